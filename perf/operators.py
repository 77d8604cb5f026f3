"""Measured cases of the cache-filling operators: block tables and slot maps,
rotary positions with the append to the paged cache, and attention of a chunk
of new tokens over that cache.

`own` chooses the side: False computes the plain forms (elementary torch
operations, 32 bits or more, rounded once), True makes the framework's calls.
Head shapes are those of the framework's workloads: 32 / 8 heads of 128, 40 / 8
heads of 128 and 8 / 2 heads of 64; pages hold 16 positions.
"""
import math

import numpy as np
import torch

own = False

PAGE = 16


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # --- block tables and slot maps (whole numbers)
        # eight sequences verifying a block of 6 tokens, as in the ragged
        # batch-8 decode step: the smallest call, made before every step
        dict(name="tables_verify_b8", op="tables", batch=8, new_lo=6, new_hi=6, cached_lo=16384,
             cached_hi=65536, prompts=0, prompt_hi=0),
        # a serving step of 300 requests: mostly single tokens, some that gave
        # pages back after rejected drafts, a dozen prompts
        dict(name="tables_mixed_b300", op="tables", batch=300, new_lo=1, new_hi=6, cached_lo=1,
             cached_hi=32768, prompts=12, prompt_hi=2048),
        # admission of long prompts: 7 fresh requests, up to 16K tokens each
        dict(name="tables_prompts_b7", op="tables", batch=7, new_lo=1, new_hi=1, cached_lo=0,
             cached_hi=0, prompts=7, prompt_hi=16384),
        # --- rotary positions and the append to the cache
        # one token of one sequence at a far position: latency
        dict(name="rope_one_token", op="rope", tokens=1, heads_q=32, heads_kv=8, dim=128, rot=128,
             axes=1, pairs="half", far=131072, fused=True, theta=500000.0),
        # a prompt chunk of 8192 tokens, split out of one fused projection
        dict(name="rope_chunk_8k", op="rope", tokens=8192, heads_q=32, heads_kv=8, dim=128,
             rot=128, axes=1, pairs="half", far=32768, fused=True, theta=500000.0),
        # an odd number of image and video tokens: time, height and width axes,
        # neighbouring pairs, half of a 64-wide head rotated
        dict(name="rope_video_d64", op="rope", tokens=5003, heads_q=8, heads_kv=2, dim=64, rot=32,
             axes=3, pairs="neighbours", far=4096, fused=False, theta=10000.0),
        # --- attention of a chunk of new tokens
        # one token over 2K positions, 8 / 2 heads of 64: latency
        dict(name="chunk_one_2k_d64", op="chunk", heads_q=8, heads_kv=2, dim=64, new="1",
             cached="2047", heavy=0.008),
        # single tokens of eight ragged sequences, 16K-64K: the cache streams
        dict(name="chunk_decode_b8", op="chunk", heads_q=32, heads_kv=8, dim=128,
             new="1,1,1,1,1,1,1,1",
             cached="17032,60211,28817,49999,33333,65535,20480,41007", heavy=0.01),
        # a serving step: seven decoding sequences beside a 1000-token chunk
        dict(name="chunk_mixed_b8", op="chunk", heads_q=32, heads_kv=8, dim=128,
             new="1,1,6,1,1000,1,6,1", cached="8000,517,4095,1,6001,2222,7777,1023", heavy=0.01),
        # fresh prompts of different lengths, nothing cached
        dict(name="chunk_prompts_b6", op="chunk", heads_q=32, heads_kv=8, dim=128,
             new="4096,2777,1311,640,129,1", cached="0,0,0,0,0,0", heavy=0.01),
        # five query heads to a KV head, odd chunks over odd prefixes
        dict(name="chunk_odd_g5", op="chunk", heads_q=40, heads_kv=8, dim=128, new="333,77,6",
             cached="4668,946,12339", heavy=0.005),
        # a 2048-token chunk at the end of a 32K context: the tensor cores
        dict(name="chunk_2k_over_32k", op="chunk", heads_q=32, heads_kv=8, dim=128, new="2048",
             cached="30720", heavy=0.01),
    ]


HEADS = ((32, 8, 128), (40, 8, 128), (8, 2, 64))


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.499)))))))


def draw(rng):
    op = rng.choice(("tables", "rope", "rope", "chunk", "chunk", "chunk"))
    if op == "tables":
        b = _log_int(rng, 1, 300)
        prompts = rng.randint(0, min(b, 12))
        lo = rng.randint(1, 3)
        return dict(op=op, batch=b, new_lo=lo, new_hi=lo + rng.randint(0, 5), cached_lo=rng.randint(0, 64),
                    cached_hi=_log_int(rng, 64, 32768), prompts=prompts,
                    prompt_hi=_log_int(rng, 16, 4096) if prompts else 0)
    hq, hkv, d = rng.choice(HEADS)
    if op == "rope":
        axes = rng.choice((1, 3))
        return dict(op=op, tokens=_log_int(rng, 1, 6500), heads_q=hq, heads_kv=hkv, dim=d,
                    rot=rng.choice((d, d // 2)), axes=axes,
                    pairs=rng.choice(("half", "neighbours")), far=_log_int(rng, 4096, 1000000),
                    fused=rng.random() < 0.5, theta=rng.choice((10000.0, 500000.0)))
    while True:
        b = _log_int(rng, 1, 8)
        top = _log_int(rng, 1, 2048)
        new = [top if i == 0 else rng.choice((1, 6, _log_int(rng, 1, top))) for i in range(b)]
        cached = [rng.choice((0, _log_int(rng, 1, 30000))) for _ in range(b)]
        rng.shuffle(new)
        case = dict(op=op, heads_q=hq, heads_kv=hkv, dim=d, new=",".join(map(str, new)),
                    cached=",".join(map(str, cached)), heavy=0.01)
        longest = max(c + n for c, n in zip(cached, new))
        # the padded score matrix of the plain form stays under the largest listed one's
        if b * hq * max(new) * longest <= 1.6e9 and work(case)["flops"] <= 1.0e12:
            return case


# ------------------------------------------------------------------ the inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _ints(text):
    return [int(x) for x in text.split(",")]


def _table_lengths(case, seed):
    """Host lengths of a table case: (cached, new, owned pages) per request."""
    r = np.random.RandomState(seed % (2 ** 31))
    b = case["batch"]
    cached = r.randint(case["cached_lo"], case["cached_hi"] + 1, b)
    new = r.randint(case["new_lo"], case["new_hi"] + 1, b)
    who = r.permutation(b)[:case["prompts"]]
    cached[who] = 0
    if case["prompts"]:
        new[who] = r.randint(max(1, case["prompt_hi"] // 4), case["prompt_hi"] + 1, case["prompts"])
    owned = (cached + PAGE - 1) // PAGE
    # one request in ten still holds a page of rejected drafts
    owned = owned + (r.rand(b) < 0.1)
    return cached, new, owned, r


def _table_sizes(case):
    """Table width, pages of the pool and rows of the padded token buffer, all
    with room for the longest lengths of the case."""
    pages = lambda n: (n + PAGE - 1) // PAGE  # noqa: E731
    few = case["batch"] - case["prompts"]
    width = max(pages(case["cached_hi"] + case["new_hi"]), pages(case["prompt_hi"])) + 2
    pool = case["batch"] * (pages(case["cached_hi"]) + 2) + few + case["prompts"] * pages(case["prompt_hi"]) + 64
    return width, pool, few * case["new_hi"] + case["prompts"] * case["prompt_hi"] + 5


def prepare(case, seed):
    op = case["op"]
    s = dict(op=op, case=case)
    if op == "tables":
        cached, new, owned, r = _table_lengths(case, seed)
        b = case["batch"]
        width, pool, room = _table_sizes(case)
        ids = r.permutation(pool).astype(np.int32)
        table = np.full((b, width), -1, np.int32)
        inside = np.arange(width)[None, :] < owned[:, None]
        used = int(owned.sum())
        table[inside] = ids[:used]
        free = np.full(pool, -1, np.int32)
        free[:pool - used] = ids[used:]
        dev = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()  # noqa: E731
        s.update(pool=pool, page_table=dev(table), owned=dev(owned), cached=dev(cached), new=dev(new),
                 free_pages=dev(free), free_count=dev([pool - used]),
                 cu_tokens=torch.zeros(b + 1, dtype=torch.int32, device="cuda"),
                 kv_lens=torch.zeros(b, dtype=torch.int32, device="cuda"),
                 positions=torch.zeros(room, dtype=torch.int32, device="cuda"),
                 slots=torch.zeros(room, dtype=torch.int32, device="cuda"))
        return s
    g = _gen(seed)
    hq, hkv, d = case["heads_q"], case["heads_kv"], case["dim"]
    rand = lambda *n: torch.randn(*n, generator=g, device="cuda")  # noqa: E731
    if op == "rope":
        t = case["tokens"]
        if case["fused"]:
            qkv = rand(t, (hq + 2 * hkv) * d).bfloat16()
            q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([hq * d, hkv * d, hkv * d], 1))
        else:
            q, k, v = rand(t, hq, d).bfloat16(), rand(t, hkv, d).bfloat16(), rand(t, hkv, d).bfloat16()
        pages = (t + PAGE - 1) // PAGE + 3
        slots = torch.randperm(pages * PAGE, generator=g, device="cuda")[:t].int()
        if t > 8:
            slots[t // 2] = -1                   # a padded token
        positions = torch.randint(0, case["far"], (case["axes"], t), generator=g, device="cuda",
                                  dtype=torch.int32)
        half = case["rot"] // 2
        inv_freq = (case["theta"] ** (-torch.arange(half, dtype=torch.float64) * 2 / case["rot"])).float().cuda()
        axis = (torch.arange(half, device="cuda") * case["axes"] // half).int()
        s.update(q=q, k=k, v=v, slots=slots, positions=positions, inv_freq=inv_freq, axis=axis,
                 k_pages=rand(pages, hkv, PAGE, d).bfloat16(), v_pages=rand(pages, hkv, PAGE, d).bfloat16(),
                 page_table=torch.arange(pages, dtype=torch.int32, device="cuda")[None],
                 q_out=torch.zeros(t, hq, d, dtype=torch.bfloat16, device="cuda"))
        return s
    new, cached = _ints(case["new"]), _ints(case["cached"])
    lens = [c + n for c, n in zip(cached, new)]
    b, t = len(new), sum(new)
    counts = [(n + PAGE - 1) // PAGE for n in lens]
    pages = sum(counts) + 5
    table = torch.full((b, max(counts)), -1, dtype=torch.int32)
    order = torch.from_numpy(np.random.RandomState(seed % (2 ** 31)).permutation(pages).astype(np.int32))
    at = 0
    for i, n in enumerate(counts):
        table[i, :n] = order[at:at + n]
        at += n
    q = rand(t, hq, d).bfloat16()
    k_pages = rand(pages, hkv, PAGE, d)
    # some keys lean towards the mean query of their group, as the ones do that attention looks for
    mean = q.float().mean(0).view(hkv, hq // hkv, d).sum(1)
    lean = (torch.rand(pages, hkv, PAGE, 1, generator=g, device="cuda") < case["heavy"]).float()
    k_pages += lean * (3.0 * math.sqrt(d)) * (mean / mean.norm(dim=-1, keepdim=True))[None, :, None, :]
    s.update(q=q, k_pages=k_pages.bfloat16(), v_pages=rand(pages, hkv, PAGE, d).bfloat16(),
             page_table=table.cuda(), kv_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
             cu=torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device="cuda"),
             max_new=max(new), scale=1.0 / math.sqrt(d), out=torch.zeros_like(q))
    return s


# ------------------------------------------------------------------- one pass
def _kept(s, make):
    """The handle that a program keeps beside its buffers."""
    if "handle" not in s:
        s["handle"] = make()
    return s["handle"]


def run(s):
    if s["op"] == "tables":
        return _tables_own(s) if own else _tables_plain(s)
    if s["op"] == "rope":
        return _rope_own(s) if own else _rope_plain(s)
    return _chunk_own(s) if own else _chunk_plain(s)


def _tables_out(s):
    return {k: s[k] for k in ("page_table", "owned", "free_pages", "free_count", "cu_tokens", "kv_lens",
                              "positions", "slots")}


def _tables_own(s):
    from self_speculative_sparse_vg_gb300 import vg
    vg.step_tables(s["page_table"], s["pool"], s["cached"], s["new"], s["cu_tokens"], s["kv_lens"],
                   s["positions"], s["slots"], owned=s["owned"], free_pages=s["free_pages"],
                   free_count=s["free_count"])
    return _tables_out(s)


def _tables_plain(s):
    """Each request's block table is resized to ceil((cached + new) / 16)
    pages: pages past that go back on the free list (requests in order, pages
    in order), then the missing ones are taken from its end.  A request whose
    pages the list no longer covers gets none and no tokens."""
    table, owned, pool = s["page_table"], s["owned"].long(), s["pool"]
    cached, new = s["cached"].long(), s["new"].long()
    room, width = s["positions"].numel(), table.shape[1]
    ends = new.cumsum(0)
    need = (cached + new + PAGE - 1) // PAGE
    fits = (ends <= room) & (need <= width)
    grow = torch.where(fits, (need - owned).clamp(min=0), 0)
    back = torch.where(fits, (owned - need).clamp(min=0), 0)
    n = s["free_count"].long()
    top = n + back.sum()
    col = torch.arange(width, device=table.device)[None, :]
    # pages that go back (the free list has one place more, for what goes nowhere)
    gives = (col >= need[:, None]) & (col < owned[:, None]) & fits[:, None]
    at = n + (back.cumsum(0) - back)[:, None] + (col - need[:, None])
    free = torch.cat((s["free_pages"], table.new_zeros(1)))
    free.scatter_(0, torch.where(gives, at, free.numel() - 1).flatten(), table.flatten())
    s["free_pages"].copy_(free[:-1])
    # pages that are taken
    want = grow.cumsum(0)
    good = fits & ((grow == 0) | (want <= top))
    takes = (col >= owned[:, None]) & (col < need[:, None]) & good[:, None]
    which = top - 1 - ((want - grow)[:, None] + (col - owned[:, None]))
    taken = free[torch.where(takes, which, 0)]
    table.copy_(torch.where(takes, taken, torch.where(gives, -1, table)))
    s["free_count"].copy_(top - torch.where(good, grow, 0).sum())
    s["owned"].copy_(torch.where(good, need, owned))
    s["cu_tokens"][1:] = ends.clamp(max=room)
    s["kv_lens"].copy_(torch.where(good, cached + new, 0))
    row = torch.arange(room, device=table.device)
    who = torch.searchsorted(ends, row, right=True)
    live = who < new.numel()
    who = who.clamp(max=new.numel() - 1)
    live = live & good[who]
    pos = cached[who] + row - (ends - new)[who]
    page = table[who, (pos // PAGE).clamp(0, width - 1)].long()
    s["positions"].copy_(torch.where(live, pos, 0))
    s["slots"].copy_(torch.where(live & (page >= 0) & (page < pool), page * PAGE + pos % PAGE, -1))
    return _tables_out(s)


def _rope_own(s):
    from self_speculative_sparse_vg_gb300 import vg
    kv = _kept(s, lambda: vg.PagedKV(s["k_pages"], s["v_pages"], s["page_table"]))
    vg.rope_append(kv, s["q"], s["k"], s["v"], s["slots"], s["q_out"], positions=s["positions"],
                   inv_freq=s["inv_freq"], freq_axis=s["axis"],
                   interleaved=s["case"]["pairs"] == "neighbours")
    return s["q_out"], s["k_pages"], s["v_pages"]


def _rope_plain(s):
    """x cos(a) + rotate(x) sin(a) with a = position(axis of the frequency) *
    frequency, in 64 bits up to the sine, then 32; the rest of the head passes."""
    angle = s["positions"].double()[s["axis"].long()].T * s["inv_freq"].double()      # [T][rot / 2]
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]
    rot, d = s["case"]["rot"], s["case"]["dim"]
    near = s["case"]["pairs"] == "neighbours"

    def turn(x):
        x = x.float()
        a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if near else (x[..., :rot // 2], x[..., rot // 2:rot])
        y, z = a * cos - b * sin, b * cos + a * sin
        turned = torch.stack((y, z), -1).flatten(-2) if near else torch.cat((y, z), -1)
        return torch.cat((turned, x[..., rot:d]), -1).bfloat16()

    s["q_out"].copy_(turn(s["q"]))
    live = s["slots"] >= 0
    slot = s["slots"][live].long()
    s["k_pages"][slot // PAGE, :, slot % PAGE] = turn(s["k"])[live]
    s["v_pages"][slot // PAGE, :, slot % PAGE] = s["v"][live]
    return s["q_out"], s["k_pages"], s["v_pages"]


def _chunk_own(s):
    from self_speculative_sparse_vg_gb300 import vg

    def make():
        kv = vg.PagedKV(s["k_pages"], s["v_pages"], s["page_table"])
        t, hq, d = s["q"].shape
        n = vg.chunk_workspace_bytes(s["kv_lens"].numel(), t, hq, kv.num_kv_heads, d)
        return kv, torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
    kv, ws = _kept(s, make)
    vg.chunk_attention(kv, s["q"], s["cu"], s["kv_lens"], s["scale"], s["out"], workspace=ws)
    return s["out"]


def _chunk_plain(s):
    """softmax(scale q k^T) v of each new token over the positions up to its
    own: sequences padded to the longest, the whole score matrix in 32 bits."""
    q, cu, lens = s["q"], s["cu"].long(), s["kv_lens"].long()
    hq, d = q.shape[1:]
    table = s["page_table"].long()
    b, hkv = table.shape[0], s["k_pages"].shape[1]
    n = cu[1:] - cu[:-1]
    i = torch.arange(s["max_new"], device=q.device)
    j = torch.arange(table.shape[1] * PAGE, device=q.device)
    row = (cu[:-1, None] + i).clamp(max=q.shape[0] - 1)
    dense = lambda x: x[table.clamp(min=0)].float().transpose(2, 3).flatten(1, 2)  # noqa: E731
    k = dense(s["k_pages"]).permute(0, 2, 3, 1)                                    # [B][Hkv][d][J]
    v = dense(s["v_pages"]).masked_fill((j >= lens[:, None])[..., None, None], 0.0).transpose(1, 2)
    x = q[row].float().view(b, -1, hkv, hq // hkv, d).permute(0, 2, 1, 3, 4).flatten(2, 3)
    p = (x @ k).mul_(s["scale"]).view(b, hkv, i.numel(), hq // hkv, j.numel())
    seen = j <= (lens[:, None] - n[:, None] + i)[..., None]                         # [B][I][J]
    p.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    p = p.sub_(p.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    total = p.sum(-1, keepdim=True)
    y = (p.flatten(2, 3) @ v).view(b, hkv, i.numel(), hq // hkv, d) / total.clamp(min=1e-30)
    t = torch.arange(q.shape[0], device=q.device)
    who = torch.searchsorted(cu[1:], t, right=True)
    s["out"].copy_(y.permute(0, 2, 1, 3, 4)[who, t - cu[who]].flatten(1, 2))
    return s["out"]


# ------------------------------------------------------------------- the work
def work(case):
    """Bytes and operations that one pass cannot do without."""
    if case["op"] == "tables":
        # lengths and owned pages in, row offsets, lengths and owned pages out, a position and
        # a slot for each token, a table entry read for each page that new tokens touch and one
        # written for each new page
        b, room = case["batch"], _table_sizes(case)[2]
        return {"bytes": 4.0 * (6 * b + 2 * room + (b + room / PAGE) * 2), "flops": 0.0}
    hq, hkv, d = case["heads_q"], case["heads_kv"], case["dim"]
    if case["op"] == "rope":
        t = case["tokens"]
        return {"bytes": t * (2.0 * (hq + 2 * hkv) * d * 2 + 4 * case["axes"] + 4) + case["rot"] * 4,
                "flops": t * 3.0 * (hq + hkv) * case["rot"]}
    new, cached = _ints(case["new"]), _ints(case["cached"])
    pairs = sum(n * c + n * (n + 1) // 2 for n, c in zip(new, cached))
    kv = sum(n + c for n, c in zip(new, cached))
    return {"bytes": 2.0 * sum(new) * hq * d * 2 + 2.0 * kv * hkv * d * 2 + kv / PAGE * 4,
            "flops": 4.0 * pairs * hq * d}


# ------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"tables": _tables_exact, "rope": _rope_exact, "chunk": _chunk_exact}[case["op"]](s)


def _tables_exact(s):
    table, free = s["page_table"].cpu().numpy().astype(np.int64), s["free_pages"].cpu().numpy().astype(np.int64)
    owned, n = s["owned"].cpu().numpy().astype(np.int64), int(s["free_count"].item())
    cached, new = s["cached"].cpu().tolist(), s["new"].cpu().tolist()
    room, width = s["positions"].numel(), table.shape[1]
    b = len(new)
    cu = [0]
    for x in new:
        cu.append(cu[-1] + x)
    need = [-(-(c + x) // PAGE) for c, x in zip(cached, new)]
    fits = [cu[i + 1] <= room and need[i] <= width for i in range(b)]
    for i in range(b):
        for p in range(need[i], int(owned[i])) if fits[i] else ():
            free[n] = table[i, p]
            table[i, p] = -1
            n += 1
    asked, top, lens = 0, n, [0] * b
    positions, slots = np.zeros(room, np.int64), np.full(room, -1, np.int64)
    for i in range(b):
        if not fits[i]:
            continue
        more = max(0, need[i] - int(owned[i]))
        asked += more
        if more and asked > top:
            continue
        for p in range(int(owned[i]), need[i]):
            n -= 1
            table[i, p] = free[n]
        owned[i], lens[i] = need[i], cached[i] + new[i]
        for x in range(new[i]):
            pos = cached[i] + x
            positions[cu[i] + x] = pos
            slots[cu[i] + x] = table[i, pos // PAGE] * PAGE + pos % PAGE
    t = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32)  # noqa: E731
    return dict(page_table=t(table), owned=t(owned), free_pages=t(free), free_count=t([n]),
                cu_tokens=t([min(x, room) for x in cu]), kv_lens=t(lens), positions=t(positions), slots=t(slots))


def _rope_exact(s):
    case = s["case"]
    rot, near = case["rot"], case["pairs"] == "neighbours"
    pos = s["positions"].double()
    freq, axis = s["inv_freq"].double(), s["axis"].tolist()

    def turned(x):
        y = x.double().clone()
        for i in range(rot // 2):
            a = (pos[axis[i]] * freq[i])[:, None]
            u, w = (2 * i, 2 * i + 1) if near else (i, i + rot // 2)
            z = torch.complex(x[..., u].double(), x[..., w].double()) * torch.polar(torch.ones_like(a), a)
            y[..., u], y[..., w] = z.real, z.imag
        return y

    kp, vp, kt = s["k_pages"].double(), s["v_pages"].double(), turned(s["k"])
    flat = lambda x: x.transpose(1, 2).reshape(-1, case["heads_kv"], case["dim"])  # noqa: E731
    kf, vf = flat(kp), flat(vp)
    live = (s["slots"] >= 0).nonzero()[:, 0]
    kf[s["slots"][live].long()] = kt[live]
    vf[s["slots"][live].long()] = s["v"][live].double()
    back = lambda x, like: x.view(like.shape[0], PAGE, case["heads_kv"], case["dim"]).transpose(1, 2).contiguous()  # noqa: E731
    return turned(s["q"]), back(kf, kp), back(vf, vp)


def _chunk_exact(s):
    q = s["q"]
    hq, d = q.shape[1:]
    hkv = s["k_pages"].shape[1]
    g = hq // hkv
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    cu, lens = s["cu"].tolist(), s["kv_lens"].tolist()
    for b, n in enumerate(lens):
        pages = s["page_table"][b, :(n + PAGE - 1) // PAGE].long()
        for h in range(hkv):
            k = s["k_pages"][pages, h].reshape(-1, d)[:n].double()
            v = s["v_pages"][pages, h].reshape(-1, d)[:n].double()
            first = n - (cu[b + 1] - cu[b])
            for r0 in range(cu[b], cu[b + 1], 512):
                r1 = min(r0 + 512, cu[b + 1])
                e = first + r1 - cu[b]                       # positions that the last of these rows sees
                x = torch.einsum("thd,jd->thj", q[r0:r1, h * g:(h + 1) * g].double(), k[:e]) * s["scale"]
                last = first + torch.arange(r0, r1, device=q.device) - cu[b]
                x = torch.where(torch.arange(e, device=q.device) <= last[:, None, None], x, -math.inf)
                w = torch.softmax(x, -1)
                out[r0:r1, h * g:(h + 1) * g] = torch.einsum("thj,jd->thd", w, v[:e])
    return out

"""Measured cases of decoding with beams: the selection over beams and
vocabulary, the reordering of the beams' block tables, the copies of their last
pages, and cross attention to an encoder's states of another length.

`own` chooses the side: False computes the plain forms (elementary torch
operations, 32 bits or more, rounded once), True makes the framework's calls.
Head shapes are those of the framework's workloads (32 / 8 and 40 / 8 heads of
128, 8 / 2 heads of 64) and, for cross attention, 16 / 16 heads of 64; pages
hold 16 positions.
"""
import math

import numpy as np
import torch

own = False

PAGE = 16
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # --- selection over beams and vocabulary
        # one request of four beams over a small vocabulary: latency
        dict(name="select_one_32k", op="select", batch=1, beams=4, out=4, vocab=32000, type="bf16", ended=0.0,
             fresh=0.0, banned=0.0),
        # a batch of five beams over an odd vocabulary (rows that start on no
        # vector's boundary); some beams have ended, some requests are at their
        # first step, where one beam lives; a tenth of the tokens is banned
        dict(name="select_odd_50k", op="select", batch=16, beams=5, out=10, vocab=50257, type="fp16", ended=0.2,
             fresh=0.2, banned=0.1),
        # logits kept in 32 bits
        dict(name="select_fp32_151k", op="select", batch=8, beams=4, out=8, vocab=151936, type="fp32", ended=0.05,
             fresh=0.0, banned=0.0),
        # a full batch: 512 rows of a large vocabulary
        dict(name="select_b64_128k", op="select", batch=64, beams=8, out=16, vocab=128256, type="bf16", ended=0.05,
             fresh=0.05, banned=0.0),
        # --- reordering of block tables (whole numbers)
        # one request of four beams: latency
        dict(name="tables_one", op="tables", batch=1, beams=4, lo=2000, hi=2100, apart=64, fresh=0.0, finished=0.0),
        # a batch of eight beams each over 1K - 32K positions: requests that
        # have just been admitted (one row is copied to all), others that end
        dict(name="tables_b32", op="tables", batch=32, beams=8, lo=1000, hi=32768, apart=400, fresh=0.1, finished=0.1),
        # --- copies of last pages
        # one layer's copies of 32 rows
        dict(name="copy_layer", op="copy", layers=1, rows=32, heads_kv=8, dim=128, share=0.7),
        # a whole model's: 32 layers in one call
        dict(name="copy_32_layers", op="copy", layers=32, rows=128, heads_kv=8, dim=128, share=0.6),
        # --- cross attention
        # one token to 1500 states, 16 heads of 64: latency
        dict(name="cross_one_1500", op="cross", heads_q=16, heads_kv=16, dim=64, type="bf16", new="1", states="1500",
             masked=0.0, fused=False, room=0),
        # five beams of 24 requests, states of 200 - 1500, keys and values
        # split out of one projection: they stream
        dict(name="cross_beams_b24", op="cross", heads_q=16, heads_kv=16, dim=64, type="fp16",
             new="5," * 23 + "5",
             states="1500,1322,207,911,1500,640,333,1500,1024,877,1500,1201,450,1499,1500,729,1500,1111,200,1500,"
                    "983,1500,601,1417", masked=0.0, fused=True, room=0),
        # blocks of six verify rows over image states that lie in slots of
        # 6404, a tenth of them masked, one request without any
        dict(name="cross_verify_b8", op="cross", heads_q=32, heads_kv=8, dim=128, type="bf16", new="6,6,6,6,6,6,6,6",
             states="6404,1601,3203,0,6404,577,4804,6404", masked=0.1, fused=False, room=6404),
        # prompts of different lengths over the states of their encoders: the
        # tensor cores
        dict(name="cross_prompts_b5", op="cross", heads_q=32, heads_kv=8, dim=128, type="bf16",
             new="2048,777,1311,1,640", states="6404,1601,4804,3203,129", masked=0.0, fused=False, room=0),
    ]


HEADS = ((32, 8, 128), (40, 8, 128), (8, 2, 64), (16, 16, 64))


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.499)))))))


def draw(rng):
    op = rng.choice(("select", "select", "select", "tables", "copy", "cross", "cross", "cross"))
    if op == "select":
        while True:
            beams = _log_int(rng, 1, 16)
            case = dict(op=op, batch=_log_int(rng, 1, 64), beams=beams, out=rng.choice((beams, 2 * beams)),
                        vocab=_log_int(rng, 900, 200000), type=rng.choice(("bf16", "fp16", "fp32")),
                        ended=rng.choice((0.0, 0.2)), fresh=rng.choice((0.0, 0.3)), banned=rng.choice((0.0, 0.5)))
            if work(case)["bytes"] <= 130e6:
                return case
    if op == "tables":
        hi = _log_int(rng, 40, 32768)
        return dict(op=op, batch=_log_int(rng, 1, 32), beams=rng.randint(1, 8), lo=rng.randint(1, min(hi, 1000)),
                    hi=hi, apart=_log_int(rng, 1, 400), fresh=rng.choice((0.0, 0.2)), finished=rng.choice((0.0, 0.2)))
    hq, hkv, d = rng.choice(HEADS)
    if op == "copy":
        return dict(op=op, layers=_log_int(rng, 1, 32), rows=_log_int(rng, 1, 128), heads_kv=min(hkv, 8), dim=d,
                    share=rng.choice((0.3, 0.6)))
    while True:
        b = _log_int(rng, 1, 24)
        top = rng.choice((1, 6, _log_int(rng, 1, 2048)))
        new = [top if i == 0 else rng.choice((1, 5, _log_int(rng, 1, top))) for i in range(b)]
        states = [_log_int(rng, 1, 6404) for _ in range(b)]
        rng.shuffle(new)
        case = dict(op=op, heads_q=hq, heads_kv=hkv, dim=d, type=rng.choice(("bf16", "fp16")),
                    new=",".join(map(str, new)), states=",".join(map(str, states)), masked=rng.choice((0.0, 0.3)),
                    fused=rng.random() < 0.5, room=rng.choice((0, 6404)))
        if work(case)["flops"] <= 2.2e11 and work(case)["bytes"] <= 1.2e8:
            return case


# ------------------------------------------------------------------ the inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _ints(text):
    return [int(x) for x in text.split(",")]


def _dev(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def prepare(case, seed):
    s = dict(op=case["op"], case=case)
    s.update({"select": _select_inputs, "tables": _tables_inputs, "copy": _copy_inputs,
              "cross": _cross_inputs}[case["op"]](case, seed))
    return s


def _select_inputs(case, seed):
    g = _gen(seed)
    b, w, v, k = case["batch"], case["beams"], case["vocab"], case["out"]
    x = torch.randn(b * w, v, generator=g, device="cuda") * 2.5
    # a few tokens stand out, as in a trained model's logits
    at = torch.randint(0, v, (b * w, 24), generator=g, device="cuda")
    x.scatter_add_(1, at, 8.0 * torch.rand(b * w, 24, generator=g, device="cuda") + 4.0)
    x = x.to(TYPES[case["type"]])
    if case["banned"]:
        x.masked_fill_(torch.rand(1, v, generator=g, device="cuda") < case["banned"], -math.inf)
    score = -(torch.rand(b, w, generator=g, device="cuda") * 2.0).cumsum(1) - 5.0
    fresh = torch.rand(b, 1, generator=g, device="cuda") < case["fresh"]
    score = torch.where(fresh & (torch.arange(w, device="cuda") > 0), -math.inf, score)
    ended = (torch.rand(b, w, generator=g, device="cuda") < case["ended"]) & ~fresh
    new = lambda t: torch.zeros(b, k, dtype=t, device="cuda")  # noqa: E731
    return dict(logits=x, score=score, ended=ended, end=2, out_score=new(torch.float32), out_token=new(torch.int32),
                out_parent=new(torch.int32), out_ended=new(torch.bool))


def _tables_inputs(case, seed):
    """Requests of `beams` rows: their pages are one row's up to a point, then
    they part, here and there again in two; the last page of a row is its own."""
    r = np.random.RandomState(seed % (2 ** 31))
    b, w = case["batch"], case["beams"]
    width = case["hi"] // PAGE + 3
    pool = b * (width + w * (case["apart"] // PAGE + 3)) + 64
    ids = r.permutation(pool)
    at = 0
    table = np.full((b * w, width), -1, np.int32)
    owned, lens = np.zeros(b * w, np.int32), np.zeros(b * w, np.int32)
    parents = np.full((b, w), -1, np.int32)
    for i in range(b):
        n = r.randint(case["lo"], case["hi"] + 1)
        cols, tail = -(-n // PAGE), n % PAGE
        kind = r.rand()
        rows = 1 if kind < case["fresh"] else w          # just admitted: one row holds the prompt
        shared = max(0, (n - r.randint(1, case["apart"] + 1)) // PAGE)
        for j in range(rows):
            row = table[i * w + j]
            if j == 0:
                row[:cols], at = ids[at:at + cols], at + cols
            else:
                mate = table[i * w + r.randint(0, j)]
                part = r.randint(shared, cols + 1)
                part = min(part, cols - 1 if tail else cols)
                row[:part] = mate[:part]
                row[part:cols], at = ids[at:at + cols - part], at + cols - part
            owned[i * w + j], lens[i * w + j] = cols, n
        if kind < case["fresh"]:
            parents[i] = 0
        elif kind < case["fresh"] + case["finished"]:
            parents[i] = -1
        else:
            parents[i] = np.minimum(r.geometric(0.45, w) - 1, w - 1)   # the better ones have more children
    free = np.full(pool, -1, np.int32)
    free[:pool - at] = ids[at:]
    return dict(pool=pool, table=_dev(table), owned=_dev(owned), lens=_dev(lens), parents=_dev(parents),
                free=_dev(free), count=_dev([pool - at]), copies=torch.zeros(b * w, 3, dtype=torch.int32, device="cuda"))


def _copy_inputs(case, seed):
    g = _gen(seed)
    r = np.random.RandomState(seed % (2 ** 31))
    n, pages = case["rows"], 2 * case["rows"] + 5
    ids = r.permutation(pages)
    copies = np.stack([ids[:n], ids[n:2 * n], r.randint(1, PAGE, n)], 1)
    copies[r.rand(n) >= case["share"]] = (-1, -1, 0)     # rows that keep their page
    pool = lambda: torch.randn(pages, case["heads_kv"], PAGE, case["dim"], generator=g, device="cuda").bfloat16()  # noqa: E731
    return dict(pools=[(pool(), pool()) for _ in range(case["layers"])], copies=_dev(copies),
                table=torch.zeros(1, 1, dtype=torch.int32, device="cuda"))


def _cross_inputs(case, seed):
    g = _gen(seed)
    hq, hkv, d, t = case["heads_q"], case["heads_kv"], case["dim"], TYPES[case["type"]]
    new, lens = _ints(case["new"]), _ints(case["states"])
    if case["room"]:                                     # slots of one size, states at their beginning
        starts, total = [i * case["room"] for i in range(len(lens))], case["room"] * len(lens)
    else:
        starts = [0] + list(np.cumsum(lens)[:-1])
        total = max(1, sum(lens))
    rand = lambda *n: torch.randn(*n, generator=g, device="cuda", dtype=torch.float32)  # noqa: E731
    q = rand(sum(new), hq, d).to(t)
    kv = rand(total, 2, hkv, d)
    # some states draw the attention of most queries of a group
    mean = q.float().mean(0).view(hkv, hq // hkv, d).sum(1)
    lean = (torch.rand(total, hkv, 1, generator=g, device="cuda") < 0.01).float()
    kv[:, 0] += lean * (3.0 * math.sqrt(d)) * (mean / mean.norm(dim=-1, keepdim=True))
    kv = kv.to(t)
    k, v = kv[:, 0], kv[:, 1]
    if not case["fused"]:
        k, v = k.contiguous(), v.contiguous()
    mask = None
    if case["masked"]:
        mask = torch.rand(total, generator=g, device="cuda") >= case["masked"]
    return dict(q=q, k=k, v=v, mask=mask, cu=_dev([0] + list(np.cumsum(new))), starts=_dev(starts), lens=_dev(lens),
                new=new, host=(starts, lens), scale=1.0 / math.sqrt(d), out=torch.zeros_like(q))


# ------------------------------------------------------------------- one pass
def _kept(s, make):
    """The handle that a program keeps beside its buffers."""
    if "handle" not in s:
        s["handle"] = make()
    return s["handle"]


def run(s):
    return _RUN[s["op"], own](s)


def _select_own(s):
    from self_speculative_sparse_vg_gb300 import vg
    x, (b, k) = s["logits"], s["out_score"].shape

    def make():
        n = vg.beam_select_workspace_bytes(b, s["case"]["beams"], x.shape[1], x.dtype, k)
        return torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
    vg.beam_select(x, s["score"], s["out_score"], s["out_token"], s["out_parent"], ended=s["ended"],
                   end_token=s["end"], out_ended=s["out_ended"], workspace=_kept(s, make))
    return s["out_score"], s["out_token"], s["out_parent"], s["out_ended"]


def _select_plain(s):
    """score + x - log sum exp x of every live beam's tokens, an ended beam's
    score with the end token, in 64 bits (candidates next to each other decide);
    the best of a request, ties to the lowest beam, then token."""
    b, w = s["score"].shape
    k, v = s["out_score"].shape[1], s["logits"].shape[1]
    x = s["logits"].double().view(b, w, v)
    top = x.amax(-1, keepdim=True).clamp(min=-1e300)
    y = s["score"].double()[..., None] + (x - top - (x - top).exp().sum(-1, keepdim=True).clamp(min=1e-300).log())
    y = torch.where(torch.isneginf(s["score"])[..., None], -math.inf, y)
    token = torch.arange(v, device=y.device)
    held = torch.where(token == s["end"], s["score"].double()[..., None], -math.inf)
    y = torch.where(s["ended"][..., None], held, y)
    y, at = y.view(b, w * v).sort(dim=1, descending=True, stable=True)
    y, at = y[:, :k], at[:, :k]
    none = torch.isneginf(y)
    parent, token = at // v, at % v
    s["out_score"].copy_(y)
    s["out_token"].copy_(torch.where(none, -1, token))
    s["out_parent"].copy_(torch.where(none, -1, parent))
    s["out_ended"].copy_(~none & (s["ended"].gather(1, parent) | (token == s["end"])))
    return s["out_score"], s["out_token"], s["out_parent"], s["out_ended"]


def _tables_out(s):
    return {k: s[k] for k in ("table", "owned", "lens", "free", "count", "copies")}


def _tables_own(s):
    from self_speculative_sparse_vg_gb300 import vg
    vg.beam_tables(s["table"], s["pool"], s["parents"], s["lens"], s["owned"], s["free"], s["count"], s["copies"])
    return _tables_out(s)


def _tables_plain(s):
    """Row j of a request takes row parents[j]'s pages and length.  Pages that
    no row holds any more go on the free list (requests, then columns, then rows
    in order).  A partly filled last page stays with the first row that takes
    it; each other one takes a page from the list's end and a copy of it."""
    table, parents = s["table"], s["parents"].long()
    b, w = parents.shape
    dev, width = table.device, table.shape[1]
    old = table.view(b, w, width).long()
    own, lens = s["owned"].view(b, w).long(), s["lens"].view(b, w).long()
    col = torch.arange(width, device=dev)
    who = torch.arange(w, device=dev)
    need = (lens + PAGE - 1) // PAGE
    held = col < own[..., None]
    alive = (parents[:, None, :] == who[None, :, None]).any(2)
    kept = alive[..., None] & (col < need[..., None])
    goes = held & ~kept
    for i in range(w):
        for j in range(w):
            if i == j:
                continue
            same = held[:, j] & (old[:, i] == old[:, j])
            goes[:, i] &= ~(same & (kept[:, j] | (j < i)))
    # the free list has one place more, for what goes nowhere
    flat = goes.transpose(1, 2).flatten()
    n = s["count"].long()
    back = flat.long().cumsum(0)
    top = n + back[-1]
    free = torch.cat((s["free"].long(), table.new_zeros(1).long()))
    free.scatter_(0, torch.where(flat, n + back - 1, free.numel() - 1), old.transpose(1, 2).flatten())
    s["free"].copy_(free[:-1])
    # the rows
    p = parents.clamp(min=0)
    live = parents >= 0
    size = torch.where(live, lens.gather(1, p), 0)
    full, tail = size // PAGE, size % PAGE
    rows = old.gather(1, p[..., None].expand(-1, -1, width))
    last = rows.gather(2, full.clamp(max=width - 1)[..., None])[..., 0]
    earlier = (who[:, None] > who[None, :]) & (last[:, :, None] == last[:, None, :]) & (tail > 0)[:, None, :]
    asks = (tail > 0) & earlier.any(2)
    rank = asks.flatten().long().cumsum(0).view(b, w) - 1
    fits = ~asks | (rank < top)
    page = free[torch.where(asks & fits, top - 1 - rank, 0)]
    mine = torch.where(asks, page, last)
    rows = torch.where(col == full[..., None], mine[..., None], rows)
    rows = torch.where((col < ((size + PAGE - 1) // PAGE)[..., None]) & fits[..., None], rows, -1)
    table.copy_(rows.view(b * w, width))
    s["copies"].copy_(torch.where((asks & fits)[..., None], torch.stack((last, page, tail), -1),
                                  torch.tensor([-1, -1, 0], device=dev)).view(b * w, 3))
    size = torch.where(fits, size, 0)
    s["lens"].copy_(size.flatten())
    s["owned"].copy_(((size + PAGE - 1) // PAGE).flatten())
    s["count"].copy_(top - torch.minimum(asks.sum(), top))
    return _tables_out(s)


def _copy_own(s):
    from self_speculative_sparse_vg_gb300 import vg
    kv = _kept(s, lambda: [vg.PagedKV(k, v, s["table"]) for k, v in s["pools"]])
    vg.copy_pages(kv, s["copies"])
    return s["pools"]


def _copy_plain(s):
    """The first `positions` positions of page `from`, in page `to`."""
    src, dst, n = s["copies"].long().unbind(1)
    row = (torch.arange(PAGE, device=src.device) < n[:, None]).nonzero()
    i, at = row[:, 0], row[:, 1]
    for k, v in s["pools"]:
        k[dst[i], :, at] = k[src[i], :, at]
        v[dst[i], :, at] = v[src[i], :, at]
    return s["pools"]


def _cross_own(s):
    from self_speculative_sparse_vg_gb300 import vg

    def make():
        t, hq, d = s["q"].shape
        n = vg.cross_workspace_bytes(s["lens"].numel(), t, hq, s["k"].shape[1], d)
        return torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
    vg.cross_attention(s["q"], s["k"], s["v"], s["cu"], s["starts"], s["lens"], s["scale"], s["out"], mask=s["mask"],
                       workspace=_kept(s, make))
    return s["out"]


def _cross_plain(s):
    """softmax(scale q k^T) v of each row over its sequence's states, 32 bits;
    a row without states is zero."""
    starts, lens = s["host"]
    hq, d = s["q"].shape[1:]
    hkv = s["k"].shape[1]
    at = 0
    for a, n, m in zip(starts, lens, s["new"]):
        if n == 0:
            s["out"][at:at + m] = 0
        elif m:
            k, v = s["k"][a:a + n].float(), s["v"][a:a + n].float()
            q = s["q"][at:at + m].float().view(m, hkv, hq // hkv, d).permute(1, 2, 0, 3).reshape(hkv, -1, d)
            p = (q @ k.permute(1, 2, 0)).mul_(s["scale"])
            if s["mask"] is not None:
                p.masked_fill_(~s["mask"][a:a + n], -math.inf)
            p = p.sub_(p.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
            y = (p @ v.transpose(0, 1)) / p.sum(-1, keepdim=True).clamp(min=1e-30)
            s["out"][at:at + m] = y.view(hkv, hq // hkv, m, d).permute(2, 0, 1, 3).reshape(m, hq, d)
        at += m
    return s["out"]


_RUN = {("select", False): _select_plain, ("select", True): _select_own, ("tables", False): _tables_plain,
        ("tables", True): _tables_own, ("copy", False): _copy_plain, ("copy", True): _copy_own,
        ("cross", False): _cross_plain, ("cross", True): _cross_own}


# ------------------------------------------------------------------- the work
def work(case):
    """Bytes and operations that one pass cannot do without."""
    if case["op"] == "select":
        # the logits of live beams; scores and marks in; four numbers out for each place
        rows = case["batch"] * ((1 - case["fresh"]) * case["beams"] * (1 - case["ended"]) + case["fresh"])
        size = 4 if case["type"] == "fp32" else 2
        return {"bytes": rows * case["vocab"] * size + case["batch"] * (5.0 * case["beams"] + 13.0 * case["out"]),
                "flops": 3.0 * rows * case["vocab"]}
    if case["op"] == "tables":
        # entries of the rows that are held, those that part written anew, five numbers a row
        rows, mean = case["batch"] * case["beams"], (case["lo"] + case["hi"]) / 2
        return {"bytes": rows * 4.0 * (mean / PAGE + min(mean, case["apart"] / 2) / PAGE + 9), "flops": 0.0}
    if case["op"] == "copy":
        each = case["heads_kv"] * case["dim"] * 2 * 8.0          # one position of K, or of V; half a page of them
        return {"bytes": case["layers"] * case["rows"] * case["share"] * each * 2 * 2 + case["rows"] * 12.0, "flops": 0.0}
    hq, hkv, d = case["heads_q"], case["heads_kv"], case["dim"]
    new, states = _ints(case["new"]), _ints(case["states"])
    seen = 1 - case["masked"]
    return {"bytes": 2.0 * sum(new) * hq * d * 2 + 2.0 * sum(n for n, m in zip(states, new) if m) * hkv * d * 2
            + (sum(states) if case["masked"] else 0),
            "flops": 4.0 * seen * sum(m * n for m, n in zip(new, states)) * hq * d}


# ------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"select": _select_exact, "tables": _tables_exact, "copy": _copy_exact, "cross": _cross_exact}[case["op"]](s)


def _select_exact(s):
    b, w = s["score"].shape
    k = s["out_score"].shape[1]
    v = s["logits"].shape[1]
    score = torch.full((b, k), -math.inf, dtype=torch.float64)
    token = torch.full((b, k), -1, dtype=torch.int32)
    parent, ended = token.clone(), torch.zeros(b, k, dtype=torch.bool)
    for i in range(b):
        found = []
        for j in range(w):
            own_score = float(s["score"][i, j])
            if own_score == -math.inf:
                continue
            if bool(s["ended"][i, j]):
                found.append((-own_score, j, s["end"], True))
                continue
            y = torch.log_softmax(s["logits"][i * w + j].double(), 0) + own_score
            least = y.topk(min(k, v)).values[-1]
            at = ((y >= least) & (y > -math.inf)).nonzero()[:, 0]
            found += [(-a, j, t, t == s["end"]) for a, t in zip(y[at].tolist(), at.tolist())]
        for n, (a, j, t, e) in enumerate(sorted(found)[:k]):
            score[i, n], token[i, n], parent[i, n], ended[i, n] = -a, t, j, e
    return score, token, parent, ended


def _tables_exact(s):
    table, owned = s["table"].cpu().numpy().astype(np.int64), s["owned"].cpu().tolist()
    lens, parents = s["lens"].cpu().tolist(), s["parents"].cpu().numpy()
    free, n = s["free"].cpu().tolist(), int(s["count"].item())
    b, w = parents.shape
    new = np.full_like(table, -1)
    new_lens = [0] * (b * w)
    for i in range(b):
        stay = set()
        for j in range(w):
            p = int(parents[i, j])
            if p >= 0:
                r = i * w + p
                new_lens[i * w + j] = lens[r]
                cols = -(-lens[r] // PAGE)
                new[i * w + j, :cols] = table[r, :cols]
                stay.update((c, int(table[r, c])) for c in range(cols))
        for c in range(max(owned[i * w:(i + 1) * w])):
            for r in range(i * w, (i + 1) * w):
                at = (c, int(table[r, c]))
                if c < owned[r] and at not in stay:
                    stay.add(at)                          # once
                    free[n] = at[1]
                    n += 1
    copies = np.tile(np.array([-1, -1, 0]), (b * w, 1))
    for i in range(b):
        taken = set()
        for r in range(i * w, (i + 1) * w):
            c, rest = divmod(new_lens[r], PAGE)
            if not rest:
                continue
            page = int(new[r, c])
            if page not in taken:
                taken.add(page)
            elif n == 0:
                new[r], new_lens[r] = -1, 0
            else:
                n -= 1
                new[r, c] = free[n]
                copies[r] = (page, free[n], rest)
    t = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32)  # noqa: E731
    return dict(table=t(new), owned=t([-(-x // PAGE) for x in new_lens]), lens=t(new_lens), free=t(free), count=t([n]),
                copies=t(copies))


def _copy_exact(s):
    out = [(k.double(), v.double()) for k, v in s["pools"]]
    for src, dst, n in s["copies"].tolist():
        for (k, v), (k0, v0) in zip(out, s["pools"]) if n else ():
            k[dst, :, :n] = k0[src, :, :n].double()
            v[dst, :, :n] = v0[src, :, :n].double()
    return out


def _cross_exact(s):
    q = s["q"]
    hq, d = q.shape[1:]
    hkv = s["k"].shape[1]
    g = hq // hkv
    starts, lens = s["host"]
    cu = s["cu"].tolist()
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    for e, n in enumerate(lens):
        pick = torch.arange(starts[e], starts[e] + n, device=q.device)
        if s["mask"] is not None:
            pick = pick[s["mask"][pick]]
        if pick.numel() == 0:
            continue
        for h in range(hkv):
            k, v = s["k"][pick, h].double(), s["v"][pick, h].double()
            for r0 in range(cu[e], cu[e + 1], 512):
                r1 = min(r0 + 512, cu[e + 1])
                x = torch.einsum("tgd,jd->tgj", q[r0:r1, h * g:(h + 1) * g].double(), k) * s["scale"]
                out[r0:r1, h * g:(h + 1) * g] = torch.einsum("tgj,jd->tgd", torch.softmax(x, -1), v)
    return out

"""Decoding with beams, all calls of a step together: block tables, rotary append,
attention over the cache and over an encoder's states, selection over beams and
vocabulary, the beams' tables and the copies of their last pages.  Every call of
every step is checked against the oracles on what the calls before it left; one
captured graph of a step is replayed and gives the same bits."""
import numpy as np
import pytest
import torch

from oracle import beam_oracle as O
from oracle import fill_oracle as F
from tests.beam_util import check_select, cross_bounds
from tests.fill_util import PAGE, chunk_bounds, i32

pytestmark = pytest.mark.gpu


class Decoder:
    """One layer of an encoder-decoder model with made-up projections: a token's
    query, key and value are rows of a table, logits a product with the outputs."""

    def __init__(self, B, W, Hq, Hkv, d, V, seed=0):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.B, self.W, self.Hq, self.Hkv, self.d, self.V = B, W, Hq, Hkv, d, V
        R = self.R = B * W
        self.pool, width = R * 14 + B * 20, 64
        self.embed = [torch.randn(V, h, d, generator=g).bfloat16().cuda() for h in (Hq, Hkv, Hkv)]
        self.project = (torch.randn(Hq * d, V, generator=g) * 0.2).cuda()
        self.freq = (1e4 ** (-torch.arange(d // 2, dtype=torch.float64) * 2 / d)).float().cuda()
        self.enc_lens = rng.integers(0, 400, B)
        self.enc_lens[0] = 300
        starts = np.concatenate([[0], np.cumsum(self.enc_lens)])
        enc = torch.randn(int(starts[-1]) + 1, 2 * Hkv, d, generator=g).bfloat16()
        self.mask = torch.rand(enc.shape[0], generator=g) < 0.9
        enc[~self.mask] = float("nan")
        self.enc, self.starts = enc, starts[:-1]
        ints = lambda *n: torch.zeros(*n, dtype=torch.int32, device="cuda")  # noqa: E731
        cache = torch.full((2, self.pool, Hkv, PAGE, d), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.dev = dict(
            table=i32(np.full((R, width), -1)), owned=ints(R), lens=ints(R), free=i32(rng.permutation(self.pool)),
            count=i32([self.pool]), cache=cache, cu=ints(R + 1), kv_lens=ints(R), positions=ints(R), slots=ints(R),
            ones=ints(R) + 1, tokens=ints(R), scores=torch.zeros(B, W, device="cuda"),
            ended=torch.zeros(B, W, dtype=torch.bool, device="cuda"), parents=ints(B, W), next=ints(B, W),
            copies=ints(R, 3), flag=ints(1), q=torch.zeros(R, Hq, d, dtype=torch.bfloat16, device="cuda"),
            self_out=torch.zeros(R, Hq, d, dtype=torch.bfloat16, device="cuda"),
            cross_out=torch.zeros(R, Hq, d, dtype=torch.bfloat16, device="cuda"),
            logits=torch.zeros(R, V, dtype=torch.bfloat16, device="cuda"))
        self.fixed = dict(enc=enc.cuda(), mask=self.mask.cuda(), starts=i32(self.starts), enc_lens=i32(self.enc_lens),
                          cu_req=i32(np.arange(B + 1) * W))

    def kv(self, s):
        from self_speculative_sparse_vg_gb300 import vg
        return vg.PagedKV(s["cache"][0], s["cache"][1], s["table"])

    def append(self, s, new, tokens, cu, kv_lens, positions, slots, q_out):
        from self_speculative_sparse_vg_gb300 import vg
        vg.step_tables(s["table"], self.pool, s["lens"], new, cu, kv_lens, positions, slots, owned=s["owned"],
                       free_pages=s["free"], free_count=s["count"], error_flag=s["flag"])
        q, k, v = (e[tokens.long()] for e in self.embed)
        vg.rope_append(self.kv(s), q, k, v, slots, q_out, positions=positions, inv_freq=self.freq, error_flag=s["flag"])
        s["lens"].copy_(kv_lens)

    def prompts(self, s, prompts):
        from self_speculative_sparse_vg_gb300 import vg
        new = np.zeros(self.R, int)
        new[::self.W] = [len(p) for p in prompts]
        n = int(new.sum())
        out = lambda *k: torch.zeros(*k, dtype=torch.int32, device="cuda")  # noqa: E731
        self.append(s, i32(new), i32(np.concatenate(prompts)), out(self.R + 1), out(self.R), out(n), out(n),
                    torch.zeros(n, self.Hq, self.d, dtype=torch.bfloat16, device="cuda"))
        vg.beam_tables(s["table"], self.pool, s["parents"], s["lens"], s["owned"], s["free"], s["count"], s["copies"],
                       error_flag=s["flag"])
        vg.copy_pages(self.kv(s), s["copies"], error_flag=s["flag"])

    def attend(self, s):
        from self_speculative_sparse_vg_gb300 import vg
        x, f, H = s, self.fixed, self.Hkv
        self.append(s, x["ones"], x["tokens"], x["cu"], x["kv_lens"], x["positions"], x["slots"], x["q"])
        vg.chunk_attention(self.kv(s), x["q"], x["cu"], x["kv_lens"], self.d ** -0.5, x["self_out"], error_flag=x["flag"])
        vg.cross_attention(x["q"], f["enc"][:, :H], f["enc"][:, H:], f["cu_req"], f["starts"], f["enc_lens"],
                           self.d ** -0.5, x["cross_out"], mask=f["mask"], error_flag=x["flag"])
        both = x["self_out"].float() + x["cross_out"].float()
        x["logits"].copy_(both.flatten(1) @ self.project)

    def choose(self, s):
        from self_speculative_sparse_vg_gb300 import vg
        vg.beam_select(s["logits"], s["scores"], s["scores"], s["next"], s["parents"], ended=s["ended"], end_token=1,
                       out_ended=s["ended"], error_flag=s["flag"])
        vg.beam_tables(s["table"], self.pool, s["parents"], s["lens"], s["owned"], s["free"], s["count"], s["copies"],
                       error_flag=s["flag"])
        vg.copy_pages(self.kv(s), s["copies"], error_flag=s["flag"])
        s["tokens"].copy_(s["next"].view(-1))


def _rows(dec, s, r):
    """Cached keys and values of row r, through its table."""
    n = int(s["lens"][r])
    pages = s["table"][r, :-(-n // PAGE)].long()
    return tuple(c[pages].transpose(1, 2).flatten(0, 1)[:n].cpu() for c in s["cache"])


@pytest.mark.parametrize("B,W,Hq,Hkv,d", [(2, 4, 8, 2, 64), (3, 3, 8, 1, 128), (1, 5, 4, 4, 64)])
def test_steps_against_the_oracles(B, W, Hq, Hkv, d):
    dec = Decoder(B, W, Hq, Hkv, d, 211, seed=B + W)
    s = dec.dev
    rng = np.random.default_rng(5)
    prompts = [rng.integers(2, dec.V, rng.integers(1, 60)) for _ in range(B)]
    history = [list(p) for p in prompts for _ in range(W)]
    dec.prompts(s, prompts)
    s["tokens"].copy_(i32(rng.integers(2, dec.V, dec.R)))
    s["scores"][:, 1:] = -float("inf")                    # the rows of a request are alike: one lives
    freq = dec.freq.double().cpu().numpy()
    for step in range(12):
        tokens = s["tokens"].cpu().tolist()
        dec.attend(s)
        for r in range(dec.R):
            history[r].append(tokens[r])
        q = s["q"].double().cpu().numpy()
        for r in range(dec.R):
            k, v = _rows(dec, s, r)
            h = torch.tensor(history[r])
            assert torch.equal(v, dec.embed[2].cpu()[h])                  # a row's cache is its history
            e = dec.embed[1].double().cpu()[h].numpy()
            turned = F.rope(e, [np.arange(len(h))], freq, [0] * (d // 2), False)
            assert (np.abs(k.double().numpy() - turned) <= 2.0 ** -8 * np.abs(turned) + 1e-4 * np.abs(e).max()).all()
            ro, rl, A, S = F.chunk_attention(q[r:r + 1], k.double().numpy(), v.double().numpy(), 1, d ** -0.5)
            tol, _ = chunk_bounds(ro, rl, A, S, np.array([[len(h)]]), d)
            assert (np.abs(s["self_out"][r:r + 1].double().cpu().numpy() - ro) <= tol).all()
        for b in range(B):
            a, n = int(dec.starts[b]), int(dec.enc_lens[b])
            kk, vv = (torch.nan_to_num(x.double()).numpy() for x in dec.enc[a:a + n].split(Hkv, 1))
            keep = dec.mask[a:a + n].numpy()
            rows = slice(b * W, (b + 1) * W)
            ro, rl, A, S = O.cross_attention(q[rows], kk, vv, keep, d ** -0.5)
            tol, _ = cross_bounds(ro, rl, A, S, int(keep.sum()), d, torch.bfloat16, 9.0)
            assert (np.abs(s["cross_out"][rows].double().cpu().numpy() - ro) <= tol).all()
        before = {k: s[k].clone() for k in ("scores", "ended", "table", "lens", "owned", "free", "count", "cache")}
        dec.choose(s)
        torch.cuda.synchronize()
        assert int(s["flag"].item()) == 0
        score, token, parent = check_select(s["logits"], before["scores"].cpu().numpy(), W,
                                            ended=before["ended"].cpu().numpy(), end_token=1)
        np.testing.assert_array_equal(s["parents"].cpu().numpy(), parent)
        np.testing.assert_array_equal(s["next"].cpu().numpy(), token)
        h = lambda k: before[k].cpu().numpy()  # noqa: E731
        want = O.beam_tables(parent, h("lens"), h("table"), dec.pool, h("owned"), h("free"), int(before["count"].item()))
        for k in ("table", "lens", "owned", "free", "copies"):
            np.testing.assert_array_equal(s[k].cpu().numpy(), want[k], err_msg=k)
        for i in range(2):
            pool = O.copy_pages(before["cache"][i].cpu().view(torch.int16).numpy(), want["copies"])
            np.testing.assert_array_equal(s["cache"][i].cpu().view(torch.int16).numpy(), pool)
        history = [list(history[b * W + parent[b, j]]) for b in range(B) for j in range(W)]
    # the search ends: every page comes back
    s["parents"].fill_(-1)
    from self_speculative_sparse_vg_gb300 import vg
    vg.beam_tables(s["table"], dec.pool, s["parents"], s["lens"], s["owned"], s["free"], s["count"], s["copies"],
                   error_flag=s["flag"])
    assert int(s["count"].item()) == dec.pool and sorted(s["free"].cpu().tolist()) == list(range(dec.pool))
    assert int(s["flag"].item()) == 0


def test_one_graph_of_a_step():
    """A whole step captured, on a stream of its own, and replayed as the search
    goes on, with work of other streams in between."""
    dec = Decoder(3, 4, 8, 2, 64, 1009, seed=3)
    rng = np.random.default_rng(1)
    prompts = [rng.integers(2, dec.V, n) for n in (17, 32, 5)]
    dec.prompts(dec.dev, prompts)
    dec.dev["tokens"].copy_(i32(rng.integers(2, dec.V, dec.R)))
    dec.dev["scores"][:, 1:] = -float("inf")
    a, b = dec.dev, {k: v.clone() for k, v in dec.dev.items()}
    warm = {k: v.clone() for k, v in dec.dev.items()}
    dec.attend(warm)
    dec.choose(warm)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dec.attend(a)
        dec.choose(a)
    for _ in range(25):
        graph.replay()
        junk = torch.full((1 << 22,), 255, dtype=torch.uint8, device="cuda")
        dec.attend(b)
        dec.choose(b)
        torch.cuda.synchronize()
        for name in a:
            x, y = a[name], b[name]
            if x.is_floating_point():
                x, y = torch.nan_to_num(x.float(), nan=7e9), torch.nan_to_num(y.float(), nan=7e9)
            assert torch.equal(x, y), name
        del junk
    assert int(a["flag"].item()) == 0

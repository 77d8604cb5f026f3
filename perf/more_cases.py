"""Device times that operators.py and more_operators.py do not show: block tables
in steps whose pages move (there a state's second pass finds them moved
already), chunk attention over hundreds of sequences, cross attention to long
states.

    python perf/more_cases.py

Each case is eight states called in one captured graph, replayed nine times
with the states put back in between: the median time of a call, microseconds.
"""
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from perf import more_operators  # noqa: E402
from self_speculative_sparse_vg_gb300 import vg  # noqa: E402

PAGE = 16
STATES, REPLAYS = 8, 9


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def pages(n):
    return -(-n // PAGE)


def decode_8(rng):
    """Eight sequences of 16K - 64K, six tokens each: a page taken now and then."""
    cached = rng.integers(16384, 65536, 8)
    return cached, np.full(8, 6), pages(cached)


def mixed_300(rng):
    """300 requests: single tokens to six, twelve prompts, eight that have finished."""
    cached, new = rng.integers(1, 32768, 300), rng.integers(1, 7, 300)
    who = rng.permutation(300)
    cached[who[:12]], new[who[:12]] = 0, rng.integers(100, 2049, 12)
    owned = pages(cached)
    cached[who[12:20]] = new[who[12:20]] = 0
    return cached, new, owned


def prompts_7(rng):
    """Seven fresh prompts of 8K - 16K tokens."""
    return np.zeros(7, int), rng.integers(8192, 16385, 7), np.zeros(7, int)


def finish_8(rng):
    """Eight requests that give back all their 1K - 4K pages."""
    return np.zeros(8, int), np.zeros(8, int), rng.integers(1000, 4097, 8)


def prompts_2000(rng):
    """2000 short prompts at once."""
    return np.zeros(2000, int), rng.integers(1, 400, 2000), np.zeros(2000, int)


class Tables:
    def __init__(self, lengths, seed):
        rng = np.random.default_rng(seed)
        cached, new, owned = lengths(rng)
        batch, width = len(cached), 4200
        spare, used = int(pages(cached + new).sum()) + 64, int(owned.sum())
        ids = rng.permutation(used + spare)
        table = np.full((batch, width), -1)
        table[np.arange(width)[None] < owned[:, None]] = ids[:used]
        room = int(new.sum()) + 3
        self.pool = used + spare
        self.lengths = i32(cached), i32(new)
        self.moved = i32(table), i32(owned), i32(np.concatenate([ids[used:], np.full(used + 8, -1)])), i32([spare])
        self.kept = [x.clone() for x in self.moved]
        self.outputs = tuple(torch.zeros(n, dtype=torch.int32, device="cuda") for n in (batch + 1, batch, room, room))

    def call(self):
        table, owned, free, count = self.moved
        vg.step_tables(table, self.pool, *self.lengths, *self.outputs, owned=owned, free_pages=free, free_count=count)

    def restore(self):
        for x, kept in zip(self.moved, self.kept):
            x.copy_(kept)


class Chunks:
    """Single tokens of `single` sequences over 0.5K - 4K positions, beside
    `chunk` tokens of one more over 6000 (none: 0); 32 / 8 heads of 128."""

    def __init__(self, single, chunk, seed):
        rng = np.random.default_rng(seed)
        new = np.array([1] * single + [chunk] * (chunk > 0))
        lens = np.concatenate([rng.integers(512, 4097, single), [6000 + chunk] * (chunk > 0)]).astype(int)
        order = rng.permutation(int(pages(lens).sum()))
        table = np.full((len(new), pages(int(lens.max()))), -1)
        table[np.arange(table.shape[1])[None] < pages(lens)[:, None]] = order
        pool = lambda: torch.randn(len(order), 8, PAGE, 128, device="cuda", dtype=torch.bfloat16)  # noqa: E731
        self.kv = vg.PagedKV(pool(), pool(), i32(table))
        self.q = torch.randn(int(new.sum()), 32, 128, device="cuda", dtype=torch.bfloat16)
        self.out = torch.empty_like(self.q)
        self.cu, self.lens = i32(np.concatenate([[0], np.cumsum(new)])), i32(lens)
        self.ws = torch.empty(vg.chunk_workspace_bytes(len(new), len(self.q), 32, 8, 128), dtype=torch.uint8,
                              device="cuda")
        self.bytes = 4 * 8 * 128 * int(lens.sum()) + 4 * self.q.numel()

    def call(self):
        vg.chunk_attention(self.kv, self.q, self.cu, self.lens, 128 ** -0.5, self.out, workspace=self.ws)

    def restore(self):
        pass


class Case:
    """A case of more_operators.py; what a call changes of a state is put back."""
    def __init__(self, name, seed, **changes):
        case = next(c for c in more_operators.listed() if c["name"] == name)
        self.state = more_operators.prepare({**case, **changes}, seed)
        self.kept = {k: self.state[k].clone() for k in ("table", "lens", "owned", "free", "count") if k in self.state}

    def call(self):
        more_operators.run(self.state)

    def restore(self):
        for k, v in self.kept.items():
            self.state[k].copy_(v)


class Cross:
    """`rows` rows of each of `batch` sequences to `states` states."""

    def __init__(self, batch, rows, states, Hq, Hkv, d):
        new = lambda n, h: torch.randn(n, h, d, device="cuda", dtype=torch.bfloat16)  # noqa: E731
        self.q, self.k, self.v = new(batch * rows, Hq), new(batch * states, Hkv), new(batch * states, Hkv)
        self.out = torch.empty_like(self.q)
        self.where = i32(np.arange(batch + 1) * rows), i32(np.arange(batch) * states), i32([states] * batch)
        self.ws = torch.empty(vg.cross_workspace_bytes(batch, batch * rows, Hq, Hkv, d), dtype=torch.uint8, device="cuda")
        self.bytes = 2 * (2 * self.k.numel() + 2 * self.q.numel())

    def call(self):
        vg.cross_attention(self.q, self.k, self.v, *self.where, self.q.shape[2] ** -0.5, self.out, workspace=self.ws)

    def restore(self):
        pass


def measure(states):
    for s in states:
        s.call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for s in states:
            s.call()
    times = []
    for _ in range(REPLAYS):
        for s in states:
            s.restore()
        torch.cuda.synchronize()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        graph.replay()
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b) * 1e3 / len(states))
    return sorted(times)[REPLAYS // 2]


def main():
    for lengths in (decode_8, mixed_300, prompts_7, finish_8, prompts_2000):
        us = measure([Tables(lengths, i) for i in range(STATES)])
        print(f"tables {lengths.__name__:14s} {us:7.2f} us", flush=True)
    for single, chunk in ((32, 0), (33, 0), (100, 0), (300, 0), (300, 1000)):
        states = [Chunks(single, chunk, i) for i in range(STATES)]
        us = measure(states)
        rate = np.mean([s.bytes for s in states]) / us * 1e-3
        print(f"chunk  {single} tokens + {chunk:4d}   {us:7.1f} us   {rate:6.0f} GB/s", flush=True)
    more_operators.own = True
    for name, changes in (("tables_b32", {}), ("tables_b32", dict(fresh=0.0, finished=0.0)), ("tables_one", {}),
                          ("select_one_32k", {}), ("select_b64_128k", {}), ("copy_layer", {}), ("copy_32_layers", {}),
                          ("cross_one_1500", {}), ("cross_beams_b24", {}), ("cross_verify_b8", {}),
                          ("cross_prompts_b5", {})):
        us = measure([Case(name, i, **changes) for i in range(STATES)])
        print(f"{name:16s} {str(changes or ''):36s} {us:7.2f} us", flush=True)
    for shape in ((64, 4, 1500, 16, 16, 64), (64, 64, 1500, 16, 16, 64), (64, 6, 6144, 16, 16, 64),
                  (64, 6, 6144, 32, 8, 128)):
        states = [Cross(*shape) for _ in range(2)]
        us = measure(states)
        print(f"cross  {shape} {us:7.1f} us   {states[0].bytes / us * 1e-3:6.0f} GB/s", flush=True)


if __name__ == "__main__":
    main()

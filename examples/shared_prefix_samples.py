"""Samples of one prompt on the paged K/V cache: shared pages, attention that reads the prompt once, pages given back.

All on the device:

    fp4idx_build_tables, fp4idx_store_kv   the prompt's tokens into the cache
    fp4idx_fork_requests, _copy_pages      samples that share the prompt's pages, each with its own unfinished page
    fp4idx_shared_prefix_attention         a decode step of all samples: the prompt is read once for all of them
    fp4idx_release_pages                   some samples end; the list of free pages
    fp4idx_compact_pages, _copy_pages      the pages in use moved to the pool's start

Model weights are stood in for by random activations.  Every step's attention is compared with plain torch.

    python examples/shared_prefix_samples.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from fp4_sparse_attention_gb300 import binding as B  # noqa: E402

PAGE = 64


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Samples:
    """One prompt (request 0) and its samples, and what a server keeps of them."""

    def __init__(self, prompt, samples, most_new, heads=32, kv_heads=4, seed=0):
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.heads, self.kv_heads, self.prompt, self.reqs = heads, kv_heads, prompt, samples + 1
        self.width = -(-(prompt + most_new) // PAGE) + 1
        self.pages = 3 * self.width + self.reqs * (-(-most_new // PAGE) + 2)
        shape = (self.pages, kv_heads, PAGE, 128)
        self.k, self.v = (torch.empty(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.cache = B.DevicePages([self.k, self.v])
        self.table = torch.full((self.reqs, self.width), -1, dtype=torch.int32, device="cuda")
        self.cached, self.lens = i32([0] * self.reqs), [0] * self.reqs     # on the device, and what the host knows
        self.free = torch.randperm(self.pages, generator=self.g, device="cuda").to(torch.int32)

    def randn(self, *shape):
        return torch.randn(shape, generator=self.g, device="cuda", dtype=torch.bfloat16)

    def step(self, new):
        """New tokens of each request through the cache and attention; returns the largest error against plain torch."""
        rows = sum(new)
        cu_q, cu_k, visible, slots, taken = B.fp4idx_build_tables(self.cached, i32(new), self.table, self.free, PAGE, rows,
                                                                  num_pages=self.pages)
        B.fp4idx_store_kv(self.randn(rows, self.kv_heads, 128), self.randn(rows, self.kv_heads, 128), slots, self.k, self.v)
        q = self.randn(rows, self.heads, 128)
        a = B.DeviceSharedAttention(q=q, k=self.k, v=self.v, cu_seqlens_q=cu_q, cu_seqlens_k=cu_k, block_table=self.table,
                                    visible_len=visible, max_seqlen_q=max(new), max_seqlen_k=max(n + m for n, m in zip(self.lens, new)),
                                    scale=128 ** -0.5, group_offsets=i32([0, self.reqs]), prefix_len=i32([self.prompt]), max_group_rows=rows)
        out, _ = B.fp4idx_shared_prefix_attention(a)
        self.cached += i32(new)
        self.lens = [n + m for n, m in zip(self.lens, new)]
        self.free = self.free[int(taken):]
        return max(self.error(q, out, visible, cu_q, t) for t in sorted({0, rows // 2, rows - 1}))

    def error(self, q, out, visible, cu_q, t):
        b, pos = int(torch.searchsorted(cu_q, t, right=True)) - 1, torch.arange(int(visible[t]), device="cuda")
        pages, worst = self.table[b].long()[pos // PAGE], 0.0
        for h in range(self.heads):
            hk = h // (self.heads // self.kv_heads)
            k, v = self.k[pages, hk, pos % PAGE].double(), self.v[pages, hk, pos % PAGE].double()
            w = torch.softmax(q[t, h].double() @ k.T * 128 ** -0.5, 0)
            worst = max(worst, float((out[t, h].double() - w @ v).abs().max()))
        return worst

    def fork(self):
        """All other requests continue request 0."""
        n = self.reqs - 1
        src, dst, taken = B.fp4idx_fork_requests(i32([0] * n), i32(list(range(1, n + 1))), self.cached, self.table, self.free, PAGE,
                                                 num_pages=self.pages)
        B.fp4idx_copy_pages(self.cache, src, dst)
        self.lens = [self.lens[0]] * self.reqs
        self.free = self.free[int(taken):]

    def release(self, gone):
        """Requests end; returns the number of free pages."""
        self.free, count = B.fp4idx_release_pages(i32(gone), self.cached, self.table, PAGE, self.pages)
        self.lens = [0 if b in gone else n for b, n in enumerate(self.lens)]
        self.free = self.free[:int(count)]
        return len(self.free)

    def compact(self, budget):
        """Pages in use to the pool's start, `budget` a time; returns the extent that is left."""
        while True:
            _, src, dst, moves, extent = B.fp4idx_compact_pages(self.cached, self.table, PAGE, self.pages, budget)
            B.fp4idx_copy_pages(self.cache, src, dst, count=moves)
            if int(moves) < budget:
                break
        self.release([])  # the free pages are others now
        return int(extent)


def main(prompt=700, samples=12, steps=3, budget=16):
    """Returns the largest error seen, the pages free after the release and the pool's extent after compaction."""
    s = Samples(prompt, samples, most_new=steps + 80)
    worst = s.step([prompt] + [0] * samples)
    s.fork()
    for _ in range(steps):
        worst = max(worst, s.step([1] * s.reqs))
    gone = list(range(0, s.reqs, 2))  # the first request, whose row the prompt was read through, among them
    free = s.release(gone)
    extent = s.compact(budget)
    left = [0 if b in gone else 1 for b in range(s.reqs)]
    worst = max(worst, s.step(left), s.step([70 * n for n in left]))  # a token, then a longer answer
    errors = B.fp4idx_get_error()
    if errors:
        raise RuntimeError(f"device error word {errors:#x}")
    print(f"{samples} samples of a prompt of {prompt}: largest error {worst:.4f}, {free} of {s.pages} pages free, extent {extent}")
    return worst, free, extent, s.pages


if __name__ == "__main__":
    main()

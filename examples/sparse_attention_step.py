"""Two steps of a serving loop on the FP4 indexer and the attention that consumes its selection.

Step 1 brings the prompts, step 2 decodes one token a request.  In each step, all on the device:

    fp4idx_build_tables                request lengths -> offsets, block table, slots, visible lengths
    fp4idx_store_k / _store_latent / _store_kv   the new tokens into the index, latent and K/V caches
    fp4idx_quantize_q, fp4idx_topk     the positions each row selects
    fp4idx_latent_attention            attention over the selected positions (latent cache)
    fp4idx_block_scores, _block_topk   the 128-key blocks each K/V head selects
    fp4idx_paged_attention             attention over the selected blocks (K/V cache)

The caches share one block table (pages of 64 tokens).  Model weights are stood in for by random
activations.  Every step's attention is compared with plain torch on a few rows.

    python examples/sparse_attention_step.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from fp4_sparse_attention_gb300 import MXFP4  # noqa: E402
from fp4_sparse_attention_gb300 import binding as B  # noqa: E402

PAGE = 64


class Caches:
    def __init__(self, pages, kv_heads):
        def empty(*shape, dtype=torch.bfloat16):
            return torch.empty(shape, dtype=dtype, device="cuda")

        self.index_k = empty(pages, 1, PAGE, 64, dtype=torch.uint8)       # packed E2M1 codes
        self.index_scale = empty(pages, 1, PAGE, 4, dtype=torch.uint8)    # E8M0 scales
        self.latent = empty(pages, PAGE, 576)
        self.k, self.v = empty(pages, kv_heads, PAGE, 128), empty(pages, kv_heads, PAGE, 128)


def step(caches, cached, new, table, free_pages, *, index_heads=8, latent_heads=16, heads=32, kv_heads=4, top_k=128,
         top_blocks=4, seed=0):
    """One step; cached and new are host lists.  Returns a dict of what it computed."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=g, device="cuda", dtype=dtype)

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    rows, longest, most_new = sum(new), max(c + n for c, n in zip(cached, new)), max(new)
    cu_q, cu_k, visible, slots, taken = B.fp4idx_build_tables(i32(cached), i32(new), table, free_pages, PAGE, rows,
                                                              num_pages=caches.latent.shape[0])
    # what the model's projections would give for the new tokens
    B.fp4idx_store_k(randn(rows, 1, 128), slots, PAGE, caches.index_k, caches.index_scale)
    latent = randn(rows, 576)
    B.fp4idx_store_latent(latent[:, :512], latent[:, 512:], slots, caches.latent)
    kv = randn(rows, 2, kv_heads, 128)
    B.fp4idx_store_kv(kv[:, 0], kv[:, 1], slots, caches.k, caches.v)
    where = dict(cu_seqlens_q=cu_q, cu_seqlens_k=cu_k, block_table=table, visible_len=visible, max_seqlen_q=most_new,
                 max_seqlen_k=longest)

    # positions: weighted-ReLU indexer, then latent attention over each row's own top-k
    q_codes, q_scale = B.fp4idx_quantize_q(randn(rows, index_heads, 128))
    index = B.DeviceProblem(format=MXFP4, num_heads=index_heads, num_kv_heads=1, page_size=PAGE, q=q_codes, q_scale=q_scale,
                            k=caches.index_k, k_scale=caches.index_scale, **where)
    positions, _, _ = B.fp4idx_topk(index, randn(rows, index_heads, dtype=torch.float32), top_k)
    q_latent = randn(rows, latent_heads, 576)
    a = B.DeviceAttention(q=q_latent, k=caches.latent, indices=positions, scale=576 ** -0.5, **where)
    out_latent, _ = B.fp4idx_latent_attention(a)

    # blocks: one index head per K/V head, then grouped-query attention over each head's own blocks
    b_codes, b_scale = B.fp4idx_quantize_q(randn(rows, kv_heads, 128))
    blocks = B.DeviceProblem(format=MXFP4, num_heads=kv_heads, num_kv_heads=1, page_size=PAGE, q=b_codes, q_scale=b_scale,
                             k=caches.index_k, k_scale=caches.index_scale, **where)
    chosen, _, _ = B.fp4idx_block_topk(B.fp4idx_block_scores(blocks), top_blocks)
    q = randn(rows, heads, 128)
    b = B.DeviceAttention(q=q, k=caches.k, v=caches.v, indices=chosen, scale=128 ** -0.5, **where)
    out, _ = B.fp4idx_paged_attention(b)
    return dict(cu_q=cu_q, visible=visible, slots=slots, taken=taken, positions=positions, q_latent=q_latent,
                out_latent=out_latent, blocks=chosen, q=q, out=out)


def check(caches, table, r, t):
    """Largest errors of row t against plain torch in 64 bits: (latent, paged)."""
    b = int(torch.searchsorted(r["cu_q"], t, right=True)) - 1
    vis, pages = int(r["visible"][t]), table[b].long()

    def gather(cache, pos):
        return cache[pages[pos // PAGE], pos % PAGE].double()

    pos = r["positions"][t].long()
    pos = pos[(pos >= 0) & (pos < vis)]
    c = gather(caches.latent, pos)
    w = torch.softmax(r["q_latent"][t].double() @ c.T * 576 ** -0.5, 1)
    worst = [float((r["out_latent"][t].double() - w @ c[:, :512]).abs().max()), 0.0]
    group = r["q"].shape[1] // caches.k.shape[1]
    for h in range(r["q"].shape[1]):
        blk = r["blocks"][h // group, t].long()
        pos = (blk[blk >= 0, None] * 128 + torch.arange(128, device="cuda")).flatten()
        pos = pos[pos < vis]
        k, v = gather(caches.k[:, h // group], pos), gather(caches.v[:, h // group], pos)
        w = torch.softmax(r["q"][t, h].double() @ k.T * 128 ** -0.5, 0)
        worst[1] = max(worst[1], float((r["out"][t, h].double() - w @ v).abs().max()))
    return worst


def main(prompts=(700, 33, 1500, 128), max_len=2048):
    """Returns the largest errors seen and the pages in use after the two steps."""
    pages = sum(-(-max_len // PAGE) for _ in prompts)
    caches = Caches(pages, kv_heads=4)
    table = torch.full((len(prompts), -(-max_len // PAGE)), -1, dtype=torch.int32, device="cuda")
    free_pages = torch.randperm(pages, device="cuda").to(torch.int32)
    used, worst = 0, [0.0, 0.0]
    for n, (cached, new) in enumerate([([0] * len(prompts), list(prompts)), (list(prompts), [1] * len(prompts))]):
        r = step(caches, cached, new, table, free_pages[used:], seed=n)
        used += int(r["taken"])
        rows = r["q"].shape[0]
        for t in sorted({0, rows // 3, rows // 2, rows - 1}):
            worst = [max(a, b) for a, b in zip(worst, check(caches, table, r, t))]
        print(f"step {n + 1}: {rows} rows, {used} pages in use, largest error latent {worst[0]:.4f} paged {worst[1]:.4f}")
    errors = B.fp4idx_get_error()
    if errors:
        raise RuntimeError(f"device error word {errors:#x}")
    return worst, used


if __name__ == "__main__":
    main()

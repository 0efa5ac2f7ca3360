"""Fork, copies, a step's tables, its keys and its attention one behind the other without a number read back: the
free pages are listed again between the calls that take some."""
import pytest
import torch

from fp4_sparse_attention_gb300 import binding as B

pytestmark = pytest.mark.gpu
PAGE, WIDTH = 64, 9


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("prompt", [1, 63, 64, 130, 300])
@pytest.mark.parametrize("samples", [1, 20])
def test_fork_and_step_in_one_graph(prompt, samples):
    reqs, P, kv, heads = samples + 1, 400, 2, 16
    g = torch.Generator(device="cuda").manual_seed(prompt + samples)
    k, v = (torch.randn((P, kv, PAGE, 128), generator=g, device="cuda").bfloat16() for _ in range(2))
    order = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
    start = torch.full((reqs, WIDTH), -1, dtype=torch.int32, device="cuda")
    start[0, :-(-prompt // PAGE)] = order[:-(-prompt // PAGE)]
    table, cached = start.clone(), i32([prompt] + [0] * samples)
    parent, child, new = i32([0] * samples), i32(list(range(1, reqs))), i32([1 + b % 70 for b in range(reqs)])
    rows = int(new.sum())
    nk, nv = (torch.randn((rows, kv, 128), generator=g, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn((rows, heads, 128), generator=g, device="cuda").bfloat16()
    pages, groups, prefix = B.DevicePages([k, v]), i32([0, reqs]), i32([prompt])

    def step():
        free, _ = B.fp4idx_release_pages(None, cached, table, PAGE, P)
        src, dst, _ = B.fp4idx_fork_requests(parent, child, cached, table, free, PAGE, num_pages=P)
        B.fp4idx_copy_pages(pages, src, dst)
        free, _ = B.fp4idx_release_pages(None, cached, table, PAGE, P)  # without the children's pages
        cu_q, cu_k, visible, slots, _ = B.fp4idx_build_tables(cached, new, table, free, PAGE, rows, num_pages=P)
        B.fp4idx_store_kv(nk, nv, slots, k, v)
        a = B.DeviceSharedAttention(q=q, k=k, v=v, cu_seqlens_q=cu_q, cu_seqlens_k=cu_k, block_table=table, visible_len=visible,
                                    max_seqlen_q=70, max_seqlen_k=prompt + 70, scale=128 ** -0.5, group_offsets=groups, prefix_len=prefix,
                                    max_group_rows=rows)
        B.fp4idx_shared_prefix_attention(a)
        return a

    kept = k.clone(), v.clone()
    step()  # (loads the kernels)
    for x, y in zip((k, v), kept):
        x.copy_(y)
    table.copy_(start)
    cached.copy_(i32([prompt] + [0] * samples))
    torch.cuda.synchronize()
    B.fp4idx_get_error(clear=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a = step()
    graph.replay()
    torch.cuda.synchronize()
    assert B.fp4idx_get_error(clear=True) == 0
    lens, t = [prompt + n for n in new.tolist()], table.tolist()
    full = prompt // PAGE
    mine = [t[b][full:-(-n // PAGE)] for b, n in enumerate(lens)]
    assert all(row[:full] == t[0][:full] for row in t)
    named = [p for m in mine for p in m]
    assert len(set(named)) == len(named) and not set(named) & set(t[0][:full]) and all(0 <= p < P for p in named)
    # each row against the formula in 64 bits; |v| stays below 6, and the weights' and the result's rounding to bf16 is 2^-8 each
    row = 0
    for b, n in enumerate(lens):
        pos = torch.arange(n, device="cuda")
        pg = table[b].long()[pos // PAGE]
        for hk in range(kv):
            kk, vv = k[pg, hk, pos % PAGE].double(), v[pg, hk, pos % PAGE].double()
            for i in range(int(new[b])):
                s = q[row + i, hk * 8:hk * 8 + 8].double() @ kk[:prompt + i + 1].T * 128 ** -0.5
                want = torch.softmax(s, 1) @ vv[:prompt + i + 1]
                assert float((a.out[row + i, hk * 8:hk * 8 + 8].double() - want).abs().max()) <= 6 * 2 * 2.0 ** -8
        row += int(new[b])

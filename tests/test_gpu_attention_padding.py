"""Batches padded to a fixed row count (a graph captured once, the tables of fp4idx_build_tables with
more rows than the requests bring): rows of no request get zeros and -inf in every form of attention."""
import math

import pytest
import torch

from fp4_sparse_attention_gb300 import binding as B
from tests import attention_ref as R

pytestmark = pytest.mark.gpu


def padded(c, extra, **over):
    """A call of the case's rows and `extra` more, whose inputs are whatever a buffer may hold."""
    T, H, dk = c["q"].shape
    q = torch.full((T + extra, H, dk), math.nan, dtype=c["q"].dtype, device="cuda")
    q[:T] = c["q"]
    a = dict(q=q, k=c["k"], v=c["v"], cu_seqlens_q=R.offsets(c["q_lens"], "cuda"), cu_seqlens_k=R.offsets(c["k_lens"], "cuda"),
             block_table=R.table_of(c), max_seqlen_q=max(c["q_lens"] + [1]), max_seqlen_k=max(c["k_lens"]), scale=c["scale"],
             causal=c.get("causal", False))
    if c.get("visible_len") is not None:
        a["visible_len"] = torch.cat([c["visible_len"], torch.full((extra,), 5, dtype=torch.int32, device="cuda")])
    if c.get("indices") is not None:
        idx = c["indices"]
        a["indices"] = torch.cat([idx, torch.zeros(idx.shape[:-2] + (extra, idx.shape[-1]), dtype=torch.int32, device="cuda")],
                                 idx.dim() - 2).contiguous()
    a.update(over)
    a = B.DeviceAttention(**a)
    a.out.fill_(math.nan)
    a.lse.fill_(math.nan)
    return a


def run(c, extra, **over):
    a = padded(c, extra, **over)
    T = c["q"].shape[0]
    B.fp4idx_get_error(clear=True)
    out, lse = (B.fp4idx_latent_attention if c["v"] is None else B.fp4idx_paged_attention)(a)
    torch.cuda.synchronize()
    assert B.fp4idx_get_error(clear=True) == 0
    assert bool((out[T:] == 0).all()) and bool((lse[T:] == -math.inf).all())
    want, want_lse, b_out, b_lse = R.reference(c)
    assert bool(((out[:T].double() - want).abs() <= b_out).all())
    none = want_lse == -math.inf
    assert torch.equal(lse[:T] == -math.inf, none)
    assert bool(((lse[:T].double() - want_lse).abs() <= b_lse)[~none].all())


@pytest.mark.parametrize("visibility", ["causal", "full", "lens"])
@pytest.mark.parametrize("kv", [None, 2])
@pytest.mark.parametrize("select", [0, 3])
@pytest.mark.parametrize("extra", [1, 7])
def test_rows_of_no_request(extra, select, kv, visibility):
    c = R.make_case(31 + extra, [2, 0, 1], [300, 5, 200], heads=6, kv_heads=kv, select=select, visibility=visibility, device="cuda")
    run(c, extra)


@pytest.mark.parametrize("kv,heads", [(None, 128), (2, 6)])
def test_more_padding_than_rows(kv, heads):
    run(R.make_case(32, [1] * 5, [2000, 9, 64, 300, 1], heads=heads, kv_heads=kv, device="cuda"), 1000)


@pytest.mark.parametrize("kv", [None, 2])
@pytest.mark.parametrize("select", [0, 3])
def test_only_padding(select, kv):
    c = R.make_case(33, [0, 0], [70, 3], heads=6, kv_heads=kv, visibility="full", device="cuda")
    if select:
        c["indices"] = torch.zeros(((0, 3) if kv is None else (kv, 0, 3)), dtype=torch.int32, device="cuda")
    run(c, 9)


@pytest.mark.parametrize("kv", [None, 2])
def test_strided_outputs_are_cleared_in_place_only(kv):
    c = R.make_case(34, [2], [100], heads=6, kv_heads=kv, device="cuda")
    wide = torch.full((2 + 4, 8, 512 if kv is None else 128), 3.0, dtype=c["q"].dtype, device="cuda")
    a = padded(c, 4, out=wide[:, 1:7])
    wide.fill_(3.0)
    (B.fp4idx_latent_attention if kv is None else B.fp4idx_paged_attention)(a)
    torch.cuda.synchronize()
    assert bool((wide[2:, 1:7] == 0).all()) and bool((wide[:, 0] == 3).all()) and bool((wide[:, 7] == 3).all())


@pytest.mark.parametrize("kv", [None, 2])
def test_replays_of_a_padded_graph_with_fewer_rows(kv):
    # captured with every row in use, replayed with fewer: no row keeps what the replay before wrote
    c = R.make_case(35, [3, 3], [200, 130], heads=6, kv_heads=kv, device="cuda")
    a = padded(c, 0)
    call = B.fp4idx_latent_attention if kv is None else B.fp4idx_paged_attention
    call(a)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(a)
    g.replay()
    torch.cuda.synchronize()
    assert bool(torch.isfinite(a.lse).all())
    a.cu_seqlens_q.copy_(torch.tensor([0, 3, 4], dtype=torch.int32, device="cuda"))
    g.replay()
    torch.cuda.synchronize()
    assert bool((a.out[4:] == 0).all()) and bool((a.lse[4:] == -math.inf).all())
    d = dict(c, q_lens=[3, 1], q=c["q"][:4])
    want, _, b_out, _ = R.reference(d)
    assert bool(((a.out[:4].double() - want).abs() <= b_out).all())


@pytest.mark.parametrize("kv", [None, 2])
def test_with_the_tables_of_a_padded_step(kv):
    c = R.make_case(36, [1, 4], [129, 64], heads=6, kv_heads=kv, device="cuda")
    lens = torch.tensor([128, 60], dtype=torch.int32, device="cuda")
    new = torch.tensor(c["q_lens"], dtype=torch.int32, device="cuda")
    table = R.table_of(c)
    free = torch.tensor(c["pages"][0][2:], dtype=torch.int32, device="cuda")
    cu_q, cu_k, visible, slots, _ = B.fp4idx_build_tables(lens, new, table, free, 64, 12, num_pages=c["k"].shape[0])
    assert visible[5:].eq(0).all() and slots[5:].eq(-1).all()
    run(c, 7, cu_seqlens_q=cu_q, cu_seqlens_k=cu_k, block_table=table, visible_len=visible)

"""Attention of requests that share a prefix: infinite and NaN values that a request alone sees stay in its own rows.

Weights, references and sums come from queries and keys, so with other values at a request's own positions the other
requests' outputs are the same bits, and every row's log-sum is."""
import math

import pytest
import torch

from fp4_sparse_attention_gb300 import binding as B
from tests import attention_ref as R
from tests import shared_ref as S
from tests.test_gpu_shared_attention import build, check

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16
BAD = (math.nan, math.inf, -math.inf)


def run(c):
    B.fp4idx_get_error(clear=True)
    out, lse = B.fp4idx_shared_prefix_attention(build(c))
    torch.cuda.synchronize()
    assert B.fp4idx_get_error(clear=True) == 0
    return out, lse


def spoil(c, b, positions, what, names=("v",)):
    """Non-finite values of request b at its own positions; a channel's bad value differs from its neighbours'."""
    for n, s in enumerate(positions):
        at = c["pages"][b][s // c["page"]]
        for name in names:
            x = c[name][at, :, s % c["page"]]
            x[...] = BAD[n % 3] if what is None else what


def rows_of(c, b):
    lo = sum(c["q_lens"][:b])
    return slice(lo, lo + c["q_lens"][b])


def check_spoiled(groups, bad, what=None, dtype=BF16, neighbours=True, **kw):
    """`bad`: requests of which some own positions are spoilt: the first, one in each tile, the last."""
    c = S.make_shared(sum(bad) + 5, groups, dtype=dtype, device="cuda", visibility="full", **kw)
    clean, clean_lse = (x.clone() for x in run(c))
    check(c, (clean, clean_lse))
    prefixes = [n for n, reqs in groups for _ in reqs]
    for b in bad:
        own = range(prefixes[b], c["k_lens"][b])
        spoil(c, b, sorted({own[0], own[-1], *own[::100]}), what)
    out, lse = run(c)
    assert torch.equal(lse, clean_lse)
    for b in range(len(c["q_lens"])):
        rows = rows_of(c, b)
        if b in bad:
            assert not bool(torch.isfinite(out[rows]).any()), b
        else:
            assert torch.equal(out[rows], clean[rows]), f"request {b}"
    if neighbours:  # the same from the call that knows no sharing
        a = build(c)
        p = B.DeviceAttention(q=a.q, k=a.k, v=a.v, cu_seqlens_q=a.cu_seqlens_q, cu_seqlens_k=a.cu_seqlens_k, block_table=a.block_table,
                              max_seqlen_q=max(c["q_lens"]), max_seqlen_k=max(c["k_lens"]), scale=c["scale"])
        paged, _ = B.fp4idx_paged_attention(p)
        assert torch.equal(torch.isfinite(paged), torch.isfinite(out))


# 8 heads a K/V head: a request of one row is 8 pairs of the 256 of a block
GROUPS = {
    "one accumulator": [(200, [(1, 31), (1, 90), (1, 5)])],
    "both accumulators": [(200, [(1, 1 + (37 * i) % 150) for i in range(32)])],
    "a request in both": [(70, [(15, 20), (3, 40), (13, 150)])],
    "blocks that end inside a request": [(70, [(20, 20), (30, 40), (13, 150), (40, 41)])],
    "no prefix": [(0, [(1, 300), (2, 17), (1, 1)])],
    "the prefix ends with a page": [(128, [(1, 64), (1, 1), (2, 128)])],
    "joined": [(64, [(1, 9000), (1, 5000), (1, 70)])],
    "joined, both accumulators": [(20011, [(1, 200 + 100 * i) for i in range(32)])],
    "several groups": [(300, [(4, 60), (1, 10), (3, 400)]), (0, [(2, 70), (2, 70)]), (129, [(2, 5), (2, 129)])],
}


@pytest.mark.parametrize("name", GROUPS)
@pytest.mark.parametrize("which", ["first", "middle", "last"])
def test_values_of_one_request_stay_in_its_rows(name, which):
    n = sum(len(reqs) for _, reqs in GROUPS[name])
    check_spoiled(GROUPS[name], {"first": [0], "middle": [n // 2], "last": [n - 1]}[which], heads=16, kv_heads=2)


@pytest.mark.parametrize("name", ["one accumulator", "both accumulators", "joined"])
@pytest.mark.parametrize("what", BAD)
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_every_value_and_type(name, what, dtype):
    check_spoiled(GROUPS[name], [1], what=what, dtype=dtype, heads=16, kv_heads=2, page=128)


@pytest.mark.parametrize("heads,kv", [(1, 1), (6, 2), (40, 8), (256, 2), (300, 1)])
def test_head_layouts(heads, kv):
    check_spoiled([(100, [(1, 40), (2, 77), (1, 9)]), (129, [(1, 3), (1, 70)])], [1, 3], heads=heads, kv_heads=kv)


def test_all_but_one_request():
    groups = [(500, [(1, 1 + (53 * i) % 300) for i in range(40)])]
    check_spoiled(groups, [i for i in range(40) if i != 17], heads=16, kv_heads=2)
    check_spoiled([(70, [(1, 1 + i % 40) for i in range(300)])], [i for i in range(300) if i % 7], heads=2, kv_heads=2, neighbours=False)


def test_long_runs():
    groups = [(1001 + 1143 * i, [(4, 5 + (331 * (6 * i + j)) % 700) for j in range(3)]) for i in range(8)]
    check_spoiled(groups, [0, 4, 8, 13, 23], heads=40, kv_heads=8)
    check_spoiled([(0, [(70, 9000), (60, 3000), (1, 17)])], [1], heads=8, kv_heads=2)


def test_keys_and_queries_of_one_request():
    # non-finite scores, too, are a matter of the rows that have them
    c = S.make_shared(3, [(200, [(1, 31), (2, 150), (1, 5)])], heads=16, kv_heads=2, device="cuda", visibility="full")
    want, want_lse, b_out, b_lse = R.reference(c)
    spoil(c, 1, [200, 270, 349], math.nan, names=("k", "v"))
    c["q"][1] = math.inf
    out, lse = run(c)
    for t in (0, 3):
        assert bool(((out[t].double() - want[t]).abs() <= b_out[t]).all()) and bool(((lse[t].double() - want_lse[t]).abs() <= b_lse[t]).all())
    assert bool(out[1:3].isnan().all()) and bool(lse[1:3].isnan().all())


def test_replays_with_changing_values():
    # a segment's rows start from zeros each time, whatever TMEM held
    c = S.make_shared(4, [(64, [(1, 500), (1, 300)] * 20)], heads=16, kv_heads=2, device="cuda", visibility="full")
    a = build(c)
    want = [x.clone() for x in B.fp4idx_shared_prefix_attention(a)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.fp4idx_shared_prefix_attention(a)
    kept = c["v"].clone()
    for b in (0, 7, 39, None):
        c["v"].copy_(kept)
        if b is not None:
            spoil(c, b, range(64, c["k_lens"][b]), math.nan)
        a.out.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        good = torch.ones(40, dtype=torch.bool, device="cuda")
        if b is not None:
            good[b] = False
        assert torch.equal(a.out[good], want[0][good]) and torch.equal(a.lse, want[1])
        assert b is None or bool(a.out[b].isnan().all())

"""Groups with more rows than the call's bound: reported, the rows up to the bound as ever, the others not written."""
import math

import pytest
import torch

from fp4_sparse_attention_gb300 import binding as B
from tests import attention_ref as R
from tests import shared_ref as S
from tests.test_gpu_shared_attention import build

pytestmark = pytest.mark.gpu


def run(groups, bound, **kw):
    c = S.make_shared(31, groups, device="cuda", visibility="full", **kw)
    B.fp4idx_get_error(clear=True)
    a = build(c, max_group_rows=bound)
    out, lse = B.fp4idx_shared_prefix_attention(a)
    torch.cuda.synchronize()
    return c, out, lse, B.fp4idx_get_error(clear=True)


@pytest.mark.parametrize("bound", [1, 3, 32, 33, 69])
def test_rows_past_the_bound(bound):
    # groups of 70, 1 and 40 rows; 16 pairs a row: blocks of 16 rows
    groups = [(100, [(50, 60), (20, 90)]), (64, [(1, 5)]), (70, [(39, 39), (1, 200)])]
    c, out, lse, err = run(groups, bound, heads=16, kv_heads=1)
    assert err == S.ERR_LENGTHS
    want, want_lse, b_out, b_lse = R.reference(c)
    first = 0
    for _, reqs in groups:
        rows = sum(r for r, _ in reqs)
        done, left = slice(first, first + min(rows, bound)), slice(first + min(rows, bound), first + rows)
        assert bool(((out[done].double() - want[done]).abs() <= b_out[done]).all())
        assert bool(((lse[done].double() - want_lse[done]).abs() <= b_lse[done]).all())
        assert bool(out[left].isnan().all()) and bool(lse[left].isnan().all())  # what build() filled them with
        first += rows


def test_bounds_that_hold():
    groups = [(100, [(5, 60), (2, 90)]), (64, []), (70, [(7, 39), (0, 9)])]
    for bound in (7, 8, 1 << 20):
        assert run(groups, bound, heads=16, kv_heads=2)[3] == 0
    # many requests of one row: a CTA plans a block
    assert run([(70, [(1, 3)] * 300)], 300, heads=2, kv_heads=2)[3] == 0
    assert run([(70, [(1, 3)] * 300)], 299, heads=2, kv_heads=2)[3] == S.ERR_LENGTHS


def test_rows_that_no_batch_has():
    # cu_seqlens_q goes past the batch's rows: only the rows that there are count
    c = S.make_shared(32, [(100, [(3, 60), (2, 90)])], device="cuda", visibility="full", heads=16, kv_heads=2)
    B.fp4idx_get_error(clear=True)
    a = build(c, max_group_rows=3, q=c["q"][:3].contiguous())
    out, _ = B.fp4idx_shared_prefix_attention(a)
    torch.cuda.synchronize()
    want, _, b_out, _ = R.reference(c)
    assert B.fp4idx_get_error(clear=True) == 0 and bool(((out.double() - want[:3]).abs() <= b_out[:3]).all())
    assert not math.isnan(float(out.float().sum()))

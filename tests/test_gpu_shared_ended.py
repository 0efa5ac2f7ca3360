"""Requests of a group that have ended or are shorter than the prefix, the first one among them: the prefix is still
read once, through a request that has it.  (The other requests' entries below it name no pages.)"""
import pytest
import torch

from fp4_sparse_attention_gb300 import binding as B
from tests import attention_ref as R
from tests import shared_ref as S
from tests.test_gpu_shared_attention import build, check

pytestmark = pytest.mark.gpu


def case(prefix, reqs, lens, through, heads=16, kv_heads=2, page=64, seed=1):
    """One group; `lens`: key counts other than the ones that it was made with, by request (0: ended, without rows)."""
    reqs = [(0 if lens.get(b) == 0 else r, n) for b, (r, n) in enumerate(reqs)]
    c = S.make_shared(seed, [(prefix, reqs)], heads=heads, kv_heads=kv_heads, page=page, visibility="full", device="cuda")
    table = R.table_of(c)
    for b, n in lens.items():
        c["k_lens"][b] = n
    for b in range(len(reqs)):  # whole pages below the prefix
        if b != through:
            table[b, :prefix // page] = -1
    return c, table


def run(c, table, **over):
    B.fp4idx_get_error(clear=True)
    a = build(c, block_table=table, max_seqlen_k=table.shape[1] * c["page"], **over)
    got = B.fp4idx_shared_prefix_attention(a)
    torch.cuda.synchronize()
    assert B.fp4idx_get_error(clear=True) == 0
    check(c, got)


REQS = [(1, 20), (2, 31), (1, 150), (1, 1)]


@pytest.mark.parametrize("prefix", [64, 300, 640, 1000])
@pytest.mark.parametrize("page", [64, 128])
def test_the_first_requests_have_ended(prefix, page):
    for ended in ([], [0], [0, 1], [0, 1, 2], [1], [3]):
        through = min(b for b in range(4) if b not in ended)
        run(*case(prefix, REQS, {b: 0 for b in ended}, through, page=page))


def test_the_first_requests_are_shorter():
    # keys 0..n of the prefix alone: their rows see those, read through another request's row
    for n in (1, 63, 64, 65, 299):
        run(*case(300, REQS, {0: n}, 1))
        run(*case(300, REQS, {0: n, 1: 64}, 2))
        run(*case(300, REQS, {0: 0, 1: n}, 2))
    run(*case(300, REQS, {0: 300}, 0))


def test_none_reaches_the_end():
    # the longest one's keys bound the prefix, the first of two alike
    for lens, through in (({0: 10, 1: 100, 2: 290, 3: 70}, 2), ({0: 290, 1: 290, 2: 290, 3: 5}, 0), ({0: 64, 1: 128, 2: 128, 3: 0}, 1)):
        c, table = case(300, REQS, lens, through)
        table[through] = R.table_of(c)[through]
        run(c, table)


@pytest.mark.parametrize("ended", [1, 31, 32, 33, 64, 95, 99])
def test_many_have_ended(ended):
    reqs = [(1, 1 + (37 * i) % 90) for i in range(100)]
    run(*case(200, reqs, {b: 0 for b in range(ended)}, ended))


def test_a_cta_plans_a_block():
    reqs = [(1, 1 + (37 * i) % 40) for i in range(300)]
    for ended in (0, 40, 270):
        run(*case(130, reqs, {b: 0 for b in range(ended)}, ended, heads=2, kv_heads=2))


def test_no_keys_at_all():
    c, table = case(300, REQS, {1: 0, 2: 0, 3: 0}, 0)
    c["k_lens"][0] = 0  # a row without keys
    run(c, table)


def test_a_request_that_ends_between_replays():
    c, table = case(300, [(0, 20)] + [(1, 1 + 17 * i) for i in range(20)], {}, 0)
    table = R.table_of(c)
    a = build(c, block_table=table, max_seqlen_k=table.shape[1] * 64)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.fp4idx_shared_prefix_attention(a)
    graph.replay()
    check(c, (a.out, a.lse))
    c["k_lens"][0] = 0
    a.cu_seqlens_k.copy_(R.offsets(c["k_lens"], "cuda"))
    table[0] = -1           # its entries are nobody's now
    table[2:, :4] = -1
    graph.replay()
    torch.cuda.synchronize()
    check(c, (a.out, a.lse))
    assert B.fp4idx_get_error(clear=True) == 0

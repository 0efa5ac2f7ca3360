"""Forks that are given free pages past the pool: none gets into a table or a copy list."""
import pytest
import torch

from fp4_sparse_attention_gb300 import binding as B
from tests import shared_ref as S

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def fork(parent, child, cached, table, free, num_pages):
    cached, table = i32(cached), i32(table)
    B.fp4idx_get_error(clear=True)
    src, dst, taken = B.fp4idx_fork_requests(i32(parent), i32(child), cached, table, i32(free), 64, num_pages=num_pages)
    return cached.tolist(), table.tolist(), src.tolist(), dst.tolist(), int(taken), B.fp4idx_get_error(clear=True)


TABLE = [[10 * b + j for j in range(3)] for b in range(8)]


@pytest.mark.parametrize("bad", [100, 101, 2 ** 31 - 1])
def test_free_pages_past_the_pool(bad):
    # as a negative entry, but for the error bit: the page is counted as taken and the next fork gets the next one
    got = fork([0, 0, 0], [1, 2, 3], [100] * 8, TABLE, [70, bad, 71], 100)
    want = S.fork([0, 0, 0], [1, 2, 3], None, [100] * 8, TABLE, [70, -1, 71], 64, 100)
    assert got[:5] == want[:5] and got[5] == S.ERR_PAGE_RANGE
    assert got[3] == [70, -1, 71] and got[2] == [1, -1, 1] and got[1][2] == [0, -1, 22]


def test_the_last_page_and_other_errors_beside_it():
    assert fork([0], [1], [100] * 8, TABLE, [99], 100)[3:] == ([99], 1, 0)
    got = fork([0, 0, 0], [1, 2, 3], [100] * 8, TABLE, [200, -1], 100)
    assert got[3] == [-1] * 3 and got[4] == 2 and got[5] == S.ERR_PAGE_RANGE | S.ERR_LENGTHS
    # forks that end with a page take none, refused ones count theirs
    got = fork([0, 4, 0, 0], [1, 2, 1, 3], [100, 0, 0, 0, 128, 0, 0, 0], TABLE, [99, 500, 98], 100)
    assert got[3] == [99, -1, -1, 98] and got[5] == S.ERR_REQUESTS


def test_many_forks():
    n = 300
    free = [1000 + i if i % 7 == 3 else i for i in range(n)]
    table = [[500, 501]] + [[0, 0] for _ in range(n)]
    got = fork([0] * n, list(range(1, n + 1)), [65] + [0] * n, table, free, 1000)
    want = [-1 if i % 7 == 3 else i for i in range(n)]
    assert got[3] == want and [row[1] for row in got[1][1:]] == want and got[4] == n and got[5] == S.ERR_PAGE_RANGE
    assert got[2] == [-1 if x < 0 else 501 for x in want] and got[0] == [65] * (n + 1)

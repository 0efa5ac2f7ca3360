"""Step tables with one long prompt among many short requests: right, and written by more than one warp."""
import pytest
import torch

from fp4_sparse_attention_gb300 import binding as B
from tests.test_gpu_cache_rows import _i32, _step, plain_tables, run_tables

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page", [64, 128])
@pytest.mark.parametrize("reqs,at,rows", [(2048, 1000, 32768), (300, 299, 5000), (64, 0, 257), (64, 63, 9001), (3, 1, 70000), (5000, 17, 12345)])
def test_one_long_prompt(reqs, at, rows, page):
    g = torch.Generator().manual_seed(reqs + rows)
    cached = torch.randint(0, 300, (reqs,), generator=g).tolist()
    new = torch.randint(0, 3, (reqs,), generator=g).tolist()
    new[at] = rows
    new[(at + reqs // 2) % reqs] = 1025  # and another one
    table, free, total, pages = _step(cached, new, page, g, extra_rows=reqs % 7)
    got, err = run_tables(cached, new, table, free, page, total, pages)
    assert err == 0
    assert got == [list(x) for x in plain_tables(cached, new, table, free, page, total)]


def test_long_prompt_with_too_few_pages_rows_and_table_columns():
    # rows 0..63 held page 3, then pages 4, 5 of the list; the table's row ends there, the list after one more
    got, err = run_tables([60, 0], [2000, 3], [[3, -5, -5], [-5, -5, -5]], [4, 5], 64, 1500, 100)
    assert err == B.ERR_LENGTHS
    assert got[2] == [[3, 4, 5], [-1, -5, -5]] and got[5] == [2]
    assert got[3] == [60 + i + 1 for i in range(1500)]
    assert got[4] == [3 * 64 + 60 + i for i in range(4)] + [4 * 64 + i for i in range(128)] + [-1] * 1368
    # an entry of the list outside the cache
    got, err = run_tables([0], [640], [[-5] * 10], [1, 2, 3, 4, 5, 6, 777, 7, 8, 9], 64, 640, 100)
    assert err == B.ERR_PAGE_RANGE
    assert got[4][:384] == [64 + i for i in range(384)] and got[4][384:448] == [-1] * 64 and got[4][448:] == [7 * 64 + i for i in range(192)]


def _device_us(cached, new):
    g = torch.Generator().manual_seed(1)
    table, free, rows, pages = _step(cached, new, 64, g)
    t, c, n, f = _i32(table), _i32(cached), _i32(new), _i32(free)
    out = B.fp4idx_build_tables(c, n, t, f, 64, rows)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        for _ in range(20):
            B.fp4idx_build_tables(c, n, t, f, 64, rows, out=out)
    best = float("inf")
    for _ in range(10):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        graph.replay()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) * 1e3 / 20)
    return best


def test_a_long_prompt_is_shared():
    # as many rows spread evenly take 4.3 us, the long prompt 12; written by one warp it took 141
    cached = [37 * i % 4096 for i in range(2048)]
    even = _device_us(cached, [17] * 2048)
    long = _device_us(cached, [1] * 1000 + [32768] + [1] * 1047)
    assert long < 8 * even, f"{long:.1f} us against {even:.1f}"

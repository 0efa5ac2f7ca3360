"""Calls on another stream while the current one still works on blocks that were just freed there."""
import pytest
import torch

from fp4_sparse_attention_gb300 import binding as B
from tests import shared_ref as S

pytestmark = pytest.mark.gpu
MANY = 1310720  # pages: a release and a compaction take scratch


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def busy(*sizes):
    """Blocks of `sizes` int32 entries, freed while the current stream has yet to write them (in about 0.1 s)."""
    blocks = [torch.empty(n, dtype=torch.int32, device="cuda") for n in sizes]
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    for x in blocks:
        x.fill_(-5)


@pytest.mark.parametrize("num_pages", [2000, MANY])
def test_release_and_compaction_beside_freed_blocks(num_pages):
    reqs, width = 30, 40
    g = torch.Generator().manual_seed(num_pages)
    cached = torch.randint(0, width * 64 + 1, (reqs,), generator=g).tolist()
    table = torch.randint(0, num_pages, (reqs, width), generator=g).tolist()
    want = S.release([3, 4], None, cached, table, 64, num_pages)
    moved = S.compact(want[0], table, 64, num_pages, 500)
    d_cached, d_table, gone = i32(cached), i32(table), i32([3, 4])
    to = torch.zeros_like(d_table)
    ws = B.fp4idx_pages_workspace_bytes(num_pages, reqs, width) // 4
    stream = torch.cuda.Stream()
    for _ in range(3):
        busy(num_pages, 1, max(1, ws))
        free, count = B.fp4idx_release_pages(gone, d_cached, d_table, 64, num_pages, stream=stream)
        busy(500, 500, 1, 1, max(1, ws))
        _, src, dst, moves, extent = B.fp4idx_compact_pages(d_cached, d_table, 64, num_pages, 500, out_table=to, stream=stream)
        torch.cuda.synchronize()
        assert free.tolist() == want[1] and count.tolist() == [want[2]]
        assert [src.tolist(), dst.tolist(), int(moves), int(extent)] == list(moved[1:5]) and to.tolist() == moved[0]


def test_fork_and_tables_beside_freed_blocks():
    stream = torch.cuda.Stream()
    table = [[10 * b + j for j in range(6)] for b in range(40)]
    cached = [100 + b for b in range(40)]
    parent, child = [0, 1] * 19, list(range(2, 40))
    free = list(range(400, 500))
    want = S.fork(parent, child, None, cached, table, free, 64, 1000)
    d = [i32(x) for x in (parent, child, cached, table, free)]
    busy(38, 38, 1)
    src, dst, taken = B.fp4idx_fork_requests(*d, 64, num_pages=1000, stream=stream)
    torch.cuda.synchronize()
    assert [src.tolist(), dst.tolist(), int(taken)] == list(want[2:5]) and d[2].tolist() == want[0] and d[3].tolist() == want[1]
    busy(41, 41, 77, 77, 1)
    cu_q, cu_k, visible, slots, taken = B.fp4idx_build_tables(d[2], i32([1] * 37 + [0, 20, 20]), d[3], d[4], 64, 77, stream=stream)
    torch.cuda.synchronize()
    new = [1] * 37 + [0, 20, 20]
    assert cu_q.tolist() == [sum(new[:b]) for b in range(41)]
    assert cu_k.tolist() == [sum(x + y for x, y in zip(want[0][:b], new)) for b in range(41)]
    rows = [(b, want[0][b] + i) for b in range(40) for i in range(new[b])]
    assert visible.tolist() == [n + 1 for _, n in rows]
    assert slots.tolist() == [int(d[3][b, n // 64]) * 64 + n % 64 for b, n in rows]


def test_captured_on_a_stream_of_its_own():
    """The call's stream is one that the capture has forked; scratch and outputs come from the graph's pool."""
    reqs, width = 30, 40
    g = torch.Generator().manual_seed(1)
    cached = torch.randint(0, width * 64 + 1, (reqs,), generator=g).tolist()
    table = torch.randint(0, MANY, (reqs, width), generator=g).tolist()
    d_cached, d_table, gone = i32(cached), i32(table), i32([3])
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        free, count = B.fp4idx_release_pages(gone, d_cached, d_table, 64, MANY, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        listed = free.clone()
    for b in (3, 17):
        gone.copy_(i32([b]))
        d_cached.copy_(i32(cached))
        graph.replay()
        torch.cuda.synchronize()
        want = S.release([b], None, cached, table, 64, MANY)
        assert listed.tolist() == want[1] and count.tolist() == [want[2]] and d_cached.tolist() == want[0]

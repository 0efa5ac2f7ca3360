"""Release and compaction of tables whose row stride is at the limit of 32 bits."""
import pytest
import torch

from fp4_sparse_attention_gb300 import binding as B
from fp4_sparse_attention_gb300 import build

MOST = 2 ** 31 - 1  # of a table's stride


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return B.load_library()


@pytest.mark.parametrize("reqs", [1, 3, 40000])
def test_workspace_of_the_widest_rows(reqs):
    # what does not fit the one launch in shared memory needs the bitmap, as a row of half the width does
    need = B.fp4idx_pages_workspace_bytes(65536, reqs, 2 ** 30)
    assert need > 0
    for stride in (MOST - 255, MOST - 254, MOST - 1, MOST):
        assert B.fp4idx_pages_workspace_bytes(65536, reqs, stride) == need


def test_wider_rows_are_refused():
    at = 1 << 20  # never dereferenced
    args = [at, None, 1, 1, 64, 64, at, at, MOST + 1, at, at, at, 1 << 20, None]
    assert B.load_library().fp4idx_release_pages(*args) == 2


@pytest.mark.gpu
def test_release_and_compaction_of_the_widest_row():
    # one request: its held entries are all that is read of the row (width bounds the compaction's copy)
    P, held = 1000, 300
    g = torch.Generator().manual_seed(1)
    pages = torch.randperm(P, generator=g)[:held].to(torch.int32)
    table, cached = pages.cuda(), torch.tensor([64 * held - 5], dtype=torch.int32, device="cuda")
    need = B.fp4idx_pages_workspace_bytes(P, 1, MOST)
    ws = torch.full((need,), 0xA5, dtype=torch.uint8, device="cuda")
    free, count = torch.full((P,), 5, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    lib, stream = B.load_library(), torch.cuda.current_stream().cuda_stream
    B.fp4idx_get_error(clear=True)
    assert lib.fp4idx_release_pages(None, None, 0, 1, 64, P, cached.data_ptr(), table.data_ptr(), MOST, free.data_ptr(), count.data_ptr(),
                                    ws.data_ptr(), need, stream) == 0
    want = sorted(set(range(P)) - set(pages.tolist()))
    assert free.tolist() == want + [-1] * held and count.tolist() == [P - held]
    src, dst = (torch.full((held,), 5, dtype=torch.int32, device="cuda") for _ in range(2))
    moves, extent = (torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2))
    assert lib.fp4idx_compact_pages(cached.data_ptr(), 1, 64, P, table.data_ptr(), MOST, held, table.data_ptr(), MOST, held, src.data_ptr(),
                                    dst.data_ptr(), moves.data_ptr(), extent.data_ptr(), ws.data_ptr(), need, stream) == 0
    high = sorted((p for p in pages.tolist() if p >= held), reverse=True)
    low = [p for p in range(held) if p not in set(pages.tolist())]
    to = dict(zip(high, low))
    assert table.tolist() == [to.get(p, p) for p in pages.tolist()] and int(moves) == len(high) and int(extent) == held
    assert src.tolist()[:len(high)] == high and dst.tolist()[:len(high)] == low
    assert B.fp4idx_get_error(clear=True) == 0

"""Arguments of the calls for requests that share a prefix that are refused on the host (no GPU needed)."""
import ctypes

import pytest
import torch

from fp4_sparse_attention_gb300 import binding as B
from fp4_sparse_attention_gb300 import build


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return B.load_library()


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def arguments(rows=2, heads=4, kv_heads=2, reqs=2, groups=1):
    cache = torch.zeros((3, kv_heads, 64, 128), dtype=torch.bfloat16)
    return dict(q=torch.zeros((rows, heads, 128), dtype=torch.bfloat16), k=cache, v=cache.clone(), cu_seqlens_q=i32(reqs + 1),
                cu_seqlens_k=i32(reqs + 1), block_table=i32(reqs, 2), max_seqlen_q=1, max_seqlen_k=128, scale=1.0,
                group_offsets=i32(groups + 1), prefix_len=i32(groups), max_group_rows=2)


def status(a, **over):
    """What the C call says of the argument checks (there is no workspace, so it never launches)."""
    x = B.DeviceSharedAttention(**a)
    for name, v in over.items():
        setattr(x.shared if hasattr(x.shared, name) else x.shared.attention, name, v)
    return B.load_library().fp4idx_shared_prefix_attention(x._ref, None, 0, None)


PAST = (3, 4, 5)  # workspace missing, or no GPU: past the argument checks


def test_attention_is_accepted():
    assert status(arguments()) in PAST
    assert status(arguments(groups=3)) in PAST


@pytest.mark.parametrize("over,want", [
    (dict(num_groups=0), 1), (dict(num_groups=-4), 1), (dict(max_group_rows=0), 1), (dict(group_offsets=None), 1), (dict(prefix_len=None), 1),
    (dict(prefix_len=(1 << 20) + 2), 1), (dict(num_groups=(1 << 20) + 1), 2), (dict(max_group_rows=(1 << 20) + 1), 2), (dict(v=None), 2),
    (dict(indices=1 << 20), 1), (dict(num_heads=3), 1), (dict(page_size=32), 2), (dict(scale=float("inf")), 1), (dict(q_row_stride=100), 1),
    (dict(k=(1 << 20) + 8), 1), (dict(max_seqlen_k=1 << 30), 1)])
def test_attention_refuses(over, want):
    assert status(arguments(), **over) == want
    assert B.load_library().fp4idx_last_error_message()


def test_attention_null():
    assert B.load_library().fp4idx_shared_prefix_attention(None, None, 0, None) == 1
    assert B.load_library().fp4idx_shared_attention_workspace_bytes(None) == 0


@pytest.mark.parametrize("name", ["group_offsets", "prefix_len"])
def test_attention_binding_refuses(name):
    a = arguments(groups=3)
    for bad in (a[name].long(), a[name].to("meta"), a[name][None], i32(2 * len(a[name]))[::2], i32(len(a[name]) + 1)):
        with pytest.raises(ValueError):
            B.DeviceSharedAttention(**{**a, name: bad})
    with pytest.raises(ValueError, match="K/V"):
        B.DeviceSharedAttention(**{**a, "v": None})
    with pytest.raises(ValueError, match="K/V"):
        B.DeviceSharedAttention(**a, indices=i32(2, 2, 1))
    with pytest.raises(ValueError, match="CUDA"):
        B.fp4idx_shared_prefix_attention(B.DeviceSharedAttention(**a))
    rest = {k: v for k, v in a.items() if k not in ("group_offsets", "prefix_len", "max_group_rows")}
    with pytest.raises(ValueError, match="DeviceSharedAttention"):
        B.fp4idx_shared_prefix_attention(B.DeviceAttention(**rest))
    with pytest.raises(ValueError, match="DeviceAttention"):  # and the other way round
        B.fp4idx_paged_attention(B.DeviceSharedAttention(**a))


def test_lists_of_the_wrong_kind_are_refused():
    n, t = i32(4), i32(4, 3)
    calls = [lambda n=n, t=t, x=n: B.fp4idx_fork_requests(x, n, n, t, n, 64), lambda n=n, t=t, x=n: B.fp4idx_fork_requests(n, n, n, t, x, 64),
             lambda n=n, t=t, x=n: B.fp4idx_release_pages(x, n, t, 64, 9), lambda n=n, t=t, x=n: B.fp4idx_release_pages(n, x, t, 64, 9),
             lambda n=n, t=t, x=n: B.fp4idx_compact_pages(x, t, 64, 9, 3)]
    for f in calls:
        with pytest.raises(ValueError, match="CUDA"):
            f()
        for bad in (n.long(), i32(8)[::2], n[:, None]):
            with pytest.raises(ValueError):
                f(x=bad)


def test_tables_of_the_wrong_kind_are_refused():
    n = i32(4)
    for table in (i32(3, 3), i32(4, 3).long(), i32(12), i32(3, 4).t(), i32(4, 6)[:, :3], i32(4, 0)):
        for f in (lambda t: B.fp4idx_fork_requests(n, n, n, t, n, 64), lambda t: B.fp4idx_release_pages(n, n, t, 64, 9),
                  lambda t: B.fp4idx_compact_pages(n, t, 64, 9, 3), lambda t: B.fp4idx_compact_pages(n, i32(4, 3), 64, 9, 3, out_table=t)):
            with pytest.raises(ValueError):
                f(table)


def test_pages_of_the_wrong_kind_are_refused():
    x = torch.zeros((4, 64), dtype=torch.uint8)
    for bad in ([], [x[0]], [x, x[:3]], [x[:, ::2]], [x.t()], [x, x.to("meta")], [x[:0]]):
        with pytest.raises(ValueError):
            B.DevicePages(bad)
    with pytest.raises(ValueError, match="CUDA"):
        B.fp4idx_copy_pages(B.DevicePages([x]), i32(2), i32(2))


# ---------------------------------------------------------------- the C calls' own checks
FAKE = 1 << 20  # an aligned address that is never dereferenced


def call(name, defaults, over):
    args = dict(defaults, **over)
    return getattr(B.load_library(), name)(*args.values())


FORK = dict(parent=FAKE, child=FAKE, fork_len=None, num_forks=2, num_reqs=4, page_size=64, num_pages=9, free_pages=FAKE, num_free=3,
            cached_len=FAKE, block_table=FAKE, table_stride=5, copy_src=FAKE, copy_dst=FAKE, pages_taken=FAKE, stream=None)
RELEASE = dict(requests=FAKE, keep_len=None, num_released=2, num_reqs=4, page_size=64, num_pages=9, cached_len=FAKE, block_table=FAKE,
               table_stride=5, free_pages=FAKE, num_free=FAKE, workspace=FAKE, workspace_bytes=1 << 20, stream=None)
COMPACT = dict(cached_len=FAKE, num_reqs=4, page_size=64, num_pages=9, block_table=FAKE, table_stride=5, width=5, new_table=FAKE, new_stride=5,
               max_moves=3, copy_src=FAKE, copy_dst=FAKE, num_moves=FAKE, extent=FAKE, workspace=FAKE, workspace_bytes=1 << 20, stream=None)
POOL = [(dict(num_reqs=0), 1), (dict(num_pages=0), 1), (dict(table_stride=0), 1), (dict(page_size=32), 2), (dict(num_pages=1 << 25), 2),
        (dict(cached_len=None), 1), (dict(block_table=FAKE + 2), 1)]


@pytest.mark.parametrize("over,want", POOL + [
    (dict(num_forks=-1), 1), (dict(num_free=-1), 1), (dict(parent=None), 1), (dict(child=FAKE + 1), 1), (dict(copy_src=None), 1),
    (dict(copy_dst=None), 1), (dict(pages_taken=None), 1), (dict(free_pages=None), 1), (dict(fork_len=FAKE + 2), 1)])
def test_fork_refuses(over, want):
    assert call("fp4idx_fork_requests", FORK, over) == want


@pytest.mark.parametrize("over,want", POOL + [
    (dict(num_released=-1), 1), (dict(requests=None), 1), (dict(keep_len=FAKE + 2), 1), (dict(free_pages=None), 1), (dict(num_free=None), 1),
    (dict(workspace=None, num_reqs=40000), 3), (dict(workspace_bytes=31, num_reqs=40000), 3), (dict(workspace=FAKE + 8, num_reqs=40000), 1)])
def test_release_refuses(over, want):
    assert call("fp4idx_release_pages", RELEASE, over) == want


@pytest.mark.parametrize("over,want", POOL + [
    (dict(width=0), 1), (dict(width=6), 1), (dict(new_stride=4), 1), (dict(new_stride=6), 1), (dict(max_moves=-1), 1), (dict(new_table=None), 1),
    (dict(copy_src=None), 1), (dict(num_moves=None), 1), (dict(extent=FAKE + 2), 1), (dict(workspace_bytes=31, num_reqs=40000), 3)])
def test_compact_refuses(over, want):
    assert call("fp4idx_compact_pages", COMPACT, over) == want


def test_copy_refuses():
    f = B.load_library().fp4idx_copy_pages

    def copy(n=1, pages=9, copies=2, src=FAKE, dst=FAKE, count=None, **over):
        spans = (B.CPageSpan * max(1, n))()
        for s in spans:
            s.base, s.page_stride, s.page_bytes = FAKE, 64, 64
        for name, v in over.items():
            setattr(spans[0], name, v)
        return f(spans, n, pages, src, dst, copies, count, None)

    for over, want in [(dict(n=0), 1), (dict(n=257), 2), (dict(pages=0), 1), (dict(pages=1 << 31), 2), (dict(copies=-1), 1), (dict(src=None), 1),
                       (dict(dst=FAKE + 2), 1), (dict(count=FAKE + 2), 1), (dict(base=None), 1), (dict(base=FAKE + 8), 1), (dict(page_bytes=0), 1),
                       (dict(page_bytes=40), 1), (dict(page_stride=48), 1), (dict(page_stride=72), 1),
                       (dict(page_bytes=1 << 33, page_stride=1 << 33), 2)]:
        assert copy(**over) == want, over
    assert f(None, 1, 9, FAKE, FAKE, 1, None, None) == 1
    assert copy(copies=0, src=None, dst=None) == 0


def test_workspace_sizes():
    f = B.fp4idx_pages_workspace_bytes
    assert f(0, 1, 1) == f(-5, 1, 1) == f(1 << 31, 1, 1) == f(9, 0, 1) == f(9, 1, 0) == 0
    assert f(10000, 64, 300) == 0  # one launch in shared memory
    for n in (1, 31, 32, 1000, 10 ** 6, 1 << 24):  # a bit a page and a rank for 128 of them
        assert n // 8 + n // 32 <= f(n, 40000, 9) <= f(n + 1, 40000, 9) and f(n, 40000, 9) % 16 == 0
        assert f(n, 40000, 9) == f(n, 200, 10 ** 6)


def test_struct_sizes():
    # the mirrors are as large as the C structs (checked by the compiler's layout rules: all fields naturally aligned)
    assert ctypes.sizeof(B.CSharedAttention) == ctypes.sizeof(B.CAttention) + 24
    assert ctypes.sizeof(B.CPageSpan) == 24

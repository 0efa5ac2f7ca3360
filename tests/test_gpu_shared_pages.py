"""Fork, page copies, release and compaction on the GPU against plain Python: whole numbers, all of them equal."""
import random

import pytest
import torch

from fp4_sparse_attention_gb300 import binding as B
from tests import shared_ref as S

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def pool(rng, reqs, stride, page, num_pages, longest):
    """Lengths and a table whose entries may be held by several requests."""
    cached = [rng.choice([0, 1, page - 1, page, page + 1, rng.randint(0, longest), rng.randint(0, longest)]) for _ in range(reqs)]
    cached = [min(n, longest) for n in cached]
    table = [[rng.randrange(num_pages) for _ in range(stride)] for _ in range(reqs)]
    for b in range(1, reqs):
        if rng.random() < 0.5:
            n = rng.randint(0, stride)
            table[b][:n] = table[rng.randrange(b)][:n]
    return cached, table


# ---------------------------------------------------------------- fork
def check_fork(parent, child, fork_len, cached, table, free, page, num_pages):
    want = S.fork(parent, child, fork_len, cached, table, free, page, num_pages)
    d_cached, d_table = i32(cached), i32(table)
    B.fp4idx_get_error(clear=True)
    for _ in range(2):  # a second call on the results gives them again
        out = [torch.full((max(1, len(parent)),), -9, dtype=torch.int32, device="cuda")[:len(parent)] for _ in range(2)]
        src, dst, taken = B.fp4idx_fork_requests(i32(parent).view(-1), i32(child).view(-1), d_cached, d_table, i32(free).view(-1), page,
                                                 fork_len=None if fork_len is None else i32(fork_len).view(-1), num_pages=num_pages,
                                                 out=out + [i32([7])])
        assert d_cached.tolist() == want[0] and d_table.tolist() == want[1]
        assert src.tolist() == want[2] and dst.tolist() == want[3] and taken.tolist() == [want[4]]
        assert B.fp4idx_get_error(clear=True) == want[5]
    return want


@pytest.mark.parametrize("seed", range(12))
def test_forks(seed):
    rng = random.Random(seed)
    page, stride = rng.choice([64, 128]), rng.choice([1, 5, 33, 200])
    reqs = rng.choice([2, 9, 40, 700])
    cached, table = pool(rng, reqs, stride, page, 5000, stride * page)
    rows = list(range(reqs))
    rng.shuffle(rows)
    n = rng.randint(1, max(1, reqs // 3))
    child = rows[n:n + rng.randint(1, reqs - n)]
    parent = [rows[rng.randrange(n)] for _ in child]
    fork_len = [rng.randint(-2, stride * page + 5) for _ in child] if seed % 2 else None
    want = check_fork(parent, child, fork_len, cached, table, [9000 + i for i in range(len(child))], page, 20000)
    assert want[5] == 0


@pytest.mark.parametrize("length", [0, 1, 63, 64, 65, 128, 129, 640])
@pytest.mark.parametrize("page", [64, 128])
def test_fork_at_page_ends(length, page):
    check_fork([1, 1, 1], [0, 2, 4], None, [5, length, 9, 7, 300], [[10 * b + j for j in range(10)] for b in range(5)], [900, 901, 902], page, 1000)


def test_forks_that_are_refused_and_padding():
    cached, table = [100, 200, 0, 0, 64, 0, 50, 0], [[10 * b + j for j in range(5)] for b in range(8)]
    # padding, a child twice, a child that is a parent, itself, numbers past the table, the smallest and largest numbers
    parent = [0, -1, 0, 1, 0, 6, 8, 0, 2 ** 31 - 1, -2 ** 31, 1, 4]
    child = [2, 3, 2, 0, 5, 6, 3, 8, 3, 3, -5, 7]
    want = check_fork(parent, child, None, cached, table, [70, 71, 72, 73, 74, 75, 76], 64, 100)
    assert want[5] == S.ERR_REQUESTS and want[2][0] == 1 and want[2][2] == -1 and want[2][4] == 1 and want[0][5] == 100


def test_fork_without_pages_or_room():
    table = [[10 * b + j for j in range(3)] for b in range(6)]
    assert check_fork([0, 0, 0], [1, 2, 3], None, [100] * 6, table, [70], 64, 100)[5] == S.ERR_LENGTHS   # one page for three
    assert check_fork([0], [1], None, [100] * 6, table, [], 64, 100)[5] == S.ERR_LENGTHS
    assert check_fork([0, 2], [1, 3], None, [193, 0, 65, 7, 7, 7], table, [70, 71], 64, 100)[5] == S.ERR_LENGTHS  # longer than its row
    assert check_fork([0, 2], [1, 3], None, [2 ** 31 - 1, 0, -5, 7, 7, 7], table, [70, 71], 64, 100)[5] == S.ERR_LENGTHS
    table[0][1] = 10 ** 6
    assert check_fork([0, 0], [1, 2], [100, 128], [130] * 6, table, [70, 71], 64, 100)[5] == S.ERR_PAGE_RANGE
    table[0][1] = -1
    assert check_fork([0, 0], [1, 2], [100, 128], [130] * 6, table, [70, 71], 64, 100)[5] == S.ERR_PAGE_RANGE


def test_forks_from_a_list_that_release_ended_with_negative_entries():
    table = [[10 * b + j for j in range(3)] for b in range(6)]
    want = check_fork([0, 0, 0, 0], [1, 2, 3, 4], None, [100] * 6, table, [70, -1, -7, -2 ** 31], 64, 100)
    assert want[5] == S.ERR_LENGTHS and want[3] == [70, -1, -1, -1] and [want[1][b][1] for b in (1, 2, 3, 4)] == [70, -1, -1, -1]


def test_no_forks():
    check_fork([], [], None, [3, 4], [[1], [2]], [5], 64, 10)


# ---------------------------------------------------------------- copy
@pytest.mark.parametrize("n", [0, 1, 5, 300])
@pytest.mark.parametrize("counted", [False, True])
def test_copies(n, counted):
    g = torch.Generator().manual_seed(n)
    P = 2 * n + 3
    latent = torch.randn((P, 2, 64, 576), generator=g).bfloat16().cuda()       # two layers; the second is copied
    k = torch.randn((P, 3, 64, 128), generator=g).half().cuda()
    fused = torch.randint(0, 256, (P, 1, 64 * 68), generator=g, dtype=torch.uint8).cuda()
    scale = torch.randint(0, 256, (P, 1, 64, 4), generator=g, dtype=torch.uint8).cuda()
    wide = torch.randint(0, 256, (P, 4096 + 48), generator=g, dtype=torch.uint8).cuda()  # a stride with a gap
    k.view(torch.int16)[0, 0, 0, :3] = torch.tensor([0x7e01, -1, 0x7c00], dtype=torch.int16)  # any bits are copied
    caches = [latent[:, 1], k, fused, scale, wide[:, :4096]]
    perm = torch.randperm(P, generator=g).to(torch.int32)
    src, dst = perm[:n].clone(), perm[n:2 * n].clone()
    if n > 4:
        src[1], dst[2], src[3] = -1, -7, -2 ** 31                               # no copies
    count = max(0, n - 2) if counted else n
    whole = [latent, k, fused, scale, wide]
    want = [x.clone() for x in whole]
    for w, part in zip(want, (lambda x: x[:, 1], lambda x: x, lambda x: x, lambda x: x, lambda x: x[:, :4096])):
        for i in range(count):
            if src[i] >= 0 and dst[i] >= 0:
                part(w)[int(dst[i])] = part(w)[int(src[i])].clone()
    B.fp4idx_get_error(clear=True)
    B.fp4idx_copy_pages(B.DevicePages(caches), src.cuda(), dst.cuda(), count=i32([count]) if counted else None)
    assert B.fp4idx_get_error(clear=True) == 0
    for x, w in zip(whole, want):
        assert torch.equal(x.view(torch.uint8), w.view(torch.uint8))


@pytest.mark.parametrize("size", [16, 32, 240, 496, 512, 528, 4080, 4096, 4112, 8192 + 16, 73728])
def test_pages_of_every_size(size):
    x = torch.randint(0, 256, (9, size), dtype=torch.uint8, device="cuda")
    want = x.clone()
    want[[4, 0]] = want[[8, 3]]
    B.fp4idx_copy_pages(B.DevicePages([x]), i32([8, 3]), i32([4, 0]))
    assert torch.equal(x, want)


def test_copies_outside_the_cache_and_counts_past_the_list():
    x = torch.randint(0, 256, (6, 64), dtype=torch.uint8, device="cuda")
    want = x.clone()
    want[1] = want[5]
    B.fp4idx_get_error(clear=True)
    B.fp4idx_copy_pages(B.DevicePages([x]), i32([6, 0, 5, 2 ** 31 - 1]), i32([0, 6, 1, 2 ** 31 - 1]), count=i32([2 ** 31 - 1]))
    assert B.fp4idx_get_error(clear=True) == B.ERR_PAGE_RANGE
    B.fp4idx_copy_pages(B.DevicePages([x]), i32([3]), i32([4]), count=i32([-5]))
    assert B.fp4idx_get_error(clear=True) == 0 and torch.equal(x, want)


def test_many_caches():
    xs = [torch.randint(0, 256, (4, 16 * (1 + i % 5)), dtype=torch.uint8, device="cuda") for i in range(256)]
    want = [x.clone() for x in xs]
    for w in want:
        w[0] = w[3]
    B.fp4idx_copy_pages(B.DevicePages(xs), i32([3]), i32([0]))
    assert all(torch.equal(x, w) for x, w in zip(xs, want))
    with pytest.raises(B.Fp4idxError):
        B.fp4idx_copy_pages(B.DevicePages(xs + xs[:1]), i32([3]), i32([0]))


def test_copies_beyond_two_to_the_31_bytes():
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB")
    x = torch.empty((70000, 64 * 576), dtype=torch.bfloat16, device="cuda")  # 2.6e9 elements
    x[69999], x[3] = torch.randn((64 * 576,), device="cuda").bfloat16(), 1.0
    x[60001] = 2.0
    B.fp4idx_copy_pages(B.DevicePages([x]), i32([69999, 60001]), i32([3, 59999]))
    assert torch.equal(x[3], x[69999]) and bool((x[59999] == 2.0).all())


# ---------------------------------------------------------------- release
def check_release(requests, keep, cached, table, page, num_pages):
    want = S.release(requests, keep, cached, table, page, num_pages)
    d_cached, d_table = i32(cached), i32(table)
    ws = torch.full((B.fp4idx_pages_workspace_bytes(num_pages, len(cached), len(table[0])),), 0xA5, dtype=torch.uint8, device="cuda")
    B.fp4idx_get_error(clear=True)
    for _ in range(2):
        free, count = B.fp4idx_release_pages(i32(requests).view(-1) if requests is not None else None, d_cached, d_table, page, num_pages,
                                             keep_len=None if keep is None else i32(keep).view(-1), workspace=ws,
                                             out=[torch.full((num_pages,), 5, dtype=torch.int32, device="cuda"), i32([-3])])
        assert d_cached.tolist() == want[0] and d_table.tolist() == [list(r) for r in table]
        assert count.tolist() == [want[2]] and free.tolist() == want[1]
        assert B.fp4idx_get_error(clear=True) == want[3]
    return want


@pytest.mark.parametrize("seed", range(12))
def test_releases(seed):
    rng = random.Random(100 + seed)
    page, stride = rng.choice([64, 128]), rng.choice([1, 7, 128, 129, 300])
    reqs, num_pages = rng.choice([1, 9, 40, 500]), rng.choice([1, 31, 32, 33, 1000, 8191, 40000])
    cached, table = pool(rng, reqs, stride, page, num_pages, stride * page)
    gone = [rng.randrange(-1, reqs) for _ in range(rng.randint(0, reqs))]  # some twice, some none
    keep = [rng.randint(-3, stride * page) for _ in gone] if seed % 2 else None
    assert check_release(gone, keep, cached, table, page, num_pages)[3] == 0


@pytest.mark.parametrize("num_pages", [1, 32, 64, 65, 300000])
def test_all_pages_free_and_all_in_use(num_pages):
    check_release([0, 1], None, [64, 64], [[0], [0]], 64, num_pages)
    stride = -(-num_pages // 2)
    table = [[j for j in range(stride)], [min(num_pages - 1, stride + j) for j in range(stride)]]
    want = check_release([], None, [stride * 64] * 2, table, 64, num_pages)
    assert want[2] == 0


def test_releases_of_broken_tables():
    table = [[3, 10 ** 6, 5], [1, -1, 2], [4, 4, 4]]
    assert check_release([3, -8, 2 ** 31 - 1], [0, 0, 0], [192, 64, 100], table, 64, 9)[3] == S.ERR_REQUESTS | S.ERR_PAGE_RANGE
    assert check_release([2], [2 ** 31 - 1], [64, 64, 2 ** 31 - 1], table, 64, 9)[3] == S.ERR_LENGTHS
    assert check_release([2], [-1], [64, -7, 100], table, 64, 9)[3] == 0


# ---------------------------------------------------------------- compaction
def check_compact(cached, table, page, num_pages, max_moves, in_place=False):
    want = S.compact(cached, table, page, num_pages, max_moves)
    d_cached, d_table = i32(cached), i32(table)
    width = d_table.shape[1]
    ws = torch.full((B.fp4idx_pages_workspace_bytes(num_pages, len(cached), len(table[0])),), 0xA5, dtype=torch.uint8, device="cuda")
    out = [torch.full((max_moves,), 5, dtype=torch.int32, device="cuda") for _ in range(2)] + [i32([-3]), i32([-3])]
    to = None if in_place else torch.full((len(cached), width + 2), -77, dtype=torch.int32, device="cuda")
    B.fp4idx_get_error(clear=True)
    for _ in range(1 if in_place else 2):
        new, src, dst, moves, extent = B.fp4idx_compact_pages(d_cached, d_table, page, num_pages, max_moves, out_table=to, out=out, workspace=ws)
        assert new[:, :width].tolist() == want[0] and src.tolist() == want[1] and dst.tolist() == want[2]
        assert moves.tolist() == [want[3]] and extent.tolist() == [want[4]]
        assert B.fp4idx_get_error(clear=True) == want[5]
        if in_place:
            assert new.data_ptr() == d_table.data_ptr()
        else:
            assert bool((new[:, width:] == -77).all()) and d_table.tolist() == [list(r) for r in table]
    return want


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("seed", range(12))
def test_compactions(seed, in_place):
    rng = random.Random(200 + seed)
    page, stride = rng.choice([64, 128]), rng.choice([1, 7, 128, 129, 300])
    reqs, num_pages = rng.choice([1, 9, 40, 300]), rng.choice([1, 31, 32, 33, 1000, 8191, 40000])
    cached, table = pool(rng, reqs, stride, page, num_pages, stride * page)
    most = rng.choice([0, 1, 100, 50000])
    want = check_compact(cached, table, page, num_pages, most, in_place)
    assert want[5] == 0
    if want[3] < most:  # everything moved: what is in use fills the pool's start
        live, _ = S.in_use(cached, want[0], page, num_pages)
        assert live == set(range(len(live))) and want[4] == len(live)


def test_compaction_in_steps_ends_where_one_does():
    rng = random.Random(5)
    cached, table = pool(rng, 20, 30, 64, 3000, 30 * 64)
    d_cached, d_table = i32(cached), i32(table)
    content = torch.arange(3000, dtype=torch.int32, device="cuda")[:, None].repeat(1, 4)  # a page's "values"
    pages = B.DevicePages([content])
    held = torch.arange(30, device="cuda")[None, :] < ((d_cached + 63) // 64)[:, None]
    for step in range(100):
        _, src, dst, moves, extent = B.fp4idx_compact_pages(d_cached, d_table, 64, 3000, 17)
        B.fp4idx_copy_pages(pages, src, dst, count=moves)
        assert torch.equal(content[d_table.long(), 0][held], i32(table)[held])  # every entry still finds its values
        if int(moves) < 17:
            break
    live, _ = S.in_use(cached, table, 64, 3000)
    assert int(extent) == len(live) and step == (S.compact(cached, table, 64, 3000, 3000)[3]) // 17


def test_compactions_of_broken_tables():
    table = [[3, 10 ** 6, 5], [1, -1, 2], [8, 8, 4]]
    assert check_compact([192, 64, 100], table, 64, 9, 10)[5] == S.ERR_PAGE_RANGE
    assert check_compact([64, 64, 2 ** 31 - 1], table, 64, 9, 10)[5] == S.ERR_LENGTHS
    assert check_compact([0, -7, 0], table, 64, 9, 10)[4] == 0


# ---------------------------------------------------------------- pools and tables past the one-launch kernel
MANY = 1310720  # pages: more than it takes


def many_requests(reqs, num_pages, longest, seed):
    """Lengths and tables of many short requests (a list for the plain form)."""
    g = torch.Generator().manual_seed(seed)
    cached = torch.randint(0, longest * 64 + 1, (reqs,), generator=g).tolist()
    return cached, torch.randint(0, num_pages, (reqs, longest), generator=g).tolist()


@pytest.mark.parametrize("reqs,num_pages", [(50, 150000), (50, MANY), (50, 3000000), (32768, 90000), (40000, 200000), (3, 250000)])
def test_large_pools_and_many_requests(reqs, num_pages):
    cached, table = many_requests(reqs, num_pages, 5 if reqs > 1000 else 1500 if reqs > 3 else 3000, reqs)
    gone = [(7 * i) % (reqs + 1) - 1 for i in range(0, reqs, 3)]  # with -1, none twice
    check_release(gone, [i % 90 for i in range(len(gone))], cached, table, 64, num_pages)
    for moves in (1000, num_pages // 2):
        want = check_compact(cached, table, 64, num_pages, moves)
    assert want[4] == len(S.in_use(cached, table, 64, num_pages)[0])


@pytest.mark.parametrize("num_pages", [65, 96, 127, 131, 131200, 131201, 131209, 160031])
@pytest.mark.parametrize("free", [0, 1, 33])
def test_compaction_of_pools_that_are_almost_full(num_pages, free):
    # every page but `free` of them, which lie at the pool's start, middle and end
    holes = {x for i in range(free) for x in [(0, num_pages // 2, num_pages - 1)[i % 3] + (i // 3 if i % 3 < 2 else -(i // 3))]}
    pages = [x for x in range(num_pages) if x not in holes]
    width = -(-len(pages) // 3)
    table = [pages[i * width:(i + 1) * width] for i in range(3)]
    cached = [64 * len(r) for r in table]
    table = [r + [7] * (width - len(r)) for r in table]
    want = check_compact(cached, table, 64, num_pages, 50)
    assert want[4] == num_pages - len(holes) and (free > 0 or want[3] == 0)
    assert check_release([], None, cached, table, 64, num_pages)[2] == len(holes)


def test_workspace_is_the_callers_or_made_for_the_call():
    cached, table = many_requests(20, MANY + 100, 50, 3)
    want = S.release([1], None, cached, table, 64, MANY + 100)
    stream = torch.cuda.Stream()
    d_cached, d_table, one = i32(cached), i32(table), i32([1])
    torch.cuda.synchronize()
    for s in (None, stream):
        free, count = B.fp4idx_release_pages(one, d_cached, d_table, 64, MANY + 100, stream=s)
        torch.cuda.synchronize()
        assert free.tolist() == want[1] and count.tolist() == [want[2]]
    short = torch.empty(B.fp4idx_pages_workspace_bytes(MANY + 100, 20, 50) - 1, dtype=torch.uint8, device="cuda")
    for f in (lambda: B.fp4idx_release_pages(one, d_cached, d_table, 64, MANY + 100, workspace=short),
              lambda: B.fp4idx_compact_pages(d_cached, d_table, 64, MANY + 100, 5, workspace=short)):
        with pytest.raises(B.Fp4idxError) as e:
            f()
        assert e.value.status == 3


# ---------------------------------------------------------------- streams and graphs
def test_graph_replays_see_new_lengths_and_another_stream():
    rng = random.Random(9)
    cached, table = pool(rng, 30, 40, 64, 2000, 40 * 64)
    d_cached, d_table = i32(cached), i32(table)
    gone, keep = i32([3, 4, 5]), i32([0, 10, 20])
    moved = torch.empty_like(d_table)
    free = [torch.empty((2000,), dtype=torch.int32, device="cuda"), i32([0])]
    moves = [i32([0] * 64), i32([0] * 64), i32([0]), i32([0])]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())

    def step(s=None):
        B.fp4idx_release_pages(gone, d_cached, d_table, 64, 2000, keep_len=keep, out=free, stream=s)
        B.fp4idx_compact_pages(d_cached, d_table, 64, 2000, 64, out_table=moved, out=moves, stream=s)

    def right(lens):
        want = S.release(gone.tolist(), keep.tolist(), lens, table, 64, 2000)
        assert d_cached.tolist() == want[0] and free[0].tolist() == want[1] and free[1].tolist() == [want[2]]
        got = S.compact(want[0], table, 64, 2000, 64)
        assert moved.tolist() == got[0] and moves[0].tolist() == got[1] and moves[1].tolist() == got[2]

    step(stream)
    stream.synchronize()
    right(cached)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n in (2560, 700, 0):
        lens = [min(n, x) for x in cached]
        d_cached.copy_(i32(lens))
        gone.copy_(i32([n % 30, 1, 1]))
        graph.replay()
        torch.cuda.synchronize()
        right(lens)

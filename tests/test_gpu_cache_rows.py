"""GPU writers of the 16-bit caches and the step tables, against plain Python."""
import pytest
import torch

from fp4_sparse_attention_gb300 import binding as B

pytestmark = pytest.mark.gpu


def _slots(n, capacity, g, skip):
    s = torch.randperm(capacity, generator=g)[:n].to(torch.int32)
    if skip:
        s[torch.rand(n, generator=g) < 0.2] = -1
        s[0] = -2 ** 31
    return s


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n,page", [(1, 64), (63, 64), (1000, 128)])
def test_store_latent(n, page, dtype):
    g = torch.Generator().manual_seed(n)
    P = n // page + 3
    src = torch.randn((n, 600), generator=g).to(dtype)
    cache = torch.randn((P, 2, page, 576), generator=g).to(dtype)  # two layers; the second is written
    slots = _slots(n, P * page, g, n > 1)
    want = cache.clone()
    for i, s in enumerate(slots.tolist()):
        if s >= 0:
            want[s // page, 1, s % page] = torch.cat([src[i, :512], src[i, 520:584]])
    d, dc = src.cuda(), cache.cuda()
    B.fp4idx_get_error(clear=True)
    B.fp4idx_store_latent(d[:, :512], d[:, 520:584], slots.cuda(), dc[:, 1])
    assert B.fp4idx_get_error(clear=True) == 0
    assert torch.equal(dc.cpu().view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("n,heads,page", [(1, 1, 64), (77, 4, 128), (1000, 3, 64)])
def test_store_kv(n, heads, page):
    g = torch.Generator().manual_seed(n + heads)
    P = n // page + 3
    kv = torch.randn((n, 2, heads, 128), generator=g).half()
    kv[0, 0, 0, :4] = torch.tensor([float("nan"), float("inf"), -0.0, 6e-8]).half()  # any bits are copied
    k, v = torch.randn((2, P, heads, page, 128), generator=g).half()
    slots = _slots(n, P * page, g, n > 1)
    wk, wv = k.clone(), v.clone()
    for i, s in enumerate(slots.tolist()):
        if s >= 0:
            wk[s // page, :, s % page], wv[s // page, :, s % page] = kv[i, 0], kv[i, 1]
    d, dk, dv = kv.cuda(), k.cuda(), v.cuda()
    B.fp4idx_get_error(clear=True)
    B.fp4idx_store_kv(d[:, 0], d[:, 1], slots.cuda(), dk, dv)
    assert B.fp4idx_get_error(clear=True) == 0
    assert torch.equal(dk.cpu().view(torch.int16), wk.view(torch.int16))
    assert torch.equal(dv.cpu().view(torch.int16), wv.view(torch.int16))


def test_no_tokens():
    cache = torch.zeros((2, 64, 576), dtype=torch.bfloat16, device="cuda")
    x = torch.ones((0, 576), dtype=torch.bfloat16, device="cuda")
    n = torch.zeros((0,), dtype=torch.int32, device="cuda")
    B.fp4idx_store_latent(x[:, :512], x[:, 512:], n, cache)
    kv = torch.zeros((2, 2, 3, 64, 128), dtype=torch.bfloat16, device="cuda")
    e = torch.zeros((0, 3, 128), dtype=torch.bfloat16, device="cuda")
    B.fp4idx_store_kv(e, e, n, kv[0], kv[1])
    assert B.fp4idx_get_error(clear=True) == 0 and not cache.any()


def test_slots_past_the_cache_are_skipped_and_reported():
    cache = torch.zeros((2, 64, 576), dtype=torch.bfloat16, device="cuda")
    x = torch.ones((4, 576), dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([128, 3, 2 ** 31 - 1, 127], dtype=torch.int32, device="cuda")
    B.fp4idx_get_error(clear=True)
    B.fp4idx_store_latent(x[:, :512], x[:, 512:], slots, cache)
    assert B.fp4idx_get_error(clear=True) == B.ERR_PAGE_RANGE
    rows = cache.view(128, 576)
    assert rows[3].eq(1).all() and rows[127].eq(1).all() and float(rows.float().sum()) == 2 * 576


# ---------------------------------------------------------------- step tables
def plain_tables(cached, new, table, free, page, rows):
    table = [r[:] for r in table]
    cu_q, cu_k, visible, slots, used = [0], [0], [], [], 0
    for b, (c, n) in enumerate(zip(cached, new)):
        has, need = -(-c // page), -(-(c + n) // page)
        for j in range(has, need):
            table[b][j] = free[used]
            used += 1
        for pos in range(c, c + n):
            visible.append(pos + 1)
            slots.append(table[b][pos // page] * page + pos % page)
        cu_q.append(cu_q[-1] + n)
        cu_k.append(cu_k[-1] + c + n)
    visible += [0] * (rows - len(visible))
    slots += [-1] * (rows - len(slots))
    return cu_q, cu_k, table, visible, slots, [used]


def _step(cached, new, page, g, extra_rows=0, spare=3):
    width = max(-(-(c + n) // page) for c, n in zip(cached, new)) + 1
    total = len(cached) * width
    perm = torch.randperm(total, generator=g).tolist()
    table, at = [], 0
    for c in cached:
        h = -(-c // page)
        table.append(perm[at:at + h] + [-1] * (width - h))
        at += h
    need = sum(-(-(c + n) // page) - -(-c // page) for c, n in zip(cached, new))
    return table, perm[at:at + need + spare], sum(new) + extra_rows, total


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def run_tables(cached, new, table, free, page, rows, pages):
    t = _i32(table)
    B.fp4idx_get_error(clear=True)
    cu_q, cu_k, visible, slots, taken = B.fp4idx_build_tables(_i32(cached), _i32(new), t, _i32(free), page, rows, num_pages=pages)
    return [x.tolist() for x in (cu_q, cu_k, t, visible, slots, taken)], B.fp4idx_get_error(clear=True)


@pytest.mark.parametrize("page", [64, 128])
@pytest.mark.parametrize("reqs,new_hi,cached_hi", [(1, 1, 0), (1, 1, 64), (1, 5000, 1), (7, 3, 200), (33, 300, 1000),
                                                   (64, 1, 5000), (700, 9, 300), (6000, 2, 100)])
def test_tables_match_plain(reqs, new_hi, cached_hi, page):
    g = torch.Generator().manual_seed(reqs + new_hi)
    cached = torch.randint(0, cached_hi + 1, (reqs,), generator=g).tolist()
    new = torch.randint(0, new_hi + 1, (reqs,), generator=g).tolist()
    new[-1] = new_hi
    table, free, rows, pages = _step(cached, new, page, g, extra_rows=reqs % 5)
    got, err = run_tables(cached, new, table, free, page, rows, pages)
    assert err == 0
    assert got == [list(x) for x in plain_tables(cached, new, table, free, page, rows)]


@pytest.mark.parametrize("held", [0, 1, 63, 64, 65, 127, 128, 129])
@pytest.mark.parametrize("fresh", [0, 1, 64, 65])
def test_tables_at_page_edges(held, fresh):
    g = torch.Generator().manual_seed(held * 100 + fresh)
    table, free, rows, pages = _step([held, 5], [fresh, 2], 64, g)
    got, err = run_tables([held, 5], [fresh, 2], table, free, 64, rows, pages)
    assert err == 0
    assert got == [list(x) for x in plain_tables([held, 5], [fresh, 2], table, free, 64, rows)]


def test_one_long_prompt_among_many():
    g = torch.Generator().manual_seed(5)
    cached, new = [100] * 50, [1] * 50
    new[20] = 40000
    table, free, rows, pages = _step(cached, new, 128, g)
    got, err = run_tables(cached, new, table, free, 128, rows, pages)
    assert err == 0
    assert got == [list(x) for x in plain_tables(cached, new, table, free, 128, rows)]


def test_too_few_free_pages():
    got, err = run_tables([64, 10], [100, 60], [[0, -5, -5, -5], [1, -5, -5, -5]], [7, 8], 64, 160, 100)
    assert err == B.ERR_LENGTHS
    assert got[2] == [[0, 7, 8, -5], [1, -1, -5, -5]]
    assert got[5] == [2]
    assert got[4][:100] == [7 * 64 + i for i in range(64)] + [8 * 64 + i for i in range(36)]
    assert got[4][100:154] == [64 + 10 + i for i in range(54)] and got[4][154:] == [-1] * 6


def test_request_longer_than_its_table_row():
    got, err = run_tables([60], [100], [[3, -5]], [4, 5], 64, 100, 100)
    assert err == B.ERR_LENGTHS
    assert got[2] == [[3, 4]]
    assert got[4] == [3 * 64 + 60 + i for i in range(4)] + [4 * 64 + i for i in range(64)] + [-1] * 32


def test_negative_lengths_and_too_few_rows():
    got, err = run_tables([-4, 3], [2, -1], [[-5], [2]], [6], 64, 2, 100)
    assert err == B.ERR_LENGTHS
    assert got[0] == [0, 2, 2] and got[1] == [0, 2, 5] and got[4] == [6 * 64, 6 * 64 + 1]
    got, err = run_tables([3, 3], [4, 4], [[0], [1]], [], 64, 6, 100)
    assert err == B.ERR_LENGTHS
    assert got[0] == [0, 4, 8] and got[4] == [3, 4, 5, 6, 64 + 3, 64 + 4]


def test_page_ids_outside_the_cache():
    got, err = run_tables([3, 64], [1, 1], [[100, -5], [0, -5]], [200], 64, 2, 100)
    assert err == B.ERR_PAGE_RANGE
    assert got[4] == [-1, -1]


def test_tables_repeat_and_graph():
    g = torch.Generator().manual_seed(9)
    cached, new = [100, 0, 64, 500], [3, 70, 1, 0]
    table, free, rows, pages = _step(cached, new, 64, g)
    want = [list(x) for x in plain_tables(cached, new, table, free, 64, rows)]
    t, c, n, f = _i32(table), _i32(cached), _i32(new), _i32(free)
    out = B.fp4idx_build_tables(c, n, t, f, 64, rows)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        B.fp4idx_build_tables(c, n, t, f, 64, rows, out=out)
    t.copy_(_i32(table))
    for x in out:
        x.fill_(-9)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        cu_q, cu_k, visible, slots, taken = out
        assert [x.tolist() for x in (cu_q, cu_k, t, visible, slots, taken)] == want

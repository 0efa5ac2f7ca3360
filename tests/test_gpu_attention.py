"""GPU attention over the paged caches (fp4idx_latent_attention, fp4idx_paged_attention)
against the plain 64-bit implementation, at the lengths, head layouts, masks and strides where
tiling can go wrong.  The tolerances are the bounds derived in tests/attention_ref.py."""
import math

import pytest
import torch

from fp4_sparse_attention_gb300 import binding as B
from tests import attention_ref as R

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16


def build(c, **over):
    dev = c["q"].device
    a = dict(q=c["q"], k=c["k"], v=c["v"], cu_seqlens_q=R.offsets(c["q_lens"], dev), cu_seqlens_k=R.offsets(c["k_lens"], dev),
             block_table=R.table_of(c), max_seqlen_q=max(c["q_lens"] + [1]), max_seqlen_k=max(c["k_lens"] + [0]),
             scale=c["scale"], visible_len=c.get("visible_len"), causal=c.get("causal", False), qo_offset=c.get("qo_offset"),
             indices=c.get("indices"))
    a.update(over)
    return B.DeviceAttention(**a)


def call(a, stream=None):
    return (B.fp4idx_latent_attention if a.v is None else B.fp4idx_paged_attention)(a, stream=stream)


def check(c, got, what=""):
    out, lse = got
    want, want_lse, b_out, b_lse = R.reference(c)
    off = (out.double() - want).abs()
    assert torch.isfinite(out).all(), what
    assert bool((off <= b_out).all()), f"{what}: out off by {float((off - b_out).max()):.3g} over the bound"
    none = want_lse == -math.inf
    assert torch.equal(lse == -math.inf, none), what
    off = (lse.double() - want_lse).abs()[~none]
    assert bool((off <= b_lse[~none]).all()), f"{what}: lse"


def run_case(*args, **kw):
    c = R.make_case(*args, device="cuda", **kw)
    B.fp4idx_get_error(clear=True)
    a = build(c)
    a.out.fill_(math.nan)
    a.lse.fill_(math.nan)
    got = call(a)
    torch.cuda.synchronize()
    assert B.fp4idx_get_error(clear=True) == 0
    check(c, got)
    return c, a


LENS = [1, 2, 63, 64, 65, 127, 128, 129, 191, 192, 193, 256, 1000]


@pytest.mark.parametrize("kv", [None, 2])
@pytest.mark.parametrize("n", LENS)
def test_one_token_at_every_tile_edge(n, kv):
    run_case(n, [1], [n], heads=16, kv_heads=kv, visibility="full", dtype=FP16 if n % 2 else BF16)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("heads", [1, 3, 8, 16, 40, 64, 65, 128, 200])
def test_latent_head_counts(heads, dtype):
    run_case(heads, [1, 2, 1], [300, 77, 513], heads=heads, dtype=dtype)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("heads,kv", [(1, 1), (8, 8), (32, 4), (6, 2), (40, 8), (64, 1), (80, 1), (256, 2)])
def test_paged_head_layouts(heads, kv, dtype):
    run_case(heads, [1, 2, 1], [300, 77, 513], heads=heads, kv_heads=kv, dtype=dtype)


@pytest.mark.parametrize("kv", [None, 2])
@pytest.mark.parametrize("page", [64, 128])
@pytest.mark.parametrize("visibility", ["causal", "full", "lens", "offset"])
def test_ragged_requests(visibility, page, kv):
    # rows without keys, requests without rows or keys, lengths past the end
    run_case(7, [4, 0, 1, 3, 2, 5], [260, 50, 0, 129, 700, 5], heads=8, kv_heads=kv, page=page, visibility=visibility)


@pytest.mark.parametrize("kv", [None, 4])
def test_many_rows_of_one_request(kv):
    run_case(8, [150], [900], heads=8, kv_heads=kv)


@pytest.mark.parametrize("kv", [None, 2])
def test_long_axis_is_split_and_joined(kv):
    run_case(9, [1, 2], [20011, 9000], heads=16, kv_heads=kv)


def test_many_requests():
    lens = [(37 * i) % 701 for i in range(400)]
    run_case(10, [1] * 400, lens, heads=8, visibility="causal")
    run_case(11, [1] * 400, lens, heads=8, kv_heads=2, visibility="causal", page=128)


@pytest.mark.parametrize("page", [64, 128])
@pytest.mark.parametrize("select", [1, 63, 64, 65, 200, 2048])
def test_latent_selected_positions(select, page):
    run_case(select, [4, 1, 0, 2], [900, 5, 10, 2500], heads=16, page=page, select=select, visibility="lens")


@pytest.mark.parametrize("heads", [8, 64, 128, 130])
def test_latent_selected_head_counts(heads):
    run_case(heads, [3], [1500], heads=heads, select=300)


@pytest.mark.parametrize("page", [64, 128])
@pytest.mark.parametrize("select", [1, 2, 5, 16])
def test_paged_selected_blocks(select, page):
    run_case(select, [4, 1, 0, 2], [1900, 5, 10, 2500], heads=16, kv_heads=4, page=page, select=select, visibility="lens")


@pytest.mark.parametrize("heads,kv", [(4, 4), (65, 1), (160, 2)])
def test_paged_selected_head_layouts(heads, kv):
    run_case(heads, [3], [1500], heads=heads, kv_heads=kv, select=4)


def test_selected_rows_of_a_prefill_chunk():
    run_case(12, [200, 100], [1400, 3000], heads=16, select=256)


@pytest.mark.parametrize("kv", [None, 2])
def test_lists_that_leave_a_row_empty_and_foreign_indices(kv):
    c = R.make_case(13, [3, 2], [500, 90], heads=8, kv_heads=kv, select=6, device="cuda")
    c["indices"][..., 0, :] = -1                                          # nothing listed
    c["indices"][..., 1, :] = torch.tensor([2 ** 31 - 1, -2 ** 31, 10 ** 6, -7, 500, 1], device="cuda")  # not the row's
    c["indices"][..., 3, :] = 0                                           # one index six times: counts six times
    a = build(c)
    B.fp4idx_get_error(clear=True)
    got = call(a)
    assert B.fp4idx_get_error(clear=True) == 0
    check(c, got)


@pytest.mark.parametrize("kv", [None, 2])
def test_scores_of_every_size(kv):
    # weights spread over the whole range: growing scores move the running maximum at every tile, falling ones never
    for order in (1, -1):
        c = R.make_case(14, [2], [700], heads=8, kv_heads=kv, visibility="full", device="cuda", gain=8.0)
        for b, pages in enumerate(c["pages"]):
            for s in range(700):
                f = 0.02 + 2.0 * (s if order > 0 else 699 - s) / 700
                if kv is None:
                    c["k"][pages[s // 64], s % 64] *= f
                else:
                    c["k"][pages[s // 64], :, s % 64] *= f
        check(c, call(build(c)), f"order {order}")
    c = R.make_case(15, [2], [300], heads=8, kv_heads=kv, visibility="full", device="cuda", scale=-0.3)
    check(c, call(build(c)), "negative scale")
    c = R.make_case(16, [2], [300], heads=8, kv_heads=kv, visibility="full", device="cuda", scale=0.0)
    check(c, call(build(c)), "scale 0")


@pytest.mark.parametrize("kv", [None, 2])
def test_infinite_and_nan_scores(kv):
    # a key whose score is -inf for a row weighs nothing; a row of only such keys has no weight at all;
    # a NaN score is the row's result, and only that row's
    c = R.make_case(17, [1, 1, 1], [130, 3, 70], heads=4, kv_heads=kv, visibility="full", device="cuda")
    c["q"] = c["q"].abs() + 0.1
    dim = 570 if kv is None else 5  # a value that the latent form reads as a key only

    def key(b, s):
        p = c["pages"][b][s // 64]
        return c["k"][p, s % 64] if kv is None else c["k"][p, :, s % 64]

    for s in (0, 64, 129):
        key(0, s)[..., dim] = -math.inf
    for s in range(3):
        key(1, s)[..., dim] = -math.inf
    key(2, 69)[..., dim] = math.nan
    out, lse = call(build(c))
    want, want_lse, b_out, _ = R.reference(c)
    assert bool(((out[:2].double() - want[:2]).abs() <= b_out[:2].nan_to_num(posinf=0.05, nan=0.05).clamp(max=0.05)).all())
    assert bool((out[1] == 0).all()) and bool((lse[1] == -math.inf).all())
    assert bool(out[2].isnan().all()) and bool(lse[2].isnan().all())


@pytest.mark.parametrize("kv", [None, 2])
def test_pages_outside_the_cache_are_not_visible(kv):
    c = R.make_case(18, [2, 1], [400, 200], heads=8, kv_heads=kv, visibility="causal", device="cuda")
    c["pages"][0][2] = 10 ** 6
    c["pages"][1][0] = -3
    a = build(c)
    B.fp4idx_get_error(clear=True)
    got = call(a)
    assert B.fp4idx_get_error(clear=True) == B.ERR_PAGE_RANGE
    check(c, got)


@pytest.mark.parametrize("kv", [None, 2])
def test_strided_tensors_and_flat_tables(kv):
    c = R.make_case(19, [2, 1], [400, 200], heads=6, kv_heads=kv, visibility="causal", device="cuda")
    T, H, dk = c["q"].shape
    dv = 512 if kv is None else 128
    q = torch.full((T, H + 2, dk + 24), math.nan, dtype=BF16, device="cuda")
    q[:, 1:1 + H, 8:8 + dk] = c["q"]
    layers = torch.full((c["k"].shape[0], 3) + c["k"].shape[1:], math.nan, dtype=BF16, device="cuda")
    layers[:, 1] = c["k"]
    v = None
    if kv is not None:
        v = torch.full_like(layers, math.nan)
        v[:, 2] = c["v"]
        v = v[:, 2]
    out = torch.zeros((T, H + 1, dv), dtype=BF16, device="cuda")
    flat = torch.tensor([7, 7] + c["pages"][0] + [9] + c["pages"][1], dtype=torch.int32, device="cuda")
    po = torch.tensor([2, 3 + len(c["pages"][0])], dtype=torch.int32, device="cuda")
    a = build(c, q=q[:, 1:1 + H, 8:8 + dk], k=layers[:, 1], v=v, out=out[:, :H], block_table=flat, page_offsets=po)
    check(c, call(a))
    assert bool((out[:, H] == 0).all())  # nothing past the call's heads is written


@pytest.mark.parametrize("select", [0, 100])
@pytest.mark.parametrize("gap", [576, 8])
def test_latent_pages_any_distance_apart(gap, select):
    # pages a whole number of rows apart, or not (selected rows cannot be gathered by row number then)
    c = R.make_case(25, [2, 1], [400, 200], heads=8, select=select, device="cuda")
    P, page, dk = c["k"].shape
    wide = torch.full((P, page * dk + gap), math.nan, dtype=BF16, device="cuda")
    wide[:, :page * dk] = c["k"].reshape(P, -1)
    check(c, call(build(c, k=wide.as_strided((P, page, dk), (page * dk + gap, dk, 1)))))


def test_cache_beyond_two_to_the_31_elements():
    # 64-bit offsets: the pages used lie at both ends of a cache of more than 2^31 elements
    free = torch.cuda.mem_get_info()[0]
    if free < 12 << 30:
        pytest.skip("needs 12 GB")
    for select in (0, 100):
        far_pages(select)


def far_pages(select):
    c = R.make_case(20, [2], [300], heads=8, select=select, device="cuda")
    big = torch.empty((2 ** 31 // (64 * 576) + 40, 64, 576), dtype=BF16, device="cuda")
    move = {p: (i if i % 2 else big.shape[0] - 1 - i) for i, p in enumerate(c["pages"][0])}
    for p, to in move.items():
        big[to] = c["k"][p]
    c["pages"][0] = [move[p] for p in c["pages"][0]]
    c["k"] = big
    check(c, call(build(c)))
    del big, c
    torch.cuda.empty_cache()


@pytest.mark.parametrize("kv", [None, 4])
@pytest.mark.parametrize("select", [0, 8])
def test_same_bits_every_call_whatever_the_workspace_holds(kv, select):
    c = R.make_case(21, [2, 1, 1], [5000, 3000, 17], heads=32, kv_heads=kv, select=select, device="cuda")
    a = build(c)
    first = [x.clone() for x in call(a)]
    for fill in (0xFF, 0x00, 0x7F):
        a.workspace.fill_(fill)
        a.out.zero_()
        again = call(a)
        assert all(torch.equal(x, y) for x, y in zip(first, again))


@pytest.mark.parametrize("kv", [None, 4])
def test_another_stream_and_graph_replay(kv):
    c = R.make_case(22, [2, 1], [900, 300], heads=16, kv_heads=kv, visibility="lens", device="cuda")
    a = build(c)
    want = [x.clone() for x in call(a)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    a.out.zero_()
    call(a, stream=s)
    s.synchronize()
    assert torch.equal(a.out, want[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(a)
    a.out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a.out, want[0]) and torch.equal(a.lse, want[1])
    c["visible_len"].copy_(torch.tensor([40, 700, 299], dtype=torch.int32, device="cuda"))  # replays see new lengths
    g.replay()
    torch.cuda.synchronize()
    check(c, (a.out, a.lse))


@pytest.mark.parametrize("kv", [None, 4])
def test_workspace_too_small_is_refused(kv):
    c = R.make_case(23, [1], [9000], heads=16, kv_heads=kv, device="cuda")
    a = build(c)
    need = a.workspace.numel()
    a.out.fill_(5)
    a._ws = (a._ws[0], need - 1)
    with pytest.raises(B.Fp4idxError) as e:
        call(a)
    assert e.value.status == 3
    a._ws = (None, need)
    with pytest.raises(B.Fp4idxError) as e:
        call(a)
    assert e.value.status == 3
    torch.cuda.synchronize()
    assert bool((a.out == 5).all())


def test_lse_is_optional():
    c = R.make_case(24, [2], [300], heads=16, device="cuda")
    a = build(c)
    want = call(a)[0].clone()
    a.c.lse = None
    a.out.zero_()
    a.lse.fill_(3)
    call(a)
    torch.cuda.synchronize()
    assert torch.equal(a.out, want) and bool((a.lse == 3).all())


@pytest.mark.parametrize("kv", [None, 2])
def test_no_rows(kv):
    c = R.make_case(26, [0, 0], [70, 3], heads=16, kv_heads=kv, visibility="full", device="cuda")
    out, lse = call(build(c))
    torch.cuda.synchronize()
    assert out.shape[0] == 0 and lse.shape[0] == 0 and B.fp4idx_get_error(clear=True) == 0


@pytest.mark.parametrize("kv,heads", [(None, 16), (None, 128), (2, 8)])
@pytest.mark.parametrize("requests,length", [(1, 128), (1, 200), (30, 256), (60, 700), (200, 300)])
def test_every_way_of_cutting_items(requests, length, kv, heads):
    # whole items, items cut alike, equal runs over all items: chosen by sizes alone
    lens = [max(1, length - 37 * (i % 5)) for i in range(requests)]
    run_case(requests + length, [1] * requests, lens, heads=heads, kv_heads=kv, visibility="full")


@pytest.mark.parametrize("kv,heads,select", [(None, 128, 0), (None, 16, 0), (None, 64, 300), (4, 32, 0), (4, 32, 3)])
def test_many_short_items_in_a_row(kv, heads, select):
    # several items of one to ten tiles per CTA, whole and cut: the ring carries on from item to item
    n = 700
    lengths = [1 + (i * 2654435761 >> 7) % 600 for i in range(n)]
    c = R.make_case(26, [1] * n, lengths, heads=heads, kv_heads=kv, select=select, device="cuda")
    a = build(c)
    first = [x.clone() for x in call(a)]
    check(c, first)
    for _ in range(20):
        a.out.zero_()
        assert all(torch.equal(x, y) for x, y in zip(first, call(a)))

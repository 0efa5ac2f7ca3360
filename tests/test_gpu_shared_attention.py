"""GPU attention of requests that share a prefix (fp4idx_shared_prefix_attention) against the plain 64-bit
implementation, which reads every request through its own table row, at the lengths, groups, head layouts, masks
and strides where it can go wrong.  The tolerances are the bounds derived in tests/attention_ref.py."""
import math

import pytest
import torch

from fp4_sparse_attention_gb300 import binding as B
from tests import attention_ref as R
from tests import shared_ref as S

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16


def build(c, **over):
    a = dict(q=c["q"], k=c["k"], v=c["v"], cu_seqlens_q=R.offsets(c["q_lens"], "cuda"), cu_seqlens_k=R.offsets(c["k_lens"], "cuda"),
             block_table=R.table_of(c), max_seqlen_q=max(c["q_lens"] + [1]), max_seqlen_k=max(c["k_lens"] + [0]), scale=c["scale"],
             visible_len=c.get("visible_len"), causal=c.get("causal", False), qo_offset=c.get("qo_offset"), **S.group_arguments(c))
    a.update(over)
    a = B.DeviceSharedAttention(**a)
    a.out.fill_(math.nan)
    a.lse.fill_(math.nan)
    return a


def check(c, got, what=""):
    out, lse = got
    want, want_lse, b_out, b_lse = R.reference(c)
    T = want.shape[0]
    assert bool((out[T:] == 0).all()) and bool((lse[T:] == -math.inf).all()), what  # rows of no request
    out, lse = out[:T], lse[:T]
    off = (out.double() - want).abs()
    assert torch.isfinite(out).all(), what
    assert bool((off <= b_out).all()), f"{what}: out off by {float((off - b_out).max()):.3g} over the bound"
    none = want_lse == -math.inf
    assert torch.equal(lse == -math.inf, none), what
    off = (lse.double() - want_lse).abs()[~none]
    assert bool((off <= b_lse[~none]).all()), f"{what}: lse"


def run_case(*args, **kw):
    c = S.make_shared(*args, device="cuda", **kw)
    B.fp4idx_get_error(clear=True)
    a = build(c)
    got = B.fp4idx_shared_prefix_attention(a)
    torch.cuda.synchronize()
    assert B.fp4idx_get_error(clear=True) == 0
    check(c, got)
    return c, a


# ---------------------------------------------------------------- lengths
@pytest.mark.parametrize("own", [0, 1, 63, 64, 65, 127, 128, 129, 200])
@pytest.mark.parametrize("prefix", [0, 1, 63, 64, 65, 127, 128, 129, 192, 257])
def test_every_tile_edge(prefix, own):
    if prefix + own == 0:
        pytest.skip("no keys: another test")
    run_case(prefix + own, [(prefix, [(1, own), (1, max(0, own - 1)), (2, own + 1)])], heads=8, kv_heads=2, page=64 if own % 2 else 128,
             visibility="full", dtype=FP16 if prefix % 2 else BF16)


@pytest.mark.parametrize("page", [64, 128])
@pytest.mark.parametrize("prefix", [1, 64, 700])
def test_one_request_is_paged_attention(prefix, page):
    c, a = run_case(3, [(prefix, [(1, 5)])], heads=16, kv_heads=2, page=page, visibility="full")
    p = B.DeviceAttention(q=a.q, k=a.k, v=a.v, cu_seqlens_q=a.cu_seqlens_q, cu_seqlens_k=a.cu_seqlens_k, block_table=a.block_table,
                          max_seqlen_q=1, max_seqlen_k=prefix + 5, scale=c["scale"])
    out, lse = B.fp4idx_paged_attention(p)
    assert torch.allclose(out.float(), a.out.float(), atol=0.03) and torch.allclose(lse, a.lse, atol=1e-4)


@pytest.mark.parametrize("visibility", ["causal", "full", "lens", "offset"])
@pytest.mark.parametrize("page", [64, 128])
def test_ragged_groups(visibility, page):
    # groups of no requests, requests without rows, keys or either, lengths past the end, rows that see less than the prefix
    groups = [(300, [(4, 60), (0, 10), (1, 0), (3, 400)]), (0, [(2, 70)]), (50, []), (129, [(2, 1), (2, 129)]), (0, [(5, 5), (0, 0), (1, 300)]),
              (1000, [(1, 64)] * 7)]
    run_case(7, groups, heads=8, kv_heads=2, page=page, visibility=visibility)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("heads,kv", [(1, 1), (8, 8), (32, 4), (6, 2), (40, 8), (64, 1), (80, 1), (256, 2), (300, 1), (1024, 4)])
def test_head_layouts(heads, kv, dtype):
    run_case(heads, [(300, [(1, 40), (2, 77)]), (129, [(1, 3)])], heads=heads, kv_heads=kv, dtype=dtype)


@pytest.mark.parametrize("rows", [1, 3])
@pytest.mark.parametrize("reqs", [1, 2, 15, 16, 17, 31, 32, 33, 64, 65, 130])
def test_requests_around_the_blocks_of_pairs(reqs, rows):
    # 8 heads a K/V head: 16 requests of one row are 128 pairs, 32 are 256; of three rows they straddle the blocks
    run_case(reqs, [(200, [(rows, 1 + (37 * i) % 150) for i in range(reqs)])], heads=16, kv_heads=2)


@pytest.mark.parametrize("page", [64, 128])
def test_many_rows_of_each_request(page):
    run_case(8, [(500, [(150, 150), (90, 200), (1, 3), (64, 64)])], heads=8, kv_heads=2, page=page)


@pytest.mark.parametrize("rows", [1, 40])
def test_long_prefix_is_split_and_joined(rows):
    run_case(9, [(20011, [(rows, rows + 500), (rows, rows)]), (64, [(1, 9000)])], heads=16, kv_heads=2)


def test_many_groups():
    groups = [((37 * i) % 701, [(1, 1 + (11 * i + 53 * j) % 90) for j in range(i % 4)]) for i in range(300)]
    run_case(10, groups, heads=8, kv_heads=2)
    run_case(11, groups, heads=4, kv_heads=4, page=128)


def test_more_blocks_than_a_cta_has_threads():
    # 800 blocks of a group: a row of 256 heads each; 900 groups, some without requests or rows
    run_case(13, [(130, [(400, 400), (400, 430)])], heads=256, kv_heads=1)
    groups = [((29 * i) % 300, [((i + j) % 3, 1 + (11 * i + 53 * j) % 70) for j in range((i // 2) % 3)]) for i in range(900)]
    run_case(14, groups, heads=4, kv_heads=2)


@pytest.mark.parametrize("reqs", [33, 300, 1023, 1025, 2500])
def test_blocks_and_groups_of_many_requests(reqs):
    # one head a K/V head: a block is 256 rows, so up to 256 requests and more where some have no rows
    run_case(reqs, [(70, [((7 * i) % 5 % 3, 1 + (37 * i) % 40) for i in range(reqs)]), (0, [(1, 5)] * 40)], heads=2, kv_heads=2)


def test_long_runs():
    # 16 tiles a CTA and more: equal runs over blocks of other lengths, and a block's own, with many requests
    groups = [(1001 + 1143 * i, [(4, 5 + (331 * (6 * i + j)) % 700) for j in range(3)]) for i in range(8)]
    run_case(17, groups, heads=40, kv_heads=8)
    run_case(18, [(16000, [(1, 1 + (53 * i) % 300) for i in range(40)])], heads=32, kv_heads=4, page=128)
    run_case(19, [(30000, [(1, 1)] * 33)], heads=32, kv_heads=2, dtype=FP16)


@pytest.mark.parametrize("groups", [33, 76, 152, 153])
def test_blocks_of_alike_lengths(groups):
    # as many CTAs as blocks, or a whole number of them each
    run_case(groups, [(64, [(1, 200 + i % 3)]) for i in range(groups)], heads=4, kv_heads=1)
    run_case(groups, [(0, [(1, 1)]) for i in range(groups)], heads=1, kv_heads=1)


def test_long_requests_without_a_prefix():
    run_case(12, [(0, [(1, 9000), (2, 3000), (1, 17)])], heads=8, kv_heads=2)


@pytest.mark.parametrize("requests,prefix,own", [(1, 128, 5), (2, 256, 130), (40, 700, 3), (60, 64, 700), (200, 300, 64)])
@pytest.mark.parametrize("per", [1, 5, 1000])
def test_every_way_of_cutting(requests, prefix, own, per):
    groups = [(prefix, [(1, 1 + (own * (j + 1)) % (own + 1)) for j in range(i, min(requests, i + per))]) for i in range(0, requests, per)]
    run_case(requests + prefix, groups, heads=32, kv_heads=4, visibility="full")


# ---------------------------------------------------------------- groups that are not what they should be
def test_prefix_longer_than_the_first_request():
    # the first request's key count bounds the prefix; the rest is read through each request's own row
    c = S.make_shared(20, [(100, [(1, 10), (2, 300)])], heads=8, kv_heads=2, visibility="full", device="cuda")
    for n in (110, 111, 5000, 2 ** 31 - 1):
        c["groups"] = [(n, c["groups"][0][1])]
        # positions 100..109 of the two requests differ: the second one's are the first one's only up to 100
        c2 = dict(c, k=c["k"].clone(), v=c["v"].clone())
        p0, p1 = c["pages"][0][1], c["pages"][1][1]
        for x in (c2["k"], c2["v"]):
            x[p1, :, 36:46] = x[p0, :, 36:46]
        check(c2, B.fp4idx_shared_prefix_attention(build(c2)), str(n))


def test_no_and_negative_prefixes():
    c = S.make_shared(21, [(0, [(1, 100), (2, 300)]), (0, [(1, 5)])], heads=8, kv_heads=2, visibility="full", device="cuda")
    check(c, B.fp4idx_shared_prefix_attention(build(c, prefix_len=torch.tensor([-5, -2 ** 31], dtype=torch.int32, device="cuda"))))


def test_requests_of_no_group():
    c = S.make_shared(22, [(100, [(1, 10), (2, 30)]), (64, [(3, 5), (1, 70)])], heads=8, kv_heads=2, visibility="full", device="cuda")
    want, want_lse, b_out, _ = R.reference(c)
    for offsets, lo, hi in (([0, 2, 3], 0, 6), ([2, 2, 4], 3, 7), ([1, 1, 1], 0, 0), ([-3, 2, 90], 0, 7), ([9, 9, 9], 0, 0)):
        a = build(c, group_offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"),
                  prefix_len=torch.tensor([0, 0], dtype=torch.int32, device="cuda"), max_group_rows=7)
        out, lse = B.fp4idx_shared_prefix_attention(a)
        inside = torch.zeros(7, dtype=torch.bool, device="cuda")
        inside[lo:hi] = True
        assert bool((out[~inside] == 0).all()) and bool((lse[~inside] == -math.inf).all()), offsets
        assert bool(((out.double() - want).abs() <= b_out)[inside].all()), offsets


@pytest.mark.parametrize("extra", [1, 7, 1000])
@pytest.mark.parametrize("visibility", ["causal", "full", "lens"])
def test_rows_of_no_request(extra, visibility):
    c = S.make_shared(23, [(100, [(1, 10), (2, 30)]), (64, [(0, 5)])], heads=6, kv_heads=2, visibility=visibility, device="cuda")
    T = c["q"].shape[0]
    q = torch.full((T + extra,) + c["q"].shape[1:], math.nan, dtype=BF16, device="cuda")
    q[:T] = c["q"]
    over = dict(q=q)
    if c.get("visible_len") is not None:
        over["visible_len"] = torch.cat([c["visible_len"], torch.full((extra,), 5, dtype=torch.int32, device="cuda")])
    check(c, B.fp4idx_shared_prefix_attention(build(c, **over)))


def test_only_padding_and_no_rows():
    c = S.make_shared(24, [(100, [(0, 10), (0, 30)])], heads=6, kv_heads=2, visibility="full", device="cuda")
    q = torch.full((9, 6, 128), math.nan, dtype=BF16, device="cuda")
    check(c, B.fp4idx_shared_prefix_attention(build(c, q=q)))
    out, lse = B.fp4idx_shared_prefix_attention(build(c))
    assert out.shape[0] == 0 and lse.shape[0] == 0 and B.fp4idx_get_error(clear=True) == 0


def test_pages_outside_the_cache_are_not_visible():
    c = S.make_shared(25, [(400, [(2, 30), (1, 200)])], heads=8, kv_heads=2, visibility="causal", device="cuda")
    # a page of the shared part (both rows name it), one of a request's own
    c["pages"][0][2] = c["pages"][1][2] = 10 ** 6
    c["pages"][1][8] = -3
    B.fp4idx_get_error(clear=True)
    got = B.fp4idx_shared_prefix_attention(build(c))
    assert B.fp4idx_get_error(clear=True) == B.ERR_PAGE_RANGE
    check(c, got)


def test_only_the_first_row_is_read_below_the_prefix():
    # the other requests' entries of whole shared pages may be anything
    c = S.make_shared(26, [(300, [(1, 30), (1, 200)])], heads=8, kv_heads=2, visibility="full", device="cuda")
    table = R.table_of(c)
    table[1, :4] = -1
    B.fp4idx_get_error(clear=True)
    got = B.fp4idx_shared_prefix_attention(build(c, block_table=table))
    assert B.fp4idx_get_error(clear=True) == 0
    check(c, got)


# ---------------------------------------------------------------- values
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_scores_of_every_size(dtype):
    for order in (1, -1):
        c = S.make_shared(14, [(500, [(2, 200), (1, 150)])], heads=8, kv_heads=2, visibility="full", device="cuda", gain=8.0, dtype=dtype)
        done = set()
        for pages, n in zip(c["pages"], c["k_lens"]):
            for s in range(n):
                if (pages[s // 64], s % 64) not in done:  # shared pages once
                    done.add((pages[s // 64], s % 64))
                    c["k"][pages[s // 64], :, s % 64] *= 0.02 + 2.0 * (s if order > 0 else 699 - s) / 700
        check(c, B.fp4idx_shared_prefix_attention(build(c)), f"order {order}")
    for scale in (-0.3, 0.0):
        c = S.make_shared(15, [(130, [(2, 70), (1, 5)])], heads=8, kv_heads=2, visibility="full", device="cuda", scale=scale, dtype=dtype)
        check(c, B.fp4idx_shared_prefix_attention(build(c)), f"scale {scale}")


def test_infinite_and_nan_scores():
    c = S.make_shared(17, [(130, [(1, 3), (1, 70)]), (0, [(1, 3)]), (64, [(1, 70)])], heads=4, kv_heads=2, visibility="full", device="cuda")
    c["q"] = c["q"].abs() + 0.1

    def key(b, s):
        return c["k"][c["pages"][b][s // 64], :, s % 64]

    for s in (0, 64):                       # shared keys
        key(0, s)[..., 5] = -math.inf
    key(0, 129)[..., 5] = key(1, 129)[..., 5] = -math.inf
    key(1, 199)[..., 5] = -math.inf
    for s in range(3):                      # every key of a request
        key(2, s)[..., 5] = -math.inf
    key(3, 133)[..., 5] = math.nan
    out, lse = B.fp4idx_shared_prefix_attention(build(c))
    want, want_lse, b_out, _ = R.reference(c)
    # (the reference's bound knows no -inf scores: as in the other attention's test, 0.05 for outputs near 1)
    assert bool(((out[:3].double() - want[:3]).abs() <= b_out[:3].nan_to_num(posinf=0.05, nan=0.05).clamp(max=0.05)).all())
    assert bool((out[2] == 0).all()) and bool((lse[2] == -math.inf).all())
    assert bool(out[3].isnan().all()) and bool(lse[3].isnan().all())


def test_fp16_shares_of_a_long_prefix_add_up():
    # one key of weight 1 and value 0 behind a prefix of keys of weight 2^-25 and values near 100
    n = 5000
    c = S.make_shared(41, [(n, [(1, 1), (1, 2)])], heads=4, kv_heads=2, visibility="full", dtype=FP16, scale=1.0, device="cuda", junk=0.0)
    g = torch.Generator().manual_seed(1)
    c["q"].zero_()
    c["q"][..., 0] = 1.0
    c["k"].zero_()
    c["k"][..., 0] = -25.2 * math.log(2)
    c["v"][:] = (100 + torch.rand(c["v"].shape, generator=g)).half().cuda()
    b1, b0 = c["pages"][1], c["pages"][0]
    for x in (c["k"], c["v"]):
        x[b1[n // 64], :, :n % 64] = x[b0[n // 64], :, :n % 64]
    for b, pages in enumerate((b0, b1)):
        at = n
        c["k"][pages[at // 64], :, at % 64, 0] = 0.0
        c["v"][pages[at // 64], :, at % 64] = 0.0
    out, lse = B.fp4idx_shared_prefix_attention(build(c))
    want, want_lse, b_out, b_lse = R.reference(c)
    # as for fp4idx_paged_attention: weights down to 2^-32 of the largest are kept, so the reference's allowance of
    # 2^-25 a key shrinks to that; the result may be subnormal
    bound = b_out - n * (2.0 ** -25 - 2.0 ** -32) * 101 + 2.0 ** -25
    assert bool((bound < 0.5 * want).all())
    assert bool(((out.double() - want).abs() <= bound).all()) and bool(((lse.double() - want_lse).abs() <= b_lse).all())


# ---------------------------------------------------------------- layouts
def test_strided_tensors_and_flat_tables():
    c = S.make_shared(19, [(129, [(2, 200), (1, 50)])], heads=6, kv_heads=2, visibility="causal", device="cuda")
    T, H, d = c["q"].shape
    q = torch.full((T, H + 2, d + 24), math.nan, dtype=BF16, device="cuda")
    q[:, 1:1 + H, 8:8 + d] = c["q"]
    layers = torch.full((c["k"].shape[0], 3) + c["k"].shape[1:], math.nan, dtype=BF16, device="cuda")
    layers[:, 1], layers[:, 2] = c["k"], c["v"]
    out = torch.zeros((T, H + 1, d), dtype=BF16, device="cuda")
    flat = torch.tensor([7, 7] + c["pages"][0] + [9] + c["pages"][1], dtype=torch.int32, device="cuda")
    po = torch.tensor([2, 3 + len(c["pages"][0])], dtype=torch.int32, device="cuda")
    a = build(c, q=q[:, 1:1 + H, 8:8 + d], k=layers[:, 1], v=layers[:, 2], out=out[:, :H], block_table=flat, page_offsets=po)
    out.zero_()
    check(c, B.fp4idx_shared_prefix_attention(a))
    assert bool((out[:, H] == 0).all())  # nothing past the call's heads is written


@pytest.mark.parametrize("rows,heads", [(1, 6), (2, 6), (70, 6), (1, 2)])
def test_queries_by_head(rows, heads):
    c = S.make_shared(51, [(100, [(rows, rows + 9), (1, 80)])], heads=heads, kv_heads=2, device="cuda")
    check(c, B.fp4idx_shared_prefix_attention(build(c, q=c["q"].transpose(0, 1).contiguous().transpose(0, 1))))


def test_cache_beyond_two_to_the_31_elements():
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    c = S.make_shared(20, [(300, [(1, 70), (2, 100)])], heads=8, kv_heads=2, device="cuda", junk=0.0)
    big_k, big_v = (torch.empty((2 ** 31 // (2 * 64 * 128) + 40, 2, 64, 128), dtype=BF16, device="cuda") for _ in range(2))
    move = {}
    for pages in c["pages"]:
        for p in pages:
            move.setdefault(p, len(move) if len(move) % 2 else big_k.shape[0] - 1 - len(move))
    for p, to in move.items():
        big_k[to], big_v[to] = c["k"][p], c["v"][p]
    c["pages"] = [[move[p] for p in pages] for pages in c["pages"]]
    c["k"], c["v"] = big_k, big_v
    check(c, B.fp4idx_shared_prefix_attention(build(c)))
    del big_k, big_v, c
    torch.cuda.empty_cache()


# ---------------------------------------------------------------- calls
CALLS = [[(5000, [(1, 40)] * 20), (300, [(2, 700), (1, 17)])], [(64, [(1, 1)])], [(1000, [(70, 100), (50, 60)])]]


@pytest.mark.parametrize("groups", CALLS)
def test_same_bits_every_call_whatever_the_workspace_holds(groups):
    c = S.make_shared(21, groups, heads=32, kv_heads=4, device="cuda")
    a = build(c)
    first = [x.clone() for x in B.fp4idx_shared_prefix_attention(a)]
    for fill in (0xFF, 0x00, 0x7F):
        a.workspace.fill_(fill)
        a.out.fill_(math.nan)
        assert all(torch.equal(x, y) for x, y in zip(first, B.fp4idx_shared_prefix_attention(a)))
    for _ in range(20):
        a.out.fill_(math.nan)
        assert all(torch.equal(x, y) for x, y in zip(first, B.fp4idx_shared_prefix_attention(a)))


def test_another_stream_two_objects_and_graph_replay():
    c = S.make_shared(22, [(900, [(2, 30), (1, 300)]), (64, [(1, 5)])], heads=16, kv_heads=4, visibility="lens", device="cuda")
    a, b = build(c), build(c)
    want = [x.clone() for x in B.fp4idx_shared_prefix_attention(a)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        a.out.zero_()
        b.out.zero_()
        torch.cuda.synchronize()
        for x, s in zip((a, b), streams):  # at the same time, a workspace each
            B.fp4idx_shared_prefix_attention(x, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(a.out, want[0]) and torch.equal(b.out, want[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.fp4idx_shared_prefix_attention(a)
        B.fp4idx_shared_prefix_attention(b)
    a.out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a.out, want[0]) and torch.equal(a.lse, want[1])
    c["visible_len"].copy_(torch.tensor([40, 929, 1100, 69], dtype=torch.int32, device="cuda"))  # replays see new lengths
    a.prefix_len.copy_(torch.tensor([130, 0], dtype=torch.int32, device="cuda"))                   # and a shorter prefix
    g.replay()
    torch.cuda.synchronize()
    check(c, (a.out, a.lse))


def test_graphs_of_different_calls_share_a_workspace():
    cases = [S.make_shared(60 + i, groups, heads=16, kv_heads=4, device="cuda") for i, groups in
             enumerate(([(5000, [(1, 40)] * 20)], [(64, [(1, 1)] * 3), (0, [(2, 900)])], [(300, [(70, 100), (50, 60)])]))]
    shared = torch.empty(max(build(c).workspace.numel() for c in cases), dtype=torch.uint8, device="cuda")
    calls = [build(c, workspace=shared) for c in cases]
    want = [[x.clone() for x in B.fp4idx_shared_prefix_attention(a)] for a in calls]
    graphs = []
    for a in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            B.fp4idx_shared_prefix_attention(a)
        graphs.append(g)
    for order in ((0, 1, 2, 1, 0, 2), (2, 2, 0, 0, 1, 1)):
        for a in calls:
            a.out.fill_(math.nan)
        for i in order:  # one behind another, no wait between
            graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for a, w in zip(calls, want) for x, y in zip((a.out, a.lse), w))
    assert B.fp4idx_get_error(clear=True) == 0


def test_workspace_too_small_is_refused():
    c = S.make_shared(23, [(900, [(1, 30)] * 40)], heads=16, kv_heads=4, device="cuda")
    a = build(c)
    need = a.workspace.numel()
    a.out.fill_(5)
    for ws in ((a._ws[0], need - 1), (None, need)):
        a._ws = ws
        with pytest.raises(B.Fp4idxError) as e:
            B.fp4idx_shared_prefix_attention(a)
        assert e.value.status == 3
    torch.cuda.synchronize()
    assert bool((a.out == 5).all())


def test_lse_is_optional():
    c = S.make_shared(24, [(300, [(2, 30), (1, 300)])], heads=16, kv_heads=4, device="cuda")
    a = build(c)
    want = B.fp4idx_shared_prefix_attention(a)[0].clone()
    a.shared.attention.lse = None
    a.out.zero_()
    a.lse.fill_(3)
    B.fp4idx_shared_prefix_attention(a)
    torch.cuda.synchronize()
    assert torch.equal(a.out, want) and bool((a.lse == 3).all())

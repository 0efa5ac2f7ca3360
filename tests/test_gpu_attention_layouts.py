"""Orders and strides of the attention operators' tensors beyond the dense ones: queries computed by
head, and dimensions of one, whose strides mean nothing."""
import pytest
import torch

from fp4_sparse_attention_gb300 import binding as B
from tests import attention_ref as R
from tests.test_gpu_attention import build, call, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", [None, 2])
@pytest.mark.parametrize("select", [0, 3])
@pytest.mark.parametrize("rows,heads", [([1], 6), ([2, 1], 6), ([70], 6), ([1], 2)])
def test_queries_by_head(rows, heads, select, kv):
    c = R.make_case(51, rows, [300] * len(rows), heads=heads, kv_heads=kv, select=select, device="cuda")
    q = c["q"].transpose(0, 1).contiguous().transpose(0, 1)  # as a product by head leaves it
    check(c, call(build(c, q=q)))
    wide = torch.zeros((heads, 2 * q.shape[0], q.shape[2] + 8), dtype=q.dtype, device="cuda")
    part = wide[:, ::2, :q.shape[2]].transpose(0, 1)
    part.copy_(q)
    check(c, call(build(c, q=part)))


@pytest.mark.parametrize("kv", [None, 1])
def test_dimensions_of_one(kv):
    c = R.make_case(52, [1], [50], heads=1, kv_heads=kv, spare=0, device="cuda")
    d, dv = c["q"].shape[2], 512 if kv is None else 128
    page = (1, 64, d) if kv is None else (1, 1, 64, d)
    over = dict(q=c["q"].as_strided((1, 1, d), (3, 5, 1)), k=c["k"].as_strided(page, (7,) * (len(page) - 2) + (d, 1)),
                out=torch.zeros((dv,), dtype=c["q"].dtype, device="cuda").as_strided((1, 1, dv), (1, 1, 1)))
    if kv is not None:
        over["v"] = c["v"].as_strided(page, (9, 4, d, 1))
    check(c, call(build(c, **over)))


def test_one_token_and_one_page():
    x = torch.randn((576,), device="cuda").bfloat16()
    cache = torch.zeros((64 * 576,), dtype=torch.bfloat16, device="cuda")
    slot = torch.tensor([9], dtype=torch.int32, device="cuda")
    B.fp4idx_store_latent(x[:512].as_strided((1, 512), (1, 1)), x[512:].as_strided((1, 64), (1, 1)), slot,
                          cache.as_strided((1, 64, 576), (5, 576, 1)))
    assert torch.equal(cache.view(64, 576)[9], x) and int((cache != 0).sum()) == int((x != 0).sum())
    kv = torch.randn((2, 128), device="cuda").bfloat16()
    k, v = torch.zeros((2, 64 * 128), dtype=torch.bfloat16, device="cuda")
    B.fp4idx_store_kv(kv[0].as_strided((1, 1, 128), (1, 2, 1)), kv[1].as_strided((1, 1, 128), (3, 4, 1)), slot,
                      k.as_strided((1, 1, 64, 128), (5, 6, 128, 1)), v.as_strided((1, 1, 64, 128), (7, 8, 128, 1)))
    assert torch.equal(k.view(64, 128)[9], kv[0]) and torch.equal(v.view(64, 128)[9], kv[1])
    lens = torch.tensor([100, 7], dtype=torch.int32, device="cuda")
    new = torch.tensor([3, 7], dtype=torch.int32, device="cuda")
    table = torch.tensor([[4, 5, -1]], dtype=torch.int32, device="cuda")
    B.fp4idx_get_error(clear=True)
    out = B.fp4idx_build_tables(lens[::2], new[::2], table.as_strided((1, 3), (1, 1)), new[:1], 64, 3)
    assert B.fp4idx_get_error(clear=True) == 0
    assert [x.tolist() for x in out] == [[0, 3], [0, 103], [101, 102, 103], [5 * 64 + 36, 5 * 64 + 37, 5 * 64 + 38], [0]]

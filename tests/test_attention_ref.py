"""Pins of the plain 64-bit attention that the GPU tests compare with, and host-side refusals of
the attention, store and table calls (no GPU needed)."""
import ctypes
import math

import pytest
import torch

from fp4_sparse_attention_gb300 import binding, build
from tests import attention_ref as R


@pytest.mark.parametrize("kv", [None, 2])
def test_equal_scores_average_the_values(kv):
    c = R.make_case(1, [1], [70], heads=4, kv_heads=kv, visibility="full")
    c["q"] = torch.zeros_like(c["q"])
    out, lse, _, _ = R.reference(c)
    assert torch.allclose(lse, torch.full_like(lse, math.log(70)))
    for h in range(4):
        v = [(c["k"][c["pages"][0][s // 64], s % 64, :512] if kv is None else
              c["v"][c["pages"][0][s // 64], h // 2, s % 64]).double() for s in range(70)]
        assert torch.allclose(out[0, h], torch.stack(v).mean(0))


def test_one_key_and_no_key():
    c = R.make_case(2, [1, 1, 2], [1, 0, 3], heads=2, visibility="causal")
    out, lse, _, _ = R.reference(c)
    k = c["k"][c["pages"][0][0], 0].double()
    assert torch.allclose(out[0, 1], k[:512])
    assert torch.allclose(lse[0, 1], c["q"][0, 1].double() @ k * c["scale"])
    assert torch.all(out[1] == 0) and torch.all(lse[1] == -math.inf)
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("kv", [None, 2])
def test_whole_prefix_is_every_key_or_block_selected(kv):
    c = R.make_case(3, [2, 1], [200, 90], heads=4, kv_heads=kv, visibility="causal")
    want = R.reference(c)
    n = 200 if kv is None else 2
    idx = torch.arange(n, dtype=torch.int32).flip(0)
    c["indices"] = idx.expand(3, n) if kv is None else idx.expand(kv, 3, n)
    got = R.reference(c)
    for a, b in zip(want[:2], got[:2]):
        assert torch.allclose(a, b, rtol=1e-12, atol=1e-12)


def test_matches_softmax():
    c = R.make_case(4, [3], [129], heads=6, kv_heads=3, visibility="full", page=128)
    out, lse, _, _ = R.reference(c)
    flat = [c["pages"][0][s // 128] * 128 + s % 128 for s in range(129)]
    for h in range(6):
        k = c["k"][:, h // 2].reshape(-1, 128)[flat].double()
        v = c["v"][:, h // 2].reshape(-1, 128)[flat].double()
        s = c["q"][:, h].double() @ k.T * c["scale"]
        assert torch.allclose(out[:, h], torch.softmax(s, 1) @ v)
        assert torch.allclose(lse[:, h], torch.logsumexp(s, 1))


# ---------------------------------------------------------------- refusals
@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load_library()


FAKE = 1 << 20  # aligned non-null placeholder address; never dereferenced


def _attention(latent, **over):
    dk = 576 if latent else 128
    kv = 1 if latent else 4
    c = binding.CAttention(
        dtype=0, num_seqs=2, num_rows=4, num_heads=16, num_kv_heads=kv, page_size=64, num_pages=32, table_stride=16,
        max_seqlen_q=2, max_seqlen_k=1024, q=FAKE, q_row_stride=16 * dk, q_head_stride=dk, k=FAKE,
        v=None if latent else FAKE, page_stride=kv * 64 * dk, cu_seqlens_q=FAKE, cu_seqlens_k=FAKE, block_table=FAKE,
        page_offsets=None, visible_len=None, qo_offset=None, causal=0, scale=0.1, indices=None, num_indices=0, out=FAKE,
        out_row_stride=16 * (512 if latent else 128), lse=None)
    for k, v in over.items():
        setattr(c, k, v)
    return c


BAD = [
    (dict(dtype=2), 1), (dict(num_seqs=0), 1), (dict(num_rows=-1), 1), (dict(num_heads=0), 1),
    (dict(num_heads=2048, q_row_stride=2048 * 576, out_row_stride=2048 * 512), 2), (dict(page_size=32), 2),
    (dict(page_size=96), 2), (dict(num_pages=0), 1), (dict(max_seqlen_q=0), 1), (dict(max_seqlen_k=-1), 1),
    (dict(max_seqlen_k=2 ** 31 - 1, table_stride=1 << 30), 2),
    (dict(q=None), 1), (dict(k=None), 1), (dict(out=None), 1), (dict(cu_seqlens_q=None), 1),
    (dict(cu_seqlens_k=None), 1), (dict(block_table=None), 1), (dict(q=FAKE + 8), 1), (dict(k=FAKE + 2), 1),
    (dict(out=FAKE + 4), 1), (dict(lse=FAKE + 2), 1), (dict(q_head_stride=64), 1), (dict(q_head_stride=577), 1),
    (dict(q_row_stride=576), 1), (dict(out_row_stride=100), 1), (dict(page_stride=64), 1),
    (dict(page_stride=4 * 128 * 576 + 4), 1), (dict(table_stride=15), 1), (dict(qo_offset=FAKE), 1),
    (dict(scale=math.inf), 1), (dict(scale=math.nan), 1), (dict(indices=FAKE), 1),
    (dict(indices=FAKE, num_indices=(1 << 20) + 1), 2), (dict(indices=FAKE + 1, num_indices=4), 1),
]


@pytest.mark.parametrize("over,status", BAD + [(dict(num_kv_heads=2), 1), (dict(v=FAKE), 1)])
def test_latent_attention_refuses(lib, over, status):
    c = _attention(True, **over)
    assert lib.fp4idx_latent_attention(ctypes.byref(c), FAKE, 1 << 40, None) == status
    assert lib.fp4idx_last_error_message()


@pytest.mark.parametrize("over,status", BAD + [(dict(num_kv_heads=3), 1), (dict(v=None), 1), (dict(v=FAKE + 2), 1)])
def test_paged_attention_refuses(lib, over, status):
    c = _attention(False, **over)
    assert lib.fp4idx_paged_attention(ctypes.byref(c), FAKE, 1 << 40, None) == status
    assert lib.fp4idx_last_error_message()


def test_attention_null_and_empty(lib):
    assert lib.fp4idx_latent_attention(None, None, 0, None) == 1
    assert lib.fp4idx_paged_attention(None, None, 0, None) == 1
    assert lib.fp4idx_attention_workspace_bytes(None) == 0
    for latent, f in ((True, lib.fp4idx_latent_attention), (False, lib.fp4idx_paged_attention)):
        assert f(ctypes.byref(_attention(latent, num_rows=0)), None, 0, None) == 0
        assert f(ctypes.byref(_attention(latent, num_rows=0, q=None, out=None)), None, 0, None) == 0


@pytest.mark.parametrize("over,status", [
    (dict(latent=None), 1), (dict(latent=FAKE + 4), 1), (dict(latent_stride=500), 1), (dict(latent_stride=516), 1),
    (dict(rope=None), 1), (dict(rope_stride=60), 1), (dict(slots=None), 1), (dict(n=-1), 1), (dict(page=16), 2),
    (dict(num_pages=0), 1), (dict(page_stride=64 * 576 - 8), 1), (dict(cache=None), 1), (dict(n=0), 0),
])
def test_store_latent_refuses(lib, over, status):
    a = dict(latent=FAKE, latent_stride=512, rope=FAKE, rope_stride=64, slots=FAKE, n=4, page=64, num_pages=8,
             page_stride=64 * 576, cache=FAKE)
    a.update(over)
    assert lib.fp4idx_store_latent(*a.values(), None) == status


@pytest.mark.parametrize("over,status", [
    (dict(k_new=None), 1), (dict(k_stride=256), 1), (dict(v_new=None), 1), (dict(v_stride=516), 1), (dict(slots=None), 1),
    (dict(n=-1), 1), (dict(heads=0), 1), (dict(heads=2000, k_stride=1 << 20, v_stride=1 << 20, page_stride=1 << 30), 2),
    (dict(page=256), 2), (dict(num_pages=0), 1), (dict(page_stride=64), 1), (dict(k=None), 1), (dict(v=None), 1),
    (dict(n=0), 0),
])
def test_store_kv_refuses(lib, over, status):
    a = dict(k_new=FAKE, k_stride=512, v_new=FAKE, v_stride=512, slots=FAKE, n=4, heads=4, page=64, num_pages=8,
             page_stride=4 * 64 * 128, k=FAKE, v=FAKE)
    a.update(over)
    assert lib.fp4idx_store_kv(*a.values(), None) == status


@pytest.mark.parametrize("over,status", [
    (dict(cached=None), 1), (dict(new=None), 1), (dict(table=None), 1), (dict(cu_q=None), 1), (dict(cu_k=None), 1),
    (dict(taken=None), 1), (dict(visible=None), 1), (dict(slots=None), 1), (dict(free=None), 1), (dict(reqs=0), 1),
    (dict(rows=-1), 1), (dict(num_free=-1), 1), (dict(stride=0), 1), (dict(num_pages=0), 1), (dict(page=32), 2),
    (dict(num_pages=1 << 26), 2), (dict(slots=FAKE + 2), 1),
])
def test_build_tables_refuses(lib, over, status):
    a = dict(cached=FAKE, new=FAKE, reqs=4, rows=8, page=64, num_pages=64, free=FAKE, num_free=10, table=FAKE, stride=8,
             cu_q=FAKE, cu_k=FAKE, visible=FAKE, slots=FAKE, taken=FAKE)
    a.update(over)
    assert lib.fp4idx_build_tables(*a.values(), None) == status


def test_binding_refuses_wrong_tensors():
    q = torch.zeros((2, 4, 576), dtype=torch.bfloat16)
    k = torch.zeros((3, 64, 576), dtype=torch.bfloat16)
    i = torch.zeros((3,), dtype=torch.int32)
    bt = torch.zeros((2, 2), dtype=torch.int32)
    ok = dict(q=q, k=k, cu_seqlens_q=i, cu_seqlens_k=i, block_table=bt, max_seqlen_q=1, max_seqlen_k=128, scale=1.0)
    for over in (dict(q=q.float()), dict(k=k.half()), dict(q=q[..., :512]), dict(k=k[:, :, :512]),
                 dict(cu_seqlens_k=i.long()), dict(cu_seqlens_k=i[:2]), dict(block_table=bt[:1]), dict(block_table=bt[0]),
                 dict(indices=torch.zeros((3, 4), dtype=torch.int32)), dict(visible_len=torch.zeros((1,), dtype=torch.int32)),
                 dict(out=torch.zeros((2, 4, 512))), dict(lse=torch.zeros((2, 5))), dict(v=k)):
        with pytest.raises(ValueError):
            binding.DeviceAttention(**{**ok, **over})
    n = torch.zeros((2,), dtype=torch.int32)
    with pytest.raises(ValueError):
        binding.fp4idx_store_latent(q[:, 0, :512], q[:, 0, :64].float(), n, k)
    with pytest.raises(ValueError):
        binding.fp4idx_store_latent(q[:, 0, :512], q[:, 0, :32], n, k)
    with pytest.raises(ValueError):
        binding.fp4idx_store_kv(q[:, :, :128], q[:, :, :128], n, k[None], k[None])
    with pytest.raises(ValueError):
        binding.fp4idx_build_tables(n, n[:1], bt, n, 64, 2)
    with pytest.raises(ValueError):
        binding.fp4idx_build_tables(n.long(), n, bt, n, 64, 2)

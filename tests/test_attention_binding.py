"""Arguments of DeviceAttention that the binding itself has to judge (no GPU needed)."""
import pytest
import torch

from fp4_sparse_attention_gb300 import binding, build


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return binding.load_library()


def arguments(latent=True, rows=2, heads=4, kv_heads=2, reqs=2):
    cache = (3, 64, 576) if latent else (3, kv_heads, 64, 128)
    i = torch.zeros((reqs + 1,), dtype=torch.int32)
    return dict(q=torch.zeros((rows, heads, cache[-1]), dtype=torch.bfloat16), k=torch.zeros(cache, dtype=torch.bfloat16),
                v=None if latent else torch.zeros(cache, dtype=torch.bfloat16), cu_seqlens_q=i, cu_seqlens_k=i,
                block_table=torch.zeros((reqs, 2), dtype=torch.int32), max_seqlen_q=1, max_seqlen_k=128, scale=1.0)


@pytest.mark.parametrize("latent", [True, False])
def test_an_empty_list_is_refused(latent):
    # an empty tensor has a null pointer, which is the C call's mark of the whole prefix
    a = arguments(latent)
    shape = (2, 0) if latent else (2, 2, 0)
    with pytest.raises(ValueError, match="at least one"):
        binding.DeviceAttention(**a, indices=torch.zeros(shape, dtype=torch.int32))
    binding.DeviceAttention(**a, indices=torch.zeros(shape[:-1] + (1,), dtype=torch.int32))


@pytest.mark.parametrize("name", ["k", "cu_seqlens_q", "cu_seqlens_k", "block_table", "visible_len", "indices", "out", "lse", "workspace"])
def test_tensors_of_another_device_are_refused(name):
    # (the meta device stands for any other device)
    more = dict(visible_len=torch.zeros((2,), dtype=torch.int32), indices=torch.zeros((2, 5), dtype=torch.int32),
                out=torch.zeros((2, 4, 512), dtype=torch.bfloat16), lse=torch.zeros((2, 4)),
                workspace=torch.zeros((1 << 20,), dtype=torch.uint8))
    a = {**arguments(), **more}
    binding.DeviceAttention(**a)
    a[name] = a[name].to("meta")
    with pytest.raises(ValueError, match="device"):
        binding.DeviceAttention(**a)


def test_host_tensors_are_refused():
    a = binding.DeviceAttention(**arguments())
    with pytest.raises(ValueError, match="CUDA"):
        binding.fp4idx_latent_attention(a)
    with pytest.raises(ValueError, match="CUDA"):
        binding.fp4idx_paged_attention(binding.DeviceAttention(**arguments(False)))
    x = torch.zeros((2, 576), dtype=torch.bfloat16)
    n = torch.zeros((2,), dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        binding.fp4idx_store_latent(x[:, :512], x[:, 512:], n, torch.zeros((1, 64, 576), dtype=torch.bfloat16))
    kv = torch.zeros((2, 2, 64, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        binding.fp4idx_store_kv(kv[:, :, 0].contiguous(), kv[:, :, 1].contiguous(), n, kv, kv.clone())
    with pytest.raises(ValueError, match="CUDA"):
        binding.fp4idx_build_tables(n, n, torch.zeros((2, 4), dtype=torch.int32), n, 64, 2)


# ---------------------------------------------------------------- strides
def accepted(a, latent=True):
    """The C call gets past its argument checks (there is no workspace, so it never launches)."""
    f = binding.load_library().fp4idx_latent_attention if latent else binding.load_library().fp4idx_paged_attention
    return f(a._ref, None, 0, None) not in (1, 2)


@pytest.mark.parametrize("latent", [True, False])
@pytest.mark.parametrize("rows,heads", [(1, 1), (1, 4), (3, 1), (3, 4)])
def test_queries_by_head_are_accepted(rows, heads, latent):
    # [H, T, d] products seen as [T, H, d]; with one row such a view is contiguous and cannot be made more so
    a = arguments(latent, rows=rows, heads=heads, kv_heads=1)
    a["q"] = torch.zeros((heads, rows, a["q"].shape[2]), dtype=torch.bfloat16).transpose(0, 1)
    assert accepted(binding.DeviceAttention(**a), latent)


def test_strides_of_dimensions_of_one_do_not_count():
    for latent in (True, False):
        a = arguments(latent, rows=1, heads=1, kv_heads=1, reqs=1)
        d, dv = a["q"].shape[2], 512 if latent else 128
        a["q"] = torch.zeros((d,), dtype=torch.bfloat16).as_strided((1, 1, d), (3, 5, 1))
        a["out"] = torch.zeros((dv,), dtype=torch.bfloat16).as_strided((1, 1, dv), (3, 5, 1))
        a["block_table"] = torch.zeros((2,), dtype=torch.int32).as_strided((1, 2), (1, 1))
        page = (1, 64, d) if latent else (1, 1, 64, d)
        strides = (7, d, 1) if latent else (7, 3, d, 1)
        a["k"] = torch.zeros((64 * d,), dtype=torch.bfloat16).as_strided(page, strides)
        if not latent:
            a["v"] = torch.zeros((64 * d,), dtype=torch.bfloat16).as_strided(page, (9, 4, d, 1))
        x = binding.DeviceAttention(**a)
        assert accepted(x, latent)
        assert x.c.table_stride == 2 and x.c.page_stride == 64 * d


def test_overlapping_queries_are_refused():
    a = arguments(True, rows=3, heads=4)
    for strides in ((576, 576, 1), (0, 576, 1), (2 * 576, 576, 1), (576, 2 * 576, 1), (576, 3 * 576 - 8, 1)):
        a["q"] = torch.zeros((1 << 14,), dtype=torch.bfloat16).as_strided((3, 4, 576), strides)
        assert not accepted(binding.DeviceAttention(**a))


# ---------------------------------------------------------------- block tables
def test_a_table_too_narrow_for_its_lengths_is_refused():
    # entries behind a row's width belong to something else, however far apart the rows are
    a = arguments()
    wide = torch.zeros((2, 8), dtype=torch.int32)
    for table in (wide[:, :1], wide[:, 7:]):
        a["block_table"] = table
        with pytest.raises(ValueError, match="block_table"):
            binding.DeviceAttention(**a)
    a["block_table"] = wide[:, 3:5]  # as many as max_seqlen_k needs
    assert accepted(binding.DeviceAttention(**a))
    a["block_table"], a["max_seqlen_k"] = wide[:, :1], 64
    assert accepted(binding.DeviceAttention(**a))


def test_tables_are_built_in_whole_rows_only():
    # the device bounds a request's pages by the distance of two rows: behind a narrower view it would write past it
    n = torch.zeros((2,), dtype=torch.int32)
    wide = torch.zeros((2, 8), dtype=torch.int32)
    with pytest.raises(ValueError, match="block_table"):
        binding.fp4idx_build_tables(n, n, wide[:, 4:], n, 64, 2)
    with pytest.raises(ValueError, match="CUDA"):  # (past that check)
        binding.fp4idx_build_tables(n, n, wide, n, 64, 2)
    with pytest.raises(ValueError, match="CUDA"):
        binding.fp4idx_build_tables(n[:1], n[:1], wide[:1, 4:], n, 64, 2)

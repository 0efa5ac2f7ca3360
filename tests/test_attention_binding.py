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

"""Keys whose score is -inf weigh nothing: the result is that of the other keys alone, to the bound that
holds for them."""
import math

import pytest
import torch

from tests import attention_ref as R
from tests.test_gpu_attention import build, call

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("kv", [None, 2])
@pytest.mark.parametrize("gone", [(0,), (1, 2), (0, 3)])  # blocks of 128 keys
def test_keys_of_minus_infinity_are_no_keys(gone, kv, dtype):
    c = R.make_case(61, [1, 2], [500, 600], heads=6, kv_heads=kv, visibility="full", dtype=dtype, device="cuda")
    c["q"] = c["q"].abs() + 0.1
    dim = 570 if kv is None else 5  # (a value that the latent form reads as a key only)
    for b, n in enumerate(c["k_lens"]):
        for s in range(n):
            if s // 128 in gone:
                page, off = c["pages"][b][s // 64], s % 64
                (c["k"][page, off] if kv is None else c["k"][page, :, off])[..., dim] = -math.inf
    left = [s for s in range(640) if s // 128 not in gone]
    listed = torch.tensor(left if kv is None else [i for i in range(5) if i not in gone], dtype=torch.int32, device="cuda")
    others = dict(c, indices=listed.expand(3, -1) if kv is None else listed.expand(kv, 3, -1))
    want, want_lse, b_out, b_lse = R.reference(others)
    assert bool(torch.isfinite(b_out).all())
    out, lse = call(build(c))
    assert bool(((out.double() - want).abs() <= b_out).all())
    assert bool(((lse.double() - want_lse).abs() <= b_lse).all())

"""Many keys of a small share beside a dominant one: what they add up to must not be lost to the 16-bit
type of the weights."""
import math

import pytest
import torch

from fp4_sparse_attention_gb300 import binding as B
from tests import attention_ref as R
from tests.test_gpu_attention import build, call

pytestmark = pytest.mark.gpu


def dominant(n, at, share, dtype, kv, seed=41):
    """One request whose key `at` has weight 1 and value 0, the n - 1 others weight 2^share and values near 100."""
    g = torch.Generator().manual_seed(seed)
    c = R.make_case(seed, [1], [n], heads=4, kv_heads=kv, visibility="full", dtype=dtype, scale=1.0, device="cuda")
    first = 512 if kv is None else 0        # score dimensions: the rotary ones of a latent key, all of a paged one
    c["q"].zero_()
    c["q"][..., first] = 1.0
    values = (100 + torch.rand((n, 512 if kv is None else 128), generator=g)).to(dtype).cuda()
    values[at] = 0
    for s in range(n):
        page, off = c["pages"][0][s // 64], s % 64
        key = c["k"][page, off] if kv is None else c["k"][page, :, off]
        key[..., first:] = 0
        key[..., first] = 0.0 if s == at else share * math.log(2)
        if kv is None:
            key[:512] = values[s]
        else:
            c["v"][page, :, off] = values[s]
    return c


@pytest.mark.parametrize("kv", [None, 2])
@pytest.mark.parametrize("n", [64, 700, 5000])
@pytest.mark.parametrize("where", ["first", "last"])
@pytest.mark.parametrize("share", [-20.3, -25.2, -28.0])
def test_fp16_shares_add_up(share, where, n, kv):
    c = dominant(n, 0 if where == "first" else n - 1, share, torch.float16, kv)
    out, lse = call(build(c))
    want, want_lse, b_out, b_lse = R.reference(c)
    # The reference's bound, which allows every weight an error of 2^-25 of the largest; here the largest is
    # at least 2^7 in a type whose smallest step is 2^-24, so 2^-32 of it.  The result may be subnormal (2^-25).
    largest = float((c["k"] if kv is None else c["v"]).nan_to_num(0)[..., :512].double().abs().amax())
    bound = b_out - n * (2.0 ** -25 - 2.0 ** -32) * largest + 2.0 ** -25
    assert bool((bound < 0.5 * want).all())  # shares that were lost would show
    off = (out.double() - want).abs()
    assert bool((off <= bound).all()), f"off by {float(off.max()):.3g}, bound {float(bound.max()):.3g}, want {float(want.min()):.3g}"
    assert bool(((lse.double() - want_lse).abs() <= b_lse).all())


@pytest.mark.parametrize("kv", [None, 2])
@pytest.mark.parametrize("keys_a_step", [64, 128])
def test_fp16_largest_weights_stay_finite(keys_a_step, kv):
    # scores that grow by just under the step that raises the reference (7.99 powers of two), tile after tile
    c = R.make_case(42, [1], [2000], heads=4, kv_heads=kv, visibility="full", dtype=torch.float16, scale=1.0, device="cuda")
    first = 512 if kv is None else 0
    c["q"].zero_()
    c["q"][..., first] = 1.0
    for s in range(2000):
        page, off = c["pages"][0][s // 64], s % 64
        key = c["k"][page, off] if kv is None else c["k"][page, :, off]
        key[..., first:] = 0
        key[..., first] = 5.54 * (s // keys_a_step)
    out, lse = call(build(c))
    want, want_lse, b_out, b_lse = R.reference(c)
    assert bool(((out.double() - want).abs() <= b_out).all()) and bool(((lse.double() - want_lse).abs() <= b_lse).all())

"""Prompt attention with queries and scores of extreme size."""
import pytest
import torch

from packed_ref import Packed, check_close

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,ctx", [([1, 1], [40, 300]), ([3, 40], [130, 20]), ([200], [77])])
@pytest.mark.parametrize("k_scale", [1.0, 2.0 ** 40])
@pytest.mark.parametrize("power", [116, 117, 126, 127, -126, -133])
def test_a_channel_of_any_size_over_zero_codes(d, lens, ctx, k_scale, power):
    """Over the 4-bit cache a query is divided by the power of two of its largest
    channel, any that bf16 has, subnormal ones too. Here that channel meets keys of
    zero: every score is zero, every key counts alike."""
    p = Packed(lens, ctx, 8, 2, d, 16, 4, seed=66, k_scale=k_scale)
    p.fill_context()
    p.fill_new()
    for r, (n, c) in enumerate(zip(p.lens, p.ctx)):
        k, v = p._normal(n + c, 2, d).bfloat16(), p._normal(n + c, 2, d).bfloat16()
        k[..., 3] = 0
        p.put(r, 0, n + c, k, v)
    p.q.zero_()
    p.q[..., 3] = -1.5 * 2.0 ** power if power > -100 else 2.0 ** power
    got = p.attend()
    want, tol = p.attention64()
    check_close(got, want, tol)
    assert p.h.ddt_device_status() == 0

"""The 4-bit append's block scales next to the midpoints of e4m3: the scale is the
number nearest to the fp32 quotient amax / (6 g), not to a product with 1 / (6 g),
which lands on a midpoint from one step below it."""
import numpy as np
import pytest
import torch

from packed_ref import MAGS, Packed, e4m3, e4m3_value
from speculative_decoding_draft_depth_gb300 import ddt

pytestmark = pytest.mark.gpu

F = np.float32


def maxima(g):
    """fp32 numbers within two steps of 6 g t, t each midpoint of e4m3 (subnormal ones too)."""
    grid = np.unique(e4m3_value(np.arange(0x7f, dtype=np.uint8)).astype(np.float64))  # 0 .. 448
    out = []
    for t in (grid[1:] + grid[:-1]) / 2:
        a = F(t * float(F(6) * F(g)))
        lo = np.nextafter(np.nextafter(a, F(0)), F(0))
        for _ in range(5):
            out.append(lo)
            lo = np.nextafter(lo, F(np.inf))
    return np.array(out, F)


@pytest.mark.parametrize("g", [1.0, 0.37, 2.0 ** -40, 2.0 ** 40, 1.0 / 1024])
def test_scales_next_to_midpoints(g):
    amax = maxima(g)
    n = len(amax)
    p = Packed([n], [0], 4, 2, 64, 16, 4, seed=61, k_scale=g)
    # keys of ones and zeros, turned by a table of cosines that hold the wanted values: x1' = cos
    p.k.zero_()
    p.k[..., :16] = 1.0
    cos = np.zeros((n, 64), F)
    cos[:, :16] = amax[:, None] * np.linspace(1.0, 0.05, 16, dtype=F)
    cos[:, 0] = amax
    p.append(ddt.Rotary(torch.from_numpy(cos).cuda(), 64))
    assert p.h.ddt_device_status() == 0
    pg, row = p.slots(0, 0, n)
    want = e4m3(np.minimum(amax / (F(6) * F(g)), F(448)))
    product = e4m3(np.minimum(amax * (F(1) / (F(6) * F(g))), F(448)))
    assert g != 1.0 or (want != product).sum() >= 14  # (the difference is there to be seen)
    got = p.kv4.k_scales[pg, :, row].cpu().numpy()
    assert (got[:, :, 0] == want[:, None]).all()
    assert (got[:, :, 1:] == 0).all()
    # the codes belong to that scale
    s = (e4m3_value(want) * F(g))[:, None]
    with np.errstate(divide="ignore", invalid="ignore"):
        a = cos[:, :16] / s
    m = ((a > .25).astype(np.uint8) + (a >= .75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5))
    m = np.where(s > 0, m, 0)
    c = p.kv4.k_codes[pg, :, row].cpu().numpy()[:, 0, :8].reshape(n, 2, 4)
    held = np.stack((c[..., 0] & 15, c[..., 2] & 15, c[..., 0] >> 4, c[..., 2] >> 4,
                     c[..., 1] & 15, c[..., 3] & 15, c[..., 1] >> 4, c[..., 3] >> 4), -1).reshape(n, 16)
    assert (held == m).all() and (MAGS[held] * s >= 0).all()

"""Prompt attention with queries and scores of extreme size."""
import pytest
import torch

from packed_ref import SENTINEL, Packed, check_close

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


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,ctx", [([1, 1], [40, 3000]), ([3, 40], [700, 20]), ([300], [900])])
def test_scores_of_the_largest_size(bits, d, lens, ctx):
    """Scores up to 2^20, of one channel alone (the products and their sums are exact),
    so far apart that every key but the row's highest has no weight; keys that tie
    have the same one. What is left of the tolerance: the tied probabilities are
    rounded alike (2^-8 of the result), the result is rounded (2^-8), the fp32 sums
    and the quotient add 2^-20 of sum p |v|. (The largest score is 0.66 of 2^20 at
    d = 64, 0.93 at 128.)"""
    p = Packed(lens, ctx, 8, 2, d, 16, bits, seed=67)
    p.fill_context()
    p.fill_new()
    top = 2688.0  # the largest value of a 4-bit block
    qv = 2.0 ** 20 / top * d ** 0.5
    qv = 2.0 ** int(torch.log2(torch.tensor(qv)))  # a power of two below it
    p.q.zero_()
    p.q[..., 0] = qv
    p.q[:, 1::2, 0] = -qv
    for r, (n, c) in enumerate(zip(p.lens, p.ctx)):
        k, v = torch.zeros(n + c, 2, d, device="cuda"), p._normal(n + c, 2, d).bfloat16()
        # -top .. top in steps of which many keys share one; from 448 / 2 * the block's scale on they are held exactly
        levels = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device="cuda") * 448
        g = torch.Generator().manual_seed(68 + r)
        at = (torch.rand(n + c, 2, generator=g) * 8).long().cuda()
        sign = torch.where(torch.rand(n + c, 2, generator=g) < 0.5, -1.0, 1.0).cuda()
        k[..., 0] = levels[at] * sign
        k[..., 1] = top  # (fixes the block's scale; the query does not look at it)
        p.put(r, 0, n + c, k.bfloat16(), v)
        kk, _ = p.rows(r, n + c)
        assert torch.equal(kk[..., 0], k[..., 0].double())  # held exactly
    got = p.attend()
    out = torch.full(got.shape, SENTINEL, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(out)
    for r, (n, c) in enumerate(zip(p.lens, p.ctx)):
        s0 = int(p.starts[r])
        k, v = p.rows(r, c + n)
        for i in range(n):
            seen = c + i + 1
            for h in range(8):
                s = float(p.q[s0 + i, h, 0]) * k[:seen, h // 4, 0]
                tied = v[:seen, h // 4][s == s.max()]
                o, A = tied.mean(0), tied.abs().mean(0)
                out[s0 + i, h] = o
                tol[s0 + i, h] = 1.01 * (2 * 2.0 ** -8 * o.abs() + 2.0 ** -20 * A)
    check_close(got, out, tol)
    assert p.h.ddt_device_status() == 0

"""Rows that two requests of an append name (q_start fell between them): the
later request has them whole, and no slot that neither names changes."""
import numpy as np
import pytest
import torch

from packed_ref import SENTINEL, Packed, quantise, turn
from speculative_decoding_draft_depth_gb300 import ddt

pytestmark = pytest.mark.gpu


def bits(t):
    return t.view(torch.int16) if t.dtype == torch.bfloat16 else t


@pytest.mark.parametrize("kv", [16, 4])
@pytest.mark.parametrize("between", [1, 45, 300])
@pytest.mark.parametrize("first_later", [False, True])
def test_the_later_request_has_the_row(kv, between, first_later):
    """Two requests far apart (looked at by one thread's neighbour, by another
    warp, in another turn of the scan) both name rows 2 .. 5; the requests in
    between are empty but for the one where q_start falls, which is skipped."""
    R = between + 2
    ctx = [4] * R
    ctx[0], ctx[-1] = (90, 40) if first_later else (40, 90)
    # the later request's range begins at row 2: rows 2 .. 8 are its own
    lens = [6] + [0] * between + [7]
    p = Packed(lens, ctx, 8, 2, 64, 16, kv, seed=60, tail=2, stale=0.0)
    p.fill_context()
    starts = [0] + [6] * between + [2, 9]
    p.q_start.copy_(torch.tensor(starts, dtype=torch.int32))
    rot = ddt.rotary_table(128, 64)
    table = rot.cpu().numpy()
    T = p.T
    pools = (p.k_cache, p.v_cache) if kv == 16 else (p.kv4.k_codes, p.kv4.v_codes, p.kv4.k_scales, p.kv4.v_scales)
    after = [t.clone() for t in pools]
    want_q = torch.full((T, 8, 64), SENTINEL).bfloat16()
    held = [torch.full((T, 2, 64), SENTINEL, device="cuda").bfloat16() for _ in range(2)]
    want_held = [h.cpu() for h in held]
    rows = {t: (0, ctx[0] + t) for t in range(2)}
    rows.update({t: (R - 1, ctx[-1] + t - 2) for t in range(2, 9)})
    for t, (r, pos) in rows.items():
        q, k, v = (x[t:t + 1].float().cpu().numpy() for x in (p.q, p.k, p.v))
        q, k = (turn(x, np.array([pos]), table, 64, False) for x in (q, k))
        want_q[t] = torch.from_numpy(q[0]).bfloat16()
        pg, row = (int(x[0]) for x in p.slots(r, pos, pos + 1))
        for i, x in enumerate((k, v)):
            if kv == 16:
                after[i][pg, row] = torch.from_numpy(x[0]).bfloat16().cuda()
            else:
                codes, scales, val = quantise(x[0], 1.0)
                after[i][pg, :, row] = torch.from_numpy(codes).cuda()
                after[2 + i][pg, :, row] = torch.from_numpy(scales).cuda()
                want_held[i][t] = torch.from_numpy(val).bfloat16()
    before = [t.clone() for t in pools]
    kw = dict(k_held=held[0], v_held=held[1]) if kv == 4 else {}
    for _ in range(20):
        for t, b in zip(pools, before):
            t.copy_(b)
        new = torch.zeros(R, dtype=torch.int32, device="cuda")
        qo = p.append(ddt.Rotary(rot, 64), new_lens=new, **kw)
        assert p.h.ddt_device_status() == ddt.DEV_BAD_LENGTH
        assert torch.equal(bits(qo).cpu(), bits(want_q))
        for g, w in zip(pools, after):
            assert torch.equal(bits(g), bits(w))
        if kv == 4:
            for g, w in zip(held, want_held):
                assert torch.equal(bits(g).cpu(), bits(w))
        assert new.tolist() == [ctx[0] + 6] + ctx[1:-1] + [ctx[-1] + 7]

"""ddt_append_kv / ddt_append_kvq on the GPU: rows, codes and scales equal the
header's formula bit for bit, nothing else of the pool changes, and what the
calls refuse or skip."""
import ctypes

import numpy as np
import pytest
import torch

from packed_ref import SENTINEL, Packed, quantise, turn
from speculative_decoding_draft_depth_gb300 import ddt

pytestmark = pytest.mark.gpu


def bits(t):
    return t.view(torch.int16) if t.dtype == torch.bfloat16 else t


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x)).bfloat16()


def state(p):
    return [t.clone() for t in ((p.k_cache, p.v_cache) if p.bits == 16 else
                                (p.kv4.k_codes, p.kv4.v_codes, p.kv4.k_scales, p.kv4.v_scales))]


def expect(p, before, rot, inter, table, q=None, skip=()):
    """The pool and q_out after an append, from the pool before it."""
    q = p.q if q is None else q
    qo = torch.full((p.T, p.Hq, p.d), SENTINEL).bfloat16()
    after = [t.cpu().clone() for t in before]
    held = [torch.full((p.T, p.Hkv, p.d), SENTINEL).bfloat16() for _ in range(2)]
    for r, (n, c) in enumerate(zip(p.lens, p.ctx)):
        if n == 0 or r in skip:
            continue
        s, pos = int(p.starts[r]), np.arange(c, c + n)
        one = [x[s:s + n].float().cpu().numpy() for x in (q, p.k, p.v)]
        if rot:
            one[0], one[1] = (turn(x, pos, table, rot, inter) for x in one[:2])
        qo[s:s + n] = bf16(one[0])
        pg, row = (x.cpu() for x in p.slots(r, c, c + n))
        for i in range(2):
            if p.bits == 16:
                after[i][pg, row] = bf16(one[1 + i])
            else:
                codes, scales, val = quantise(one[1 + i], (p.kv4.k_scale, p.kv4.v_scale)[i])
                after[i][pg, :, row] = torch.from_numpy(codes)
                after[2 + i][pg, :, row] = torch.from_numpy(scales)
                held[i][s:s + n] = bf16(val)
    return qo, after, held


def check(p, rot, inter, **kw):
    table = ddt.rotary_table(max(c + n for c, n in zip(p.ctx, p.lens)) + 1, rot) if rot else None
    before = state(p)
    if p.bits == 4:
        held = [torch.full((p.T, p.Hkv, p.d), SENTINEL, device="cuda").bfloat16() for _ in range(2)]
        kw.update(k_held=held[0], v_held=held[1])
    new = torch.full((p.R,), -5, dtype=torch.int32, device="cuda")
    qo = p.append(ddt.Rotary(table, rot, inter) if rot else None, new_lens=new, **kw)
    want_q, want, want_held = expect(p, before, rot, inter, table.cpu().numpy() if rot else None)
    assert p.h.ddt_device_status() == 0
    assert torch.equal(bits(qo).cpu(), bits(want_q))
    for g, w in zip(state(p), want):
        assert torch.equal(bits(g).cpu(), bits(w))
    if p.bits == 4:
        for g, w in zip(held, want_held):
            g = g.cpu()
            # (a NaN's sign and payload say nothing)
            assert bool(((bits(g) == bits(w)) | (g.isnan() & w.isnan())).all())
    assert new.tolist() == [c + n for c, n in zip(p.ctx, p.lens)]


@pytest.mark.parametrize("kv", [16, 4])
@pytest.mark.parametrize("lens,ctx,Hq,Hkv,d,page,rot,inter", [
    ([1], [0], 4, 1, 64, 16, 64, False),
    ([1, 1, 1], [15, 16, 4000], 32, 8, 128, 16, 128, False),
    ([5, 0, 33, 1, 0], [0, 7, 13, 100, 0], 8, 2, 64, 16, 32, True),
    ([17, 3], [31, 64], 16, 1, 128, 32, 96, False),
    ([2, 70, 9], [3, 250, 0], 5, 5, 128, 256, 64, False),
    ([40, 1], [1, 30], 6, 3, 64, 64, 0, False),
    ([300], [77], 2, 2, 128, 16, 128, True),
    ([0, 0], [3, 0], 4, 1, 64, 16, 64, False),
])
def test_append_is_exact(kv, lens, ctx, Hq, Hkv, d, page, rot, inter):
    check(Packed(lens, ctx, Hq, Hkv, d, page, kv, seed=3, lead=2, tail=3), rot, inter)


@pytest.mark.parametrize("kv", [16, 4])
def test_append_of_many_requests(kv):
    """More requests than a CTA has threads, most of one or no token."""
    rng = np.random.default_rng(5)
    check(Packed(rng.integers(0, 4, 700).tolist(), rng.integers(0, 60, 700).tolist(), 4, 2, 64, 16, kv, seed=4), 64,
          False)


def test_global_scales():
    check(Packed([9, 20], [3, 40], 4, 2, 128, 16, 4, seed=6, k_scale=0.37, v_scale=1.0 / 1024, v_gain=1e-3), 128,
          False)


def test_blocks_of_every_kind():
    """Zero blocks, ties between codes, values past the largest, subnormal and
    NaN blocks: codes and scales follow the rule."""
    p = Packed([24], [0], 4, 2, 64, 16, 4, seed=7)
    x = p.k.float()
    x[0] = 0.0
    x[1] = -0.0
    x[2, :, :16] = torch.tensor([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, 0])
    x[3] = 1e5
    x[4] = float("inf")
    x[5, 0, 3] = float("nan")
    x[6] *= 2.0 ** -9
    x[7] *= 2.0 ** -11
    x[8] *= 2.0 ** -130
    x[9, 0, 20], x[9, 1, 40] = -float("inf"), 2688.0
    p.k.copy_(x)
    p.v.copy_(x.flip(0))
    check(p, 0, False)


def test_strided_rows_and_in_place():
    p = Packed([5, 40], [9, 100], 8, 2, 128, 16, 16, seed=8)
    rows = torch.cat([x.flatten(1) for x in (p.q, p.k, p.v)], 1)
    q, k, v = (x.unflatten(1, (-1, 128)) for x in rows.split((8 * 128, 256, 256), 1))
    assert not k.is_contiguous()
    check(p, 128, False, q=q, k=k, v=v)
    # in place: q_out is q
    table = ddt.rotary_table(200, 128)
    want, _, _ = expect(p, state(p), 128, False, table.cpu().numpy())
    q = p.q.clone()
    p.append(ddt.Rotary(table, 128), q=q, q_out=q)
    assert torch.equal(bits(q).cpu(), bits(want))


@pytest.mark.parametrize("kv", [16, 4])
def test_keys_alone(kv):
    p = Packed([3, 8], [2, 9], 8, 2, 64, 16, kv, seed=9)
    table = ddt.rotary_table(64, 64)
    before = state(p)
    kw = dict(q=None, q_out=None)
    p.append(ddt.Rotary(table, 64), **kw)
    _, want, _ = expect(p, before, 64, False, table.cpu().numpy())
    for g, w in zip(state(p), want):
        assert torch.equal(bits(g).cpu(), bits(w))


@pytest.mark.parametrize("kv", [16, 4])
def test_bad_pages_drop_their_rows(kv):
    p = Packed([20, 20], [0, 0], 4, 2, 64, 16, kv, seed=10)
    before = state(p)
    p.table[0, 0], p.table[1, 1] = p.num_pages, -1
    good = [(0, 16, 20), (1, 0, 16)]
    p.append()
    assert p.h.ddt_device_status() == ddt.DEV_BAD_PAGE
    want = [t.clone() for t in before]
    for r, a, b in good:
        pg, row = p.slots(r, a, b)
        s = int(p.starts[r])
        for i, x in enumerate((p.k, p.v)):
            if kv == 16:
                want[i][pg, row] = x[s + a:s + b]
            else:
                c, sc, _ = quantise(x[s + a:s + b].float().cpu().numpy(), 1.0)
                want[i][pg, :, row] = torch.from_numpy(c).cuda()
                want[2 + i][pg, :, row] = torch.from_numpy(sc).cuda()
    for g, w in zip(state(p), want):
        assert torch.equal(bits(g), bits(w))


@pytest.mark.parametrize("kind", ["negative", "past_the_table", "past_the_angles", "descending", "past_T"])
def test_bad_lengths_skip_their_request(kind):
    p = Packed([4, 6, 5], [3, 8, 2], 4, 2, 64, 16, 16, seed=11)
    table = ddt.rotary_table(14 if kind != "past_the_angles" else 13, 64)
    before, skip = state(p), (1,)
    if kind == "negative":
        p.ctx_lens[1] = -1
    elif kind == "past_the_table":
        p.ctx_lens[1] = p.max_pages * p.page - 5
    elif kind == "descending":
        p.q_start[2] = 3
        p.lens[2], p.starts = 12, np.array([0, 4, 3, 15])  # request 2 now begins at row 3
        skip = None
    elif kind == "past_T":
        p.q_start[3] = 99
        skip = (2,)
    new = torch.zeros(3, dtype=torch.int32, device="cuda")
    qo = p.append(ddt.Rotary(table, 64), new_lens=new)
    assert p.h.ddt_device_status() == ddt.DEV_BAD_LENGTH
    if skip is None:
        # row 3 belongs to two requests; the others' rows are as they should be
        assert bool((bits(qo)[4:] != bits(torch.full_like(qo, SENTINEL))[4:]).any())
        return
    want_q, want, _ = expect(p, before, 64, False, table.cpu().numpy(), skip=skip)
    assert torch.equal(bits(qo).cpu(), bits(want_q))
    for g, w in zip(state(p), want):
        assert torch.equal(bits(g).cpu(), bits(w))
    ctx = p.ctx_lens.tolist()
    assert new.tolist() == [c if r in skip else c + n for r, (c, n) in enumerate(zip(ctx, p.lens))]


def test_refusals():
    p = Packed([4, 4], [0, 3], 4, 2, 64, 16, 16, seed=12)
    lib = ddt.load()
    fake = p.h.alloc_kv4()

    def call(**kw):
        qs, ks, vs = 0, 0, 0
        a = p.h._append_args(p.q, p.k, p.v, p.q_start, p.ctx_lens, p.table, p.R, torch.empty_like(p.q),
                             ddt.Rotary(ddt.rotary_table(64, 64), 64), None)
        a.q_stride, a.k_stride, a.v_stride = qs, ks, vs
        for n, v in kw.items():
            if n not in ("kc", "cache"):
                setattr(a, n, v)
        if "cache" in kw:
            return lib.ddt_append_kvq(p.h._h, ctypes.byref(a), ctypes.byref(kw["cache"]), None, None, None)
        return lib.ddt_append_kv(p.h._h, ctypes.byref(a), kw.get("kc", p.k_cache.data_ptr()), p.v_cache.data_ptr(),
                                 None)

    assert call() == ddt.OK
    q = p.q.data_ptr()
    for bad in (dict(R=3), dict(R=-1), dict(T=-1), dict(T=2 ** 31 - 1), dict(q_stride=8), dict(k_stride=129),
                dict(v_stride=-128), dict(k=None), dict(v=None), dict(q_start=None), dict(ctx_lens=None),
                dict(block_table=None), dict(q_out=None), dict(q=None), dict(k=p.k.data_ptr() + 2),
                dict(q_out=q + 16), dict(q_out=p.k.data_ptr()), dict(q_out=p.v.data_ptr()),
                dict(q_start=p.q_start.data_ptr() + 2), dict(new_lens=p.ctx_lens.data_ptr()),
                dict(new_lens=p.ctx_lens.data_ptr() + 4), dict(rotary_dim=48), dict(rotary_dim=0),
                dict(rotary_dim=96), dict(max_pos=0), dict(interleaved=2), dict(kc=None),
                dict(kc=p.k_cache.data_ptr() + 8)):
        assert call(**bad) == ddt.EINVAL, bad
    k4 = p.h._kv4(fake)
    assert call(cache=k4) == ddt.OK
    for name, v in (("k_codes", None), ("v_scales", None), ("v_codes", fake.v_codes.data_ptr() + 8),
                    ("k_scale", 0.0), ("k_scale", float("nan")), ("v_scale", float("inf")), ("v_scale", -1.0)):
        bad = p.h._kv4(fake)
        setattr(bad, name, v)
        assert call(cache=bad) == ddt.EINVAL, (name, v)
    # what the cache holds is written apart from every other tensor
    qo = torch.empty_like(p.q)
    args = p.h._append_args(p.q, p.k, p.v, p.q_start, p.ctx_lens, p.table, p.R, qo, None, None)
    kh, vh = torch.empty_like(p.k), torch.empty_like(p.v)

    def held(k, v):
        return lib.ddt_append_kvq(p.h._h, ctypes.byref(args), ctypes.byref(k4), k, v, None)

    assert held(kh.data_ptr(), vh.data_ptr()) == ddt.OK
    for k, v in ((kh.data_ptr(), None), (kh.data_ptr(), kh.data_ptr()), (p.k.data_ptr(), vh.data_ptr()),
                 (kh.data_ptr(), p.v.data_ptr()), (kh.data_ptr(), args.q_out), (p.q.data_ptr(), vh.data_ptr()),
                 (kh.data_ptr() + 8, vh.data_ptr())):
        assert held(k, v) == ddt.EINVAL
    with pytest.raises(ValueError):
        p.append(k=p.k.cpu())
    torch.cuda.synchronize()
    assert p.h.ddt_device_status() == 0


def test_no_rows():
    """T = 0: only the lengths are written; R = 0: nothing."""
    p = Packed([0, 0], [5, 2], 4, 2, 64, 16, 16, seed=13)
    new = torch.full((2,), -1, dtype=torch.int32, device="cuda")
    p.append(ddt.Rotary(ddt.rotary_table(8, 64), 64), new_lens=new)
    assert new.tolist() == [5, 2]
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    p.h.ddt_append_kv(None, p.k, p.v, torch.zeros(1, dtype=torch.int32, device="cuda"), e, p.table[:0], 0, p.k_cache,
                      p.v_cache)
    assert p.h.ddt_device_status() == 0


def test_slots_past_32_bits():
    """A pool of more than 2^32 bytes (2^31 elements): rows at its end."""
    p = Packed([3], [30], 8, 8, 128, 16, 16, seed=14, stale=0.0, extra_pages=2 ** 31 // (16 * 8 * 128) + 4)
    p.table[0, :3] = torch.tensor([p.num_pages - 1, p.num_pages - 3, p.num_pages - 2], dtype=torch.int32)
    p.append()
    for r, a, b in ((0, 30, 33),):
        pg, row = p.slots(r, a, b)
        assert torch.equal(p.k_cache[pg, row], p.k) and torch.equal(p.v_cache[pg, row], p.v)
    assert int((bits(p.k_cache[:-3]) != 0).any()) == 0
    assert p.h.ddt_device_status() == 0

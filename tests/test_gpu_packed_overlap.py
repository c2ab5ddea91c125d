"""What the packed calls write must lie apart from what they read and from each
other: every pair that a call could race on is refused before anything runs."""
import ctypes

import pytest
import torch

from packed_ref import Packed
from speculative_decoding_draft_depth_gb300 import ddt

pytestmark = pytest.mark.gpu


def at(t):
    return t.data_ptr()


def case(kv, seed):
    p = Packed([4, 4], [0, 3], 4, 2, 64, 16, kv, seed=seed)
    return p, ddt.load()


def append_call(p, lib, pools, held=(None, None), **kw):
    qo = torch.empty_like(p.q)
    a = p.h._append_args(p.q, p.k, p.v, p.q_start, p.ctx_lens, p.table, p.R, qo,
                         ddt.Rotary(ddt.rotary_table(64, 64), 64), None)
    for n, v in kw.items():
        assert hasattr(a, n)
        setattr(a, n, v)
    if p.bits == 16:
        return lib.ddt_append_kv(p.h._h, ctypes.byref(a), pools[0], pools[1], None)
    c = p.h._kv4(p.kv4)
    for n, v in zip(("k_codes", "v_codes", "k_scales", "v_scales"), pools):
        setattr(c, n, v)
    return lib.ddt_append_kvq(p.h._h, ctypes.byref(a), ctypes.byref(c), held[0], held[1], None)


def pools_of(p):
    return (p.k_cache, p.v_cache) if p.bits == 16 else (p.kv4.k_codes, p.kv4.v_codes, p.kv4.k_scales, p.kv4.v_scales)


@pytest.mark.parametrize("kv", [16, 4])
def test_append(kv):
    p, lib = case(kv, 62)
    good = [at(t) for t in pools_of(p)]
    before = [t.clone() for t in pools_of(p)]
    new = torch.empty(p.R, dtype=torch.int32, device="cuda")
    # the lengths after the call: over the requests' rows, lengths and pages, the tokens, a pool
    for t in (p.q_start, p.ctx_lens, p.table, p.q, p.k, p.v) + pools_of(p):
        for off in (0, 4):
            assert append_call(p, lib, good, new_lens=at(t) + off) == ddt.EINVAL
    # the angles: the last bytes of the table
    rot = ddt.rotary_table(64, 64)
    assert append_call(p, lib, good, cos_sin=at(rot), new_lens=at(rot) + 64 * 64 * 4 - 4) == ddt.EINVAL
    assert append_call(p, lib, good, cos_sin=at(rot), q_out=at(rot)) == ddt.EINVAL
    # queries over a pool, another's pool, or the tables
    for t in pools_of(p) + (p.q_start, p.table):
        if at(t) % 16 == 0:
            assert append_call(p, lib, good, q_out=at(t)) == ddt.EINVAL
    # keys, values and queries that lie in a pool
    for n in ("q", "k", "v"):
        assert append_call(p, lib, good, **{n: good[0]}) == ddt.EINVAL
    # two pools that are one, or that share their last 16 bytes
    for i in range(len(good)):
        for j in range(i):
            for off in (0, pools_of(p)[j].numel() * pools_of(p)[j].element_size() - 16):
                bad = list(good)
                bad[i] = good[j] + off
                assert append_call(p, lib, bad) == ddt.EINVAL, (i, j, off)
    if kv == 4:
        kh, vh = torch.empty_like(p.k), torch.empty_like(p.v)
        for t in pools_of(p) + (p.q_start, p.table):
            if at(t) % 16 == 0:
                assert append_call(p, lib, good, held=(at(t), at(vh))) == ddt.EINVAL
                assert append_call(p, lib, good, held=(at(kh), at(t))) == ddt.EINVAL
        assert append_call(p, lib, good, held=(at(kh), at(vh)), new_lens=at(vh)) == ddt.EINVAL
    torch.cuda.synchronize()
    for t, b in zip(pools_of(p), before):
        assert torch.equal(t.view(torch.uint8), b.view(torch.uint8))
    # what lies side by side, and queries turned in place, are as good as before
    assert append_call(p, lib, good, new_lens=at(new), q=at(p.q), q_out=at(p.q)) == ddt.OK
    assert new.tolist() == [4, 7] and p.h.ddt_device_status() == 0


@pytest.mark.parametrize("kv", [16, 4])
def test_attention(kv):
    p, lib = case(kv, 63)
    p.fill_context()
    p.fill_new()
    before = [t.clone() for t in pools_of(p)]

    def call(o):
        if kv == 16:
            return lib.ddt_prompt_attention(p.h._h, at(p.q), 0, at(p.q_start), at(p.ctx_lens), p.R, p.T, at(p.k_cache),
                                            at(p.v_cache), at(p.table), o, None)
        c = p.h._kv4(p.kv4)
        return lib.ddt_prompt_attention_kvq(p.h._h, at(p.q), 0, at(p.q_start), at(p.ctx_lens), p.R, p.T,
                                            ctypes.byref(c), at(p.table), o, None)

    for t in pools_of(p) + (p.q, p.q_start, p.ctx_lens, p.table):
        last = (t.numel() * t.element_size() - 1) // 16 * 16
        for o in (at(t), at(t) + last):
            if o % 16 == 0:
                assert call(o) == ddt.EINVAL
    torch.cuda.synchronize()
    for t, b in zip(pools_of(p), before):
        assert torch.equal(t.view(torch.uint8), b.view(torch.uint8))
    out = torch.empty_like(p.q)
    assert call(at(out)) == ddt.OK and p.h.ddt_device_status() == 0
    # one pool for both keys and values is only read
    if kv == 16:
        p.h.ddt_prompt_attention(p.q, p.q_start, p.ctx_lens, p.table, p.R, p.k_cache, p.k_cache, out)
        assert p.h.ddt_device_status() == 0

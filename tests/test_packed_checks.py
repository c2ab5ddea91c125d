"""The packed-sequence operators' host side, without a GPU: the layout of their
argument structures, the binding's checks of types and shapes, the library's
refusal of a missing context, the rotation table, and which requests' lengths
the kernels take (the header's plain function, compiled here)."""
import ctypes
import os
import subprocess
import types

import numpy as np
import pytest
import torch

from speculative_decoding_draft_depth_gb300 import build as ddt_build
from speculative_decoding_draft_depth_gb300 import ddt

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "speculative_decoding_draft_depth_gb300", "csrc")


@pytest.fixture(scope="module")
def lib():
    ddt_build.build()
    return ddt.load()


def _run_c(tmp_path, body, cxx=False):
    src = tmp_path / ("a.cpp" if cxx else "a.c")
    src.write_text(body)
    exe = str(tmp_path / "a")
    subprocess.run(["g++" if cxx else "gcc", "-I", os.path.join(ROOT, "include"), "-I", CSRC, str(src), "-o", exe],
                   check=True)
    return subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split()


def test_structures_match_the_header(tmp_path):
    for name, st in (("ddt_append_args", ddt.AppendArgs), ("ddt_kv4", ddt.Kv4)):
        fields = [f for f, _ in st._fields_]
        out = _run_c(tmp_path, '#include <stdio.h>\n#include <stddef.h>\n#include "ddt.h"\nint main(void) {\n' +
                     "".join('printf("%%zu\\n", offsetof(%s, %s));\n' % (name, f) for f in fields) +
                     'printf("%%zu\\n", sizeof(%s));return 0;}\n' % name)
        assert [int(x) for x in out] == [getattr(st, f).offset for f in fields] + [ctypes.sizeof(st)], name


def test_packed_ok(tmp_path):
    """Against the same rule in unbounded integers, at the limits of 32 bits."""
    big = 2 ** 31 - 1
    vals = [-2 ** 31, -1, 0, 1, 5, 6, 7, big - 1, big]
    rows = [(a, b, T, c, cap) for a in vals for b in vals for T in (0, 6, big) for c in vals for cap in (1, 6, big)]
    body = '#include <stdio.h>\n#include "packed_seq.h"\nstatic int x[][5] = {%s};\nint main() {\n' % ",".join(
        "{%s}" % ",".join("(-2147483647-1)" if v == -2 ** 31 else str(v) for v in r) for r in rows)
    body += 'for (auto &r : x) printf("%d\\n", (int)packed_ok(r[0], r[1], r[2], r[3], r[4]));return 0;}\n'
    got = [int(x) for x in _run_c(tmp_path, body, cxx=True)]
    want = [int(0 <= a <= b <= T and c >= 0 and c + b - a <= cap) for a, b, T, c, cap in rows]
    assert got == want


def _cfg():
    return types.SimpleNamespace(R_max=4, Hq=8, Hkv=2, d=64, page_size=16, max_pages_per_req=3, num_pages=9)


def _tensors(T=6, R=2):
    bf = dict(dtype=torch.bfloat16)
    i32 = dict(dtype=torch.int32)
    return dict(q=torch.zeros(T, 8, 64, **bf), k=torch.zeros(T, 2, 64, **bf), v=torch.zeros(T, 2, 64, **bf),
                q_start=torch.zeros(R + 1, **i32), ctx_lens=torch.zeros(R, **i32),
                block_table=torch.zeros(R, 3, **i32), R=R, q_out=torch.zeros(T, 8, 64, **bf), rotary=None,
                new_lens=None)


def test_strides_of_a_fused_projection():
    t = _tensors()
    rows = torch.zeros(6, (8 + 2 + 2) * 64, dtype=torch.bfloat16)
    t["q"], t["k"], t["v"] = (x.unflatten(1, (-1, 64)) for x in rows.split((512, 128, 128), 1))
    assert ddt.check_append(_cfg(), **t) == (768, 768, 768)
    assert ddt.check_append(_cfg(), **_tensors()) == (0, 0, 0)  # (dense)
    # one row has no next one: its stride says nothing
    t = _tensors(T=1)
    t["k"] = torch.zeros(1, 2, 64, dtype=torch.bfloat16).as_strided((1, 2, 64), (1, 64, 1))
    assert ddt.check_append(_cfg(), **t)[1] == 0


@pytest.mark.parametrize("name,value", [
    ("q", torch.zeros(6, 8, 64)), ("q", None), ("q_out", None), ("q", torch.zeros(5, 8, 64, dtype=torch.bfloat16)),
    ("k", torch.zeros(6, 3, 64, dtype=torch.bfloat16)), ("v", torch.zeros(6, 2, 32, dtype=torch.bfloat16)),
    ("v", torch.zeros(6, 64, 2, dtype=torch.bfloat16).transpose(1, 2)),
    ("k", torch.zeros(6, 4, 64, dtype=torch.bfloat16)[:, ::2]),
    ("q_start", torch.zeros(2, dtype=torch.int32)), ("q_start", torch.zeros(3, dtype=torch.int64)),
    ("ctx_lens", torch.zeros(3, dtype=torch.int32)), ("block_table", torch.zeros(2, 4, dtype=torch.int32)),
    ("new_lens", torch.zeros(1, dtype=torch.int32)), ("R", 5), ("R", -1),
    ("rotary", ddt.Rotary(torch.zeros(4, 48), 48)), ("rotary", ddt.Rotary(torch.zeros(4, 96), 96)),
])
def test_append_shapes_are_checked(name, value):
    t = _tensors()
    t[name] = value
    with pytest.raises(ValueError):
        ddt.check_append(_cfg(), **t)


@pytest.mark.parametrize("name,value", [
    ("q", torch.zeros(6, 8, 64)), ("out", torch.zeros(6, 8, 64)), ("out", torch.zeros(7, 8, 64, dtype=torch.bfloat16)),
    ("q", torch.zeros(6, 64, 8, dtype=torch.bfloat16).transpose(1, 2)), ("R", 9),
])
def test_prompt_shapes_are_checked(name, value):
    t = {k: v for k, v in _tensors().items() if k in ("q", "q_start", "ctx_lens", "block_table", "R")}
    t["out"] = torch.zeros(6, 8, 64, dtype=torch.bfloat16)
    assert ddt.check_prompt(_cfg(), **t) == 0
    t[name] = value
    with pytest.raises(ValueError):
        ddt.check_prompt(_cfg(), **t)


@pytest.mark.parametrize("name", ["q", "k", "v"])
def test_rows_that_share_memory_are_refused(name):
    """One row expanded over the tokens, and rows that begin inside the last one:
    a stride of 0 would otherwise stand for dense rows."""
    heads = 8 if name == "q" else 2
    row = torch.zeros(1, heads, 64, dtype=torch.bfloat16)
    half = torch.zeros(7 * heads * 32, dtype=torch.bfloat16).as_strided((6, heads, 64), (heads * 32, 64, 1))
    for bad in (row.expand(6, heads, 64), half):
        t = _tensors()
        t[name] = bad
        with pytest.raises(ValueError):
            ddt.check_append(_cfg(), **t)
        if name == "q":
            p = {k: v for k, v in t.items() if k in ("q", "q_start", "ctx_lens", "block_table", "R")}
            with pytest.raises(ValueError):
                ddt.check_prompt(_cfg(), out=torch.zeros(6, 8, 64, dtype=torch.bfloat16), **p)


def test_cache_shapes_are_checked():
    def u8(*s):
        return torch.zeros(*s, dtype=torch.uint8)
    ddt.Kv4Cache(u8(9, 2, 16, 32), u8(9, 2, 16, 32), u8(9, 2, 16, 4), u8(9, 2, 16, 4)).check(_cfg())
    for bad in ((u8(9, 16, 2, 32), u8(9, 2, 16, 32), u8(9, 2, 16, 4), u8(9, 2, 16, 4)),
                (u8(9, 2, 16, 32), u8(9, 2, 16, 32), u8(9, 2, 16, 4), u8(9, 2, 16, 8)),
                (u8(9, 2, 16, 32), u8(8, 2, 16, 32), u8(9, 2, 16, 4), u8(9, 2, 16, 4))):
        with pytest.raises(ValueError):
            ddt.Kv4Cache(*bad).check(_cfg())


def test_a_missing_context_is_refused(lib):
    a = ddt.AppendArgs()
    c = ddt.Kv4()
    n = None
    assert lib.ddt_append_kv(n, ctypes.byref(a), n, n, n) == ddt.EINVAL
    assert lib.ddt_append_kvq(n, ctypes.byref(a), ctypes.byref(c), n, n, n) == ddt.EINVAL
    assert lib.ddt_prompt_attention(n, n, 0, n, n, 1, 1, n, n, n, n, n) == ddt.EINVAL
    assert lib.ddt_prompt_attention_kvq(n, n, 0, n, n, 1, 1, ctypes.byref(c), n, n, n) == ddt.EINVAL


def test_rotary_table_far_positions():
    """Rows of the table are the angles' cosines and sines at fp32's accuracy, far positions among them."""
    t = ddt.rotary_table(200001, 64, base=500000.0, device="cpu").numpy()
    for p in (0, 1, 4097, 200000):
        for j in (0, 1, 17, 31):
            ang = np.longdouble(p) * np.longdouble(500000.0) ** (-np.longdouble(2 * j) / 64)
            # fp32 rounding, and an fp64 angle off by two parts in 2^53
            tol = 2.0 ** -24 + float(ang) * 2.0 ** -51
            assert abs(float(t[p, j]) - float(np.cos(ang))) <= tol
            assert abs(float(t[p, 32 + j]) - float(np.sin(ang))) <= tol
    assert ddt.rotary_table(3, 32, inv_freq=[0.5] * 16, device="cpu").shape == (3, 32)
    with pytest.raises(ValueError):
        ddt.rotary_table(3, 32, inv_freq=[0.5] * 15, device="cpu")

"""The host side of sampling and of attention over shared prefixes, without a GPU: the
layout of the settings' structure, the binding's checks of types and shapes, and the
library's refusal of a missing context."""
import ctypes
import os
import subprocess
import types

import pytest
import torch

from speculative_decoding_draft_depth_gb300 import build as ddt_build
from speculative_decoding_draft_depth_gb300 import ddt

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    ddt_build.build()
    return ddt.load()


def test_structure_matches_the_header(tmp_path):
    fields = [f for f, _ in ddt.FilterArgs._fields_]
    src = tmp_path / "a.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "ddt.h"\nint main(void) {\n' +
                   "".join('printf("%%zu\\n", offsetof(ddt_filter, %s));\n' % f for f in fields) +
                   'printf("%zu %zu %zu\\n", sizeof(ddt_filter), offsetof(ddt_config, prefix_tokens), sizeof(ddt_config));'
                   "return 0;}\n")
    exe = str(tmp_path / "a")
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", exe], check=True)
    out = [int(x) for x in subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split()]
    assert out == [getattr(ddt.FilterArgs, f).offset for f in fields] + [
        ctypes.sizeof(ddt.FilterArgs), ddt.Config.prefix_tokens.offset, ctypes.sizeof(ddt.Config)]


def test_a_missing_context_is_refused(lib):
    f = ctypes.byref(ddt.FilterArgs())
    assert lib.ddt_sample(None, None, 0, 1, f, None, None, None, None) == ddt.EINVAL
    assert lib.ddt_accept_sampled(None, None, None, None, None, None, 1, f, f, None, None, None, None) == ddt.EINVAL
    assert lib.ddt_prefix_attention(None, None, 0, None, None, 1, 1, None, None, None, None, None, 0, None, None) == ddt.EINVAL
    assert lib.ddt_prefix_attention_kvq(None, None, 0, None, None, 1, 1, None, None, None, None, 0, None, None) == ddt.EINVAL


def cfg():
    return types.SimpleNamespace(R_max=4, L=3, V=50, draft_dtype=ddt.BF16, target_dtype=ddt.F32)


def f32(*s):
    return torch.zeros(*s)


def i32(*s):
    return torch.zeros(*s, dtype=torch.int32)


def bf16(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


def test_sample_takes_either_type():
    assert ddt.check_sample(cfg(), bf16(7, 50), f32(7), i32(7), None, None) == ddt.BF16
    assert ddt.check_sample(cfg(), f32(7, 50), f32(7), i32(7), ddt.Filter(temperature=f32(7), top_k=i32(7)), f32(7)) == ddt.F32


@pytest.mark.parametrize("name,value", [
    ("logits", bf16(7, 49)), ("logits", torch.zeros(7, 50, dtype=torch.float16)), ("logits", bf16(50, 7)),
    ("u", f32(6)), ("u", f32(7).double()), ("tokens", i32(7).long()),
    ("tokens", i32(7, 1)), ("logprobs", f32(8)), ("logprobs", bf16(7)),
    ("filter", ddt.Filter(temperature=f32(6))), ("filter", ddt.Filter(top_k=f32(7))), ("filter", ddt.Filter(top_p=i32(7))),
])
def test_sample_shapes_are_checked(name, value):
    t = dict(logits=bf16(7, 50), u=f32(7), tokens=i32(7), filter=None, logprobs=f32(7))
    ddt.check_sample(cfg(), **t)
    t[name] = value
    with pytest.raises(ValueError):
        ddt.check_sample(cfg(), **t)


@pytest.mark.parametrize("name,value", [
    ("draft_logits", f32(4, 3, 50)), ("target_logits", bf16(4, 4, 50)), ("target_logits", f32(4, 3, 50)),
    ("draft_tokens", i32(4, 4)), ("u", f32(4)), ("r", f32(4, 1)), ("acc_len", i32(3)), ("acc_tokens", i32(4, 3)),
    ("n_guess", i32(5)), ("n_guess", f32(4)), ("draft_filter", ddt.Filter(min_p=f32(3))),
    ("target_filter", ddt.Filter(top_k=i32(5))), ("R", 5), ("R", -1), ("R", 3),
])
def test_accept_sampled_shapes_are_checked(name, value):
    t = dict(draft_logits=bf16(4, 3, 50), target_logits=f32(4, 4, 50), draft_tokens=i32(4, 3), u=f32(4, 3), r=f32(4), R=4,
             acc_len=i32(4), acc_tokens=i32(4, 4), draft_filter=ddt.Filter(top_p=f32(4)), target_filter=None, n_guess=i32(4))
    ddt.check_accept_sampled(cfg(), **t)
    t[name] = value
    with pytest.raises(ValueError):
        ddt.check_accept_sampled(cfg(), **t)


def test_group_shapes_are_checked():
    assert ddt.check_groups(cfg(), i32(3), i32(2)) == 2
    assert ddt.check_groups(cfg(), i32(1), i32(0)) == 0
    for bad in ((i32(2), i32(2)), (i32(3), f32(2)), (i32(3).long(), i32(2)), (i32(6), i32(5))):
        with pytest.raises(ValueError):
            ddt.check_groups(cfg(), *bad)


PLAN = r"""
#include <stdio.h>
#include <stdlib.h>
#include "prompt_plan.h"
#define NEED(x) do { if (!(x)) { printf("line %d: %s\n", __LINE__, #x); exit(1); } } while (0)
int main() {
    // a prefix (every query tile has the same tiles), and requests without their first ones
    for (int tq = 1; tq <= 256; tq *= 2)
        for (int len = 1; len < 700; len += 37)
            for (int ctx = 0; ctx < 3000; ctx += 211)
                for (int kind = 0; kind < 3; ++kind)
                    for (int hkv = 1; hkv <= 8; hkv *= 8) {
                        PpReq q = {0, len, ctx, 0, 0};
                        if (kind == 0) q.flat = ctx / 128 + 1;
                        if (kind == 1) q.off = ctx / 128;
                        int64_t at = 0;
                        for (int qt = 0; qt * tq < len; ++qt) {
                            const int end = ctx + ((qt + 1) * tq < len ? (qt + 1) * tq : len);
                            const int n = kind == 0 ? q.flat : (end + 127) / 128 - q.off;
                            NEED(pp_tiles(q, qt, tq) == n && n > 0);
                            NEED(pp_units_before(q, qt, tq) * hkv == at);
                            for (int h = 0; h < hkv; ++h, at += n + PP_ITEM)
                                for (int64_t u = at; u < at + n + PP_ITEM; u += n + PP_ITEM - 1) {
                                    const PpItem it = pp_find(q, u, tq, hkv);
                                    NEED(it.qt == qt && it.h == h && it.n == n && it.start == at);
                                }
                        }
                        NEED(pp_units(q, tq, hkv) == at);
                    }
    printf("ok\n");
    return 0;
}
"""


def test_plan_of_prefixes_and_of_what_is_behind_them(tmp_path):
    src = tmp_path / "a.cpp"
    src.write_text(PLAN)
    exe = str(tmp_path / "a")
    csrc = os.path.join(ROOT, "speculative_decoding_draft_depth_gb300", "csrc")
    subprocess.run(["g++", "-O1", "-I", csrc, str(src), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True)
    assert out.stdout == "ok\n" and out.returncode == 0, out.stdout

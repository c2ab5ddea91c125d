"""Which tensors of a packed call share memory: the header's plain functions,
compiled here, against sets of bytes."""
import itertools
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "speculative_decoding_draft_depth_gb300", "csrc")

PROGRAM = r"""
#include <stdio.h>
#include "packed_seq.h"
static PsBytes at(int a, int n) { PsBytes b = {a < 0 ? (const void *)0 : (const void *)(uintptr_t)(4096 + a), n}; return b; }
int main(void)
{
    static const int x[][8] = {%s};
    for (unsigned i = 0; i < sizeof x / sizeof x[0]; ++i) {
        const PsBytes w[2] = {at(x[i][0], x[i][1]), at(x[i][2], x[i][3])}, r[2] = {at(x[i][4], x[i][5]), at(x[i][6], x[i][7])};
        printf("%%d\n", (int)ps_apart(w, 2, r, 2));
    }
    // the ends of the address space, and sizes past 32 bits
    const PsBytes top = {(const void *)(UINTPTR_MAX - 15), 15}, big = {(const void *)4096, (int64_t)1 << 40},
                  in = {(const void *)(4096 + ((uintptr_t)1 << 40) - 1), 1}, out = {(const void *)(4096 + ((uintptr_t)1 << 40)), 1};
    printf("%%d %%d %%d\n", (int)ps_apart(&top, 1, &big, 1), (int)ps_apart(&in, 1, &big, 1), (int)ps_apart(&out, 1, &big, 1));
    return 0;
}
"""


def test_written_tensors_lie_apart(tmp_path):
    """Every arrangement of two written and two read ranges of up to three bytes,
    missing (-1) and empty ones among them; read ones may share with each other."""
    ranges = [(-1, 3), (0, 0), (0, 1), (0, 3), (1, 1), (2, 2), (3, 1), (3, 0)]
    rows = [a + b + c + d for a, b, c, d in itertools.product(ranges, repeat=4)]

    def cells(a, n):
        return set(range(a, a + n)) if a >= 0 else set()

    want = []
    for x in rows:
        w0, w1, r0, r1 = (cells(x[i], x[i + 1]) for i in (0, 2, 4, 6))
        want.append(int(not (w0 & w1 or w0 & (r0 | r1) or w1 & (r0 | r1))))
    src = tmp_path / "a.cpp"
    src.write_text(PROGRAM % ",".join("{%s}" % ",".join(map(str, x)) for x in rows))
    subprocess.run(["g++", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover", "-I", CSRC, str(src), "-o",
                    str(tmp_path / "a")], check=True)
    out = subprocess.run([str(tmp_path / "a")], check=True, capture_output=True, text=True).stdout.split()
    assert [int(x) for x in out[:-3]] == want
    assert out[-3:] == ["1", "0", "1"]

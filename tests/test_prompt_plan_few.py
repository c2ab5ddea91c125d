"""The share arithmetic at the sizes of the kernel of few rows: query tiles of one
token up, two CTAs an SM; the same program as for the larger tiles."""
import os
import re
import subprocess

from test_prompt_plan import PROGRAM

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "speculative_decoding_draft_depth_gb300", "csrc")

MAIN = r"""
int main()
{
    const int grid_max = %d;
    for (int k = 0; k < 4000; ++k) {
        const int tq = 1 << rnd(9), hkv = 1 + rnd(9), R = 1 + rnd(12);
        std::vector<PpReq> qs;
        for (int r = 0; r < R; ++r) {
            const int len = rnd(4) == 0 ? rnd(3) : rnd(2) ? rnd(20) : rnd(tq < 8 ? 150 : 900);
            qs.push_back({0, len, rnd(3) == 0 ? rnd(3) : rnd(2000)});
        }
        one(qs, tq, hkv, 1 + rnd(grid_max), 1 + PP_ITEM);
    }
    // the limits: 2048 requests of 262144 tokens, 255 heads, every tile
    for (int tq = 1; tq <= 256; tq *= 2) {
        PpReq q = {0, 262144, 0};
        const int64_t per = pp_units(q, tq, 255);
        int64_t want = 0;
        for (int64_t t = 1; t <= 262144 / tq; ++t) want += (t * tq + 127) / 128 + PP_ITEM;
        NEED(per == want * 255);
        NEED(per < ((int64_t)1 << 62) / 2048 / grid_max);  // shares of the total, times a CTA's number
        const int64_t total = per * 2048;
        for (int c = 0; c < grid_max; ++c) {
            const int64_t lo = pp_share(total, c, grid_max), hi = pp_share(total, c + 1, grid_max);
            NEED(lo >= 0 && lo < hi && pp_cta_of(lo, total, grid_max) == c && pp_cta_of(hi - 1, total, grid_max) == c);
        }
        PpItem it = pp_find(q, per - 1, tq, 255);
        NEED(it.qt == 262144 / tq - 1 && it.h == 254 && it.n == 2048 && it.start == per - 2048 - PP_ITEM);
        it = pp_find(q, 0, tq, 255);
        NEED(it.qt == 0 && it.h == 0 && it.start == 0);
    }
    printf("ok\n");
}
"""


def test_shares_of_few_rows(tmp_path):
    body = PROGRAM[:PROGRAM.index("int main()")]
    assert "static void one(" in body
    ctas = re.search(r"PR_MAX_CTAS = (\d+);", open(os.path.join(CSRC, "ddt_internal.h")).read())
    (tmp_path / "a.cpp").write_text(body + MAIN % (2 * int(ctas.group(1))))
    subprocess.run(["g++", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover", "-I", CSRC, str(tmp_path / "a.cpp"),
                    "-o", str(tmp_path / "a")], check=True)
    r = subprocess.run([str(tmp_path / "a")], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr

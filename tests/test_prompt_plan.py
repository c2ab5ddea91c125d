"""Prompt attention's share arithmetic (plain functions, compiled here): the
shares cover every key tile of every item once, a cut item's parts are where
the merge looks for them, and totals near the limits do not overflow."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "speculative_decoding_draft_depth_gb300", "csrc")

PROGRAM = r"""
#include <stdio.h>
#include <stdlib.h>
#include <map>
#include <vector>
#include "prompt_plan.h"
#define NEED(x) do { if (!(x)) { printf("line %d: %s\n", __LINE__, #x); exit(1); } } while (0)
static unsigned long long seed = 12345;
static int rnd(int n) { seed = seed * 6364136223846793005ULL + 1442695040888963407ULL; return (int)((seed >> 33) % n); }

static void one(const std::vector<PpReq> &qs, int tq, int hkv, int grid, int min_units)
{
    // the items, listed plainly
    struct It { int r, qt, h, n; int64_t s; };
    std::vector<It> items;
    int64_t total = 0;
    for (int r = 0; r < (int)qs.size(); ++r) {
        const PpReq &q = qs[r];
        int64_t here = 0;
        for (int qt = 0; qt * tq < q.len; ++qt) {
            int end = q.ctx + ((qt + 1) * tq < q.len ? (qt + 1) * tq : q.len);
            int n = (end + 127) / 128;
            NEED(n == pp_tiles(q, qt, tq));
            NEED(pp_units_before(q, qt, tq) * hkv == here);
            for (int h = 0; h < hkv; ++h) {
                items.push_back({r, qt, h, n, total + here});
                here += n + PP_ITEM;
            }
        }
        NEED(here == pp_units(q, tq, hkv));
        total += here;
    }
    if (total == 0) return;
    const int nc = pp_ctas(total, grid, min_units);
    NEED(nc >= 1 && nc <= grid && (nc == 1 || total / nc >= min_units));
    NEED(pp_share(total, 0, nc) == 0 && pp_share(total, nc, nc) == total);
    // every unit's item is found; every tile lies in one share; slots are unique
    std::map<int, int> slots;
    size_t i = 0;
    for (int c = 0; c < nc; ++c) {
        const int64_t lo = pp_share(total, c, nc), hi = pp_share(total, c + 1, nc);
        NEED(lo < hi);
        NEED(pp_cta_of(lo, total, nc) == c && pp_cta_of(hi - 1, total, nc) == c);
    }
    int64_t base = 0;
    for (int r = 0; r < (int)qs.size(); ++r) {
        const int64_t u = pp_units(qs[r], tq, hkv);
        for (int64_t x = 0; x < u; x += 1 + (u > 3000 ? rnd(50) : 0)) {
            PpItem it = pp_find(qs[r], x, tq, hkv);
            NEED(it.start <= x && x < it.start + it.n + PP_ITEM);
            while (items[i].s + items[i].n + PP_ITEM <= base + x) ++i;
            NEED(items[i].r == r && items[i].qt == it.qt && items[i].h == it.h && items[i].n == it.n &&
                 items[i].s == base + it.start);
        }
        base += u;
    }
    for (auto &it : items) {
        int next = 0;
        const int64_t e = it.s + it.n + PP_ITEM;
        const int c0 = pp_cta_of(it.s + PP_ITEM, total, nc), c1 = pp_cta_of(e - 1, total, nc);
        int parts = 0;
        for (int c = 0; c < nc; ++c) {
            const int64_t lo = pp_share(total, c, nc), hi = pp_share(total, c + 1, nc);
            if (hi <= it.s || lo >= e) continue;
            const int a = pp_tile_at((lo > it.s ? lo : it.s) - it.s), b = pp_tile_at((hi < e ? hi : e) - it.s);
            if (a == b) continue;
            NEED(a == next);
            next = b;
            NEED(c == c0 + parts);
            ++parts;
            if (a != 0 || b != it.n)  // a part: where the merge looks for it
                NEED(slots[a > 0 ? 2 * c : 2 * c + 1]++ == 0);
        }
        NEED(next == it.n && parts == c1 - c0 + 1);
    }
}

int main()
{
    for (int k = 0; k < 3000; ++k) {
        const int tq = 16 << rnd(5), hkv = 1 + rnd(9), R = 1 + rnd(12);
        std::vector<PpReq> qs;
        for (int r = 0; r < R; ++r) {
            const int len = rnd(4) == 0 ? rnd(3) : rnd(2) ? rnd(40) : rnd(900);
            qs.push_back({0, len, rnd(3) == 0 ? rnd(3) : rnd(2000)});
        }
        one(qs, tq, hkv, 1 + rnd(160), 1 + rnd(6));
    }
    // the limits: 2048 requests of 262144 tokens, 255 heads, 16-token tiles
    PpReq q = {0, 262144, 0};
    const int64_t per = pp_units(q, 16, 255);
    int64_t want = 0;
    for (int t = 0; t < 262144 / 16; ++t) want += (16 * (t + 1) + 127) / 128 + PP_ITEM;
    NEED(per == want * 255);
    NEED(per > 0 && per * 2048 < ((int64_t)1 << 62) / 256);  // times a CTA count stays in 64 bits
    PpItem it = pp_find(q, per - 1, 16, 255);
    NEED(it.qt == 262144 / 16 - 1 && it.h == 254 && it.n == 2048);
    printf("ok\n");
}
"""


def test_shares_cover_every_tile(tmp_path):
    (tmp_path / "a.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover", "-I", CSRC, str(tmp_path / "a.cpp"),
                    "-o", str(tmp_path / "a")], check=True)
    r = subprocess.run([str(tmp_path / "a")], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr

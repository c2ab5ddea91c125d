// prompt_plan.h -- how prompt attention's work is cut into equal shares. Plain
// integer arithmetic, the same on the host (where a test runs it) and on the
// device.
//
// An item is (request r, query tile qt, KV head h): up to TQ = 256 / G tokens
// of the request with the G query heads of the KV head, so 256 rows, against
// n(qt) = ceil((ctx + tokens up to the tile's last) / 128) tiles of 128 keys.
// Items lie one behind the other, request by request, query tile by query
// tile, head by head (neighbouring CTAs then read the same tokens' cache rows
// at about the same time). An item counts n + PP_ITEM units: its tiles, behind
// PP_ITEM units for what it costs once. CTA c of nc takes units
// [total c / nc, total (c + 1) / nc).
#pragma once

#include <stdint.h>

#include "packed_seq.h"

constexpr int PP_TILE = 128;   // keys of a tile
constexpr int PP_ROWS = 256;   // rows of a query tile
constexpr int PP_ITEM = 3;     // units of an item besides its tiles

struct PpReq {   // one request, and where its units begin
    int q0, len, ctx;  // first packed row, tokens (0: none, or skipped), cached tokens
};

PS_FN int pp_tiles(const PpReq &q, int qt, int tq)
{
    const int64_t last = (int64_t)(qt + 1) * tq;
    const int end = q.ctx + (last < q.len ? (int)last : q.len);
    return (end + PP_TILE - 1) / PP_TILE;
}

PS_FN int pp_qtiles(const PpReq &q, int tq) { return (q.len + tq - 1) / tq; }

// sum of floor(j / w), j = 0 .. x
PS_FN int64_t pp_floor_sum(int64_t x, int w)
{
    const int64_t q = x / w, r = x % w;
    return w * (q * (q - 1) / 2) + q * (r + 1);
}

// tiles of query tiles 0 .. m - 1, all of them full (m TQ <= len)
PS_FN int64_t pp_tiles_before(const PpReq &q, int m, int tq)
{
    if (tq >= PP_TILE) {
        const int64_t c = (q.ctx + PP_TILE - 1) / PP_TILE, k = tq / PP_TILE;
        return m * c + k * ((int64_t)m * (m + 1) / 2);
    }
    const int w = PP_TILE / tq;
    const int64_t b = (q.ctx + PP_TILE - 1) / tq;
    return pp_floor_sum(b + m, w) - pp_floor_sum(b, w);
}

// units of one head's items of query tiles 0 .. m - 1 (m <= pp_qtiles)
PS_FN int64_t pp_units_before(const PpReq &q, int m, int tq)
{
    if (m == 0)
        return 0;
    const int nq = pp_qtiles(q, tq);
    const int64_t t = m < nq ? pp_tiles_before(q, m, tq)
                             : pp_tiles_before(q, nq - 1, tq) + pp_tiles(q, nq - 1, tq);
    return t + (int64_t)m * PP_ITEM;
}

PS_FN int64_t pp_units(const PpReq &q, int tq, int hkv)
{
    return q.len > 0 ? hkv * pp_units_before(q, pp_qtiles(q, tq), tq) : 0;
}

// CTAs that share `total` units: at most `grid`, each with at least min_units
PS_FN int pp_ctas(int64_t total, int grid, int min_units)
{
    const int64_t n = total / min_units;
    return n < 1 ? 1 : n > grid ? grid : (int)n;
}

PS_FN int64_t pp_share(int64_t total, int c, int nc) { return total * c / nc; }

// the CTA whose share holds unit u
PS_FN int pp_cta_of(int64_t u, int64_t total, int nc)
{
    return (int)(((u + 1) * nc + total - 1) / total - 1);
}

struct PpItem {
    int qt, h, n;      // query tile, KV head, key tiles
    int64_t start;     // the item's first unit, from the request's first
};

// the item that holds unit u of a request (0 <= u < pp_units)
PS_FN PpItem pp_find(const PpReq &q, int64_t u, int tq, int hkv)
{
    int lo = 0, hi = pp_qtiles(q, tq) - 1;  // the last query tile whose units begin at or before u
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (hkv * pp_units_before(q, mid, tq) <= u)
            lo = mid;
        else
            hi = mid - 1;
    }
    PpItem it;
    it.qt = lo;
    it.n = pp_tiles(q, lo, tq);
    const int64_t base = hkv * pp_units_before(q, lo, tq);
    it.h = (int)((u - base) / (it.n + PP_ITEM));
    it.start = base + (int64_t)it.h * (it.n + PP_ITEM);
    return it;
}

// key tiles before unit x of an item
PS_FN int pp_tile_at(int64_t x) { return x > PP_ITEM ? (int)(x - PP_ITEM) : 0; }

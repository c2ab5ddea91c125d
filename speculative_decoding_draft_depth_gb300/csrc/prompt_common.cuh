// prompt_common.cuh -- what the prompt attention kernels share: their arguments,
// the walk over a CTA's share of the work (prompt_plan.h), the 4-bit codes'
// values, and the merge of items that share boundaries cut.
#pragma once

#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "ddt_device.cuh"
#include "ddt_internal.h"
#include "prompt_plan.h"

struct PtArgs {
    const int32_t *q_start, *ctx_lens, *block_table;
    const uint16_t *v_cache;
    const uint8_t *codes[2], *scales[2];  // of K, V
    uint16_t *out;
    float *part_o;
    float2 *part_ml;
    int32_t *status;
    int R, T, Hq, Hkv, g_shift, page_shift, max_pages, cap;
    int64_t num_pages;
    float scale_log2, out_scale;
    long long debug_wait;  // > 0 (tests only): each CTA starts with a wait that runs out after this many cycles
};

// few rows of each request over the 4-bit cache (prompt_few.cu): items of up to 8
// rows, or 16
cudaError_t launch_prompt_few(ddt_ctx *c, const PtArgs &a, const uint16_t *q, int64_t q_stride, int rows,
                              cudaStream_t s);

namespace {

// Units of a share at least: an item of one tile is not cut (one token behind 10 takes
// 9 us; cut, 11.5).
constexpr int MIN_UNITS = 1 + PP_ITEM;
constexpr float TAU = 8.0f;   // growth of a maximum that the running one may lag behind (log2 units)
// 4-bit cache: probabilities are held times 2^7, at most 2^(7 + TAU) (fp16 ends at
// 65504), so that what fp16 cannot hold lies 2^-32 below the row's largest
constexpr float PBIAS = 7.0f;

// a segment of an item: ring words
//   0: request (-1: end of the share)   1: head | split << 8 | whole << 9 | slot << 10
//   2: first packed row  3: tokens  4: position of the first  5, 6: key tiles [t0, t1)
struct Seg {
    int r, h, row0, ntok, pos0, t0, t1, slot;
    bool split, whole;
    DDT_DEVINL int steps(int g) const  // key tiles of group g
    {
        const int n = t1 - t0;
        return split ? (n + 1 - g) >> 1 : n;
    }
    DDT_DEVINL int tile(int g, int j) const { return t0 + (split ? 2 * j + g : j); }
};

DDT_DEVINL void seg_decode(const int *w, Seg &s)
{
    s.r = w[0];
    s.h = w[1] & 0xFF;
    s.split = (w[1] >> 8) & 1;
    s.whole = (w[1] >> 9) & 1;
    s.slot = w[1] >> 10;
    s.row0 = w[2];
    s.ntok = w[3];
    s.pos0 = w[4];
    s.t0 = w[5];
    s.t1 = w[6];
}

// 4-bit cache: what a score is multiplied by whose query was divided by `power`. Finite:
// an infinity would make a score of zero NaN.
DDT_DEVINL float row_scale(const PtArgs &a, float power) { return fminf(a.scale_log2 * power, 3.402823466e38f); }

DDT_DEVINL PpReq load_req(const PtArgs &a, int r)
{
    const int s0 = __ldg(&a.q_start[r]), s1 = __ldg(&a.q_start[r + 1]), c = __ldg(&a.ctx_lens[r]);
    PpReq q;
    q.q0 = s0;
    q.ctx = c;
    q.len = packed_ok(s0, s1, a.T, c, a.cap) ? s1 - s0 : 0;
    return q;
}

// the page of 16-token group u of key tile j (NO_PAGE: past the item's last key)
constexpr int NO_PAGE = -0x7fffffff - 1;
DDT_DEVINL int group_page(const PtArgs &a, const Seg &s, int j, int u)
{
    const int t16 = j * PP_TILE + 16 * u;  // never straddles a page (page % 16 == 0)
    return t16 >= s.pos0 + s.ntok ? NO_PAGE
                                  : __ldg(&a.block_table[(int64_t)s.r * a.max_pages + (t16 >> a.page_shift)]);
}
// whether the group has rows to read; a page out of range is reported
DDT_DEVINL bool page_ok(const PtArgs &a, int pg)
{
    if (pg >= 0 && pg < a.num_pages)
        return true;
    if (pg != NO_PAGE)
        atomicOr(a.status, DDT_DEV_BAD_PAGE);
    return false;
}
// this CTA's share: the totals by a scan over the requests (whole block), then
// the request that holds the share's first unit. found: [0] request, [1..2] its
// first unit, [3..4] total
DDT_DEVINL void find_share(const PtArgs &a, int tq, int grid, int cta, long long *sums,
                           volatile long long *found, int tid, int nthreads)
{
    const int per = (a.R + nthreads - 1) / nthreads;
    const int r0 = min(tid * per, a.R), r1 = min(r0 + per, a.R);
    long long mine = 0;
    for (int r = r0; r < r1; ++r)
        mine += pp_units(load_req(a, r), tq, a.Hkv);
    long long incl = mine;
    const int lane = tid & 31, warp = tid >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o)
            incl += y;
    }
    if (lane == 31)
        sums[warp] = incl;
    __syncthreads();
    long long before = 0, total = 0;
    for (int w = 0; w < nthreads / 32; ++w) {
        before += w < warp ? sums[w] : 0;
        total += sums[w];
    }
    const long long excl = before + incl - mine;
    if (tid == 0) {
        found[0] = -1;
        found[2] = total;
    }
    __syncthreads();
    if (total > 0) {
        const int nc = pp_ctas(total, grid, MIN_UNITS);
        const long long lo = pp_share(total, cta, nc);
        if (cta < nc && excl <= lo && lo < excl + mine) {
            long long acc = excl;
            for (int r = r0; r < r1; ++r) {
                const long long u = pp_units(load_req(a, r), tq, a.Hkv);
                if (lo < acc + u) {
                    found[0] = r;
                    found[1] = acc;
                    break;
                }
                acc += u;
            }
        }
    }
    __syncthreads();
}

// the segments of a CTA's share, one behind the other (every thread that walks holds
// the same state)
struct ShareWalk {
    int r;
    long long base, cur, hi;  // the request's first unit; the walk's place and end
    PpReq rq;
    PpItem it;
    int cta;

    DDT_DEVINL void begin(const PtArgs &a, const volatile long long *found, int tq, int grid, int c)
    {
        const long long total = found[2];
        r = (int)found[0];
        base = found[1];
        cta = c;
        cur = hi = 0;
        if (r >= 0) {
            const int nc = pp_ctas(total, grid, MIN_UNITS);
            cur = pp_share(total, c, nc);
            hi = pp_share(total, c + 1, nc);
            rq = load_req(a, r);
            it = pp_find(rq, cur - base, tq, a.Hkv);
        }
    }

    // the next segment that holds tiles; s.r = -1 at the end. An item of at most
    // split_rows rows is `split`.
    DDT_DEVINL void next(const PtArgs &a, int tq, int split_rows, Seg &s)
    {
        s.r = -1;
        while (cur < hi) {
            const long long i0 = base + it.start, i1 = i0 + it.n + PP_ITEM;
            const int t0 = pp_tile_at(cur - i0), t1 = pp_tile_at(min(hi, i1) - i0);
            s.h = it.h;
            s.row0 = rq.q0 + it.qt * tq;
            s.ntok = min(tq, rq.len - it.qt * tq);
            s.pos0 = rq.ctx + it.qt * tq;
            s.t0 = t0;
            s.t1 = t1;
            s.whole = t0 == 0 && t1 == it.n;
            s.split = (s.ntok << a.g_shift) <= split_rows;
            s.slot = 2 * cta + (t0 > 0 ? 0 : 1);
            const int sr = r;
            cur = min(hi, i1);
            if (cur < hi) {  // the item behind it
                it.start += it.n + PP_ITEM;
                if (++it.h == a.Hkv) {
                    it.h = 0;
                    if (++it.qt == pp_qtiles(rq, tq)) {
                        base += it.start;
                        it.start = 0;
                        it.qt = 0;
                        do {  // (units remain, so a request with tokens follows)
                            if (++r >= a.R) {
                                cur = hi;  // (not so: lengths that changed under the call)
                                break;
                            }
                            rq = load_req(a, r);
                        } while (rq.len == 0);
                    }
                    it.n = pp_tiles(rq, it.qt, tq);
                }
            }
            if (t1 > t0) {
                s.r = sr;
                return;
            }
        }
    }
};

// eight 4-bit codes to four fp16 pairs times sc; byte b holds channels in the
// order 0 2 4 6 1 3 5 7, which the fp16 tiles keep (Q's channels are laid out the
// same way, and the output's are put back by naming)
DDT_DEVINL uint4 values8(uint32_t w, uint32_t sc)
{
    uint4 r;
    asm("{\n .reg .b8 a, b, c, d;\n .reg .b32 w0, w1, w2, w3;\n mov.b32 {a, b, c, d}, %4;\n"
        " cvt.rn.f16x2.e2m1x2 w0, a;\n cvt.rn.f16x2.e2m1x2 w1, b;\n"
        " cvt.rn.f16x2.e2m1x2 w2, c;\n cvt.rn.f16x2.e2m1x2 w3, d;\n"
        " mul.rn.f16x2 %0, w0, %5;\n mul.rn.f16x2 %1, w1, %5;\n"
        " mul.rn.f16x2 %2, w2, %5;\n mul.rn.f16x2 %3, w3, %5;\n}\n"
        : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
        : "r"(w), "r"(sc));
    return r;
}
// channel of position e of the fp16 tiles, within its 8
DDT_DEVINL constexpr int channel_of(int e) { return (e & ~7) | ((e & 3) * 2 + ((e >> 2) & 1)); }
DDT_DEVINL constexpr int position_of(int c) { return (c & ~7) | ((c & 6) >> 1) | ((c & 1) << 2); }

DDT_DEVINL uint32_t pack_f16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Merge of a cut item: boundary b (between CTAs b - 1 and b) takes the j-th of
// the nb row blocks of the item that it cuts, if it lies among the item's tiles
// (nb: the boundaries that do). Partials come from L2; what counts is how many CTAs
// read them: with up to 1, 2, 4, 8 CTAs a boundary 32 packed prompts take 134, 123, 119,
// 122 us, one prompt of 512 tokens 50, 34, 30, 28, and 64 tokens behind a thousand
// cached 56, 56, 57, 61 (many CTAs of few rows).
constexpr int MG_THREADS = 256, MG_SPLIT = 4;

template <int D>
__global__ void __launch_bounds__(MG_THREADS) prompt_merge_kernel(const PtArgs a, int grid, int rows)
{
    __shared__ long long s_sums[MG_THREADS / 32], s_found[3];
    const int tq = rows >> a.g_shift, tid = threadIdx.x, b = blockIdx.x + 1;
    find_share(a, tq, grid, b, s_sums, s_found, tid, MG_THREADS);
    const long long total = s_found[2], base = s_found[1];
    int nc = 0;
    PpReq rq = {0, 0, 0};
    PpItem it = {0, 0, 0, 0};
    long long i0 = 0;
    bool cuts = s_found[0] >= 0;  // (else no such share)
    if (cuts) {
        nc = pp_ctas(total, grid, MIN_UNITS);
        rq = load_req(a, (int)s_found[0]);
        const long long at = pp_share(total, b, nc);
        it = pp_find(rq, at - base, tq, a.Hkv);
        i0 = base + it.start;
        cuts = pp_tile_at(at - i0) > 0;  // (else the item's tiles all lie behind this boundary)
    }
    // The main kernel let this one start early: every CTA waits for it, one without
    // work too, or what comes next in the stream could begin before it has ended.
    pdl_wait();
    if (!cuts)
        return;
    const int c0 = pp_cta_of(i0 + PP_ITEM, total, nc), c1 = pp_cta_of(i0 + PP_ITEM + it.n - 1, total, nc);
    const int ntok = min(tq, rq.len - it.qt * tq), nrows = ntok << a.g_shift, ns = c1 - c0 + 1;
    const int nb = ns - 1, j = b - c0 - 1;
    // of the boundary's rows, this CTA's part
    const int y = j * gridDim.y + blockIdx.y, ny = nb * gridDim.y;
    const int lo = (int)((long long)y * nrows / ny), hi = (int)((long long)(y + 1) * nrows / ny);
    // a warp: eight rows by four float4 columns (the partials' rows lie side by
    // side, the output's columns do)
    constexpr int C4 = D / 4;
    const int lane = tid & 31, r8 = lane & 7;
    for (int e = tid >> 5; e < ((hi - lo + 7) >> 3) * (C4 / 4); e += MG_THREADS / 32) {
        const int row = lo + (e / (C4 / 4)) * 8 + r8, c4 = (e % (C4 / 4)) * 4 + (lane >> 3);
        if (row >= hi)
            continue;
        float M = DDT_NEG_INF, L = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int s = 0; s < ns; ++s) {
            const int64_t slot = s == 0 ? 2 * c0 + 1 : 2 * (c0 + s);
            const float2 ml = __ldcg(&a.part_ml[slot * rows + row]);
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(a.part_o + slot * rows * D) + c4 * rows + row);
            const float Mn = fmaxf(M, ml.x);
            const float f = M == DDT_NEG_INF ? 0.f : ex2(M - Mn), w = ml.x == DDT_NEG_INF ? 0.f : ex2(ml.x - Mn);
            L = L * f + ml.y * w;
            o.x = o.x * f + v.x * w;
            o.y = o.y * f + v.y * w;
            o.z = o.z * f + v.z * w;
            o.w = o.w * f + v.w * w;
            M = Mn;
        }
        const float inv = L > 0.f || L != L ? a.out_scale / L : 0.f;
        const int tok = row >> a.g_shift, h = (it.h << a.g_shift) + (row & ((1 << a.g_shift) - 1));
        uint32_t *dst = reinterpret_cast<uint32_t *>(
            a.out + ((int64_t)(rq.q0 + it.qt * tq + tok) * a.Hq + h) * D) + c4 * 2;
        *reinterpret_cast<uint2 *>(dst) =
            make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    }
}

// devices for which a kernel's attributes have been set (setting them twice does no
// harm, so two threads may come at once)
struct DeviceFlags {
    std::atomic<uint64_t> bits{0};
    bool test(int dev) const { return dev < 64 && ((bits.load(std::memory_order_relaxed) >> dev) & 1); }
    void set(int dev)
    {
        if (dev < 64)
            bits.fetch_or((uint64_t)1 << dev, std::memory_order_relaxed);
    }
};

// the merge as a programmatic dependent of the main kernel (which lets it stage
// itself at once); grid: the main kernel's
template <int D>
cudaError_t launch_merge(const PtArgs &a, int grid, int rows, cudaStream_t s)
{
    cudaLaunchConfig_t lc = {};
    // CTAs of a boundary: one for about 32 of the rows that an item can have
    const int64_t most = std::min((int64_t)rows, (int64_t)a.T << a.g_shift);
    lc.gridDim = dim3(grid - 1, (unsigned)std::max((int64_t)1, std::min((int64_t)MG_SPLIT, most / 32)));
    lc.blockDim = dim3(MG_THREADS);
    lc.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = at;
    lc.numAttrs = 1;
    return cudaLaunchKernelEx(&lc, prompt_merge_kernel<D>, a, grid, rows);
}

}  // namespace

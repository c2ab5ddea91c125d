// prompt_tc.cu -- causal attention of packed sequences over the paged cache on
// the 5th-generation tensor cores (tcgen05 + TMEM + TMA), D = 128 and 64.
//
// Work split (prompt_plan.h): an item is up to 256 rows (256 / G tokens of a
// request with the G heads of one KV head) against the request's key tiles of
// 128; the items of the batch, laid end to end, are cut into equal shares, one
// per CTA (one CTA per SM), each CTA computing its share from q_start and
// ctx_lens. An item cut by a share boundary leaves partial outputs (two slots
// per CTA), merged by prompt_merge_kernel.
//
// Inside a CTA:
//  * two groups, A and B, of 128 rows each (rows in TMEM lanes): S = Q K^T into
//    the group's 128 TMEM columns, softmax by the group's four warps (one row
//    per thread, no exchange between threads), P (bf16) over the first 64 of the same
//    columns, O += P V from there. While one group's softmax runs, the tensor
//    cores work for the other. An item of at most 128 rows (a token or a chain
//    of a few) gives both groups the same rows and alternate key tiles; group A
//    merges the two at the end, reading B's O from TMEM.
//  * K and V tiles of 128 tokens arrive by TMA in a 2-deep K ring and a 3-deep V
//    ring, one box per 16-token page run and 64-channel half.
//  * the running maximum is followed lazily: O and the sum are rescaled only when
//    a row's maximum grows by more than 2^8. P V of the tile before has then
//    completed, since the tile's S was issued behind it.
//  * warps 0-3: group A; 4-7: group B; 8: MMA issuer; 9: walks the share, loads Q
//    and K; 10: loads V, with the rows past the item's last key zeroed (whatever
//    the page holds there must not meet a probability of zero).
//  * every wait is bounded; on timeout the CTA raises DDT_DEV_TIMEOUT, waits
//    (bounded) for its own copies and MMAs, frees its TMEM and returns.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "ddt_device.cuh"
#include "ddt_internal.h"
#include "prompt_plan.h"
#include "tc_ptx.cuh"

namespace {

template <bool KV4>
constexpr int NT = KV4 ? 512 : 384;
constexpr int W_MMA = 8, W_WALK = 9, W_VLOAD = 10, W_DQ = 12;
constexpr int NDQ = 4;  // 4-bit cache: warps that turn codes into fp16 tiles (one warpgroup)
// registers per thread of the two softmax warpgroups and of the others, and what
// the kernel has to be launched with: they add up to no more than that
template <bool KV4>
constexpr int REGS_SM = KV4 ? 176 : 208;
template <bool KV4>
constexpr int REGS_OTHER = KV4 ? 80 : 88;
template <bool KV4>
constexpr int REGS_LAUNCH = KV4 ? 128 : 168;
static_assert(256 * REGS_SM<true> + 256 * REGS_OTHER<true> <= REGS_LAUNCH<true> * NT<true>, "register split");
static_assert(256 * REGS_SM<false> + 128 * REGS_OTHER<false> <= REGS_LAUNCH<false> * NT<false>, "register split");
constexpr int NRING = 4;
template <bool KV4>
constexpr int RING_CONSUMERS = 8 + 1 + (KV4 ? 0 : 1);  // softmax warps, MMA issuer, V loader
constexpr int MIN_UNITS = 4;               // of a share
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t TM_S = 0;    // S (and P) of A, B: 128 columns each
constexpr uint32_t TM_O = 256;  // O of A, B: 128 columns each
constexpr float TAU = 8.0f;     // lazy-rescale threshold (log2 units)
constexpr long long WAIT_LIMIT = 4000000000LL;  // cycles (about 2 s)
constexpr long long DRAIN_LIMIT = 200000000LL;

// shared memory (offsets from a 1024-byte aligned base)
constexpr int NK = 2;
template <bool KV4>
constexpr int NV = KV4 ? 2 : 3;
constexpr int NRAW = 6;          // 4-bit cache: tiles of codes and scales in flight
constexpr uint32_t RAW = 9216;   // 128 rows of 64 bytes of codes, then of 8 scales
constexpr uint32_t SM_Q = 0;     // A, B: 32 KB each (two 16 KB halves); 4 bits: one for both
template <bool KV4>
constexpr uint32_t SM_K = KV4 ? 32768 : 65536;
template <bool KV4>
constexpr uint32_t SM_V = SM_K<KV4> + NK * 32768;
template <bool KV4>
constexpr uint32_t SM_RAW = SM_V<KV4> + NV<KV4> * 32768;
template <bool KV4>
constexpr uint32_t SM_BAR = SM_RAW<KV4> + (KV4 ? NRAW * RAW : 0);
constexpr uint32_t B_QFULL = 0, B_QEMPTY = 8, B_KFULL = 16, B_KEMPTY = 32, B_VFULL = 48, B_VEMPTY = 72,
                   B_SFULL = 96,   // [2 groups]
                   B_PFULL = 112,  // [2] 4 arrivals: the group's warps
                   B_OFULL = 128,  // [2]
                   B_XB = 144,     // B's (m, l) published and its O complete (4 arrivals)
                   B_XA = 152,     // A has read them (4 arrivals)
                   B_RFULL = 160,  // [NRING]
                   B_REMPTY = 192,
                   B_FINAL = 224, B_TMEM = 232, B_ABORT = 236, B_FOUND = 240,  // 32 bytes
                   B_RING = 272,   // [NRING][8] ints
                   B_ML = 400,     // [128] float2: B's (m, l); before the roles start, the scan's sums
                   // 4-bit cache only:
                   B_RAWFULL = 1424,           // [NRAW]
                   B_RAWEMPTY = 1424 + 48,     // [NRAW] NDQ arrivals
                   B_QREADY = 1424 + 96,       // NDQ arrivals
                   B_META = 1424 + 104,        // [NRAW] int: what the slot holds
                   B_ROWSC = 1424 + 128;       // [2][128] floats: the row's factor, by item parity
template <bool KV4>
constexpr uint32_t B_END = KV4 ? B_ROWSC + 1024 : B_RAWFULL;
template <bool KV4>
constexpr uint32_t SM_ALLOC = SM_BAR<KV4> + B_END<KV4> + 1024;
static_assert(SM_ALLOC<false> <= 232448 && SM_ALLOC<true> <= 232448, "shared memory of one CTA");

template <bool KV4>
constexpr uint32_t IDESC_QK = KV4 ? idesc_f16(128, 128, false, false) : idesc_bf16(128, 128, false, false);
template <int D, bool KV4>
constexpr uint32_t IDESC_PV = KV4 ? idesc_f16(128, D, false, true) : idesc_bf16(128, D, false, true);
// 4-bit cache: probabilities are held times 2^7, at most 2^(7 + TAU) (fp16 ends at
// 65504), so that what fp16 cannot hold lies 2^-32 below the row's largest
constexpr float PBIAS = 7.0f;

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
};

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

DDT_DEVINL PpReq load_req(const PtArgs &a, int r)
{
    const int s0 = __ldg(&a.q_start[r]), s1 = __ldg(&a.q_start[r + 1]), c = __ldg(&a.ctx_lens[r]);
    PpReq q;
    q.q0 = s0;
    q.ctx = c;
    q.len = packed_ok(s0, s1, a.T, c, a.cap) ? s1 - s0 : 0;
    return q;
}

// bounded mbarrier wait; false (and the abort flag raised) on timeout
DDT_DEVINL bool wait_bar(uint32_t bar, uint32_t parity, volatile int *abort_flag, int32_t *status)
{
    if (mbar_try_wait(bar, parity))
        return true;
    const long long t0 = clock64();
    while (!mbar_try_wait(bar, parity)) {
        if (*abort_flag)
            return false;
        if (clock64() - t0 > WAIT_LIMIT) {
            *abort_flag = 1;
            atomicOr(status, DDT_DEV_TIMEOUT);
            return false;
        }
    }
    return true;
}
DDT_DEVINL bool wait_warp(uint32_t bar, uint32_t parity, volatile int *abort_flag, int32_t *status)
{
    return __all_sync(0xFFFFFFFFu, wait_bar(bar, parity, abort_flag, status));
}
DDT_DEVINL void drain_bar(uint32_t bar, uint32_t parity)
{
    const long long t0 = clock64();
    while (!mbar_try_wait(bar, parity))
        if (clock64() - t0 > DRAIN_LIMIT)
            return;
}

// ring entry k for a whole warp; false: the end, or abort
DDT_DEVINL bool ring_get(const PtArgs &a, uint32_t bar, const volatile int *ring, int k, int lane,
                         volatile int *abort_flag, Seg &s)
{
    const int slot = k & (NRING - 1);
    if (!wait_warp(bar + B_RFULL + 8 * slot, (k / NRING) & 1, abort_flag, a.status))
        return false;
    int w[7];
#pragma unroll
    for (int i = 0; i < 7; ++i)
        w[i] = ring[8 * slot + i];
    __syncwarp();
    if (lane == 0)
        mbar_arrive(bar + B_REMPTY + 8 * slot);
    seg_decode(w, s);
    return s.r >= 0;
}

// the pool row of 16-token group u of key tile j; -16: past the item's last key,
// or a page out of range (the TMA fills zeros)
DDT_DEVINL int group_row(const PtArgs &a, const Seg &s, int j, int u)
{
    const int t16 = j * PP_TILE + 16 * u;  // never straddles a page (page % 16 == 0)
    if (t16 >= s.pos0 + s.ntok)
        return -16;
    const int pg = __ldg(&a.block_table[(int64_t)s.r * a.max_pages + (t16 >> a.page_shift)]);
    if (pg < 0 || pg >= a.num_pages) {
        atomicOr(a.status, DDT_DEV_BAD_PAGE);
        return -16;
    }
    return (pg << a.page_shift) + (t16 & ((1 << a.page_shift) - 1));
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

// whole warp: one thread issues a tile's boxes, 16 tokens by 64 channels each, but
// for group `skip`; z: lane u holds group u's pool row
template <int D>
DDT_DEVINL void load_boxes(const void *map, uint32_t dst, int h, int z, int skip, uint32_t fb, uint32_t bytes)
{
    int zu[8];
#pragma unroll
    for (int u = 0; u < 8; ++u)
        zu[u] = __shfl_sync(0xFFFFFFFFu, z, u);
    if (elect_one()) {
        mbar_arrive_expect_tx(fb, bytes);
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (u != skip) {
                tma_load_3d(dst + u * 2048, map, 0, h, zu[u], fb);
                if (D == 128)
                    tma_load_3d(dst + 16384 + u * 2048, map, 64, h, zu[u], fb);
            }
    }
    __syncwarp();
}

// what a raw slot holds (B_META): its kind, and for K and V the rows that count
// and, by 16-row groups, the ones whose page is out of range
constexpr int CMD_K = 0, CMD_V = 1, CMD_Q = 2, CMD_END = 3;

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

// a warp's part of a tile of codes and scales -> its fp16 tile (128-byte swizzle)
template <int D>
DDT_DEVINL void dequant_tile(const unsigned char *rawp, unsigned char *dst, int meta, int wq, int lane)
{
    constexpr int CH = D / 32;  // 16-byte vectors of codes in a row
    const int nvalid = (meta >> 8) & 0xFF, bad = (meta >> 16) & 0xFF;
#pragma unroll
    for (int i = 0; i < 128 * CH / (NDQ * 32); ++i) {
        const int idx = (i * NDQ + wq) * 32 + lane, row = idx / CH, q = idx % CH;
        uint4 w = *reinterpret_cast<const uint4 *>(rawp + idx * 16);
        uint32_t two = *reinterpret_cast<const uint16_t *>(rawp + 128 * (D / 2) + row * (D / 16) + 2 * q), sc;
        if (row >= nvalid || ((bad >> (row >> 4)) & 1)) {
            w = make_uint4(0u, 0u, 0u, 0u);
            two = 0u;
        }
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(sc) : "h"((uint16_t)two));
        const uint32_t s0 = __byte_perm(sc, sc, 0x1010), s1 = __byte_perm(sc, sc, 0x3232);
        // vectors 4 q + x of the row; lanes of its upper half go in another order,
        // so that eight lanes' stores fall into eight bank groups
        const bool up = D == 128 && (q & 2);
        const uint32_t wx[4] = {up ? w.z : w.x, up ? w.w : w.y, up ? w.x : w.z, up ? w.y : w.w};
        const uint32_t sa = up ? s1 : s0, sb = up ? s0 : s1;
        unsigned char *d = dst + (D == 128 ? (q >> 1) * 16384 : 0) + row * 128;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int ch = ((q & 1) * 4 + x) ^ (up ? 2 : 0);
            *reinterpret_cast<uint4 *>(d + ((ch ^ (row & 7)) << 4)) = values8(wx[x], x < 2 ? sa : sb);
        }
    }
}

// one row of Q: bf16 -> fp16 in place (128-byte swizzle), divided by the power of
// two of its largest magnitude, channels in the tiles' order; returns that power
template <int D>
DDT_DEVINL float halve_row(unsigned char *q, int row)
{
    uint32_t amax = 0;
#pragma unroll 4
    for (int c = 0; c < D / 8; ++c) {
        const uint4 w = *reinterpret_cast<const uint4 *>(q + (c >> 3) * 16384 + row * 128 + (((c & 7) ^ (row & 7)) << 4));
        const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            amax = max(amax, max(v[i] & 0x7FFFu, (v[i] >> 16) & 0x7FFFu));
    }
    int e = (int)(amax >> 7) - 127;
    e = amax >= 0x7F80u ? 0 : max(-100, min(100, e));  // (rows with NaN or inf as they are)
    const float f = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll 4
    for (int c = 0; c < D / 8; ++c) {
        uint4 *at = reinterpret_cast<uint4 *>(q + (c >> 3) * 16384 + row * 128 + (((c & 7) ^ (row & 7)) << 4));
        const uint4 w = *at;
        const float x[8] = {bf16lo(w.x), bf16hi(w.x), bf16lo(w.y), bf16hi(w.y),
                            bf16lo(w.z), bf16hi(w.z), bf16lo(w.w), bf16hi(w.w)};
        *at = make_uint4(pack_f16x2(x[channel_of(0)] * f, x[channel_of(1)] * f),
                         pack_f16x2(x[channel_of(2)] * f, x[channel_of(3)] * f),
                         pack_f16x2(x[channel_of(4)] * f, x[channel_of(5)] * f),
                         pack_f16x2(x[channel_of(6)] * f, x[channel_of(7)] * f));
    }
    return __uint_as_float((uint32_t)(127 + e) << 23);
}

template <int D, bool KV4>
__global__ void __launch_bounds__(NT<KV4>, 1)
prompt_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, const PtArgs a)
{
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = (uint32_t)__cvta_generic_to_shared(smem_raw);
    const uint32_t sb = (raw + 1023u) & ~1023u;
    unsigned char *sgen = smem_raw + (sb - raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sgen + SM_BAR<KV4> + B_ABORT);
    volatile int *ring = reinterpret_cast<volatile int *>(sgen + SM_BAR<KV4> + B_RING);
    const uint32_t bar = sb + SM_BAR<KV4>;
    constexpr int ROWS = KV4 ? 128 : PP_ROWS;  // of an item
    const int tq = ROWS >> a.g_shift;

    if (tid == 0) {
        mbar_init(bar + B_QFULL, 1);
        mbar_init(bar + B_QEMPTY, 1);
        for (int i = 0; i < NK; ++i) {
            mbar_init(bar + B_KFULL + 8 * i, KV4 ? NDQ : 1);
            mbar_init(bar + B_KEMPTY + 8 * i, 1);
        }
        for (int i = 0; i < NV<KV4>; ++i) {
            mbar_init(bar + B_VFULL + 8 * i, KV4 ? NDQ : 1);
            mbar_init(bar + B_VEMPTY + 8 * i, 1);
        }
        for (int g = 0; g < 2; ++g) {
            mbar_init(bar + B_SFULL + 8 * g, 1);
            mbar_init(bar + B_PFULL + 8 * g, 4);
            mbar_init(bar + B_OFULL + 8 * g, 1);
        }
        mbar_init(bar + B_XB, 4);
        mbar_init(bar + B_XA, 4);
        for (int i = 0; i < NRING; ++i) {
            mbar_init(bar + B_RFULL + 8 * i, 1);
            mbar_init(bar + B_REMPTY + 8 * i, RING_CONSUMERS<KV4>);
        }
        mbar_init(bar + B_FINAL, 1);
        if (KV4) {
            for (int i = 0; i < NRAW; ++i) {
                mbar_init(bar + B_RAWFULL + 8 * i, 1);
                mbar_init(bar + B_RAWEMPTY + 8 * i, NDQ);
            }
            mbar_init(bar + B_QREADY, NDQ);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == W_MMA) {
        tmem_alloc(bar + B_TMEM, TMEM_COLS);
        tmem_relinquish();
    }
    if (warp == W_WALK && lane == 0) {
        prefetch_tmap(&tm_q);
        if (!KV4) {
            prefetch_tmap(&tm_k);
            prefetch_tmap(&tm_v);
        }
    }
    volatile long long *found = reinterpret_cast<volatile long long *>(sgen + SM_BAR<KV4> + B_FOUND);
    find_share(a, tq, gridDim.x, blockIdx.x, reinterpret_cast<long long *>(sgen + SM_BAR<KV4> + B_ML), found, tid, NT<KV4>);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(sgen + SM_BAR<KV4> + B_TMEM);

    if (warp >= 8)
        regs_dec<REGS_OTHER<KV4>>();

    if (warp == W_WALK) {
        // ============================================================ share walk, Q and K loads
        if (blockIdx.x == 0)
            for (int r = lane; r < a.R; r += 32) {
                const int s0 = __ldg(&a.q_start[r]), s1 = __ldg(&a.q_start[r + 1]);
                if (!packed_ok(s0, s1, a.T, __ldg(&a.ctx_lens[r]), a.cap))
                    atomicOr(a.status, DDT_DEV_BAD_LENGTH);
            }
        const long long total = found[2];
        int r = (int)found[0];
        long long base = found[1], cur = 0, hi = 0;
        PpReq rq = {0, 0, 0};
        PpItem it = {0, 0, 0, 0};
        if (r >= 0) {
            const int nc = pp_ctas(total, gridDim.x, MIN_UNITS);
            cur = pp_share(total, blockIdx.x, nc);
            hi = pp_share(total, blockIdx.x + 1, nc);
            rq = load_req(a, r);
            it = pp_find(rq, cur - base, tq, a.Hkv);
        }
        int k = 0, kn = 0;
        bool ok = true;
        // 4-bit cache: the next raw slot gets a tile's codes and scales, or a word
        // (Q has been asked for; the end) for the dequantising warps
        int nraw = 0;
        Seg pend;      // the tile whose K has been asked for, but not its V
        int pend_j = -1;
        auto raw_slot = [&]() {
            ok = ok && (nraw < NRAW ||
                        wait_warp(bar + B_RAWEMPTY + 8 * (nraw % NRAW), ((nraw / NRAW) - 1) & 1, abort_flag, a.status));
            return nraw % NRAW;
        };
        volatile int *metas = reinterpret_cast<volatile int *>(sgen + SM_BAR<KV4> + B_META);
        auto say = [&](int cmd) {
            const int sl = raw_slot();
            if (ok) {
                if (lane == 0) {
                    metas[sl] = cmd;
                    mbar_arrive(bar + B_RAWFULL + 8 * sl);
                }
                ++nraw;
            }
        };
        auto load_raw = [&](const Seg &s, int j, int kind) {
            const int z = lane < 8 ? group_row(a, s, j, lane) : -16;
            const int valid = min(PP_TILE, s.pos0 + s.ntok - j * PP_TILE);
            const bool in = lane < 8 && 16 * lane < valid;
            const unsigned copies = __ballot_sync(0xFFFFFFFFu, in && z >= 0);
            const unsigned bad = __ballot_sync(0xFFFFFFFFu, in && z < 0);
            // pool row -> the head's rows of its page
            const int64_t mine = (((int64_t)(z >> a.page_shift) * a.Hkv + s.h) << a.page_shift) +
                                 (z & ((1 << a.page_shift) - 1));
            int64_t row[8];
#pragma unroll
            for (int u = 0; u < 8; ++u)
                row[u] = __shfl_sync(0xFFFFFFFFu, mine, u);
            const int sl = raw_slot();
            if (!ok)
                return;
            const uint32_t fb = bar + B_RAWFULL + 8 * sl, dst = sb + SM_RAW<KV4> + sl * RAW;
            if (elect_one()) {
                metas[sl] = kind | (valid << 8) | ((int)bad << 16);
                mbar_arrive_expect_tx(fb, __popc(copies) * 16 * (D / 2 + D / 16));
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    if ((copies >> u) & 1) {
                        bulk_load(dst + u * 16 * (D / 2), a.codes[kind] + row[u] * (D / 2), 16 * (D / 2), fb);
                        bulk_load(dst + 128 * (D / 2) + u * 16 * (D / 16), a.scales[kind] + row[u] * (D / 16),
                                  16 * (D / 16), fb);
                    }
            }
            __syncwarp();
            ++nraw;
        };
        while (ok) {
            // the next segment that holds tiles
            Seg s;
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
                s.split = KV4 || (s.ntok << a.g_shift) <= 128;
                s.slot = 2 * blockIdx.x + (t0 > 0 ? 0 : 1);
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
                            do
                                rq = load_req(a, ++r);  // (units remain, so a request with tokens follows)
                            while (rq.len == 0);
                        }
                        it.n = pp_tiles(rq, it.qt, tq);
                    }
                }
                if (t1 > t0) {
                    s.r = sr;
                    break;
                }
            }
            const int slot = k & (NRING - 1);
            if (k >= NRING && !wait_warp(bar + B_REMPTY + 8 * slot, ((k / NRING) - 1) & 1, abort_flag, a.status))
                break;
            if (lane == 0) {
                volatile int *w = ring + 8 * slot;
                w[0] = s.r;
                if (s.r >= 0) {
                    w[1] = s.h | (s.split ? 256 : 0) | (s.whole ? 512 : 0) | (s.slot << 10);
                    w[2] = s.row0;
                    w[3] = s.ntok;
                    w[4] = s.pos0;
                    w[5] = s.t0;
                    w[6] = s.t1;
                }
                mbar_arrive(bar + B_RFULL + 8 * slot);
            }
            if (s.r < 0)
                break;
            if (k >= 1 && !wait_warp(bar + B_QEMPTY, (k - 1) & 1, abort_flag, a.status))
                break;
            if (elect_one()) {
                const int y = s.h << a.g_shift;
                mbar_arrive_expect_tx(bar + B_QFULL, 16384u * (D / 64) * (s.split ? 1 : 2));
                for (int g = 0; g < (s.split ? 1 : 2); ++g)
                    for (int x = 0; x < D / 64; ++x)
                        tma_load_3d(sb + SM_Q + g * 32768 + x * 16384, &tm_q, x * 64, y, s.row0 + g * (tq / 2),
                                    bar + B_QFULL);
            }
            ++k;
            if constexpr (KV4) {
                // K one tile ahead of V, across items too
                say(CMD_Q);
                for (int j = s.t0; ok && j < s.t1; ++j) {
                    load_raw(s, j, CMD_K);
                    if (pend_j >= 0)
                        load_raw(pend, pend_j, CMD_V);
                    pend = s;
                    pend_j = j;
                }
            }
            for (int j = s.t0; !KV4 && j < s.t1; ++j, ++kn) {
                const int sl = kn % NK;
                const int z = lane < 8 ? group_row(a, s, j, lane) : 0;
                if (kn >= NK && !wait_warp(bar + B_KEMPTY + 8 * sl, ((kn / NK) - 1) & 1, abort_flag, a.status)) {
                    ok = false;
                    break;
                }
                const uint32_t fb = bar + B_KFULL + 8 * sl, dst = sb + SM_K<KV4> + sl * 32768u;
                load_boxes<D>(&tm_k, dst, s.h, z, -1, fb, 16384u * (D / 64));
            }
        }
        if constexpr (KV4) {
            if (ok && pend_j >= 0)
                load_raw(pend, pend_j, CMD_V);
            say(CMD_END);
            for (int m = max(0, nraw - NRAW); m < nraw; ++m)
                drain_bar(bar + B_RAWFULL + 8 * (m % NRAW), (m / NRAW) & 1);
        }
        // wind down: the copies that this warp issued have landed
        if (k > 0)
            drain_bar(bar + B_QFULL, (k - 1) & 1);
        for (int m = max(0, kn - NK); m < kn; ++m)
            drain_bar(bar + B_KFULL + 8 * (m % NK), (m / NK) & 1);
    } else if (!KV4 && warp == W_VLOAD) {
        // ============================================================ V loads
        int vn = 0;
        bool ok = true;
        for (int k = 0; ok; ++k) {
            Seg s;
            if (!ring_get(a, bar, ring, k, lane, abort_flag, s))
                break;
            const int end = s.pos0 + s.ntok;
            for (int j = s.t0; j < s.t1; ++j, ++vn) {
                const int sl = vn % NV<KV4>;
                const int z = lane < 8 ? group_row(a, s, j, lane) : 0;
                if (vn >= NV<KV4> && !wait_warp(bar + B_VEMPTY + 8 * sl, ((vn / NV<KV4>) - 1) & 1, abort_flag, a.status)) {
                    ok = false;
                    break;
                }
                const uint32_t fb = bar + B_VFULL + 8 * sl, dst = sb + SM_V<KV4> + sl * 32768u;
                // the 16-token group that holds the item's last key and rows behind it
                const int cut = (end & 15) != 0 && (end >> 7) == j ? (end & 127) >> 4 : -1;
                if (cut >= 0) {
                    const int zc = __shfl_sync(0xFFFFFFFFu, z, cut), nrow = end & 15;
                    unsigned char *d = sgen + SM_V<KV4> + sl * 32768u + cut * 2048;
#pragma unroll
                    for (int i = 0; i < 16 * (D / 8) / 32; ++i) {
                        const int c = lane + 32 * i, row = c / (D / 8), ch = c % (D / 8);
                        uint4 w = make_uint4(0u, 0u, 0u, 0u);
                        if (zc >= 0 && row < nrow)
                            w = __ldg(reinterpret_cast<const uint4 *>(
                                          a.v_cache + (((int64_t)zc + row) * a.Hkv + s.h) * D) + ch);
                        *reinterpret_cast<uint4 *>(d + (ch >> 3) * 16384 + row * 128 +
                                                   (((ch & 7) ^ (row & 7)) << 4)) = w;
                    }
                    fence_proxy_async_smem();
                }
                __syncwarp();
                load_boxes<D>(&tm_v, dst, s.h, z, cut, fb, (cut >= 0 ? 14336u : 16384u) * (D / 64));
            }
        }
        for (int m = max(0, vn - NV<KV4>); m < vn; ++m)
            drain_bar(bar + B_VFULL + 8 * (m % NV<KV4>), (m / NV<KV4>) & 1);
    } else if (warp == W_MMA) {
        // ============================================================ MMA issuer
        if (elect_one()) {
            const uint64_t dQ = sdesc_sw128(sb + SM_Q, 16, 1024);
            const uint64_t dK = sdesc_sw128(sb + SM_K<KV4>, 16, 1024);
            const uint64_t dV = sdesc_sw128(sb + SM_V<KV4>, 16384, 1024);
            int kbase = 0, vbase = 0;  // K tiles before the item of the next S, V tiles before the current one
            int kseen = 0, vseen = 0;  // tiles waited for
            uint32_t pbits = 0;        // phase of each group's next P
            bool ok = true;
            auto need = [&](uint32_t b, uint32_t parity) { ok = ok && wait_bar(b, parity, abort_flag, a.status); };
            auto fetch = [&](int k, Seg &s) {
                const int slot = k & (NRING - 1);
                need(bar + B_RFULL + 8 * slot, (k / NRING) & 1);
                s.r = -1;
                if (!ok)
                    return;
                int w[7];
                for (int i = 0; i < 7; ++i)
                    w[i] = ring[8 * slot + i];
                mbar_arrive(bar + B_REMPTY + 8 * slot);
                seg_decode(w, s);
            };
            Seg cur, nxt;
            fetch(0, cur);
            // one body for every product (the thread's code stays in the instruction
            // cache): step j of item k, P V of group g, then that group's next S, which
            // may be the next item's first (j = -1: only the first item's)
            int k = 0, j = -1, g = 0, steps = cur.r >= 0 ? cur.steps(0) : 0;
            nxt.r = -1;
#pragma unroll 1
            while (ok && cur.r >= 0) {
                const bool last = j == steps - 1;
                if (last && g == 0)
                    fetch(k + 1, nxt);
                if (j >= 0 && j < cur.steps(g)) {
                    const int t = vbase + cur.tile(g, j) - cur.t0, sl = t % NV<KV4>;
                    need(bar + B_PFULL + 8 * g, (pbits >> g) & 1);
                    pbits ^= 1u << g;
                    if (t >= vseen) {
                        need(bar + B_VFULL + 8 * sl, (t / NV<KV4>) & 1);
                        vseen = t + 1;
                    }
                    if (!ok)
                        break;
                    tc_fence_after();
                    const uint64_t v = dV + (uint64_t)sl * (32768u >> 4);
                    const uint32_t o = tmem + TM_O + 128u * g, pp = tmem + TM_S + 128u * g;
                    const uint32_t more = j > 0 ? 1u : 0u;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        mma_bf16_ts(o, pp + 8u * i, v + i * (2048u >> 4), IDESC_PV<D, KV4>, i > 0 ? 1u : more);
                    if (cur.split || g == 1)
                        mma_commit(bar + B_VEMPTY + 8 * sl);
                    if (j == cur.steps(g) - 1)
                        mma_commit(bar + B_OFULL + 8 * g);
                }
                // the group's next S: (item, step)
                const bool over = last;
                const Seg &s = over ? nxt : cur;
                const int js = over ? 0 : j + 1;
                if (s.r >= 0 && js < s.steps(g)) {
                    const int t = (over ? kbase + cur.t1 - cur.t0 : kbase) + s.tile(g, js) - s.t0, sl = t % NK;
                    if (js == 0 && g == 0)
                        need(bar + (KV4 ? B_QREADY : B_QFULL), (over ? k + 1 : k) & 1);
                    if (t >= kseen) {
                        need(bar + B_KFULL + 8 * sl, (t / NK) & 1);
                        kseen = t + 1;
                    }
                    if (!ok)
                        break;
                    tc_fence_after();
                    const uint64_t q = dQ + (uint64_t)((!KV4 && !s.split && g) ? (32768u >> 4) : 0u);
                    const uint64_t kk = dK + (uint64_t)sl * (32768u >> 4);
                    const uint32_t d = tmem + TM_S + 128u * g;
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        const uint32_t off = ((i >> 2) * 16384u + (i & 3) * 32u) >> 4;
                        mma_bf16(d, q + off, kk + off, IDESC_QK<KV4>, i > 0 ? 1u : 0u);
                    }
                    mma_commit(bar + B_SFULL + 8 * g);
                    if (s.split || g == 1)
                        mma_commit(bar + B_KEMPTY + 8 * sl);
                    // the item's last S: its Q is free
                    if (s.split ? s.tile(g, js) == s.t1 - 1 : (g == 1 && js == s.steps(1) - 1))
                        mma_commit(bar + B_QEMPTY);
                }
                g ^= 1;
                if (g == 0) {
                    ++j;
                    if (last) {
                        kbase += cur.t1 - cur.t0;
                        vbase = kbase;
                        cur = nxt;
                        ++k;
                        j = 0;
                        steps = cur.r >= 0 ? cur.steps(0) : 0;
                    }
                }
            }
            // wind down: every MMA issued here has completed
            mma_commit(bar + B_FINAL);
            drain_bar(bar + B_FINAL, 0);
        }
        __syncwarp();
    } else if (KV4 && warp >= W_DQ) {
        // ============================================================ codes to fp16 tiles
        const int wq = warp - W_DQ;
        const volatile int *metas = reinterpret_cast<const volatile int *>(sgen + SM_BAR<KV4> + B_META);
        int kn = 0, vn = 0, qn = 0;
        for (int c = 0;; ++c) {
            const int sl = c % NRAW;
            if (!wait_warp(bar + B_RAWFULL + 8 * sl, (c / NRAW) & 1, abort_flag, a.status))
                break;
            const int meta = metas[sl], kind = meta & 0xFF;
            if (kind == CMD_END)
                break;
            uint32_t full;
            if (kind == CMD_Q) {
                if (!wait_warp(bar + B_QFULL, qn & 1, abort_flag, a.status))
                    break;
                const int row = wq * 32 + lane;
                float *rowsc = reinterpret_cast<float *>(sgen + SM_BAR<KV4> + B_ROWSC) + (qn & 1) * 128;
                rowsc[row] = halve_row<D>(sgen + SM_Q, row);
                ++qn;
                full = bar + B_QREADY;
            } else {
                const bool v = kind == CMD_V;
                int &n = v ? vn : kn;
                const int at = n & 1;
                const uint32_t empty = bar + (v ? B_VEMPTY : B_KEMPTY) + 8 * at;
                if (n >= 2 && !wait_warp(empty, ((n >> 1) - 1) & 1, abort_flag, a.status))
                    break;
                dequant_tile<D>(sgen + SM_RAW<KV4> + sl * RAW, sgen + (v ? SM_V<KV4> : SM_K<KV4>) + at * 32768u, meta,
                                wq, lane);
                full = bar + (v ? B_VFULL : B_KFULL) + 8 * at;
                ++n;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(full);
                mbar_arrive(bar + B_RAWEMPTY + 8 * sl);
            }
        }
    } else if (warp < 8) {
        // ============================================================ softmax and epilogue
        regs_inc<REGS_SM<KV4>>();
        const int g = warp >> 2, qw = warp & 3, row = qw * 32 + lane;
        const uint32_t lane_addr = (uint32_t)(qw * 32) << 16;
        const uint32_t s_addr = tmem + lane_addr + TM_S + 128u * g;
        const uint32_t o_addr = tmem + lane_addr + TM_O + 128u * g;
        float2 *ml = reinterpret_cast<float2 *>(sgen + SM_BAR<KV4> + B_ML);
        int n = 0, no = 0, nx = 0;  // tiles, items with tiles, split items so far
        for (int k = 0;; ++k) {
            Seg s;
            if (!ring_get(a, bar, ring, k, lane, abort_flag, s))
                break;
            const int steps = s.steps(g);
            // this row's token, head and last key (rows without a token: the last one's)
            const int tok = ((s.split ? 0 : 128 * g) + row) >> a.g_shift, hl = row & ((1 << a.g_shift) - 1);
            const int pos = s.pos0 + min(tok, s.ntok - 1);
            const int pos_warp = __shfl_sync(0xFFFFFFFFu, pos, 0);  // the warp's least
            float m_used = DDT_NEG_INF, l = 0.f;
            float scale = a.scale_log2;
            bool alive = true;
            for (int j = 0; j < steps; ++j, ++n) {
                if (!wait_warp(bar + B_SFULL + 8 * g, n & 1, abort_flag, a.status)) {
                    alive = false;
                    break;
                }
                tc_fence_after();
                if (KV4 && j == 0)
                    scale = a.scale_log2 * reinterpret_cast<const volatile float *>(sgen + SM_BAR<KV4> + B_ROWSC)[(k & 1) * 128 + row];
                uint32_t sv[128];
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    tmem_ld32(s_addr + 32u * c, sv + 32 * c);
                tmem_wait_ld();
                const int key0 = s.tile(g, j) * PP_TILE;
                if (key0 + PP_TILE - 1 > pos_warp) {
                    const int lim = pos - key0;
#pragma unroll
                    for (int c = 0; c < 128; ++c)
                        if (c > lim)
                            sv[c] = __float_as_uint(DDT_NEG_INF);
                }
                float m4[4] = {DDT_NEG_INF, DDT_NEG_INF, DDT_NEG_INF, DDT_NEG_INF};
#pragma unroll
                for (int c = 0; c < 128; c += 8)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        m4[e] = fmaxf(m4[e], fmaxf(__uint_as_float(sv[c + 2 * e]), __uint_as_float(sv[c + 2 * e + 1])));
                const float mcand = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * scale;
                float alpha = 1.f;
                const bool grow = mcand > m_used + TAU;
                if (grow) {
                    alpha = ex2(m_used - mcand);  // 0 while m_used is -inf
                    m_used = mcand;
                }
                // O rescale (rare): P V of the tile before completed before this S did
                if (__any_sync(0xFFFFFFFFu, grow && j > 0)) {
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t ov[32];
                        tmem_ld32(o_addr + 32u * c, ov);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
                        tmem_st32(o_addr + 32u * c, ov);
                    }
                }
                // P = exp2(scale S - m), rounded to bf16 for the tensor cores (the sum
                // takes the unrounded values); a row with nothing yet has m = -inf
                const float off = (KV4 ? PBIAS : 0.f) - (m_used == DDT_NEG_INF ? 0.f : m_used);
                const uint64_t sc2 = f2pack(scale, scale), nm2 = f2pack(off, off);
                uint64_t sum0 = f2pack(0.f, 0.f), sum1 = sum0;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t pw[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        float x0, x1;
                        f2unpack(f2fma(f2pack(__uint_as_float(sv[64 * c + 2 * e]), __uint_as_float(sv[64 * c + 2 * e + 1])),
                                       sc2, nm2), x0, x1);
                        x0 = ex2(x0);
                        x1 = ex2(x1);
                        pw[e] = KV4 ? pack_f16x2(x0, x1) : pack_bf16x2(x0, x1);
                        if (e & 1)
                            sum1 = f2add(sum1, f2pack(x0, x1));
                        else
                            sum0 = f2add(sum0, f2pack(x0, x1));
                    }
                    tmem_st32(s_addr + 32u * c, pw);
                }
                float r0, r1;
                f2unpack(f2add(sum0, sum1), r0, r1);
                l = l * alpha + (r0 + r1);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar + B_PFULL + 8 * g);
            }
            if (!alive)
                break;
            // ---- epilogue
            if (steps > 0) {
                if (!wait_warp(bar + B_OFULL + 8 * g, no & 1, abort_flag, a.status))
                    break;
                ++no;
                tc_fence_after();
            }
            float fa = 1.f, fb = 0.f;
            bool two = false;
            if (s.split) {
                if (g == 1) {
                    // hand B's (m, l) and O over, and wait until A has read them
                    ml[row] = make_float2(m_used, l);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(bar + B_XB);
                    if (!wait_warp(bar + B_XA, nx & 1, abort_flag, a.status))
                        break;
                    ++nx;
                    continue;
                }
                if (!wait_warp(bar + B_XB, nx & 1, abort_flag, a.status))
                    break;
                ++nx;
                tc_fence_after();
                two = s.steps(1) > 0;
                if (two) {
                    const float2 o = ml[row];
                    const float M = fmaxf(m_used, o.x);
                    fa = m_used == DDT_NEG_INF ? 0.f : ex2(m_used - M);
                    fb = o.x == DDT_NEG_INF ? 0.f : ex2(o.x - M);
                    l = l * fa + o.y * fb;
                    m_used = M;
                }
            }
            const bool row_ok = tok < s.ntok;
            const float inv = s.whole ? (l > 0.f || l != l ? a.out_scale / l : 0.f) : 1.f;
            uint16_t *dst = a.out + ((int64_t)(s.row0 + tok) * a.Hq + (s.h << a.g_shift) + hl) * D;
            const int64_t prow = (int64_t)s.slot * PR_ROWS + (s.split ? 0 : 128 * g) + row;
            float *pdst = a.part_o + prow * D;
            auto at = [](int c) { return KV4 ? position_of(c) : c; };  // column of channel c
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t ov[32];
                tmem_ld32(o_addr + 32u * c, ov);
                if (two) {
                    uint32_t bv[32];
                    tmem_ld32(o_addr + 128u + 32u * c, bv);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        ov[e] = __float_as_uint((__uint_as_float(ov[e]) * fa + __uint_as_float(bv[e]) * fb) * inv);
                } else {
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        ov[e] = __float_as_uint(__uint_as_float(ov[e]) * inv);
                }
                if (row_ok && s.whole) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t w[4];
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            w[x] = pack_bf16x2(__uint_as_float(ov[at(8 * e + 2 * x)]), __uint_as_float(ov[at(8 * e + 2 * x + 1)]));
                        reinterpret_cast<uint4 *>(dst + 32 * c)[e] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                } else if (row_ok) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        reinterpret_cast<uint4 *>(pdst + 32 * c)[e] =
                            make_uint4(ov[at(4 * e)], ov[at(4 * e + 1)], ov[at(4 * e + 2)], ov[at(4 * e + 3)]);
                }
            }
            if (row_ok && !s.whole)
                a.part_ml[prow] = make_float2(m_used, l);
            tc_fence_before();
            if (s.split) {
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar + B_XA);
            }
        }
    }
    // ---- every role has finished or given up
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == W_MMA)
        tmem_dealloc(tmem, TMEM_COLS);
}

// Merge of a cut item: boundary b (between CTAs b - 1 and b) takes the j-th of
// the nb row blocks of the item that it cuts, if it lies among the item's tiles
// (nb: the boundaries that do).
constexpr int MG_THREADS = 256;

template <int D>
__global__ void __launch_bounds__(MG_THREADS) prompt_merge_kernel(const PtArgs a, int grid, int rows)
{
    __shared__ long long s_sums[MG_THREADS / 32], s_found[3];
    const int tq = rows >> a.g_shift, tid = threadIdx.x, b = blockIdx.x + 1;
    find_share(a, tq, grid, b, s_sums, s_found, tid, MG_THREADS);
    if (s_found[0] < 0)
        return;  // no such share
    const long long total = s_found[2], base = s_found[1];
    const int nc = pp_ctas(total, grid, MIN_UNITS);
    const PpReq rq = load_req(a, (int)s_found[0]);
    const long long at = pp_share(total, b, nc);
    const PpItem it = pp_find(rq, at - base, tq, a.Hkv);
    const long long i0 = base + it.start;
    if (pp_tile_at(at - i0) == 0)
        return;  // the item's tiles all lie behind this boundary
    const int c0 = pp_cta_of(i0 + PP_ITEM, total, nc), c1 = pp_cta_of(i0 + PP_ITEM + it.n - 1, total, nc);
    const int ntok = min(tq, rq.len - it.qt * tq), nrows = ntok << a.g_shift, ns = c1 - c0 + 1;
    const int nb = ns - 1, j = b - c0 - 1;
    const int lo = (int)((long long)j * nrows / nb), hi = (int)((long long)(j + 1) * nrows / nb);
    pdl_wait();  // the partials, once the main kernel has completed
    constexpr int C4 = D / 4, RPB = MG_THREADS / C4;  // float4 of a row; rows at a time
    for (int row = lo + tid / C4; row < hi; row += RPB) {
        const int c4 = tid % C4;
        float M = DDT_NEG_INF, L = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int s = 0; s < ns; ++s) {
            const int64_t pr = (int64_t)(s == 0 ? 2 * c0 + 1 : 2 * (c0 + s)) * PR_ROWS + row;
            const float2 ml = __ldcg(&a.part_ml[pr]);
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(a.part_o + pr * D) + c4);
            const float Mn = fmaxf(M, ml.x);
            const float f = M == DDT_NEG_INF ? 0.f : ex2(M - Mn), e = ml.x == DDT_NEG_INF ? 0.f : ex2(ml.x - Mn);
            L = L * f + ml.y * e;
            o.x = o.x * f + v.x * e;
            o.y = o.y * f + v.y * e;
            o.z = o.z * f + v.z * e;
            o.w = o.w * f + v.w * e;
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

// ------------------------------------------------------------------ host side
typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn()
{
    static EncodeTiledFn fn = nullptr;
    if (fn == nullptr) {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = (EncodeTiledFn)p;
    }
    return fn;
}

// 3-D bf16 map: (d, heads, rows) with row_stride elements from row to row and
// a (64, bh, brows) box, 128-byte swizzle
bool make_map(CUtensorMap *m, const void *base, int d, int heads, int64_t rows, int64_t row_stride, int bh, int brows)
{
    EncodeTiledFn f = encode_fn();
    if (f == nullptr)
        return false;
    const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)rows};
    const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)row_stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)bh, (cuuint32_t)brows};
    const cuuint32_t es[3] = {1, 1, 1};
    return f(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box,
             es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool KV4>
cudaError_t launch_d(int grid, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, const PtArgs &a,
                     cudaStream_t s)
{
    cudaError_t e = cudaFuncSetAttribute(prompt_tc_kernel<D, KV4>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)SM_ALLOC<KV4>);
    if (e != cudaSuccess)
        return e;
    // a block launched with fewer registers would wait forever for its split
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, prompt_tc_kernel<D, KV4>);
    if (e != cudaSuccess)
        return e;
    if (fa.numRegs < REGS_LAUNCH<KV4>)
        return cudaErrorLaunchOutOfResources;
    prompt_tc_kernel<D, KV4><<<grid, NT<KV4>, SM_ALLOC<KV4>, s>>>(tq, tk, tv, a);
    e = cudaGetLastError();
    if (e != cudaSuccess || grid == 1)
        return e;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(grid - 1);
    lc.blockDim = dim3(MG_THREADS);
    lc.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = at;
    lc.numAttrs = 1;
    return cudaLaunchKernelEx(&lc, prompt_merge_kernel<D>, a, grid, KV4 ? 128 : PP_ROWS);
}

}  // namespace

cudaError_t launch_prompt_attention(ddt_ctx *c, const uint16_t *q, int64_t q_stride,
                                    const int32_t *q_start, const int32_t *ctx_lens, int R, int T,
                                    const uint16_t *k_cache, const uint16_t *v_cache,
                                    const ddt_kv4 *kv4, const int32_t *block_table, uint16_t *out,
                                    cudaStream_t s)
{
    const ddt_config &cfg = c->cfg;
    const int G = cfg.Hq / cfg.Hkv, d = cfg.d;
    const int64_t rows = cfg.num_pages * cfg.page_size;
    const int64_t dense = (int64_t)cfg.Hkv * d;
    CUtensorMap tq, tk = {}, tv = {};
    if (!make_map(&tq, q, d, cfg.Hq, T, q_stride, G, 128 / G))
        return cudaErrorInvalidValue;
    if (!kv4 && (!make_map(&tk, k_cache, d, cfg.Hkv, rows, dense, 1, 16) ||
                 !make_map(&tv, v_cache, d, cfg.Hkv, rows, dense, 1, 16)))
        return cudaErrorInvalidValue;
    PtArgs a = {};
    a.q_start = q_start;
    a.ctx_lens = ctx_lens;
    a.block_table = block_table;
    a.v_cache = v_cache;
    a.out = out;
    a.part_o = c->att_part_o;
    a.part_ml = c->att_part_ml;
    a.status = c->status;
    a.R = R;
    a.T = T;
    a.Hq = cfg.Hq;
    a.Hkv = cfg.Hkv;
    while ((1 << a.g_shift) < G)
        ++a.g_shift;
    while ((1 << a.page_shift) < cfg.page_size)
        ++a.page_shift;
    a.max_pages = cfg.max_pages_per_req;
    a.cap = cfg.max_pages_per_req * cfg.page_size;
    a.num_pages = cfg.num_pages;
    a.scale_log2 = 1.4426950408889634f / sqrtf((float)d);
    a.out_scale = 1.f;
    if (kv4) {
        a.codes[0] = kv4->k_codes;
        a.codes[1] = kv4->v_codes;
        a.scales[0] = kv4->k_scales;
        a.scales[1] = kv4->v_scales;
        a.scale_log2 *= kv4->k_scale;
        a.out_scale = kv4->v_scale;
    }
    const int grid = c->num_sms < PR_MAX_CTAS ? c->num_sms : PR_MAX_CTAS;
    if (kv4)
        return d == 128 ? launch_d<128, true>(grid, tq, tk, tv, a, s) : launch_d<64, true>(grid, tq, tk, tv, a, s);
    return d == 128 ? launch_d<128, false>(grid, tq, tk, tv, a, s) : launch_d<64, false>(grid, tq, tk, tv, a, s);
}

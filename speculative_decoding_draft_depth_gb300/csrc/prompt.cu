// prompt.cu -- causal attention of packed sequences over the paged cache on the
// 5th-generation tensor cores (tcgen05 + TMEM + TMA), D = 128 and 64.
//
//   O = softmax(scale Q K^T + mask) V, one pass over the keys: with a running m and
//   P = exp2(scale log2(e) S - m), O and l (the row's sum) are sums over the keys,
//   multiplied by exp2(m_old - m_new) when m moves.
//
// Work split (prompt_plan.h): an item is up to 256 rows (256 / G tokens of a
// request with the G heads of one KV head) against the request's key tiles of
// 128; the items of the batch, laid end to end, are cut into equal shares, one
// per CTA (one CTA per SM), each CTA computing its share from q_start and
// ctx_lens. An item cut by a share boundary leaves partial outputs (two slots
// per CTA), merged by prompt_merge_kernel.
//
// Inside a CTA:
//  * two groups, A and B, of 128 rows each (rows in TMEM lanes), worked on in steps
//    of 64 keys: S = Q K^T into one of the group's two buffers of 64 TMEM columns,
//    softmax by the group's four warps (one row per thread, no exchange between
//    threads), P (bf16; fp16 for the 4-bit cache) over the buffer's first 32 columns,
//    O += P V from there. S of the next step is issued before P of this one is
//    waited for, so the softmax warps find their next S ready. An item of at most
//    128 rows (a token or a chain of a few) gives both groups the same rows and
//    alternate key tiles; group A merges the two at the end, reading B's O from TMEM.
//  * m is followed loosely. The common step looks for no maximum: while a row's
//    weights of a step add up to no more than a limit, none of them can overflow or
//    swamp the sums, and m stays. The first step, steps with masked keys and those
//    above the limit read S once more and take the maximum.
//  * bf16 cache: K and V tiles of 128 tokens arrive by TMA in a ring of two K and of
//    three V tiles, one box per 16 tokens and 64 channels.
//  * 4-bit cache: codes and scales arrive by cp.async; eight warps turn them into
//    fp16 tiles (exact) in the same places. Q goes to fp16 by a power of two for
//    each row, in the channel order that the codes' pairs come out in.
//  * warps 0-3: group A; 4-7: group B; 8 and 11: MMA issuers of A and of B; 9: walks
//    the share, loads Q and K; 10: loads V, with the rows past the item's last key
//    zeroed (whatever the page holds there must not meet a probability of zero).
//    4 bits: 9 walks, 10 loads Q, 12-15 make K's tiles and 16-19 V's.
//  * every wait is bounded; on timeout the CTA raises DDT_DEV_TIMEOUT, waits
//    (bounded) for its own copies and MMAs, frees its TMEM and returns.
//
// Measured (GB300; a step of both groups is 2 x 128 rows x 64 keys):
//  * 16384 tokens, 32 heads of 128 over 8 KV heads: 1.34 to 1.50 ms by board and
//    temperature, 1470 to 1640 TFLOP/s. Alone, a launch takes 1300 cycles a step, and the
//    tensor pipe 1286 of them (8 MMAs of N = 64 for S, bound by shared memory at 48
//    cycles each, and 4 of N = 128 for P V, both groups); repeated, the board's power
//    limit lowers the clock (a large bf16 matrix product repeated for seconds: 1740).
//    S of a whole tile at once (N = 128, 32 cycles per 64 keys) needs both buffers, so
//    a group has no next S while its softmax runs: 1.66 ms.
//  * 32 prompts of up to 2047 tokens, 8 heads of 64: 119 to 121 us, of which 132 steps a
//    CTA and its items' outputs account for about 84 (the rest, a quarter, has not been
//    taken apart: first scores of an item, its queries' way, the shares' ends). A step
//    takes 1080 cycles:
//    the softmax of two warps a scheduler (700 to 900, of which 512 are exponentials) and
//    the chain from P over P V to the next S are about as long, so that sixteen softmax
//    warps, a third buffer of S, or sums made by the tensor core each gave 1% or nothing.
//    With the mask and the maximum as branches of one path (registers copied at their
//    joins) 137; the common path by itself 127; zeros at once where a warp's rows have
//    no key 123; an item at three units in the shares 119.
//  * 64 tokens behind 512 to 16384 cached: 361 to 371 us, 6.5 to 6.7 TB/s.
//  * 4-bit cache, four chunks of 1500 to 2048 tokens behind 4000 to 16000: 0.88 to 0.90
//    ms, 1320 to 1350 TFLOP/s; issue slots 60% and the tensor core 65% busy. Each query
//    tile turns the codes into fp16 anew.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "ddt_device.cuh"
#include "ddt_internal.h"
#include "prompt_common.cuh"
#include "tc_ptx.cuh"

namespace {

template <bool KV4>
constexpr int NT = KV4 ? 640 : 384;
constexpr int W_MMA = 8, W_WALK = 9, W_VLOAD = 10, W_MMB = 11, W_DQ = 12;  // (4 bits: 10 loads Q)
constexpr int NDQ = 4;  // 4-bit cache: warps that fetch codes and turn them into fp16 tiles, of K and of V each
// registers per thread of the two softmax warpgroups, of the one with the issuers
// and loaders and of the two that make fp16 tiles, and what the kernel has to be
// launched with: they add up to no more than that
template <bool KV4>
constexpr int REGS_SM = KV4 ? 112 : 208;
template <bool KV4>
constexpr int REGS_OTHER = KV4 ? 64 : 88;
constexpr int REGS_DQ = 96;
template <bool KV4>
constexpr int REGS_LAUNCH = KV4 ? 96 : 168;
static_assert(256 * REGS_SM<true> + 128 * REGS_OTHER<true> + 256 * REGS_DQ <= REGS_LAUNCH<true> * NT<true>, "registers");
static_assert(256 * REGS_SM<false> + 128 * REGS_OTHER<false> <= REGS_LAUNCH<false> * NT<false>, "registers");
constexpr int NRING = 8;
template <bool KV4>
constexpr int RING_CONSUMERS = 8 + 2 + 1 + (KV4 ? 2 * NDQ : 0);  // softmax warps, MMA issuers, V or Q loader, ...
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t TM_S = 0;    // S (and P) of A, B: two buffers of SUB columns each
constexpr uint32_t TM_O = 256;  // O of A, B: 128 columns each
constexpr long long WAIT_LIMIT = 4000000000LL;  // cycles (about 2 s)
constexpr long long DRAIN_LIMIT = 200000000LL;

// shared memory (offsets from a 1024-byte aligned base)
constexpr int NK = 2;
constexpr int SUB = 64;  // keys of a softmax step: half a tile
// scores of a step that a thread holds at a time (64 of them spill beside the 4-bit
// cache's 112 registers: 0.90 ms for four chunks of prompts, in halves 0.88)
template <bool KV4>
constexpr int CHUNK = KV4 ? 32 : SUB;
// what a step's weights of a row may add up to before the maximum is looked for again
template <bool KV4>
constexpr float LIMIT = KV4 ? 32768.f : 256.f;
template <bool KV4>
constexpr int NV = KV4 ? 2 : 3;
constexpr int NRK = 2, NRV = 1;  // 4-bit cache: tiles of K's and of V's codes and scales in flight
constexpr uint32_t RAW = 9216;   // 128 rows of 64 bytes of codes, then of 8 scales
constexpr uint32_t SM_Q = 0;     // A, B: 32 KB each (two 16 KB halves)
constexpr uint32_t SM_K = 65536;
constexpr uint32_t SM_V = SM_K + NK * 32768;
template <bool KV4>
constexpr uint32_t SM_RAW = SM_V + NV<KV4> * 32768;
template <bool KV4>
constexpr uint32_t SM_BAR = SM_RAW<KV4> + (KV4 ? (NRK + NRV) * RAW : 0);
constexpr uint32_t B_QFULL = 0, B_QEMPTY = 8, B_KFULL = 16, B_KEMPTY = 32, B_VFULL = 48, B_VEMPTY = 72,
                   B_SFULL = 96,   // [2 groups][2 buffers]
                   B_PFULL = 128,  // [2][2] 4 arrivals (the group's warps)
                   B_ODONE = 160,  // [2] every P V of the group
                   B_XB = 176,     // B's (m, l) published and its O complete (4 arrivals)
                   B_XA = 184,     // A has read them (4 arrivals)
                   B_FINAL = 192,  // [2]
                   B_OFULL = 208,  // [2] the last P V of an item
                   B_TMEM = 224, B_ABORT = 228,
                   B_QREADY = 232,    // 4 bits: Q is fp16 (NDQ arrivals)
                   B_RFULL = 240,     // [NRING]
                   B_REMPTY = 304,    // [NRING]
                   B_RING = 368,      // [NRING][8] ints
                   B_FOUND = 624,     // three 64-bit words of the share search: apart from the ring, whose first
                                      // entry one lane of the walker writes while others may still read them
                   B_ML = 648,        // [128] float2: B's (m, l); before the roles start, the scan's sums
                   B_ROWSC = 1672;    // 4 bits: [2][256] floats: the row's factor, by item parity
template <bool KV4>
constexpr uint32_t B_END = B_ROWSC + (KV4 ? 2048 : 0);
template <bool KV4>
constexpr uint32_t SM_ALLOC = SM_BAR<KV4> + B_END<KV4> + 1024;
static_assert(B_FOUND >= B_RING + NRING * 8 * 4 && B_ML >= B_FOUND + 3 * 8, "the share search's words are their own");
static_assert(B_ML % 8 == 0 && B_ROWSC >= B_ML + 128 * 8, "(m, l) pairs");
static_assert(SM_ALLOC<false> <= 232448 && SM_ALLOC<true> <= 232448, "shared memory of one CTA");

template <bool KV4>
constexpr uint32_t IDESC_QK = KV4 ? idesc_f16(128, SUB, false, false) : idesc_bf16(128, SUB, false, false);
template <int D, bool KV4>
constexpr uint32_t IDESC_PV = KV4 ? idesc_f16(128, D, false, true) : idesc_bf16(128, D, false, true);

// bounded mbarrier wait; false (and the abort flag raised) on timeout
DDT_DEVINL bool wait_bar_for(uint32_t bar, uint32_t parity, volatile int *abort_flag, int32_t *status, long long limit)
{
    if (mbar_try_wait(bar, parity))
        return true;
    const long long t0 = clock64();
    while (!mbar_try_wait(bar, parity)) {
        if (*abort_flag)
            return false;
        if (clock64() - t0 > limit) {
            *abort_flag = 1;
            atomicOr(status, DDT_DEV_TIMEOUT);
            return false;
        }
    }
    return true;
}
DDT_DEVINL bool wait_bar(uint32_t bar, uint32_t parity, volatile int *abort_flag, int32_t *status)
{
    return wait_bar_for(bar, parity, abort_flag, status, WAIT_LIMIT);
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

// the pool row of that group; -16: none (the TMA fills zeros)
DDT_DEVINL int group_row(const PtArgs &a, const Seg &s, int j, int u)
{
    const int pg = group_page(a, s, j, u);
    return page_ok(a, pg) ? (pg << a.page_shift) + ((j * PP_TILE + 16 * u) & ((1 << a.page_shift) - 1)) : -16;
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

// A warp's part of a tile of codes and scales: 16-byte vectors of codes, CH to a
// row, numbered so that eight neighbouring lanes' stores of the fp16 rows fall into
// eight bank groups; each row's first lane also fetches the row's scales. The
// warp that fetches a part is the one that turns it into values.
template <int D>
struct Part {
    static constexpr int CH = D / 32, N = 128 * CH / (NDQ * 32);
    DDT_DEVINL static int index(int i, int wq, int lane) { return (i * NDQ + wq) * 32 + lane; }
};

// base: lane u holds the byte offset of the tile's 16-token group u in the codes
// (-1: zeros; the scales' is an eighth of it); rows from `valid` on become zeros
template <int D>
DDT_DEVINL void fetch_part(const uint8_t *codes, const uint8_t *scales, long long base, int valid, uint32_t dst, int wq,
                           int lane)
{
    using P = Part<D>;
    long long b[P::N];
#pragma unroll
    for (int i = 0; i < P::N; ++i)
        b[i] = __shfl_sync(0xFFFFFFFFu, base, P::index(i, wq, lane) / P::CH >> 4);
    // this warp's rows' scales: 16 bytes (SR rows) a lane, four lanes to a part
    constexpr int SR = 256 / D;
    const int srow = P::index((lane >> 2) % P::N, wq, 0) / P::CH + (lane & 3) * SR;
    const long long sbase = __shfl_sync(0xFFFFFFFFu, base, srow >> 4);
#pragma unroll
    for (int i = 0; i < P::N; ++i) {
        const int idx = P::index(i, wq, lane), row = idx / P::CH, q = idx % P::CH;
        const bool in = b[i] >= 0 && row < valid;
        cp_async_16(dst + idx * 16, codes + (in ? b[i] + (row & 15) * (D / 2) + q * 16 : 0), in ? 16u : 0u);
    }
    if (lane < 4 * P::N) {
        const int n = sbase >= 0 ? max(0, min(SR, valid - srow)) : 0;
        cp_async_16(dst + 128 * (D / 2) + srow * (D / 16),
                    scales + (n > 0 ? (sbase >> 3) + (srow & 15) * (D / 16) : 0), n * (D / 16));
    }
}

template <int D>
DDT_DEVINL void dequant_part(const unsigned char *rawp, unsigned char *dst, int wq, int lane)
{
    using P = Part<D>;
    uint4 w[P::N];
    uint32_t two[P::N];
#pragma unroll
    for (int i = 0; i < P::N; ++i) {
        const int idx = P::index(i, wq, lane), row = idx / P::CH, q = idx % P::CH;
        w[i] = *reinterpret_cast<const uint4 *>(rawp + idx * 16);
        two[i] = *reinterpret_cast<const uint16_t *>(rawp + 128 * (D / 2) + row * (D / 16) + 2 * q);
    }
#pragma unroll
    for (int i = 0; i < P::N; ++i) {
        const int idx = P::index(i, wq, lane), row = idx / P::CH, q = idx % P::CH;
        uint32_t sc;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(sc) : "h"((uint16_t)two[i]));
        const uint32_t s0 = __byte_perm(sc, sc, 0x1010), s1 = __byte_perm(sc, sc, 0x3232);
        // vectors 4 q + x of the row; lanes of its upper half go in another order
        const bool up = D == 128 && (q & 2);
        const uint32_t wx[4] = {up ? w[i].z : w[i].x, up ? w[i].w : w[i].y, up ? w[i].x : w[i].z,
                                up ? w[i].y : w[i].w};
        const uint32_t sa = up ? s1 : s0, sb = up ? s0 : s1;
        unsigned char *d = dst + (D == 128 ? (q >> 1) * 16384 : 0) + row * 128;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int ch = ((q & 1) * 4 + x) ^ (up ? 2 : 0);
            *reinterpret_cast<uint4 *>(d + ((ch ^ (row & 7)) << 4)) = values8(wx[x], x < 2 ? sa : sb);
        }
    }
}

// lane i of four holds w = quarters 0..3 (four words each) of its own row; after it
// has quarter i of the four lanes' rows
DDT_DEVINL void quads_transpose(uint32_t *w, int lane)
{
    // exchange with lane ^ 2, then lane ^ 1: swap the off-diagonal blocks of 2x2 quarters
#pragma unroll
    for (int x = 2; x >= 1; x >>= 1) {
        const bool up = lane & x;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (q & x)
                continue;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint32_t &lo = w[4 * q + e], &hi = w[4 * (q | x) + e];
                const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, up ? lo : hi, x);
                if (up)
                    lo = got;
                else
                    hi = got;
            }
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
    e = amax >= 0x7F80u ? 0 : max(-100, min(126, e));  // (rows with NaN or inf as they are; 2^-126 is normal)
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
    const int tq = PP_ROWS >> a.g_shift;

    if (tid == 0) {
        mbar_init(bar + B_QFULL, 1);
        mbar_init(bar + B_QEMPTY, 2);
        for (int i = 0; i < NK; ++i) {
            mbar_init(bar + B_KFULL + 8 * i, KV4 ? NDQ : 1);
            mbar_init(bar + B_KEMPTY + 8 * i, 2);
        }
        for (int i = 0; i < NV<KV4>; ++i) {
            mbar_init(bar + B_VFULL + 8 * i, KV4 ? NDQ : 1);
            mbar_init(bar + B_VEMPTY + 8 * i, 2);
        }
        for (int g = 0; g < 2; ++g) {
            for (int b = 0; b < 2; ++b) {
                mbar_init(bar + B_SFULL + 16 * g + 8 * b, 1);
                mbar_init(bar + B_PFULL + 16 * g + 8 * b, 4);
            }
            mbar_init(bar + B_ODONE + 8 * g, 1);
            mbar_init(bar + B_OFULL + 8 * g, 1);
        }
        mbar_init(bar + B_XB, 4);
        mbar_init(bar + B_XA, 4);
        for (int i = 0; i < NRING; ++i) {
            mbar_init(bar + B_RFULL + 8 * i, 1);
            mbar_init(bar + B_REMPTY + 8 * i, RING_CONSUMERS<KV4>);
        }
        mbar_init(bar + B_FINAL, 1);
        mbar_init(bar + B_FINAL + 8, 1);
        mbar_init(bar + B_QREADY, NDQ);
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
    pdl_trigger();  // (the merge stages itself; it waits for this grid before it reads)
    find_share(a, tq, gridDim.x, blockIdx.x, reinterpret_cast<long long *>(sgen + SM_BAR<KV4> + B_ML), found, tid, NT<KV4>);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(sgen + SM_BAR<KV4> + B_TMEM);

    // a whole warp: Q of item k, once the item before is done with its own
    auto load_q = [&](const Seg &s, int k) {
        if (k >= 1 && !wait_warp(bar + B_QEMPTY, (k - 1) & 1, abort_flag, a.status))
            return false;
        if (elect_one()) {
            mbar_arrive_expect_tx(bar + B_QFULL, 16384u * (D / 64) * (s.split ? 1 : 2));
            for (int g = 0; g < (s.split ? 1 : 2); ++g)
                for (int x = 0; x < D / 64; ++x)
                    tma_load_3d(sb + SM_Q + g * 32768 + x * 16384, &tm_q, x * 64, s.h << a.g_shift,
                                s.row0 + g * (tq / 2), bar + B_QFULL);
        }
        __syncwarp();
        return true;
    };

    if (warp >= W_DQ)
        regs_dec<REGS_DQ>();
    else if (warp >= 8)
        regs_dec<REGS_OTHER<KV4>>();

    if (warp == W_WALK) {
        // ============================================================ share walk, Q and K loads
        if (blockIdx.x == 0)
            for (int r = lane; r < a.R; r += 32) {
                const int s0 = __ldg(&a.q_start[r]), s1 = __ldg(&a.q_start[r + 1]);
                if (!packed_ok(s0, s1, a.T, __ldg(&a.ctx_lens[r]), a.cap))
                    atomicOr(a.status, DDT_DEV_BAD_LENGTH);
            }
        ShareWalk walk;
        walk.begin(a, found, tq, gridDim.x, blockIdx.x);
        int k = 0, kn = 0;
        bool ok = true;
        if (a.debug_wait > 0)  // (armed by a test) nothing is announced: this wait runs out, and the other roles give up
            ok = __all_sync(0xFFFFFFFFu, wait_bar_for(bar + B_RFULL, 0, abort_flag, a.status, a.debug_wait));
        while (ok) {
            Seg s;
            walk.next(a, tq, 128, s);
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
            ++k;
            if constexpr (KV4)
                continue;
            if (!load_q(s, k - 1)) {
                --k;  // (k counts the loads of Q under way or over; the parity of one more would pass at once)
                break;
            }
            for (int j = s.t0; j < s.t1; ++j, ++kn) {
                const int sl = kn % NK;
                const int z = lane < 8 ? group_row(a, s, j, lane) : 0;
                if (kn >= NK && !wait_warp(bar + B_KEMPTY + 8 * sl, ((kn / NK) - 1) & 1, abort_flag, a.status)) {
                    ok = false;
                    break;
                }
                const uint32_t fb = bar + B_KFULL + 8 * sl, dst = sb + SM_K + sl * 32768u;
                load_boxes<D>(&tm_k, dst, s.h, z, -1, fb, 16384u * (D / 64));
            }
        }
        // wind down: the copies that this warp issued have landed
        if (!KV4 && k > 0)
            drain_bar(bar + B_QFULL, (k - 1) & 1);
        for (int m = max(0, kn - NK); m < kn; ++m)
            drain_bar(bar + B_KFULL + 8 * (m % NK), (m / NK) & 1);
    } else if (KV4 && warp == W_VLOAD) {
        // ============================================================ Q loads
        int k = 0;
        for (;; ++k) {
            Seg s;
            if (!ring_get(a, bar, ring, k, lane, abort_flag, s) || !load_q(s, k))
                break;
        }
        if (k > 0)
            drain_bar(bar + B_QFULL, (k - 1) & 1);
    } else if (warp == W_VLOAD) {
        // ============================================================ V loads
        uint32_t vfill = 0;  // phase of each slot's next fill
        bool ok = true;
        for (int k = 0; ok; ++k) {
            Seg s;
            if (!ring_get(a, bar, ring, k, lane, abort_flag, s))
                break;
            const int end = s.pos0 + s.ntok;
            int sl = 0;  // the ring of three from the start, or a slot for each group
            for (int j = s.t0; j < s.t1; ++j) {
                const int z = lane < 8 ? group_row(a, s, j, lane) : 0;
                // (a slot never filled passes: its phase "before" is complete)
                if (!wait_warp(bar + B_VEMPTY + 8 * sl, ((vfill >> sl) & 1) ^ 1, abort_flag, a.status)) {
                    ok = false;
                    break;
                }
                vfill ^= 1u << sl;
                const uint32_t fb = bar + B_VFULL + 8 * sl, dst = sb + SM_V + sl * 32768u;
                // the 16-token group that holds the item's last key and rows behind it
                const int cut = (end & 15) != 0 && (end >> 7) == j ? (end & 127) >> 4 : -1;
                if (cut >= 0) {
                    const int zc = __shfl_sync(0xFFFFFFFFu, z, cut), nrow = end & 15;
                    unsigned char *d = sgen + SM_V + sl * 32768u + cut * 2048;
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
                if (++sl == (s.split ? 2 : NV<KV4>))
                    sl = 0;
            }
        }
        for (int m = 0; m < NV<KV4>; ++m)
            drain_bar(bar + B_VFULL + 8 * m, ((vfill >> m) & 1) ^ 1);
    } else if (warp == W_MMA || warp == W_MMB) {
        // ============================================================ MMA issuers, one per group
        if (elect_one()) {
            const uint32_t g = warp == W_MMB;
            const uint64_t dQ = sdesc_sw128(sb + SM_Q, 16, 1024);
            const uint64_t dK = sdesc_sw128(sb + SM_K, 16, 1024);
            const uint64_t dV = sdesc_sw128(sb + SM_V, 16384, 1024);
            const uint32_t o = tmem + TM_O + 128u * g, sp = tmem + TM_S + 128u * g;
            // A parity wait is sound only if the phase before is known to be complete. So
            // in a split item every K and V slot belongs to one group; K's fills of
            // earlier items are complete once this item's Q is there (it waited for both
            // groups' last S), V's once the group's P is (its softmax has finished the
            // item before, with the other group's last product): P is waited for first.
            uint32_t base = 0, n = 0;    // tiles before the item; the group's steps so far
            uint32_t vfill = 0;          // phase of each V slot's next fill, at the item's start
            bool ok = true;
            // (after a wait that gave up, what the body still issues reads and writes
            // this CTA's own memory; the loop then ends)
            auto need = [&](uint32_t b, uint32_t parity) { ok &= wait_bar(b, parity, abort_flag, a.status); };
            for (int k = 0; ok; ++k) {
                const int slot = k & (NRING - 1);
                need(bar + B_RFULL + 8 * slot, (k / NRING) & 1);
                if (!ok)
                    break;
                int w[7];
                for (int i = 0; i < 7; ++i)
                    w[i] = ring[8 * slot + i];
                mbar_arrive(bar + B_REMPTY + 8 * slot);
                Seg s;
                seg_decode(w, s);
                if (s.r < 0)
                    break;
                const int steps = 2 * s.steps(g);
                // the group's first tile and its slots; then every tile, or every second
                const uint32_t first = base + (s.split ? g : 0u), by = s.split ? 2u : 1u;
                uint32_t ks = first % NK, kph = (first / NK) & 1;
                uint32_t vs = s.split ? g : 0u, vbits = vfill;
                const uint64_t q = dQ + (uint64_t)((!s.split && g) ? (32768u >> 4) : 0u);
                need(bar + (KV4 ? B_QREADY : B_QFULL), k & 1);
                // S of step u (into the buffer that P of step u - 2 has left), then P V of
                // step u - 1
#pragma unroll 1
                for (int u = 0; u <= steps && ok; ++u) {
                    const uint32_t b = (n + u) & 1;
                    if (u < steps) {
                        const uint64_t kk = dK + (uint64_t)(ks * (32768u >> 4) + (u & 1) * (SUB * 128u >> 4));
                        const uint32_t d = sp + SUB * b;
                        if ((u & 1) == 0)
                            need(bar + B_KFULL + 8 * ks, kph);
                        tc_fence_after();
#pragma unroll
                        for (int i = 0; i < D / 16; ++i) {
                            const uint32_t off = ((i >> 2) * 16384u + (i & 3) * 32u) >> 4;
                            mma_bf16(d, q + off, kk + off, IDESC_QK<KV4>, i > 0 ? 1u : 0u);
                        }
                        mma_commit(bar + B_SFULL + 16 * g + 8 * b);
                        if (u & 1) {
                            mma_commit(bar + B_KEMPTY + 8 * ks);
                            if (s.split)  // (a slot counts two releases: of both groups, or two of its one)
                                mbar_arrive(bar + B_KEMPTY + 8 * ks);
                            ks += by;
                            if (ks >= NK) {
                                ks -= NK;
                                kph ^= 1;
                            }
                            if (u == steps - 1)  // the group is done with the item's Q
                                mma_commit(bar + B_QEMPTY);
                        }
                    }
                    if (u > 0) {
                        const uint32_t m = n + u - 1, h = (u - 1) & 1, pp = sp + SUB * (m & 1);
                        const uint64_t v = dV + (uint64_t)(vs * (32768u >> 4) + h * (SUB * 128u >> 4));
                        const uint32_t more = u > 1 ? 1u : 0u;
                        need(bar + B_PFULL + 16 * g + 8 * (m & 1), (m >> 1) & 1);
                        if (h == 0)
                            need(bar + B_VFULL + 8 * vs, (vbits >> vs) & 1);
                        tc_fence_after();
#pragma unroll
                        for (int i = 0; i < SUB / 16; ++i)
                            mma_bf16_ts(o, pp + 8u * i, v + i * (2048u >> 4), IDESC_PV<D, KV4>, i > 0 ? 1u : more);
                        mma_commit(bar + B_ODONE + 8 * g);
                        if (u == steps)
                            mma_commit(bar + B_OFULL + 8 * g);
                        if (h) {
                            mma_commit(bar + B_VEMPTY + 8 * vs);
                            if (s.split)
                                mbar_arrive(bar + B_VEMPTY + 8 * vs);
                            vbits ^= 1u << vs;
                            if (!s.split && ++vs == NV<KV4>)
                                vs = 0;
                        }
                    }
                }
                if (steps == 0)  // (the wait for this item's Q keeps this arrival in its phase)
                    mbar_arrive(bar + B_QEMPTY);
                n += steps;
                const uint32_t tiles = s.t1 - s.t0;
                base += tiles;
                vfill = s.split ? vfill ^ (((tiles + 1) >> 1) & 1u) ^ (((tiles >> 1) & 1u) << 1) : vbits;
            }
            // wind down: every MMA issued here has completed
            mma_commit(bar + B_FINAL + 8 * g);
            drain_bar(bar + B_FINAL + 8 * g, 0);
        }
        __syncwarp();
    } else if (KV4 && warp >= W_DQ) {
        // ============================================================ codes to fp16 tiles
        // (one warpgroup K's, the other V's). Fetches run ahead: cp.async into this
        // warp's part of the raw slots, one group a tile.
        const bool v = warp >= W_DQ + NDQ;
        const int wq = warp & 3, ahead = v ? NRV : NRK;
        const uint32_t raws = SM_RAW<KV4> + (v ? NRK * RAW : 0);
        const uint32_t tiles = v ? SM_V : SM_K;
        const uint32_t full = bar + (v ? B_VFULL : B_KFULL), empty = bar + (v ? B_VEMPTY : B_KEMPTY);
        const uint8_t *codes = v ? a.codes[1] : a.codes[0], *scales = v ? a.scales[1] : a.scales[0];
        Seg f;  // the fetched item, and its next tile
        int fk = 0, fj = 0, fend = 0, total = 0x7fffffff;
        int fpage = NO_PAGE;  // lane u: page of group u of that tile (looked at when it is fetched)
        uint32_t info = 0;    // by raw slot: bit 0, tile is its item's first; bit 1, item has both groups' rows
        auto look_up = [&]() { fpage = fj < fend && lane < 8 ? group_page(a, f, fj, lane) : NO_PAGE; };
        auto fetch = [&](int t, int raw) {
            if (total > t) {
                const bool first = fj == fend;
                if (first) {
                    if (ring_get(a, bar, ring, fk, lane, abort_flag, f)) {
                        ++fk;
                        fj = f.t0;
                        fend = f.t1;
                        look_up();
                    } else {
                        total = t;
                    }
                }
                if (total > t) {
                    info = (info & ~(3u << (2 * raw))) | ((first ? 1u : 0u) | (f.split ? 0u : 2u)) << (2 * raw);
                    const long long page0 = ((long long)fpage * a.Hkv + f.h) << a.page_shift;
                    const int in_page = (fj * PP_TILE + 16 * lane) & ((1 << a.page_shift) - 1);
                    const long long fbase = page_ok(a, fpage) ? (page0 + in_page) * (D / 2) : -1;
                    fetch_part<D>(codes, scales, fbase, f.pos0 + f.ntok - fj * PP_TILE, sb + raws + raw * RAW, wq, lane);
                    ++fj;
                    look_up();  // (for the next one)
                }
            }
            cp_async_commit();
        };
        for (int t = 0; t < ahead; ++t)
            fetch(t, t);
        uint32_t fill = 0;  // phase of each fp16 slot's next fill
        int qn = 0, raw = 0, sl = 0;
        for (int t = 0; t < total; ++t) {
            if (v)
                cp_async_wait_group<NRV - 1>();
            else
                cp_async_wait_group<NRK - 1>();
            __syncwarp();
            const uint32_t now = info >> (2 * raw);
            if (now & 1) {
                if (v) {
                    sl = 0;  // (V's slots begin anew with each item)
                } else {
                    if (!wait_warp(bar + B_QFULL, qn & 1, abort_flag, a.status))
                        break;
                    float *rowsc = reinterpret_cast<float *>(sgen + SM_BAR<KV4> + B_ROWSC) + (qn & 1) * 256;
                    for (int g = 0; g < ((now & 2) ? 2 : 1); ++g)
                        rowsc[128 * g + wq * 32 + lane] = halve_row<D>(sgen + SM_Q + g * 32768, wq * 32 + lane);
                    ++qn;
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(bar + B_QREADY);
                }
            }
            // (a slot never filled passes: its phase "before" is complete)
            if (!wait_warp(empty + 8 * sl, ((fill >> sl) & 1) ^ 1, abort_flag, a.status))
                break;
            fill ^= 1u << sl;
            dequant_part<D>(sgen + raws + raw * RAW, sgen + tiles + sl * 32768u, wq, lane);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(full + 8 * sl);
            sl ^= 1;
            fetch(t + ahead, raw);
            raw = raw + 1 == ahead ? 0 : raw + 1;
        }
        cp_async_wait_all();
    } else if (warp < 8) {
        // ============================================================ softmax and epilogue
        regs_inc<REGS_SM<KV4>>();
        const int g = warp >> 2, qw = warp & 3, row = qw * 32 + lane;
        const uint32_t lane_addr = (uint32_t)(qw * 32) << 16;
        const uint32_t s_addr = tmem + lane_addr + TM_S + 128u * g;
        const uint32_t o_addr = tmem + lane_addr + TM_O + 128u * g;
        constexpr int CH = CHUNK<KV4>;
        float2 *ml = reinterpret_cast<float2 *>(sgen + SM_BAR<KV4> + B_ML);
        int n = 0, no = 0, nx = 0;  // the group's steps, items with steps, split items so far
        for (int k = 0;; ++k) {
            Seg s;
            if (!ring_get(a, bar, ring, k, lane, abort_flag, s))
                break;
            const int steps = 2 * s.steps(g);
            // this row's token, head and last key (rows without a token: the last one's)
            const int tok = ((s.split ? 0 : 128 * g) + row) >> a.g_shift, hl = row & ((1 << a.g_shift) - 1);
            const int pos = s.pos0 + min(tok, s.ntok - 1);
            const int pos_warp = __shfl_sync(0xFFFFFFFFu, pos, 0);  // the warp's least and greatest
            const int pos_top = __shfl_sync(0xFFFFFFFFu, pos, 31);
            float m_used = DDT_NEG_INF, l = 0.f;
            float scale = a.scale_log2;
            bool alive = true;
            for (int j = 0; j < steps; ++j, ++n) {
                const uint32_t buf = s_addr + SUB * (n & 1);
                if (!wait_warp(bar + B_SFULL + 16 * g + 8 * (n & 1), (n >> 1) & 1, abort_flag, a.status)) {
                    alive = false;
                    break;
                }
                tc_fence_after();
                if (KV4 && j == 0)
                    scale = row_scale(a, reinterpret_cast<const volatile float *>(
                                             sgen + SM_BAR<KV4> + B_ROWSC)[(k & 1) * 256 + (s.split ? 0 : 128 * g) + row]);
                const int key0 = s.tile(g, j >> 1) * PP_TILE + SUB * (j & 1);
                // P = exp2(scale S - m), rounded to bf16 (fp16 with its range moved up) for
                // the tensor cores; the sum takes the unrounded values. A row with nothing
                // yet has m = -inf.
                auto weigh = [&](const uint32_t (&sv)[CH], uint32_t *pw) {
                    const float off = (KV4 ? PBIAS : 0.f) - (m_used == DDT_NEG_INF ? 0.f : m_used);
                    const uint64_t sc2 = f2pack(scale, scale), nm2 = f2pack(off, off);
                    uint64_t sum0 = f2pack(0.f, 0.f), sum1 = sum0;
#pragma unroll
                    for (int e = 0; e < CH / 2; ++e) {
                        float x0, x1;
                        f2unpack(f2fma(f2pack(__uint_as_float(sv[2 * e]), __uint_as_float(sv[2 * e + 1])), sc2, nm2), x0, x1);
                        x0 = ex2(x0);
                        x1 = ex2(x1);
                        pw[e] = KV4 ? pack_f16x2(x0, x1) : pack_bf16x2(x0, x1);
                        if (e & 1)
                            sum1 = f2add(sum1, f2pack(x0, x1));
                        else
                            sum0 = f2add(sum0, f2pack(x0, x1));
                    }
                    float r0, r1;
                    f2unpack(f2add(sum0, sum1), r0, r1);
                    return r0 + r1;
                };
                auto load = [&](int c, uint32_t (&sv)[CH]) {  // CH columns from c on
#pragma unroll
                    for (int x = 0; x < CH; x += 32)
                        tmem_ld32(buf + c + x, sv + x);
                    tmem_wait_ld();
                };
                auto load_masked = [&](int c, uint32_t (&sv)[CH]) {
                    load(c, sv);
#pragma unroll
                    for (int w = 0; w < CH / 32; ++w) {
                        const int last = pos - key0 - c - 32 * w;  // the row's last key, in these columns
                        const uint32_t mk = last < 0 ? 0u : last >= 31 ? 0xFFFFFFFFu : (2u << last) - 1u;
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!(mk & (1u << e)))
                                sv[32 * w + e] = __float_as_uint(DDT_NEG_INF);
                    }
                };
                // m need not be the row's maximum, only near enough to it: while a step's
                // weights add up to no more than LIMIT, none of them is larger. So the
                // maximum is looked for on the item's first step, with the mask, and when
                // a sum says so (NaN does); S is then read anew, so that no register of
                // the common path outlives a branch (that cost 250 cycles of 1000 a step).
                bool done = false;
                const bool common = j > 0 && key0 + SUB - 1 <= pos_warp;
                if (common) {
                    uint32_t sv[CH], pw[SUB / 2];
                    float sum = 0.f;
#pragma unroll
                    for (int c = 0; c < SUB; c += CH) {
                        load(c, sv);
                        sum += weigh(sv, pw + c / 2);
                    }
                    done = __all_sync(0xFFFFFFFFu, sum <= LIMIT<KV4> && m_used != DDT_NEG_INF);
                    if (done) {
                        l += sum;
                        tmem_st32(buf, pw);
                    }
                }
                if (!KV4 && !common && key0 > pos_top) {
                    // nothing for these rows
                    uint32_t pw[SUB / 2];
#pragma unroll
                    for (int e = 0; e < SUB / 2; ++e)
                        pw[e] = 0;
                    tmem_st32(buf, pw);
                } else if (!done) {
                    uint32_t sv[CH], pw[SUB / 2];
                    float top = DDT_NEG_INF;
#pragma unroll
                    for (int c = 0; c < SUB; c += CH) {
                        load_masked(c, sv);
                        float m4[4] = {DDT_NEG_INF, DDT_NEG_INF, DDT_NEG_INF, DDT_NEG_INF};
#pragma unroll
                        for (int x = 0; x < CH; x += 8)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                m4[e] = fmaxf(m4[e], fmaxf(__uint_as_float(sv[x + 2 * e]), __uint_as_float(sv[x + 2 * e + 1])));
                        top = fmaxf(top, fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])));
                    }
                    top *= scale;
                    // (a sum above the limit moves m even by less than TAU: the next one
                    // would be above it again)
                    if (__any_sync(0xFFFFFFFFu, top > m_used + (common ? 0.f : TAU))) {
                        const float m = fmaxf(m_used, top), alpha = m == m_used ? 1.f : ex2(m_used - m);  // 0 from -inf
                        m_used = m;
                        l *= alpha;
                        if (j > 0) {
                            // O must not have P V of the step before under way (that of the one
                            // before it is complete: this S was issued behind it)
                            if (!wait_warp(bar + B_ODONE + 8 * g, (n - 1) & 1, abort_flag, a.status)) {
                                alive = false;
                                break;
                            }
                            tc_fence_after();
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
                    }
                    if (CH == SUB) {
                        l += weigh(sv, pw);
                    } else {
#pragma unroll
                        for (int c = 0; c < SUB; c += CH) {
                            load_masked(c, sv);
                            l += weigh(sv, pw + c / 2);
                        }
                    }
                    tmem_st32(buf, pw);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar + B_PFULL + 16 * g + 8 * (n & 1));
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
            const int64_t row_off = row_ok ? ((int64_t)(s.row0 + tok) * a.Hq + (s.h << a.g_shift) + hl) * D : -1;
            const int64_t prow = (int64_t)s.slot * PR_ROWS + (s.split ? 0 : 128 * g) + row;
            float4 *pdst = reinterpret_cast<float4 *>(a.part_o + (int64_t)s.slot * PR_ROWS * D) + prow % PR_ROWS;
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
                if (s.whole) {
                    // 64 bytes of this lane's row; four lanes exchange 16-byte quarters so
                    // that each store covers eight rows' whole 64 bytes
                    uint32_t w[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        w[e] = pack_bf16x2(__uint_as_float(ov[at(2 * e)]), __uint_as_float(ov[at(2 * e + 1)]));
                    quads_transpose(w, lane);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int src = (lane & ~3) + e;  // the lane whose row this is
                        const int64_t off = __shfl_sync(0xFFFFFFFFu, row_off, src);
                        if (off >= 0)
                            *reinterpret_cast<uint4 *>(a.out + off + 32 * c + 8 * (lane & 3)) =
                                make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
                    }
                } else if (row_ok) {
                    // partials: float4 columns, rows side by side (coalesced here and in the merge)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        pdst[(8 * c + e) * PR_ROWS] =
                            make_float4(__uint_as_float(ov[at(4 * e)]), __uint_as_float(ov[at(4 * e + 1)]),
                                        __uint_as_float(ov[at(4 * e + 2)]), __uint_as_float(ov[at(4 * e + 3)]));
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
cudaError_t launch_d(int dev, int grid, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, const PtArgs &a,
                     cudaStream_t s)
{
    static DeviceFlags ready;
    cudaError_t e = cudaSuccess;
    if (!ready.test(dev)) {
        e = cudaFuncSetAttribute(prompt_tc_kernel<D, KV4>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)SM_ALLOC<KV4>);
        // a block launched with fewer registers would wait forever for its split
        cudaFuncAttributes fa;
        if (e == cudaSuccess)
            e = cudaFuncGetAttributes(&fa, prompt_tc_kernel<D, KV4>);
        if (e != cudaSuccess)
            return e;
        if (fa.numRegs < REGS_LAUNCH<KV4>)
            return cudaErrorLaunchOutOfResources;
        ready.set(dev);
    }
    prompt_tc_kernel<D, KV4><<<grid, NT<KV4>, SM_ALLOC<KV4>, s>>>(tq, tk, tv, a);
    e = cudaGetLastError();
    if (e != cudaSuccess || grid == 1)
        return e;
    return launch_merge<D>(a, grid, PP_ROWS, s);
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
    // Few rows of a request (on average: lengths are the device's) over the 4-bit
    // cache have a kernel of their own. 64 requests behind 8000, 32/8 heads of 128, this
    // kernel and that one: one token (4 rows) 363 and 140 us, two 364 and 142, four (16
    // rows) 366 and 197, eight (32: it reads the cache twice) 370 and 377. Uneven lengths
    // can lose by it: 63 single tokens and a chunk of 190 behind 8000 171 and 203, 16
    // chains of 16 among 48 empty requests 113 and 194; and 16 single tokens among 48
    // empty requests 109 and 48.
    if (kv4 && (int64_t)T * G <= (int64_t)R * 16)
        return launch_prompt_few(c, a, q, q_stride, G <= 8 && (int64_t)T * G <= (int64_t)R * 8 ? 8 : 16, s);
    CUtensorMap tq, tk = {}, tv = {};
    if (!make_map(&tq, q, d, cfg.Hq, T, q_stride, G, 128 / G))
        return cudaErrorInvalidValue;
    if (!kv4 && (!make_map(&tk, k_cache, d, cfg.Hkv, rows, dense, 1, 16) ||
                 !make_map(&tv, v_cache, d, cfg.Hkv, rows, dense, 1, 16)))
        return cudaErrorInvalidValue;
    const int grid = c->num_sms < PR_MAX_CTAS ? c->num_sms : PR_MAX_CTAS;
    a.debug_wait = c->debug_pr_wait;  // one-shot test setting
    c->debug_pr_wait = 0;
    if (kv4)
        return d == 128 ? launch_d<128, true>(c->device, grid, tq, tk, tv, a, s) : launch_d<64, true>(c->device, grid, tq, tk, tv, a, s);
    return d == 128 ? launch_d<128, false>(c->device, grid, tq, tk, tv, a, s) : launch_d<64, false>(c->device, grid, tq, tk, tv, a, s);
}

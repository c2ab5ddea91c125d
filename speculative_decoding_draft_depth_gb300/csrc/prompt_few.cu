// prompt_few.cu -- attention of few rows over the cache held in 4 bits (a decoding
// step, short chains): at most 8 NR rows of an item, keys as the long side of
// warp-level products, values made in registers.
//
// Why not the kernel of prompt.cu: with few rows the cache's bytes are the bound,
// and there each 128-key tile costs 64 KB of fp16 written to shared memory and as
// much read back by the products, about 1600 cycles at 128 bytes a cycle, against
// 900 for the tile's codes from HBM. Here a warp takes 16 keys at a time straight
// from global memory to registers, where the codes become the products' A operand:
//   S^T (16 keys x 8 rows) = K Q^T:  lane (i, c) = (lane / 4, lane % 4) holds keys i
//     and i + 8, channels [c D/4, (c + 1) D/4) -- 16 bytes of codes of a key, whose
//     pairs go to the products as they come; Q's are laid out alike, once an item;
//   O^T (channels x 8 rows) += V^T P^T: lane (i, c) holds keys 2c, 2c + 1, 2c + 8,
//     2c + 9, channels [i D/8, (i + 1) D/8); two keys' codes of one channel are
//     put into one byte, so that they come out as the pair the product takes, and
//     P^T is transposed in the warp.
// Eight warps of a CTA take the 16-key blocks of a segment in turn, each with its
// own running maximum and sum, and meet at the segment's end; four blocks a warp
// are in flight (cp.async into a ring of the warp's own). Shares of the work and the merge of
// cut items as in prompt.cu.
//
// Measured (64 tokens behind 512 to 16384, 32/8 heads of 128, 680 MB): 160 us, 4.25 TB/s;
// the bytes alone would take 101. No pipe is full: issue slots 63%, the ALU pipe (half of
// it the codes' way to fp16 and the byte shuffles for V) 56%, HBM 50%. Four warps a
// scheduler are what hides the dependent chains, and in 37% of the cycles none of them can
// issue. Two CTAs of 8 rows an SM (registers and shared memory); 16 rows (four tokens)
// need twice the registers and go one to an SM.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "prompt_common.cuh"
#include "tc_ptx.cuh"

namespace {

constexpr int FW = 8;  // warps of a CTA
constexpr int FT = FW * 32;
constexpr int FS = 4;  // blocks that a warp has in flight

struct FewArgs {
    PtArgs a;
    const uint16_t *q;
    int64_t q_stride;
};

DDT_DEVINL void mma_f16(float *d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// an 8 x 8 matrix of 16-bit values (lane: row lane / 4, columns 2 (lane % 4), + 1), transposed
DDT_DEVINL uint32_t transpose8(uint32_t x)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
DDT_DEVINL uint32_t scales2(uint32_t two)  // e4m3 pair -> fp16 pair
{
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
    return r;
}

// one lane's codes of a 16-key block
template <int D>
struct Block {
    static constexpr int KW = D / 32;  // words of a key's codes (K); V: half as many
    uint32_t k[2][KW], ks[2];
    uint32_t v[4][KW / 2], vs[4];
};

// A raw block in shared memory: 16 keys' codes of K, of V, then their scales. A key's
// row of V lies in the line of its pair of keys, at a half and a quarter that spread
// the eight-byte reads of four even (or odd) keys over all banks (D = 128).
template <int D>
constexpr uint32_t RAW_CODES = 16 * (D / 2);
template <int D>
constexpr uint32_t RAW_SCALES = 16 * (D / 16);
template <int D>
constexpr uint32_t RAW_BYTES = 2 * (RAW_CODES<D> + RAW_SCALES<D>);
template <int D>
DDT_DEVINL uint32_t v_place(int key, int q)  // of 16-byte vector q of the key's codes
{
    if (D == 128)
        return (key >> 1) * 128 + (((key & 1) ^ ((key >> 2) & 1)) << 6) + ((q ^ (key & 2)) << 4);
    return key * 32 + q * 16;
}

// Where a lane's copies of a block begin: vectors lane, lane + 32 of the codes (of K
// and V alike), and one vector of scales for the first lanes.
template <int D>
struct Copier {
    static constexpr int CH = D / 32, RS = 256 / D, NS = 16 / RS;  // vectors of a key's codes; keys, vectors of scales
    const uint8_t *k, *v, *s;  // the pools' bases, moved by the lane's place (s: K's or V's scales)
    uint32_t vdst[16 * CH / 32], sdst;

    DDT_DEVINL void begin(const PtArgs &a, int lane)
    {
        k = a.codes[0] + lane * 16;
        v = a.codes[1] + lane * 16;
        const int sv = lane / NS, first = lane % NS * RS;
        s = (sv ? a.scales[1] : a.scales[0]) + first * (D / 16);
        sdst = 2 * RAW_CODES<D> + sv * RAW_SCALES<D> + first * (D / 16);
#pragma unroll
        for (int x = 0; x < 16 * CH / 32; ++x)
            vdst[x] = RAW_CODES<D> + v_place<D>((x * 32 + lane) / CH, (x * 32 + lane) % CH);
    }

    // start the copies of a block into dst; page: the block's (NO_PAGE: no rows); rows
    // of keys from `end` on become zeros
    DDT_DEVINL void fetch(const PtArgs &a, uint32_t dst, int page, int key0, int end, int h, int lane) const
    {
        const bool ok = page_ok(a, page);
        const int64_t row = (((int64_t)(ok ? page : 0) * a.Hkv + h) << a.page_shift) + (key0 & ((1 << a.page_shift) - 1));
        const int n = ok ? end - key0 : 0;  // keys that count
        const int64_t at = row * (D / 2);
        if (n >= 16) {
#pragma unroll
            for (int x = 0; x < 16 * CH / 32; ++x) {
                cp_async_16(dst + lane * 16 + x * 512, k + at + x * 512, 16);
                cp_async_16(dst + vdst[x], v + at + x * 512, 16);
            }
            if (lane < 2 * NS)
                cp_async_16(dst + sdst, s + (at >> 3), 16);
            return;
        }
#pragma unroll
        for (int x = 0; x < 16 * CH / 32; ++x) {
            const bool in = (x * 32 + lane) / CH < n;
            cp_async_16(dst + lane * 16 + x * 512, k + (in ? at + x * 512 : 0), in ? 16u : 0u);
            cp_async_16(dst + vdst[x], v + (in ? at + x * 512 : 0), in ? 16u : 0u);
        }
        if (lane < 2 * NS) {
            const int c = max(0, min(RS, n - lane % NS * RS));
            cp_async_16(dst + sdst, s + (c > 0 ? at >> 3 : 0), c * (D / 16));
        }
    }
};

template <int D>
DDT_DEVINL void read_block(const unsigned char *raw, Block<D> &b, int lane)
{
    const int i = lane >> 2, c = lane & 3;
    const unsigned char *vr = raw + RAW_CODES<D>, *ks = vr + RAW_CODES<D>, *vs = ks + RAW_SCALES<D>;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int key = i + 8 * x;
        if constexpr (D == 128) {
            const uint4 w = *reinterpret_cast<const uint4 *>(raw + key * 64 + c * 16);
            b.k[x][0] = w.x, b.k[x][1] = w.y, b.k[x][2] = w.z, b.k[x][3] = w.w;
            b.ks[x] = *reinterpret_cast<const uint16_t *>(ks + key * 8 + c * 2);
        } else {
            const uint2 w = *reinterpret_cast<const uint2 *>(raw + key * 32 + c * 8);
            b.k[x][0] = w.x, b.k[x][1] = w.y;
            b.ks[x] = ks[key * 4 + c];
        }
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        const int key = 2 * c + (x & 1) + 8 * (x >> 1);
        if constexpr (D == 128) {
            const uint2 w = *reinterpret_cast<const uint2 *>(vr + v_place<D>(key, i >> 1) + (i & 1) * 8);
            b.v[x][0] = w.x, b.v[x][1] = w.y;
            b.vs[x] = vs[key * 8 + i];
        } else {
            b.v[x][0] = *reinterpret_cast<const uint32_t *>(vr + key * 32 + i * 4);
            b.vs[x] = vs[key * 4 + (i >> 1)];
        }
    }
}

template <int D, int NR>
__global__ void __launch_bounds__(FT, NR == 1 ? 2 : 1) prompt_few_kernel(const FewArgs f)
{
    constexpr int ROWS = 8 * NR, KW = Block<D>::KW, KS = D / 16, CH = D / 8;  // CH: channels of a lane's V
    extern __shared__ float4 few_smem[];
    float *so = reinterpret_cast<float *>(few_smem);  // [FW][ROWS][D]
    float2 *sml = reinterpret_cast<float2 *>(so + FW * ROWS * D);  // [FW][ROWS]
    unsigned char *rawp = reinterpret_cast<unsigned char *>(sml + FW * ROWS) + (threadIdx.x >> 5) * FS * RAW_BYTES<D>;
    const uint32_t raws = (uint32_t)__cvta_generic_to_shared(rawp);
    __shared__ long long s_sums[FW], s_found[3];
    const PtArgs &a = f.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, i = lane >> 2, c = lane & 3;
    const int tq = ROWS >> a.g_shift, G = 1 << a.g_shift;
    if (blockIdx.x == 0)
        for (int r = tid; r < a.R; r += FT) {
            const int s0 = __ldg(&a.q_start[r]), s1 = __ldg(&a.q_start[r + 1]);
            if (!packed_ok(s0, s1, a.T, __ldg(&a.ctx_lens[r]), a.cap))
                set_status(a.status, DDT_DEV_BAD_LENGTH);
        }
    pdl_trigger();  // (the merge stages itself; it waits for this grid before it reads)
    find_share(a, tq, gridDim.x, blockIdx.x, s_sums, s_found, tid, FT);
    Copier<D> copier;
    copier.begin(a, lane);
    ShareWalk walk;
    walk.begin(a, s_found, tq, gridDim.x, blockIdx.x);
    // this warp's blocks of a segment: the next one, their end, the page of the one FS
    // turns ahead; their copies begin while the segment before is merged
    int blk = 0, bend = 0, page = NO_PAGE;
    Seg s = {};
    auto page_of = [&](int b) {
        return b < bend ? __ldg(a.block_table + (int64_t)s.r * a.max_pages + ((b * 16) >> a.page_shift)) : NO_PAGE;
    };
    auto fetch = [&](int b, int pg, int slot) {  // (nothing beyond the end: a slot has one copy under way)
        if (b < bend)
            copier.fetch(a, raws + slot * RAW_BYTES<D>, pg, b * 16, s.pos0 + s.ntok, s.h, lane);
        cp_async_commit();
    };
    auto start = [&]() {
        walk.next(a, tq, 0, s);
        if (s.r < 0)
            return;
        bend = (min(s.pos0 + s.ntok, s.t1 * PP_TILE) + 15) >> 4;
        blk = s.t0 * (PP_TILE / 16) + warp;
        int pg[FS];
#pragma unroll
        for (int x = 0; x < FS; ++x)
            pg[x] = page_of(blk + x * FW);
        page = page_of(blk + FS * FW);
#pragma unroll
        for (int x = 0; x < FS; ++x)
            fetch(blk + x * FW, pg[x], x);
    };
    start();
    while (s.r >= 0) {
        const int nrows = s.ntok << a.g_shift;
        int slot = 0;
        // ---- Q: row 8 y + i, channels [c D/4, + D/4), divided by a power of two of the
        //      row's largest magnitude, to fp16 in the order of the codes' pairs
        uint32_t qf[NR][2 * KS];
        float sc[NR][2], m[NR][2], l[NR][2], o[NR][KS][4];
        float top[NR][2], off[NR][2];  // the score that moves the reference; what is added in the exponent
        int pos[NR][2];
#pragma unroll
        for (int y = 0; y < NR; ++y) {
            const int row = 8 * y + i;
            uint4 w[D / 32];
#pragma unroll
            for (int x = 0; x < D / 32; ++x)
                w[x] = make_uint4(0u, 0u, 0u, 0u);
            if (row < nrows) {
                const uint16_t *src = f.q + (int64_t)(s.row0 + (row >> a.g_shift)) * f.q_stride +
                                      ((s.h << a.g_shift) + (row & (G - 1))) * D + c * (D / 4);
#pragma unroll
                for (int x = 0; x < D / 32; ++x)
                    w[x] = __ldg(reinterpret_cast<const uint4 *>(src) + x);
            }
            uint32_t amax = 0;
#pragma unroll
            for (int x = 0; x < D / 32; ++x) {
                const uint32_t u[4] = {w[x].x, w[x].y, w[x].z, w[x].w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    amax = max(amax, max(u[e] & 0x7FFFu, (u[e] >> 16) & 0x7FFFu));
            }
            amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
            amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
            int e2 = (int)(amax >> 7) - 127;
            e2 = amax >= 0x7F80u ? 0 : max(-100, min(126, e2));  // (rows with NaN or inf as they are; 2^-126 is normal)
            const float down = __uint_as_float((uint32_t)(127 - e2) << 23);
            const float up = row_scale(a, __uint_as_float((uint32_t)(127 + e2) << 23));
#pragma unroll
            for (int x = 0; x < D / 32; ++x) {
                const float v[8] = {bf16lo(w[x].x), bf16hi(w[x].x), bf16lo(w[x].y), bf16hi(w[x].y),
                                    bf16lo(w[x].z), bf16hi(w[x].z), bf16lo(w[x].w), bf16hi(w[x].w)};
                qf[y][4 * x] = pack_f16x2(v[0] * down, v[2] * down);
                qf[y][4 * x + 1] = pack_f16x2(v[4] * down, v[6] * down);
                qf[y][4 * x + 2] = pack_f16x2(v[1] * down, v[3] * down);
                qf[y][4 * x + 3] = pack_f16x2(v[5] * down, v[7] * down);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {  // this lane's columns of S^T: rows 8 y + 2 c, + 1
                sc[y][e] = __shfl_sync(0xFFFFFFFFu, up, (2 * c + e) * 4);
                m[y][e] = top[y][e] = DDT_NEG_INF;
                off[y][e] = PBIAS;
                l[y][e] = 0.f;
                pos[y][e] = s.pos0 + min((8 * y + 2 * c + e) >> a.g_shift, s.ntok - 1);
            }
#pragma unroll
            for (int j = 0; j < KS; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    o[y][j][e] = 0.f;
        }
        for (; blk < bend; blk += FW) {
            cp_async_wait_group<FS - 1>();
            __syncwarp();
            Block<D> b;
            read_block<D>(rawp + slot * RAW_BYTES<D>, b, lane);
            __syncwarp();
            fetch(blk + FS * FW, page, slot);
            page = page_of(blk + (FS + 1) * FW);
            slot = slot + 1 == FS ? 0 : slot + 1;
            // ---- S^T
            float st[NR][4], su[NR][4];  // (two sums: half the products wait for one another)
#pragma unroll
            for (int y = 0; y < NR; ++y)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    st[y][e] = su[y][e] = 0.f;
            uint32_t s2[2];
#pragma unroll
            for (int x = 0; x < 2; ++x)
                s2[x] = scales2(D == 128 ? b.ks[x] : b.ks[x] * 0x0101u);
#pragma unroll
            for (int w = 0; w < KW; ++w) {
                // (D = 128: words 0, 1 lie in the first of the lane's two blocks)
                const uint32_t sel = (D == 128 && w >= 2) ? 0x3232u : 0x1010u;
                const uint4 x0 = values8(b.k[0][w], __byte_perm(s2[0], s2[0], sel));
                const uint4 x1 = values8(b.k[1][w], __byte_perm(s2[1], s2[1], sel));
#pragma unroll
                for (int y = 0; y < NR; ++y) {
                    mma_f16(st[y], x0.x, x1.x, x0.y, x1.y, qf[y][4 * w], qf[y][4 * w + 1]);
                    mma_f16(su[y], x0.z, x1.z, x0.w, x1.w, qf[y][4 * w + 2], qf[y][4 * w + 3]);
                }
            }
#pragma unroll
            for (int y = 0; y < NR; ++y)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    st[y][e] += su[y][e];
            // ---- softmax: keys key0 + i and + 8, rows 2 c and 2 c + 1
            const int key0 = blk * 16;
            if (key0 + 15 > s.pos0) {
#pragma unroll
                for (int y = 0; y < NR; ++y)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (key0 + i + 8 * (e >> 1) > pos[y][e & 1])
                            st[y][e] = DDT_NEG_INF;
            }
            bool grow = false;
#pragma unroll
            for (int y = 0; y < NR; ++y)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    grow |= fmaxf(st[y][e], st[y][e + 2]) > top[y][e];
            if (__any_sync(0xFFFFFFFFu, grow)) {
#pragma unroll
                for (int y = 0; y < NR; ++y)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float mx = fmaxf(st[y][e], st[y][e + 2]);
#pragma unroll
                        for (int x = 4; x <= 16; x <<= 1)
                            mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, x));
                        mx *= sc[y][e];
                        if (mx > m[y][e]) {
                            const float alpha = ex2(m[y][e] - mx);
                            m[y][e] = mx;
                            off[y][e] = PBIAS - mx;
                            top[y][e] = (mx + TAU) / sc[y][e];
                            l[y][e] *= alpha;
#pragma unroll
                            for (int j = 0; j < KS; ++j) {
                                o[y][j][e] *= alpha;
                                o[y][j][e + 2] *= alpha;
                            }
                        }
                    }
            }
            uint32_t pb[NR][2];
#pragma unroll
            for (int y = 0; y < NR; ++y) {
                float p[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    p[e] = ex2(fmaf(st[y][e], sc[y][e & 1], off[y][e & 1]));
                    l[y][e & 1] += p[e];
                }
                pb[y][0] = transpose8(pack_f16x2(p[0], p[1]));
                pb[y][1] = transpose8(pack_f16x2(p[2], p[3]));
            }
            // ---- O^T
            // keys 2c, 2c + 1 (and + 8) pair up before they are converted: a byte takes one
            // channel's code of either key
            uint32_t vsc[2];
#pragma unroll
            for (int x = 0; x < 2; ++x)
                vsc[x] = scales2(b.vs[2 * x + 1] * 256u + b.vs[2 * x]);
#pragma unroll
            for (int w = 0; w < KW / 2; ++w) {
                uint4 lo[2], hi[2];  // of either pair of keys: channels {0, 4, 1, 5}, and those + 2
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const uint32_t ka = b.v[2 * x][w], kb = b.v[2 * x + 1][w], mask = 0x0F0F0F0Fu;
                    lo[x] = values8((ka & mask) | ((kb * 16u) & ~mask), vsc[x]);
                    hi[x] = values8(((ka >> 4) & mask) | (kb & ~mask), vsc[x]);
                }
                const uint32_t l0[4] = {lo[0].x, lo[0].y, lo[0].z, lo[0].w}, h0[4] = {hi[0].x, hi[0].y, hi[0].z, hi[0].w};
                const uint32_t l1[4] = {lo[1].x, lo[1].y, lo[1].z, lo[1].w}, h1[4] = {hi[1].x, hi[1].y, hi[1].z, hi[1].w};
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int y = 0; y < NR; ++y)
                        mma_f16(o[y][4 * w + q], l0[q], h0[q], l1[q], h1[q], pb[y][0], pb[y][1]);
            }
        }
        const Seg was = s;
        start();
        // ---- the warps' parts to shared memory: O row by row, (m, l)
#pragma unroll
        for (int y = 0; y < NR; ++y)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = 8 * y + 2 * c + e;
#pragma unroll
                for (int x = 4; x <= 16; x <<= 1)
                    l[y][e] += __shfl_xor_sync(0xFFFFFFFFu, l[y][e], x);
                if (i == 0)
                    sml[warp * ROWS + row] = make_float2(m[y][e], l[y][e]);
                float *dst = so + (warp * ROWS + row) * D + i * CH;
                // product 4 w + q holds channels {0, 4, 1, 5}[q] and those + 2 of word w
#pragma unroll
                for (int w = 0; w < KW / 2; ++w) {
                    reinterpret_cast<float4 *>(dst)[2 * w] =
                        make_float4(o[y][4 * w][e], o[y][4 * w + 2][e], o[y][4 * w][e + 2], o[y][4 * w + 2][e + 2]);
                    reinterpret_cast<float4 *>(dst)[2 * w + 1] =
                        make_float4(o[y][4 * w + 1][e], o[y][4 * w + 3][e], o[y][4 * w + 1][e + 2], o[y][4 * w + 3][e + 2]);
                }
            }
        __syncthreads();
        for (int e = tid; e < nrows * (D / 4); e += FT) {
            const int row = e / (D / 4), c4 = e % (D / 4);
            float M = DDT_NEG_INF, L = 0.f;
#pragma unroll
            for (int w = 0; w < FW; ++w)
                M = fmaxf(M, sml[w * ROWS + row].x);
            float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < FW; ++w) {
                const float2 ml = sml[w * ROWS + row];
                const float k = ml.x == DDT_NEG_INF ? 0.f : ex2(ml.x - M);
                const float4 v = reinterpret_cast<const float4 *>(so + (w * ROWS + row) * D)[c4];
                L += ml.y * k;
                r.x += v.x * k;
                r.y += v.y * k;
                r.z += v.z * k;
                r.w += v.w * k;
            }
            if (was.whole) {
                const float inv = L > 0.f || L != L ? a.out_scale / L : 0.f;
                uint32_t *dst = reinterpret_cast<uint32_t *>(
                    a.out + ((int64_t)(was.row0 + (row >> a.g_shift)) * a.Hq + (was.h << a.g_shift) + (row & (G - 1))) * D) + 2 * c4;
                *reinterpret_cast<uint2 *>(dst) =
                    make_uint2(pack_bf16x2(r.x * inv, r.y * inv), pack_bf16x2(r.z * inv, r.w * inv));
            } else {
                reinterpret_cast<float4 *>(a.part_o + (int64_t)was.slot * ROWS * D)[c4 * ROWS + row] = r;
                if (c4 == 0)
                    a.part_ml[(int64_t)was.slot * ROWS + row] = make_float2(M, L);
            }
        }
        __syncthreads();
    }
    cp_async_wait_all();
}

template <int D, int NR>
cudaError_t launch_few(const FewArgs &f, int dev, int num_sms, cudaStream_t s)
{
    constexpr int ROWS = 8 * NR, BYTES = FW * (ROWS * (D * 4 + 8) + FS * RAW_BYTES<D>);
    static_assert(ROWS * 2 * 2 * PR_MAX_CTAS <= 2 * PR_MAX_CTAS * PR_ROWS, "partial slots");
    static DeviceFlags ready;
    cudaError_t e = cudaSuccess;
    if (!ready.test(dev)) {
        e = cudaFuncSetAttribute(prompt_few_kernel<D, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize, BYTES);
        if (e != cudaSuccess)
            return e;
        ready.set(dev);
    }
    const int grid = (num_sms < PR_MAX_CTAS ? num_sms : PR_MAX_CTAS) * (NR == 1 ? 2 : 1);
    prompt_few_kernel<D, NR><<<grid, FT, BYTES, s>>>(f);
    e = cudaGetLastError();
    if (e != cudaSuccess || grid == 1)
        return e;
    return launch_merge<D>(f.a, grid, ROWS, s);
}

}  // namespace

cudaError_t launch_prompt_few(ddt_ctx *c, const PtArgs &a, const uint16_t *q, int64_t q_stride, int rows, cudaStream_t s)
{
    FewArgs f;
    f.a = a;
    f.q = q;
    f.q_stride = q_stride;
    if (c->cfg.d == 128)
        return rows <= 8 ? launch_few<128, 1>(f, c->device, c->num_sms, s) : launch_few<128, 2>(f, c->device, c->num_sms, s);
    return rows <= 8 ? launch_few<64, 1>(f, c->device, c->num_sms, s) : launch_few<64, 2>(f, c->device, c->num_sms, s);
}

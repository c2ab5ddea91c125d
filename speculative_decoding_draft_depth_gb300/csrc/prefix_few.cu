// prefix_few.cu -- attention of few rows over their requests' own bf16 keys, behind a
// shared prefix: a decoding step's part that is not shared. At most 8 NR rows of an item.
//
// Why not the kernel of prompt_tc.cuh: own keys are short (some hundreds), so its items are
// a few tiles each, and an item costs it 5 us besides its tiles: its queries' way, the
// first scores, the accumulators' way out. Here a warp takes 16 keys at a time, each warp on
// its own, and an item ends with one exchange through shared memory:
//   S^T (16 keys x 8 rows) = K Q^T, K's rows by ldmatrix, Q's in registers;
//   O^T (16 channels x 8 rows) += V^T P^T, V by transposing ldmatrix, P^T transposed in the
//   warp.
// Four warps of a CTA take the 16-key blocks of a segment in turn, each with its own running
// maximum and sum; blocks come by cp.async into a ring of the warp's own, 16-byte vectors of
// a key's row exchanged by the key's low bits (the ldmatrix rows then lie in all banks).
// Shares of the work as in prompt_plan.h; the parts are added up by prefix_merge_kernel.
// Measured: own keys of 64 requests, 1 to 1024 each, 32/8 heads of 128: 36 us alone and cold
// (47 % of HBM's rate).
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "prompt_common.cuh"
#include "tc_ptx.cuh"

namespace {

constexpr int OW = 4;  // warps of a CTA (two CTAs an SM)
constexpr int OT = OW * 32;
template <int NR>
constexpr int OS = NR == 1 ? 3 : 2;  // blocks that a warp has in flight

struct OwnArgs {
    PtArgs a;
    const uint16_t *q, *k_cache;
    int64_t q_stride;
};

DDT_DEVINL void mma_b16(float *d, const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
DDT_DEVINL void ldmatrix4(uint32_t (&r)[4], uint32_t at)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
DDT_DEVINL void ldmatrix4_t(uint32_t (&r)[4], uint32_t at)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
DDT_DEVINL uint32_t transpose8(uint32_t x)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// a block in shared memory: 16 keys' rows of K, then of V
template <int D>
constexpr uint32_t OWN_ROW = 2 * D;
template <int D>
constexpr uint32_t OWN_BLOCK = 2 * 16 * OWN_ROW<D>;
// of 16-byte vector x of key's row
template <int D>
DDT_DEVINL uint32_t own_place(int key, int x) { return key * OWN_ROW<D> + ((x ^ (key & 7)) << 4); }

template <int D, int NR>
__global__ void __launch_bounds__(OT, 2) own_few_kernel(const OwnArgs f)
{
    constexpr int ROWS = 8 * NR, KS = D / 16, S = OS<NR>;
    extern __shared__ float4 own_smem[];
    float *so = reinterpret_cast<float *>(own_smem);               // [OW][ROWS][D]
    float2 *sml = reinterpret_cast<float2 *>(so + OW * ROWS * D);  // [OW][ROWS]
    const uint32_t raws = (uint32_t)__cvta_generic_to_shared(sml + OW * ROWS) + (threadIdx.x >> 5) * S * OWN_BLOCK<D>;
    __shared__ long long s_sums[OW], s_found[4];
    const PtArgs &a = f.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, i = lane >> 2, c = lane & 3;
    const int tq = ROWS >> a.g_shift, G = 1 << a.g_shift;
    if (blockIdx.x == 0)
        for (int r = tid; r < a.R; r += OT) {
            bool sound;
            load_req<OWN>(a, r, &sound);
            if (!sound)
                set_status(a.status, DDT_DEV_BAD_LENGTH);
        }
    pdl_trigger();  // (the merge stages itself; it waits for this grid before it reads)
    find_share<OWN>(a, tq, gridDim.x, blockIdx.x, s_sums, s_found, tid, OT);
    ShareWalk<OWN> walk;
    walk.begin(a, s_found, tq, blockIdx.x);
    int blk = 0, bend = 0, page = NO_PAGE;
    Seg s = {};
    auto page_of = [&](int b) {
        return b < bend ? __ldg(a.block_table + (int64_t)s.r * a.max_pages + ((b * 16) >> a.page_shift)) : NO_PAGE;
    };
    // start the copies of block b into a slot (nothing beyond the end); rows of keys past the
    // item's last, and of pages out of range, become zeros
    auto fetch = [&](int b, int pg, int slot) {
        if (b < bend) {
            const bool ok = page_ok(a, pg);
            const int key0 = b * 16, n = ok ? s.end() - key0 : 0;
            const int64_t row = (((int64_t)(ok ? pg : 0) << a.page_shift) + (key0 & ((1 << a.page_shift) - 1))) * a.Hkv + s.h;
            const uint32_t dst = raws + slot * OWN_BLOCK<D>;
#pragma unroll
            for (int x = 0; x < 16 * D / 8 / 32; ++x) {
                const int v = x * 32 + lane, key = v / (D / 8), ch = v % (D / 8);
                const int64_t at = (row + (int64_t)key * a.Hkv) * D + ch * 8;
                const uint32_t bytes = key < n ? 16 : 0;
                cp_async_16(dst + own_place<D>(key, ch), f.k_cache + (bytes ? at : 0), bytes);
                cp_async_16(dst + 16 * OWN_ROW<D> + own_place<D>(key, ch), a.v_cache + (bytes ? at : 0), bytes);
            }
        }
        cp_async_commit();
    };
    auto start = [&]() {
        walk.next(a, tq, 0, s);
        if (s.r < 0)
            return;
        bend = (min(s.end(), s.t1 * PP_TILE) + 15) >> 4;
        blk = s.t0 * (PP_TILE / 16) + warp;
        int pg[S];
#pragma unroll
        for (int x = 0; x < S; ++x)
            pg[x] = page_of(blk + x * OW);
        page = page_of(blk + S * OW);
#pragma unroll
        for (int x = 0; x < S; ++x)
            fetch(blk + x * OW, pg[x], x);
    };
    start();
    while (s.r >= 0) {
        const int nrows = s.ntok << a.g_shift;
        int slot = 0;
        // ---- Q: row 8 y + i, channels 16 j + 2 c, + 1 and + 8, + 9
        uint32_t qf[NR][2 * KS];
        float m[NR][2], l[NR][2], o[NR][KS][4], off[NR][2], top[NR][2];
        int pos[NR][2];
#pragma unroll
        for (int y = 0; y < NR; ++y) {
            const int row = 8 * y + i;
            const uint16_t *src = f.q + (int64_t)(s.row0 + (row >> a.g_shift)) * f.q_stride +
                                  ((s.h << a.g_shift) + (row & (G - 1))) * D + 2 * c;
#pragma unroll
            for (int j = 0; j < 2 * KS; ++j)
                qf[y][j] = row < nrows ? __ldg(reinterpret_cast<const uint32_t *>(src + 8 * j)) : 0u;
#pragma unroll
            for (int e = 0; e < 2; ++e) {  // this lane's columns of S^T: rows 8 y + 2 c, + 1
                m[y][e] = top[y][e] = DDT_NEG_INF;
                off[y][e] = l[y][e] = 0.f;
                pos[y][e] = s.last_key((8 * y + 2 * c + e) >> a.g_shift);
            }
#pragma unroll
            for (int j = 0; j < KS; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    o[y][j][e] = 0.f;
        }
        const float sc = a.scale_log2;
        for (; blk < bend; blk += OW) {
            cp_async_wait_group<S - 1>();
            __syncwarp();
            const uint32_t kb = raws + slot * OWN_BLOCK<D>, vb = kb + 16 * OWN_ROW<D>;
            // ---- S^T: ldmatrix's four 8 x 8 parts: keys 0-7 and 8-15 of channels 16 j .. + 7, then + 8 ..
            float st[NR][4];
#pragma unroll
            for (int y = 0; y < NR; ++y)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    st[y][e] = 0.f;
#pragma unroll
            for (int j = 0; j < KS; ++j) {
                uint32_t k4[4];
                ldmatrix4(k4, kb + own_place<D>(lane & 15, 2 * j + (lane >> 4)));
#pragma unroll
                for (int y = 0; y < NR; ++y)
                    mma_b16(st[y], k4, qf[y][2 * j], qf[y][2 * j + 1]);
            }
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
                        mx *= sc;
                        if (mx > m[y][e]) {
                            const float alpha = ex2(m[y][e] - mx);
                            m[y][e] = mx;
                            off[y][e] = -mx;
                            top[y][e] = (mx + TAU) / sc;
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
                    p[e] = ex2(fmaf(st[y][e], sc, off[y][e & 1]));
                    l[y][e & 1] += p[e];
                }
                pb[y][0] = transpose8(pack_bf16x2(p[0], p[1]));
                pb[y][1] = transpose8(pack_bf16x2(p[2], p[3]));
            }
            // ---- O^T: V^T's parts: channels 16 j .. + 7 and + 8 .. of keys 0-7, then of keys 8-15
#pragma unroll
            for (int j = 0; j < KS; ++j) {
                uint32_t v4[4];
                ldmatrix4_t(v4, vb + own_place<D>((lane & 7) + ((lane >> 4) << 3), 2 * j + ((lane >> 3) & 1)));
#pragma unroll
                for (int y = 0; y < NR; ++y)
                    mma_b16(o[y][j], v4, pb[y][0], pb[y][1]);
            }
            __syncwarp();
            fetch(blk + S * OW, page, slot);
            page = page_of(blk + (S + 1) * OW);
            slot = slot + 1 == S ? 0 : slot + 1;
        }
        const Seg was = s;
        if (tid == 0)
            note_ctas(a, was, blockIdx.x);
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
                float *dst = so + (warp * ROWS + row) * D + i;
#pragma unroll
                for (int j = 0; j < KS; ++j) {
                    dst[16 * j] = o[y][j][e];
                    dst[16 * j + 8] = o[y][j][e + 2];
                }
            }
        __syncthreads();
        for (int e = tid; e < nrows * (D / 4); e += OT) {
            const int row = e / (D / 4), c4 = e % (D / 4);
            float M = DDT_NEG_INF, L = 0.f;
#pragma unroll
            for (int w = 0; w < OW; ++w)
                M = fmaxf(M, sml[w * ROWS + row].x);
            float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < OW; ++w) {
                const float2 ml = sml[w * ROWS + row];
                const float k = ml.x == DDT_NEG_INF ? 0.f : ex2(ml.x - M);
                const float4 v = reinterpret_cast<const float4 *>(so + (w * ROWS + row) * D)[c4];
                L += ml.y * k;
                r.x += v.x * k;
                r.y += v.y * k;
                r.z += v.z * k;
                r.w += v.w * k;
            }
            if (was.whole && !was.part) {
                const float inv = L > 0.f || L != L ? 1.f / L : 0.f;
                uint32_t *dst = reinterpret_cast<uint32_t *>(
                    a.out + ((int64_t)(was.row0 + (row >> a.g_shift)) * a.Hq + (was.h << a.g_shift) + (row & (G - 1))) * D) + 2 * c4;
                *reinterpret_cast<uint2 *>(dst) =
                    make_uint2(pack_bf16x2(r.x * inv, r.y * inv), pack_bf16x2(r.z * inv, r.w * inv));
            } else if (was.whole) {
                const int64_t at = (((int64_t)was.h * a.T + was.row0) << a.g_shift) + row;
                a.store_o[1][(int64_t)c4 * a.T * a.Hq + at] = r;
                if (c4 == 0)
                    a.store_ml[1][at] = make_float2(M, L);
            } else {
                const int64_t sl = (int64_t)was.slot * ROWS;
                reinterpret_cast<float4 *>(a.own_o + sl * D)[c4 * ROWS + row] = r;
                if (c4 == 0)
                    a.own_ml[sl + row] = make_float2(M, L);
            }
        }
        __syncthreads();
    }
    cp_async_wait_all();
    own_done();  // (the prefixes' kernel is before this one; the merge waits for this one only)
}

template <int D, int NR>
cudaError_t launch_own(const OwnArgs &f, int dev, int num_sms, cudaStream_t s)
{
    constexpr int ROWS = 8 * NR, BYTES = OW * (ROWS * (D * 4 + 8) + OS<NR> * (int)OWN_BLOCK<D>);
    static_assert(BYTES <= 115200, "shared memory of one CTA of two");
    static DeviceFlags ready;
    if (!ready.test(dev)) {
        const cudaError_t e = cudaFuncSetAttribute(own_few_kernel<D, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize, BYTES);
        if (e != cudaSuccess)
            return e;
        ready.set(dev);
    }
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3((num_sms < PR_MAX_CTAS ? num_sms : PR_MAX_CTAS) * OWN_FEW_CTAS);
    lc.blockDim = dim3(OT);
    lc.dynamicSmemBytes = BYTES;
    lc.stream = s;
    cudaLaunchAttribute at[1];  // (beside the prefixes' kernel, which reads and writes elsewhere)
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = at;
    lc.numAttrs = 1;
    return cudaLaunchKernelEx(&lc, own_few_kernel<D, NR>, f);
}

}  // namespace

cudaError_t launch_own_few(ddt_ctx *c, const PtArgs &a, const uint16_t *q, int64_t q_stride, const uint16_t *k_cache,
                           int rows, cudaStream_t s)
{
    OwnArgs f;
    f.a = a;
    f.q = q;
    f.q_stride = q_stride;
    f.k_cache = k_cache;
    if (c->cfg.d == 128)
        return rows <= 8 ? launch_own<128, 1>(f, c->device, c->num_sms, s)
                         : launch_own<128, 2>(f, c->device, c->num_sms, s);
    return rows <= 8 ? launch_own<64, 1>(f, c->device, c->num_sms, s)
                     : launch_own<64, 2>(f, c->device, c->num_sms, s);
}

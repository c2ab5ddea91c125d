// prompt.cu -- causal attention of packed sequences over the paged cache.
//
// One warp per query row (token, head): lane l holds channels l D/32 .. of the
// query and of the running output; keys are taken one at a time with the
// running maximum and sum of the softmax.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "ddt_device.cuh"
#include "ddt_internal.h"
#include "packed_seq.h"

namespace {

struct PrArgs {
    const uint16_t *q;
    int64_t q_stride;
    const int32_t *q_start, *ctx_lens, *block_table;
    const uint16_t *k_cache, *v_cache;
    ddt_kv4 kv4;
    uint16_t *out;
    int32_t *status;
    int R, T, Hq, Hkv, G, page_shift, max_pages, cap;
    int64_t num_pages;
    float scale_log2, out_scale;
};

DDT_DEVINL float value4(uint32_t code, uint32_t e4m3)
{
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)e4m3));
    float f;
    asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n cvt.f32.f16 %0, l;\n}\n" : "=f"(f) : "r"(h2));
    const uint32_t m = code & 7u;
    const float v = m < 2 ? 0.5f * (float)m : __uint_as_float(((126u + (m >> 1)) << 23) | ((m & 1u) << 22));
    return f * ((code & 8u) ? -v : v);
}

template <int D, bool KV4>
__global__ void __launch_bounds__(256) prompt_rows_kernel(const PrArgs p)
{
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (blockIdx.x == 0)
        for (int r = threadIdx.x; r < p.R; r += 256)
            if (!packed_ok(p.q_start[r], p.q_start[r + 1], p.T, p.ctx_lens[r], p.cap))
                set_status(p.status, DDT_DEV_BAD_LENGTH);
    if (w >= (int64_t)p.T * p.Hq)
        return;
    const int t = (int)(w / p.Hq), h = (int)(w % p.Hq), g = h / p.G;
    int req = -1;
    for (int r0 = 0; r0 < p.R && req < 0; r0 += 32) {
        const int r = r0 + lane;
        const bool in = r < p.R && p.q_start[r] <= t && t < p.q_start[r + 1] &&
                        packed_ok(p.q_start[r], p.q_start[r + 1], p.T, p.ctx_lens[r], p.cap);
        const unsigned b = __ballot_sync(0xFFFFFFFFu, in);
        if (b)
            req = r0 + __ffs(b) - 1;
    }
    if (req < 0)
        return;
    const int n = p.ctx_lens[req] + (t - p.q_start[req]) + 1;
    float q[E], o[E], m = DDT_NEG_INF, l = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        q[i] = bf16_to_f32(p.q[(int64_t)t * p.q_stride + h * D + lane * E + i]) * p.scale_log2;
        o[i] = 0.f;
    }
    for (int j = 0; j < n; ++j) {
        const int pg = p.block_table[(int64_t)req * p.max_pages + (j >> p.page_shift)];
        const int in_page = j & ((1 << p.page_shift) - 1);
        float k[E], v[E];
        if (pg < 0 || pg >= p.num_pages) {
            set_status(p.status, DDT_DEV_BAD_PAGE);
#pragma unroll
            for (int i = 0; i < E; ++i)
                k[i] = v[i] = 0.f;
        } else if (KV4) {
            const int64_t row = ((((int64_t)pg * p.Hkv) + g) << p.page_shift) + in_page;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const int c = lane * E + i, sh = ((c & 7) >> 1) * 4 + (c & 1) * 16;
                const int64_t at = row * (D / 8) + c / 8;
                k[i] = value4((reinterpret_cast<const uint32_t *>(p.kv4.k_codes)[at] >> sh) & 15u,
                              p.kv4.k_scales[row * (D / 16) + c / 16]);
                v[i] = value4((reinterpret_cast<const uint32_t *>(p.kv4.v_codes)[at] >> sh) & 15u,
                              p.kv4.v_scales[row * (D / 16) + c / 16]);
            }
        } else {
            const int64_t row = ((((int64_t)pg << p.page_shift) + in_page) * p.Hkv + g) * D + lane * E;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                k[i] = bf16_to_f32(p.k_cache[row + i]);
                v[i] = bf16_to_f32(p.v_cache[row + i]);
            }
        }
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i)
            s = fmaf(q[i], k[i], s);
#pragma unroll
        for (int x = 16; x > 0; x >>= 1)
            s += __shfl_xor_sync(0xFFFFFFFFu, s, x);
        const float mn = fmaxf(m, s), f = exp2f(m - mn), e = exp2f(s - mn);
        l = l * f + e;
#pragma unroll
        for (int i = 0; i < E; ++i)
            o[i] = fmaf(o[i], f, e * v[i]);
        m = mn;
    }
#pragma unroll
    for (int i = 0; i < E; i += 2)
        reinterpret_cast<uint32_t *>(p.out)[(((int64_t)t * p.Hq + h) * D + lane * E + i) / 2] =
            pack_bf16x2(o[i] / l * p.out_scale, o[i + 1] / l * p.out_scale);
}

}  // namespace

cudaError_t launch_prompt_tc(ddt_ctx *c, const uint16_t *q, int64_t q_stride, const int32_t *q_start,
                             const int32_t *ctx_lens, int R, int T, const uint16_t *k_cache,
                             const uint16_t *v_cache, const int32_t *block_table, uint16_t *out, cudaStream_t s);

cudaError_t launch_prompt_attention(ddt_ctx *c, const uint16_t *q, int64_t q_stride,
                                    const int32_t *q_start, const int32_t *ctx_lens, int R, int T,
                                    const uint16_t *k_cache, const uint16_t *v_cache,
                                    const ddt_kv4 *kv4, const int32_t *block_table, uint16_t *out,
                                    cudaStream_t s)
{
    if (!kv4)
        return launch_prompt_tc(c, q, q_stride, q_start, ctx_lens, R, T, k_cache, v_cache, block_table, out, s);
    const ddt_config &cfg = c->cfg;
    PrArgs p = {};
    p.q = q;
    p.q_stride = q_stride;
    p.q_start = q_start;
    p.ctx_lens = ctx_lens;
    p.block_table = block_table;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.out = out;
    p.status = c->status;
    p.R = R;
    p.T = T;
    p.Hq = cfg.Hq;
    p.Hkv = cfg.Hkv;
    p.G = cfg.Hq / cfg.Hkv;
    while ((1 << p.page_shift) < cfg.page_size)
        ++p.page_shift;
    p.max_pages = cfg.max_pages_per_req;
    p.cap = cfg.max_pages_per_req * cfg.page_size;
    p.num_pages = cfg.num_pages;
    p.scale_log2 = 1.4426950408889634f / sqrtf((float)cfg.d);
    p.out_scale = 1.f;
    if (kv4) {
        p.kv4 = *kv4;
        p.scale_log2 *= kv4->k_scale;
        p.out_scale = kv4->v_scale;
    }
    const int64_t warps = (int64_t)T * cfg.Hq;
    const int64_t grid = (warps + 7) / 8;
    if (grid > 0x7fffffff)
        return cudaErrorInvalidValue;
    if (kv4) {
        if (cfg.d == 128)
            prompt_rows_kernel<128, true><<<(int)grid, 256, 0, s>>>(p);
        else
            prompt_rows_kernel<64, true><<<(int)grid, 256, 0, s>>>(p);
    } else {
        if (cfg.d == 128)
            prompt_rows_kernel<128, false><<<(int)grid, 256, 0, s>>>(p);
        else
            prompt_rows_kernel<64, false><<<(int)grid, 256, 0, s>>>(p);
    }
    return cudaGetLastError();
}

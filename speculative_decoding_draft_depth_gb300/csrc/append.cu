// append.cu -- new tokens' keys and values into the paged cache, queries and
// keys turned by their positions on the way; the cache is bf16, or held in 4
// bits (16-channel blocks of e2m1 codes under one e4m3 scale).
//
// A token's row of Hq + 2 Hkv heads is cut into pieces of 16 channels, one per
// thread: for paired halves (j, j + rd/2) the two 8-channel vectors that turn
// into each other, otherwise 16 neighbouring channels. So every thread reads
// and writes 2 x 16 bytes, holds both members of its pairs, and q_out may be q.
//
// Bound by memory: 24083 ragged tokens of 32/8 heads of 128 (593 MB with the angles)
// take 98.5 us, 6.0 TB/s. Five CTAs of 256 threads an SM (48 registers) hide the
// loads; four take 106 us, six 101, and a thread that keeps its piece over four
// tokens, for more loads in flight, 115. Into 4 bits (16/16 heads of 64, 324 MB): 65
// us, 5.0 TB/s, where the codes' arithmetic (three multiply-adds a channel for the
// exact quotient, a conversion for two) and short stores cost the rest.
#include <cuda_runtime.h>
#include <stdint.h>

#include "ddt_device.cuh"
#include "ddt_internal.h"
#include "packed_seq.h"

namespace {

constexpr int AP_THREADS = 256;
constexpr int AP_TOKENS = 4;  // tokens of one CTA, at most

struct ApArgs {
    ddt_append_args a;
    uint16_t *k_cache, *v_cache;
    ddt_kv4 kv4;
    uint16_t *k_held, *v_held;
    int32_t *status;
    int Hq, Hkv, page_shift, max_pages, cap;  // Hq: 0 when there are no queries
    int64_t num_pages;
    float k_inv6, v_inv6;  // 1 / (6 g)
    int tokens;            // of a CTA
};

// x1' = x1 cos - x2 sin, x2' = x2 cos + x1 sin, every product and sum rounded
// (no fused multiply-add: the result is the one the header's formula gives)
DDT_DEVINL void turn(float &x1, float &x2, float c, float s)
{
    const float a = __fsub_rn(__fmul_rn(x1, c), __fmul_rn(x2, s));
    const float b = __fadd_rn(__fmul_rn(x2, c), __fmul_rn(x1, s));
    x1 = a;
    x2 = b;
}

DDT_DEVINL float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
DDT_DEVINL float min_nan(float a, float b)
{
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// fp32 -> e4m3 bits (to nearest even; NaN -> 0x7f) and back
DDT_DEVINL uint32_t to_e4m3(float x)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
    return r & 0xFFu;
}
DDT_DEVINL float from_e4m3(uint32_t b)
{
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)b));
    float f;
    asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n cvt.f32.f16 %0, l;\n}\n" : "=f"(f) : "r"(h2));
    return f;
}

// two fp32 to a byte of e2m1 codes, to nearest even, at most 6 in magnitude
DDT_DEVINL uint32_t to_e2m1x2(float lo, float hi)
{
    uint32_t r;
    asm("{\n .reg .b8 b;\n cvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n cvt.u32.u8 %0, b;\n}\n" : "=r"(r) : "f"(lo), "f"(hi));
    return r;
}
// and back: a byte's two values
DDT_DEVINL void from_e2m1x2(uint32_t b, float &lo, float &hi)
{
    uint32_t h2;
    asm("{\n .reg .b8 b;\n cvt.u8.u32 b, %1;\n cvt.rn.f16x2.e2m1x2 %0, b;\n}\n" : "=r"(h2) : "r"(b));
    asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, h;\n}\n"
        : "=f"(lo), "=f"(hi)
        : "r"(h2));
}

// A block's scale and what its codes need. The scale is the e4m3 number nearest to
// RN(amax / (6 g)): the product amax RN(1 / (6 g)) alone can be a midpoint of e4m3 where
// the quotient is one step below it, so it gets one residual as the codes' do. With q = RN(x / s) the nearest code of q
// (ties to even) is the nearest code of x / s for g = 1: a midpoint t and s have at
// most three and four significant bits, so t s is an fp32 number, and an x next to it
// is at least as far from it, in units of x / s, as half a step of q at t. q comes from
// the correctly rounded reciprocal y by one residual, q0 + (x - q0 s) y with
// q0 = RN(x y), which is RN(x / s) (Markstein).
struct Scale {
    uint32_t bits;  // e4m3
    float s, y;     // scale * g; 1 / s
    bool plain;     // neither zero, NaN nor saturated
};
DDT_DEVINL Scale make_scale(float amax, float inv6, float g)
{
    Scale r;
    const float raw0 = __fmul_rn(amax, inv6);
    // (beyond e4m3 the product will do: infinity would have no residual)
    const float raw = raw0 <= 512.f ? __fmaf_rn(__fmaf_rn(-raw0, __fmul_rn(6.f, g), amax), inv6, raw0) : raw0;
    r.bits = to_e4m3(min_nan(raw, 448.f));
    r.s = __fmul_rn(from_e4m3(r.bits), g);
    r.y = __frcp_rn(r.s);
    r.plain = r.s > 0.f && raw <= 448.f;
    return r;
}

DDT_DEVINL void unpack8(const uint4 &w, float *f)
{
    f[0] = bf16lo(w.x), f[1] = bf16hi(w.x), f[2] = bf16lo(w.y), f[3] = bf16hi(w.y);
    f[4] = bf16lo(w.z), f[5] = bf16hi(w.z), f[6] = bf16lo(w.w), f[7] = bf16hi(w.w);
}
DDT_DEVINL uint4 pack8(const float *f)
{
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}
// the codes of 8 neighbouring channels: bytes of channels (0, 2), (4, 6), (1, 3), (5, 7)
DDT_DEVINL uint32_t codes8(const float *f, const Scale &c)
{
    float q[8];
    if (c.plain) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float q0 = __fmul_rn(f[i], c.y);
            q[i] = __fmaf_rn(__fmaf_rn(-q0, c.s, f[i]), c.y, q0);
        }
    } else {
        // zero or NaN scale: zeros with their signs; saturated: the quotient may be
        // beyond fp32
#pragma unroll
        for (int i = 0; i < 8; ++i)
            q[i] = c.s > 0.f ? __fdiv_rn(f[i], c.s) : copysignf(0.f, f[i]);
    }
    return to_e2m1x2(q[0], q[2]) | to_e2m1x2(q[4], q[6]) << 8 | to_e2m1x2(q[1], q[3]) << 16 | to_e2m1x2(q[5], q[7]) << 24;
}
DDT_DEVINL void held8(uint32_t w, float s, float *f)
{
    from_e2m1x2(w & 255u, f[0], f[2]);
    from_e2m1x2((w >> 8) & 255u, f[4], f[6]);
    from_e2m1x2((w >> 16) & 255u, f[1], f[3]);
    from_e2m1x2(w >> 24, f[5], f[7]);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        f[i] = __fmul_rn(f[i], s);
}

template <int D, bool KV4>
__global__ void __launch_bounds__(AP_THREADS, 5) append_kernel(const ApArgs p)
{
    constexpr int PIECES = D / 16;  // of a head
    __shared__ int s_r[AP_TOKENS], s_pos[AP_TOKENS];  // the token's request and position, -1: no request
    __shared__ int64_t s_row[AP_TOKENS];  // the token's row of the pool, -1: no slot
    const ddt_append_args &a = p.a;
    const int tid = threadIdx.x, t0 = blockIdx.x * p.tokens;
    if (tid < p.tokens)
        s_r[tid] = -1;
    __syncthreads();
    // every thread looks at some of the requests: one round of independent
    // loads instead of a chain of dependent ones
    for (int r = tid; r < a.R; r += AP_THREADS) {
        const int q0 = __ldg(&a.q_start[r]), q1 = __ldg(&a.q_start[r + 1]);
        const int ctx = __ldg(&a.ctx_lens[r]);
        const bool ok = packed_ok(q0, q1, a.T, ctx, p.cap);
        if (blockIdx.x == 0) {
            if (!ok)
                set_status(p.status, DDT_DEV_BAD_LENGTH);
            if (a.new_lens)
                a.new_lens[r] = ok ? ctx + (q1 - q0) : ctx;
        }
        // Of two requests that name the row (q_start fell between them) the later one has
        // it; the position follows from the owner, so that the two belong together.
        if (ok)
            for (int t = max(q0, t0); t < min(q1, t0 + p.tokens); ++t)
                atomicMax(&s_r[t - t0], r);
    }
    __syncthreads();
    if (tid < p.tokens) {
        const int r = s_r[tid];
        s_pos[tid] = r < 0 ? -1 : __ldg(&a.ctx_lens[r]) + (t0 + tid - __ldg(&a.q_start[r]));
    }
    if (tid < p.tokens && s_r[tid] >= 0) {
        const int pos = s_pos[tid], r = s_r[tid];
        const int pg = __ldg(&a.block_table[(int64_t)r * p.max_pages + (pos >> p.page_shift)]);
        const bool ok = pg >= 0 && pg < p.num_pages;
        if (!ok)
            set_status(p.status, DDT_DEV_BAD_PAGE);
        const int in_page = pos & ((1 << p.page_shift) - 1);
        // row of [num_pages, page_size] (bf16), of [num_pages, Hkv, page_size] at head 0 (4 bits)
        s_row[tid] = !ok ? -1 : ((((int64_t)pg * (KV4 ? p.Hkv : 1)) << p.page_shift) + in_page);
    }
    __syncthreads();

    const int per_token = (p.Hq + 2 * p.Hkv) * PIECES, half = a.rotary_dim / 2;
    const int n = min(p.tokens, a.T - t0) * per_token;
    // the last round is padded to whole warps: lanes exchange block maxima
    for (int e0 = 0; e0 < n; e0 += AP_THREADS) {
        const int e = min(e0 + tid, n - 1);
        static_assert(AP_TOKENS == 4, "the token by comparison");
        const int tk = (e >= per_token) + (e >= 2 * per_token) + (e >= 3 * per_token);
        const int h = (e - tk * per_token) / PIECES, piece = e % PIECES;  // (whole heads: pieces stay aligned)
        const bool live = e0 + tid < n && s_r[tk] >= 0;
        const bool is_q = h < p.Hq, is_k = !is_q && h < p.Hq + p.Hkv;
        const int hk = is_q ? h : (h - p.Hq) - (is_k ? 0 : p.Hkv);
        const bool turned = (is_q || is_k) && piece * 16 < a.rotary_dim;
        const bool halves = turned && !a.interleaved;
        const int o0 = halves ? piece * 8 : piece * 16, o1 = halves ? half + piece * 8 : piece * 16 + 8;
        float x[16];
        if (live) {
            const uint16_t *src = is_q ? a.q + (t0 + tk) * a.q_stride
                                       : is_k ? a.k + (t0 + tk) * a.k_stride : a.v + (t0 + tk) * a.v_stride;
            src += hk * D;
            unpack8(__ldcs(reinterpret_cast<const uint4 *>(src + o0)), x);
            unpack8(__ldcs(reinterpret_cast<const uint4 *>(src + o1)), x + 8);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                x[i] = 0.f;
        }
        if (live && turned) {
            const float4 *row = reinterpret_cast<const float4 *>(a.cos_sin + (int64_t)s_pos[tk] * a.rotary_dim +
                                                                 piece * 8);
            const float4 c0 = __ldg(row), c1 = __ldg(row + 1);
            const float4 n0 = __ldg(row + half / 4), n1 = __ldg(row + half / 4 + 1);
            const float c[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
            const float s[8] = {n0.x, n0.y, n0.z, n0.w, n1.x, n1.y, n1.z, n1.w};
            if (halves) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    turn(x[i], x[8 + i], c[i], s[i]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    turn(x[2 * i], x[2 * i + 1], c[i], s[i]);
            }
        }
        if ((is_q || !KV4) && live) {
            uint16_t *dst = nullptr;
            if (is_q)
                dst = a.q_out + ((int64_t)(t0 + tk) * p.Hq + h) * D;
            else if (s_row[tk] >= 0)
                dst = (is_k ? p.k_cache : p.v_cache) + (s_row[tk] * p.Hkv + hk) * D;
            if (dst) {
                *reinterpret_cast<uint4 *>(dst + o0) = pack8(x);
                *reinterpret_cast<uint4 *>(dst + o1) = pack8(x + 8);
            }
        }
        if (KV4) {
            if (__all_sync(0xFFFFFFFFu, is_q))
                continue;
            float m0 = 0.f, m1 = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                m0 = max_nan(m0, fabsf(x[i]));
                m1 = max_nan(m1, fabsf(x[8 + i]));
            }
            // a block's other 8 channels: the neighbour's vector when halves pair up
            // (pieces 2i and 2i + 1 sit in lanes 2i and 2i + 1), else this thread's
            // second one
            const float u0 = __shfl_xor_sync(0xFFFFFFFFu, m0, 1), u1 = __shfl_xor_sync(0xFFFFFFFFu, m1, 1);
            const float b0 = max_nan(m0, halves ? u0 : m1), b1 = max_nan(m1, halves ? u1 : m0);
            if (live && !is_q) {
                const float g = is_k ? p.kv4.k_scale : p.kv4.v_scale, inv6 = is_k ? p.k_inv6 : p.v_inv6;
                const Scale s0 = make_scale(b0, inv6, g);
                const Scale s1 = halves ? make_scale(b1, inv6, g) : s0;
                const uint32_t w0 = codes8(x, s0), w1 = codes8(x + 8, s1);
                if (s_row[tk] >= 0) {
                    const int64_t row = s_row[tk] + ((int64_t)hk << p.page_shift);
                    uint8_t *cd = (is_k ? p.kv4.k_codes : p.kv4.v_codes) + row * (D / 2);
                    uint8_t *sc = (is_k ? p.kv4.k_scales : p.kv4.v_scales) + row * (D / 16);
                    if (!halves) {
                        *reinterpret_cast<uint2 *>(cd + o0 / 2) = make_uint2(w0, w1);
                        sc[piece] = (uint8_t)s0.bits;
                    } else {
                        *reinterpret_cast<uint32_t *>(cd + o0 / 2) = w0;
                        *reinterpret_cast<uint32_t *>(cd + o1 / 2) = w1;
                        if ((piece & 1) == 0) {
                            sc[o0 / 16] = (uint8_t)s0.bits;
                            sc[o1 / 16] = (uint8_t)s1.bits;
                        }
                    }
                }
                if (p.k_held) {
                    uint16_t *hd = (is_k ? p.k_held : p.v_held) + ((int64_t)(t0 + tk) * p.Hkv + hk) * D;
                    float y[8];
                    held8(w0, s0.s, y);
                    *reinterpret_cast<uint4 *>(hd + o0) = pack8(y);
                    held8(w1, s1.s, y);
                    *reinterpret_cast<uint4 *>(hd + o1) = pack8(y);
                }
            }
        }
    }
}

}  // namespace

cudaError_t launch_append(const ddt_ctx *c, const ddt_append_args &a, uint16_t *k_cache,
                          uint16_t *v_cache, const ddt_kv4 *kv4, uint16_t *k_held,
                          uint16_t *v_held, cudaStream_t s)
{
    const ddt_config &cfg = c->cfg;
    ApArgs p = {};
    p.a = a;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    if (kv4) {
        p.kv4 = *kv4;
        p.k_inv6 = 1.0f / (6.0f * kv4->k_scale);
        p.v_inv6 = 1.0f / (6.0f * kv4->v_scale);
    }
    p.k_held = k_held;
    p.v_held = v_held;
    p.status = c->status;
    p.Hq = a.q ? cfg.Hq : 0;
    p.Hkv = cfg.Hkv;
    while ((1 << p.page_shift) < cfg.page_size)
        ++p.page_shift;
    p.max_pages = cfg.max_pages_per_req;
    p.cap = cfg.max_pages_per_req * cfg.page_size;
    if (a.cos_sin && a.max_pos < p.cap)
        p.cap = a.max_pos;
    p.num_pages = cfg.num_pages;
    // (T = 0 still writes new_lens)
    // Tokens of a CTA: each CTA first finds its requests and pages, which takes longer
    // than one token's pieces; few tokens want all SMs all the same. Measured (32/8
    // heads of 128, bf16; 1, 2, 4 tokens a CTA): 256 tokens 3.6, 4.0, 5.9 us; 1024
    // 7.4, 6.5, 7.9; 4096 22.3, 18.3, 19.0; 8192 45.1, 38.4, 37.0.
    p.tokens = a.T >= 40 * c->num_sms ? AP_TOKENS : a.T >= 3 * c->num_sms ? 2 : 1;
    const int grid = a.T > 0 ? (a.T - 1) / p.tokens + 1 : 1;
    if (kv4) {
        if (cfg.d == 128)
            append_kernel<128, true><<<grid, AP_THREADS, 0, s>>>(p);
        else
            append_kernel<64, true><<<grid, AP_THREADS, 0, s>>>(p);
    } else {
        if (cfg.d == 128)
            append_kernel<128, false><<<grid, AP_THREADS, 0, s>>>(p);
        else
            append_kernel<64, false><<<grid, AP_THREADS, 0, s>>>(p);
    }
    return cudaGetLastError();
}

// sample_row.cuh -- one row of logits held by a thread-block cluster: the tokens that
// temperature, top-k, top-p and min-p keep, their weights, and the draw of one.
//
// With z_max the row's largest logit and T the temperature, token i's weight is
//   w_i = exp((z_i - z_max) / T).
// All three filters keep a front part of the order (z descending, index ascending):
// min-p the tokens with w_i >= min_p, top-k the first k of those, top-p the shortest
// front part of these whose weights reach p times their sum. So the kept set is one
// border (value, index): z above the value, or equal to it and an index up to the
// border's. The draw takes the kept tokens in index order: the first whose running sum
// exceeds u times the sum.
//
// The border and the draw are decisions: an error in a sum decides wrongly whenever a
// border lies within it, and a vocabulary has 10^5 of them. So weights are made to about
// 2^-40 of themselves, from pairs of fp32 numbers (one fma more for each rounding that
// is kept), and added up as 64-bit integers in units of 2^-44, whose sums do not depend
// on an order. What is below 2^-64 of the largest weight counts as zero.
//
// A row is read from HBM once (but see FAR below): the CTAs of its cluster hold it in shared
// memory (sub-chunks of 512 bytes: 16 bytes a lane), and every further look at it reads that. What
// the CTAs have to tell one another goes through distributed shared memory, one cluster
// barrier an exchange, and each CTA then comes to the same decision by itself.
#pragma once

#include <stdint.h>
#include <string.h>

#include "ddt_device.cuh"
#include "ddt_internal.h"

namespace {

constexpr int SR_THREADS = 256, SR_WARPS = SR_THREADS / 32;
constexpr int SR_SUB = 512;       // bytes of a sub-chunk
constexpr int SR_FAR = 512;       // threads of a CTA that reads a row from global memory (1984 rows of 151936 bf16,
                                  // greedy: 222 us; 1024, one CTA an SM: 270; under top-p 256, three an SM: 767 for 543)
constexpr int SR_GROUP = 4;       // sub-chunks that a warp takes at once from there (64 chains of 15 guesses, mixed
                                  // settings: 427 us; two 442, eight 500)
constexpr int SR_OWN = 8;         // parts of a thread's logits of which it knows the largest there
constexpr int SR_MAX_CL = 16;     // CTAs of a cluster
constexpr int SR_CAP = 512;       // candidates that are sorted in one place
constexpr int SR_PROBE = 256;     // how many the first collection asks for, and the largest k that it serves
constexpr int SR_BINS = 512;      // (two a thread)
constexpr int SR_FLAT = 8;        // rows that weigh more than so many of their largest tokens are flat
constexpr int SR_SMALL = 256;     // candidates of which each has a thread
constexpr int SR_ONE = 44;        // a weight of 1 is 2^44
constexpr float SR_MAX_FLOAT = 3.402823466e38f;
constexpr float SR_TINY = 8.077935669e-28f;  // 2^-90: differences of logits stay far above what 1 / x can take

// ---------------------------------------------------------------- cluster
DDT_DEVINL uint32_t cl_rank()
{
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
DDT_DEVINL uint32_t cl_size()
{
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
DDT_DEVINL void cl_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
DDT_DEVINL void cl_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
DDT_DEVINL void cl_sync()
{
    cl_arrive();
    cl_wait();
}
DDT_DEVINL uint32_t cl_map(const void *p, uint32_t rank)
{
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    return r;
}
DDT_DEVINL void cl_st64(uint32_t at, uint64_t v)
{
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(v) : "memory");
}
DDT_DEVINL uint32_t cl_ld32(uint32_t at)
{
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at));  // (stays between the barriers around it)
    return v;
}
DDT_DEVINL uint64_t cl_ld64(uint32_t at)
{
    uint64_t v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(at));
    return v;
}
DDT_DEVINL void cp16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
DDT_DEVINL void cp_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

DDT_DEVINL uint64_t f2mul(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
DDT_DEVINL uint64_t f2both(float x) { return f2pack(x, x); }

// order-preserving map of floats to unsigned integers
DDT_DEVINL uint32_t order_key(float z)
{
    const uint32_t b = __float_as_uint(z == 0.f ? 0.f : z);  // (-0 and 0 are equal)
    return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
DDT_DEVINL float key_value(uint32_t k)
{
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

// ---------------------------------------------------------------- weights
struct Scale {
    float zmax, ch, cl;  // log2(e) / T = ch + cl
    float zfloor;        // smaller values have no weight (finite)
};

// (fp32 throughout: the fp64 units take 16 cycles a warp's instruction)
DDT_DEVINL Scale make_scale(float zmax, float T)
{
    Scale s;
    s.zmax = zmax;
    const float LH = 1.44269502162933349609375f, LL = 1.92596299112661746887e-8f;  // log2(e)
    s.ch = LH / T;
    s.cl = (fmaf(-s.ch, T, LH) + LL) / T;
    // 2^-64 is 44.36 T below; rounded up, so that no exponent is below -64. A difference of
    // two values stays finite.
    s.zfloor = fmaxf(__fsub_ru(zmax, 44.3614195f * T), fmaxf(-SR_MAX_FLOAT, zmax - SR_MAX_FLOAT));
    return s;
}

// 2^(j / 32) as a pair of floats, j = 0 .. 31
__device__ const float2 SR_TABLE[32] = {
    {1.f, 0.f}, {1.0218972f, -4.81155986e-08f}, {1.04427373f, 4.83347016e-08f},
    {1.06714046f, -5.93375198e-08f}, {1.09050775f, -1.30775399e-08f}, {1.1143868f, -5.43554002e-08f},
    {1.13878858f, 5.38622231e-08f}, {1.1637249f, -4.05144149e-08f}, {1.18920708f, 3.79763527e-08f},
    {1.21524739f, -3.26739489e-08f}, {1.24185777f, 4.4968381e-08f}, {1.26905096f, 1.41933332e-09f},
    {1.29683959f, -4.01899953e-08f}, {1.32523668f, -3.49637332e-08f}, {1.35425556f, -1.01233493e-08f},
    {1.38390994f, -5.87557736e-08f}, {1.41421354f, 2.4203235e-08f}, {1.44518077f, 3.32419994e-08f},
    {1.47682619f, -4.50089885e-08f}, {1.50916445f, -2.49593732e-08f}, {1.54221082f, 8.07090483e-09f},
    {1.5759809f, -5.66102543e-08f}, {1.61049032f, 9.83621717e-09f}, {1.64575553f, -5.12497209e-08f},
    {1.68179286f, -2.47553267e-08f}, {1.71861935f, -4.8496176e-08f}, {1.75625217f, -9.23577037e-09f},
    {1.79470909f, -1.14150449e-08f}, {1.8340081f, -1.1239278e-08f}, {1.87416768f, -4.66300563e-08f},
    {1.91520655f, 9.84532811e-09f}, {1.95714414f, -1.70218044e-08f}};

// Sums of weights. A weight of up to 1 is cut at 2^-18: the front parts add up without an
// error (up to 16 of them), what is behind it in fp32 (2^-42 of 1 at most, each time).
struct Sum2 {
    uint64_t hi, lo;  // two lanes each
};
constexpr float SR_CUT = 48.0f;  // 1.5 * 2^5: fp32 numbers next to it are 2^-18 apart

// weights of two logits; k0, k1: whether they count. EXACT: the error of z - z_max for any
// floats (else the shorter form, which serves z of few bits, as bf16 numbers have)
template <bool EXACT>
DDT_DEVINL void add_weights(const Scale &sc, const float2 *tab, float x0, float x1, bool k0, bool k1, Sum2 &sum)
{
    const uint64_t m1 = f2both(-1.f);
    const uint64_t z = f2pack(k0 ? x0 : sc.zmax, k1 ? x1 : sc.zmax), nz = f2both(-sc.zmax);
    // d + dl = z - zmax
    const uint64_t d = f2add(z, nz);
    uint64_t dl;
    if (EXACT) {
        const uint64_t bb = f2fma(z, m1, d);                     // the part of -zmax that d took
        dl = f2add(f2fma(f2fma(bb, m1, d), m1, z), f2fma(bb, m1, nz));
    } else {
        dl = f2fma(f2add(d, f2both(sc.zmax)), m1, z);
    }
    // y + yl = (d + dl) (ch + cl), the exponent
    const uint64_t nch = f2both(-sc.ch);
    const uint64_t y = f2mul(d, f2both(sc.ch));
    uint64_t nyl = f2fma(d, nch, y);  // -yl
    nyl = f2fma(d, f2both(-sc.cl), nyl);
    nyl = f2fma(dl, nch, nyl);
    // y = n / 32 + r; s + re = r + yl, |s| <= 2^-6
    const float C5 = 393216.0f;  // 1.5 * 2^18: fp32 numbers next to it are 2^-5 apart
    const uint64_t t = f2add(y, f2both(C5));
    const uint64_t r = f2fma(f2add(t, f2both(-C5)), m1, y);
    const uint64_t s = f2fma(nyl, m1, r);
    const uint64_t nre = f2add(nyl, f2fma(r, m1, s));
    // 2^(s + re) - 1 = h + he, h = s ln 2 in fp32 (ln 2 as a pair), the rest of the series
    const float LH = 0.693147182464599609375f, LL = -1.90465429995776804525e-9f;
    const uint64_t h = f2mul(s, f2both(LH));
    uint64_t nhe = f2fma(s, f2both(-LH), h);
    nhe = f2fma(s, f2both(-LL), nhe);
    nhe = f2fma(nre, f2both(LH), nhe);
    uint64_t g = f2fma(s, f2both(-9.6181291076e-3f), f2both(-5.5504108665e-2f));
    g = f2fma(s, g, f2both(-0.24022650696f));
    nhe = f2fma(f2mul(s, s), g, nhe);
    float t0, t1;
    f2unpack(t, t0, t1);
    const int i0 = __float_as_int(t0), i1 = __float_as_int(t1);
    const float2 a = tab[i0 & 31], b = tab[i1 & 31];
    const uint64_t th = f2pack(a.x, b.x), tl = f2pack(a.y, b.y);
    // (th + tl) (1 + h + he) = w + wl
    const uint64_t w = f2fma(th, h, th);
    uint64_t wl = f2fma(th, h, f2fma(w, m1, th));  // th + th h - w
    wl = f2fma(th, f2mul(nhe, m1), wl);
    wl = f2add(f2fma(tl, h, wl), tl);
    // times 2^n
    const float e0 = __int_as_float(((i0 << 18) & 0xFF800000) + 0x3F800000);
    const float e1 = __int_as_float(((i1 << 18) & 0xFF800000) + 0x3F800000);
    const uint64_t e = f2pack(k0 ? e0 : 0.f, k1 ? e1 : 0.f);
    const uint64_t ws = f2mul(w, e);
    const uint64_t front = f2add(f2add(ws, f2both(SR_CUT)), f2both(-SR_CUT));
    sum.hi = f2add(sum.hi, front);
    sum.lo = f2add(sum.lo, f2fma(wl, e, f2fma(front, m1, ws)));
}

DDT_DEVINL uint64_t to_fixed(float hi, float lo)
{
    const long long v = __float2ll_rn(hi * 17592186044416.0f) + __float2ll_rn(lo * 17592186044416.0f);  // 2^44
    return v > 0 ? (uint64_t)v : 0;
}
DDT_DEVINL uint64_t to_fixed(const Sum2 &s)
{
    float a, b, c, d;
    f2unpack(s.hi, a, b);
    f2unpack(s.lo, c, d);
    return to_fixed(a + b, c + d);
}

// two weights in fixed point
template <bool EXACT>
DDT_DEVINL void fixed_pair(const Scale &sc, const float2 *tab, float x0, float x1, bool k0, bool k1, uint64_t &w0,
                           uint64_t &w1)
{
    Sum2 s = {0, 0};
    add_weights<EXACT>(sc, tab, x0, x1, k0, k1, s);
    float h0, h1, l0, l1;
    f2unpack(s.hi, h0, h1);
    f2unpack(s.lo, l0, l1);
    w0 = to_fixed(h0, l0);
    w1 = to_fixed(h1, l1);
}

// one weight (z counts)
template <bool EXACT>
DDT_DEVINL uint64_t weight_of(const Scale &sc, const float2 *tab, float z)
{
    Sum2 s = {0, 0};
    add_weights<EXACT>(sc, tab, z, z, z >= sc.zfloor, false, s);
    return to_fixed(s);
}

// The weights of two logits by the hardware's 2^x, the exponent's rounding carried: off by at
// most 2^-22 of themselves (ex2), and 2^-24 each for the product's rounding, what is left of
// the exponent's and (bf16) z - z_max where it has more than 24 bits.
template <bool EXACT>
DDT_DEVINL uint64_t quick_weights(const Scale &sc, float x0, float x1, bool k0, bool k1)
{
    const uint64_t z = f2pack(k0 ? x0 : sc.zmax, k1 ? x1 : sc.zmax), nz = f2both(-sc.zmax);
    const uint64_t d = f2add(z, nz);
    const uint64_t y = f2mul(d, f2both(sc.ch));
    uint64_t nyl = f2fma(d, f2both(-sc.ch), y);  // -(what y lacks)
    nyl = f2fma(d, f2both(-sc.cl), nyl);
    if (EXACT) {
        const uint64_t m1 = f2both(-1.f), bb = f2fma(z, m1, d);
        nyl = f2fma(f2add(f2fma(f2fma(bb, m1, d), m1, z), f2fma(bb, m1, nz)), f2both(-sc.ch), nyl);
    }
    float a, b, la, lb;
    f2unpack(y, a, b);
    f2unpack(nyl, la, lb);
    const float LN2 = 0.693147182464599609375f;
    a = ex2(a);
    b = ex2(b);
    return f2pack(k0 ? fmaf(-a * LN2, la, a) : 0.f, k1 ? fmaf(-b * LN2, lb, b) : 0.f);
}
// What a sum of such weights may be off by: 2^-22 + 3 * 2^-24 of itself for the weights, and
// 4 * 2^-24 for sums of up to eight in fp32 (then they are integers): below 2^-20.
DDT_DEVINL uint64_t quick_slack(uint64_t mass) { return mass >> 20; }

// x m for 0 < x < 1, rounded down or up
DDT_DEVINL uint64_t fraction_of(float x, uint64_t m, bool up)
{
    const uint32_t b = __float_as_uint(x);
    const int sh = 126 - (int)(b >> 23);  // x = mantissa 2^-24 2^-sh (a subnormal x: 0)
    if (sh > 125)
        return up && x > 0.f ? 1 : 0;
    const uint64_t a = (uint64_t)((b & 0x7FFFFFu) | 0x800000u) << 40;
    const uint64_t hi = __umul64hi(a, m), lo = a * m;
    if (sh >= 64)
        return up ? 1 : 0;
    const bool rest = lo != 0 || (hi & ((1ull << sh) - 1)) != 0;
    return (hi >> sh) + (up && rest ? 1 : 0);
}

// floor(u mass), within the running sums: the draw's token is the first whose sum exceeds it
DDT_DEVINL uint64_t draw_target(float u, uint64_t mass)
{
    return u < 1.f ? min(u > 0.f ? fraction_of(u, mass, false) : 0, mass - 1) : u == u ? mass - 1 : 0;
}

// the settings of a row. k = 1 and T = 1 stand for T = 0 (the largest logit, the lowest
// index of it)
struct Settings {
    float T, p, m;
    int k;
    bool good;
};
DDT_DEVINL Settings load_settings(const ddt_filter &f, int i)
{
    Settings s;
    s.T = f.temperature ? __ldg(f.temperature + i) : 1.f;
    s.k = f.top_k ? __ldg(f.top_k + i) : 0;
    s.p = f.top_p ? __ldg(f.top_p + i) : 1.f;
    s.m = f.min_p ? __ldg(f.min_p + i) : 0.f;
    s.good = s.T >= 0.f && s.T <= SR_MAX_FLOAT && s.p >= 0.f && s.p <= 1.f && s.m >= 0.f && s.m <= 1.f;
    if (s.T == 0.f) {
        s.T = 1.f;
        s.k = 1;
    }
    s.T = fmaxf(s.T, SR_TINY);
    return s;
}
// ---------------------------------------------------------------- border
struct Border {
    float z;   // kept: above this value, or equal to it
    int last;  //   with an index up to this
};
DDT_DEVINL bool kept(const Border &b, float z, int i) { return z > b.z || (z == b.z && i <= b.last); }

// ---------------------------------------------------------------- a row in shared memory
struct Xchg {
    uint64_t w[2][SR_MAX_CL][4];  // what the CTAs tell one another, by turns
};
struct RowShared {
    float2 tab[32];
    Xchg x;
    uint64_t warp[SR_FAR / 32][4];
    uint64_t list[SR_CAP];   // candidates: (order_key << 32) | ~index
    uint64_t mine[SR_CAP];   //   of this CTA's slice
    uint32_t hist[SR_BINS];
    uint32_t count;          //   how many
    int found[4];
    float2 off;              // T ln(min_p)
    uint64_t kept[SR_SMALL]; // the candidates' weights
};

// 16 bytes of logits. Range: the largest and the least that look() has seen; odd(): there may
// be odd ones among them: NaN (which is then the largest), or not 0 and next to 0 (SR_TINY)
template <typename T> struct Vec;
template <> struct Vec<uint16_t> {
    static constexpr int E = 8;
    static constexpr bool EXACT = false;
    static constexpr uint32_t NONE = 0xFF80FF80u;
    struct Range {
        uint32_t hi, lo, odd;  // odd: the least of (bits of the magnitude) - 1, of either half
    };
    DDT_DEVINL static void begin(Range &r) { r = {NONE, 0x7F7F7F7Fu, 0xFFFFFFFFu}; }
    DDT_DEVINL static void look(Range &r, const uint4 &v)
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(r.hi) : "r"(w[i]));
            asm("min.bf16x2 %0, %0, %1;" : "+r"(r.lo) : "r"(w[i]));
            // (a zero in the low half takes one more from the high half, which then counts as
            // odd one bit pattern early)
            asm("min.u16x2 %0, %0, %1;" : "+r"(r.odd) : "r"((w[i] & 0x7FFF7FFFu) - 0x00010001u));
        }
    }
    DDT_DEVINL static bool odd(const Range &r)
    {
        const uint32_t a = r.odd & 0xFFFFu, b = r.odd >> 16;
        const float x = bf16lo(r.hi), y = bf16hi(r.hi);
        return a < (37u << 7) - 1 || b < (37u << 7) - 1 || x != x || y != y;
    }
    DDT_DEVINL static void end(const Range &r, float &hi, float &lo)
    {
        hi = fmaxf(bf16lo(r.hi), bf16hi(r.hi));
        lo = fminf(bf16lo(r.lo), bf16hi(r.lo));
    }
    DDT_DEVINL static uint4 put(const uint16_t *x)
    {
        return make_uint4(x[0] | (uint32_t)x[1] << 16, x[2] | (uint32_t)x[3] << 16, x[4] | (uint32_t)x[5] << 16,
                          x[6] | (uint32_t)x[7] << 16);
    }
    // whether one of them reaches `from`
    DDT_DEVINL static bool reaches(const uint4 &v, float from)
    {
        uint32_t m;
        asm("{\n .reg .b32 a, b;\n max.bf16x2 a, %1, %2;\n max.bf16x2 b, %3, %4;\n max.bf16x2 %0, a, b;\n}\n"
            : "=r"(m) : "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w));
        return bf16lo(m) >= from || bf16hi(m) >= from;
    }
    DDT_DEVINL static void get(const uint4 &v, float *z)
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            z[2 * i] = bf16lo(w[i]);
            z[2 * i + 1] = bf16hi(w[i]);
        }
    }
};
template <> struct Vec<float> {
    static constexpr int E = 4;
    static constexpr bool EXACT = true;
    static constexpr uint32_t NONE = 0xFF800000u;
    struct Range {
        float hi, lo;
        uint32_t odd;
    };
    DDT_DEVINL static void begin(Range &r) { r = {DDT_NEG_INF, SR_MAX_FLOAT, 0xFFFFFFFFu}; }
    DDT_DEVINL static void look(Range &r, const uint4 &v)
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < E; ++e) {
            asm("max.NaN.f32 %0, %0, %1;" : "+f"(r.hi) : "f"(__uint_as_float(w[e])));
            r.lo = fminf(r.lo, __uint_as_float(w[e]));
            r.odd = min(r.odd, (w[e] & 0x7FFFFFFFu) - 1u);
        }
    }
    DDT_DEVINL static bool odd(const Range &r) { return r.odd < (37u << 23) - 1 || r.hi != r.hi; }
    DDT_DEVINL static void end(const Range &r, float &hi, float &lo)
    {
        hi = r.hi;
        lo = r.lo;
    }
    DDT_DEVINL static uint4 put(const float *x)
    {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
    DDT_DEVINL static bool reaches(const uint4 &v, float from)
    {
        float z[E];
        get(v, z);
        return fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3])) >= from;
    }
    DDT_DEVINL static void get(const uint4 &v, float *z)
    {
        z[0] = __uint_as_float(v.x);
        z[1] = __uint_as_float(v.y);
        z[2] = __uint_as_float(v.z);
        z[3] = __uint_as_float(v.w);
    }
};

// a logit as the row in shared memory holds it (Row::top, Row::only_infinite)
DDT_DEVINL float held_value(float z, bool infinite)
{
    if (infinite)
        return z == -DDT_NEG_INF ? 0.f : DDT_NEG_INF;
    return z != z ? DDT_NEG_INF : fabsf(z) < SR_TINY ? 0.f : z;
}
DDT_DEVINL float logit_value(const uint16_t *p, int64_t i) { return bf16_to_f32(__ldg(p + i)); }
DDT_DEVINL float logit_value(const float *p, int64_t i) { return __ldg(p + i); }

// sub-chunks of a row of V logits that begins anywhere (the row's first 16 bytes may hold
// up to E - 1 of the row before), and how many of them one of cl CTAs holds at most
template <typename T>
__host__ __device__ constexpr int row_subs(int V) { return (int)(((int64_t)V + Vec<T>::E - 1) * sizeof(T) + SR_SUB - 1) / SR_SUB; }
template <typename T>
__host__ __device__ constexpr int slice_subs(int V, int cl) { return (row_subs<T>(V) + cl - 1) / cl; }

// The slice of a row that a CTA holds. Element (sub-chunk s, lane, e) has index
// index0(s, lane) + e. FAR: the whole row, where it is in global memory.
template <typename T, bool FAR>
struct Slice {
    static constexpr int E = Vec<T>::E, SE = SR_SUB / (int)sizeof(T);
    static constexpr int G = FAR ? SR_GROUP : 1;  // sub-chunks of a group
    unsigned char *at;  // ns sub-chunks
    const T *base;      // the tensor's 16-byte vector that the row begins in
    int s0, ns, off, V;
    bool odd, infinite;  // FAR: the row has odd values; infinities

    DDT_DEVINL void place(unsigned char *smem, const T *row, int V_, uint32_t rank, uint32_t cl)
    {
        at = smem;
        odd = infinite = false;
        V = V_;
        off = (int)(((uintptr_t)row & 15) / sizeof(T));
        const int subs = (int)(((int64_t)off + V + SE - 1) / SE);
        s0 = (int)((int64_t)subs * rank / cl);
        ns = (int)((int64_t)subs * (rank + 1) / cl) - s0;
        base = row - off;
    }
    DDT_DEVINL int groups() const { return (ns + G - 1) / G; }
    // start this thread's copies. Whole 16-byte vectors of the row; what is before the
    // row's first element comes from the row before it (the tensor begins on 16 bytes)
    DDT_DEVINL void fetch(int tid) const
    {
        const uint32_t dst = (uint32_t)__cvta_generic_to_shared(at);
        const int64_t end = (int64_t)off + V;
        for (int v = tid; v < ns * 32; v += SR_THREADS) {
            const int64_t j = ((int64_t)s0 * 32 + v) * E;  // the vector's first element, from base
            if (j + E <= end) {
                cp16(dst + v * 16, base + j);
            } else {
                T *d = reinterpret_cast<T *>(at + v * 16);
                for (int e = 0; e < E; ++e)
                    d[e] = j + e < end ? base[j + e] : (T)none();
            }
        }
    }
    DDT_DEVINL static T none()
    {
        if constexpr (sizeof(T) == 2)
            return (T)0xFF80u;
        else
            return DDT_NEG_INF;
    }
    // after the copies and a barrier: elements before the row's first
    DDT_DEVINL void mend(int tid) const
    {
        if (s0 == 0 && ns > 0 && tid < off)
            reinterpret_cast<T *>(at)[tid] = none();
    }
    // a lane's vector of a sub-chunk (FAR: any sub-chunk; what is not the row's is -infinity)
    DDT_DEVINL uint4 raw(int s, int lane) const
    {
        if (!FAR)
            return *reinterpret_cast<const uint4 *>(at + s * SR_SUB + lane * 16);
        const int j = s * SE + lane * E;  // its first element, from base (off + V stays below 2^31)
        if (j >= off && j - off <= V - E)
            return __ldg(reinterpret_cast<const uint4 *>(base + j));
        T x[E];
#pragma unroll
        for (int e = 0; e < E; ++e)
            x[e] = j + e >= off && j + e - off < V ? __ldg(base + j + e) : none();
        return Vec<T>::put(x);
    }
    // those of N sub-chunks (FAR: where all of it is the row's, loads with no branch between)
    template <int N>
    DDT_DEVINL void raws(int s, int lane, uint4 (&x)[N]) const
    {
        if (FAR && s * SE >= off && (s + N) * SE <= off + V) {
            const uint4 *p = reinterpret_cast<const uint4 *>(base) + s * 32 + lane;
#pragma unroll
            for (int b = 0; b < N; ++b)
                x[b] = __ldg(p + b * 32);
        } else {
#pragma unroll
            for (int b = 0; b < N; ++b)
                x[b] = raw(s + b, lane);
        }
    }
    // a vector without odd values: a NaN is -infinity, what is next to 0 is 0
    DDT_DEVINL static uint4 mended(const uint4 &v)
    {
        T x[E];
        memcpy(x, &v, 16);
        float z[E];
        Vec<T>::get(v, z);
#pragma unroll
        for (int e = 0; e < E; ++e)
            x[e] = z[e] != z[e] ? none() : fabsf(z[e]) < SR_TINY ? (T)0 : x[e];
        return Vec<T>::put(x);
    }
    // its logits, as the row holds them
    DDT_DEVINL void values(const uint4 &v, float *z) const
    {
        Vec<T>::get(v, z);
        if (FAR && odd) {
#pragma unroll
            for (int e = 0; e < E; ++e)
                z[e] = held_value(z[e], infinite);
        }
    }
    DDT_DEVINL void get(int s, int lane, float *z) const { values(raw(s, lane), z); }
    DDT_DEVINL int index0(int s, int lane) const { return (s0 + s) * SE + lane * E - off; }
};

// totals over a warp
DDT_DEVINL uint64_t warp_sum64(uint64_t v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}
DDT_DEVINL uint64_t warp_incl64(uint64_t v, int lane)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t y = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o)
            v += y;
    }
    return v;
}

// One row of a cluster: what its threads share in doing it. FAR: of one CTA that reads it
// from global memory each time.
template <typename T, bool FAR = false>
struct Row {
    static constexpr int THREADS = FAR ? SR_FAR : SR_THREADS, WARPS = THREADS / 32;
    static constexpr int OWN = FAR ? SR_OWN : 1;
    static constexpr int E = Vec<T>::E;
    static constexpr bool EXACT = Vec<T>::EXACT;
    RowShared *sh;
    using Part = Slice<T, FAR>;
    Part sl;
    int tid, lane, warp;
    uint32_t rank, cl, turn;

    DDT_DEVINL void begin(RowShared *s)
    {
        sh = s;
        tid = threadIdx.x;
        lane = tid & 31;
        warp = tid >> 5;
        rank = FAR ? 0 : cl_rank();
        cl = FAR ? 1 : cl_size();
        turn = 0;
        if (!FAR)
            cl_arrive();  // (ended by started(): a CTA's shared memory is there once it runs)
    }
    // before the first access to another CTA's shared memory
    DDT_DEVINL void started()
    {
        if (!FAR)
            cl_wait();
    }
    DDT_DEVINL void sync_row()
    {
        if (FAR)
            __syncthreads();
        else
            cl_sync();
    }
    // f(sub-chunk, its raw 16 bytes) over this warp's part; end(group) after each group
    template <typename F, typename End>
    DDT_DEVINL void each(F f, End end) const
    {
        constexpr int G = Part::G;
        const int n = sl.groups();
        for (int g = warp; g < n; g += WARPS) {
            uint4 x[G];
            sl.raws(g * G, lane, x);
#pragma unroll
            for (int b = 0; b < G; ++b)
                f(g * G + b, x[b]);
            end(g);
        }
    }
    template <typename F>
    DDT_DEVINL void each(F f) const
    {
        each(f, [](int) {});
    }

    // Every CTA tells the others up to four words (held by every thread). A place is
    // written again only two exchanges later, behind a barrier that its readers reach
    // after they have read. Returns the words of all CTAs.
    DDT_DEVINL const uint64_t (*exchange(uint64_t a, uint64_t b, uint64_t c, uint64_t d))[4]
    {
        const uint32_t p = turn++ & 1;
        if (FAR) {
            if (tid < 4)
                sh->x.w[p][0][tid] = tid == 0 ? a : tid == 1 ? b : tid == 2 ? c : d;
            __syncthreads();
            return sh->x.w[p];
        }
        if (tid < (int)cl * 4) {
            const int q = tid & 3;
            cl_st64(cl_map(&sh->x.w[p][rank][q], tid >> 2), q == 0 ? a : q == 1 ? b : q == 2 ? c : d);
        }
        cl_sync();
        return sh->x.w[p];
    }

    // hold a row: copies started, and waited for
    DDT_DEVINL void load(unsigned char *smem, const T *row, int V)
    {
        sl.place(smem, row, V, rank, cl);
        if (!FAR)
            sl.fetch(tid);
        if (tid < 32)
            sh->tab[tid] = SR_TABLE[tid];
    }
    DDT_DEVINL void loaded()
    {
        if (FAR) {
            __syncthreads();
            return;
        }
        cp_wait_all();
        __syncthreads();
        sl.mend(tid);
        __syncthreads();
    }

    // ---- the row's largest and least (finite) value, the largest of each thread's (FAR: of
    // each of SR_OWN parts of them)
    struct Top {
        float zmax, own[OWN], low;
        bool nan;
    };
    DDT_DEVINL Top top()
    {
        Top r;
        bool nan = false;
        float m, lo;
        if (__syncthreads_or(look(r, m, lo))) {
            // from here on a NaN is -infinity, and what is next to 0 is 0
            sl.odd = FAR;
            each([&](int s, const uint4 &v) {
                float z[E];
                Vec<T>::get(v, z);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    nan |= z[e] != z[e];
                if (!FAR)
                    mend_vector(s);
            });
            __syncthreads();
            look(r, m, lo);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
            lo = fminf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, o));
        }
        nan = __any_sync(0xFFFFFFFFu, nan);
        if (lane == 0)
            sh->warp[warp][0] = ((uint64_t)__float_as_uint(m) << 32) | __float_as_uint(lo), sh->warp[warp][1] = nan;
        __syncthreads();
        nan = false;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            const uint64_t x = sh->warp[w][0];
            m = fmaxf(m, __uint_as_float((uint32_t)(x >> 32)));
            lo = fminf(lo, __uint_as_float((uint32_t)x));
            nan |= sh->warp[w][1] != 0;
        }
        const uint64_t(*all)[4] = exchange(((uint64_t)__float_as_uint(m) << 32) | __float_as_uint(lo), nan, 0, 0);
        for (uint32_t c = 0; c < cl; ++c) {
            const uint64_t x = all[c][0];
            m = fmaxf(m, __uint_as_float((uint32_t)(x >> 32)));
            lo = fminf(lo, __uint_as_float((uint32_t)x));
            nan |= all[c][1] != 0;
        }
        r.zmax = m;
        r.low = lo;
        r.nan = nan;
        return r;
    }
    // this thread's part of that; whether there are odd values
    DDT_DEVINL bool look(Top &r, float &m, float &lo)
    {
        typename Vec<T>::Range range[OWN];
#pragma unroll
        for (int o = 0; o < OWN; ++o)
            Vec<T>::begin(range[o]);
        // (sub-chunks at once; near ones may be looked at twice)
        constexpr int N = FAR ? SR_OWN : 2;
        for (int s = warp * (FAR ? N : 1); s < sl.ns; s += WARPS * N) {
            uint4 x[N];
            if (FAR) {
                sl.raws(s, lane, x);
                if (sl.odd) {
#pragma unroll
                    for (int o = 0; o < N; ++o)
                        x[o] = sl.mended(x[o]);
                }
            } else {
#pragma unroll
                for (int o = 0; o < N; ++o)
                    x[o] = sl.raw(s + o * WARPS < sl.ns ? s + o * WARPS : s, lane);
            }
#pragma unroll
            for (int o = 0; o < N; ++o)
                Vec<T>::look(range[FAR ? o : 0], x[o]);
        }
        bool odd = false;
        m = DDT_NEG_INF;
        lo = SR_MAX_FLOAT;
#pragma unroll
        for (int o = 0; o < OWN; ++o) {
            float l;
            odd |= Vec<T>::odd(range[o]);
            Vec<T>::end(range[o], r.own[o], l);
            m = fmaxf(m, r.own[o]);
            lo = fminf(lo, l);
        }
        return odd;
    }
    // a lane's vector with odd values
    DDT_DEVINL void mend_vector(int s) { *reinterpret_cast<uint4 *>(sl.at + s * SR_SUB + lane * 16) = sl.mended(sl.raw(s, lane)); }
    // a row with +infinity: those tokens have equal weights, the others none
    DDT_DEVINL void only_infinite(Top &t)
    {
        if (FAR)
            sl.odd = sl.infinite = true;
        else
            for (int s = warp; s < sl.ns; s += WARPS) {
                T *d = reinterpret_cast<T *>(sl.at + s * SR_SUB + lane * 16);
                float z[E];
                sl.get(s, lane, z);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    d[e] = z[e] == t.zmax ? (T)0 : Part::none();
            }
        __syncthreads();
#pragma unroll
        for (int o = 0; o < OWN; ++o)
            t.own[o] = t.own[o] == t.zmax ? 0.f : DDT_NEG_INF;
        t.zmax = t.low = 0.f;
    }

    // block-wide sum of one word a thread, known to all
    DDT_DEVINL uint64_t block_sum(uint64_t v)
    {
        v = warp_sum64(v);
        __syncthreads();  // (the words before have been read)
        if (lane == 0)
            sh->warp[warp][0] = v;
        __syncthreads();
        uint64_t t = 0;
#pragma unroll
        for (int w = 0; w < WARPS; ++w)
            t += sh->warp[w][0];
        return t;
    }

    // ---- sum of the weights of the kept tokens, over the row. sub: each sub-chunk's
    // (or null). all: every CTA's total
    DDT_DEVINL uint64_t mass(const Scale &sc, const Border &b, uint64_t *sub, const uint64_t (**all)[4])
    {
        uint64_t own = 0;
        const bool cut = b.last < sl.V - 1;
        uint64_t group = 0;
        each([&](int s, const uint4 &v) {
            float z[E];
            sl.values(v, z);
            const int i0 = sl.index0(s, lane);
            bool k[E], some = false;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                k[e] = z[e] >= b.z;
                if (cut && z[e] == b.z)
                    k[e] = i0 + e <= b.last;
                some |= k[e];
            }
            if (__any_sync(0xFFFFFFFFu, some)) {
                Sum2 sum = {0, 0};
#pragma unroll
                for (int e = 0; e < E; e += 2)
                    add_weights<EXACT>(sc, sh->tab, z[e], z[e + 1], k[e], k[e + 1], sum);
                group += to_fixed(sum);
            }
        }, [&](int g) {
            own += group;
            if (sub && __any_sync(0xFFFFFFFFu, group != 0))
                group = warp_sum64(group);
            if (sub && lane == 0)
                sub[g] = group;
            group = 0;
        });
        const uint64_t mine = block_sum(own);
        const uint64_t(*a)[4] = exchange(mine, 0, 0, 0);
        uint64_t t = 0;
        for (uint32_t c = 0; c < cl; ++c)
            t += a[c][0];
        if (all)
            *all = a;
        return t;
    }

    // ---- the same in plain fp32 (see quick_slack)
    DDT_DEVINL uint64_t quick_mass(const Scale &sc, const Border &b, uint64_t *sub, const uint64_t (**all)[4])
    {
        uint64_t own = 0, group = 0;
        const bool cut = b.last < sl.V - 1;
        each([&](int s, const uint4 &v) {
            float z[E];
            sl.values(v, z);
            group += cut ? quick_fixed(sc, b, z, sl.index0(s, lane), E - 1) : quick_fixed(sc, {b.z, 0x7FFFFFFF}, z, 0, E - 1);
        }, [&](int g) {
            own += group;
            if (sub) {
                group = warp_sum64(group);
                if (lane == 0)
                    sub[g] = group;
            }
            group = 0;
        });
        const uint64_t(*a)[4] = exchange(block_sum(own), 0, 0, 0);
        uint64_t t = 0;
        for (uint32_t c = 0; c < cl; ++c)
            t += a[c][0];
        if (all)
            *all = a;
        return t;
    }
    DDT_DEVINL static uint64_t quick_fixed(const Scale &sc, const Border &b, const float *z, int i0, int last)
    {
        uint64_t w = 0;
        const auto in = [&](int e) { return e <= last && (b.last == 0x7FFFFFFF ? z[e] >= b.z : kept(b, z[e], i0 + e)); };
#pragma unroll
        for (int e = 0; e < E; e += 2)
            w = f2add(w, quick_weights<EXACT>(sc, z[e], z[e + 1], in(e), in(e + 1)));
        float w0, w1;
        f2unpack(w, w0, w1);
        return __float2ull_rn((w0 + w1) * 17592186044416.0f);
    }
    struct QuickWeight {  // adds these up
        Scale sc;
        Border b;
        DDT_DEVINL uint64_t sum_to(const float *z, int i0, int last) const { return quick_fixed(sc, b, z, i0, last); }
        DDT_DEVINL uint64_t lane_sum(const float *z, int i0) const { return quick_fixed(sc, b, z, i0, E - 1); }
    };

    // ---- histogram of values from vhi down, and the first bin at which the tokens so far
    // reach `want` (-1: never). Bins are even in value: (vhi - z) * scale, cut off.
    DDT_DEVINL static int bin_of(float vhi, float scale, float z) { return min(SR_BINS - 1, (int)((vhi - z) * scale)); }
    DDT_DEVINL static float bin_scale(float vhi, float vlo)
    {
        const float r = vhi - vlo;  // (finite: both within the floats' half range, or the difference is cut)
        return r > 0.f ? (SR_BINS - 1) / fminf(r, SR_MAX_FLOAT) : 0.f;
    }
    DDT_DEVINL void clear_hist()
    {
        for (int i = tid; i < SR_BINS; i += THREADS)
            sh->hist[i] = 0;
        __syncthreads();
    }
    // after a cluster barrier: this thread's two bins over the whole row
    DDT_DEVINL void row_bins(uint32_t &n0, uint32_t &n1)
    {
        n0 = n1 = 0;
        if (FAR) {
            if (2 * tid < SR_BINS) {
                n0 = sh->hist[2 * tid];
                n1 = sh->hist[2 * tid + 1];
            }
            return;
        }
        for (uint32_t b = 0; b < cl; b += 4) {  // (four at a time: the loads overlap)
            uint32_t x[4], y[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const uint32_t at = cl_map(&sh->hist[2 * tid], min(b + c, cl - 1));
                x[c] = cl_ld32(at);
                y[c] = cl_ld32(at + 4);
            }
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (b + c < cl)
                    n0 += x[c], n1 += y[c];
        }
    }
    // inclusive running sum over the threads of one word each
    DDT_DEVINL uint64_t block_incl(uint64_t v)
    {
        v = warp_incl64(v, lane);
        __syncthreads();
        if (lane == 31)
            sh->warp[warp][0] = v;
        __syncthreads();
        for (int w = 0; w < warp; ++w)
            v += sh->warp[w][0];
        return v;
    }
    // the smallest of the threads' candidates (none: 0x7fffffff), known to all
    DDT_DEVINL int block_least(int v)
    {
        v = __reduce_min_sync(0xFFFFFFFFu, v);
        __syncthreads();
        if (lane == 0)
            sh->warp[warp][0] = (uint64_t)(uint32_t)v;
        __syncthreads();
        int r = 0x7FFFFFFF;
#pragma unroll
        for (int w = 0; w < WARPS; ++w)
            r = min(r, (int)(uint32_t)sh->warp[w][0]);
        return r;
    }

    // ---- collect the tokens that `in` names, all of them at or above `from`, in the first
    // CTA (in any order); returns how many there are, which may be more than the list holds
    // (then it holds none). Each CTA lists its own; the first one fetches them: the others
    // may not leave before fetched().
    template <typename In>
    DDT_DEVINL uint32_t collect(float from, In in)
    {
        if (tid == 0)
            sh->count = 0;
        __syncthreads();
        uint64_t *to = FAR ? sh->list : sh->mine;
        each([&](int s, const uint4 &v) {
            if (!(FAR && sl.odd) && !Vec<T>::reaches(v, from))
                return;
            float z[E];
            sl.values(v, z);
            const int i0 = sl.index0(s, lane);
            bool k[E];
            uint32_t n = 0;
#pragma unroll
            for (int e = 0; e < E; ++e)
                n += k[e] = in(z[e], i0 + e);
            if (n > 0) {
                uint32_t p = atomicAdd(&sh->count, n);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (k[e]) {
                        if (p < SR_CAP)
                            to[p] = ((uint64_t)order_key(z[e]) << 32) | (uint32_t)~(i0 + e);
                        ++p;
                    }
            }
        });
        __syncthreads();
        if (FAR)
            return sh->count;
        const uint64_t(*all)[4] = exchange(sh->count, 0, 0, 0);
        uint32_t n = 0;
        for (uint32_t c = 0; c < cl; ++c)
            n += (uint32_t)all[c][0];
        if (n <= SR_CAP) {
            if (rank == 0) {
                for (uint32_t i = tid; i < n; i += THREADS) {
                    uint32_t c = 0, j = i;
                    while (j >= (uint32_t)all[c][0])
                        j -= (uint32_t)all[c++][0];
                    sh->list[i] = cl_ld64(cl_map(&sh->mine[j], c));
                }
                __syncthreads();
            }
            cl_arrive();
        }
        return n;
    }
    // (after a collection that the list holds, before anything else between CTAs)
    DDT_DEVINL void fetched()
    {
        if (FAR)
            __syncthreads();
        else
            cl_wait();
    }

    // the first CTA: its list's n candidates in descending order (value, then lower index)
    DDT_DEVINL void sort_list(int n)
    {
        int p2 = 32;
        while (p2 < n)
            p2 <<= 1;
        for (int i = n + tid; i < p2; i += THREADS)
            sh->list[i] = 0;
        __syncthreads();
        for (int k = 2; k <= p2; k <<= 1)
            for (int j = k >> 1; j > 0; j >>= 1) {
                for (int i = tid; i < p2 / 2; i += THREADS) {
                    const int lo = 2 * j * (i / j) + i % j, hi = lo + j;
                    const uint64_t a = sh->list[lo], b = sh->list[hi];
                    if ((a < b) == ((lo & k) == 0)) {
                        sh->list[lo] = b;
                        sh->list[hi] = a;
                    }
                }
                __syncthreads();
            }
    }

    // ---- the border among the collected candidates (the first CTA), and the draw. They are
    // all tokens from some value up. At most `limit` of them count; p < 1: the fewest that
    // reach p of `base` (0: of the sum of those that count), within `slack` of which no
    // border may lie.
    struct Cut {
        Border b;
        uint64_t mass;  // of all that is kept
        bool ok;        // the border was found
    };
    // up to SR_SMALL of them, a thread each: its place in the order and what comes before it
    // by looking at all. u >= 0: the token drawn, in one thread (-1 elsewhere)
    DDT_DEVINL Cut small_list(const Scale &sc, int n, int limit, float p, uint64_t base, uint64_t slack, float u, int &token)
    {
        token = -1;
        const uint64_t key = tid < n ? sh->list[tid] : 0;
        const float z = key_value((uint32_t)(key >> 32));
        const uint64_t w = tid < n ? weight_of<EXACT>(sc, sh->tab, z) : 0;
        if (tid < SR_SMALL)
            sh->kept[tid] = w;
        if (tid == 0)
            sh->found[0] = 0;
        __syncthreads();
        int place = 0;
        uint64_t before = 0;
        for (int j = 0; j < n; ++j) {
            const bool b = sh->list[j] > key;
            place += b;
            before += b ? sh->kept[j] : 0;
        }
        bool in = tid < n && place < limit;
        bool ok = true;
        if (p < 1.f) {
            const uint64_t own = block_sum(in ? w : 0), want = max(share_of(p, base ? base : own), (uint64_t)1);
            const uint64_t gap = base ? slack : 0;
            // reached, and by no doubtful step
            ok = !base || own >= want + gap;
            const bool doubt = in && gap > 0 && ((before < want + gap && want < before + gap) ||
                                                 (before + w < want + gap && want < before + w + gap));
            ok = ok && !__syncthreads_or(doubt);
            in = in && before < want;
        }
        const int m = __syncthreads_count(in);
        if (in && place == m - 1) {
            sh->found[0] = tid;
            sh->warp[0][3] = before + w;
        }
        if (tid < SR_SMALL)
            sh->kept[tid] = in ? w : 0;
        __syncthreads();
        Cut c;
        const uint64_t last = sh->list[sh->found[0]];
        c.b.z = key_value((uint32_t)(last >> 32));
        c.b.last = (int)~(uint32_t)last;
        c.mass = sh->warp[0][3];
        c.ok = ok;
        if (u >= 0.f && ok) {
            const uint64_t target = draw_target(u, c.mass);
            uint64_t sum = 0;  // of the kept tokens of lower index
            for (int j = 0; j < n; ++j)
                sum += (uint32_t)sh->list[j] > (uint32_t)key ? sh->kept[j] : 0;
            if (in && sum <= target && target < sum + w)
                token = (int)~(uint32_t)key;
        }
        return c;
    }
    // any number that the list holds, sorted; what is above them weighs `above`, the sum has
    // to reach `want` (0: `limit` is the border). Known to all CTAs afterwards
    DDT_DEVINL Cut cut_list(const Scale &sc, int n, int limit, uint64_t above, uint64_t want)
    {
        float z = 0.f;
        int last = 0;
        uint64_t mass = 0;
        if (rank == 0) {
            sort_list(n);
            const int n2 = min(n, limit), r0 = 2 * tid;
            uint64_t w0 = 0, w1 = 0;
            if (r0 < n2)
                w0 = weight_of<EXACT>(sc, sh->tab, key_value((uint32_t)(sh->list[r0] >> 32)));
            if (r0 + 1 < n2)
                w1 = weight_of<EXACT>(sc, sh->tab, key_value((uint32_t)(sh->list[r0 + 1] >> 32)));
            const uint64_t incl = above + block_incl(w0 + w1);
            int first = n2 - 1;
            if (want > 0) {
                first = block_least(r0 < n2 && incl - w1 >= want ? r0 : r0 + 1 < n2 && incl >= want ? r0 + 1 : 0x7FFFFFFF);
                if (first == 0x7FFFFFFF)  // (rounding in `want`)
                    first = n2 - 1;
            }
            const uint64_t key = sh->list[first];
            z = key_value((uint32_t)(key >> 32));
            last = (int)~(uint32_t)key;
            __syncthreads();
            if (tid == (first >> 1))
                sh->warp[0][2] = first & 1 ? incl : incl - w1;
            __syncthreads();
            mass = sh->warp[0][2];
        }
        const uint64_t(*a)[4] = exchange(((uint64_t)__float_as_uint(z) << 32) | (uint32_t)last, mass, 0, 0);
        Cut c;
        c.b.z = __uint_as_float((uint32_t)(a[0][0] >> 32));
        c.b.last = (int)(uint32_t)a[0][0];
        c.mass = a[0][1];
        c.ok = true;
        return c;
    }
    DDT_DEVINL static uint64_t share_of(float p, uint64_t mass) { return fraction_of(p, mass, true); }

    // ---- a value that at least `need` tokens reach (lo, if fewer than that many reach lo),
    // and not many more: from the threads' largest ones (each a different token), or, where
    // these are too few, from all tokens
    DDT_DEVINL float probe(const Top &t, float lo, uint32_t need)
    {
        const float vlo = fmaxf(t.low, lo), scale = bin_scale(t.zmax, vlo);
        clear_hist();
        if ((int64_t)sl.V >= (int64_t)4 * need * E && cl * THREADS * OWN >= 4 * need) {
#pragma unroll
            for (int o = 0; o < OWN; ++o)
                if (t.own[o] >= vlo)
                    atomicAdd(&sh->hist[bin_of(t.zmax, scale, t.own[o])], 1u);
        } else {
            each([&](int, const uint4 &v) {
                float z[E];
                sl.values(v, z);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (z[e] >= vlo)
                        atomicAdd(&sh->hist[bin_of(t.zmax, scale, z[e])], 1u);
            });
        }
        sync_row();
        uint32_t n0, n1;
        row_bins(n0, n1);
        const uint64_t incl = block_incl(n0 + n1);
        const int b = block_least(incl - n1 >= need ? 2 * tid : incl >= need ? 2 * tid + 1 : 0x7FFFFFFF);
        if (b == 0x7FFFFFFF)
            return lo;
        // (a hundredth of a bin covers the rounding of bin_of: 511 * 2^-23 of one)
        return scale > 0.f ? fmaxf(lo, t.zmax - (b + 1.01f) / scale) : t.zmax;
    }

    // members of an interval of values: how many, the least and the greatest, and the weight
    // of the tokens that come before them (and, ALL, of all that a border keeps)
    struct Members {
        uint32_t n;
        float lo, hi;
        uint64_t before, all;
    };
    template <bool ALL, typename Before, typename In>
    DDT_DEVINL Members members(const Scale &sc, const Border &keep, Before before, In in)
    {
        uint64_t w = 0, all = 0;
        uint32_t n = 0;
        float lo = SR_MAX_FLOAT, hi = -SR_MAX_FLOAT;
        each([&](int s, const uint4 &v) {
            float z[E];
            sl.values(v, z);
            const int i0 = sl.index0(s, lane);
            bool k[E], some = false;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                some |= k[e] = before(z[e], i0 + e);
                if (in(z[e], i0 + e)) {
                    ++n;
                    lo = fminf(lo, z[e]);
                    hi = fmaxf(hi, z[e]);
                }
            }
            if (__any_sync(0xFFFFFFFFu, some)) {
                Sum2 sum = {0, 0};
#pragma unroll
                for (int e = 0; e < E; e += 2)
                    add_weights<EXACT>(sc, sh->tab, z[e], z[e + 1], k[e], k[e + 1], sum);
                w += to_fixed(sum);
            }
            if (ALL) {
                Sum2 sum = {0, 0};
#pragma unroll
                for (int e = 0; e < E; e += 2)
                    add_weights<EXACT>(sc, sh->tab, z[e], z[e + 1], !k[e] && kept(keep, z[e], i0 + e),
                                       !k[e + 1] && kept(keep, z[e + 1], i0 + e + 1), sum);
                all += to_fixed(sum);
            }
        });
        w = warp_sum64(w);
        all = warp_sum64(all) + w;
        n = __reduce_add_sync(0xFFFFFFFFu, n);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            lo = fminf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, o));
            hi = fmaxf(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, o));
        }
        __syncthreads();
        if (lane == 0) {
            sh->warp[warp][0] = w;
            sh->warp[warp][1] = n;
            sh->warp[warp][2] = ((uint64_t)__float_as_uint(hi) << 32) | __float_as_uint(lo);
            sh->warp[warp][3] = all;
        }
        __syncthreads();
        auto sum = [&](const uint64_t(*a)[4], uint32_t count) {
            Members m = {0, SR_MAX_FLOAT, -SR_MAX_FLOAT, 0, 0};
            for (uint32_t c = 0; c < count; ++c) {
                m.before += a[c][0];
                m.n += (uint32_t)a[c][1];
                m.lo = fminf(m.lo, __uint_as_float((uint32_t)a[c][2]));
                m.hi = fmaxf(m.hi, __uint_as_float((uint32_t)(a[c][2] >> 32)));
                m.all += a[c][3];
            }
            return m;
        };
        const Members m = sum(sh->warp, WARPS);
        return sum(exchange(m.before, m.n, ((uint64_t)__float_as_uint(m.hi) << 32) | __float_as_uint(m.lo), m.all), cl);
    }

    // ---- the CTA whose part holds `target` (the running sum first exceeds it there) finds
    // the token. sub: the sub-chunks' sums; all: the CTAs'. F gives a lane's sum and the sum
    // up to an element. Returns the index in one thread of one CTA, -1 elsewhere.
    template <typename F>
    DDT_DEVINL int locate(const uint64_t *sub, const uint64_t (*all)[4], uint64_t target, F f, uint64_t *from = nullptr,
                          uint64_t *to_ = nullptr)
    {
        uint64_t before = 0;
        for (uint32_t c = 0; c < rank; ++c)
            before += all[c][0];
        if (!(before <= target && target < before + all[rank][0]))
            return -1;
        const int ng = sl.groups(), per = (ng + THREADS - 1) / THREADS, a = min(ng, tid * per), b = min(ng, a + per);
        uint64_t own = 0;
        for (int s = a; s < b; ++s)
            own += sub[s];
        uint64_t at = before + block_incl(own) - own;
        if (at <= target && target < at + own) {
            int s = a;
            while (target >= at + sub[s])
                at += sub[s++];
            sh->found[0] = s;
            sh->warp[0][3] = at;
        }
        __syncthreads();
        if (warp > 0)
            return -1;
        int s = sh->found[0] * Part::G;
        at = sh->warp[0][3];
        float z[E];
        uint64_t sum, to;
        uint32_t hit;
        for (int end = s + Part::G;;) {  // (the group's sum is its lanes': one is hit)
            sl.get(s, lane, z);
            sum = f.lane_sum(z, sl.index0(s, lane));
            to = at + warp_incl64(sum, lane);
            hit = __ballot_sync(0xFFFFFFFFu, target < to);
            if (Part::G == 1 || hit != 0 || s + 1 == end)
                break;
            at = __shfl_sync(0xFFFFFFFFu, to, 31);
            ++s;
        }
        const int who = __ffs(hit) - 1;
        at = __shfl_sync(0xFFFFFFFFu, to - sum, who);
#pragma unroll
        for (int e = 0; e < E; ++e)
            z[e] = __shfl_sync(0xFFFFFFFFu, z[e], who);
        const int i0 = sl.index0(s, who), e = lane & (E - 1);
        const uint64_t sum_e = at + f.sum_to(z, i0, e);
        const uint32_t over = __ballot_sync(0xFFFFFFFFu, target < sum_e);
        const int pick = __ffs(over) - 1;
        if (from) {  // the running sum ahead of the token and with it
            const uint64_t ahead = __shfl_up_sync(0xFFFFFFFFu, sum_e, 1);
            *from = lane > 0 ? ahead : at;
            *to_ = sum_e;
        }
        return lane == pick ? i0 + pick : -1;
    }

    // ---- the same sum for any weights: F gives a lane's, over a sub-chunk's 16 bytes
    template <typename F>
    DDT_DEVINL uint64_t total(const F &f, uint64_t *sub, const uint64_t (**all)[4])
    {
        uint64_t own = 0, group = 0;
        each([&](int s, const uint4 &v) {
            float z[E];
            sl.values(v, z);
            group += f.lane_sum(z, sl.index0(s, lane));
        }, [&](int g) {
            own += group;
            group = warp_sum64(group);
            if (lane == 0)
                sub[g] = group;
            group = 0;
        });
        const uint64_t(*a)[4] = exchange(block_sum(own), 0, 0, 0);
        uint64_t t = 0;
        for (uint32_t c = 0; c < cl; ++c)
            t += a[c][0];
        *all = a;
        return t;
    }

    struct Equal {  // counts the tokens of one value that a border keeps
        Border b;
        float v;
        DDT_DEVINL uint64_t sum_to(const float *z, int i0, int last) const
        {
            uint64_t n = 0;
#pragma unroll
            for (int e = 0; e < E; ++e)
                n += e <= last && z[e] == v && kept(b, z[e], i0 + e);
            return n;
        }
        DDT_DEVINL uint64_t lane_sum(const float *z, int i0) const { return sum_to(z, i0, E - 1); }
    };
    // the index of the m-th token (1, 2, ...) of value v that b keeps; known to all
    DDT_DEVINL int nth_equal(const Border &b, float v, uint64_t m, uint64_t *sub)
    {
        const Equal eq = {b, v};
        const uint64_t(*all)[4];
        total(eq, sub, &all);
        const int i = locate(sub, all, m - 1, eq);
        __syncthreads();
        if (tid == 0)
            sh->found[1] = -1;
        __syncthreads();
        if (i >= 0)
            sh->found[1] = i;
        __syncthreads();
        const uint64_t(*who)[4] = exchange((uint64_t)(int64_t)sh->found[1], 0, 0, 0);
        int r = -1;
        for (uint32_t c = 0; c < cl; ++c)
            r = max(r, (int)(int64_t)who[c][0]);
        return r;
    }

    // ---- the border of the first k tokens at or above lo, by counts: histograms of ever
    // smaller intervals, until their tokens fit the list or have one value
    DDT_DEVINL Border count_border(const Top &t, const Scale &sc, float lo, int64_t k, uint64_t *sub)
    {
        float vhi = t.zmax, vlo = fmaxf(lo, t.low);
        uint64_t before = 0;
        for (int it = 0; it < 64; ++it) {
            const float scale = bin_scale(vhi, vlo);
            clear_hist();
            each([&](int, const uint4 &v) {
                float z[E];
                sl.values(v, z);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (z[e] >= vlo && z[e] <= vhi)
                        atomicAdd(&sh->hist[bin_of(vhi, scale, z[e])], 1u);
            });
            sync_row();
            uint32_t n0, n1;
            row_bins(n0, n1);
            const uint64_t incl = before + block_incl(n0 + n1);
            const uint64_t want = (uint64_t)k;
            const int b = block_least(incl - n1 >= want ? 2 * tid : incl >= want ? 2 * tid + 1 : 0x7FFFFFFF);
            if (b == 0x7FFFFFFF)
                break;  // fewer than k
            if (tid == (b >> 1)) {
                sh->warp[0][1] = b & 1 ? incl - n1 : incl - n1 - n0;
                sh->warp[0][2] = b & 1 ? n1 : n0;
            }
            __syncthreads();
            before = sh->warp[0][1];
            const uint64_t n = sh->warp[0][2];
            auto in = [=](float z, int) { return z >= vlo && z <= vhi && bin_of(vhi, scale, z) == b; };
            if (n <= SR_CAP) {
                collect(vlo, in);
                fetched();
                return cut_list(sc, (int)n, (int)(want - before), 0, 0).b;
            }
            const Members m = members<false>(sc, Border{0.f, 0}, [](float, int) { return false; }, in);
            if (m.lo == m.hi) {
                Border r = {m.lo, 0x7FFFFFFF};
                if (want - before < n)
                    r.last = nth_equal(r, m.lo, want - before, sub);
                return r;
            }
            vlo = m.lo;
            vhi = m.hi;
        }
        return Border{lo, 0x7FFFFFFF};
    }

    // ---- the border of the front part of what b keeps whose weights first reach p of their
    // sum, by bounds of the bins' weights (tokens times the bin's ends). about: that sum by
    // quick weights; the first look at all tokens' weights makes it exact
    DDT_DEVINL Cut mass_border(const Top &t, const Scale &sc, const Border &b, float p, uint64_t about, uint64_t *sub)
    {
        float vhi = t.zmax, vlo = fmaxf(b.z, t.low);
        uint64_t above = 0, least = share_of(p, about - quick_slack(about)), most = share_of(p, about + quick_slack(about));
        for (int it = 0; it < 64; ++it) {
            const float scale = bin_scale(vhi, vlo);
            clear_hist();
            each([&](int s, const uint4 &v) {
                float z[E];
                sl.values(v, z);
                const int i0 = sl.index0(s, lane);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (z[e] >= vlo && z[e] <= vhi && kept(b, z[e], i0 + e))
                        atomicAdd(&sh->hist[bin_of(vhi, scale, z[e])], 1u);
            });
            sync_row();
            uint32_t n[2];
            row_bins(n[0], n[1]);
            uint64_t up[2], low[2];
            const float inv = scale > 0.f ? 1.f / scale : 0.f;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int bin = 2 * tid + x;
                // (a hundredth of a bin and 2^-16 of the weight cover what fp32 rounds here)
                const float hi = fminf(0.f, (vhi - sc.zmax) - (bin - 0.01f) * inv), lo = (vhi - sc.zmax) - (bin + 1.01f) * inv;
                up[x] = __float2ull_ru((float)n[x] * fminf(1.f, ex2(hi * sc.ch) * 1.0000153f) * 17592186044416.0f);
                low[x] = __float2ull_rd((float)n[x] * (ex2(lo * sc.ch) * 0.9999847f) * 17592186044416.0f);
            }
            const uint64_t iu = above + block_incl(up[0] + up[1]);
            int first = block_least(iu - up[1] >= least ? 2 * tid : iu >= least ? 2 * tid + 1 : 0x7FFFFFFF);
            const uint64_t il = above + block_incl(low[0] + low[1]);
            int final_ = block_least(il - low[1] >= most ? 2 * tid : il >= most ? 2 * tid + 1 : 0x7FFFFFFF);
            first = min(first, SR_BINS - 1);
            final_ = min(final_, SR_BINS - 1);
            auto front = [=](float z, int i) { return z >= vlo && z <= vhi && bin_of(vhi, scale, z) < first && kept(b, z, i); };
            auto in = [=](float z, int i) {
                if (!(z >= vlo && z <= vhi && kept(b, z, i)))
                    return false;
                const int x = bin_of(vhi, scale, z);
                return x >= first && x <= final_;
            };
            Members m;
            if (it == 0) {
                m = members<true>(sc, b, front, in);
                least = most = max(share_of(p, m.all), (uint64_t)1);
            } else {
                m = members<false>(sc, b, front, in);
            }
            above += m.before;
            if (m.n == 0)  // (not so: the bounds hold)
                break;
            if (m.n <= SR_CAP) {
                collect(vlo, in);
                fetched();
                return cut_list(sc, (int)m.n, (int)m.n, above, least);
            }
            if (m.lo == m.hi) {
                const uint64_t w = weight_of<EXACT>(sc, sh->tab, m.lo);
                uint64_t c = least > above && w > 0 ? (least - above + w - 1) / w : 1;
                c = min(c, (uint64_t)m.n);
                Border r = {m.lo, m.lo == b.z ? b.last : 0x7FFFFFFF};
                if (c < m.n)
                    r.last = nth_equal(r, m.lo, c, sub);
                return Cut{r, above + c * w, true};
            }
            vlo = m.lo;
            vhi = m.hi;
        }
        return Cut{b, 0, false};
    }

    // ---- What the settings keep, and (u >= 0) the token drawn: in one thread of the cluster
    // token >= 0, and that thread's mass. u < 0: the border and the mass, in the first CTA.
    // COUNTS: false is returned where counting values serves better (nothing has been found,
    // and this CTA's part of the row may be overwritten).
    struct Found {
        Border b;
        uint64_t mass;
        int token;
        bool quick;
    };
    template <bool COUNTS>
    DDT_DEVINL bool solve(const Top &t, const Scale &sc, const Settings &set, float min_z, float u, uint64_t *sub, Found &r)
    {
        const float lo = fmaxf(min_z, sc.zfloor), p = set.p;
        const int k = set.k <= 0 || set.k >= sl.V ? 0 : set.k;
        Border b = {lo, 0x7FFFFFFF};
        r.token = -1;
        r.mass = 0;
        r.quick = false;
        if (k > 0 && k <= SR_PROBE) {
            const float tau = probe(t, lo, k);
            const uint32_t n = collect(tau, [=](float z, int) { return z >= tau; });
            if (n <= SR_SMALL) {
                if (rank == 0) {
                    const Cut c = small_list(sc, (int)n, k, p, 0, 0, u, r.token);
                    r.b = c.b;
                    r.mass = c.mass;
                }
                fetched();
                return true;
            }
            if (n <= SR_CAP)
                fetched();
            if (n <= SR_CAP && !(p < 1.f)) {
                const Cut c = cut_list(sc, (int)n, k, 0, 0);
                b = c.b;
                r.mass = c.mass;
            } else {
                if (COUNTS)
                    return false;
                b = count_border(t, sc, lo, k, sub);
            }
        } else if (k > 0) {
            if (COUNTS)
                return false;
            b = count_border(t, sc, lo, k, sub);
        }
        if (FAR && COUNTS && p < 1.f)
            return false;
        if (p < 1.f) {
            const bool whole = b.last == 0x7FFFFFFF && b.z == lo;
            const uint64_t about = whole ? quick_mass(sc, b, nullptr, nullptr) : mass(sc, b, nullptr, nullptr);
            // (a share of which more tokens are needed than the list takes, as no token weighs
            // more than 1, or very likely so, is not looked for there)
            uint32_t n = SR_CAP + 1;
            float tau = b.z;
            if (about < (uint64_t)SR_FLAT << SR_ONE) {
                tau = probe(t, b.z, SR_PROBE / 2);
                n = collect(tau, [=](float z, int i) { return z >= tau && kept(b, z, i); });
            }
            if (n <= SR_SMALL) {
                // (all that is kept: its own sum is exact)
                Cut c = {};
                if (rank == 0) {
                    c = small_list(sc, (int)n, (int)n, p, tau <= b.z ? 0 : about, whole ? quick_slack(about) : 0, u, r.token);
                    r.b = c.b;
                    r.mass = c.mass;
                }
                fetched();
                if (exchange(c.ok, 0, 0, 0)[0][0])
                    return true;
                r.token = -1;
            } else if (n <= SR_CAP) {
                fetched();
            }
            if (COUNTS)
                return false;
            const Cut c = mass_border(t, sc, b, p, about, sub);
            b = c.b;
            r.mass = c.mass;
        }
        r.b = b;
        finish(sc, u, k > 0 || p < 1.f, sub, r);
        return true;
    }
    // The border and (or 0) the mass are known: the mass where no token is asked for (FAR: by
    // quick weights, which r.quick tells), or the token. exact: the mass is to be exact
    DDT_DEVINL void finish(const Scale &sc, float u, bool exact, uint64_t *sub, Found &r)
    {
        const Border b = r.b;
        if (u < 0.f) {
            if (r.mass == 0) {
                r.quick = FAR;
                r.mass = FAR ? quick_mass(sc, b, nullptr, nullptr) : mass(sc, b, nullptr, nullptr);
            }
            return;
        }
        const uint64_t(*all)[4];
        if (r.mass > 0 || !exact) {
            // by quick weights; they stand unless the token's ends lie within their error
            const QuickWeight f = {sc, b};
            const uint64_t q = quick_mass(sc, b, sub, &all);
            const uint64_t target = draw_target(u, q), slack = 2 * quick_slack(q);
            uint64_t from = 0, to = 0;
            r.token = locate(sub, all, target, f, &from, &to);
            __syncthreads();
            if (tid == 0)
                sh->found[1] = 0;
            __syncthreads();
            if (r.token >= 0)
                sh->found[1] = (from == 0 || target - from >= slack) && (to == q || to - target > slack);
            __syncthreads();
            const uint64_t(*sure)[4] = exchange(sh->found[1], 0, 0, 0);
            uint64_t any = 0;
            for (uint32_t c = 0; c < cl; ++c)
                any |= sure[c][0];
            if (any) {
                if (r.mass == 0)
                    r.mass = q;
                return;
            }
        }
        r.mass = mass(sc, b, sub, &all);
        const Weight w = {sc, b, sh->tab};
        r.token = locate(sub, all, draw_target(u, r.mass), w);
    }

    struct Weight {  // adds up the kept tokens' weights
        Scale sc;
        Border b;
        const float2 *tab;
        DDT_DEVINL uint64_t sum_to(const float *z, int i0, int last) const
        {
            Sum2 sum = {0, 0};
#pragma unroll
            for (int e = 0; e < E; e += 2)
                add_weights<EXACT>(sc, tab, z[e], z[e + 1], e <= last && kept(b, z[e], i0 + e),
                                   e + 1 <= last && kept(b, z[e + 1], i0 + e + 1), sum);
            return to_fixed(sum);
        }
        DDT_DEVINL uint64_t lane_sum(const float *z, int i0) const { return sum_to(z, i0, E - 1); }
    };
};

// T ln m as a pair of floats (one thread: fp64)
DDT_DEVINL float2 min_offset(const Settings &s)
{
    const double v = (double)s.T * log((double)s.m);
    const float h = (float)v;
    return make_float2(h, (float)(v - (double)h));
}
// the smallest float at or above zmax + T ln m: exp((z - zmax) / T) >= m from there on
DDT_DEVINL float min_value(float zmax, float2 off)
{
    float s = zmax + off.x, bb = s - zmax;
    float e = ((zmax - (s - bb)) + (off.x - bb)) + off.y;
    const float s2 = s + e;
    bb = s2 - s;
    e = (s - (s2 - bb)) + (e - bb);
    return e > 0.f ? nextafterf(s2, SR_MAX_FLOAT) : s2;
}

}  // namespace

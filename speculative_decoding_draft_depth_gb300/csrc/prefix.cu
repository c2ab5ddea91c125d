// prefix.cu -- attention of requests that share prefixes (ddt_prefix_attention and
// ddt_prefix_attention_kvq): the result of prompt attention, each group's prefix read once
// for all its members' rows.
//
// A row's keys are its group's prefix (whole tiles of 128) and what its request holds
// behind it; softmax over both is one merge of (m, l, O) parts, as for any cut of the keys:
//   M = max m_i,  O = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i.
// The prefix is one more item of the tensor-core kernel (prompt_tc.cuh): the group's
// tokens, packed one behind the other, fill its tiles of 256 rows, against keys without a
// mask; its members' items begin behind it. One launch does both, in equal shares, or, where
// requests have few rows, two launches: prefixes there, own keys in a kernel of few rows
// (prefix_few.cu, prompt_few.cu). Items leave their parts in a store by rows, cut ones in the
// CTAs' slots, and prefix_merge_kernel adds each row's up.
#include "prompt_tc.cuh"

namespace {

constexpr int PM_THREADS = 256;

// what one item left of a row: whole (c0 == c1), in the store, or in the slots of CTAs c0..c1
struct RowPart {
    int c0, c1, row;  // row: of the item's tile
};

struct Acc {
    float M, L;
    float4 o;
    DDT_DEVINL void add(float2 ml, const float4 &v)
    {
        const float n = fmaxf(M, ml.x);
        const float f = M == DDT_NEG_INF ? 0.f : ex2(M - n), w = ml.x == DDT_NEG_INF ? 0.f : ex2(ml.x - n);
        L = L * f + ml.y * w;
        o.x = o.x * f + v.x * w;
        o.y = o.y * f + v.y * w;
        o.z = o.z * f + v.z * w;
        o.w = o.w * f + v.w * w;
        M = n;
    }
};

// what was cut: slots of `rows` rows
struct Slots {
    const float *o;
    const float2 *ml;
    int rows;
};
template <int D>
DDT_DEVINL void add_part(const PtArgs &a, const RowPart &p, const Slots &sl, int store, int64_t srow, int c4, Acc &acc)
{
    if (p.c0 == p.c1) {
        acc.add(__ldcg(a.store_ml[store] + srow), __ldcg(a.store_o[store] + (int64_t)c4 * a.T * a.Hq + srow));
        return;
    }
#pragma unroll 4
    for (int c = p.c0; c <= p.c1; ++c) {
        const int64_t slot = 2 * (int64_t)c + (c == p.c0 ? 1 : 0);
        acc.add(__ldcg(&sl.ml[slot * sl.rows + p.row]),
                __ldcg(reinterpret_cast<const float4 *>(sl.o + slot * sl.rows * D) + c4 * sl.rows + p.row));
    }
}

// the units' places in the shares: their first units, and (returned) all units
template <Units U>
DDT_DEVINL long long unit_places(const PtArgs &a, int tq, long long *base, long long *sums)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int count = num_units<U>(a), per = (count + PM_THREADS - 1) / PM_THREADS;
    const int u0 = min(tid * per, count), u1 = min(u0 + per, count);
    long long mine = 0;
    for (int u = u0; u < u1; ++u) {
        base[u] = mine;
        mine += pp_units(load_req<U>(a, u), tq, a.Hkv);
    }
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o)
            incl += y;
    }
    __syncthreads();
    if (lane == 31)
        sums[warp] = incl;
    __syncthreads();
    long long before = incl - mine, total = 0;
    for (int w = 0; w < PM_THREADS / 32; ++w) {
        before += w < warp ? sums[w] : 0;
        total += sums[w];
    }
    for (int u = u0; u < u1; ++u)
        base[u] += before;
    return total;
}

// A CTA: items (request, KV head) by turns. rows: of an item of own keys (PP_ROWS: the same
// launch did both, with `grid` CTAs; else a launch of its own with `own_grid`).
template <int D>
__global__ void __launch_bounds__(PM_THREADS) prefix_merge_kernel(const PtArgs a, int grid, int rows, int own_grid)
{
    extern __shared__ long long s_base[];  // each unit's first share unit: prefixes, then requests
    __shared__ long long s_sums[PM_THREADS / 32];
    __shared__ RowPart s_part[PP_ROWS];    // of each token of an item: the prefix's
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int tp = PP_ROWS >> a.g_shift, tq = rows >> a.g_shift, G = 1 << a.g_shift;
    const bool both = rows == PP_ROWS;
    long long total, own_total;
    if (both) {
        total = own_total = unit_places<BOTH>(a, tp, s_base, s_sums);
    } else {
        total = unit_places<PREFIXES>(a, tp, s_base, s_sums);
        own_total = unit_places<OWN>(a, tq, s_base + a.ngroups, s_sums);
    }
    __syncthreads();
    pdl_wait();  // (every CTA: what comes next in the stream must find the main kernel done)
    if (own_total == 0)
        return;
    const int nc = total > 0 ? pp_ctas(total, grid, MIN_UNITS) : 1;
    const int own_nc = both ? nc : pp_ctas(own_total, own_grid, MIN_UNITS);
    const Slots ps = {a.part_o, a.part_ml, PP_ROWS}, os = {both ? a.part_o : a.few_o, both ? a.part_ml : a.few_ml, rows};
    auto part_of = [&](const PpReq &q, int unit, int t, long long all, int ctas, int qt, int h, int row) {
        const int n = pp_tiles(q, qt, t);
        const long long i0 = s_base[unit] + a.Hkv * pp_units_before(q, qt, t) + (long long)h * (n + PP_ITEM) + PP_ITEM;
        return RowPart{pp_cta_of(i0, all, ctas), pp_cta_of(i0 + n - 1, all, ctas), row};
    };
    for (int x = blockIdx.x; x < a.R * a.Hkv; x += gridDim.x) {
        const int r = x / a.Hkv, h = x - r * a.Hkv;
        const PpReq q = load_req<OWN>(a, r);
        if (q.len == 0)
            continue;
        const int g = q.off > 0 ? group_of(a, r) : 0;
        PpReq pre = {0, 0, 0, 0, 0};
        if (q.off > 0)
            pre = load_group(a, g);
        for (int qt = 0; qt * tq < q.len; ++qt) {
            const int ntok = min(tq, q.len - qt * tq), nrows = ntok << a.g_shift;
            const RowPart own = part_of(q, a.ngroups + r, tq, own_total, own_nc, qt, h, 0);
            if (q.off == 0 && own.c0 == own.c1)
                continue;  // (the kernel before wrote the result)
            if (q.off > 0) {
                __syncthreads();
                for (int t = tid; t < ntok; t += PM_THREADS) {
                    const int i = q.q0 + qt * tq + t - pre.q0;
                    s_part[t] = part_of(pre, g, tp, total, nc, i / tp, h, (i % tp) << a.g_shift);
                }
                __syncthreads();
            }
            // a warp: up to eight rows (side by side in the parts), the rest of its lanes
            // columns of four channels (side by side in the output)
            constexpr int least = D == 128 ? 0 : 1;  // (a row of 64 channels has 16 such columns)
            const int rw = nrows > 1 ? max(least, min(3, 32 - __clz(nrows - 1))) : least, cw = 5 - rw;
            const int blocks = (nrows + (1 << rw) - 1) >> rw, cols = (D / 4) >> cw;
            for (int e = warp; e < blocks * cols; e += PM_THREADS / 32) {
                const int row = ((e / cols) << rw) + (lane & ((1 << rw) - 1)), c4 = ((e % cols) << cw) + (lane >> rw);
                if (row >= nrows)
                    continue;
                const int tok = row >> a.g_shift, hl = row & (G - 1);
                const int64_t t = q.q0 + qt * tq + tok;
                const int64_t srow = (((int64_t)h * a.T + t) << a.g_shift) + hl;
                Acc acc = {DDT_NEG_INF, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
                if (q.off > 0) {
                    RowPart p = s_part[tok];
                    p.row += hl;
                    add_part<D>(a, p, ps, 0, srow, c4, acc);
                }
                add_part<D>(a, RowPart{own.c0, own.c1, row}, os, 1, srow, c4, acc);
                const float inv = acc.L > 0.f || acc.L != acc.L ? a.out_scale / acc.L : 0.f;
                *reinterpret_cast<uint2 *>(a.out + (t * a.Hq + (h << a.g_shift) + hl) * D + 4 * c4) =
                    make_uint2(pack_bf16x2(acc.o.x * inv, acc.o.y * inv), pack_bf16x2(acc.o.z * inv, acc.o.w * inv));
            }
        }
    }
}

template <int D>
cudaError_t launch_merge_rows(const ddt_ctx *c, const PtArgs &a, int grid, int rows, int own_grid, cudaStream_t s)
{
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3((unsigned)std::min((int64_t)a.R * a.Hkv, (int64_t)c->num_sms * 6));
    lc.blockDim = dim3(PM_THREADS);
    lc.dynamicSmemBytes = (size_t)(a.R + a.ngroups) * sizeof(long long);
    lc.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = at;
    lc.numAttrs = 1;
    return cudaLaunchKernelEx(&lc, prefix_merge_kernel<D>, a, grid, rows, own_grid);
}

// few: own keys by a kernel of few rows, this many an item (0: everything in one launch)
template <int D, bool KV4>
cudaError_t launch_d(ddt_ctx *c, int grid, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                     const PtArgs &a, const uint16_t *q, int64_t q_stride, const uint16_t *k_cache, int few, cudaStream_t s)
{
    cudaError_t e;
    int own_grid = grid;
    if (few > 0) {
        e = launch_main<D, KV4, PREFIXES>(c->device, grid, tq, tk, tv, a, s);
        if (e == cudaSuccess)
            e = KV4 ? launch_own_few_kvq(c, a, q, q_stride, few, &own_grid, s)
                    : launch_own_few(c, a, q, q_stride, k_cache, few, &own_grid, s);
    } else {
        e = launch_main<D, KV4, BOTH>(c->device, grid, tq, tk, tv, a, s);
    }
    return e != cudaSuccess ? e : launch_merge_rows<D>(c, a, grid, few > 0 ? few : PP_ROWS, own_grid, s);
}

}  // namespace

cudaError_t launch_prefix_attention(ddt_ctx *c, const uint16_t *q, int64_t q_stride, const int32_t *q_start,
                                    const int32_t *ctx_lens, int R, int T, const uint16_t *k_cache,
                                    const uint16_t *v_cache, const ddt_kv4 *kv4, const int32_t *block_table,
                                    const int32_t *group_start, const int32_t *prefix_lens, int ngroups, uint16_t *out,
                                    cudaStream_t s)
{
    const ddt_config &cfg = c->cfg;
    PtArgs a = make_args(c, q_start, ctx_lens, R, T, v_cache, kv4, block_table, out);
    a.group_start = group_start;
    a.prefix_lens = prefix_lens;
    a.ngroups = ngroups;
    for (int i = 0; i < 2; ++i) {
        a.store_o[i] = reinterpret_cast<float4 *>(c->px_store_o) + (int64_t)i * cfg.prefix_tokens * cfg.Hq * cfg.d / 4;
        a.store_ml[i] = c->px_store_ml + (int64_t)i * cfg.prefix_tokens * cfg.Hq;
    }
    CUtensorMap tq, tk = {}, tv = {};
    if (!make_maps(cfg, q, q_stride, T, k_cache, v_cache, kv4 != nullptr, &tq, &tk, &tv))
        return cudaErrorInvalidValue;
    const int grid = c->num_sms < PR_MAX_CTAS ? c->num_sms : PR_MAX_CTAS;
    a.debug_wait = c->debug_pr_wait;  // one-shot test setting
    c->debug_pr_wait = 0;
    a.few_o = c->px_few_o;
    a.few_ml = c->px_few_ml;
    const int G = cfg.Hq / cfg.Hkv;
    // Few rows of a request on average (lengths are the device's) go to a kernel of their own.
    const int few = (int64_t)T * G > (int64_t)R * 16 ? 0 : G <= 8 && (int64_t)T * G <= (int64_t)R * 8 ? 8 : 16;
    if (kv4)
        return cfg.d == 128 ? launch_d<128, true>(c, grid, tq, tk, tv, a, q, q_stride, nullptr, few, s)
                            : launch_d<64, true>(c, grid, tq, tk, tv, a, q, q_stride, nullptr, few, s);
    return cfg.d == 128 ? launch_d<128, false>(c, grid, tq, tk, tv, a, q, q_stride, k_cache, few, s)
                        : launch_d<64, false>(c, grid, tq, tk, tv, a, q, q_stride, k_cache, few, s);
}

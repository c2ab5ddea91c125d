// prefix.cu -- attention of requests that share prefixes (ddt_prefix_attention and
// ddt_prefix_attention_kvq): the result of prompt attention, each group's prefix read once
// for all its members' rows.
//
// A row's keys are its group's prefix (whole tiles of 128) and what its request holds
// behind it; softmax over both is one merge of (m, l, O) parts, as for any cut of the keys:
//   M = max m_i,  O = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i.
// The prefix is one more item of the tensor-core kernel (prompt_tc.cuh): the group's
// tokens, packed one behind the other, fill its tiles of 256 rows, against keys without a
// mask. Own keys are a launch that begins beside that one, of the same kernel or, where
// requests have few rows, of one for few rows (prefix_few.cu, prompt_few.cu). Items leave
// their parts in a store by rows, cut ones in the CTAs' slots, and prefix_merge_kernel adds
// each row's up.
//
// What bounds it: 64 requests of a token behind 8192 shared keys (32/8 heads of 128) take 60 us
// where the bytes take 25: a tile of the prefix 2 us on its SM, own keys in waves beside and
// behind them, the merge 5 to 10. Prompt attention of the same requests, a prefix each (in
// L2 mostly), takes 210 us.
#include "prompt_tc.cuh"

namespace {

constexpr int PM_THREADS = 256;
constexpr int PM_WARPS = PM_THREADS / 32;
constexpr int PM_AHEAD = 4;  // parts of a row whose loads are in flight

// a row's sum so far: of columns of four channels
struct Acc {
    float M, L;
    float4 o;
    DDT_DEVINL void add(float m, float l, const float4 &v)
    {
        const float n = fmaxf(M, m);
        const float f = M == DDT_NEG_INF ? 0.f : ex2(M - n), w = m == DDT_NEG_INF ? 0.f : ex2(m - n);
        L = L * f + l * w;
        o.x = o.x * f + v.x * w;
        o.y = o.y * f + v.y * w;
        o.z = o.z * f + v.z * w;
        o.w = o.w * f + v.w * w;
        M = n;
    }
};

// add what an item left of a row, of its parts every `by`-th from `from` on. The parts lie in
// slots of `rows` rows, of CTA c0 the second one, of those up to c1 the first ones.
template <int D>
DDT_DEVINL void add_parts(const float *so, const float2 *sml, int rows, int c0, int c1, int row, int c4, int from, int by, Acc &acc)
{
    const int64_t slot = (int64_t)rows * D;
    const float *o = so + (int64_t)c4 * rows * 4 + row * 4;
    for (int c = c0 + from; c <= c1; c += PM_AHEAD * by) {
        float2 ml[PM_AHEAD];
        float4 v[PM_AHEAD];
#pragma unroll
        for (int y = 0; y < PM_AHEAD; ++y) {
            const int x = min(c + y * by, c1), at = 2 * x + (x == c0 ? 1 : 0);
            ml[y] = __ldcg(sml + (int64_t)at * rows + row);
            v[y] = __ldcg(reinterpret_cast<const float4 *>(o + at * slot));
        }
#pragma unroll
        for (int y = 0; y < PM_AHEAD; ++y)
            if (c + y * by <= c1)
                acc.add(ml[y].x, ml[y].y, v[y]);
    }
}

// A CTA: items (request, KV head) by turns. What counts is the parts' way from L2: where an
// item has few rows, several warps share a row's parts.
// (Four CTAs an SM against three: 64 requests of a token 60.4 and 62.9 us a call, over 4 bits
// 59.9 and 62.2; 8 prefixes of chains 193 and 186, 8 tokens 21.8 and 20.9.)
template <int D>
__global__ void __launch_bounds__(PM_THREADS, 4) prefix_merge_kernel(const PtArgs a)
{
    __shared__ Acc s_acc[PM_WARPS][32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int tp = PP_ROWS >> a.g_shift, tq = a.own_rows >> a.g_shift, G = 1 << a.g_shift;
    bool waited = false;
    for (int x = blockIdx.x; x < a.R * a.Hkv; x += gridDim.x) {
        const int r = x / a.Hkv, h = x - r * a.Hkv;
        const PpReq q = load_req<OWN>(a, r);
        PpReq pre = {0, 0, 0, 0, 0};
        if (q.off > 0)
            pre = load_group(a, group_of(a, r));
        if (!waited)  // (every CTA: what comes next in the stream must find the kernels before done)
            pdl_wait();
        waited = true;
        for (int qt = 0; qt * tq < q.len; ++qt) {
            const int ntok = min(tq, q.len - qt * tq), nrows = ntok << a.g_shift, row0 = q.q0 + qt * tq;
            const int2 oc = __ldcg(a.item_ctas[1] + (int64_t)h * a.T + row0);
            // (its tokens lie in two query tiles of the prefix at most: tq <= tp)
            int first_in = 0;
            int2 pcs[2] = {{0, 0}, {0, 0}};
            if (q.off > 0) {
                const int last_in = (row0 + ntok - 1 - pre.q0) % tp;
                first_in = (row0 - pre.q0) % tp;
                pcs[0] = __ldcg(a.item_ctas[0] + (int64_t)h * a.T + row0 - first_in);
                pcs[1] = __ldcg(a.item_ctas[0] + (int64_t)h * a.T + row0 + ntok - 1 - last_in);
            }
            if (q.off == 0 && oc.x == oc.y)
                continue;  // (the kernel before wrote the result)
            // a warp: up to eight rows (side by side in the parts), the rest of its lanes
            // columns of four channels (side by side in the output)
            constexpr int least = D == 128 ? 0 : 1;  // (a row of 64 channels has 16 such columns)
            const int rw = nrows > 1 ? max(least, min(3, 32 - __clz(nrows - 1))) : least, cw = 5 - rw;
            const int cols = (D / 4) >> cw, tasks = ((nrows + (1 << rw) - 1) >> rw) * cols;
            const int by = tasks > PM_WARPS / 2 ? 1 : tasks > PM_WARPS / 4 ? 2 : 4;  // warps to a task
            for (int e0 = 0; e0 < tasks; e0 += PM_WARPS / by) {
                const int e = e0 + warp / by, from = warp % by;
                const int row = ((e / cols) << rw) + (lane & ((1 << rw) - 1)), c4 = ((e % cols) << cw) + (lane >> rw);
                const int tok = row >> a.g_shift, hl = row & (G - 1);
                const int64_t t = row0 + tok, srow = (((int64_t)h * a.T + t) << a.g_shift) + hl;
                Acc acc = {DDT_NEG_INF, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
                if (e < tasks && row < nrows) {
                    auto stored = [&](int i) {
                        const float2 ml = __ldcg(a.store_ml[i] + srow);
                        acc.add(ml.x, ml.y, __ldcg(a.store_o[i] + (int64_t)c4 * a.T * a.Hq + srow));
                    };
                    if (q.off > 0) {
                        const int in = (int)(t - pre.q0) % tp;
                        const int2 pc = pcs[first_in + tok >= tp];
                        if (pc.x != pc.y)
                            add_parts<D>(a.part_o, a.part_ml, PP_ROWS, pc.x, pc.y, (in << a.g_shift) + hl, c4, from, by, acc);
                        else if (from == 0)
                            stored(0);
                    }
                    if (oc.x != oc.y)
                        add_parts<D>(a.own_o, a.own_ml, a.own_rows, oc.x, oc.y, row, c4, from, by, acc);
                    else if (from == by - 1)
                        stored(1);
                }
                if (by > 1) {
                    __syncthreads();  // (of the round before: read)
                    s_acc[warp][lane] = acc;
                    __syncthreads();
                    if (from > 0)
                        continue;
                    for (int w = 1; w < by; ++w)
                        acc.add(s_acc[warp + w][lane].M, s_acc[warp + w][lane].L, s_acc[warp + w][lane].o);
                }
                if (e < tasks && row < nrows) {
                    const float inv = acc.L > 0.f || acc.L != acc.L ? a.out_scale / acc.L : 0.f;
                    *reinterpret_cast<uint2 *>(a.out + (t * a.Hq + (h << a.g_shift) + hl) * D + 4 * c4) =
                        make_uint2(pack_bf16x2(acc.o.x * inv, acc.o.y * inv), pack_bf16x2(acc.o.z * inv, acc.o.w * inv));
                }
            }
        }
    }
    if (!waited)
        pdl_wait();
}

template <int D>
cudaError_t launch_merge_rows(const ddt_ctx *c, const PtArgs &a, cudaStream_t s)
{
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3((unsigned)std::min((int64_t)a.R * a.Hkv, (int64_t)c->num_sms * 6));
    lc.blockDim = dim3(PM_THREADS);
    lc.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = at;
    lc.numAttrs = 1;
    return cudaLaunchKernelEx(&lc, prefix_merge_kernel<D>, a);
}

template <int D, bool KV4>
cudaError_t launch_d(ddt_ctx *c, int grid, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                     const PtArgs &a, const uint16_t *q, int64_t q_stride, const uint16_t *k_cache, cudaStream_t s)
{
    cudaError_t e = launch_main<D, KV4, PREFIXES>(c->device, grid, tq, tk, tv, a, s);
    if (e != cudaSuccess)
        return e;
    if (a.own_rows == PP_ROWS) {
        PtArgs own = a;
        own.part_o = a.own_o;
        own.part_ml = a.own_ml;
        own.debug_wait = 0;
        e = launch_main<D, KV4, OWN>(c->device, grid, tq, tk, tv, own, s);
    } else {
        e = KV4 ? launch_own_few_kvq(c, a, q, q_stride, a.own_rows, s) : launch_own_few(c, a, q, q_stride, k_cache, a.own_rows, s);
    }
    return e != cudaSuccess ? e : launch_merge_rows<D>(c, a, s);
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
    for (int i = 0; i < 2; ++i)
        a.item_ctas[i] = c->px_item_ctas + (int64_t)i * cfg.Hkv * cfg.prefix_tokens;
    a.own_o = c->px_own_o;
    a.own_ml = c->px_own_ml;
    const int G = cfg.Hq / cfg.Hkv;
    // Few rows of a request on average (lengths are the device's) go to a kernel of their own.
    a.own_rows = (int64_t)T * G > (int64_t)R * 16 ? PP_ROWS : G <= 8 && (int64_t)T * G <= (int64_t)R * 8 ? 8 : 16;
    // Measured: a prefix's tile 2 us of an SM (4 bits as well), a unit of own keys 0.9 us, a
    // CTA of the prefixes' 6 us besides.
    if (a.own_rows < PP_ROWS) {
        a.cost[0] = 20;
        a.cost[1] = 9;
        a.cost[2] = 60;
    }
    if (kv4)
        return cfg.d == 128 ? launch_d<128, true>(c, grid, tq, tk, tv, a, q, q_stride, nullptr, s)
                            : launch_d<64, true>(c, grid, tq, tk, tv, a, q, q_stride, nullptr, s);
    return cfg.d == 128 ? launch_d<128, false>(c, grid, tq, tk, tv, a, q, q_stride, k_cache, s)
                        : launch_d<64, false>(c, grid, tq, tk, tv, a, q, q_stride, k_cache, s);
}

// sample.cu -- sampled decoding: a token of each logit row under temperature, top-k,
// top-p and min-p. The mathematics and the work on one row are in sample_row.cuh; a row is
// done by a cluster that holds it, or, where there are many, by a CTA that reads it where
// it lies (sample_solve.cuh).
//
// What bounds it: the row's bytes are little (64 rows of 151936 bf16 logits: 3 us of HBM),
// the chain of decisions on them is long: each exchange between a cluster's CTAs takes 1 us,
// the passes between them 1 to 5 us each. Measured, rows of 151936 bf16 logits, 1 and 64 of
// them: temperature alone 11 and 33 us, greedy 12 and 20, top-k 50 13 and 24, top-p 0.9 36
// and 58 (its counts are 150000 additions in shared memory a row).
#include "sample_solve.cuh"

namespace {

template <typename T>
struct SampleArgs {
    const T *logits;  // [N, V]
    ddt_filter f;
    const float *u;
    int32_t *tokens;
    float *logprobs;  // or null
    int32_t *status;
    int V, subs;      // subs: sub-chunks that a CTA has room for
};

template <typename T>
DDT_DEVINL void store_token(const SampleArgs<T> &a, int64_t n, int token, float logprob)
{
    a.tokens[n] = token;
    if (a.logprobs)
        a.logprobs[n] = logprob;
}

template <typename T, int CL>
__global__ void __launch_bounds__(CL == FAR ? SR_FAR : SR_THREADS, CL == FAR ? FAR_CTAS : 4) sample_kernel(const SampleArgs<T> a)
{
    __shared__ RowShared sh;
    __shared__ BinShared<(CL > 0 ? CL : 1)> bs;
    const int64_t n = blockIdx.x / cl_size();
    const Settings set = load_settings(a.f, (int)n);
    Solved r;
    r.none = !set.good;
    r.token = -1;
    if (set.good) {
        bool here;
        const float u = __ldg(a.u + n);
        const T *z = a.logits + n * a.V;
        whole_row<CL>(&sh, &bs, z, a.V, a.subs, set, u > 0.f ? u : 0.f, a.status, r, here);
        // log of the token's weight over all that is kept (the largest weight is 2^44, so
        // the sum is about that at least)
        if (r.token >= 0) {
            const float over = (float)(int64_t)(r.mass - (1ull << SR_ONE)) * 5.684341886e-14f;
            store_token(a, n, r.token, (held_value(logit_value(z, r.token), r.infinite) - r.sc.zmax) / set.T - log1pf(over));
        }
    }
    if (r.none && cl_rank() == 0 && threadIdx.x == 0) {
        store_token(a, n, -1, DDT_NEG_INF);
        if (!set.good)
            set_status(a.status, DDT_DEV_BAD_SETTING);
    }
}

template <typename T, int CL>
cudaError_t sample_rows_cl(const ddt_ctx *c, const SampleArgs<T> &a, int N, int cl, int smem, cudaStream_t s)
{
    static DeviceFlags ready;
    return launch_rows(sample_kernel<T, CL>, ready, c->device, N, cl, CL == FAR ? SR_FAR : SR_THREADS, smem, false, a, s);
}
template <typename T>
cudaError_t sample_rows(const ddt_ctx *c, const void *logits, int N, const ddt_filter &f, const float *u, int32_t *tokens,
                        float *logprobs, cudaStream_t s)
{
    const int V = c->cfg.V, bins = sizeof(T) == 2 ? bins_cluster(V) : 0;
    if (const int far = far_groups<T>(V, N, c->num_sms)) {
        const SampleArgs<T> a = {(const T *)logits, f, u, tokens, logprobs, c->status, V, (far + 1) / 2 * 2};
        return sample_rows_cl<T, FAR>(c, a, N, 1, far_bytes(far), s);
    }
    const int cl = bins > 0 ? bins : pick_cluster<T>(V, N, c->num_sms, 0);
    const SampleArgs<T> a = {(const T *)logits, f, u, tokens, logprobs, c->status, V, slice_subs<T>(V, cl)};
    const int smem = std::max(slice_bytes<T>(V, cl, 0), bins > 0 ? sb_bytes(cl) : 0);
    if constexpr (sizeof(T) == 2) {
        if (bins == 8)
            return sample_rows_cl<T, 8>(c, a, N, cl, smem, s);
        if (bins == 16)
            return sample_rows_cl<T, 16>(c, a, N, cl, smem, s);
    }
    return sample_rows_cl<T, 0>(c, a, N, cl, smem, s);
}

}  // namespace

cudaError_t launch_sample(const ddt_ctx *c, const void *logits, int dtype, int N, const ddt_filter &f, const float *u,
                          int32_t *tokens, float *logprobs, cudaStream_t s)
{
    return dtype == DDT_BF16 ? sample_rows<uint16_t>(c, logits, N, f, u, tokens, logprobs, s)
                             : sample_rows<float>(c, logits, N, f, u, tokens, logprobs, s);
}

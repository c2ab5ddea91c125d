// prompt.cu -- ddt_prompt_attention and ddt_prompt_attention_kvq: the kernel of few rows
// (prompt_few.cu) or the tensor cores' (prompt_tc.cuh), and the merge of cut items.
#include "prompt_tc.cuh"

namespace {

template <int D, bool KV4>
cudaError_t launch_d(int dev, int grid, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, const PtArgs &a,
                     cudaStream_t s)
{
    const cudaError_t e = launch_main<D, KV4, PLAIN>(dev, grid, tq, tk, tv, a, s);
    return e != cudaSuccess || grid == 1 ? e : launch_merge<D>(a, grid, PP_ROWS, s);
}

}  // namespace

cudaError_t launch_prompt_attention(ddt_ctx *c, const uint16_t *q, int64_t q_stride,
                                    const int32_t *q_start, const int32_t *ctx_lens, int R, int T,
                                    const uint16_t *k_cache, const uint16_t *v_cache,
                                    const ddt_kv4 *kv4, const int32_t *block_table, uint16_t *out,
                                    cudaStream_t s)
{
    const ddt_config &cfg = c->cfg;
    const int G = cfg.Hq / cfg.Hkv;
    PtArgs a = make_args(c, q_start, ctx_lens, R, T, v_cache, kv4, block_table, out);
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
    if (!make_maps(cfg, q, q_stride, T, k_cache, v_cache, kv4 != nullptr, &tq, &tk, &tv))
        return cudaErrorInvalidValue;
    const int grid = c->num_sms < PR_MAX_CTAS ? c->num_sms : PR_MAX_CTAS;
    a.debug_wait = c->debug_pr_wait;  // one-shot test setting
    c->debug_pr_wait = 0;
    if (kv4)
        return cfg.d == 128 ? launch_d<128, true>(c->device, grid, tq, tk, tv, a, s)
                            : launch_d<64, true>(c->device, grid, tq, tk, tv, a, s);
    return cfg.d == 128 ? launch_d<128, false>(c->device, grid, tq, tk, tv, a, s)
                        : launch_d<64, false>(c->device, grid, tq, tk, tv, a, s);
}

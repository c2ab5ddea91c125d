// sample.cu -- sampled decoding: a token of each logit row under temperature, top-k,
// top-p and min-p (sample_kernel), and the probability rule on drafted chains whose
// drafter and target both sample under such settings (keep_kernel, chain_kernel).
// The mathematics and the work on one row are in sample_row.cuh.
//
//  * sample_kernel: one cluster a row: read once, the border of the kept tokens, their
//    weights' running sums, the drawn token.
//  * keep_kernel: one cluster for each draft and target row that a chain verifies: the
//    border, the kept weights' sum and the guess's weight, 32 bytes a row.
//  * chain_kernel (a dependent launch): one cluster a request. Each CTA takes the
//    request's decisions itself, u < (w_p(x) / W_p) / (w_q(x) / W_q), and the cluster draws
//    from max(0, w_p - (W_p / W_q) w_q) over the first rejected row, or from w_p behind the
//    last guess, in 64-bit integers.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "device_flags.h"
#include "sample_bins.cuh"
#include "sample_row.cuh"

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

extern __shared__ __align__(16) unsigned char sr_smem[];

template <typename T>
DDT_DEVINL void store_token(const SampleArgs<T> &a, int64_t n, int token, float logprob)
{
    a.tokens[n] = token;
    if (a.logprobs)
        a.logprobs[n] = logprob;
}

// what became of a row in shared memory
struct Solved {
    Scale sc;
    Border b;
    uint64_t mass;
    int token;
    bool infinite, none;  // none: no token has a weight
};

// a row in place in shared memory (see Row::solve). false: to be counted
template <bool COUNTS, typename T>
DDT_DEVINL bool solve_row(Row<T> &row, const Settings &set, float u, uint64_t *sub, int32_t *status, Solved &r)
{
    typename Row<T>::Top t = row.top();
    if (t.nan && row.rank == 0 && row.tid == 0)
        set_status(status, DDT_DEV_NAN_LOGITS);
    r.none = t.zmax == DDT_NEG_INF;
    r.token = -1;
    if (r.none)
        return true;
    r.infinite = t.zmax == -DDT_NEG_INF;
    if (r.infinite)
        row.only_infinite(t);
    r.sc = make_scale(t.zmax, set.T);
    typename Row<T>::Found f;
    if (!row.template solve<COUNTS>(t, r.sc, set, set.m > 0.f ? min_value(t.zmax, row.sh->off) : DDT_NEG_INF, u, sub, f))
        return false;
    r.b = f.b;
    r.mass = f.mass;
    r.token = f.token;
    return true;
}
// the same for a row that cannot be counted after all (apart, for the registers of the rest)
__device__ __noinline__ void solve_general(Row<uint16_t> row, const uint16_t *z, int V, const Settings &set, float u,
                                           uint64_t *sub, int32_t *status, Solved &r)
{
    __syncthreads();
    row.load(sr_smem, z, V);
    row.loaded();
    solve_row<false>(row, set, u, sub, status, r);
}

// A row from its logits on. CL > 0: the cluster's size, of rows that may be counted. In
// r.token >= 0 the drawn token, in one thread; for u < 0 the border and the mass, in `here`.
template <int CL, typename T>
DDT_DEVINL void whole_row(Row<T> &row, RowShared *sh, BinShared<(CL > 0 ? CL : 1)> *bs, const T *z, int V, int subs,
                          const Settings &set, float u, int32_t *status, Solved &r, bool &here)
{
    uint64_t *sub = reinterpret_cast<uint64_t *>(sr_smem + subs * SR_SUB);
    row.begin(sh);
    row.load(sr_smem, z, V);
    if (row.tid == 0 && set.m > 0.f)
        sh->off = min_offset(set);
    row.loaded();
    row.started();
    here = row.rank == 0 && row.tid == 0;
    if constexpr (CL == 0) {
        solve_row<false>(row, set, u, sub, status, r);
    } else if (!solve_row<true>(row, set, u, sub, status, r)) {
        BinRow<CL> bins(row, bs, sr_smem, z, V);
        typename BinRow<CL>::Kept k;
        if (!bins.run(set, r.sc, k)) {
            Solved g;
            solve_general(row, z, V, set, u, sub, status, g);
            r = g;
            return;
        }
        r.mass = k.mass;
        if (u >= 0.f) {
            r.token = bins.draw(r.sc, k, u, r.b);
            return;
        }
        // the thread that knows the border answers: the last kept index's, or the first
        const bool cut = k.d != SB_VALUES && k.count != k.of;
        const int last = bins.last_kept(k);
        r.b = {k.d == SB_VALUES ? bins.least : sb_value(k.d), cut ? last : 0x7FFFFFFF};
        here = cut ? last >= 0 : here;
        cl_sync();  // (the counts have been read by other CTAs)
    }
}

template <typename T, int CL>
__global__ void __launch_bounds__(SR_THREADS, 4) sample_kernel(const SampleArgs<T> a)
{
    __shared__ RowShared sh;
    __shared__ BinShared<(CL > 0 ? CL : 1)> bs;
    const int64_t n = blockIdx.x / cl_size();
    const Settings set = load_settings(a.f, (int)n);
    Solved r;
    r.none = !set.good;
    r.token = -1;
    if (set.good) {
        Row<T> row;
        bool here;
        const float u = __ldg(a.u + n);
        const T *z = a.logits + n * a.V;
        whole_row<CL>(row, &sh, &bs, z, a.V, a.subs, set, u > 0.f ? u : 0.f, a.status, r, here);
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

// what keep_kernel leaves of a row
struct __align__(16) KeptRow {
    float zmax;
    Border b;
    int flags;
    uint64_t mass, guess;  // the kept weights' sum; the guess's weight (0: not kept)
};
constexpr int KR_BAD = 1, KR_INF = 2;

template <typename T>
struct KeepArgs {
    const T *draft, *target;  // [R, L, V], [R, L + 1, V]; either may be null (then none of its rows is done here)
    ddt_filter fd, ft;
    const int32_t *tokens, *n_guess;
    KeptRow *rows;  // [R, 2 L + 1]
    int32_t *status;
    int L, V, subs;
};

DDT_DEVINL int guess_count(const int32_t *n_guess, int i, int L)
{
    return n_guess ? max(0, min(L, __ldg(n_guess + i))) : L;
}

// which row a cluster has; false: one that is not verified
template <typename T>
struct KeepRow {
    const T *z;
    KeptRow *to;
    Settings set;
    int x;  // the guess, -1: none

    DDT_DEVINL bool find(const KeepArgs<T> &a, int64_t n)
    {
        const int L = a.L, per = (a.draft ? L : 0) + (a.target ? L + 1 : 0);
        const int i = (int)(n / per), j = (int)(n % per);
        const bool isd = a.draft && j < L;
        const int k = isd || !a.draft ? j : j - L;
        const int guesses = guess_count(a.n_guess, i, L);
        if (isd ? k >= guesses : k > guesses)
            return false;
        to = a.rows + (int64_t)i * (2 * L + 1) + (isd ? k : L + k);
        z = isd ? a.draft + ((int64_t)i * L + k) * a.V : a.target + ((int64_t)i * (L + 1) + k) * a.V;
        set = load_settings(isd ? a.fd : a.ft, i);
        x = k < guesses ? __ldg(a.tokens + (int64_t)i * L + k) : -1;
        if (x >= a.V)
            x = -1;
        if (!set.good && cl_rank() == 0 && threadIdx.x == 0)
            *to = KeptRow{0.f, {0.f, 0}, KR_BAD, 0, 0};
        return set.good;
    }
};

template <typename T, int CL>
__global__ void __launch_bounds__(SR_THREADS, 4) keep_kernel(const KeepArgs<T> a)
{
    __shared__ RowShared sh;
    pdl_trigger();
    KeepRow<T> kr;
    if (kr.find(a, blockIdx.x / cl_size())) {
        Row<T> row;
        Solved r;
        bool here;
        whole_row<CL>(row, &sh, (BinShared<(CL > 0 ? CL : 1)> *)nullptr, kr.z, a.V, a.subs, kr.set, -1.f, a.status, r, here);
        if (here) {
            KeptRow k = {0.f, {0.f, 0}, 0, 0, 0};
            if (!r.none) {
                k = {r.sc.zmax, r.b, r.infinite ? KR_INF : 0, r.mass, 0};
                if (kr.x >= 0) {
                    const float v = held_value(logit_value(kr.z, kr.x), r.infinite);
                    if (kept(r.b, v, kr.x))
                        k.guess = weight_of<Row<T>::EXACT>(r.sc, sh.tab, v);
                }
            }
            *kr.to = k;
        }
    }
    pdl_wait();  // (rows of the other type may be done by the launch before; what follows waits for both)
}

template <typename TD, typename TT>
struct ChainArgs {
    const TD *draft;
    const TT *target;
    ddt_filter fd, ft;
    const int32_t *tokens, *n_guess;
    const float *u, *r;
    const KeptRow *rows;
    int32_t *acc_len, *acc_tokens, *status;
    int L, V, subs;
};

// 64 x 64 -> a quotient's product: x * (num / den) in integers, x and the result in units
// of 2^-44; what does not fit becomes the largest number
struct Ratio {
    uint64_t m;  // num / den = m 2^-64 2^e, 2^63 <= m
    int e;
    DDT_DEVINL uint64_t times(uint64_t x) const
    {
        const uint64_t h = __umul64hi(x << 16, m);  // (x < 2^45)
        const int sh = 16 - e;
        if (sh >= 0)
            return sh < 64 ? h >> sh : 0;
        return -sh < 64 && h <= (~0ull >> -sh) ? h << -sh : ~0ull;
    }
};
// (one thread: a quotient of up to 2^64 by long division)
DDT_DEVINL Ratio make_ratio(uint64_t num, uint64_t den)
{
    Ratio r;
    const int a = __clzll(num), b = __clzll(den);
    num <<= a;
    den <<= b;
    r.e = b - a;
    // num / den in (1/2, 2): 2^63 <= m < 2^64
    const bool big = num >= den;
    uint64_t rem = big ? num - den : num, q = big ? 1 : 0;
    for (int k = 0; k < (big ? 63 : 64); ++k) {
        const bool carry = rem >> 63;
        rem <<= 1;
        q <<= 1;
        if (carry || rem >= den) {
            rem -= den;
            q |= 1;
        }
    }
    r.m = q;
    r.e += big ? 1 : 0;
    return r;
}

// weights of the draw: p's, less p's share of q's where there is a q
template <typename TD, typename TT>
struct Leftover {
    static constexpr int E = Vec<TT>::E;
    Scale p, q;
    Border bp, bq;
    const float2 *tab;
    const TD *zq;  // shared memory: element i of q's row is zq[i]
    Ratio ratio;
    bool two, inf_p, inf_q;

    DDT_DEVINL uint64_t sum_to(const float *z, int i0, int last) const
    {
        uint64_t t = 0;
#pragma unroll
        for (int e = 0; e < E; e += 2) {
            const float x0 = held_value(z[e], inf_p), x1 = held_value(z[e + 1], inf_p);
            const bool k0 = e <= last && kept(bp, x0, i0 + e), k1 = e + 1 <= last && kept(bp, x1, i0 + e + 1);
            if (!(k0 || k1))
                continue;
            uint64_t w0, w1;
            fixed_pair<Vec<TT>::EXACT>(p, tab, x0, x1, k0, k1, w0, w1);
            if (two) {
                // (a kept index lies within the row, and so within q's part)
                const float y0 = k0 ? held_value(value(i0 + e), inf_q) : 0.f, y1 = k1 ? held_value(value(i0 + e + 1), inf_q) : 0.f;
                const bool j0 = k0 && kept(bq, y0, i0 + e), j1 = k1 && kept(bq, y1, i0 + e + 1);
                if (j0 || j1) {
                    uint64_t v0, v1;
                    fixed_pair<Vec<TD>::EXACT>(q, tab, y0, y1, j0, j1, v0, v1);
                    v0 = ratio.times(v0);
                    v1 = ratio.times(v1);
                    w0 = w0 > v0 ? w0 - v0 : 0;
                    w1 = w1 > v1 ? w1 - v1 : 0;
                }
            }
            t += w0 + w1;
        }
        return t;
    }
    DDT_DEVINL uint64_t lane_sum(const float *z, int i0) const { return sum_to(z, i0, E - 1); }
    DDT_DEVINL float value(int i) const
    {
        if constexpr (sizeof(TD) == 2)
            return bf16_to_f32(zq[i]);
        else
            return zq[i];
    }
};

// Start this thread's copies of elements [lo, hi) of a row of V (whole 16-byte vectors
// around them, within the tensor); returns where element 0 of the row would lie.
template <typename T>
DDT_DEVINL const T *fetch_range(unsigned char *smem, const T *row, int V, int lo, int hi, int tid)
{
    constexpr int E = Vec<T>::E;
    const int skip = (int)(((uintptr_t)(row + lo) & 15) / sizeof(T));
    const T *from = row + lo - skip;
    const uint32_t dst = (uint32_t)__cvta_generic_to_shared(smem);
    for (int v = tid; v * E < hi - lo + skip; v += SR_THREADS) {
        if (lo - skip + (v + 1) * E <= V) {
            cp16(dst + v * 16, from + v * E);
        } else {
            T *d = reinterpret_cast<T *>(smem + v * 16);
            for (int e = 0; e < E && lo - skip + v * E + e < V; ++e)
                d[e] = from[v * E + e];
        }
    }
    return reinterpret_cast<const T *>(smem) + skip - lo;
}

template <typename TD, typename TT>
__global__ void __launch_bounds__(SR_THREADS) chain_kernel(const ChainArgs<TD, TT> a)
{
    __shared__ RowShared sh;
    __shared__ Ratio s_ratio;
    __shared__ int s_first, s_bad;
    Row<TT> row;
    row.begin(&sh);
    const int L = a.L, V = a.V, i = blockIdx.x / row.cl, lane = row.lane;
    const int n = guess_count(a.n_guess, i, L);
    const bool writer = row.rank == 0;
    pdl_wait();  // the kept rows come from keep_kernel
    const KeptRow *rows = a.rows + (int64_t)i * (2 * L + 1);
    if (row.warp == 0) {
        if (writer && lane == 0 && a.n_guess && n != a.n_guess[i])
            set_status(a.status, DDT_DEV_BAD_TREE);
        bool keep = false, bad = false;
        if (lane <= n)
            bad = rows[L + lane].flags & KR_BAD;
        if (lane < n) {
            const KeptRow q = rows[lane], p = rows[L + lane];
            bad |= (q.flags & KR_BAD) != 0;
            const int x = a.tokens[(int64_t)i * L + lane];
            const bool in = x >= 0 && x < V;
            if (!in && writer)
                set_status(a.status, DDT_DEV_BAD_TREE);
            // (q(x) = 0 counts as a ratio of 1)
            double ratio = 1.0;
            if (q.guess > 0)
                ratio = fmin(1.0, p.mass > 0 ? ((double)p.guess * (double)q.mass) / ((double)p.mass * (double)q.guess) : 0.0);
            keep = in && (double)a.u[(int64_t)i * L + lane] < ratio;
        }
        bad = __any_sync(0xFFFFFFFFu, bad);
        const uint32_t kept_ = __ballot_sync(0xFFFFFFFFu, keep && !bad);
        const int first = __ffs(~kept_) - 1;  // (lanes from n on keep nothing)
        if (lane == 0) {
            s_first = first;
            s_bad = bad;
            if (first < n && !bad) {
                const uint64_t mp = rows[L + first].mass, mq = rows[first].mass;
                if (mp > 0 && mq > 0)
                    s_ratio = make_ratio(mp, mq);
            }
        }
        if (writer) {
            if (lane == 0)
                a.acc_len[i] = first + 1;
            if (bad && lane == 0)
                set_status(a.status, DDT_DEV_BAD_SETTING);
            for (int t = lane; t <= L; t += 32)
                if (t != first)
                    a.acc_tokens[(int64_t)i * (L + 1) + t] = t < first ? a.tokens[(int64_t)i * L + t] : -1;
        }
    }
    __syncthreads();
    const int first = s_first;
    int32_t *to = a.acc_tokens + (int64_t)i * (L + 1) + first;
    const KeptRow kp = rows[L + first];
    Leftover<TD, TT> f;
    f.two = first < n && rows[first].mass > 0;
    if (s_bad || kp.mass == 0) {
        row.started();
        if (writer && row.tid == 0)
            *to = -1;
        return;
    }
    uint64_t *sub = reinterpret_cast<uint64_t *>(sr_smem + a.subs * SR_SUB);
    unsigned char *smem_q = reinterpret_cast<unsigned char *>(sub + a.subs + (a.subs & 1));
    row.load(sr_smem, a.target + ((int64_t)i * (L + 1) + first) * V, V);
    f.p = make_scale(kp.zmax, load_settings(a.ft, i).T);
    f.bp = kp.b;
    f.inf_p = kp.flags & KR_INF;
    f.tab = sh.tab;
    if (f.two) {
        const KeptRow kq = rows[first];
        f.q = make_scale(kq.zmax, load_settings(a.fd, i).T);
        f.bq = kq.b;
        f.inf_q = kq.flags & KR_INF;
        f.ratio = s_ratio;
        const int lo = max(0, row.sl.index0(0, 0)), hi = min(V, row.sl.index0(row.sl.ns, 0));
        f.zq = fetch_range(smem_q, a.draft + ((int64_t)i * L + first) * V, V, lo, hi, row.tid);
    }
    row.loaded();
    row.started();
    const uint64_t(*all)[4];
    const uint64_t mass = row.total(f, sub, &all);
    if (mass == 0) {
        if (writer && row.tid == 0)
            *to = -1;
        return;
    }
    const int token = row.locate(sub, all, draw_target(__ldg(a.r + i), mass), f);
    if (token >= 0)
        *to = token;
}

// ------------------------------------------------------------------ host side
constexpr int SR_SMEM_MAX = 227 * 1024 - (int)sizeof(RowShared) - (int)sizeof(BinShared<SR_MAX_CL>) - 256;

// Bytes of shared memory of a CTA that holds a slice of a row of V: the slice, its sub-
// chunks' sums, and (bytes_q > 0) as many elements of another row of that element size.
template <typename T>
int slice_bytes(int V, int cl, int bytes_q)
{
    const int subs = slice_subs<T>(V, cl);
    const int q = bytes_q ? (subs * (SR_SUB / (int)sizeof(T)) * bytes_q + 32) : 0;
    return subs * SR_SUB + (subs + (subs & 1)) * 8 + (q + 15) / 16 * 16;
}

// CTAs of a row's cluster
template <typename T>
int pick_cluster(int V, int64_t rows, int num_sms, int bytes_q)
{
    const int subs = row_subs<T>(V);
    int cl = 1;
    // as many as leave two sub-chunks a warp
    while (cl < 8 && subs >= 2 * cl * 2 * SR_WARPS)
        cl *= 2;
    while (cl < SR_MAX_CL && slice_bytes<T>(V, cl, bytes_q) > SR_SMEM_MAX)
        cl *= 2;
    return cl;
}

// Rows of bf16 logits from this length on may be counted by their values: their cluster has
// eight CTAs, sixteen where a slice's counts would pass 16 bits (0: not even then).
constexpr int SB_LEAST = 8192;
int bins_cluster(int V)
{
    if (V < SB_LEAST)
        return 0;
    for (int cl = 8; cl <= SR_MAX_CL; cl *= 2)
        if ((V + 14) / 8 / cl * 8 + 8 <= 65535 && slice_bytes<uint16_t>(V, cl, 0) <= SR_SMEM_MAX)
            return cl;
    return 0;
}

template <typename Args>
cudaError_t launch_rows(void (*kernel)(Args), DeviceFlags &ready, int dev, int64_t rows, int cl, int smem, bool dependent,
                        const Args &args, cudaStream_t s)
{
    if (rows * cl > 0x7FFFFFFF)
        return cudaErrorInvalidConfiguration;
    if (!ready.test(dev)) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SR_SMEM_MAX);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess)
            return e;
        ready.set(dev);
    }
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = cl;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3((unsigned)(rows * cl));
    lc.blockDim = dim3(SR_THREADS);
    lc.dynamicSmemBytes = smem;
    lc.stream = s;
    lc.attrs = at;
    lc.numAttrs = dependent ? 2 : 1;
    return cudaLaunchKernelEx(&lc, kernel, args);
}

template <typename T, int CL>
cudaError_t sample_rows_cl(const ddt_ctx *c, const SampleArgs<T> &a, int N, int cl, int smem, cudaStream_t s)
{
    static DeviceFlags ready;
    return launch_rows(sample_kernel<T, CL>, ready, c->device, N, cl, smem, false, a, s);
}
template <typename T>
cudaError_t sample_rows(const ddt_ctx *c, const void *logits, int N, const ddt_filter &f, const float *u, int32_t *tokens,
                        float *logprobs, cudaStream_t s)
{
    const int V = c->cfg.V, bins = sizeof(T) == 2 ? bins_cluster(V) : 0;
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

template <typename T, int CL>
cudaError_t keep_rows_cl(const ddt_ctx *c, const KeepArgs<T> &a, int64_t rows, int cl, int smem, bool dependent, cudaStream_t s)
{
    static DeviceFlags ready;
    return launch_rows(keep_kernel<T, CL>, ready, c->device, rows, cl, smem, dependent, a, s);
}
template <typename T>
cudaError_t keep_rows(const ddt_ctx *c, const void *draft, const void *target, const ddt_filter &fd, const ddt_filter &ft,
                      const int32_t *tokens, const int32_t *n_guess, int R, bool dependent, cudaStream_t s)
{
    const int V = c->cfg.V, L = c->cfg.L, bins = sizeof(T) == 2 ? bins_cluster(V) : 0;
    const int64_t rows = (int64_t)R * ((draft ? L : 0) + (target ? L + 1 : 0));
    const int cl = bins > 0 ? bins : pick_cluster<T>(V, rows, c->num_sms, 0);
    const KeepArgs<T> a = {(const T *)draft, (const T *)target, fd, ft, tokens, n_guess, (KeptRow *)c->sm_rows,
                           c->status, L, V, slice_subs<T>(V, cl)};
    const int smem = std::max(slice_bytes<T>(V, cl, 0), bins > 0 ? sb_bytes(cl) : 0);
    if constexpr (sizeof(T) == 2) {
        if (bins == 8)
            return keep_rows_cl<T, 8>(c, a, rows, cl, smem, dependent, s);
        if (bins == 16)
            return keep_rows_cl<T, 16>(c, a, rows, cl, smem, dependent, s);
    }
    return keep_rows_cl<T, 0>(c, a, rows, cl, smem, dependent, s);
}

template <typename TD, typename TT>
cudaError_t chains(const ddt_ctx *c, const void *draft, const void *target, const ddt_filter &fd, const ddt_filter &ft,
                   const int32_t *tokens, const float *u, const float *r, int R, const int32_t *n_guess, int32_t *acc_len,
                   int32_t *acc_tokens, cudaStream_t s)
{
    static DeviceFlags ready;
    cudaError_t e;
    if constexpr (sizeof(TD) == sizeof(TT)) {
        e = keep_rows<TT>(c, draft, target, fd, ft, tokens, n_guess, R, false, s);
    } else {
        e = keep_rows<TD>(c, draft, nullptr, fd, ft, tokens, n_guess, R, false, s);
        if (e == cudaSuccess)
            e = keep_rows<TT>(c, nullptr, target, fd, ft, tokens, n_guess, R, true, s);
    }
    if (e != cudaSuccess)
        return e;
    const int V = c->cfg.V, cl = pick_cluster<TT>(V, R, c->num_sms, sizeof(TD));
    const ChainArgs<TD, TT> a = {(const TD *)draft, (const TT *)target, fd, ft, tokens, n_guess, u, r,
                                 (const KeptRow *)c->sm_rows, acc_len, acc_tokens, c->status, c->cfg.L, V,
                                 slice_subs<TT>(V, cl)};
    return launch_rows(chain_kernel<TD, TT>, ready, c->device, R, cl, slice_bytes<TT>(V, cl, sizeof(TD)), true, a, s);
}

}  // namespace

size_t sample_row_bytes() { return sizeof(KeptRow); }

cudaError_t launch_sample(const ddt_ctx *c, const void *logits, int dtype, int N, const ddt_filter &f, const float *u,
                          int32_t *tokens, float *logprobs, cudaStream_t s)
{
    return dtype == DDT_BF16 ? sample_rows<uint16_t>(c, logits, N, f, u, tokens, logprobs, s)
                             : sample_rows<float>(c, logits, N, f, u, tokens, logprobs, s);
}

cudaError_t launch_accept_sampled(const ddt_ctx *c, const void *draft, const void *target, const ddt_filter &fd,
                                  const ddt_filter &ft, const int32_t *tokens, const float *u, const float *r, int R,
                                  const int32_t *n_guess, int32_t *acc_len, int32_t *acc_tokens, cudaStream_t s)
{
    const bool bd = c->cfg.draft_dtype == DDT_BF16, bt = c->cfg.target_dtype == DDT_BF16;
    if (bd && bt)
        return chains<uint16_t, uint16_t>(c, draft, target, fd, ft, tokens, u, r, R, n_guess, acc_len, acc_tokens, s);
    if (bd)
        return chains<uint16_t, float>(c, draft, target, fd, ft, tokens, u, r, R, n_guess, acc_len, acc_tokens, s);
    if (bt)
        return chains<float, uint16_t>(c, draft, target, fd, ft, tokens, u, r, R, n_guess, acc_len, acc_tokens, s);
    return chains<float, float>(c, draft, target, fd, ft, tokens, u, r, R, n_guess, acc_len, acc_tokens, s);
}

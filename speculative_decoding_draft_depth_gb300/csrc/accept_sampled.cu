// accept_sampled.cu -- the probability rule on drafted chains whose drafter and target both
// sample under temperature, top-k, top-p and min-p.
//
//  * keep_kernel: each draft and target row that a chain verifies: the border of what its
//    settings keep, the kept weights' sum and the guess's weight, 32 bytes a row. Rows enough
//    to have a CTA each may leave a quick sum (off by less than 2^-20 of itself).
//  * chain_kernel (a dependent launch): one cluster a request. Each CTA takes the request's
//    decisions itself, u < (w_p(x) / W_p) / (w_q(x) / W_q); one that lies within the error of
//    quick sums is taken again with exact ones. The cluster then draws from max(0, w_p -
//    (W_p / W_q) w_q) over the first rejected row, or from w_p behind the last guess, in
//    64-bit integers.
//
// What bounds it, for many rows: two reads of each row, the second of which hits L2 for a
// quarter (greedy: 220 us for 1984 rows of 151936 bf16 logits, 5.5 TB/s from HBM); under
// top-p the instructions (40 a logit: 580 us); the draws from what is left, 50 to 180 us of
// pairs of weights. For one chain of 15 guesses, the exchanges: 27 to 70 us.
#include "sample_solve.cuh"

namespace {

// what keep_kernel leaves of a row
struct __align__(16) KeptRow {
    float zmax;
    Border b;
    int flags;
    uint64_t mass, guess;  // the kept weights' sum; the guess's weight (0: not kept)
};
constexpr int KR_BAD = 1, KR_INF = 2, KR_QUICK = 4;  // KR_QUICK: the sum is by quick weights

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
__global__ void __launch_bounds__(CL == FAR ? SR_FAR : SR_THREADS, CL == FAR ? FAR_CTAS : 4) keep_kernel(const KeepArgs<T> a)
{
    __shared__ RowShared sh;
    pdl_trigger();
    KeepRow<T> kr;
    if (kr.find(a, blockIdx.x / cl_size())) {
        Solved r;
        bool here;
        whole_row<CL>(&sh, (BinShared<(CL > 0 ? CL : 1)> *)nullptr, kr.z, a.V, a.subs, kr.set, -1.f, a.status, r, here);
        if (here) {
            KeptRow k = {0.f, {0.f, 0}, 0, 0, 0};
            if (!r.none) {
                k = {r.sc.zmax, r.b, (r.infinite ? KR_INF : 0) | (r.quick ? KR_QUICK : 0), r.mass, 0};
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
    // both rows' kept weights, exactly
    DDT_DEVINL void sums(Row<TT> &row, uint64_t &mp, uint64_t &mq) const
    {
        uint64_t sp = 0, sq = 0;
        row.each([&](int s, const uint4 &v) {
            float z[E];
            row.sl.values(v, z);
            const int i0 = row.sl.index0(s, row.lane);
            Sum2 wp = {0, 0}, wq = {0, 0};
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const float x0 = held_value(z[e], inf_p), x1 = held_value(z[e + 1], inf_p);
                add_weights<Vec<TT>::EXACT>(p, tab, x0, x1, kept(bp, x0, i0 + e), kept(bp, x1, i0 + e + 1), wp);
                const int j0 = i0 + e, j1 = i0 + e + 1;
                const bool in0 = j0 >= 0 && j0 < row.sl.V, in1 = j1 >= 0 && j1 < row.sl.V;
                const float y0 = in0 ? held_value(value(j0), inf_q) : 0.f, y1 = in1 ? held_value(value(j1), inf_q) : 0.f;
                add_weights<Vec<TD>::EXACT>(q, tab, y0, y1, in0 && kept(bq, y0, j0), in1 && kept(bq, y1, j1), wq);
            }
            sp += to_fixed(wp);
            sq += to_fixed(wq);
        });
        sp = row.block_sum(sp);
        sq = row.block_sum(sq);
        const uint64_t(*all)[4] = row.exchange(sp, sq, 0, 0);
        mp = mq = 0;
        for (uint32_t c = 0; c < row.cl; ++c) {
            mp += all[c][0];
            mq += all[c][1];
        }
    }
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
__global__ void __launch_bounds__(SR_THREADS, 4) chain_kernel(const ChainArgs<TD, TT> a)
{
    __shared__ RowShared sh;
    __shared__ Ratio s_ratio;
    __shared__ int s_first, s_bad, s_doubt;
    Row<TT> row;
    row.begin(&sh);
    const int L = a.L, V = a.V, i = blockIdx.x / row.cl, lane = row.lane;
    const int n = guess_count(a.n_guess, i, L);
    const bool writer = row.rank == 0;
    pdl_wait();  // the kept rows come from keep_kernel
    const KeptRow *rows = a.rows + (int64_t)i * (2 * L + 1);
    uint64_t *sub = reinterpret_cast<uint64_t *>(sr_smem + a.subs * SR_SUB);
    unsigned char *smem_q = reinterpret_cast<unsigned char *>(sub + a.subs + (a.subs & 1));
    int held = -1;     // whose rows this CTA holds, and their exact sums
    int settled = -1;  // a lane's guess: 0 or 1 once its exact sums have decided it
    uint64_t mp = 0, mq = 0;
    Leftover<TD, TT> f;
    f.tab = sh.tab;
    // (each turn but the last settles one more guess: L turns and one at most)
    for (;;) {
        if (row.warp == 0) {
            bool keep = false, bad = false, doubt = false;
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
                const double u = (double)a.u[(int64_t)i * L + lane];
                const double wp = (double)(lane == held ? mp : p.mass), wq = (double)(lane == held ? mq : q.mass);
                double ratio = 1.0;
                if (q.guess > 0)
                    ratio = p.mass > 0 ? ((double)p.guess * wq) / (wp * (double)q.guess) : 0.0;
                keep = settled >= 0 ? settled == 1 : in && u < fmin(1.0, ratio);
                if (lane == held)
                    settled = keep;
                // (a ratio of two quick sums is off by less than 2^-18 of itself)
                doubt = in && settled < 0 && p.mass > 0 && q.guess > 0 && ((q.flags | p.flags) & KR_QUICK) &&
                        fabs(u - ratio) <= ratio * 3.8147e-6;
            }
            bad = __any_sync(0xFFFFFFFFu, bad);
            const uint32_t kept_ = __ballot_sync(0xFFFFFFFFu, keep && !bad);
            const uint32_t doubts = __ballot_sync(0xFFFFFFFFu, doubt && !bad);
            if (lane == 0) {
                const int first = __ffs(~kept_) - 1;  // (lanes from n on keep nothing)
                s_first = first;
                s_bad = bad;
                s_doubt = doubts != 0 && __ffs(doubts) - 1 <= first ? __ffs(doubts) - 1 : -1;
            }
        }
        __syncthreads();
        const int first = s_doubt >= 0 ? s_doubt : s_first;
        const KeptRow kp = rows[L + first];
        f.two = first < n && rows[first].mass > 0;
        if (s_bad || kp.mass == 0)
            break;
        if (held != first) {
            if (held >= 0)
                __syncthreads();  // (the rows before have been read)
            held = first;
            mp = kp.mass;
            row.load(sr_smem, a.target + ((int64_t)i * (L + 1) + first) * V, V);
            f.p = make_scale(kp.zmax, load_settings(a.ft, i).T);
            f.bp = kp.b;
            f.inf_p = kp.flags & KR_INF;
            bool quick = false;
            if (f.two) {
                const KeptRow kq = rows[first];
                mq = kq.mass;
                f.q = make_scale(kq.zmax, load_settings(a.fd, i).T);
                f.bq = kq.b;
                f.inf_q = kq.flags & KR_INF;
                const int lo = max(0, row.sl.index0(0, 0)), hi = min(V, row.sl.index0(row.sl.ns, 0));
                f.zq = fetch_range(smem_q, a.draft + ((int64_t)i * L + first) * V, V, lo, hi, row.tid);
                quick = (kp.flags | kq.flags) & KR_QUICK;
            }
            row.loaded();
            if (row.turn == 0)
                row.started();
            if (quick)
                f.sums(row, mp, mq);
        }
        if (s_doubt < 0)
            break;
        __syncthreads();  // (what has been decided has been read)
    }
    if (row.turn == 0 && held < 0)
        row.started();
    const int first = s_first;
    if (writer && row.warp == 0) {
        if (lane == 0)
            a.acc_len[i] = first + 1;
        if (lane == 0 && a.n_guess && n != a.n_guess[i])
            set_status(a.status, DDT_DEV_BAD_TREE);
        if (lane == 0 && s_bad)
            set_status(a.status, DDT_DEV_BAD_SETTING);
        for (int t = lane; t <= L; t += 32)
            if (t != first)
                a.acc_tokens[(int64_t)i * (L + 1) + t] = t < first ? a.tokens[(int64_t)i * L + t] : -1;
    }
    int32_t *to = a.acc_tokens + (int64_t)i * (L + 1) + first;
    if (s_bad || rows[L + first].mass == 0) {
        if (writer && row.tid == 0)
            *to = -1;
        return;
    }
    if (f.two) {
        if (row.tid == 0)
            s_ratio = make_ratio(mp, mq);
        __syncthreads();
        f.ratio = s_ratio;
    }
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

template <typename T, int CL>
cudaError_t keep_rows_cl(const ddt_ctx *c, const KeepArgs<T> &a, int64_t rows, int cl, int smem, bool dependent, cudaStream_t s)
{
    static DeviceFlags ready;
    return launch_rows(keep_kernel<T, CL>, ready, c->device, rows, cl, CL == FAR ? SR_FAR : SR_THREADS, smem, dependent, a, s);
}
template <typename T>
cudaError_t keep_rows(const ddt_ctx *c, const void *draft, const void *target, const ddt_filter &fd, const ddt_filter &ft,
                      const int32_t *tokens, const int32_t *n_guess, int R, bool dependent, cudaStream_t s)
{
    const int V = c->cfg.V, L = c->cfg.L, bins = sizeof(T) == 2 ? bins_cluster(V) : 0;
    const int64_t rows = (int64_t)R * ((draft ? L : 0) + (target ? L + 1 : 0));
    if (const int far = far_groups<T>(V, rows, c->num_sms)) {
        const KeepArgs<T> a = {(const T *)draft, (const T *)target, fd, ft, tokens, n_guess, (KeptRow *)c->sm_rows,
                               c->status, L, V, (far + 1) / 2 * 2};
        return keep_rows_cl<T, FAR>(c, a, rows, 1, far_bytes(far), dependent, s);
    }
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
    return launch_rows(chain_kernel<TD, TT>, ready, c->device, R, cl, SR_THREADS, slice_bytes<TT>(V, cl, sizeof(TD)), true, a, s);
}

}  // namespace

size_t sample_row_bytes() { return sizeof(KeptRow); }

// chain_kernel holds a row of both
bool accept_sampled_fits(const ddt_config &c)
{
    const int q = c.draft_dtype == DDT_BF16 ? 2 : 4;
    return (c.target_dtype == DDT_BF16 ? slice_bytes<uint16_t>(c.V, SR_MAX_CL, q) : slice_bytes<float>(c.V, SR_MAX_CL, q)) <=
           SR_SMEM_MAX;
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

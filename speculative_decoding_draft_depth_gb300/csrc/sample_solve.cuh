// sample_solve.cuh -- what the settings keep of a row and the token drawn, by one of three
// ways of going about the row (whole_row), and the launches of kernels over rows.
//
//  * A cluster holds the row in shared memory (sample_row.cuh): few rows, where what counts
//    is how soon one is done.
//  * The same, and bf16 rows that need it are counted by their values (sample_bins.cuh).
//  * Rows enough to fill every SM twice have a CTA each, which reads the row from global
//    memory in each pass: no exchange between CTAs (2000 cycles each), and nothing waits for
//    a cluster's place. 1984 rows of 151936 bf16 logits, greedy: 220 us against 450; under
//    the mixed settings of 64 chains 400 against 763. 256 rows of 100003 fp32 logits take 112
//    against 91, as the last rows are alone on their SMs.
#pragma once

#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "device_flags.h"
#include "sample_bins.cuh"
#include "sample_row.cuh"

namespace {

extern __shared__ __align__(16) unsigned char sr_smem[];

// Rows of bf16 logits from this length on may be counted by their values. (64 rows under top-p
// 0.9, with counts and without: of 32768 tokens 42 and 64 us, of 16384 43 and 46, of 4096 43 and
// 41; under top-k 50, whose rows then take the cluster of eight too, 20 and 19, 19 and 12, 20
// and 10)
constexpr int SB_LEAST = 24576;

// what became of a row
struct Solved {
    Scale sc;
    Border b;
    uint64_t mass;
    float low;  // the least logit
    int token;
    bool infinite, none;  // none: no token has a weight
    bool quick;           // the mass is by quick weights
};

// a row in place in shared memory (see Row::solve). false: to be counted
template <bool COUNTS, typename T, bool FAR>
DDT_DEVINL bool solve_row(Row<T, FAR> &row, const Settings &set, float u, uint64_t *sub, int32_t *status, Solved &r)
{
    typename Row<T, FAR>::Top t = row.top();
    if (t.nan && row.rank == 0 && row.tid == 0)
        set_status(status, DDT_DEV_NAN_LOGITS);
    r.none = t.zmax == DDT_NEG_INF;
    r.quick = false;
    r.token = -1;
    if (r.none)
        return true;
    r.infinite = t.zmax == -DDT_NEG_INF;
    if (r.infinite)
        row.only_infinite(t);
    r.sc = make_scale(t.zmax, set.T);
    typename Row<T, FAR>::Found f;
    if (!row.template solve<COUNTS>(t, r.sc, set, set.m > 0.f ? min_value(t.zmax, row.sh->off) : DDT_NEG_INF, u, sub, f)) {
        r.low = t.low;
        return false;
    }
    r.b = f.b;
    r.mass = f.mass;
    r.token = f.token;
    r.quick = f.quick;
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
__device__ __noinline__ void solve_general(Row<uint16_t, true> row, const Settings &set, float u, uint64_t *sub,
                                           int32_t *status, Solved &r)
{
    solve_row<false>(row, set, u, sub, status, r);
}

// The same by one CTA that reads the row from where it lies. subs: its groups
template <typename T>
DDT_DEVINL void far_row(RowShared *sh, const T *z, int V, int subs, const Settings &set, float u, int32_t *status, Solved &r,
                        bool &here)
{
    Row<T, true> row;
    uint64_t *sub = reinterpret_cast<uint64_t *>(sr_smem);
    row.begin(sh);
    row.load(nullptr, z, V);
    if (row.tid == 0 && set.m > 0.f)
        sh->off = min_offset(set);
    row.loaded();
    here = row.tid == 0;
    if constexpr (sizeof(T) == 2) {
        if (V < SB_LEAST) {
            solve_general(row, set, u, sub, status, r);
        } else if (!solve_row<true>(row, set, u, sub, status, r)) {
            __syncthreads();
            FarBins bins = {row, r.sc, reinterpret_cast<uint32_t *>(sub + subs)};
            Kept k;
            if (!bins.solve(set, r.low, k)) {
                solve_general(row, set, u, sub, status, r);
                return;
            }
            typename Row<T, true>::Found f = {bins.border(k, sub), k.mass, -1, false};
            row.finish(r.sc, u, true, sub, f);
            r.b = f.b;
            r.mass = f.mass;
            r.token = f.token;
        }
    } else {
        solve_row<false>(row, set, u, sub, status, r);
    }
}

// A row from its logits on. CL > 0: the cluster's size, of rows that may be counted; FAR: one
// CTA. In r.token >= 0 the drawn token, in one thread; for u < 0 the border and the mass, in
// `here`.
constexpr int FAR = -1, FAR_CTAS = 2;
template <int CL, typename T>
DDT_DEVINL void whole_row(RowShared *sh, BinShared<(CL > 0 ? CL : 1)> *bs, const T *z, int V, int subs, const Settings &set,
                          float u, int32_t *status, Solved &r, bool &here)
{
    if constexpr (CL == FAR) {
        far_row(sh, z, V, subs, set, u, status, r, here);
        return;
    }
    Row<T> row;
    uint64_t *sub = reinterpret_cast<uint64_t *>(sr_smem + subs * SR_SUB);
    row.begin(sh);
    row.load(sr_smem, z, V);
    if (row.tid == 0 && set.m > 0.f)
        sh->off = min_offset(set);
    row.loaded();
    row.started();
    here = row.rank == 0 && row.tid == 0;
    if constexpr (CL <= 0) {
        solve_row<false>(row, set, u, sub, status, r);
    } else if (!solve_row<true>(row, set, u, sub, status, r)) {
        BinRow<CL> bins(row, bs, sr_smem, z, V);
        Kept k;
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
    // as many as leave two sub-chunks a warp (with another row beside it up to 16: 64 chains of
    // 15 guesses over 151936 take 400 us so, 427 with eight; alone 33, 36)
    while (cl < (bytes_q ? SR_MAX_CL : 8) && subs >= 2 * cl * 2 * SR_WARPS)
        cl *= 2;
    while (cl < SR_MAX_CL && slice_bytes<T>(V, cl, bytes_q) > SR_SMEM_MAX)
        cl *= 2;
    return cl;
}

// The cluster of bf16 rows that may be counted: eight CTAs, sixteen where a slice's counts
// would pass 16 bits (0: not even then).
int bins_cluster(int V)
{
    if (V < SB_LEAST)
        return 0;
    for (int cl = 8; cl <= SR_MAX_CL; cl *= 2)
        if ((V + 14) / 8 / cl * 8 + 8 <= 65535 && slice_bytes<uint16_t>(V, cl, 0) <= SR_SMEM_MAX)
            return cl;
    return 0;
}

// Rows enough for every SM's CTAs twice over, or of which a cluster cannot hold one: a CTA each
// (0: not so). Its groups of sub-chunks, and its bytes of shared memory
template <typename T>
int far_groups(int V, int64_t rows, int num_sms)
{
    const int groups = (row_subs<T>(V) + SR_GROUP - 1) / SR_GROUP;
    const bool far = rows >= 2 * FAR_CTAS * num_sms || slice_bytes<T>(V, SR_MAX_CL, 0) > SR_SMEM_MAX;
    return far && groups * 8 <= SR_SMEM_MAX / FAR_CTAS - FB_BYTES ? groups : 0;
}
int far_bytes(int groups) { return (groups * 8 + 15) / 16 * 16 + FB_BYTES; }

template <typename Args>
cudaError_t launch_rows(void (*kernel)(Args), DeviceFlags &ready, int dev, int64_t rows, int cl, int threads, int smem,
                        bool dependent, const Args &args, cudaStream_t s)
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
    lc.blockDim = dim3(threads);
    lc.dynamicSmemBytes = smem;
    lc.stream = s;
    lc.attrs = at;
    lc.numAttrs = dependent ? 2 : 1;
    return cudaLaunchKernelEx(&lc, kernel, args);
}

}  // namespace

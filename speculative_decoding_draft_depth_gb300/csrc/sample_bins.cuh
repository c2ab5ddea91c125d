// sample_bins.cuh -- a row of bf16 logits by its values: what the settings keep of it, and
// the draw, from how often each value occurs.
//
// A bf16 row of 10^5 logits has a few thousand different values, and a token's weight is
// its value's: the order, its borders and all sums follow from the counts. So the pass
// over the row does one shared-memory addition a logit (some ten instructions; a weight to
// 2^-40 costs forty), each CTA of the cluster counts a slice, each then adds up a part of
// the values over all CTAs and makes their weights, and the borders are found in running
// sums over the values. A draw finds the CTA whose slice holds the token from the same
// counts; only that slice is read again, by all CTAs together, with weights token by token.
//
// Counted are zeros and magnitudes from 2^-30 to below 128, by all their bits, one 32-bit
// word a magnitude: positive values in its low half, negative ones in its high half.
// Values of -128 and less are left out (with temperatures up to 2.88 no row whose largest
// logit is positive gives them a weight). What this cannot hold (a nonzero magnitude below
// 2^-30, a logit of 128 or more, a row wholly at -128 or below, a hot row with values down
// there) is left to the general way of sample_row.cuh: run() says so.
#pragma once

#include "sample_row.cuh"

namespace {

constexpr int SB_LOW = 97 << 7;       // bits of 2^-30
constexpr int SB_MAGS = 37 << 7;      // magnitudes: 2^-30 up to 128
// words of the histogram: 0 zeros, 1 smaller magnitudes, 2 .. SB_MAGS + 1, above
constexpr int SB_WORDS = SB_MAGS + 3;
// values in descending order: positive ones 0 .. SB_MAGS - 1, zero, negative ones
constexpr int SB_VALUES = 2 * SB_MAGS + 1;
constexpr int SB_UNROLL = 4;          // 16-byte vectors that a thread has in flight

// the word and half of value d, and the value
DDT_DEVINL int sb_word(int d) { return d < SB_MAGS ? SB_MAGS + 1 - d : d == SB_MAGS ? 0 : d - SB_MAGS + 1; }
DDT_DEVINL float sb_value(int d)
{
    if (d == SB_MAGS)
        return 0.f;
    const uint32_t mag = sb_word(d) - 2 + SB_LOW;
    return __uint_as_float((mag | (d > SB_MAGS ? 0x8000u : 0u)) << 16);
}
DDT_DEVINL uint32_t sb_count(uint32_t word, int d)
{
    return d < SB_MAGS ? word & 0xFFFFu : d > SB_MAGS ? word >> 16 : (word & 0xFFFFu) + (word >> 16);
}

// values of a CTA's part, and its bytes of shared memory: the histogram, then of each value
// of the part how often it occurs in the row and its weight
__host__ __device__ constexpr int sb_part(int cl) { return (SB_VALUES + cl - 1) / cl; }
__host__ __device__ constexpr int sb_bytes(int cl) { return (SB_WORDS * 4 + 15) / 16 * 16 + sb_part(cl) * 12 + 16; }

// where a logit's bits are counted (0: zeros, 1: what is smaller than 2^-30, SB_WORDS - 1: what
// is larger), and whether they are
DDT_DEVINL int sb_place(uint32_t b)
{
    const uint32_t mag = b & 0x7FFFu;
    return min(max((int)mag - (SB_LOW - 2), min((int)mag, 1)), SB_WORDS - 1);
}
DDT_DEVINL bool sb_counts(uint32_t b) { return b < 0x8000u + SB_LOW + SB_MAGS; }  // (not the negative ones beyond)

// what the settings keep, as a value of which so many count, and its sum
struct Kept {
    int d;           // SB_VALUES: everything
    uint64_t count;  // of value d
    uint64_t of;     //   out of so many
    uint64_t mass;
};

template <int CL>
struct BinShared {
    uint64_t mass[CL][CL];  // [of a part of the values][in a CTA's slice]
    uint64_t sum[SR_WARPS][CL];
};

template <int CL>
struct BinRow {
    using Base = Row<uint16_t>;
    Base &row;  // its exchanges and block sums
    BinShared<CL> *bs;
    uint32_t *hist;
    uint64_t *w;       // of this CTA's values
    uint32_t *n;
    const uint16_t *z;  // the row
    int V, off, v0, v1;  // this CTA's vectors: vector v holds elements v * 8 - off ..
    int d0, d1;          // its values
    float least;         // values from here on count

    DDT_DEVINL BinRow(Base &r, BinShared<CL> *b, unsigned char *smem, const uint16_t *z_, int V_) : row(r), bs(b), z(z_), V(V_)
    {
        hist = reinterpret_cast<uint32_t *>(smem);
        w = reinterpret_cast<uint64_t *>(smem + (SB_WORDS * 4 + 15) / 16 * 16);
        const int part = sb_part(CL);
        n = reinterpret_cast<uint32_t *>(w + part);
        d0 = min(SB_VALUES, (int)row.rank * part);
        d1 = min(SB_VALUES, d0 + part);
        off = (int)(((uintptr_t)z & 15) / 2);
        const int vecs = (off + V + 7) / 8;
        v0 = (int)((int64_t)vecs * row.rank / CL);
        v1 = (int)((int64_t)vecs * (row.rank + 1) / CL);
    }
    // a word of every CTA's histogram
    DDT_DEVINL void read(int word, uint32_t (&x)[CL]) const
    {
#pragma unroll
        for (int c = 0; c < CL; ++c)
            x[c] = cl_ld32(cl_map(&hist[word], c));
    }
    DDT_DEVINL bool inner(int v) const { return v * 8 >= off && v * 8 + 8 <= off + V; }

    DDT_DEVINL void add(uint32_t b) const  // one logit's bits
    {
        if (sb_counts(b))
            atomicAdd(&hist[sb_place(b)], b & 0x8000u ? 0x10000u : 1u);
    }
    DDT_DEVINL void add2(uint32_t x, uint32_t &least2) const
    {
        asm("min.bf16x2 %0, %0, %1;" : "+r"(least2) : "r"(x));
        add(x & 0xFFFFu);
        add(x >> 16);
    }
    DDT_DEVINL void add8(const uint4 &x, uint32_t &least2) const
    {
        add2(x.x, least2);
        add2(x.y, least2);
        add2(x.z, least2);
        add2(x.w, least2);
    }
    DDT_DEVINL void edge(int v, uint32_t &least2) const  // a vector that is partly the row's
    {
        for (int i = max(0, v * 8 - off); i < min(V, v * 8 + 8 - off); ++i) {
            const uint32_t b = __ldg(z + i);
            asm("min.bf16x2 %0, %0, %1;" : "+r"(least2) : "r"(b * 0x10001u));
            add(b);
        }
    }

    // counts, weights, borders. false: this row is not one for counting
    DDT_DEVINL bool run(const Settings &set, const Scale &sc, Kept &k)
    {
        const int tid = row.tid;
        for (int i = tid; i < SB_WORDS; i += SR_THREADS)
            hist[i] = 0;
        if (tid == 0)
            row.sh->list[0] = 0;  // (see hold)
        __syncthreads();
        uint32_t least2 = 0x7F807F80u;  // pairs of the least (numbers)
        const uint4 *at = reinterpret_cast<const uint4 *>(z - off);
        int v = v0 + tid;
        for (; v + (SB_UNROLL - 1) * SR_THREADS < v1; v += SB_UNROLL * SR_THREADS) {
            uint4 x[SB_UNROLL];
#pragma unroll
            for (int u = 0; u < SB_UNROLL; ++u) {
                const int vu = v + u * SR_THREADS;
                x[u] = inner(vu) ? __ldg(at + vu) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int u = 0; u < SB_UNROLL; ++u) {
                if (inner(v + u * SR_THREADS))
                    add8(x[u], least2);
                else
                    edge(v + u * SR_THREADS, least2);
            }
        }
        for (; v < v1; v += SR_THREADS) {
            if (inner(v))
                add8(__ldg(at + v), least2);
            else
                edge(v, least2);
        }
        bool low = fminf(bf16lo(least2), bf16hi(least2)) <= -128.f;
        low = __syncthreads_or(low);
        const bool odd = hist[1] != 0 || (hist[SB_WORDS - 1] & 0xFFFFu) != 0;
        const uint64_t(*all)[4] = row.exchange(odd || (low && sc.zfloor < -128.f), 0, 0, 0);
        bool general = sc.zmax <= -128.f;
        for (int c = 0; c < CL; ++c)
            general |= all[c][0] != 0;
        if (general)
            return false;
        least = fmaxf(sc.zfloor, set.m > 0.f ? min_value(sc.zmax, row.sh->off) : DDT_NEG_INF);

        // ---- this CTA's values, over all slices
        for (int i = tid; i < d1 - d0; i += SR_THREADS) {
            const int d = d0 + i, word = sb_word(d);
            uint32_t x[CL], t = 0;
            read(word, x);
#pragma unroll
            for (int c = 0; c < CL; ++c)
                t += sb_count(x[c], d);
            const float y = sb_value(d);
            const bool in = t > 0 && y >= least;
            n[i] = in ? t : 0;
            w[i] = in ? weight_of<false>(sc, row.sh->tab, y) : 0;
        }
        __syncthreads();
        const int per = (d1 - d0 + SR_THREADS - 1) / SR_THREADS, a = min(d1 - d0, tid * per), b = min(d1 - d0, a + per);
        uint64_t cnt = 0, mass = 0;
        for (int i = a; i < b; ++i) {
            cnt += n[i];
            mass += n[i] * w[i];
        }
        const uint64_t cnt1 = row.block_incl(cnt), mass1 = row.block_incl(mass);
        if (tid == SR_THREADS - 1) {
            row.sh->warp[0][1] = cnt1;
            row.sh->warp[0][2] = mass1;
        }
        __syncthreads();
        all = row.exchange(row.sh->warp[0][1], row.sh->warp[0][2], 0, 0);
        uint64_t cnt0 = 0, mass0 = 0, cnt_all = 0, mass_all = 0;  // before this CTA's values, of all
        for (int c = 0; c < CL; ++c) {
            if (c < row.rank)
                cnt0 += all[c][0], mass0 += all[c][1];
            cnt_all += all[c][0];
            mass_all += all[c][1];
        }
        cnt0 += cnt1 - cnt;  // before this thread's
        mass0 += mass1 - mass;
        k = {SB_VALUES, 0, 0, mass_all};
        // ---- top-k: the value that holds the k-th token
        if (set.k > 0 && (uint64_t)set.k < cnt_all) {
            const uint64_t want = set.k;
            uint64_t q = cnt0, m = mass0;
            for (int i = a; i < b; ++i) {
                if (q < want && want <= q + n[i])
                    hold(d0 + i, want - q, n[i], m + (want - q) * w[i]);
                q += n[i];
                m += n[i] * w[i];
            }
            k = told();
        }
        // ---- top-p: the value at which the sum reaches its share
        if (set.p < 1.f) {
            const uint64_t want = max(Base::share_of(set.p, k.mass), (uint64_t)1);
            uint64_t m = mass0;
            for (int i = a; i < b; ++i) {
                if (m < want && want <= m + n[i] * w[i]) {
                    const uint64_t c = (want - m + w[i] - 1) / w[i];
                    hold(d0 + i, c, n[i], m + c * w[i]);
                }
                m += n[i] * w[i];
            }
            k = told();
        }
        return true;
    }

    // one thread of the cluster has the answer; all know it afterwards (told() also makes
    // the place free again: its reset comes before the barrier of the next exchange)
    DDT_DEVINL void hold(int d, uint64_t count, uint64_t of, uint64_t mass)
    {
        uint64_t *q = row.sh->list;
        q[0] = 1;
        q[1] = ((uint64_t)d << 32) | (uint32_t)count;
        q[2] = of;
        q[3] = mass;
    }
    DDT_DEVINL Kept told()
    {
        uint64_t *q = row.sh->list;
        __syncthreads();
        const bool mine = q[0] != 0;
        const uint64_t x = mine ? q[1] : 0, y = mine ? q[2] : 0, m = mine ? q[3] : 0;
        const uint64_t(*all)[4] = row.exchange(x, y, m, mine);
        if (row.tid == 0)
            q[0] = 0;
        __syncthreads();
        Kept k = {SB_VALUES, 0, 0, 0};
        for (int c = 0; c < CL; ++c)
            if (all[c][3])
                k = {(int)(all[c][0] >> 32), (uint32_t)all[c][0], all[c][1], all[c][2]};
        return k;
    }

    // The last kept index of value k.d, where not all of it is kept: in one thread of one
    // CTA, -1 elsewhere.
    DDT_DEVINL int last_kept(const Kept &k) const
    {
        if (k.d == SB_VALUES || k.count == k.of)
            return -1;
        uint64_t m = k.count;  // of those in this slice and behind it
        const int word = sb_word(k.d);
        uint32_t y[CL];
        read(word, y);
        bool here = false;
#pragma unroll
        for (int c = 0; c < CL; ++c) {
            const uint32_t h = sb_count(y[c], k.d);
            if (c < (int)row.rank)
                m = h >= m ? 0 : m - h;
            if (c == (int)row.rank)
                here = m > 0 && h >= m;
        }
        if (!here)
            return -1;
        const float x = sb_value(k.d);
        const int nv = v1 - v0, per = (nv + SR_THREADS - 1) / SR_THREADS;
        const int a = min(nv, row.tid * per), b = min(nv, a + per);
        uint32_t own = 0;
        for (int v = a; v < b; ++v) {
            float y[8];
            get(v0 + v, y);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                own += y[e] == x;
        }
        uint64_t at = row.block_incl(own) - own;
        if (!(at < m && m <= at + own))
            return -1;
        for (int v = a; v < b; ++v) {
            float y[8];
            get(v0 + v, y);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (y[e] == x && ++at == m)
                    return (v0 + v) * 8 + e - off;
        }
        return -1;
    }
    // a vector's logits (-infinity outside the row; NaN and what is next to 0 as counted)
    DDT_DEVINL void get(int v, float *y) const
    {
        if (inner(v)) {
            Vec<uint16_t>::get(__ldg(reinterpret_cast<const uint4 *>(z - off) + v), y);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int i = v * 8 + e - off;
                y[e] = i >= 0 && i < V ? logit_value(z, i) : DDT_NEG_INF;
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
            y[e] = held_value(y[e], false);
    }

    // ---- the token that u draws, in one thread of one CTA; -1 elsewhere. b: the border
    DDT_DEVINL int draw(const Scale &sc, const Kept &k, float u, Border &b)
    {
        // what is kept of each slice: of this CTA's values, then over all
        uint64_t acc[CL];
#pragma unroll
        for (int c = 0; c < CL; ++c)
            acc[c] = 0;
        for (int i = row.tid; i < d1 - d0; i += SR_THREADS) {
            const int d = d0 + i, word = sb_word(d);
            if (n[i] == 0 || d > k.d)
                continue;
            uint64_t left = d == k.d ? k.count : ~0ull;
            uint32_t x[CL];
            read(word, x);
#pragma unroll
            for (int c = 0; c < CL; ++c) {
                const uint64_t t = min((uint64_t)sb_count(x[c], d), left);
                left -= t;
                acc[c] += t * w[i];
            }
        }
#pragma unroll
        for (int c = 0; c < CL; ++c) {
            const uint64_t t = warp_sum64(acc[c]);
            if (row.lane == 0)
                bs->sum[row.warp][c] = t;
        }
        const int last = last_kept(k);
        __syncthreads();
        if (row.tid == 0)
            row.sh->found[2] = -1;
        __syncthreads();
        if (last >= 0)
            row.sh->found[2] = last;
        if (row.tid < (int)(CL * CL)) {
            const int c = row.tid % CL, to = row.tid / CL;
            uint64_t t = 0;
#pragma unroll
            for (int q = 0; q < SR_WARPS; ++q)
                t += bs->sum[q][c];
            cl_st64(cl_map(&bs->mass[row.rank][c], to), t);
        }
        __syncthreads();
        const uint64_t(*all)[4] = row.exchange((uint64_t)(int64_t)row.sh->found[2], 0, 0, 0);
        b.z = k.d == SB_VALUES ? least : sb_value(k.d);
        b.last = 0x7FFFFFFF;
        for (int c = 0; c < CL; ++c)
            if ((int64_t)all[c][0] >= 0)
                b.last = (int)all[c][0];
        const uint64_t target = draw_target(u, k.mass);
        uint64_t at = 0;
        int owner = 0;
        for (int c = 0; c < CL; ++c) {
            uint64_t t = 0;
            for (int q = 0; q < CL; ++q)
                t += bs->mass[q][c];
            if (at + t > target) {
                owner = c;
                break;
            }
            at += t;
        }
        // the owner's slice, in parts
        const int vecs = (off + V + 7) / 8;
        const int o0 = (int)((int64_t)vecs * owner / CL), o1 = (int)((int64_t)vecs * (owner + 1) / CL);
        const int p0 = o0 + (int)((int64_t)(o1 - o0) * row.rank / CL), p1 = o0 + (int)((int64_t)(o1 - o0) * (row.rank + 1) / CL);
        const int per = (p1 - p0 + SR_THREADS - 1) / SR_THREADS, a = min(p1, p0 + row.tid * per), e1 = min(p1, a + per);
        uint64_t own = 0;
        for (int v = a; v < e1; ++v)
            own += vector_mass(sc, b, v);
        const uint64_t incl = row.block_incl(own);
        if (row.tid == SR_THREADS - 1)
            row.sh->warp[0][1] = incl;
        __syncthreads();
        all = row.exchange(row.sh->warp[0][1], 0, 0, 0);
        for (uint32_t c = 0; c < row.rank; ++c)
            at += all[c][0];
        at += incl - own;
        if (!(at <= target && target < at + own))
            return -1;
        for (int v = a; v < e1; ++v) {
            float y[8];
            uint64_t x[8];
            weights(sc, b, v, y, x);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (target < at + x[e])
                    return v * 8 + e - off;
                at += x[e];
            }
        }
        return -1;
    }
    DDT_DEVINL void weights(const Scale &sc, const Border &b, int v, float *y, uint64_t *x) const
    {
        get(v, y);
        const int i0 = v * 8 - off;
#pragma unroll
        for (int e = 0; e < 8; e += 2)
            fixed_pair<false>(sc, row.sh->tab, y[e], y[e + 1], kept(b, y[e], i0 + e), kept(b, y[e + 1], i0 + e + 1), x[e], x[e + 1]);
    }
    DDT_DEVINL uint64_t vector_mass(const Scale &sc, const Border &b, int v) const
    {
        float y[8];
        uint64_t x[8], t = 0;
        weights(sc, b, v, y, x);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            t += x[e];
        return t;
    }
};

// The same for a row that one CTA reads from global memory: a 32-bit count each of a
// magnitude's two signs; weights are made where they are needed (a thread has some twenty
// values, few of which occur). Under top-p alone only the front of the row is counted, and
// the tokens behind it are added up by quick weights: a sixteenth of the row tells from where
// up the tokens hold more than p of the sum, and the border stands unless two tokens lie
// within the error of that small rest.
struct FarBins {
    using Base = Row<uint16_t, true>;
    static constexpr int T = Base::THREADS, SAMPLE = 16;
    Base &row;
    const Scale &sc;
    uint32_t *hist;      // 2 SB_WORDS
    float least;         // values from here up may count
    float from;          //   and are counted from here up
    int a, b;            // this thread's values
    uint64_t cnt, mass;  //   their tokens and weights
    uint64_t cnt0, mass0, cnt_all, mass_all;  // before them, and of all that are counted
    uint64_t rest;       // weights of the others, quick ones

    DDT_DEVINL uint32_t count(int d) const
    {
        const int w = 2 * sb_word(d);
        return d < SB_MAGS ? hist[w] : d > SB_MAGS ? hist[w + 1] : hist[w] + hist[w + 1];
    }
    DDT_DEVINL uint64_t weight(int d) const { return weight_of<false>(sc, row.sh->tab, sb_value(d)); }

    // a value from which up the tokens very likely weigh more than p of all
    DDT_DEVINL float front(float p, float low)
    {
        const float vlo = fmaxf(low, least), scale = row.bin_scale(sc.zmax, vlo);
        row.clear_hist();
        const int ng = row.sl.groups(), n_look = min(ng, max(Base::WARPS, ng / SAMPLE));
        for (int g = row.warp; g < n_look; g += Base::WARPS) {
            uint4 x[SR_GROUP];
            row.sl.raws((int)((int64_t)g * ng / n_look) * SR_GROUP, row.lane, x);
#pragma unroll
            for (int i = 0; i < SR_GROUP; ++i) {
                float z[8];
                row.sl.values(x[i], z);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (z[e] >= vlo)
                        atomicAdd(&row.sh->hist[row.bin_of(sc.zmax, scale, z[e])], 1u);
            }
        }
        __syncthreads();
        uint32_t n[2];
        row.row_bins(n[0], n[1]);
        const float inv = scale > 0.f ? 1.f / scale : 0.f, share = (float)ng / n_look;
        uint64_t w[2];
#pragma unroll
        for (int x = 0; x < 2; ++x)
            w[x] = __float2ull_rn((float)n[x] * share * ex2(-(2 * row.tid + x) * inv * sc.ch) * 17592186044416.0f);
        const uint64_t incl = row.block_incl(w[0] + w[1]);
        __syncthreads();
        if (row.tid == T - 1)
            row.sh->warp[0][1] = incl;
        __syncthreads();
        const uint64_t all = row.sh->warp[0][1], tail = (uint64_t)((1.f - p) * 0.5f * (float)all);
        // the first bin behind which no more than `tail` lies
        const int bin = row.block_least(all - (incl - w[1]) <= tail ? 2 * row.tid : all - incl <= tail ? 2 * row.tid + 1 : 0x7FFFFFFF);
        return bin >= SR_BINS - 1 || !(scale > 0.f) ? least : fmaxf(least, sc.zmax - (bin + 1) * inv);
    }
    // count the tokens from `from` up. false: not a row for this
    DDT_DEVINL bool run()
    {
        const int tid = row.tid;
        for (int i = tid; i < 2 * SB_WORDS; i += T)
            hist[i] = 0;
        __syncthreads();
        uint32_t least2 = 0x7F807F80u;
        const bool some = from > least, positive = some && from >= 9.313225746e-10f && sc.zmax < 128.f;  // (2^-30)
        rest = 0;
        row.each([&](int, const uint4 &v) {
            if (some) {
                float z[8];
                Vec<uint16_t>::get(v, z);
                uint64_t w = 0;
#pragma unroll
                for (int e = 0; e < 8; e += 2)
                    w = f2add(w, quick_weights<false>(sc, z[e], z[e + 1], z[e] >= least && z[e] < from,
                                                      z[e + 1] >= least && z[e + 1] < from));
                float w0, w1;
                f2unpack(w, w0, w1);
                rest += __float2ull_rn((w0 + w1) * 17592186044416.0f);
                if (!Vec<uint16_t>::reaches(v, from))
                    return;
            }
            const uint32_t x[4] = {v.x, v.y, v.z, v.w};
            if (positive) {  // (the same, in fewer instructions)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (bf16lo(x[i]) >= from)
                        atomicAdd(&hist[2 * ((int)(x[i] & 0xFFFFu) - (SB_LOW - 2))], 1u);
                    if (bf16hi(x[i]) >= from)
                        atomicAdd(&hist[2 * ((int)(x[i] >> 16) - (SB_LOW - 2))], 1u);
                }
                return;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                asm("min.bf16x2 %0, %0, %1;" : "+r"(least2) : "r"(x[i]));
                const uint32_t lo = x[i] & 0xFFFFu, hi = x[i] >> 16;
                if (some ? bf16lo(x[i]) >= from : sb_counts(lo))
                    atomicAdd(&hist[2 * sb_place(lo) + (lo >> 15)], 1u);
                if (some ? bf16hi(x[i]) >= from : sb_counts(hi))
                    atomicAdd(&hist[2 * sb_place(hi) + (hi >> 15)], 1u);
            }
        });
        const bool low = __syncthreads_or(fminf(bf16lo(least2), bf16hi(least2)) <= -128.f);
        if (hist[2] != 0 || hist[3] != 0 || hist[2 * SB_WORDS - 2] != 0 || sc.zmax <= -128.f || (low && fmaxf(from, sc.zfloor) < -128.f))
            return false;
        // (with the front alone, its values only: that of `from` rounded down, and above)
        const int d_end = positive ? SB_MAGS + 2 - sb_place(__float_as_uint(from) >> 16) : SB_VALUES;
        const int d_first = positive ? SB_MAGS + 1 - sb_place(__float_as_uint(sc.zmax) >> 16) : 0;
        const int per = (d_end - d_first + T - 1) / T;
        a = min(d_end, d_first + tid * per);
        b = min(d_end, a + per);
        cnt = mass = 0;
        for (int d = a; d < b; ++d) {
            const uint32_t n = count(d);
            if (n > 0 && sb_value(d) >= least) {
                cnt += n;
                mass += n * weight(d);
            }
        }
        cnt0 = row.block_incl(cnt) - cnt;
        mass0 = row.block_incl(mass) - mass;
        __syncthreads();
        if (tid == T - 1) {
            row.sh->warp[0][1] = cnt0 + cnt;
            row.sh->warp[0][2] = mass0 + mass;
        }
        __syncthreads();
        cnt_all = row.sh->warp[0][1];
        mass_all = row.sh->warp[0][2];
        if (some)
            rest = row.block_sum(rest);
        return true;
    }
    // the value at which the tokens (or their weights) reach `want`, which they do
    DDT_DEVINL Kept find(bool tokens, uint64_t want)
    {
        const uint64_t before = tokens ? cnt0 : mass0, own = tokens ? cnt : mass;
        uint64_t *to = row.sh->list;
        __syncthreads();
        if (before < want && want <= before + own) {
            uint64_t q = cnt0, m = mass0;
            for (int d = a; d < b; ++d) {
                const uint32_t n = count(d);
                if (n == 0 || !(sb_value(d) >= least))
                    continue;
                const uint64_t w = weight(d);
                const uint64_t c = tokens ? want - q : w > 0 ? (want - m + w - 1) / w : n + 1ull;
                if (c <= n) {
                    to[0] = ((uint64_t)d << 32) | (uint32_t)c;
                    to[1] = n;
                    to[2] = m + c * w;
                    break;
                }
                q += n;
                m += n * w;
            }
        }
        __syncthreads();
        return {(int)(to[0] >> 32), (uint32_t)to[0], to[1], to[2]};
    }
    DDT_DEVINL bool solve(const Settings &set, float low, Kept &k)
    {
        least = fmaxf(sc.zfloor, set.m > 0.f ? min_value(sc.zmax, row.sh->off) : DDT_NEG_INF);
        if (!(set.k > 0 && set.k < row.sl.V)) {
            from = front(set.p, low);
            if (!run())
                return false;
            const uint64_t slack = quick_slack(rest) + 1, most = Base::share_of(set.p, mass_all + rest + slack);
            if (from > least && most <= mass_all) {
                k = find(false, max(Base::share_of(set.p, mass_all + rest - min(rest, slack)), (uint64_t)1));
                const Kept other = find(false, max(most, (uint64_t)1));
                if (k.d == other.d && k.count == other.count)
                    return true;
            }
            if (!(from > least)) {  // (all of it has been counted)
                k = find(false, max(Base::share_of(set.p, mass_all), (uint64_t)1));
                return true;
            }
        }
        from = least;
        if (!run())
            return false;
        k = {SB_VALUES, 0, 0, mass_all};
        if (set.k > 0 && (uint64_t)set.k < cnt_all)
            k = find(true, set.k);
        if (set.p < 1.f)
            k = find(false, max(Base::share_of(set.p, k.mass), (uint64_t)1));
        return true;
    }
    // the border that this is
    DDT_DEVINL Border border(const Kept &k, uint64_t *sub)
    {
        Border r = {k.d == SB_VALUES ? least : sb_value(k.d), 0x7FFFFFFF};
        if (k.d != SB_VALUES && k.count != k.of)
            r.last = row.nth_equal(r, r.z, k.count, sub);
        return r;
    }
};
constexpr int FB_BYTES = 2 * SB_WORDS * 4;

}  // namespace

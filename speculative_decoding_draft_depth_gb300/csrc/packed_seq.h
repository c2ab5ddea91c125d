// packed_seq.h -- which requests' lengths are sound, and which tensors of a call lie
// apart. Plain integer arithmetic, the same on the host (where a test runs it) and on
// the device.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define PS_FN __host__ __device__ __forceinline__
#else
#define PS_FN static inline
#endif

// request r: rows [s0, s1) of T packed ones behind ctx cached tokens, with room
// for `cap` slots (cap <= 2^31 - 1: no sum below overflows)
PS_FN bool packed_ok(int s0, int s1, int T, int ctx, int cap)
{
    return s0 >= 0 && s0 <= s1 && s1 <= T && ctx >= 0 && ctx <= cap && s1 - s0 <= cap - ctx;
}

// the bytes of a tensor: none if it is not given
struct PsBytes {
    const void *at;
    int64_t n;
};

PS_FN bool ps_share(const PsBytes &a, const PsBytes &b)
{
    const uintptr_t x = (uintptr_t)a.at, y = (uintptr_t)b.at;
    return a.at && b.at && a.n > 0 && b.n > 0 && x < y + (uintptr_t)b.n && y < x + (uintptr_t)a.n;
}

// each of the nw written tensors shares no byte with another one or with any of the nr
// that are read (those may share with each other)
PS_FN bool ps_apart(const PsBytes *w, int nw, const PsBytes *r, int nr)
{
    for (int i = 0; i < nw; ++i) {
        for (int j = 0; j < i; ++j)
            if (ps_share(w[i], w[j]))
                return false;
        for (int j = 0; j < nr; ++j)
            if (ps_share(w[i], r[j]))
                return false;
    }
    return true;
}

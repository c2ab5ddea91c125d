// packed_seq.h -- which request a packed row belongs to, and which requests'
// lengths are sound. Plain integer arithmetic, the same on the host (where a
// test runs it) and on the device.
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

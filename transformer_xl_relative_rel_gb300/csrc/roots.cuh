// roots.cuh -- square roots and reciprocals to nearest, in fewer instructions
// than the functions take: an approximation of the hardware and one Newton
// step whose residual a fused multiply-add gives exactly (P. Markstein,
// "Computation of elementary functions on the IBM RISC System/6000", IBM
// Journal of Research and Development 34, 1990).
//
// That one step is enough on this hardware is not proved but tested: with
// every float of the ranges below the results are __frcp_rn's and __fsqrt_rn's
// (tests/test_gpu_roots.py).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "rows.cuh"

namespace txl {

// 1 / x to an ulp, for normal x; 0 above 2^126
__device__ __forceinline__ float reciprocal(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// 1 / x to nearest, for a normal x of a normal reciprocal: the same to an ulp
// and one Newton step with its exact residual
__device__ __forceinline__ float exact_reciprocal(float x)
{
    const float r = reciprocal(x);
    return fmaf(r, fmaf(-x, r, 1.f), r);
}

// The square roots of two numbers, 0 or at least 2^-100, to nearest: a root of
// about 22 bits and one Newton step with its exact residual.  NaN for infinity.
__device__ __forceinline__ uint64_t pair_sqrt(uint64_t v)
{
    float a, b, ra, rb;
    unpair(pair_add(v, pair(0x1p-126f, 0x1p-126f)), a, b);      // (only 0 is changed: it has no reciprocal root)
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(ra) : "f"(a));
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(rb) : "f"(b));
    const uint64_t r = pair(ra, rb), s = pair_mul(v, r), half = pair_mul(r, pair(0.5f, 0.5f));
    const uint64_t residual = pair_fma(pair_sub(0, s), s, v);
    return pair_fma(residual, half, s);
}

// eight numbers' roots; by the function where one is so small (below 2^-100,
// but not 0) that the Newton step's residual has no room, or infinite (the sum
// then is; one that overflows of finite numbers costs time only)
__device__ __forceinline__ void eight_sqrt(const uint64_t (&v)[4], uint64_t (&root)[4])
{
    uint32_t least = 0xffffffffu;      // (the bits of 0, less one, are the largest)
    float x[8], lo, hi;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        unpair(v[k], x[2 * k], x[2 * k + 1]);
        least = min(min(least, __float_as_uint(x[2 * k]) - 1u), __float_as_uint(x[2 * k + 1]) - 1u);
    }
    unpair(pair_add(pair_add(v[0], v[1]), pair_add(v[2], v[3])), lo, hi);
    if (least < (27u << 23) - 1u || !(lo + hi <= 3.4028234e38f)) {
#pragma unroll
        for (int k = 0; k < 4; ++k) root[k] = pair(__fsqrt_rn(x[2 * k]), __fsqrt_rn(x[2 * k + 1]));
        return;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) root[k] = pair_sqrt(v[k]);
}

}  // namespace txl

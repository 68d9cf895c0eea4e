// rows.cuh -- vectors of a row's neighbouring elements, held as fp32 in
// registers, for the kernels that stream rows of a tensor (embedding, layer
// norm, optimiser): each lane loads and stores W bytes at a time.
//
// Plain loads and stores (no read-only path): the kernels are resident while
// their predecessor still writes (chain.h).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace txl {

template <int BYTES>
struct RawVec;
template <>
struct RawVec<16> { typedef uint4 type; };
template <>
struct RawVec<8> { typedef uint2 type; };
template <>
struct RawVec<4> { typedef uint32_t type; };
template <>
struct RawVec<2> { typedef uint16_t type; };

template <typename T, int V>
using raw_t = typename RawVec<(int)sizeof(T) * V>::type;

template <typename T, int V>
__device__ __forceinline__ raw_t<T, V> load_raw(const T *p)
{
    return *reinterpret_cast<const raw_t<T, V> *>(p);
}

// the V elements of a raw vector as fp32
template <typename T, int V>
__device__ __forceinline__ void unpack(const raw_t<T, V> &r, float (&x)[V])
{
    if constexpr (sizeof(T) == 4) {
        const float *f = reinterpret_cast<const float *>(&r);
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = f[i];
    } else if constexpr (V == 1) {
        x[0] = __uint_as_float((uint32_t)r << 16);
    } else {
        const uint32_t *w = reinterpret_cast<const uint32_t *>(&r);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
}

// V fp32 values as a raw vector of T: one rounding to nearest
template <typename T, int V>
__device__ __forceinline__ raw_t<T, V> pack(const float (&x)[V])
{
    raw_t<T, V> r;
    if constexpr (sizeof(T) == 4) {
        float *f = reinterpret_cast<float *>(&r);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = x[i];
    } else if constexpr (V == 1) {
        r = __bfloat16_as_ushort(__float2bfloat16_rn(x[0]));
    } else {
        __nv_bfloat162 *w = reinterpret_cast<__nv_bfloat162 *>(&r);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) w[i] = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    }
    return r;
}

template <typename T, int V>
__device__ __forceinline__ void store_vec(T *p, const float (&x)[V])
{
    *reinterpret_cast<raw_t<T, V> *>(p) = pack<T, V>(x);
}

// V fp32 values to p, which lies at a multiple of 4 V bytes (of 16 at most)
template <int V>
__device__ __forceinline__ void store_floats(float *p, const float (&x)[V])
{
    if constexpr (V >= 4) {
#pragma unroll
        for (int i = 0; i < V; i += 4)
            *reinterpret_cast<float4 *>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
    } else if constexpr (V == 2) {
        *reinterpret_cast<float2 *>(p) = make_float2(x[0], x[1]);
    } else {
        *p = x[0];
    }
}

// V fp32 values from p (as store_floats)
template <int V>
__device__ __forceinline__ void load_floats(const float *p, float (&x)[V])
{
    if constexpr (V >= 4) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const float4 f = *reinterpret_cast<const float4 *>(p + i);
            x[i] = f.x;
            x[i + 1] = f.y;
            x[i + 2] = f.z;
            x[i + 3] = f.w;
        }
    } else if constexpr (V == 2) {
        const float2 f = *reinterpret_cast<const float2 *>(p);
        x[0] = f.x;
        x[1] = f.y;
    } else {
        x[0] = *p;
    }
}

// Two fp32 values in one 64-bit register: one instruction, two operations.
__device__ __forceinline__ uint64_t pair(float lo, float hi)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float &lo, float &hi)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t pair_add(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t pair_sub(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t pair_mul(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t pair_fma(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
// a b + c where k < n, else c
__device__ __forceinline__ uint64_t pair_fma_below(uint64_t a, uint64_t b, uint64_t c, int k, int n)
{
    asm("{\n\t.reg .pred below;\n\tsetp.lt.s32 below, %3, %4;\n\t@below fma.rn.f32x2 %0, %1, %2, %0;\n\t}"
        : "+l"(c) : "l"(a), "l"(b), "r"(k), "r"(n));
    return c;
}
// a + b towards zero
__device__ __forceinline__ uint64_t pair_add_rz(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rz.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

}  // namespace txl

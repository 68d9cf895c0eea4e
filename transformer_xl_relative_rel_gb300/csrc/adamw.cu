// adamw.cu -- the optimiser step over many tensors at once (AdamW:
// Loshchilov and Hutter's decoupled weight decay), with moments in 32 or 8
// bits, and the global norm of their gradients.
//
//     g = grad grad_scale
//     m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2
//     p = p - lr (wd p + (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps))
//
// HBM-bound: every value is read and written once, 8 neighbouring elements
// per thread.  All tensors of a call share a launch: their descriptions are a
// kernel argument (up to kMostTensors of them), work is cut into rounds of
// 2048 elements, and a block finds its rounds' tensors by bisection.
//
// Measured: 229 M weights (bf16 with masters, 32-bit moments) 905 us for 6.4 GB
// (7.1 TB/s, a little above the measured copy rate), the norm of their
// gradients 84 us for 458 MB; 34 M weights with 8-bit moments 100 us for 547 MB
// (5.5 TB/s), bound by the arithmetic of the codes next to the memory (some 70
// instructions an element, issued in 0.7 of the cycles).
//
// 8-bit moments: e4m3 codes of m and of sqrt(v) (half the exponent range of
// v), times a scale per 256 elements that maps the largest to 448.  Rounding
// is stochastic: at b2 = 0.999 a step changes sqrt(v) by 0.05% where
// neighbouring codes are 6 to 12% apart, so rounding to nearest would leave v
// where it is.  The random bits are a hash of seed, tensor, step and element.
// What a code depends on is computed operation by operation, each rounded to
// fp32 (no fused multiply-adds), so that the formulas in plain fp32
// arithmetic give the same codes.
#include <cuda_runtime.h>
#include <cuda_fp8.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <iterator>
#include <new>
#include <vector>

#include "buffers.h"
#include "chain.h"
#include "internal.h"
#include "roots.cuh"
#include "rows.cuh"

namespace txl {
namespace {

constexpr int NT = 256;
constexpr int kPer = 8;                         // elements per thread and round
constexpr int kRound = NT * kPer;
constexpr int kBlockElems = 256;                // elements that share a scale: one warp's
constexpr float kTop = 448.f;                   // the largest e4m3 value
constexpr int kCodesResident = 4;               // blocks per SM where moments have 8 bits
constexpr int kResident = 4;                    // ... 32 bits
constexpr int kRounds = 4;                      // rounds of a block, at most
constexpr int kMostTensors = 384, kFewTensors = 48;   // per launch: 30 KB of arguments, 4 KB
constexpr int64_t kMaxElements = (int64_t)1 << 40;    // of one tensor

// ---------------------------------------------------------------- descriptions
struct Tensor {
    void *param;             // F32 or BF16
    float *master;           // NULL: param itself is what the step acts on
    const void *grad;
    void *m, *v;             // float32, or e4m3 codes
    float *m_scale, *v_scale;   // NULL: float32 moments
    int64_t n;
    float decay;
    uint32_t key;            // of its random numbers
    uint8_t param_f32, grad_f32, wide, pad[5];   // wide: every buffer at a 16-byte boundary (codes: 8)
};

// A launch's tensors, cut into rounds of kRound elements.  The rounds that
// they begin at lie together: the search of a block whose SM has not looked at
// them yet waits for few lines.
template <int N>
struct Tensors {
    int first[N];
    int count, rounds;
    Tensor t[N];
};

struct GradTensor {
    const void *grad;
    int64_t n;
    uint8_t f32, wide, pad[6];
};

template <int N>
struct GradTensors {
    int first[N];
    int count, chunks;
    uint64_t one;                // as StepScalars'
    GradTensor t[N];
};

struct StepScalars {
    const float *lr_at, *grad_scale;
    const int64_t *step_at;
    uint64_t b1, b2, c1, c2, eps;    // twice each, as pairs; c1 = 1 - b1, c2 = 1 - b2
    uint64_t one;                    // of 1, unknown to the compiler (pair_sum)
    float lr, log_b1, log_b2;
    int64_t step;
};

// A permutation of 32-bit numbers whose outputs' bits depend evenly on all of
// the input's: two rounds of xor-shift and multiplication with the constants
// that C. Wellons found by search and published as public domain ("Prospecting
// for Hash Functions", 2018).
__host__ __device__ __forceinline__ uint32_t mix(uint32_t x)
{
    x = (x ^ (x >> 16)) * 0x7feb352du;
    x = (x ^ (x >> 15)) * 0x846ca68bu;
    return x ^ (x >> 16);
}

// the tensor of a round (in the norm, of a chunk)
template <typename List>
__device__ __forceinline__ int tensor_of(const List &l, int chunk)
{
    int lo = 0, hi = l.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (l.first[mid] <= chunk) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// ---------------------------------------------------------------- eight elements
// from element i on, of which `n` exist; `wide`: all of them, aligned
template <typename T>
__device__ __forceinline__ void load8(const T *p, int64_t i, int n, bool wide, float (&x)[8])
{
    if (wide) {
        if constexpr (sizeof(T) == 4) {
            load_floats<8>((const float *)p + i, x);
        } else {
            unpack<T, 8>(load_raw<T, 8>(p + i), x);
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float v[1] = {0.f};
        if (j < n) unpack<T, 1>(load_raw<T, 1>(p + i + j), v);
        x[j] = v[0];
    }
}

template <typename T>
__device__ __forceinline__ void store8(T *p, int64_t i, int n, bool wide, const float (&x)[8])
{
    if (wide) {
        if constexpr (sizeof(T) == 4) {
            store_floats<8>((float *)p + i, x);
        } else {
            store_vec<T, 8>(p + i, x);
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float v[1] = {x[j]};
        if (j < n) store_vec<T, 1>(p + i + j, v);
    }
}

__device__ __forceinline__ void load_codes(const void *p, int64_t i, int n, bool wide, uint32_t (&raw)[2])
{
    const uint8_t *c = (const uint8_t *)p + i;
    if (wide) {
        const uint2 r = *reinterpret_cast<const uint2 *>(c);
        raw[0] = r.x;
        raw[1] = r.y;
        return;
    }
    raw[0] = raw[1] = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j < n) raw[j / 4] |= (uint32_t)c[j] << (8 * (j % 4));
}

__device__ __forceinline__ void store_codes(void *p, int64_t i, int n, bool wide, const uint32_t (&raw)[2])
{
    uint8_t *c = (uint8_t *)p + i;
    if (wide) {
        *reinterpret_cast<uint2 *>(c) = make_uint2(raw[0], raw[1]);
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j < n) c[j] = (uint8_t)(raw[j / 4] >> (8 * (j % 4)));
}

// codes 2 k and 2 k + 1 of eight, times their scale
__device__ __forceinline__ uint64_t decode(const uint32_t (&raw)[2], int k, uint64_t scale)
{
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(raw[k / 2] >> (16 * (k % 2))), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    return pair_mul(pair(f.x, f.y), scale);
}

// The warp's 256 values x (8 per lane) as codes of x times one scale, which is
// returned.  h: random bits, of which the low halves are used, for roots
// (which are not negative, and keep at least one step) the high ones.
//
// Steps are counted as floats: |y| / 2^(e-3) + u, added to 2^23 towards zero,
// has the whole steps as its low bits.  8 (e + 6) more is the code, since a
// code's exponent field is e + 7 and its 3 bits of mantissa are steps - 8, or,
// below the normal numbers (e = -6), its bits are the steps; a step too many
// runs over into the exponent, as it should.  The largest y, 448 or a few
// 2^-22 of it more, plus u < 1 - 2^-17 stays below 15 steps: no code is past 448.
// (A warp's integer and logic operations are issued every other cycle: there
// are as few of them as of the others.)
template <bool ROOT>
__device__ __forceinline__ float encode(const uint64_t (&x)[4], const uint32_t (&h)[8], uint32_t (&raw)[2])
{
    uint32_t bits[8], top = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float lo, hi;
        unpair(x[k], lo, hi);
        bits[2 * k] = __float_as_uint(lo);
        bits[2 * k + 1] = __float_as_uint(hi);
        if (ROOT) top = max(max(top, bits[2 * k]), bits[2 * k + 1]);
        else top = max(max(top, bits[2 * k] & 0x7fffffffu), bits[2 * k + 1] & 0x7fffffffu);
    }
    top = __reduce_max_sync(0xffffffffu, top);        // (magnitudes are ordered as their bits are)
    const float most = __uint_as_float(top);
    raw[0] = raw[1] = 0;
    if (most < 0x1p-100f) return 0.f;
    // a block with a value that is not finite (or of 2^126, whose reciprocal is no normal number) is lost
    if (top >= 0x7e800000u) return __uint_as_float(0x7fffffffu);
    const float inverse = __fmul_rn(exact_reciprocal(most), kTop);
    uint32_t code[8];     // in the low bytes
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint64_t mag = ROOT ? x[k] : pair(__uint_as_float(bits[2 * k] & 0x7fffffffu),
                                                __uint_as_float(bits[2 * k + 1] & 0x7fffffffu));
        const uint64_t y2 = pair_mul(mag, pair(inverse, inverse));
        float y[2], one[2], u[2], steps[2];
        uint32_t e[2];
        unpair(y2, y[0], y[1]);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            e[j] = max(__float_as_uint(y[j]) & 0x7f800000u, (127u - 6u) << 23);
            one[j] = __uint_as_float((257u << 23) - e[j]);                               // 2^(3 - e)
            u[j] = __uint_as_float(__byte_perm(h[2 * k + j], 0x4b000000u, ROOT ? 0x7432 : 0x7410));   // 2^23 + 16 bits
        }
        const uint64_t u2 = pair_fma(pair(u[0], u[1]), pair(0x1p-16f, 0x1p-16f), pair(-128.f, -128.f));
        const uint64_t s2 = pair_fma(y2, pair(one[0], one[1]), u2);      // (the product is exact: one rounding)
        // 56: -8 * (127 - 6) in the low byte
        unpair(pair_add_rz(s2, pair(0x1p23f + 56.f, 0x1p23f + 56.f)), steps[0], steps[1]);
        code[2 * k] = __float_as_uint(steps[0]) + (e[0] >> 20);
        code[2 * k + 1] = __float_as_uint(steps[1]) + (e[1] >> 20);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const uint32_t *c = code + 4 * k, *b = bits + 4 * k;
        raw[k] = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
        if (!ROOT) {
            raw[k] |= __byte_perm(__byte_perm(b[0], b[1], 0x0073), __byte_perm(b[2], b[3], 0x0073), 0x5410) & 0x80808080u;
        } else if (((raw[k] - 0x01010101u) & ~raw[k] & 0x80808080u) != 0) {      // a code of 0
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (b[j] != 0 && (raw[k] >> (8 * j) & 0xffu) == 0) raw[k] |= 1u << (8 * j);
        }
    }
    return __fmul_rn(most, 1.f / kTop);
}

// a + b of products, each rounded by itself: the assembler fuses a packed
// product and a packed addition (not scalar ones), but not a product and a
// fused multiply-add by a 1 that it does not know
__device__ __forceinline__ uint64_t pair_sum(uint64_t one, uint64_t a, uint64_t b) { return pair_fma(one, a, b); }

// ---------------------------------------------------------------- the step
struct Rates {
    float lr, factor, r1, r2;     // r1 = 1 / (1 - b1^t), r2 = 1 / sqrt(1 - b2^t)
    int go;
};

// eight elements of a thread
struct Eight {
    float g[8], p[8];
    float m[8], v[8];          // 32-bit moments, or
    uint32_t cm[2], cv[2];     // codes, and
    float ms, vs;              // their scales
};

// from i on (n of them exist; WHOLE: the block's are all there and aligned)
template <bool CODES, bool WHOLE>
__device__ __forceinline__ void load_eight(const Tensor &t, int64_t i, int n, Eight &x)
{
    const bool wide = WHOLE || (t.wide && n == kPer);
    if (t.grad_f32) load8((const float *)t.grad, i, n, wide, x.g);
    else load8((const __nv_bfloat16 *)t.grad, i, n, wide, x.g);
    if (t.master) load8((const float *)t.master, i, n, wide, x.p);
    else if (t.param_f32) load8((const float *)t.param, i, n, wide, x.p);
    else load8((const __nv_bfloat16 *)t.param, i, n, wide, x.p);
    if (CODES) {
        load_codes(t.m, i, n, wide, x.cm);
        load_codes(t.v, i, n, wide, x.cv);
        x.ms = x.vs = 0.f;
        if (WHOLE || i / kBlockElems * kBlockElems < t.n) {       // (the same for a warp)
            x.ms = t.m_scale[i / kBlockElems];
            x.vs = t.v_scale[i / kBlockElems];
        }
    } else {
        load8((const float *)t.m, i, n, wide, x.m);
        load8((const float *)t.v, i, n, wide, x.v);
    }
}

// the step of what load_eight gave
template <bool CODES, bool WHOLE>
__device__ __forceinline__ void step_eight(const Tensor &t, const StepScalars &s, const Rates &r, uint32_t key, int64_t i,
                                           int n, Eight &x)
{
    const bool wide = WHOLE || (t.wide && n == kPer);
    const auto both = [](float y) { return pair(y, y); };
    uint64_t m2[4], v2[4], root2[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint64_t g2 = pair_mul(pair(x.g[2 * k], x.g[2 * k + 1]), both(r.factor));
        if (CODES) {
            m2[k] = decode(x.cm, k, both(x.ms));
            v2[k] = decode(x.cv, k, both(x.vs));
            v2[k] = pair_mul(v2[k], v2[k]);
        } else {
            m2[k] = pair(x.m[2 * k], x.m[2 * k + 1]);
            v2[k] = pair(x.v[2 * k], x.v[2 * k + 1]);
        }
        m2[k] = pair_sum(s.one, pair_mul(s.b1, m2[k]), pair_mul(s.c1, g2));
        v2[k] = pair_sum(s.one, pair_mul(s.b2, v2[k]), pair_mul(pair_mul(s.c2, g2), g2));
        if (!CODES) {
            unpair(v2[k], x.v[2 * k], x.v[2 * k + 1]);
            root2[k] = pair(__fsqrt_rn(x.v[2 * k]), __fsqrt_rn(x.v[2 * k + 1]));
        }
    }
    if (CODES) eight_sqrt(v2, root2);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        uint64_t p2 = pair(x.p[2 * k], x.p[2 * k + 1]);
        float a, b;
        unpair(pair_fma(root2[k], both(r.r2), s.eps), a, b);
        const uint64_t update = pair_mul(pair_mul(m2[k], both(r.r1)), pair(reciprocal(a), reciprocal(b)));
        // (1 - lr wd as a factor would lose the small lr wd: it is added to the update)
        p2 = pair_fma(both(-r.lr), pair_fma(both(t.decay), p2, update), p2);
        unpair(p2, x.p[2 * k], x.p[2 * k + 1]);
        if (!CODES) unpair(m2[k], x.m[2 * k], x.m[2 * k + 1]);
    }
    if (t.master) store8(t.master, i, n, wide, x.p);
    if (t.param_f32) store8((float *)t.param, i, n, wide, x.p);
    else store8((__nv_bfloat16 *)t.param, i, n, wide, x.p);
    if (!CODES) {
        store8((float *)t.m, i, n, wide, x.m);
        store8((float *)t.v, i, n, wide, x.v);
        return;
    }
    uint32_t h[8];
    const uint32_t base = key + (uint32_t)i + (uint32_t)(i >> 32) * 0x9e3779b9u;    // (8 elements share i >> 32)
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = mix(base + j);
    // elements behind the end are zero: codes of zeros stay zeros, gradients were read as zeros
    const float ms = encode<false>(m2, h, x.cm), vs = encode<true>(root2, h, x.cv);
    store_codes(t.m, i, n, wide, x.cm);
    store_codes(t.v, i, n, wide, x.cv);
    if ((threadIdx.x & 31) == 0 && n > 0) {
        t.m_scale[i / kBlockElems] = ms;
        t.v_scale[i / kBlockElems] = vs;
    }
}

template <bool CODES, bool WHOLE>
__device__ __forceinline__ void eight(const Tensor &t, const StepScalars &s, const Rates &r, uint32_t key, int64_t i, int n)
{
    Eight x;
    load_eight<CODES, WHOLE>(t, i, n, x);
    step_eight<CODES, WHOLE>(t, s, r, key, i, n, x);
}

// Blocks take up to kRounds rounds, gridDim.x apart: the blocks at work are
// then next to one another in all of a tensor's buffers.  CODES: for lists with
// any 8-bit moments.
template <int N, bool CODES>
__global__ void __launch_bounds__(NT, CODES ? kCodesResident : kResident)
adamw_kernel(const __grid_constant__ Tensors<N> list, const __grid_constant__ StepScalars s)
{
    chain_begin();
    __shared__ Rates shared;
    __shared__ int tensor[kRounds];
    __shared__ uint32_t keys[kRounds];
    chain_wait();
    if (threadIdx.x < 32) {      // (one warp's instructions, not eight's)
        Rates r;
        r.lr = s.lr_at ? *s.lr_at : s.lr;
        r.factor = s.grad_scale ? *s.grad_scale : 1.f;
        const int64_t step = s.step_at ? *s.step_at : s.step;
        if (threadIdx.x < kRounds) {
            const unsigned round = blockIdx.x + threadIdx.x * gridDim.x;
            const int at = round < (unsigned)list.rounds ? tensor_of(list, (int)round) : 0;
            tensor[threadIdx.x] = at;
            keys[threadIdx.x] = mix(list.t[at].key + (uint32_t)step);
        }
        // 1 - b^t = -expm1(t log b)
        r.r1 = -1.f / expm1f((float)step * s.log_b1);
        r.r2 = rsqrtf(-expm1f((float)step * s.log_b2));
        // gradients without a finite norm, or no step's number: nothing is done
        r.go = fabsf(r.factor) <= 3.4028234e38f && step >= 1;
        shared = r;
    }
    __syncthreads();
    const Rates r = shared;
    if (!r.go) return;
#pragma unroll 1
    for (int k = 0; k < kRounds; ++k) {
        const unsigned round = blockIdx.x + k * gridDim.x;      // (past 2^31 for a list of 2^30)
        if (round >= (unsigned)list.rounds) return;
        const int at = tensor[k];
        const Tensor &t = list.t[at];
        const int64_t base = (int64_t)((int)round - list.first[at]) * kRound, i = base + threadIdx.x * kPer;
        const int n = i >= t.n ? 0 : t.n - i < kPer ? (int)(t.n - i) : kPer;
        const bool whole = t.wide && base + kRound <= t.n;
        if (CODES && t.m_scale) {
            if (whole) eight<true, true>(t, s, r, keys[k], i, kPer);
            else eight<true, false>(t, s, r, keys[k], i, n);
        } else {
            if (whole) eight<false, true>(t, s, r, 0, i, kPer);
            else eight<false, false>(t, s, r, 0, i, n);
        }
    }
}

// ---------------------------------------------------------------- the norm
// sum + low += x (in pairs), the rounding of the addition kept in low (Knuth's
// exact difference of a sum): a thread's fp32 sums are as exact as one in
// double, which the chip has few units for
__device__ __forceinline__ void add_exactly(uint64_t x, uint64_t one, uint64_t &sum, uint64_t &low)
{
    const uint64_t s = pair_sum(one, x, sum), back = pair_sub(s, sum);
    low = pair_add(low, pair_add(pair_sub(sum, pair_sub(s, back)), pair_sum(one, x, pair_sub(0, back))));
    sum = s;
}

__device__ __forceinline__ void add_exactly(float x, float &sum, float &low)
{
    const float s = __fadd_rn(sum, x), back = __fsub_rn(s, sum);
    low = __fadd_rn(low, __fadd_rn(__fsub_rn(sum, __fsub_rn(s, back)), __fsub_rn(x, back)));
    sum = s;
}

__device__ __forceinline__ void add_squares(const float (&g)[8], uint64_t one, uint64_t &sum, uint64_t &low)
{
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        const uint64_t x = pair(g[j], g[j + 1]);
        add_exactly(pair_mul(x, x), one, sum, low);
    }
}

constexpr int kNormRounds = 4;      // rounds of a chunk, all asked for at once
constexpr int kNormResident = 6;    // blocks per SM

// part[block]: the sum of the squares of a range of chunks' gradients
template <int N>
__global__ void __launch_bounds__(NT, kNormResident) square_kernel(const __grid_constant__ GradTensors<N> list, double *part)
{
    chain_begin();
    chain_wait();
    uint64_t sum = 0, low = 0;
    const int end = (int)((int64_t)list.chunks * (blockIdx.x + 1) / gridDim.x);
    int chunk = (int)((int64_t)list.chunks * blockIdx.x / gridDim.x), at = tensor_of(list, chunk);
    for (; chunk < end; ++chunk) {
        while (at + 1 < list.count && list.first[at + 1] <= chunk) ++at;
        const GradTensor &t = list.t[at];
        const int64_t i = (int64_t)(chunk - list.first[at]) * kNormRounds * kRound + threadIdx.x * kPer;
        if (t.wide && !t.f32 && i + (kNormRounds - 1) * kRound + kPer <= t.n) {
            raw_t<__nv_bfloat16, 8> raw[kNormRounds];
#pragma unroll
            for (int k = 0; k < kNormRounds; ++k)
                raw[k] = load_raw<__nv_bfloat16, 8>((const __nv_bfloat16 *)t.grad + i + k * kRound);
#pragma unroll
            for (int k = 0; k < kNormRounds; ++k) {
                float g[8];
                unpack<__nv_bfloat16, 8>(raw[k], g);
                add_squares(g, list.one, sum, low);
            }
        } else {
#pragma unroll
            for (int k = 0; k < kNormRounds; ++k) {
                const int64_t j = i + k * kRound;
                const int n = j >= t.n ? 0 : t.n - j < kPer ? (int)(t.n - j) : kPer;
                float g[8];
                if (t.f32) load8((const float *)t.grad, j, n, t.wide && n == kPer, g);
                else load8((const __nv_bfloat16 *)t.grad, j, n, t.wide && n == kPer, g);
                add_squares(g, list.one, sum, low);
            }
        }
    }
    float s[2], l[2];
    unpair(sum, s[0], s[1]);
    unpair(low, l[0], l[1]);
    float low_sum = l[0] + l[1], high = s[0];
    add_exactly(s[1], high, low_sum);
    // in fp32 as far as it goes: the chip adds two doubles per SM and cycle
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const float other = __shfl_xor_sync(0xffffffffu, high, o);
        low_sum += __shfl_xor_sync(0xffffffffu, low_sum, o);
        add_exactly(other, high, low_sum);
    }
    __shared__ float2 sums[NT / 32];
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = make_float2(high, low_sum);
    __syncthreads();
    if (threadIdx.x == 0) {
        double total = 0.0;
#pragma unroll
        for (int x = 0; x < NT / 32; ++x)      // (an infinite sum has NaN in its low part)
            total += sums[x].x <= 3.4028234e38f ? (double)sums[x].x + (double)sums[x].y : (double)sums[x].x;
        part[blockIdx.x] = total;
    }
}

__global__ void __launch_bounds__(NT) norm_kernel(const double *part, int count, float max_norm, float *norm, float *clip)
{
    chain_begin();
    chain_wait();
    __shared__ double shared[NT / 32];
    double sum = 0.0;
    for (int x = threadIdx.x; x < count; x += NT) sum += part[x];
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        sum = 0.0;
        for (int x = 0; x < NT / 32; ++x) sum += shared[x];
        const float total = (float)sqrt(sum);
        if (norm) *norm = total;
        // (a norm that is not finite gives NaN: a step that takes it as its factor does nothing)
        if (clip) *clip = !(total <= 3.4028234e38f) ? __int_as_float(0x7fffffff) : total > max_norm ? max_norm / total : 1.f;
    }
}

// ---------------------------------------------------------------- host side
size_t up(size_t n) { return (n + 255) / 256 * 256; }

// a pair of the same number, as the kernels hold it
uint64_t twice(float x)
{
    uint32_t b;
    memcpy(&b, &x, 4);
    return (uint64_t)b << 32 | b;
}

txl_status finish(cudaError_t e)
{
    if (e == cudaSuccess) return TXL_OK;
    note_cuda_error(e);
    return TXL_ERR_CUDA;
}

bool dtype_known(txl_dtype t) { return t == TXL_F32 || t == TXL_BF16; }
size_t size_of(txl_dtype t) { return t == TXL_F32 ? 4 : 2; }

int64_t chunks_of(int64_t n, int rounds) { return (n + (int64_t)rounds * kRound - 1) / ((int64_t)rounds * kRound); }

txl_status check_ranges(std::vector<CallBuffer> &ins, std::vector<CallBuffer> &outs)
{
    for (const auto *list : {&ins, &outs})
        for (const CallBuffer &b : *list)
            if ((b.need && b.bytes && !b.p) || !at_boundary(b.p, b.align)) return TXL_ERR_INVALID;
    // outputs overlap neither one another nor an input: in order of address, an output's end may
    // lie behind no later buffer's start, an input's behind no later output's
    struct Range {
        uintptr_t from, to;
        bool out;
    };
    std::vector<Range> all;
    all.reserve(ins.size() + outs.size());
    for (const CallBuffer &b : ins)
        if (b.p && b.bytes) all.push_back({(uintptr_t)b.p, (uintptr_t)b.p + b.bytes, false});
    for (const CallBuffer &b : outs)
        if (b.p && b.bytes) all.push_back({(uintptr_t)b.p, (uintptr_t)b.p + b.bytes, true});
    std::sort(all.begin(), all.end(), [](const Range &a, const Range &b) { return a.from < b.from; });
    uintptr_t end_in = 0, end_out = 0;
    for (const Range &r : all) {
        if (r.from < end_out || (r.out && r.from < end_in)) return TXL_ERR_INVALID;
        uintptr_t &end = r.out ? end_out : end_in;
        end = std::max(end, r.to);
    }
    return TXL_OK;
}

// a tensor's buffers: its gradient, and what the step writes
constexpr int kBuffers = 7;
CallBuffer buffer_of(const txl_adamw_tensor &x, int which)
{
    const size_t n = (size_t)x.size, blocks = (n + kBlockElems - 1) / kBlockElems;
    const bool codes = x.exp_avg_scale != nullptr;
    const size_t p = size_of(x.param_dtype), g = size_of(x.grad_dtype), m = codes ? 1 : 4;
    switch (which) {
    case 0: return {x.grad, n * g, g, true};
    case 1: return {x.param, n * p, p, true};
    case 2: return {x.master, n * 4, 4, false};
    case 3: return {x.exp_avg, n * m, m, true};
    case 4: return {x.exp_avg_sq, n * m, m, true};
    case 5: return {x.exp_avg_scale, blocks * 4, 4, codes};
    default: return {x.exp_avg_sq_scale, blocks * 4, 4, codes};
    }
}

// Whether the buffers are aligned and plainly apart: those of each kind in
// order of address, and no kind's whole range over another's or over a scalar
// (tensors that are parts of one allocation per kind).  Otherwise check_ranges
// decides, which sorts them: 20 us of a call over 270 tensors.
template <size_t S>
bool apart(const txl_adamw_tensor *t, const std::vector<int> &order, const CallBuffer (&scalars)[S])
{
    uintptr_t from[kBuffers + S], to[kBuffers + S];
    int ranges = 0;
    for (int which = 0; which < kBuffers; ++which) {
        uintptr_t begin = 0, end = 0;
        for (int k : order) {
            const CallBuffer b = buffer_of(t[k], which);
            if (!b.p) {
                if (b.need) return false;
                continue;
            }
            const uintptr_t at = (uintptr_t)b.p;
            if (at < end || !at_boundary(b.p, b.align)) return false;
            if (!begin) begin = at;
            end = at + b.bytes;
        }
        if (begin) from[ranges] = begin, to[ranges++] = end;
    }
    for (const CallBuffer &b : scalars) {
        if (!at_boundary(b.p, b.align)) return false;
        if (b.p) from[ranges] = (uintptr_t)b.p, to[ranges++] = (uintptr_t)b.p + b.bytes;
    }
    for (int x = 0; x < ranges; ++x)
        for (int y = 0; y < x; ++y)
            if (from[x] < to[y] && from[y] < to[x]) return false;
    return true;
}

txl_status tensors_known(int tensors, const txl_adamw_tensor *t)
{
    if (tensors < 0 || (tensors > 0 && !t)) return TXL_ERR_INVALID;
    for (int k = 0; k < tensors; ++k) {
        if (t[k].size < 0) return TXL_ERR_INVALID;
        if (!dtype_known(t[k].param_dtype) || !dtype_known(t[k].grad_dtype) || t[k].size > kMaxElements)
            return TXL_ERR_UNSUPPORTED;
    }
    return TXL_OK;
}

template <int N>
cudaError_t launch_step(const txl_adamw_tensor *t, const int *order, int count, uint32_t seed, const StepScalars &sc,
                        cudaStream_t s)
{
    Tensors<N> list;
    int rounds = 0;
    bool codes = false;
    for (int k = 0; k < count; ++k) {
        const txl_adamw_tensor &x = t[order[k]];
        Tensor &y = list.t[k];
        y.param = x.param;
        y.master = x.master;
        y.grad = x.grad;
        y.m = x.exp_avg;
        y.v = x.exp_avg_sq;
        y.m_scale = x.exp_avg_scale;
        y.v_scale = x.exp_avg_sq_scale;
        y.n = x.size;
        y.decay = x.weight_decay;
        list.first[k] = rounds;
        y.key = mix(seed + (uint32_t)order[k]);
        y.param_f32 = x.param_dtype == TXL_F32;
        y.grad_f32 = x.grad_dtype == TXL_F32;
        const uintptr_t state = y.m_scale ? 8 : 16;
        y.wide = at_boundary(y.param, 16) && at_boundary(y.master, 16) && at_boundary(y.grad, 16) &&
                 at_boundary(y.m, state) && at_boundary(y.v, state);
        rounds += (int)chunks_of(x.size, 1);
        codes = codes || y.m_scale;
    }
    list.count = count;
    list.rounds = rounds;
    // One round per block where that is few blocks.  Several where they are many, for fewer searches
    // and rates: 2 and 4 rounds take 106 and 100 us for 34 M weights with 8-bit moments, but 1004
    // and 1014 us for 229 M with 32-bit ones, which have less to compute.
    const int per = rounds <= 152 * 16 ? 1 : codes ? kRounds : 2;
    return chain_launch(codes ? adamw_kernel<N, true> : adamw_kernel<N, false>, (unsigned)((rounds + per - 1) / per), NT, 0,
                        1, s, list, sc);
}

template <int N>
cudaError_t launch_squares(const txl_adamw_tensor *t, const int *order, int count, unsigned blocks, double *part,
                           cudaStream_t s)
{
    GradTensors<N> list;
    int chunks = 0;
    for (int k = 0; k < count; ++k) {
        const txl_adamw_tensor &x = t[order[k]];
        GradTensor &y = list.t[k];
        y.grad = x.grad;
        y.n = x.size;
        list.first[k] = chunks;
        y.f32 = x.grad_dtype == TXL_F32;
        y.wide = at_boundary(x.grad, 16);
        chunks += (int)chunks_of(x.size, kNormRounds);
    }
    list.count = count;
    list.chunks = chunks;
    list.one = twice(1.f);
    return chain_launch(square_kernel<N>, blocks, NT, 0, 1, s, list, part);
}

// The launches of a call: its tensors with elements, so many per launch that
// neither they nor their chunks are too many.
struct Launch {
    int at, count;               // in the order of the tensors
    int64_t chunks;
};

struct Launches {
    std::vector<int> order;
    std::vector<Launch> each;
};

void deal(int tensors, const txl_adamw_tensor *t, int rounds, Launches *l)
{
    l->order.reserve(tensors);
    for (int k = 0; k < tensors; ++k)
        if (t[k].size > 0) l->order.push_back(k);
    for (int at = 0; at < (int)l->order.size();) {
        Launch one = {at, 0, 0};
        while (at < (int)l->order.size() && one.count < kMostTensors) {
            const int64_t more = chunks_of(t[l->order[at]].size, rounds);
            if (one.count && one.chunks + more > (1 << 30)) break;
            one.chunks += more;
            ++one.count;
            ++at;
        }
        l->each.push_back(one);
    }
}

// Blocks of a launch of the norm: what the SMs hold at once, so that the last
// launch has few sums to add.
constexpr int64_t kNormBlocks = 152 * kNormResident;
unsigned norm_blocks(const Launch &l) { return (unsigned)std::min(l.chunks, kNormBlocks); }

size_t norm_bytes(const Launches &l)
{
    size_t blocks = 0;
    for (const Launch &x : l.each) blocks += norm_blocks(x);
    return up(blocks * sizeof(double));
}

txl_status grad_norm(int tensors, const txl_adamw_tensor *t, float max_norm, float *norm, float *clip, void *workspace,
                     size_t workspace_bytes, cudaStream_t s)
{
    txl_status st = tensors_known(tensors, t);
    if (st != TXL_OK) return st;
    if (!(max_norm > 0.f)) return TXL_ERR_INVALID;
    if (!norm && !clip) return TXL_OK;
    Launches l;
    deal(tensors, t, kNormRounds, &l);
    const size_t need = norm_bytes(l);
    std::vector<CallBuffer> ins, outs;
    ins.reserve(l.order.size());
    for (int k : l.order) ins.push_back({t[k].grad, (size_t)t[k].size * size_of(t[k].grad_dtype), size_of(t[k].grad_dtype), true});
    outs.push_back({norm, 4, 4, false});
    outs.push_back({clip, 4, 4, false});
    outs.push_back({workspace, need, 256, need > 0});
    st = check_ranges(ins, outs);
    if (st != TXL_OK) return st;
    if (workspace_bytes < need) return TXL_ERR_INVALID;
    cudaError_t e = cudaSuccess;
    int blocks = 0;
    for (const Launch &x : l.each) {
        double *part = (double *)workspace + blocks;
        blocks += (int)norm_blocks(x);
        e = x.count <= kFewTensors ? launch_squares<kFewTensors>(t, &l.order[x.at], x.count, norm_blocks(x), part, s)
                                   : launch_squares<kMostTensors>(t, &l.order[x.at], x.count, norm_blocks(x), part, s);
        if (e != cudaSuccess) return finish(e);
    }
    return finish(chain_launch(norm_kernel, 1, NT, 0, 1, s, (const double *)workspace, blocks, max_norm, norm, clip));
}

txl_status adamw_step(int tensors, const txl_adamw_tensor *t, const txl_adamw_options *o, cudaStream_t s)
{
    txl_status st = tensors_known(tensors, t);
    if (st != TXL_OK) return st;
    if (!o) return TXL_ERR_INVALID;
    if (!(o->beta1 >= 0.0 && o->beta1 < 1.0 && o->beta2 >= 0.0 && o->beta2 < 1.0)) return TXL_ERR_INVALID;
    if (!(o->eps >= 0x1p-126f && o->eps <= 3.4028234e38f)) return TXL_ERR_INVALID;
    if (!o->step_device && o->step < 1) return TXL_ERR_INVALID;
    if (!o->lr_device && !(o->lr >= 0.f && o->lr <= 3.4028234e38f)) return TXL_ERR_INVALID;
    Launches l;
    deal(tensors, t, 1, &l);
    for (int k : l.order) {
        const txl_adamw_tensor &x = t[k];
        if ((x.exp_avg_scale != nullptr) != (x.exp_avg_sq_scale != nullptr)) return TXL_ERR_INVALID;
        if (x.master && x.param_dtype == TXL_F32) return TXL_ERR_INVALID;
        if (!(x.weight_decay >= 0.f && x.weight_decay <= 3.4028234e38f)) return TXL_ERR_INVALID;
    }
    const CallBuffer scalars[] = {{o->lr_device, 4, 4, false}, {o->grad_scale, 4, 4, false}, {o->step_device, 8, 8, false}};
    if (!apart(t, l.order, scalars)) {
        std::vector<CallBuffer> ins(std::begin(scalars), std::end(scalars)), outs;
        ins.reserve(l.order.size() + 3);
        outs.reserve(l.order.size() * 6);
        for (int k : l.order)
            for (int which = 0; which < kBuffers; ++which) (which ? outs : ins).push_back(buffer_of(t[k], which));
        st = check_ranges(ins, outs);
        if (st != TXL_OK) return st;
    }
    StepScalars sc;
    sc.lr_at = o->lr_device;
    sc.grad_scale = o->grad_scale;
    sc.step_at = o->step_device;
    sc.lr = o->lr;
    sc.b1 = twice((float)o->beta1);
    sc.b2 = twice((float)o->beta2);
    sc.c1 = twice((float)(1.0 - o->beta1));
    sc.c2 = twice((float)(1.0 - o->beta2));
    sc.log_b1 = (float)log(o->beta1);
    sc.log_b2 = (float)log(o->beta2);
    sc.eps = twice(o->eps);
    sc.one = twice(1.f);
    sc.step = o->step;
    const uint32_t seed = mix(mix((uint32_t)o->seed) + (uint32_t)(o->seed >> 32));
    for (const Launch &x : l.each) {
        const int *order = &l.order[x.at];
        const cudaError_t e = x.count <= kFewTensors ? launch_step<kFewTensors>(t, order, x.count, seed, sc, s)
                                                     : launch_step<kMostTensors>(t, order, x.count, seed, sc, s);
        if (e != cudaSuccess) return finish(e);
    }
    return TXL_OK;
}

}  // namespace
}  // namespace txl

using namespace txl;

extern "C" {

txl_status txl_grad_norm_workspace(int tensors, const txl_adamw_tensor *t, size_t *bytes)
{
    if (!bytes) return TXL_ERR_INVALID;
    const txl_status st = tensors_known(tensors, t);
    if (st != TXL_OK) return st;
    try {
        Launches l;
        deal(tensors, t, kNormRounds, &l);
        *bytes = std::max(norm_bytes(l), (size_t)256);
    } catch (const std::bad_alloc &) {
        return TXL_ERR_UNSUPPORTED;
    }
    return TXL_OK;
}

txl_status txl_grad_norm(int tensors, const txl_adamw_tensor *t, float max_norm, float *norm, float *clip,
                         void *workspace, size_t workspace_bytes, void *stream)
{
    try {
        return grad_norm(tensors, t, max_norm, norm, clip, workspace, workspace_bytes, (cudaStream_t)stream);
    } catch (const std::bad_alloc &) {
        return TXL_ERR_UNSUPPORTED;
    }
}

txl_status txl_adamw_step(int tensors, const txl_adamw_tensor *t, const txl_adamw_options *options, void *stream)
{
    try {
        return adamw_step(tensors, t, options, (cudaStream_t)stream);
    } catch (const std::bad_alloc &) {
        return TXL_ERR_UNSUPPORTED;
    }
}

}  // extern "C"

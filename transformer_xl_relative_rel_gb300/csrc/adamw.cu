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
// kernel argument (up to kMostTensors of them), work is cut into chunks, and
// a block finds its chunk's tensor by bisection.
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

#include <algorithm>
#include <new>
#include <vector>

#include "buffers.h"
#include "chain.h"
#include "internal.h"
#include "rows.cuh"

namespace txl {
namespace {

constexpr int NT = 256;
constexpr int kPer = 8;                         // elements per thread and round
constexpr int kRound = NT * kPer;
constexpr int kBlockElems = 256;                // elements that share a scale: one warp's
constexpr float kTop = 448.f;                   // the largest e4m3 value
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
    int first;               // its first chunk in the launch
    uint32_t key;            // of its random numbers
    uint8_t param_f32, grad_f32, wide, pad;   // wide: every buffer at a 16-byte boundary (codes: 8)
};

template <int N>
struct Tensors {
    Tensor t[N];
    int count, chunks, rounds;   // a chunk is so many rounds of kRound elements
};

struct GradTensor {
    const void *grad;
    int64_t n;
    int first;
    uint8_t f32, wide, pad[2];
};

template <int N>
struct GradTensors {
    GradTensor t[N];
    int count, chunks, rounds;
};

struct StepScalars {
    const float *lr_at, *grad_scale;
    const int64_t *step_at;
    float lr, b1, b2, c1, c2;        // c1 = 1 - b1, c2 = 1 - b2
    float log_b1, log_b2, eps;
    int64_t step;
};

__host__ __device__ __forceinline__ uint32_t mix(uint32_t x)
{
    x = (x ^ (x >> 16)) * 0x7feb352du;
    x = (x ^ (x >> 15)) * 0x846ca68bu;
    return x ^ (x >> 16);
}

template <typename List>
__device__ __forceinline__ int tensor_of(const List &l, int chunk)
{
    int lo = 0, hi = l.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (l.t[mid].first <= chunk) lo = mid;
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

__device__ __forceinline__ void load_codes(const void *p, int64_t i, int n, bool wide, float scale, float (&x)[8])
{
    const uint8_t *c = (const uint8_t *)p + i;
    uint8_t raw[8];
    if (wide) {
        *reinterpret_cast<uint2 *>(raw) = *reinterpret_cast<const uint2 *>(c);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) raw[j] = j < n ? c[j] : 0;
    }
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(raw[j] | raw[j + 1] << 8), __NV_E4M3);
        const float2 f = __half22float2(__half2(h));
        x[j] = __fmul_rn(f.x, scale);
        x[j + 1] = __fmul_rn(f.y, scale);
    }
}

// |y| <= 448 (1 + 2^-22), or NaN, to one of its two neighbours in e4m3: up
// where the fraction of the way and u make a whole
__device__ __forceinline__ float round_code(float y, float u, bool keep)
{
    const uint32_t mag = __float_as_uint(y) & 0x7fffffffu;
    const uint32_t e = max(mag & 0x7f800000u, (127u - 6u) << 23);
    // neighbours are 2^(exponent - 3) apart (the product is exact)
    float steps = floorf(fmaf(__uint_as_float(mag), __uint_as_float((257u << 23) - e), u));
    if (keep && mag != 0 && steps == 0.f) steps = 1.f;
    const float value = steps * __uint_as_float(e - (3u << 23));
    return copysignf(value > kTop ? kTop : value, y);      // (NaN stays NaN)
}

// the warp's 256 elements (8 per lane) as codes times one scale; h: random bits
template <bool ROOT>
__device__ __forceinline__ void store_codes(void *p, float *scale, int64_t i, int n, bool wide, const float (&x)[8],
                                            const uint32_t (&h)[8])
{
    float top = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(x[j]));
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (top < 0x1p-100f) top = 0.f;
    const float inverse = top > 0.f ? __fmul_rn(__frcp_rn(top), kTop) : 0.f;
    uint8_t raw[8];
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        float2 f;
        const float u0 = (ROOT ? h[j] >> 16 : h[j] & 0xffffu) * 0x1p-16f;
        const float u1 = (ROOT ? h[j + 1] >> 16 : h[j + 1] & 0xffffu) * 0x1p-16f;
        f.x = round_code(__fmul_rn(x[j], inverse), u0, ROOT);
        f.y = round_code(__fmul_rn(x[j + 1], inverse), u1, ROOT);
        const uint16_t c = __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
        raw[j] = (uint8_t)c;
        raw[j + 1] = (uint8_t)(c >> 8);
    }
    uint8_t *c = (uint8_t *)p + i;
    if (wide) {
        *reinterpret_cast<uint2 *>(c) = *reinterpret_cast<const uint2 *>(raw);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n) c[j] = raw[j];
    }
    if ((threadIdx.x & 31) == 0 && n > 0) *scale = __fmul_rn(top, 1.f / kTop);
}

// ---------------------------------------------------------------- the step
template <int N>
__global__ void __launch_bounds__(NT)
adamw_kernel(const __grid_constant__ Tensors<N> list, const __grid_constant__ StepScalars s)
{
    chain_begin();
    const Tensor &t = list.t[tensor_of(list, blockIdx.x)];
    chain_wait();
    const float lr = s.lr_at ? *s.lr_at : s.lr;
    const int64_t step = s.step_at ? *s.step_at : s.step;
    const float factor = s.grad_scale ? *s.grad_scale : 1.f;
    // gradients without a finite norm, or no step's number: nothing is done
    if (!(fabsf(factor) <= 3.4028234e38f) || step < 1) return;
    // 1 - b^t = -expm1(t log b)
    const float r1 = -1.f / expm1f((float)step * s.log_b1), r2 = rsqrtf(-expm1f((float)step * s.log_b2));
    const uint32_t key = mix(t.key + (uint32_t)step);
    const bool codes = t.m_scale != nullptr;
    const int64_t first = (int64_t)(blockIdx.x - t.first) * list.rounds * kRound;
    for (int round = 0; round < list.rounds; ++round) {
        const int64_t base = first + (int64_t)round * kRound;
        if (base >= t.n) return;
        const int64_t i = base + threadIdx.x * kPer;
        const int n = i >= t.n ? 0 : t.n - i < kPer ? (int)(t.n - i) : kPer;
        const bool wide = t.wide && n == kPer;
        const int64_t block = i / kBlockElems;       // (the same for a warp)
        float g[8], p[8], m[8], v[8];
        if (t.grad_f32) load8((const float *)t.grad, i, n, wide, g);
        else load8((const __nv_bfloat16 *)t.grad, i, n, wide, g);
        if (t.master) load8((const float *)t.master, i, n, wide, p);
        else if (t.param_f32) load8((const float *)t.param, i, n, wide, p);
        else load8((const __nv_bfloat16 *)t.param, i, n, wide, p);
        if (codes) {
            const bool any = block * kBlockElems < t.n;
            load_codes(t.m, i, n, wide, any ? t.m_scale[block] : 0.f, m);
            load_codes(t.v, i, n, wide, any ? t.v_scale[block] : 0.f, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(v[j], v[j]);
        } else {
            load8((const float *)t.m, i, n, wide, m);
            load8((const float *)t.v, i, n, wide, v);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            g[j] = __fmul_rn(g[j], factor);
            m[j] = __fadd_rn(__fmul_rn(s.b1, m[j]), __fmul_rn(s.c1, g[j]));
            v[j] = __fadd_rn(__fmul_rn(s.b2, v[j]), __fmul_rn(__fmul_rn(s.c2, g[j]), g[j]));
            const float root = __fsqrt_rn(v[j]);
            // (1 - lr wd as a factor would lose the small lr wd: it is added to the update)
            p[j] = fmaf(-lr, fmaf(t.decay, p[j], m[j] * r1 / fmaf(root, r2, s.eps)), p[j]);
            if (codes) v[j] = root;
        }
        if (t.master) store8(t.master, i, n, wide, p);
        if (t.param_f32) store8((float *)t.param, i, n, wide, p);
        else store8((__nv_bfloat16 *)t.param, i, n, wide, p);
        if (codes) {
            uint32_t h[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                h[j] = mix(key + (uint32_t)(i + j) + (uint32_t)(i >> 32) * 0x9e3779b9u);
            store_codes<false>(t.m, t.m_scale + block, i, n, wide, m, h);
            store_codes<true>(t.v, t.v_scale + block, i, n, wide, v, h);
        } else {
            store8((float *)t.m, i, n, wide, m);
            store8((float *)t.v, i, n, wide, v);
        }
    }
}

// ---------------------------------------------------------------- the norm
__device__ __forceinline__ double block_sum(double v)
{
    __shared__ double part[NT / 32];
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int x = 0; x < NT / 32; ++x) v += part[x];
    return v;
}

// sum + low += x, the rounding of the addition kept in low (Knuth's exact
// difference of a sum): a thread's fp32 sum as exact as one in double, which
// the chip has few units for
__device__ __forceinline__ void add_exactly(float x, float &sum, float &low)
{
    const float s = __fadd_rn(sum, x), back = __fsub_rn(s, sum);
    low = __fadd_rn(low, __fadd_rn(__fsub_rn(sum, __fsub_rn(s, back)), __fsub_rn(x, back)));
    sum = s;
}

// part[chunk]: the sum of the squares of a chunk's gradients
template <int N>
__global__ void __launch_bounds__(NT) square_kernel(const __grid_constant__ GradTensors<N> list, double *part)
{
    chain_begin();
    const GradTensor &t = list.t[tensor_of(list, blockIdx.x)];
    chain_wait();
    const int64_t first = (int64_t)(blockIdx.x - t.first) * list.rounds * kRound;
    float sum = 0.f, low = 0.f;
    for (int round = 0; round < list.rounds; ++round) {
        const int64_t i = first + (int64_t)round * kRound + threadIdx.x * kPer;
        const int n = i >= t.n ? 0 : t.n - i < kPer ? (int)(t.n - i) : kPer;
        float g[8];
        if (t.f32) load8((const float *)t.grad, i, n, t.wide && n == kPer, g);
        else load8((const __nv_bfloat16 *)t.grad, i, n, t.wide && n == kPer, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) add_exactly(__fmul_rn(g[j], g[j]), sum, low);
    }
    // (an infinite sum has NaN in low)
    const double total = block_sum(sum <= 3.4028234e38f ? (double)sum + (double)low : (double)sum);
    if (threadIdx.x == 0) part[blockIdx.x] = total;
}

__global__ void __launch_bounds__(1024) norm_kernel(const double *part, long count, float max_norm, float *norm, float *clip)
{
    chain_begin();
    chain_wait();
    __shared__ double shared[32];
    double sum = 0.0;
    for (long x = threadIdx.x; x < count; x += 1024) sum += part[x];
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        sum = 0.0;
        for (int x = 0; x < 32; ++x) sum += shared[x];
        const float total = (float)sqrt(sum);
        if (norm) *norm = total;
        // (a norm that is not finite gives NaN: a step that takes it as its factor does nothing)
        if (clip) *clip = !(total <= 3.4028234e38f) ? __int_as_float(0x7fffffff) : total > max_norm ? max_norm / total : 1.f;
    }
}

// ---------------------------------------------------------------- host side
size_t up(size_t n) { return (n + 255) / 256 * 256; }

txl_status finish(cudaError_t e)
{
    if (e == cudaSuccess) return TXL_OK;
    note_cuda_error(e);
    return TXL_ERR_CUDA;
}

bool dtype_known(txl_dtype t) { return t == TXL_F32 || t == TXL_BF16; }
size_t size_of(txl_dtype t) { return t == TXL_F32 ? 4 : 2; }

// Rounds per chunk: one where that leaves every SM no more than some blocks,
// up to 4 where blocks are many (fewer searches).
int rounds_for(int64_t elements)
{
    const int64_t rounds = (elements + kRound - 1) / kRound;
    return rounds <= 152 * 16 ? 1 : 4;
}

// (chunks of all launches together, which the norm's workspace holds a double for each of)
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
cudaError_t launch_step(const txl_adamw_tensor *t, const int *order, int count, int rounds, uint32_t seed,
                        const StepScalars &sc, cudaStream_t s)
{
    Tensors<N> list;
    int chunks = 0;
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
        y.first = chunks;
        y.key = mix(seed + (uint32_t)order[k]);
        y.param_f32 = x.param_dtype == TXL_F32;
        y.grad_f32 = x.grad_dtype == TXL_F32;
        const uintptr_t state = y.m_scale ? 8 : 16;
        y.wide = at_boundary(y.param, 16) && at_boundary(y.master, 16) && at_boundary(y.grad, 16) &&
                 at_boundary(y.m, state) && at_boundary(y.v, state);
        y.pad = 0;
        chunks += (int)chunks_of(x.size, rounds);
    }
    list.count = count;
    list.chunks = chunks;
    list.rounds = rounds;
    return chain_launch(adamw_kernel<N>, (unsigned)chunks, NT, 0, 1, s, list, sc);
}

template <int N>
cudaError_t launch_squares(const txl_adamw_tensor *t, const int *order, int count, int rounds, double *part, cudaStream_t s)
{
    GradTensors<N> list;
    int chunks = 0;
    for (int k = 0; k < count; ++k) {
        const txl_adamw_tensor &x = t[order[k]];
        GradTensor &y = list.t[k];
        y.grad = x.grad;
        y.n = x.size;
        y.first = chunks;
        y.f32 = x.grad_dtype == TXL_F32;
        y.wide = at_boundary(x.grad, 16);
        y.pad[0] = y.pad[1] = 0;
        chunks += (int)chunks_of(x.size, rounds);
    }
    list.count = count;
    list.chunks = chunks;
    list.rounds = rounds;
    return chain_launch(square_kernel<N>, (unsigned)chunks, NT, 0, 1, s, list, part);
}

// how a call's tensors are dealt out to launches
struct Launches {
    std::vector<int> order;      // the tensors with elements
    int64_t total = 0, chunks = 0;
    int rounds = 1;
};

void deal(int tensors, const txl_adamw_tensor *t, Launches *l)
{
    for (int k = 0; k < tensors; ++k)
        if (t[k].size > 0) {
            l->order.push_back(k);
            l->total += t[k].size;
        }
    l->rounds = rounds_for(l->total);
    for (int k : l->order) l->chunks += chunks_of(t[k].size, l->rounds);
}

// calls launch(first, count, chunks before) for groups of at most kMostTensors tensors
template <typename F>
cudaError_t each_launch(const Launches &l, const txl_adamw_tensor *t, F launch)
{
    int64_t before = 0;
    for (size_t at = 0; at < l.order.size();) {
        int count = 0;
        int64_t chunks = 0;
        while (at + count < l.order.size() && count < kMostTensors) {
            const int64_t more = chunks_of(t[l.order[at + count]].size, l.rounds);
            if (count && chunks + more > INT32_MAX) break;
            chunks += more;
            ++count;
        }
        const cudaError_t e = launch((int)at, count, before);
        if (e != cudaSuccess) return e;
        before += chunks;
        at += count;
    }
    return cudaSuccess;
}

txl_status grad_norm(int tensors, const txl_adamw_tensor *t, float max_norm, float *norm, float *clip, void *workspace,
                     size_t workspace_bytes, cudaStream_t s)
{
    txl_status st = tensors_known(tensors, t);
    if (st != TXL_OK) return st;
    if (!(max_norm > 0.f)) return TXL_ERR_INVALID;
    if (!norm && !clip) return TXL_OK;
    Launches l;
    deal(tensors, t, &l);
    const size_t need = up((size_t)l.chunks * 8);
    std::vector<CallBuffer> ins, outs;
    for (int k : l.order) ins.push_back({t[k].grad, (size_t)t[k].size * size_of(t[k].grad_dtype), size_of(t[k].grad_dtype), true});
    outs.push_back({norm, 4, 4, false});
    outs.push_back({clip, 4, 4, false});
    outs.push_back({workspace, need, 256, need > 0});
    st = check_ranges(ins, outs);
    if (st != TXL_OK) return st;
    if (workspace_bytes < need) return TXL_ERR_INVALID;
    cudaError_t e = each_launch(l, t, [&](int at, int count, int64_t before) {
        double *part = (double *)workspace + before;
        return count <= kFewTensors ? launch_squares<kFewTensors>(t, &l.order[at], count, l.rounds, part, s)
                                    : launch_squares<kMostTensors>(t, &l.order[at], count, l.rounds, part, s);
    });
    if (e == cudaSuccess)
        e = chain_launch(norm_kernel, 1, 1024, 0, 1, s, (const double *)workspace, (long)l.chunks, max_norm, norm, clip);
    return finish(e);
}

txl_status adamw_step(int tensors, const txl_adamw_tensor *t, const txl_adamw_options *o, cudaStream_t s)
{
    txl_status st = tensors_known(tensors, t);
    if (st != TXL_OK) return st;
    if (!o) return TXL_ERR_INVALID;
    if (!(o->beta1 >= 0.0 && o->beta1 < 1.0 && o->beta2 >= 0.0 && o->beta2 < 1.0)) return TXL_ERR_INVALID;
    if (!(o->eps > 0.f && o->eps <= 3.4028234e38f)) return TXL_ERR_INVALID;
    if (!o->step_device && o->step < 1) return TXL_ERR_INVALID;
    if (!o->lr_device && !(o->lr >= 0.f && o->lr <= 3.4028234e38f)) return TXL_ERR_INVALID;
    Launches l;
    deal(tensors, t, &l);
    std::vector<CallBuffer> ins, outs;
    outs.reserve(l.order.size() * 6);
    for (int k : l.order) {
        const txl_adamw_tensor &x = t[k];
        const size_t n = (size_t)x.size, blocks = (n + kBlockElems - 1) / kBlockElems;
        const bool codes = x.exp_avg_scale != nullptr;
        if (codes != (x.exp_avg_sq_scale != nullptr) || (x.master && x.param_dtype == TXL_F32)) return TXL_ERR_INVALID;
        if (!(x.weight_decay >= 0.f && x.weight_decay <= 3.4028234e38f)) return TXL_ERR_INVALID;
        const size_t p = size_of(x.param_dtype), g = size_of(x.grad_dtype), m = codes ? 1 : 4;
        ins.push_back({x.grad, n * g, g, true});
        outs.push_back({x.param, n * p, p, true});
        outs.push_back({x.master, n * 4, 4, false});
        outs.push_back({x.exp_avg, n * m, m, true});
        outs.push_back({x.exp_avg_sq, n * m, m, true});
        if (codes) {
            outs.push_back({x.exp_avg_scale, blocks * 4, 4, true});
            outs.push_back({x.exp_avg_sq_scale, blocks * 4, 4, true});
        }
    }
    ins.push_back({o->lr_device, 4, 4, false});
    ins.push_back({o->grad_scale, 4, 4, false});
    ins.push_back({o->step_device, 8, 8, false});
    st = check_ranges(ins, outs);
    if (st != TXL_OK) return st;
    StepScalars sc;
    sc.lr_at = o->lr_device;
    sc.grad_scale = o->grad_scale;
    sc.step_at = o->step_device;
    sc.lr = o->lr;
    sc.b1 = (float)o->beta1;
    sc.b2 = (float)o->beta2;
    sc.c1 = (float)(1.0 - o->beta1);
    sc.c2 = (float)(1.0 - o->beta2);
    sc.log_b1 = (float)log(o->beta1);
    sc.log_b2 = (float)log(o->beta2);
    sc.eps = o->eps;
    sc.step = o->step;
    const uint32_t seed = mix(mix((uint32_t)o->seed) + (uint32_t)(o->seed >> 32));
    return finish(each_launch(l, t, [&](int at, int count, int64_t) {
        return count <= kFewTensors ? launch_step<kFewTensors>(t, &l.order[at], count, l.rounds, seed, sc, s)
                                    : launch_step<kMostTensors>(t, &l.order[at], count, l.rounds, seed, sc, s);
    }));
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
        deal(tensors, t, &l);
        *bytes = up((size_t)l.chunks * 8 + 1);
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

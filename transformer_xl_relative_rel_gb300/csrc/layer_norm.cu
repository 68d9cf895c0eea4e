// layer_norm.cu -- layer norm of a residual sum, and its gradients.
//
//     s = x + residual            (rounded to the element type where it is kept, and then used as kept)
//     y = (s - mean) rstd gamma + beta,  rstd = 1 / sqrt(var + eps)
//     ds = rstd (g - mean_d(g) - xh mean_d(g xh)) + dsum,   g = dy gamma, xh = (s - mean) rstd
//     dgamma = sum_i dy xh, dbeta = sum_i dy
//
// HBM-bound: a row is read once and stays in registers, as fp32, from its
// loads to its result; G threads share it (a warp up to 1024 columns).  The
// variance is the mean of the squared differences from the mean.  The
// backward's groups of threads each take many rows and keep their columns'
// sums for dgamma and dbeta in registers; a block adds its groups' up and
// writes them, and a second launch adds the blocks' in a fixed order.
#include <cuda_runtime.h>
#include <stdint.h>

#include "buffers.h"
#include "chain.h"
#include "internal.h"
#include "rows.cuh"

namespace txl {
namespace {

constexpr int kMaxRows = 1 << 30;
constexpr int kMaxNormWidth = 8192;    // 1024 threads hold 8 columns each
constexpr int kMostBlocks = 304;       // of the backward: two per SM
constexpr int kWarpBlock = 256;        // threads of a block whose warps take a row each

struct NormArgs {
    const void *x, *residual, *dy, *dsum;
    const float *gamma, *beta;
    void *out, *sum;            // y or dx; the kept sum
    float *mean, *rstd;
    float *part;                // [blocks][2][pitch] column sums
    float eps;
    int rows, d, pitch, weights;
};

// the sum of v over the group's G threads
template <int G>
__device__ __forceinline__ float group_sum(float v, float *shared)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if constexpr (G > 32) {
        const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
        __syncthreads();          // (the places may still be read)
        if (lane == 0) shared[w] = v;
        __syncthreads();
        v = lane < G / 32 ? shared[lane] : 0.f;
#pragma unroll
        for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    }
    return v;
}

// threads of a block: 8 groups of a warp, or one group
template <int G>
constexpr int kBlock = G == 32 ? kWarpBlock : G;

template <typename T, int V, int K, int G>
__global__ void __launch_bounds__(kBlock<G>) norm_fwd_kernel(const __grid_constant__ NormArgs a)
{
    chain_begin();
    __shared__ float shared[32];
    const int t = G == 32 ? threadIdx.x & 31 : threadIdx.x;
    const long row = G == 32 ? (long)blockIdx.x * (kWarpBlock / 32) + (threadIdx.x >> 5) : (long)blockIdx.x;
    chain_wait();
    if (row >= a.rows) return;    // (a whole group)
    const T *x = (const T *)a.x + row * a.d, *res = (const T *)a.residual + row * a.d;
    float s[K][V];
    raw_t<T, V> raw[K], raw2[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (k * G + t) * V;
        if (c < a.d) {
            raw[k] = load_raw<T, V>(x + c);
            if (a.residual) raw2[k] = load_raw<T, V>(res + c);
        }
    }
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (k * G + t) * V;
#pragma unroll
        for (int i = 0; i < V; ++i) s[k][i] = 0.f;
        if (c < a.d) {
            unpack<T, V>(raw[k], s[k]);
            if (a.residual) {
                float r[V];
                unpack<T, V>(raw2[k], r);
#pragma unroll
                for (int i = 0; i < V; ++i) s[k][i] += r[i];
            }
            if (a.sum) {
                const raw_t<T, V> kept = pack<T, V>(s[k]);
                *reinterpret_cast<raw_t<T, V> *>((T *)a.sum + row * a.d + c) = kept;
                unpack<T, V>(kept, s[k]);
            }
#pragma unroll
            for (int i = 0; i < V; ++i) sum += s[k][i];
        }
    }
    const float mean = group_sum<G>(sum, shared) / (float)a.d;
    float square = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k)
        if ((k * G + t) * V < a.d) {
#pragma unroll
            for (int i = 0; i < V; ++i) square = fmaf(s[k][i] - mean, s[k][i] - mean, square);
        }
    const float rstd = rsqrtf(group_sum<G>(square, shared) / (float)a.d + a.eps);
    if (t == 0 && a.mean) {
        a.mean[row] = mean;
        a.rstd[row] = rstd;
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (k * G + t) * V;
        if (c < a.d) {
            float g[V], b[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                g[i] = 1.f;
                b[i] = 0.f;
            }
            if (a.gamma) load_floats<V>(a.gamma + c, g);
            if (a.beta) load_floats<V>(a.beta + c, b);
#pragma unroll
            for (int i = 0; i < V; ++i) g[i] = fmaf((s[k][i] - mean) * rstd, g[i], b[i]);
            store_vec<T, V>((T *)a.out + row * a.d + c, g);
        }
    }
}

template <typename T, int V, int K, int G>
__global__ void __launch_bounds__(kBlock<G>) norm_bwd_kernel(const __grid_constant__ NormArgs a)
{
    chain_begin();
    __shared__ float shared[32];
    extern __shared__ float columns[];      // G = 32: [8 warps][2][32 V K]
    constexpr int kGroups = kBlock<G> / G;
    const int t = G == 32 ? threadIdx.x & 31 : threadIdx.x, w = G == 32 ? threadIdx.x >> 5 : 0;
    float dg[K][V], db[K][V];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) dg[k][i] = db[k][i] = 0.f;
    chain_wait();
    const float inverse = 1.f / (float)a.d;
    for (long row = (long)blockIdx.x * kGroups + w; row < a.rows; row += (long)gridDim.x * kGroups) {
        const size_t at = (size_t)row * a.d;
        raw_t<T, V> rx[K], rr[K], ry[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * G + t) * V;
            if (c < a.d) {
                rx[k] = load_raw<T, V>((const T *)a.x + at + c);
                ry[k] = load_raw<T, V>((const T *)a.dy + at + c);
                if (a.residual) rr[k] = load_raw<T, V>((const T *)a.residual + at + c);
            }
        }
        const float mean = a.mean[row], rstd = a.rstd[row];
        float hat[K][V], g[K][V], sum = 0.f, along = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * G + t) * V;
            if (c < a.d) {
                unpack<T, V>(rx[k], hat[k]);
                unpack<T, V>(ry[k], g[k]);
                if (a.residual) {
                    float r[V];
                    unpack<T, V>(rr[k], r);
#pragma unroll
                    for (int i = 0; i < V; ++i) hat[k][i] += r[i];
                }
                float gamma[V];
#pragma unroll
                for (int i = 0; i < V; ++i) gamma[i] = 1.f;
                if (a.gamma) load_floats<V>(a.gamma + c, gamma);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    hat[k][i] = (hat[k][i] - mean) * rstd;
                    dg[k][i] = fmaf(g[k][i], hat[k][i], dg[k][i]);
                    db[k][i] += g[k][i];
                    g[k][i] *= gamma[i];
                    sum += g[k][i];
                    along = fmaf(g[k][i], hat[k][i], along);
                }
            }
        }
        sum = group_sum<G>(sum, shared) * inverse;
        along = group_sum<G>(along, shared) * inverse;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * G + t) * V;
            if (c < a.d) {
#pragma unroll
                for (int i = 0; i < V; ++i) g[k][i] = (g[k][i] - sum - hat[k][i] * along) * rstd;
                if (a.dsum) {
                    float r[V];
                    unpack<T, V>(load_raw<T, V>((const T *)a.dsum + at + c), r);
#pragma unroll
                    for (int i = 0; i < V; ++i) g[k][i] += r[i];
                }
                store_vec<T, V>((T *)a.out + at + c, g[k]);
            }
        }
    }
    if (!a.weights) return;
    float *part = a.part + (size_t)blockIdx.x * 2 * a.pitch;
    if constexpr (G == 32) {
        constexpr int kWide = 32 * V * K;
        float *mine = columns + (size_t)w * 2 * kWide;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            store_floats<V>(mine + (k * 32 + t) * V, dg[k]);
            store_floats<V>(mine + kWide + (k * 32 + t) * V, db[k]);
        }
        __syncthreads();
        for (int c = threadIdx.x; c < 2 * kWide; c += kWarpBlock) {
            float sum = 0.f;
#pragma unroll
            for (int x = 0; x < kGroups; ++x) sum += columns[(size_t)x * 2 * kWide + c];
            const int column = c % kWide;
            if (column < a.d) part[(c / kWide) * a.pitch + column] = sum;
        }
    } else {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * G + t) * V;
            if (c < a.d) {
                store_floats<V>(part + c, dg[k]);
                store_floats<V>(part + a.pitch + c, db[k]);
            }
        }
    }
}

// adds the blocks' column sums: 32 threads per column
__global__ void __launch_bounds__(1024)
norm_columns_kernel(const float *part, int blocks, int d, int pitch, float *dgamma, float *dbeta)
{
    chain_begin();
    chain_wait();
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5, strips = (d + 31) / 32;
    const int which = blockIdx.x / strips, c = (blockIdx.x % strips) * 32 + x;
    float sum = 0.f;
    if (c < d)
        for (int b = y; b < blocks; b += 32) sum += part[((size_t)b * 2 + which) * pitch + c];
    __shared__ float sums[32][33];
    sums[y][x] = sum;
    __syncthreads();
    sum = sums[x][y];
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    float *out = which ? dbeta : dgamma;
    const int column = (blockIdx.x % strips) * 32 + y;
    if (x == 0 && column < d && out) out[column] = sum;
}

// ---------------------------------------------------------------- host side
int norm_pitch(int d) { return (d + 3) / 4 * 4; }

// blocks of the backward: groups of 8 warps, or one row at a time
int norm_blocks(int rows, int d)
{
    const int groups = d <= 1024 ? kWarpBlock / 32 : 1;
    const long want = ((long)rows + groups - 1) / groups, most = d <= 4096 ? kMostBlocks : kMostBlocks / 2;
    return (int)(want < most ? want : most);
}

size_t norm_bytes(int rows, int d) { return (size_t)norm_blocks(rows, d) * 2 * norm_pitch(d) * 4 + 256; }

txl_status norm_sizes(int rows, int d, txl_dtype dtype)
{
    if (dtype != TXL_F32 && dtype != TXL_BF16) return TXL_ERR_UNSUPPORTED;
    if (rows < 0 || d < 1) return TXL_ERR_INVALID;
    if (rows > kMaxRows || d > kMaxNormWidth) return TXL_ERR_UNSUPPORTED;
    return TXL_OK;
}

template <typename T, int V, int K, int G>
cudaError_t launch_norm(const NormArgs &a, bool backward, int blocks, cudaStream_t s)
{
    if (!backward) {
        const unsigned grid = (unsigned)(G == 32 ? ((long)a.rows + kWarpBlock / 32 - 1) / (kWarpBlock / 32) : a.rows);
        return chain_launch(norm_fwd_kernel<T, V, K, G>, grid, kBlock<G>, 0, 1, s, a);
    }
    const size_t smem = G == 32 ? (size_t)(kWarpBlock / 32) * 2 * 32 * V * K * 4 : 0;
    if (smem > 48 << 10) {
        const cudaError_t e = cudaFuncSetAttribute(norm_bwd_kernel<T, V, K, G>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    return chain_launch(norm_bwd_kernel<T, V, K, G>, (unsigned)blocks, kBlock<G>, smem, 1, s, a);
}

// K vectors of V columns per thread for the smallest group that holds a row
template <typename T, int V>
cudaError_t pick_norm(const NormArgs &a, bool backward, int blocks, cudaStream_t s)
{
    if constexpr (V >= 4) {
        if (a.d <= 256) return launch_norm<T, V, 8 / V, 32>(a, backward, blocks, s);
        if (a.d <= 512) return launch_norm<T, V, 16 / V, 32>(a, backward, blocks, s);
    } else if (a.d <= 512) {
        return launch_norm<T, V, 16 / V, 32>(a, backward, blocks, s);
    }
    if (a.d <= 1024) return launch_norm<T, V, 32 / V, 32>(a, backward, blocks, s);
    if (a.d <= 4096) return launch_norm<T, V, 16 / V, 256>(a, backward, blocks, s);
    return launch_norm<T, V, 8 / V, 1024>(a, backward, blocks, s);
}

// the widest vector that every row of every tensor can be read by
cudaError_t run_norm(const NormArgs &a, txl_dtype dtype, bool backward, int blocks, cudaStream_t s)
{
    const size_t esz = dtype == TXL_F32 ? 4 : 2;
    int wide = (int)esz;
    for (int n : {16, 4}) {
        bool fits = (size_t)a.d * esz % n == 0;
        for (const void *p : {a.x, a.residual, a.dy, a.dsum, (const void *)a.out, (const void *)a.sum})
            fits = fits && at_boundary(p, n);
        const size_t floats = n / esz * 4 < 16 ? n / esz * 4 : 16;
        for (const void *p : {a.gamma, a.beta}) fits = fits && at_boundary(p, floats);
        if (fits) {
            wide = n;
            break;
        }
    }
    if (dtype == TXL_F32)
        return wide == 16 ? pick_norm<float, 4>(a, backward, blocks, s) : pick_norm<float, 1>(a, backward, blocks, s);
    return wide == 16  ? pick_norm<__nv_bfloat16, 8>(a, backward, blocks, s)
           : wide == 4 ? pick_norm<__nv_bfloat16, 2>(a, backward, blocks, s)
                       : pick_norm<__nv_bfloat16, 1>(a, backward, blocks, s);
}

txl_status finish(cudaError_t e)
{
    if (e == cudaSuccess) return TXL_OK;
    note_cuda_error(e);
    return TXL_ERR_CUDA;
}

}  // namespace
}  // namespace txl

using namespace txl;

extern "C" {

txl_status txl_layer_norm_fwd(const void *x, const void *residual, const float *gamma, const float *beta, float eps,
                              int rows, int d_model, txl_dtype dtype, void *y, void *sum, float *mean, float *rstd,
                              void *stream)
{
    txl_status st = norm_sizes(rows, d_model, dtype);
    if (st != TXL_OK) return st;
    if (!(eps > 0.f) || eps > 3.4028234e38f || (mean == nullptr) != (rstd == nullptr)) return TXL_ERR_INVALID;
    const size_t esz = dtype == TXL_F32 ? 4 : 2, n = (size_t)rows, all = n * d_model * esz, w = rows ? (size_t)d_model * 4 : 0;
    st = check_buffers({{x, all, esz, true}, {residual, all, esz, false}, {gamma, w, 4, false}, {beta, w, 4, false}},
                       {{y, all, esz, true}, {sum, all, esz, false}, {mean, n * 4, 4, false}, {rstd, n * 4, 4, false}});
    if (st != TXL_OK || rows == 0) return st;
    const NormArgs a = {x, residual, nullptr, nullptr, gamma, beta, y, sum, mean, rstd, nullptr, eps, rows, d_model, 0, 0};
    return finish(run_norm(a, dtype, false, 0, (cudaStream_t)stream));
}

txl_status txl_layer_norm_bwd_workspace(int rows, int d_model, txl_dtype dtype, size_t *bytes)
{
    if (!bytes) return TXL_ERR_INVALID;
    const txl_status st = norm_sizes(rows, d_model, dtype);
    if (st != TXL_OK) return st;
    *bytes = rows ? norm_bytes(rows, d_model) : 256;
    return TXL_OK;
}

txl_status txl_layer_norm_bwd(const void *dy, const void *x, const void *residual, const void *dsum, const float *gamma,
                              const float *mean, const float *rstd, int rows, int d_model, txl_dtype dtype, void *dx,
                              float *dgamma, float *dbeta, void *workspace, size_t workspace_bytes, void *stream)
{
    txl_status st = norm_sizes(rows, d_model, dtype);
    if (st != TXL_OK) return st;
    const size_t esz = dtype == TXL_F32 ? 4 : 2, n = (size_t)rows, all = n * d_model * esz, w = (size_t)d_model * 4;
    const bool weights = dgamma || dbeta, scratch = weights && rows > 0;
    st = check_buffers({{dy, all, esz, true}, {x, all, esz, true}, {residual, all, esz, false}, {dsum, all, esz, false},
                        {gamma, rows ? w : 0, 4, false}, {mean, n * 4, 4, true}, {rstd, n * 4, 4, true}},
                       {{dx, all, esz, true}, {dgamma, w, 4, false}, {dbeta, w, 4, false},
                        {workspace, scratch ? workspace_bytes : 0, 256, scratch}});
    if (st != TXL_OK) return st;
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e = cudaSuccess;
    if (rows == 0) {     // sums over no rows
        if (dgamma) e = cudaMemsetAsync(dgamma, 0, w, s);
        if (dbeta && e == cudaSuccess) e = cudaMemsetAsync(dbeta, 0, w, s);
        return finish(e);
    }
    if (scratch && (!workspace || workspace_bytes < norm_bytes(rows, d_model))) return TXL_ERR_INVALID;
    const int blocks = norm_blocks(rows, d_model), pitch = norm_pitch(d_model);
    const NormArgs a = {x, residual, dy, dsum, gamma, nullptr, dx, nullptr, (float *)mean, (float *)rstd,
                        (float *)workspace, 0.f, rows, d_model, pitch, weights};
    e = run_norm(a, dtype, true, blocks, s);
    if (e == cudaSuccess && weights)
        e = chain_launch(norm_columns_kernel, (unsigned)(2 * ((d_model + 31) / 32)), 1024, 0, 1, s,
                         (const float *)workspace, blocks, d_model, pitch, dgamma, dbeta);
    return finish(e);
}

}  // extern "C"

// layer_norm.cu -- layer norm of a residual sum, and its gradients.
//
//     s = x + residual            (rounded to the element type where it is kept, and then used as kept)
//     y = (s - mean) rstd gamma + beta,  rstd = 1 / sqrt(var + eps)
//     ds = rstd (g - mean_d(g) - xh mean_d(g xh)) + dsum,   g = dy gamma, xh = (s - mean) rstd
//     dgamma = sum_i dy xh, dbeta = sum_i dy
//
// HBM-bound, above some 256 columns.  The variance is the mean of the squared
// differences from the mean.  G threads share a row, which stays in registers,
// as fp32, from its loads to its result:
//     forward: a warp up to 1024 columns (rows read by single elements: up to
//     256), 128 threads up to 2048, 256 up to 4096, 512 above;
//     backward: a warp up to 1024 columns (bf16 rows read by single elements:
//     up to 512), 256 threads up to 2048, 512 up to 4096, 1024 above.
// A row takes a whole warp however narrow it is: 262144 rows of 64 bf16
// columns take 69 us forward and 79 backward where their bytes are worth 15
// and 20, of 33 columns 80 and 88 (8 and 10).
//
// The backward's warps (groups of threads) take many rows each and keep their
// columns' sums for dgamma and dbeta in registers; a block adds its warps' up
// and writes them, and a second launch adds the blocks' in a fixed order.
// Those registers leave room for few warps, so a warp of the backward asks for
// its next rows (asynchronous copies into shared memory, each lane its own
// columns; not bf16 rows that are only 2-byte aligned, which such copies do
// not serve) before it computes one: 6144 x 1024 pre-norm rows 27.7 -> 15.0 us
// (the forward gained nothing by it, 12 -> 14 us, and keeps a row per warp).
// It reads two rows ahead where three stages of dy, x, the residual and dsum
// fit beside another block's, one where two do, and none (one stage) for fp32
// rows of more than 512 columns, and for fp32 rows of 257 to 512 and bf16 ones
// of more than 512 with both the residual and dsum: other warps' rows are then
// all that hides a load (fp32 262144 x 1024 with a residual 690 us, 633 at the
// copy rate).
//
// Measured one by one under a profiler (about 2.5 us of each a launch; several
// GB300s): 16896 x 512 bf16 with residual forward 11.8 to 12.7 us (52 MB),
// backward 15.1 to 15.8 us (70 MB), column sums 3.6 to 4.3 us; 6144 x 1024 with
// the sum kept 11.4 to 13.5 us (50 MB), 15.0 to 15.7 us (50 MB, bound by its
// instructions: a row's xh is computed twice) and 3.7 to 4.3 us.
// Wider rows as 16 columns a thread in the forward, 8 in the backward: 65536 x
// 8192 forward 665 us (1024 threads of 8 columns: 1034), 65536 x 2048 forward
// 148 (256 threads: 270), backward 198 (256 threads of up to 16 columns and
// more barriers per row: 297).
// Some kernels spill registers: the forward of 16 columns a thread in fp32 (76
// bytes; 104 by pairs, 20 by bf16 pairs), the backward's of 1024 threads (88 to
// 148) and the read-ahead one of fp32 rows above 512 columns (12; 108 by single
// elements).  The forward runs at the copy rate all the same (fp32 262144 x 512
// 227 us, x 1024 446, 65536 x 2048 228, x 4096 471); the backward of 65536 x
// 8192 fp32 takes 1.41 times its floor where x 4096, which does not spill,
// takes 1.33.
#include <cuda_runtime.h>
#include <stdint.h>

#include "buffers.h"
#include "chain.h"
#include "internal.h"
#include "rows.cuh"

namespace txl {
namespace {

constexpr int kMaxRows = 1 << 30;
constexpr int kMaxNormWidth = 8192;    // 1024 threads of the backward hold 8 columns each
constexpr int kMostBlocks = 608;       // of the backward: four per SM
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

// The warp's sums of a and of b: half the lanes go on with either.
__device__ __forceinline__ void two_sums(float &a, float &b)
{
    const bool low = (threadIdx.x & 16) == 0;
    float v = (low ? a : b) + __shfl_xor_sync(0xffffffffu, low ? b : a, 16);
#pragma unroll
    for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    a = __shfl_sync(0xffffffffu, v, 0);
    b = __shfl_sync(0xffffffffu, v, 16);
}

// The sum of v over the group's G threads, through shared[G / 32], which the
// sum after the next may use again (one barrier each: two places in turn).
template <int G>
__device__ __forceinline__ float group_sum(float v, float *shared)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if constexpr (G > 32) {
        const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
        if (lane == 0) shared[w] = v;
        __syncthreads();
        v = lane < G / 32 ? shared[lane] : 0.f;
#pragma unroll
        for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    }
    return v;
}

// ... of a and of b
template <int G>
__device__ __forceinline__ void group_sums(float &a, float &b, float2 *shared)
{
    two_sums(a, b);
    if constexpr (G > 32) {
        const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
        if (lane == 0) shared[w] = make_float2(a, b);
        __syncthreads();
        const float2 v = lane < G / 32 ? shared[lane] : make_float2(0.f, 0.f);
        a = v.x;
        b = v.y;
        two_sums(a, b);
    }
}

// threads of a block: 8 groups of a warp, or one group
template <int G>
constexpr int kBlock = G == 32 ? kWarpBlock : G;

template <typename T, int V, int K, int G>
__global__ void __launch_bounds__(kBlock<G>, G == 32 ? (K * V <= 16 ? 4 : 1) : V * sizeof(T) == 16 || K * V <= 8 ? 1024 / G : 1)
norm_fwd_kernel(const __grid_constant__ NormArgs a)
{
    chain_begin();
    __shared__ float shared[2][32];
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
    // gamma and beta too, where the registers allow it
    constexpr bool EARLY = K * V <= 16;
    float gm[EARLY ? K : 1][V], bt[EARLY ? K : 1][V];
    const auto affine = [&](int c, float (&g)[V], float (&b)[V]) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            g[i] = 1.f;
            b[i] = 0.f;
        }
        if (a.gamma && c < a.d) load_floats<V>(a.gamma + c, g);
        if (a.beta && c < a.d) load_floats<V>(a.beta + c, b);
    };
    if (EARLY) {
#pragma unroll
        for (int k = 0; k < K; ++k) affine((k * G + t) * V, gm[EARLY ? k : 0], bt[EARLY ? k : 0]);
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
    const float mean = group_sum<G>(sum, shared[0]) / (float)a.d;
    float square = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k)
        if ((k * G + t) * V < a.d) {
#pragma unroll
            for (int i = 0; i < V; ++i) square = fmaf(s[k][i] - mean, s[k][i] - mean, square);
        }
    const float rstd = rsqrtf(group_sum<G>(square, shared[1]) / (float)a.d + a.eps);
    if (t == 0 && a.mean) {
        a.mean[row] = mean;
        a.rstd[row] = rstd;
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (k * G + t) * V;
        float(&g)[V] = gm[EARLY ? k : 0], (&b)[V] = bt[EARLY ? k : 0];
        if (!EARLY) affine(c, g, b);
        if (c < a.d) {
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
    __shared__ float2 shared[2][32];
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
    int place = 0;
    for (long row = (long)blockIdx.x * kGroups + w; row < a.rows; row += (long)gridDim.x * kGroups) {
        const size_t at = (size_t)row * a.d;
        raw_t<T, V> rx[K], rr[K], ry[K], rs[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * G + t) * V;
            if (c < a.d) {
                rx[k] = load_raw<T, V>((const T *)a.x + at + c);
                ry[k] = load_raw<T, V>((const T *)a.dy + at + c);
                if (a.residual) rr[k] = load_raw<T, V>((const T *)a.residual + at + c);
                if (a.dsum) rs[k] = load_raw<T, V>((const T *)a.dsum + at + c);
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
        group_sums<G>(sum, along, shared[place]);
        place ^= 1;
        sum *= inverse;
        along *= inverse;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * G + t) * V;
            if (c < a.d) {
#pragma unroll
                for (int i = 0; i < V; ++i) g[k][i] = (g[k][i] - sum - hat[k][i] * along) * rstd;
                if (a.dsum) {
                    float r[V];
                    unpack<T, V>(rs[k], r);
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

// ---------------------------------------------------------------- a warp per row, read ahead
// A lane's columns are G groups of 8: J = 8 / V vectors of V columns each,
// vector k of all at column (k 32 + lane) V.
constexpr int kRowWarps = kWarpBlock / 32;
constexpr int kMostStages = 3;

// shared memory of one row of one tensor; a stage: its tensors' rows, mean and rstd
template <typename T, int G>
constexpr int kRowBytes = 32 * 8 * G * (int)sizeof(T);
template <typename T, int G>
__host__ __device__ __forceinline__ int stage_bytes(int tensors) { return tensors * kRowBytes<T, G> + 16; }

template <int BYTES>
__device__ __forceinline__ void copy_async(void *to, const void *from)
{
    const uint32_t at = (uint32_t)__cvta_generic_to_shared(to);
    if constexpr (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(from) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(at), "l"(from), "n"(BYTES) : "memory");
}

// until at most n (0 .. kMostStages - 1) of the lane's groups of copies are under way
__device__ __forceinline__ void wait_copies(int n)
{
    if (n == 0) asm volatile("cp.async.wait_group 0;" ::: "memory");
    else if (n == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 2;" ::: "memory");
}

template <typename T, int V, int G>
__device__ __forceinline__ void copy_row(unsigned char *to, const void *from, long row, int d, int lane)
{
    const T *x = (const T *)from + row * d;
#pragma unroll
    for (int k = 0; k < G * 8 / V; ++k) {
        const int v = k * 32 + lane;
        if (v * V < d) copy_async<V * (int)sizeof(T)>((T *)to + v * V, x + v * V);
    }
}

// the lane's group g of a row in shared memory
template <typename T, int V>
__device__ __forceinline__ void group_of(const unsigned char *row, int g, int lane, float (&x)[8])
{
#pragma unroll
    for (int j = 0; j < 8 / V; ++j) {
        float v[V];
        unpack<T, V>(load_raw<T, V>((const T *)row + ((g * (8 / V) + j) * 32 + lane) * V), v);
#pragma unroll
        for (int i = 0; i < V; ++i) x[j * V + i] = v[i];
    }
}

// ... and of gamma or beta
template <int V>
__device__ __forceinline__ void floats_of(const float *row, int g, int lane, float (&x)[8])
{
#pragma unroll
    for (int j = 0; j < 8 / V; ++j) {
        float v[V];
        load_floats<V>(row + ((g * (8 / V) + j) * 32 + lane) * V, v);
#pragma unroll
        for (int i = 0; i < V; ++i) x[j * V + i] = v[i];
    }
}

template <typename T, int V>
__device__ __forceinline__ void store_group(T *row, int g, int lane, int d, const float (&x)[8])
{
#pragma unroll
    for (int j = 0; j < 8 / V; ++j) {
        const int c = ((g * (8 / V) + j) * 32 + lane) * V;
        float v[V];
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = x[j * V + i];
        if (c < d) store_vec<T, V>(row + c, v);
    }
}

// columns past the row's end are zero in every stage: nothing copies there
template <typename T, int V, int G>
__device__ __forceinline__ void clear_ends(unsigned char *mine, int stages, int bytes, int tensors, int d, int lane)
{
    const float none[V] = {};
    for (int x = 0; x < stages; ++x)
        for (int y = 0; y < tensors; ++y)
#pragma unroll
            for (int k = 0; k < G * 8 / V; ++k) {
                const int v = k * 32 + lane;
                if (v * V >= d) store_vec<T, V>((T *)(mine + x * bytes + y * kRowBytes<T, G>) + v * V, none);
            }
}

// a float vector of the columns in shared memory, zero past the row's end
template <int G>
__device__ __forceinline__ void load_columns(float *to, const float *from, float otherwise, int d)
{
    for (int c = threadIdx.x; c < 32 * 8 * G; c += kWarpBlock) to[c] = c < d ? (from ? from[c] : otherwise) : 0.f;
}

template <typename T, int V, int G>
__global__ void __launch_bounds__(kWarpBlock, 2) norm_bwd_rows_kernel(const __grid_constant__ NormArgs a, int stages)
{
    chain_begin();
    constexpr int kWide = 32 * 8 * G;
    constexpr bool KEEP = G <= 2;
    extern __shared__ __align__(16) unsigned char dynamic[];
    float *gamma = (float *)dynamic;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    // tensors in a stage: dy, x, residual, dsum
    const int at_dsum = a.residual ? 3 : 2, tensors = at_dsum + (a.dsum ? 1 : 0);
    const int bytes = stage_bytes<T, G>(tensors);
    unsigned char *mine = (unsigned char *)(gamma + kWide) + w * stages * bytes;
    const long step = (long)gridDim.x * kRowWarps;
    long row = (long)blockIdx.x * kRowWarps + w;
    clear_ends<T, V, G>(mine, stages, bytes, tensors, a.d, lane);
    chain_wait();
    const auto ask = [&](long r, int stage) {
        unsigned char *to = mine + stage * bytes;
        if (r < a.rows) {
            copy_row<T, V, G>(to, a.dy, r, a.d, lane);
            copy_row<T, V, G>(to + kRowBytes<T, G>, a.x, r, a.d, lane);
            if (a.residual) copy_row<T, V, G>(to + 2 * kRowBytes<T, G>, a.residual, r, a.d, lane);
            if (a.dsum) copy_row<T, V, G>(to + at_dsum * kRowBytes<T, G>, a.dsum, r, a.d, lane);
            if (lane < 2) copy_async<4>(to + tensors * kRowBytes<T, G> + 4 * lane, (lane ? a.rstd : a.mean) + r);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    for (int x = 0; x + 1 < stages; ++x) ask(row + x * step, x);
    load_columns<G>(gamma, a.gamma, 1.f, a.d);
    __syncthreads();
    uint64_t dg[G][4], db[G][4];
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
        for (int j = 0; j < 4; ++j) dg[g][j] = db[g][j] = 0;
    const float inverse = 1.f / (float)a.d;
    const int vectors = (a.d / V - lane + 31) / 32;      // of this lane, the first ones of each row
    int stage = 0, next = stages - 1;
    for (; row < a.rows; row += step) {
        ask(row + (stages - 1) * step, next);
        wait_copies(stages - 1);
        __syncwarp();           // (mean and rstd are two lanes' copies)
        const unsigned char *x = mine + stage * bytes;
        const float2 stats = *(const float2 *)(x + tensors * kRowBytes<T, G>);
        const uint64_t mean2 = pair(stats.x, stats.x), rstd2 = pair(stats.y, stats.y);
        // xh and dy gamma of a group (dy also by itself): computed for the sums and, where keeping them
        // would take too many registers, again for dx
        const auto load = [&](int g, uint64_t (&hat)[4], uint64_t (&dy)[4], uint64_t (&t)[4]) {
            float v[8], u[8];
            group_of<T, V>(x + kRowBytes<T, G>, g, lane, v);
            if (a.residual) {
                group_of<T, V>(x + 2 * kRowBytes<T, G>, g, lane, u);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    unpair(pair_add(pair(v[2 * j], v[2 * j + 1]), pair(u[2 * j], u[2 * j + 1])), v[2 * j], v[2 * j + 1]);
            }
            group_of<T, V>(x, g, lane, u);
            float gm[8];
            floats_of<V>(gamma, g, lane, gm);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                hat[j] = pair_mul(pair_sub(pair(v[2 * j], v[2 * j + 1]), mean2), rstd2);
                dy[j] = pair(u[2 * j], u[2 * j + 1]);
                t[j] = pair_mul(dy[j], pair(gm[2 * j], gm[2 * j + 1]));
            }
        };
        uint64_t sums = 0, alongs = 0, hats[KEEP ? G : 1][4], ts[KEEP ? G : 1][4];
#pragma unroll
        for (int g = 0; g < G; ++g) {
            uint64_t(&hat)[4] = hats[KEEP ? g : 0], (&t)[4] = ts[KEEP ? g : 0], dy[4];
            load(g, hat, dy, t);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                dg[g][j] = pair_fma(dy[j], hat[j], dg[g][j]);
                db[g][j] = pair_add(db[g][j], dy[j]);
                sums = pair_add(sums, t[j]);
                // (behind the row's end t is 0, but (0 - mean) rstd may be infinite: it is left out)
                if constexpr (V == 1) {
                    float lo, hi;
                    unpair(hat[j], lo, hi);
                    const int k = g * 8 + 2 * j;
                    alongs = pair_fma(t[j], pair(k < vectors ? lo : 0.f, k + 1 < vectors ? hi : 0.f), alongs);
                } else {
                    alongs = pair_fma_below(t[j], hat[j], alongs, g * (8 / V) + 2 * j / V, vectors);
                }
            }
            if (!KEEP) asm volatile("" ::: "memory");      // (one group's values in registers at a time)
        }
        float lo, hi;
        unpair(sums, lo, hi);
        float sum = lo + hi;
        unpair(alongs, lo, hi);
        float along = lo + hi;
        two_sums(sum, along);
        sum *= inverse;
        along *= inverse;
        const uint64_t sum2 = pair(sum, sum), minus2 = pair(-along, -along);
#pragma unroll(KEEP ? G : 1)
        for (int g = 0; g < G; ++g) {
            uint64_t(&hat)[4] = hats[KEEP ? g : 0], (&t)[4] = ts[KEEP ? g : 0], dy[4];
            if (!KEEP) load(g, hat, dy, t);
            float out[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) t[j] = pair_mul(pair_fma(hat[j], minus2, pair_sub(t[j], sum2)), rstd2);
            if (a.dsum) {
                float u[8];
                group_of<T, V>(x + at_dsum * kRowBytes<T, G>, g, lane, u);
#pragma unroll
                for (int j = 0; j < 4; ++j) t[j] = pair_add(t[j], pair(u[2 * j], u[2 * j + 1]));
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) unpair(t[j], out[2 * j], out[2 * j + 1]);
            store_group<T, V>((T *)a.out + row * a.d, g, lane, a.d, out);
        }
        __syncwarp();           // (before another row's mean and rstd arrive here)
        stage = stage + 1 == stages ? 0 : stage + 1;
        next = next + 1 == stages ? 0 : next + 1;
    }
    if (!a.weights) return;
    // the block's sums: the stages' memory is free once every warp is through
    wait_copies(0);
    __syncthreads();
    float *columns = gamma + kWide;       // [8 warps][2][kWide]
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
        for (int j = 0; j < 8 / V; ++j) {
            const int c = ((g * (8 / V) + j) * 32 + lane) * V;
            float x[2][V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int at = j * V + i;
                float lo, hi;
                unpair(dg[g][at / 2], lo, hi);
                x[0][i] = at % 2 ? hi : lo;
                unpair(db[g][at / 2], lo, hi);
                x[1][i] = at % 2 ? hi : lo;
            }
            store_floats<V>(columns + (w * 2) * kWide + c, x[0]);
            store_floats<V>(columns + (w * 2 + 1) * kWide + c, x[1]);
        }
    __syncthreads();
    float *part = a.part + (size_t)blockIdx.x * 2 * a.pitch;
    for (int c = threadIdx.x; c < 2 * kWide; c += kWarpBlock) {
        float sum = 0.f;
#pragma unroll
        for (int x = 0; x < kRowWarps; ++x) sum += columns[x * 2 * kWide + c];
        const int column = c % kWide;
        if (column < a.d) part[(c / kWide) * a.pitch + column] = sum;
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
    // (all asked for at once: one wait for memory, not ten)
    constexpr int kEach = (kMostBlocks + 31) / 32;
    float v[kEach], sum = 0.f;
#pragma unroll
    for (int k = 0; k < kEach; ++k)
        v[k] = c < d && y + 32 * k < blocks ? part[((size_t)(y + 32 * k) * 2 + which) * pitch + c] : 0.f;
#pragma unroll
    for (int k = 0; k < kEach; ++k) sum += v[k];
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

// Blocks of the backward, as many as the SMs hold: of 8 warps that take a row
// each, two per SM; of 8, 16 or 32 that share one, four, two and one.  (bf16
// rows of an odd width are read by single elements, and above 512 columns 8
// warps share one; so are those of an even width that start at an odd element,
// by the blocks that their width has.)
int norm_blocks(int rows, int d, txl_dtype dtype)
{
    const bool warps = d <= 512 || (d <= 1024 && (d % 2 == 0 || dtype == TXL_F32));
    const int groups = warps ? kWarpBlock / 32 : 1;
    const long want = ((long)rows + groups - 1) / groups;
    const long most = 152 * (warps ? 2 : d <= 2048 ? 4 : d <= 4096 ? 2 : 1);
    return (int)(want < most ? want : most);
}

size_t norm_bytes(int rows, int d, txl_dtype dtype)
{
    return (size_t)norm_blocks(rows, d, dtype) * 2 * norm_pitch(d) * 4 + 256;
}

txl_status norm_sizes(int rows, int d, txl_dtype dtype)
{
    if (dtype != TXL_F32 && dtype != TXL_BF16) return TXL_ERR_UNSUPPORTED;
    if (rows < 0 || d < 1) return TXL_ERR_INVALID;
    if (rows > kMaxRows || d > kMaxNormWidth) return TXL_ERR_UNSUPPORTED;
    return TXL_OK;
}

template <typename T, int V, int K, int G>
cudaError_t launch_fwd(const NormArgs &a, cudaStream_t s)
{
    const unsigned grid = (unsigned)(G == 32 ? ((long)a.rows + kRowWarps - 1) / kRowWarps : a.rows);
    return chain_launch(norm_fwd_kernel<T, V, K, G>, grid, kBlock<G>, 0, 1, s, a);
}

// `bytes`: the most that any call gives this kernel.  The limit is the kernel's
// on its device and not a call's: host threads that call at once set the same.
template <typename K>
cudaError_t allow_shared(K kernel, size_t bytes)
{
    return bytes > 48 << 10 ? cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes)
                            : cudaSuccess;
}

// stages that leave room for `blocks` blocks per SM (less, for a single stage of wide rows)
int stages_for(size_t stage, size_t other, int blocks)
{
    const size_t most = (224 << 10) / blocks - 1024;
    int stages = kMostStages;
    while (stages > 1 && other + stages * kRowWarps * stage > most) --stages;
    return stages;
}

// stages and shared memory of norm_bwd_rows_kernel for so many tensors
struct RowsPlan {
    int stages;
    size_t smem;
};

template <typename T, int G>
RowsPlan rows_plan(int tensors)
{
    constexpr size_t kWide = 32 * 8 * G * 4;
    const size_t stage = stage_bytes<T, G>(tensors);
    const int stages = stages_for(stage, kWide, 2);
    const size_t rows = stages * kRowWarps * stage, sums = 2 * kRowWarps * kWide;      // (the column sums, at the end)
    return {stages, kWide + (rows > sums ? rows : sums)};
}

template <typename T, int V, int G>
cudaError_t launch_rows(const NormArgs &a, int blocks, cudaStream_t s)
{
    size_t most = 0;       // (of 2 to 4 tensors, not always 4: that may leave room for fewer stages)
    for (int n = 2; n <= 4; ++n) {
        const size_t smem = rows_plan<T, G>(n).smem;
        most = smem > most ? smem : most;
    }
    const cudaError_t e = allow_shared(norm_bwd_rows_kernel<T, V, G>, most);
    if (e != cudaSuccess) return e;
    const RowsPlan q = rows_plan<T, G>(2 + (a.residual ? 1 : 0) + (a.dsum ? 1 : 0));
    return chain_launch(norm_bwd_rows_kernel<T, V, G>, (unsigned)blocks, kWarpBlock, q.smem, 1, s, a, q.stages);
}

template <typename T, int V, int K, int G>
cudaError_t launch_bwd(const NormArgs &a, int blocks, cudaStream_t s)
{
    const size_t smem = G == 32 ? (size_t)kRowWarps * 2 * 32 * V * K * 4 : 0;
    const cudaError_t e = allow_shared(norm_bwd_kernel<T, V, K, G>, smem);
    if (e != cudaSuccess) return e;
    return chain_launch(norm_bwd_kernel<T, V, K, G>, (unsigned)blocks, kBlock<G>, smem, 1, s, a);
}

// the smallest kernels that hold a row
template <typename T, int V>
cudaError_t pick_fwd(const NormArgs &a, cudaStream_t s)
{
    if constexpr (V != 2) {
        if (a.d <= 256) return launch_fwd<T, V, 8 / V, 32>(a, s);
    }
    if constexpr (V == 1) {
        // single elements take as many loads as columns: few of them a thread,
        // for enough warps to wait for each other (262144 x 1023 bf16 rows 727
        // -> 420 us, x 411 fp32 350 -> 276, against a warp per row)
        if (a.d <= 512) return launch_fwd<T, V, 4, 128>(a, s);
        if (a.d <= 1024) return launch_fwd<T, V, 8, 128>(a, s);
    } else {
        if (a.d <= 512) return launch_fwd<T, V, 16 / V, 32>(a, s);
        if (a.d <= 1024) return launch_fwd<T, V, 32 / V, 32>(a, s);
    }
    if (a.d <= 2048) return launch_fwd<T, V, 16 / V, 128>(a, s);
    if (a.d <= 4096) return launch_fwd<T, V, 16 / V, 256>(a, s);
    return launch_fwd<T, V, 16 / V, 512>(a, s);
}

template <typename T, int V>
cudaError_t pick_bwd(const NormArgs &a, int blocks, cudaStream_t s)
{
    if constexpr (sizeof(T) * V >= 4) {
        if (a.d <= 256) return launch_rows<T, V, 1>(a, blocks, s);
        if (a.d <= 512) return launch_rows<T, V, 2>(a, blocks, s);
        if (a.d <= 1024) return launch_rows<T, V, 4>(a, blocks, s);
    } else {
        // as many loads as columns: 262144 x 255 rows 488 -> 162 us with 8
        // columns a lane instead of 16, x 1023 1794 -> 684 with 8 warps to a
        // row instead of one (x 411 568 by one warp, 977 by 8)
        if (a.d <= 256) return launch_bwd<T, V, 8, 32>(a, blocks, s);
        if (a.d <= 512) return launch_bwd<T, V, 16, 32>(a, blocks, s);
        if (a.d <= 1024) return launch_bwd<T, V, 4, 256>(a, blocks, s);
    }
    if (a.d <= 2048) return launch_bwd<T, V, 8 / V, 256>(a, blocks, s);
    if (a.d <= 4096) return launch_bwd<T, V, 8 / V, 512>(a, blocks, s);
    return launch_bwd<T, V, 8 / V, 1024>(a, blocks, s);
}

template <typename T, int V>
cudaError_t pick_norm(const NormArgs &a, bool backward, int blocks, cudaStream_t s)
{
    return backward ? pick_bwd<T, V>(a, blocks, s) : pick_fwd<T, V>(a, s);
}

// the widest vector that every row of every tensor can be read by
cudaError_t run_norm(const NormArgs &a, txl_dtype dtype, bool backward, int blocks, cudaStream_t s)
{
    const size_t esz = dtype == TXL_F32 ? 4 : 2;
    int wide = (int)esz;
    for (int n : {16, 8, 4}) {
        if (n == 8 && esz == 2) continue;
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
        return wide == 16  ? pick_norm<float, 4>(a, backward, blocks, s)
               : wide == 8 ? pick_norm<float, 2>(a, backward, blocks, s) : pick_norm<float, 1>(a, backward, blocks, s);
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
    *bytes = rows ? norm_bytes(rows, d_model, dtype) : 256;
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
    if (scratch && (!workspace || workspace_bytes < norm_bytes(rows, d_model, dtype))) return TXL_ERR_INVALID;
    const int blocks = norm_blocks(rows, d_model, dtype), pitch = norm_pitch(d_model);
    const NormArgs a = {x, residual, dy, dsum, gamma, nullptr, dx, nullptr, (float *)mean, (float *)rstd,
                        (float *)workspace, 0.f, rows, d_model, pitch, weights};
    e = run_norm(a, dtype, true, blocks, s);
    if (e == cudaSuccess && weights)
        e = chain_launch(norm_columns_kernel, (unsigned)(2 * ((d_model + 31) / 32)), 1024, 0, 1, s,
                         (const float *)workspace, blocks, d_model, pitch, dgamma, dbeta);
    return finish(e);
}

}  // extern "C"

// output_loss.cu -- the output layer's losses without their logits
// (txl_softmax_xent_*, txl_distill_*):
//
//   z = h W^T + bias,  lse_i = log sum_j exp(z_ij / t),
//   loss_i = t^2 sum_k p_ik (log p_ik - z_{i,idx_ik} / t + lse_i)
//
// with p the teacher's softmax over its kept entries; cross entropy is the
// same with one entry of weight 1 and t = 1.  Both reduce to a sparse list
// of (column, weight) per row, so one set of kernels serves both:
//
//   loss_rows_kernel   the row lists (for the backward also the row's factor
//                      t * dloss and lse in base-2 units);
//   lse pass           per 64-row block and strip of vocabulary tiles, the
//                      running maximum and sum of the softmax; the logits of
//                      the listed columns are kept on the way;
//   loss_merge_kernel  joins the strips, loss and lse;
//   backward           for each piece of the vocabulary: dz (one piece of it
//                      in the workspace), dh += dz W, dW = dz^T h, and the
//                      column sums of dz.
//
// Everything is scaled so that exponentials are powers of two:
// y_ij = z_ij * log2(e) / t.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "internal.h"
#include "txl.h"

namespace txl {
namespace {

constexpr int kMaxTopK = 256;
constexpr int kNoColumn = INT32_MAX;   // an invalid list entry: sorts behind every column
constexpr float kLn2 = 0.693147180559945309f;

template <typename T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16(x); }

// One call's rows, as the kernels see them.
struct LossRows {
    int *col;        // [rows][K] listed columns, ascending; kNoColumn behind them
    float *p;        // [rows][K] their weights
    float *ent;      // [rows] sum_k p log p
    float *coef;     // [rows] t * dloss, 0 for an empty row (backward)
    float *l2;       // [rows] lse * log2(e) (backward)
    int K;
};

// cross entropy: one entry of weight 1
__global__ void __launch_bounds__(256)
xent_rows_kernel(const int64_t *__restrict__ target, const float *__restrict__ lse,
                 const float *__restrict__ dloss, LossRows r, int rows, int vocab)
{
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i >= rows) return;
    const int64_t y = target[i];
    const bool valid = y >= 0 && y < vocab;
    r.col[i] = valid ? (int)y : kNoColumn;
    r.p[i] = valid ? 1.f : 0.f;
    r.ent[i] = 0.f;
    if (dloss) {
        const float l = lse[i];
        r.coef[i] = valid && l != -INFINITY ? dloss[i] : 0.f;
        r.l2[i] = l * (1.f / kLn2);
    }
}

// distillation: the softmax of a row's valid entries at temperature t, then
// the entries sorted by column (a bitonic network over the next power of
// two).  One warp per row; K2 entries of shared memory per warp.
template <typename TT>
__global__ void __launch_bounds__(128)
distill_rows_kernel(const int64_t *__restrict__ idx, const TT *__restrict__ logits, float inv_t, float t,
                    const float *__restrict__ lse, const float *__restrict__ dloss, LossRows r, int rows, int vocab,
                    int K2)
{
    extern __shared__ unsigned char sm[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int *sc = reinterpret_cast<int *>(sm) + warp * K2;
    float *sp = reinterpret_cast<float *>(sm) + (4 + warp) * K2;
    const int i = blockIdx.x * 4 + warp;
    if (i >= rows) return;
    const int K = r.K;
    const long base = (long)i * K;
    float top = -INFINITY;
    for (int k = lane; k < K2; k += 32) {
        int c = kNoColumn;
        float y = -INFINITY;
        if (k < K) {
            const int64_t e = idx[base + k];
            const float v = to_f(logits[base + k]);
            if (e >= 0 && e < vocab && v != -INFINITY) {
                c = (int)e;
                y = v * inv_t;
            }
        }
        sc[k] = c;
        sp[k] = y;
        top = fmaxf(top, y);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    float sum = 0.f;
    int any = 0;
    for (int k = lane; k < K2; k += 32)
        if (sc[k] != kNoColumn) {
            any = 1;
            sum += expf(sp[k] - top);
        }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        any |= __shfl_xor_sync(0xffffffffu, any, o);
    }
    const float lt = logf(sum);
    float ent = 0.f;
    for (int k = lane; k < K2; k += 32) {
        float p = 0.f;
        if (sc[k] != kNoColumn) {
            const float lp = sp[k] - top - lt;
            p = expf(lp);
            if (p != 0.f) ent += p * lp;   // (a NaN teacher logit stays NaN)
        }
        sp[k] = p;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) ent += __shfl_xor_sync(0xffffffffu, ent, o);
    __syncwarp();
    for (int len = 2; len <= K2; len <<= 1)
        for (int step = len >> 1; step; step >>= 1) {
            for (int x = lane; x < K2 / 2; x += 32) {
                const int a = 2 * x - (x & (step - 1)), b = a + step;
                const bool up = (a & len) == 0;
                const int ca = sc[a], cb = sc[b];
                if ((ca > cb) == up && ca != cb) {
                    sc[a] = cb;
                    sc[b] = ca;
                    const float q = sp[a];
                    sp[a] = sp[b];
                    sp[b] = q;
                }
            }
            __syncwarp();
        }
    for (int k = lane; k < K; k += 32) {
        r.col[base + k] = sc[k];
        r.p[base + k] = sp[k];
    }
    if (lane == 0) {
        r.ent[i] = ent;
        if (dloss) {
            const float l = lse[i];
            r.coef[i] = any && l != -INFINITY ? t * dloss[i] : 0.f;
            r.l2[i] = l * (1.f / kLn2);
        }
    }
}

// bz[j] = bias_j log2(e) / t (0 without a bias)
__global__ void __launch_bounds__(256) bias_scale_kernel(const float *__restrict__ bias, float alpha,
                                                         float *__restrict__ bz, int vocab)
{
    const int j = blockIdx.x * 256 + threadIdx.x;
    if (j < vocab) bz[j] = bias ? bias[j] * alpha : 0.f;
}

// ------------------------------------------------------------------ products
// 64 x 64 tiles of sum_k A[m][k] B[k][n], 256 threads, 4 x 4 elements each.
constexpr int TM = 64, TN = 64, TK = 16;
struct TileSmem {
    float a[TK][TM + 1], b[TK][TN + 1];
};

template <typename FA, typename FB>
__device__ __forceinline__ void tile_product(TileSmem &s, int K, FA fa, FB fb, float (&acc)[4][4])
{
    const int tid = threadIdx.x, tr = tid / 16, tc = tid % 16;
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y) acc[x][y] = 0.f;
    for (int k0 = 0; k0 < K; k0 += TK) {
        for (int x = tid; x < TK * TM; x += 256) {
            s.a[x % TK][x / TK] = k0 + x % TK < K ? fa(x / TK, k0 + x % TK) : 0.f;
            s.b[x % TK][x / TK] = k0 + x % TK < K ? fb(x / TK, k0 + x % TK) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < TK; ++k) {
            float av[4], bv[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                av[x] = s.a[k][tr + 16 * x];
                bv[x] = s.b[k][tc + 16 * x];
            }
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int y = 0; y < 4; ++y) acc[x][y] = fmaf(av[x], bv[y], acc[x][y]);
        }
        __syncthreads();
    }
}

struct LossShape {
    int rows, d, vocab, strips;
    float alpha;    // log2(e) / t
};

// the tile's y_ij in shared memory, -infinity past the vocabulary
template <typename T>
__device__ __forceinline__ void logits_tile(TileSmem &s, float (*y)[TN + 1], const T *h, const T *w, const float *bz,
                                            const LossShape &q, int m0, int n0)
{
    float acc[4][4];
    tile_product(s, q.d,
                 [&](int m, int k) { return m0 + m < q.rows ? to_f(h[(long)(m0 + m) * q.d + k]) : 0.f; },
                 [&](int n, int k) { return n0 + n < q.vocab ? to_f(w[(long)(n0 + n) * q.d + k]) : 0.f; }, acc);
    const int tr = threadIdx.x / 16, tc = threadIdx.x % 16;
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int n = n0 + tc + 16 * c;
            y[tr + 16 * x][tc + 16 * c] = n < q.vocab ? fmaf(acc[x][c], q.alpha, bz[n]) : -INFINITY;
        }
    __syncthreads();
}

// part[strip][row] = (maximum, sum of 2^(y - maximum)) over the strip's
// columns; ysel[row][k] = y at the row's listed columns
template <typename T>
__global__ void __launch_bounds__(256)
lse_kernel(const T *__restrict__ h, const T *__restrict__ w, const float *__restrict__ bz, LossRows r,
           float *__restrict__ ysel, float2 *__restrict__ part, LossShape q)
{
    __shared__ TileSmem s;
    __shared__ float y[TM][TN + 1];
    const int m0 = blockIdx.x * TM, strip = blockIdx.y;
    const int tiles = (q.vocab + TN - 1) / TN;
    const int t0 = (int)((long)strip * tiles / q.strips), t1 = (int)((long)(strip + 1) * tiles / q.strips);
    const int row = threadIdx.x >> 2, sub = threadIdx.x & 3, i = m0 + row;
    float m = -INFINITY, l = 0.f;
    for (int t = t0; t < t1; ++t) {
        const int n0 = t * TN;
        logits_tile(s, y, h, w, bz, q, m0, n0);
        float cm = m;
        for (int c = sub; c < TN; c += 4) cm = fmaxf(cm, y[row][c]);
        if (cm != -INFINITY) {
            l *= exp2f(m - cm);
            for (int c = sub; c < TN; c += 4) l += exp2f(y[row][c] - cm);
            m = cm;
        } else {
            for (int c = sub; c < TN; c += 4) l += exp2f(y[row][c]);   // all -infinity, or NaN
        }
        if (i < q.rows)
            for (int k = sub; k < r.K; k += 4) {
                const int c = r.col[(long)i * r.K + k];
                if (c >= n0 && c < n0 + TN) ysel[(long)i * r.K + k] = y[row][c - n0];
            }
        __syncthreads();
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, m, o), l2 = __shfl_xor_sync(0xffffffffu, l, o);
        const float mm = fmaxf(m, m2), ref = mm == -INFINITY ? 0.f : mm;
        l = l * exp2f(m - ref) + l2 * exp2f(m2 - ref);
        m = mm;
    }
    if (sub == 0 && i < q.rows) part[(long)strip * q.rows + i] = make_float2(m, l);
}

__global__ void __launch_bounds__(256)
loss_merge_kernel(const float2 *__restrict__ part, int slots, const float *__restrict__ ysel, LossRows r, float t2,
                  float *__restrict__ loss, float *__restrict__ lse, int rows)
{
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i >= rows) return;
    float m = -INFINITY;
    for (int x = 0; x < slots; ++x) m = fmaxf(m, part[(long)x * rows + i].x);
    const float ref = m == -INFINITY ? 0.f : m;
    float l = 0.f;
    for (int x = 0; x < slots; ++x) {
        const float2 e = part[(long)x * rows + i];
        l += e.y * exp2f(e.x - ref);
    }
    const float y_lse = ref + log2f(l);
    lse[i] = y_lse * kLn2;
    float dot = 0.f;
    bool any = false;
    for (int k = 0; k < r.K; ++k) {
        if (r.col[(long)i * r.K + k] == kNoColumn) continue;
        any = true;
        const float p = r.p[(long)i * r.K + k];
        if (p != 0.f) dot += p * (y_lse - ysel[(long)i * r.K + k]);
    }
    loss[i] = any && y_lse != -INFINITY ? t2 * (r.ent[i] + kLn2 * dot) : 0.f;
}

// one piece of dz (columns v0 .. v0+cols) and its column sums per row block
template <typename T>
__global__ void __launch_bounds__(256)
dz_kernel(const T *__restrict__ h, const T *__restrict__ w, const float *__restrict__ bz, LossRows r,
          T *__restrict__ dz, float *__restrict__ dbpart, LossShape q, int v0, int cols)
{
    __shared__ TileSmem s;
    __shared__ float y[TM][TN + 1];
    const int m0 = blockIdx.x * TM, c0 = blockIdx.y * TN, n0 = v0 + c0;
    LossShape qq = q;
    qq.vocab = v0 + cols;
    logits_tile(s, y, h, w, bz, qq, m0, n0);
    const int row = threadIdx.x >> 2, sub = threadIdx.x & 3, i = m0 + row;
    const float coef = i < q.rows ? r.coef[i] : 0.f, l2 = i < q.rows ? r.l2[i] : 0.f;
    for (int c = sub; c < TN; c += 4) y[row][c] = coef != 0.f ? coef * exp2f(y[row][c] - l2) : 0.f;
    __syncwarp();
    if (coef != 0.f)   // entries of one column: the same thread, in order
        for (int k = 0; k < r.K; ++k) {
            const int c = r.col[(long)i * r.K + k] - n0;
            if (c >= 0 && c < TN && (c & 3) == sub) y[row][c] -= coef * r.p[(long)i * r.K + k];
        }
    __syncthreads();
    for (int x = threadIdx.x; x < TM * TN; x += 256)
        if (m0 + x / TN < q.rows && c0 + x % TN < cols)
            dz[(long)(m0 + x / TN) * cols + c0 + x % TN] = from_f<T>(y[x / TN][x % TN]);
    if (dbpart && threadIdx.x < TN && c0 + threadIdx.x < cols) {
        float sum = 0.f;
        for (int m = 0; m < TM; ++m) sum += y[m][threadIdx.x];
        dbpart[(long)blockIdx.x * cols + c0 + threadIdx.x] = sum;
    }
}

__global__ void __launch_bounds__(256)
dbias_kernel(const float *__restrict__ dbpart, int parts, int cols, float *__restrict__ db)
{
    const int j = blockIdx.x * 256 + threadIdx.x;
    if (j >= cols) return;
    float sum = 0.f;
    for (int x = 0; x < parts; ++x) sum += dbpart[(long)x * cols + j];
    db[j] = sum;
}

// dh += dz W over one piece, in fp32; the last piece rounds
template <typename T>
__global__ void __launch_bounds__(256)
dh_kernel(const T *__restrict__ dz, const T *__restrict__ w, float *__restrict__ acc, T *__restrict__ dh, int rows,
          int d, int cols, int first, int last)
{
    __shared__ TileSmem s;
    const int m0 = blockIdx.x * TM, n0 = blockIdx.y * TN;
    float a[4][4];
    tile_product(s, cols, [&](int m, int k) { return m0 + m < rows ? to_f(dz[(long)(m0 + m) * cols + k]) : 0.f; },
                 [&](int n, int k) { return n0 + n < d ? to_f(w[(long)k * d + n0 + n]) : 0.f; }, a);
    const int tr = threadIdx.x / 16, tc = threadIdx.x % 16;
    for (int x = 0; x < 4; ++x)
        for (int c = 0; c < 4; ++c) {
            const int m = m0 + tr + 16 * x, n = n0 + tc + 16 * c;
            if (m >= rows || n >= d) continue;
            float v = a[x][c];
            if (!first) v += acc[(long)m * d + n];
            if (last)
                dh[(long)m * d + n] = from_f<T>(v);
            else
                acc[(long)m * d + n] = v;
        }
}

// dW of one piece; rows whose factor is 0 are left out whatever h holds there
template <typename T>
__global__ void __launch_bounds__(256)
dw_kernel(const T *__restrict__ dz, const T *__restrict__ h, const float *__restrict__ coef, T *__restrict__ dw,
          int rows, int d, int cols)
{
    __shared__ TileSmem s;
    const int m0 = blockIdx.x * TM, n0 = blockIdx.y * TN;
    float a[4][4];
    tile_product(s, rows, [&](int m, int k) { return m0 + m < cols ? to_f(dz[(long)k * cols + m0 + m]) : 0.f; },
                 [&](int n, int k) { return n0 + n < d && coef[k] != 0.f ? to_f(h[(long)k * d + n0 + n]) : 0.f; }, a);
    const int tr = threadIdx.x / 16, tc = threadIdx.x % 16;
    for (int x = 0; x < 4; ++x)
        for (int c = 0; c < 4; ++c) {
            const int m = m0 + tr + 16 * x, n = n0 + tc + 16 * c;
            if (m < cols && n < d) dw[(long)m * d + n] = from_f<T>(a[x][c]);
        }
}

// ---------------------------------------------------------------- host side
bool al(const void *p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

bool overlap(const void *a, size_t na, const void *b, size_t nb)
{
    if (!a || !b || na == 0 || nb == 0) return false;
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return x < y + nb && y < x + na;
}

constexpr size_t kPieceBytes = (size_t)64 << 20;   // one piece of dz
constexpr int kMaxSize = 1 << 30;                  // rows and vocabulary

// Where things lie in the workspace, from the shape alone.
struct LossPlan {
    int strips, piece;     // vocabulary strips of the forward, columns of a backward piece
    size_t col, p, ent, coef, l2, bz, ysel, part, dz, acc, dbpart, bytes;
};

LossPlan loss_plan(int rows, int d, int vocab, int K, size_t esz, bool backward)
{
    LossPlan q;
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t o = at;
        at += (n + 255) / 256 * 256;
        return o;
    };
    const int tiles = (vocab + TN - 1) / TN;
    q.strips = tiles < 64 ? tiles : 64;
    const size_t n = (size_t)rows;
    q.col = take(n * K * 4);
    q.p = take(n * K * 4);
    q.ent = take(n * 4);
    q.bz = take((size_t)vocab * 4);
    const size_t common = at;
    q.ysel = take(n * K * 4);
    q.part = take(n * q.strips * 8);
    const size_t fwd = at;
    size_t piece = kPieceBytes / (n * esz > 0 ? n * esz : 1) / TN * TN;
    if (piece < (size_t)TN) piece = TN;
    if (piece > (size_t)TN * 65535) piece = (size_t)TN * 65535;
    q.piece = piece < (size_t)vocab ? (int)piece : vocab;
    q.coef = q.l2 = q.dz = q.acc = q.dbpart = 0;
    if (backward) {
        at = common;
        q.coef = take(n * 4);
        q.l2 = take(n * 4);
        q.dz = take(n * q.piece * esz);
        q.acc = take(q.piece < vocab ? n * d * 4 : 0);
        q.dbpart = take((n + TM - 1) / TM * q.piece * 4);
    }
    q.bytes = at > fwd ? at : fwd;
    if (q.bytes == 0) q.bytes = 256;
    return q;
}

struct LossArgs {
    const void *h, *w;
    const float *bias;
    const int64_t *idx;            // [rows][K]
    const void *t_logits;          // NULL: cross entropy
    txl_dtype t_dtype;
    float temp;
    int rows, d, vocab, K;
    txl_dtype dtype;
    float *loss, *lse_out;         // forward
    const float *lse, *dloss;      // backward
    void *dh, *dw;
    float *db;
    void *ws;
    size_t ws_bytes;
    cudaStream_t s;
};

txl_status loss_sizes(int rows, int d, int vocab, int K, txl_dtype dtype)
{
    if (dtype != TXL_F32 && dtype != TXL_BF16) return TXL_ERR_UNSUPPORTED;
    if (rows < 0 || d < 1 || vocab < 1 || K < 1) return TXL_ERR_INVALID;
    if (K > kMaxTopK || rows > kMaxSize || vocab > kMaxSize) return TXL_ERR_UNSUPPORTED;
    return TXL_OK;
}

txl_status loss_workspace(int rows, int d, int vocab, int K, txl_dtype dtype, int backward, size_t *bytes)
{
    if (!bytes) return TXL_ERR_INVALID;
    const txl_status st = loss_sizes(rows, d, vocab, K, dtype);
    if (st != TXL_OK) return st;
    *bytes = loss_plan(rows, d, vocab, K, dtype == TXL_F32 ? 4 : 2, backward != 0).bytes;
    return TXL_OK;
}

txl_status loss_checks(const LossArgs &a, bool backward)
{
    const txl_status st = loss_sizes(a.rows, a.d, a.vocab, a.K, a.dtype);
    if (st != TXL_OK) return st;
    const bool distill = a.temp != 0.f;
    if (distill) {
        if (a.t_dtype != TXL_F32 && a.t_dtype != TXL_BF16) return TXL_ERR_UNSUPPORTED;
        if (!(a.temp > 0.f) || isinf(a.temp)) return TXL_ERR_INVALID;
    }
    const size_t esz = a.dtype == TXL_F32 ? 4 : 2, tsz = a.t_dtype == TXL_F32 ? 4 : 2;
    const size_t n = (size_t)a.rows;
    struct Buf {
        const void *p;
        size_t bytes, align;
        bool need;
    };
    const Buf ins[] = {{a.h, n * a.d * esz, esz, true},
                       {a.w, (size_t)a.vocab * a.d * esz, esz, a.rows > 0},
                       {a.bias, (size_t)a.vocab * 4, 4, false},
                       {a.idx, n * a.K * 8, 8, true},
                       {a.t_logits, distill ? n * a.K * tsz : 0, tsz, distill},
                       {backward ? a.lse : nullptr, n * 4, 4, backward},
                       {backward ? a.dloss : nullptr, n * 4, 4, backward}};
    const Buf outs[] = {{backward ? nullptr : a.loss, n * 4, 4, !backward},
                        {backward ? nullptr : a.lse_out, n * 4, 4, !backward},
                        {backward ? a.dh : nullptr, n * a.d * esz, esz, false},
                        {backward ? a.dw : nullptr, (size_t)a.vocab * a.d * esz, esz, false},
                        {backward ? a.db : nullptr, (size_t)a.vocab * 4, 4, false},
                        {a.ws, a.rows > 0 ? a.ws_bytes : 0, 256, a.rows > 0}};
    for (const Buf &b : ins)
        if ((b.need && b.bytes && !b.p) || !al(b.p, b.align)) return TXL_ERR_INVALID;
    for (const Buf &b : outs)
        if ((b.need && b.bytes && !b.p) || !al(b.p, b.align)) return TXL_ERR_INVALID;
    for (const Buf &o : outs) {
        for (const Buf &i : ins)
            if (overlap(o.p, o.bytes, i.p, i.bytes)) return TXL_ERR_INVALID;
        for (const Buf &p : outs)
            if (&p != &o && overlap(o.p, o.bytes, p.p, p.bytes)) return TXL_ERR_INVALID;
    }
    if (a.rows > 0 && a.ws_bytes < loss_plan(a.rows, a.d, a.vocab, a.K, esz, backward).bytes) return TXL_ERR_INVALID;
    return TXL_OK;
}

LossRows rows_at(const LossArgs &a, const LossPlan &q)
{
    unsigned char *ws = (unsigned char *)a.ws;
    LossRows r;
    r.col = (int *)(ws + q.col);
    r.p = (float *)(ws + q.p);
    r.ent = (float *)(ws + q.ent);
    r.coef = (float *)(ws + q.coef);
    r.l2 = (float *)(ws + q.l2);
    r.K = a.K;
    return r;
}

cudaError_t launch_rows(const LossArgs &a, const LossRows &r, const LossPlan &q, bool backward)
{
    const float *lse = backward ? a.lse : nullptr, *dloss = backward ? a.dloss : nullptr;
    if (a.temp == 0.f) {
        xent_rows_kernel<<<(a.rows + 255) / 256, 256, 0, a.s>>>(a.idx, lse, dloss, r, a.rows, a.vocab);
    } else {
        int K2 = 2;
        while (K2 < a.K) K2 <<= 1;
        const int grid = (a.rows + 3) / 4;
        const size_t sm = (size_t)K2 * 8 * 4;
        if (a.t_dtype == TXL_F32)
            distill_rows_kernel<float><<<grid, 128, sm, a.s>>>(a.idx, (const float *)a.t_logits, 1.f / a.temp, a.temp,
                                                               lse, dloss, r, a.rows, a.vocab, K2);
        else
            distill_rows_kernel<__nv_bfloat16><<<grid, 128, sm, a.s>>>(a.idx, (const __nv_bfloat16 *)a.t_logits,
                                                                       1.f / a.temp, a.temp, lse, dloss, r, a.rows,
                                                                       a.vocab, K2);
    }
    const float alpha = 1.f / (kLn2 * (a.temp != 0.f ? a.temp : 1.f));
    bias_scale_kernel<<<(a.vocab + 255) / 256, 256, 0, a.s>>>(a.bias, alpha, (float *)((unsigned char *)a.ws + q.bz),
                                                              a.vocab);
    return cudaGetLastError();
}

LossShape shape_of(const LossArgs &a, const LossPlan &q)
{
    return {a.rows, a.d, a.vocab, q.strips, 1.f / (kLn2 * (a.temp != 0.f ? a.temp : 1.f))};
}

template <typename T>
cudaError_t run_fwd(const LossArgs &a)
{
    const LossPlan q = loss_plan(a.rows, a.d, a.vocab, a.K, sizeof(T), false);
    unsigned char *ws = (unsigned char *)a.ws;
    const LossRows r = rows_at(a, q);
    cudaError_t e = launch_rows(a, r, q, false);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)((a.rows + TM - 1) / TM), (unsigned)q.strips);
    lse_kernel<T><<<grid, 256, 0, a.s>>>((const T *)a.h, (const T *)a.w, (const float *)(ws + q.bz), r,
                                         (float *)(ws + q.ysel), (float2 *)(ws + q.part), shape_of(a, q));
    const float t2 = a.temp != 0.f ? a.temp * a.temp : 1.f;
    loss_merge_kernel<<<(a.rows + 255) / 256, 256, 0, a.s>>>((const float2 *)(ws + q.part), q.strips,
                                                             (const float *)(ws + q.ysel), r, t2, a.loss, a.lse_out,
                                                             a.rows);
    return cudaGetLastError();
}

template <typename T>
cudaError_t run_bwd(const LossArgs &a)
{
    const LossPlan q = loss_plan(a.rows, a.d, a.vocab, a.K, sizeof(T), true);
    unsigned char *ws = (unsigned char *)a.ws;
    const LossRows r = rows_at(a, q);
    cudaError_t e = launch_rows(a, r, q, true);
    const T *w = (const T *)a.w;
    T *dz = (T *)(ws + q.dz);
    const unsigned rb = (unsigned)((a.rows + TM - 1) / TM), db = (unsigned)((a.d + TN - 1) / TN);
    for (long v0 = 0; e == cudaSuccess && v0 < a.vocab; v0 += q.piece) {
        const int cols = (int)(a.vocab - v0 < q.piece ? a.vocab - v0 : q.piece);
        const unsigned cb = (unsigned)((cols + TN - 1) / TN);
        float *dbp = a.db ? (float *)(ws + q.dbpart) : nullptr;
        dz_kernel<T><<<dim3(rb, cb), 256, 0, a.s>>>((const T *)a.h, w, (const float *)(ws + q.bz), r, dz, dbp,
                                                    shape_of(a, q), (int)v0, cols);
        if (a.db) dbias_kernel<<<(cols + 255) / 256, 256, 0, a.s>>>(dbp, (int)rb, cols, a.db + v0);
        if (a.dh)
            dh_kernel<T><<<dim3(rb, db), 256, 0, a.s>>>(dz, w + v0 * a.d, (float *)(ws + q.acc), (T *)a.dh, a.rows,
                                                        a.d, cols, v0 == 0, v0 + cols == a.vocab);
        if (a.dw)
            dw_kernel<T><<<dim3(cb, db), 256, 0, a.s>>>(dz, (const T *)a.h, r.coef, (T *)a.dw + v0 * a.d, a.rows, a.d,
                                                        cols);
        e = cudaGetLastError();
    }
    return e;
}

txl_status loss_fwd(const LossArgs &a)
{
    const txl_status st = loss_checks(a, false);
    if (st != TXL_OK || a.rows == 0) return st;
    const cudaError_t e = a.dtype == TXL_F32 ? run_fwd<float>(a) : run_fwd<__nv_bfloat16>(a);
    if (e == cudaSuccess) return TXL_OK;
    note_cuda_error(e);
    return TXL_ERR_CUDA;
}

txl_status loss_bwd(const LossArgs &a)
{
    const txl_status st = loss_checks(a, true);
    if (st != TXL_OK) return st;
    cudaError_t e = cudaSuccess;
    if (a.rows == 0) {   // sums over no rows
        if (a.dw) e = cudaMemsetAsync(a.dw, 0, (size_t)a.vocab * a.d * (a.dtype == TXL_F32 ? 4 : 2), a.s);
        if (e == cudaSuccess && a.db) e = cudaMemsetAsync(a.db, 0, (size_t)a.vocab * 4, a.s);
    } else if (a.dh || a.dw || a.db) {
        e = a.dtype == TXL_F32 ? run_bwd<float>(a) : run_bwd<__nv_bfloat16>(a);
    }
    if (e == cudaSuccess) return TXL_OK;
    note_cuda_error(e);
    return TXL_ERR_CUDA;
}

}  // namespace
}  // namespace txl

using namespace txl;

extern "C" {

txl_status txl_softmax_xent_workspace(int rows, int d_model, int vocab, txl_dtype dtype, int backward, size_t *bytes)
{
    return loss_workspace(rows, d_model, vocab, 1, dtype, backward, bytes);
}

txl_status txl_distill_workspace(int rows, int d_model, int vocab, int top_k, txl_dtype dtype, int backward,
                                 size_t *bytes)
{
    return loss_workspace(rows, d_model, vocab, top_k, dtype, backward, bytes);
}

txl_status txl_softmax_xent_fwd(const void *h, const void *w, const float *bias, const int64_t *target, int rows,
                                int d_model, int vocab, txl_dtype dtype, float *loss, float *lse, void *workspace,
                                size_t workspace_bytes, void *stream)
{
    return loss_fwd({h, w, bias, target, nullptr, TXL_F32, 0.f, rows, d_model, vocab, 1, dtype, loss, lse, nullptr,
                     nullptr, nullptr, nullptr, nullptr, workspace, workspace_bytes, (cudaStream_t)stream});
}

txl_status txl_softmax_xent_bwd(const void *h, const void *w, const float *bias, const int64_t *target,
                                const float *lse, const float *dloss, int rows, int d_model, int vocab,
                                txl_dtype dtype, void *dh, void *dw, float *dbias, void *workspace,
                                size_t workspace_bytes, void *stream)
{
    return loss_bwd({h, w, bias, target, nullptr, TXL_F32, 0.f, rows, d_model, vocab, 1, dtype, nullptr, nullptr, lse,
                     dloss, dh, dw, dbias, workspace, workspace_bytes, (cudaStream_t)stream});
}

txl_status txl_distill_fwd(const void *h, const void *w, const float *bias, const int64_t *teacher_idx,
                           const void *teacher_logits, txl_dtype teacher_dtype, float temperature, int rows,
                           int d_model, int vocab, int top_k, txl_dtype dtype, float *loss, float *lse,
                           void *workspace, size_t workspace_bytes, void *stream)
{
    if (!(temperature > 0.f)) return TXL_ERR_INVALID;
    return loss_fwd({h, w, bias, teacher_idx, teacher_logits, teacher_dtype, temperature, rows, d_model, vocab, top_k,
                     dtype, loss, lse, nullptr, nullptr, nullptr, nullptr, nullptr, workspace, workspace_bytes,
                     (cudaStream_t)stream});
}

txl_status txl_distill_bwd(const void *h, const void *w, const float *bias, const int64_t *teacher_idx,
                           const void *teacher_logits, txl_dtype teacher_dtype, float temperature, const float *lse,
                           const float *dloss, int rows, int d_model, int vocab, int top_k, txl_dtype dtype,
                           void *dh, void *dw, float *dbias, void *workspace, size_t workspace_bytes, void *stream)
{
    if (!(temperature > 0.f)) return TXL_ERR_INVALID;
    return loss_bwd({h, w, bias, teacher_idx, teacher_logits, teacher_dtype, temperature, rows, d_model, vocab, top_k,
                     dtype, nullptr, nullptr, lse, dloss, dh, dw, dbias, workspace, workspace_bytes,
                     (cudaStream_t)stream});
}

}  // extern "C"

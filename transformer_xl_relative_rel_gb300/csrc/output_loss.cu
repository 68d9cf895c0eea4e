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
//   *_rows_kernel      the row lists (for the backward also the row's factor
//                      t * dloss and lse in base-2 units);
//   forward            one pass over the vocabulary (loss_products.cu) leaves
//                      a maximum and a sum per row and strip of vocabulary
//                      tiles and the logits of the listed columns;
//                      loss_merge_kernel joins them;
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
#include <string.h>

#include <mutex>

#include "internal.h"
#include "loss_products.h"
#include "txl.h"

namespace txl {
namespace {

constexpr int kMaxTopK = 256;
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

// bz[j] = bias_j log2(e) / t
__global__ void __launch_bounds__(256) bias_scale_kernel(const float *__restrict__ bias, float alpha,
                                                         float *__restrict__ bz, int vocab)
{
    const int j = blockIdx.x * 256 + threadIdx.x;
    if (j < vocab) bz[j] = bias[j] * alpha;
}

// The bf16 parts of an element: itself, or the three parts of an fp32 value,
// each the bf16 nearest to what the parts before it leave (a finite value
// that would round to infinity rounds down instead); v keeps what is left.
template <typename T>
__device__ __forceinline__ __nv_bfloat16 next_part(float &v)
{
    __nv_bfloat16 r = __float2bfloat16(v);
    if (sizeof(T) == 4) {
        float f = __bfloat162float(r);
        if (isinf(f) && !isinf(v)) {
            f = __uint_as_float(__float_as_uint(v) & 0xffff0000u);
            r = __float2bfloat16(f);
        }
        v = isfinite(v) ? v - f : 0.f;
    }
    return r;
}

// An operand of the products that the TMA unit cannot read as it lies (fp32,
// row pitch or base not a multiple of 16 bytes): dst[part][row][dp] with
// zeros past d.  One thread per 8 elements; HBM-bound.
template <typename T>
__global__ void __launch_bounds__(256)
operand_kernel(const T *__restrict__ src, __nv_bfloat16 *__restrict__ dst, int rows, int d, int dp, long part_stride,
               int vec)
{
    const int per = dp / 8;
    const long n = (long)rows * per;
    for (long x = (long)blockIdx.x * 256 + threadIdx.x; x < n; x += (long)gridDim.x * 256) {
        const long i = x / per;
        const int c = (int)(x - i * per) * 8;
        float v[8];
        if (vec) {   // 16-byte aligned rows
            __align__(16) T t[8];
#pragma unroll
            for (int j = 0; j < (int)sizeof(T) / 2; ++j)
                reinterpret_cast<uint4 *>(t)[j] = reinterpret_cast<const uint4 *>(src + i * d + c)[j];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = to_f(t[j]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = c + j < d ? to_f(src[i * d + c + j]) : 0.f;
        }
        const long at = i * dp + c;
#pragma unroll
        for (int part = 0; part < (sizeof(T) == 4 ? 3 : 1); ++part) {
            __align__(16) __nv_bfloat16 b[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) b[j] = next_part<T>(v[j]);
            *reinterpret_cast<uint4 *>(dst + part * part_stride + at) = *reinterpret_cast<const uint4 *>(b);
        }
    }
}

// h transposed for dW: dst[part][column][rp], rows of factor 0 as zeros
// whatever they hold, zeros from `rows` to rp (a multiple of 8).  64 x 64
// elements per block through shared memory, 16 bytes per access of memory
// (element loads where rows are not aligned); HBM-bound.
template <typename T>
__global__ void __launch_bounds__(256)
transpose_kernel(const T *__restrict__ src, __nv_bfloat16 *__restrict__ dst, int rows, int d, long rp,
                 long part_stride, const float *__restrict__ coef, int vec)
{
    constexpr int kParts = sizeof(T) == 4 ? 3 : 1;
    __shared__ __nv_bfloat16 s[kParts][64][65];   // [column][row]
    const long i0 = (long)blockIdx.x * 64;
    const int c0 = blockIdx.y * 64;
#pragma unroll
    for (int x = threadIdx.x; x < 512; x += 256) {
        const int y = x >> 3, c = (x & 7) * 8;
        const long i = i0 + y;
        float v[8];
        const bool live = i < rows && coef[i] != 0.f;
        if (live && vec && c0 + c < d) {
            __align__(16) T t[8];
#pragma unroll
            for (int j = 0; j < (int)sizeof(T) / 2; ++j)
                reinterpret_cast<uint4 *>(t)[j] = reinterpret_cast<const uint4 *>(src + i * d + c0 + c)[j];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = to_f(t[j]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = live && c0 + c + j < d ? to_f(src[i * d + c0 + c + j]) : 0.f;
        }
#pragma unroll
        for (int part = 0; part < kParts; ++part)
#pragma unroll
            for (int j = 0; j < 8; ++j) s[part][c + j][y] = next_part<T>(v[j]);
    }
    __syncthreads();
#pragma unroll
    for (int x = threadIdx.x; x < 512; x += 256) {
        const int c = x >> 3, y = (x & 7) * 8;
        if (c0 + c >= d || i0 + y >= rp) continue;
#pragma unroll
        for (int part = 0; part < kParts; ++part) {
            __align__(16) __nv_bfloat16 b[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) b[j] = s[part][c][y + j];
            *reinterpret_cast<uint4 *>(dst + part * part_stride + (c0 + c) * rp + i0 + y) =
                *reinterpret_cast<const uint4 *>(b);
        }
    }
}

// out[row][c] = the sum of the slots' [row][dp] partial products, in order
template <typename T>
__global__ void __launch_bounds__(256)
slots_kernel(const float *__restrict__ slot, int slots, long slot_stride, T *__restrict__ out, int rows, int d, int dp)
{
    const int per = (d + 3) / 4;
    const long n = (long)rows * per;
    for (long x = (long)blockIdx.x * 256 + threadIdx.x; x < n; x += (long)gridDim.x * 256) {
        const long i = x / per;
        const int c = (int)(x - i * per) * 4;
        float4 sum = *reinterpret_cast<const float4 *>(slot + i * dp + c);
        for (int k = 1; k < slots; ++k) {
            const float4 e = *reinterpret_cast<const float4 *>(slot + k * slot_stride + i * dp + c);
            sum.x += e.x, sum.y += e.y, sum.z += e.z, sum.w += e.w;
        }
        const float v[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (c + j < d) out[i * d + c + j] = from_f<T>(v[j]);
    }
}

// Joins the strips of a row's softmax and its listed logits: 32 rows per
// block (coalesced over rows), 32 threads of a column of the block share a
// row's slots and entries.
__global__ void __launch_bounds__(1024)
loss_merge_kernel(const float2 *__restrict__ part, int slots, const float *__restrict__ ysel, LossRows r, float t2,
                  float *__restrict__ loss, float *__restrict__ lse, int rows)
{
    __shared__ float sm[32][33], sl[32][33];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const long i = (long)blockIdx.x * 32 + tx;
    float m = -INFINITY, l = 0.f;
    if (i < rows)
        for (int x = ty; x < slots; x += 32) {
            const float2 e = part[(long)x * rows + i];
            const float mm = fmaxf(m, e.x), ref = mm == -INFINITY ? 0.f : mm;
            l = l * exp2f(m - ref) + e.y * exp2f(e.x - ref);
            m = mm;
        }
    sm[ty][tx] = m;
    sl[ty][tx] = l;
    __syncthreads();
    // warp ty takes row ty of the block: lane tx one thread's part of it
    const long row = (long)blockIdx.x * 32 + ty;
    if (row >= rows) return;
    m = sm[tx][ty];
    l = sl[tx][ty];
    float mm = m;
#pragma unroll
    for (int o = 16; o; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
    const float ref = mm == -INFINITY ? 0.f : mm;
    l *= exp2f(m - ref);
#pragma unroll
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    const float y_lse = ref + log2f(l);
    float dot = 0.f;
    int any = 0;
    for (int k = tx; k < r.K; k += 32) {
        if (r.col[row * r.K + k] == kNoColumn) continue;
        any = 1;
        const float p = r.p[row * r.K + k];
        if (p != 0.f) dot += p * (y_lse - ysel[row * r.K + k]);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        dot += __shfl_xor_sync(0xffffffffu, dot, o);
        any |= __shfl_xor_sync(0xffffffffu, any, o);
    }
    if (tx == 0) {
        lse[row] = y_lse * kLn2;
        loss[row] = any && y_lse != -INFINITY ? t2 * (r.ent[row] + kLn2 * dot) : 0.f;
    }
}

// db[j] = the sum of the row groups' sums: 32 columns per block, 32 threads
// per column
__global__ void __launch_bounds__(1024)
dbias_kernel(const float *__restrict__ dbpart, int parts, long pitch, int cols, float *__restrict__ db)
{
    __shared__ float s[32][33];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const long j = (long)blockIdx.x * 32 + tx;
    float sum = 0.f;
    if (j < cols)
        for (int x = ty; x < parts; x += 32) sum += dbpart[x * pitch + j];
    s[ty][tx] = sum;
    __syncthreads();
    if (ty == 0 && j < cols) {
        float all = 0.f;
        for (int x = 0; x < 32; ++x) all += s[x][tx];
        db[j] = all;
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

constexpr size_t kPieceBytes = (size_t)256 << 20;  // at most this for one piece of dz and of copied weights
constexpr size_t kWeightBytes = (size_t)64 << 20;  // ... for the forward's copied weights
constexpr int kMaxSize = 1 << 30;                  // rows and vocabulary

long up(long a, long b) { return (a + b - 1) / b * b; }

// How a call is divided and where things lie in the workspace; from sizes,
// alignment and the number of SMs alone.
struct LossPlan {
    int parts, dp;          // bf16 parts of an element; operand row pitch (d rounded up to 8)
    bool copy_h, copy_w;
    int piece;              // vocabulary columns per piece
    int slots;              // forward: partial softmaxes per row over all pieces
    LossTiling dh;          // of a whole piece
    bool dh_slots;
    size_t col, p, ent, coef, l2, bz, ysel, part, h, ht, w, dz, dh_acc, dw_acc, dbpart, bytes;
};

LossPlan make_plan(int rows, int d, int vocab, int K, txl_dtype dtype, bool backward, bool h_ok, bool w_ok)
{
    LossPlan q;
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t o = at;
        at += (n + 255) / 256 * 256;
        return o;
    };
    const size_t n = (size_t)rows;
    q.parts = dtype == TXL_F32 ? 3 : 1;
    q.dp = (int)up(d, 8);
    const bool tma = dtype == TXL_BF16 && d % 8 == 0;
    q.copy_h = !tma || !h_ok;
    q.copy_w = !tma || !w_ok;
    // what a vocabulary column of a piece takes; pieces start at multiples of the widest tile
    const size_t per = ((backward ? n : 0) + (q.copy_w ? (size_t)q.dp : 0)) * q.parts * 2;
    size_t most = per ? (backward ? kPieceBytes : kWeightBytes) / per / kLossPieceUnit * kLossPieceUnit : (size_t)vocab;
    if (most < (size_t)kLossPieceUnit) most = kLossPieceUnit;
    if (backward)
        q.piece = gradient_piece(rows, d, vocab, q.parts, most < (size_t)kMaxSize ? (int)most : kMaxSize);
    else
        q.piece = most < (size_t)vocab ? (int)most : vocab;
    q.col = take(n * K * 4);
    q.p = take(n * K * 4);
    q.ent = take(n * 4);
    q.bz = take((size_t)vocab * 4 + 256);   // read in fours past the last column
    q.h = take(q.copy_h ? n * q.dp * q.parts * 2 : 0);
    q.w = take(q.copy_w ? (size_t)q.piece * q.dp * q.parts * 2 : 0);
    q.coef = q.l2 = q.ht = q.dz = q.dh_acc = q.dw_acc = q.dbpart = q.ysel = q.part = 0;
    q.slots = 0;
    q.dh_slots = false;
    if (!backward) {
        for (long v0 = 0; v0 < vocab; v0 += q.piece)
            q.slots += kSlotsPerStrip *
                       vocab_strips(vocab_tiling(rows, (int)(vocab - v0 < q.piece ? vocab - v0 : q.piece), d, q.parts));
        q.ysel = take(n * K * 4);
        q.part = take(n * q.slots * 8);
    } else {
        q.coef = take(n * 4);
        q.l2 = take(n * 4);
        q.ht = take((size_t)d * up(rows, 8) * q.parts * 2);
        q.dz = take(n * up(q.piece, 64) * q.parts * 2);
        q.dh_slots = q.piece < vocab;
        // the last, narrower piece may split dW further
        LossTiling dw, dh_last, dw_last;
        const int last = vocab % q.piece ? vocab % q.piece : q.piece;
        gradient_tiling(rows, d, q.piece, q.piece, q.parts, q.dh_slots, 0, &q.dh, &dw);
        gradient_tiling(rows, d, last, q.piece, q.parts, q.dh_slots, q.dh.splits, &dh_last, &dw_last);
        const size_t dw_whole = (size_t)dw.splits * q.piece, dw_rest = (size_t)dw_last.splits * last;
        // whatever the output's alignment: the products go to the slots where TMA cannot write it
        q.dh_acc = take((size_t)q.dh.splits * n * q.dp * 4);
        q.dw_acc = take((dw_whole > dw_rest ? dw_whole : dw_rest) * q.dp * 4);
        q.dbpart = take((size_t)up(rows, 32) / 32 * up(q.piece, 64) * 4);
    }
    q.bytes = at ? at : 256;
    return q;
}

// The plans of the shapes used last (a plan's search takes up to a
// millisecond of host time).
struct PlanKey {
    int rows, d, vocab, K, dtype, flags, sms;
};
std::mutex g_plan_mu;
struct PlanEntry {
    PlanKey key;
    LossPlan plan;
};
PlanEntry g_plans[64];
int g_plan_n = 0, g_plan_next = 0;

LossPlan loss_plan(int rows, int d, int vocab, int K, txl_dtype dtype, bool backward, bool h_ok, bool w_ok)
{
    const PlanKey key = {rows, d, vocab, K, (int)dtype, backward * 4 + h_ok * 2 + w_ok, device_sm_count()};
    {
        std::lock_guard<std::mutex> lock(g_plan_mu);
        for (int x = 0; x < g_plan_n; ++x)
            if (!memcmp(&g_plans[x].key, &key, sizeof(key))) return g_plans[x].plan;
    }
    const LossPlan plan = make_plan(rows, d, vocab, K, dtype, backward, h_ok, w_ok);
    std::lock_guard<std::mutex> lock(g_plan_mu);
    g_plans[g_plan_next].key = key;
    g_plans[g_plan_next].plan = plan;
    g_plan_next = (g_plan_next + 1) % 64;
    if (g_plan_n < 64) ++g_plan_n;
    return plan;
}

// The bytes either direction may need whatever the buffers' alignment.
size_t loss_bytes(int rows, int d, int vocab, int K, txl_dtype dtype, bool backward)
{
    size_t most = 0;
    for (int b = 0; b <= (backward ? 1 : 0); ++b)
        for (int ok = 0; ok < 4; ++ok) {
            const size_t n = loss_plan(rows, d, vocab, K, dtype, b, ok & 1, ok & 2).bytes;
            most = n > most ? n : most;
        }
    return most;
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
    *bytes = loss_bytes(rows, d, vocab, K, dtype, backward != 0);
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
    if (a.rows > 0 && a.ws_bytes < loss_plan(a.rows, a.d, a.vocab, a.K, a.dtype, backward, al(a.h, 16), al(a.w, 16)).bytes)
        return TXL_ERR_INVALID;
    return TXL_OK;
}

float alpha_of(const LossArgs &a) { return 1.f / (kLn2 * (a.temp != 0.f ? a.temp : 1.f)); }

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
    if (a.bias)
        bias_scale_kernel<<<(a.vocab + 255) / 256, 256, 0, a.s>>>(a.bias, alpha_of(a),
                                                                  (float *)((unsigned char *)a.ws + q.bz), a.vocab);
    return cudaGetLastError();
}

// a copied operand: h, or a piece of W
cudaError_t copy_operand(const LossArgs &a, const LossPlan &q, const void *src, size_t at, int rows, long part_stride)
{
    __nv_bfloat16 *dst = (__nv_bfloat16 *)((unsigned char *)a.ws + at);
    const long n = (long)rows * (q.dp / 8), want = (n + 255) / 256, most = 16L * device_sm_count();
    const int grid = (int)(want < most ? want : most);
    if (a.dtype == TXL_F32)
        operand_kernel<float><<<grid, 256, 0, a.s>>>((const float *)src, dst, rows, a.d, q.dp, part_stride,
                                                     a.d % 8 == 0 && al(src, 16));
    else
        operand_kernel<__nv_bfloat16><<<grid, 256, 0, a.s>>>((const __nv_bfloat16 *)src, dst, rows, a.d, q.dp,
                                                             part_stride, a.d % 8 == 0 && al(src, 16));
    return cudaGetLastError();
}

cudaError_t h_operand(const LossArgs &a, const LossPlan &q, LossMatrix *m)
{
    if (!q.copy_h) {
        *m = {a.h, a.d, 0, a.rows, a.d, 1};
        return cudaSuccess;
    }
    const long stride = (long)a.rows * q.dp;
    *m = {(unsigned char *)a.ws + q.h, q.dp, stride, a.rows, q.dp, q.parts};
    return copy_operand(a, q, a.h, q.h, a.rows, stride);
}

// h^T for dW
cudaError_t ht_operand(const LossArgs &a, const LossPlan &q, const float *coef, LossMatrix *m)
{
    const long rp = up(a.rows, 8), stride = a.d * rp;
    __nv_bfloat16 *dst = (__nv_bfloat16 *)((unsigned char *)a.ws + q.ht);
    *m = {dst, rp, stride, a.d, (int)rp, q.parts};
    const dim3 grid((unsigned)((a.rows + 63) / 64), (unsigned)((a.d + 63) / 64));
    const int vec = a.d % 8 == 0 && al(a.h, 16);
    if (grid.y > 65535) return cudaErrorNotSupported;
    if (a.dtype == TXL_F32)
        transpose_kernel<float><<<grid, 256, 0, a.s>>>((const float *)a.h, dst, a.rows, a.d, rp, stride, coef, vec);
    else
        transpose_kernel<__nv_bfloat16><<<grid, 256, 0, a.s>>>((const __nv_bfloat16 *)a.h, dst, a.rows, a.d, rp, stride,
                                                               coef, vec);
    return cudaGetLastError();
}

// columns v0 .. v0+cols of the vocabulary
cudaError_t w_operand(const LossArgs &a, const LossPlan &q, long v0, int cols, LossMatrix *m)
{
    const size_t esz = a.dtype == TXL_F32 ? 4 : 2;
    const void *src = (const unsigned char *)a.w + (size_t)v0 * a.d * esz;
    if (!q.copy_w) {
        *m = {src, a.d, 0, cols, a.d, 1};
        return cudaSuccess;
    }
    const long stride = (long)q.piece * q.dp;
    *m = {(unsigned char *)a.ws + q.w, q.dp, stride, cols, q.dp, q.parts};
    return copy_operand(a, q, src, q.w, cols, stride);
}

cudaError_t sum_slots(const LossArgs &a, const LossPlan &q, const float *slot, int slots, long stride, void *out,
                      int rows)
{
    const long n = (long)rows * ((a.d + 3) / 4), want = (n + 255) / 256, most = 16L * device_sm_count();
    const int grid = (int)(want < most ? want : most);
    if (a.dtype == TXL_F32)
        slots_kernel<float><<<grid, 256, 0, a.s>>>(slot, slots, stride, (float *)out, rows, a.d, q.dp);
    else
        slots_kernel<__nv_bfloat16><<<grid, 256, 0, a.s>>>(slot, slots, stride, (__nv_bfloat16 *)out, rows, a.d, q.dp);
    return cudaGetLastError();
}

cudaError_t run_fwd(const LossArgs &a)
{
    const LossPlan q = loss_plan(a.rows, a.d, a.vocab, a.K, a.dtype, false, al(a.h, 16), al(a.w, 16));
    unsigned char *ws = (unsigned char *)a.ws;
    const LossRows r = rows_at(a, q);
    const float *bz = (const float *)(ws + q.bz);
    float2 *part = (float2 *)(ws + q.part);
    LossMatrix h, w;
    cudaError_t e = launch_rows(a, r, q, false);
    if (e == cudaSuccess) e = h_operand(a, q, &h);
    long slot = 0;
    for (long v0 = 0; e == cudaSuccess && v0 < a.vocab; v0 += q.piece) {
        const int cols = (int)(a.vocab - v0 < q.piece ? a.vocab - v0 : q.piece);
        const LossTiling t = vocab_tiling(a.rows, cols, a.d, q.parts);
        e = w_operand(a, q, v0, cols, &w);
        if (e == cudaSuccess)
            e = launch_loss_lse(h, w, a.bias ? bz + v0 : nullptr, (int)v0, alpha_of(a), r, (float *)(ws + q.ysel),
                                part + slot * a.rows, t, a.s);
        slot += kSlotsPerStrip * vocab_strips(t);
    }
    if (e != cudaSuccess) return e;
    const float t2 = a.temp != 0.f ? a.temp * a.temp : 1.f;
    loss_merge_kernel<<<(a.rows + 31) / 32, 1024, 0, a.s>>>(part, q.slots, (const float *)(ws + q.ysel), r, t2, a.loss,
                                                            a.lse_out, a.rows);
    return cudaGetLastError();
}

LossOutput direct_out(const LossArgs &a, void *p)
{
    LossOutput o;
    o.base = p;
    o.pitch = a.d;
    o.slot_stride = 0;
    o.f32 = a.dtype == TXL_F32;
    o.add = false;
    return o;
}

LossOutput slot_out(float *p, long pitch, long stride, bool add)
{
    LossOutput o;
    o.base = p;
    o.pitch = pitch;
    o.slot_stride = stride;
    o.f32 = true;
    o.add = add;
    return o;
}

cudaError_t run_bwd(const LossArgs &a)
{
    const LossPlan q = loss_plan(a.rows, a.d, a.vocab, a.K, a.dtype, true, al(a.h, 16), al(a.w, 16));
    unsigned char *ws = (unsigned char *)a.ws;
    const LossRows r = rows_at(a, q);
    const float *bz = (const float *)(ws + q.bz);
    const size_t esz = a.dtype == TXL_F32 ? 4 : 2;
    const bool tma_out = ((size_t)a.d * esz) % 16 == 0;   // rows that a TMA store can address
    LossMatrix h, ht, w;
    cudaError_t e = launch_rows(a, r, q, true);
    if (e == cudaSuccess) e = h_operand(a, q, &h);
    if (e == cudaSuccess && a.dw) e = ht_operand(a, q, r.coef, &ht);
    for (long v0 = 0; e == cudaSuccess && v0 < a.vocab; v0 += q.piece) {
        const int cols = (int)(a.vocab - v0 < q.piece ? a.vocab - v0 : q.piece);
        const long pitch = up(cols, 64);
        const LossMatrix dz = {ws + q.dz, pitch, (long)a.rows * pitch, a.rows, cols, q.parts};
        float *dbp = a.db ? (float *)(ws + q.dbpart) : nullptr;
        e = w_operand(a, q, v0, cols, &w);
        if (e == cudaSuccess)
            e = launch_loss_dz(h, w, a.bias ? bz + v0 : nullptr, (int)v0, alpha_of(a), r, dz, dbp,
                               vocab_tiling(a.rows, cols, a.d, q.parts), a.s);
        if (e == cudaSuccess && a.db) {
            dbias_kernel<<<(cols + 31) / 32, 1024, 0, a.s>>>(dbp, (a.rows + 31) / 32, pitch, cols, a.db + v0);
            e = cudaGetLastError();
        }
        // both gradients of the piece in one launch
        LossContraction job[2];
        int n = 0;
        LossTiling dh, dw;
        gradient_tiling(a.rows, a.d, cols, q.piece, q.parts, q.dh_slots, q.dh.splits, &dh, &dw);
        const long hs = (long)a.rows * q.dp, ws_stride = (long)cols * q.dp;
        float *acc_h = (float *)(ws + q.dh_acc), *acc_w = (float *)(ws + q.dw_acc);
        // every piece splits dh the same way, so that each adds to the same slots
        const bool h_direct = !q.dh_slots && dh.splits == 1 && tma_out && al(a.dh, 16);
        void *dw_out = a.dw ? (unsigned char *)a.dw + (size_t)v0 * a.d * esz : nullptr;
        const bool w_direct = dw.splits == 1 && tma_out && al(dw_out, 16);
        if (a.dh) {
            LossContraction &j = job[a.dw && dw.first ? 1 : 0];
            ++n;
            j.a = dh.turned ? w : dz;
            j.b = dh.turned ? dz : w;
            j.a_t = j.b_t = j.out_t = dh.turned;
            j.m = dh.turned ? a.d : a.rows;
            j.n = dh.turned ? a.rows : a.d;
            j.k = cols;
            j.out = h_direct ? direct_out(a, a.dh) : slot_out(acc_h, q.dp, hs, v0 > 0);
            j.t = dh;
        }
        if (a.dw) {
            LossContraction &j = job[a.dh && !dw.first ? 1 : 0];
            ++n;
            j.a = dz;
            j.b = ht;
            j.a_t = j.b_t = true;
            j.out_t = false;
            j.m = cols;
            j.n = a.d;
            j.k = a.rows;
            j.out = w_direct ? direct_out(a, dw_out) : slot_out(acc_w, q.dp, ws_stride, false);
            j.t = dw;
        }
        if (e == cudaSuccess && n) e = launch_loss_gradients(job, n, q.parts, a.s);
        if (e == cudaSuccess && a.dh && !h_direct && v0 + cols == a.vocab)
            e = sum_slots(a, q, acc_h, dh.splits, hs, a.dh, a.rows);
        if (e == cudaSuccess && a.dw && !w_direct) e = sum_slots(a, q, acc_w, dw.splits, ws_stride, dw_out, cols);
    }
    return e;
}

txl_status loss_fwd(const LossArgs &a)
{
    const txl_status st = loss_checks(a, false);
    if (st != TXL_OK || a.rows == 0) return st;
    const cudaError_t e = run_fwd(a);
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
        e = run_bwd(a);
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

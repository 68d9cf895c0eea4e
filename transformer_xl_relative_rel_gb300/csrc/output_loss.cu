// output_loss.cu -- the output layer's losses without their logits
// (txl_softmax_xent_*, txl_distill_*):
//
//   z = h W^T + bias,  lse_i = log sum_j exp(z_ij / t),
//   loss_i = t^2 sum_k p_ik (log p_ik - z_{i,idx_ik} / t + lse_i)
//
// with p the teacher's softmax over its kept entries; cross entropy is the
// same with one entry of weight 1 (the target itself) and t = 1, so one set
// of kernels serves both:
//
//   loss_prep_kernel   the row lists, operands laid out for the products;
//   forward            one pass over the vocabulary (loss_products.cu) leaves
//                      a maximum and a sum per row and strip of vocabulary
//                      tiles and the logits of the listed columns;
//                      loss_merge_kernel joins them;
//   backward           for each piece of the vocabulary: dz (one piece of it
//                      in the workspace), then dh += dz W and dW = dz^T h in
//                      one launch; loss_finish_kernel adds up what lies in
//                      parts (the column sums of dz, split products).
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

// ------------------------------------------------------------ preparation
// What has to be ready before the products, in one launch whose blocks take
// different parts (none of them for a forward cross entropy of aligned bf16
// operands): the teacher's row lists, unaligned biases, operands that the TMA
// unit cannot read as they lie, and (backward) h transposed.  Bound by memory
// latency (each element is read and written once): h^T of 6144 x 1024 in 11
// us, with 16384 rows of 64 listed columns and 16384 x 512 in 47 us.
struct CopyJob {
    const void *src;
    __nv_bfloat16 *dst;
    int rows, blocks;
    long part_stride;
    int vec;
};
struct PrepArgs {
    const int64_t *idx;
    const void *logits;   // NULL: cross entropy
    int logits_f32;
    float inv_t;
    LossRows r;
    int rows, vocab, K2;
    const float *bias;          // copied where it is not 16-byte aligned
    float *bias_copy;
    int d, dp;
    CopyJob copy[2];
    // h^T
    const void *h;
    __nv_bfloat16 *ht;
    long rp, ht_stride;
    int h_vec, t_cols;    // column blocks of the transpose
    int twice;            // with h's rows once more behind the first (for the second part of dz)
    int row_blocks, bias_blocks, t_blocks;
};

__device__ __forceinline__ float teacher_logit(const PrepArgs &p, long at)
{
    return p.logits_f32 ? static_cast<const float *>(p.logits)[at]
                        : to_f(static_cast<const __nv_bfloat16 *>(p.logits)[at]);
}
__device__ __forceinline__ bool teacher_valid(const PrepArgs &p, long at)
{
    const int64_t e = p.idx[at];
    return e >= 0 && e < p.vocab && teacher_logit(p, at) != -INFINITY;
}

// distillation: the softmax of a row's valid entries at temperature t, then
// the entries sorted by the parity of their column's 64-column chunk and the
// column (a bitonic network over the next power of two).  One warp per row;
// K2 entries of shared memory per warp.  Logits are scaled as differences from
// the row's largest: scaled first, a row of the type's lowest values at t < 1
// would be -infinity throughout, and its weights NaN instead of alike.
constexpr unsigned kNoKey = 0xffffffffu, kOdd = 1u << 31;
__device__ __forceinline__ void distill_rows(const PrepArgs &p, unsigned *sc, float *sp)
{
    const int lane = threadIdx.x & 31, K = p.r.K, K2 = p.K2;
    const long i = (long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (i >= p.rows) return;
    const long base = i * K;
    float top = -INFINITY;
    for (int k = lane; k < K2; k += 32) {
        const bool valid = k < K && teacher_valid(p, base + k);
        const unsigned c = valid ? (unsigned)p.idx[base + k] : 0u;
        sc[k] = valid ? c | (c & 64u ? kOdd : 0u) : kNoKey;
        sp[k] = valid ? teacher_logit(p, base + k) : -INFINITY;
        top = fmaxf(top, sp[k]);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    float sum = 0.f;
    for (int k = lane; k < K2; k += 32)
        if (sc[k] != kNoKey) sum += expf((sp[k] - top) * p.inv_t);
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float lt = logf(sum);
    float ent = 0.f;
    for (int k = lane; k < K2; k += 32) {
        float w = 0.f;
        if (sc[k] != kNoKey) {
            const float lp = (sp[k] - top) * p.inv_t - lt;
            w = expf(lp);
            if (w != 0.f) ent += w * lp;   // (a NaN teacher logit stays NaN)
        }
        sp[k] = w;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) ent += __shfl_xor_sync(0xffffffffu, ent, o);
    __syncwarp();
    for (int len = 2; len <= K2; len <<= 1)
        for (int step = len >> 1; step; step >>= 1) {
            for (int x = lane; x < K2 / 2; x += 32) {
                const int a = 2 * x - (x & (step - 1)), b = a + step;
                const bool up = (a & len) == 0;
                const unsigned ca = sc[a], cb = sc[b];
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
    int even = 0;
    for (int k = lane; k < K; k += 32) {
        const unsigned c = sc[k];
        p.r.col[base + k] = c == kNoKey ? kNoColumn : (int)(c & ~kOdd);
        p.r.p[base + k] = sp[k];
        even += !(c & kOdd);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) even += __shfl_xor_sync(0xffffffffu, even, o);
    if (lane == 0) {
        p.r.ent[i] = ent;
        p.r.even[i] = even;
    }
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

// 8 elements of a row from column c on, zeros past d; vec: bytes at a time
// that the rows' alignment and length allow (16, 4 or an element)
template <typename T>
__device__ __forceinline__ void load8(const T *row, int c, int d, int vec, float (&v)[8])
{
    if (sizeof(T) == 2 && vec == 4) {
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const uint32_t w = c + j < d ? *reinterpret_cast<const uint32_t *>(row + c + j) : 0u;
            v[j] = __uint_as_float(w << 16);
            v[j + 1] = __uint_as_float(w & 0xffff0000u);
        }
    } else if (vec == 16 && c < d) {
        __align__(16) T t[8];
#pragma unroll
        for (int j = 0; j < (int)sizeof(T) / 2; ++j)
            reinterpret_cast<uint4 *>(t)[j] = reinterpret_cast<const uint4 *>(row + c)[j];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = to_f(t[j]);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = c + j < d ? to_f(row[c + j]) : 0.f;
    }
}

// dst[part][row][dp], zeros past d; one thread per 8 elements
template <typename T>
__device__ __forceinline__ void copy_rows(const CopyJob &c, int d, int dp, int block)
{
    const int per = dp / 8;
    const long n = (long)c.rows * per;
    for (long x = (long)block * 256 + threadIdx.x; x < n; x += (long)c.blocks * 256) {
        const long i = x / per;
        const int at = (int)(x - i * per) * 8;
        float v[8];
        load8(static_cast<const T *>(c.src) + i * d, at, d, c.vec, v);
#pragma unroll
        for (int part = 0; part < (sizeof(T) == 4 ? 3 : 1); ++part) {
            __align__(16) __nv_bfloat16 b[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) b[j] = next_part<T>(v[j]);
            *reinterpret_cast<uint4 *>(c.dst + part * c.part_stride + i * dp + at) = *reinterpret_cast<const uint4 *>(b);
        }
    }
}

// h transposed for dW: ht[part][column][rp], rows of factor 0 as zeros
// whatever they hold, zeros from `rows` to rp (a multiple of 8).  64 x 64
// elements per block through shared memory (s: [part][column][65]), 16 bytes
// per access of memory.
template <typename T>
__device__ __forceinline__ void transpose_rows(const PrepArgs &p, int block, __nv_bfloat16 *s, int *live)
{
    constexpr int kParts = sizeof(T) == 4 ? 3 : 1;
    const long i0 = (long)(block / p.t_cols) * 64;
    const int c0 = (block % p.t_cols) * 64;
    if (threadIdx.x < 64) {
        const long i = i0 + threadIdx.x;
        bool valid = false;
        if (i < p.rows) {
            if (p.r.target)
                valid = target_column(p.r, i) != kNoColumn;
            else
                for (int k = 0; k < p.r.K && !valid; ++k) valid = teacher_valid(p, i * p.r.K + k);
            valid = row_factor(p.r, i, valid) != 0.f;
        }
        live[threadIdx.x] = valid;
    }
    __syncthreads();
    for (int x = threadIdx.x; x < 512; x += 256) {
        const int y = x >> 3, c = (x & 7) * 8;
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (live[y]) load8(static_cast<const T *>(p.h) + (i0 + y) * p.d, c0 + c, p.d, p.h_vec, v);
#pragma unroll
        for (int part = 0; part < kParts; ++part)
#pragma unroll
            for (int j = 0; j < 8; ++j) s[(part * 64 + c + j) * 65 + y] = next_part<T>(v[j]);
    }
    __syncthreads();
    for (int x = threadIdx.x; x < 512; x += 256) {
        const int c = x >> 3, y = (x & 7) * 8;
        if (c0 + c >= p.d || i0 + y >= p.rp) continue;
        if (p.twice) {
            __nv_bfloat16 *to = p.ht + (c0 + c) * p.rp + i0 + y;
            for (int j = 0; j < 8 && i0 + y + j < p.rows; ++j) to[j] = to[p.rows + j] = s[c * 65 + y + j];
            continue;
        }
#pragma unroll
        for (int part = 0; part < kParts; ++part) {
            __align__(16) __nv_bfloat16 b[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) b[j] = s[(part * 64 + c) * 65 + y + j];
            *reinterpret_cast<uint4 *>(p.ht + part * p.ht_stride + (c0 + c) * p.rp + i0 + y) =
                *reinterpret_cast<const uint4 *>(b);
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(256) loss_prep_kernel(const __grid_constant__ PrepArgs p)
{
    // the lists of 8 rows, or a transposed block
    constexpr int kBlock = (sizeof(T) == 4 ? 3 : 1) * 64 * 65 * 2, kLists = 8 * kMaxTopK * 8;
    __shared__ __align__(16) unsigned char s[kBlock > kLists ? kBlock : kLists];
    __shared__ int live[64];
    loss_kernel_begin();
    loss_kernel_wait();
    int b = (int)blockIdx.x;
    if (b < p.row_blocks) {
        distill_rows(p, reinterpret_cast<unsigned *>(s) + (threadIdx.x >> 5) * p.K2,
                     reinterpret_cast<float *>(s) + (8 + (threadIdx.x >> 5)) * p.K2);
        return;
    }
    b -= p.row_blocks;
    if (b < p.bias_blocks) {
        const long j = (long)b * 256 + threadIdx.x;
        if (j < p.vocab) p.bias_copy[j] = p.bias[j];
        return;
    }
    b -= p.bias_blocks;
    if (b < p.t_blocks) {
        transpose_rows<T>(p, b, reinterpret_cast<__nv_bfloat16 *>(s), live);
        return;
    }
    b -= p.t_blocks;
    if (b < p.copy[0].blocks)
        copy_rows<T>(p.copy[0], p.d, p.dp, b);
    else
        copy_rows<T>(p.copy[1], p.d, p.dp, b - p.copy[0].blocks);
}

// ------------------------------------------------------------ finishing
// What follows the products of a vocabulary piece, in one launch: the column
// sums of dz from those of its row groups, and gradients that lie in slots.
// Bound by the latency of reading them: 192 row groups of 32768 columns (25
// MB, none of it in L2) in 11 us.
struct SumJob {
    const float *slot;
    void *out;
    int slots, rows, blocks;
    long stride;
};
struct FinishArgs {
    const float *dbpart;
    float *db;
    int parts, cols, db_blocks, db_lanes;
    long pitch;
    int d, dp;
    SumJob sum[2];
};

// out[row][c] = the sum of the slots' [row][dp] partial products, in order
template <typename T>
__device__ __forceinline__ void sum_slots(const SumJob &j, int d, int dp, int block)
{
    const int per = (d + 3) / 4;
    const long n = (long)j.rows * per;
    for (long x = (long)block * 1024 + threadIdx.x; x < n; x += (long)j.blocks * 1024) {
        const long i = x / per;
        const int c = (int)(x - i * per) * 4;
        float4 sum = *reinterpret_cast<const float4 *>(j.slot + i * dp + c);
        for (int k = 1; k < j.slots; ++k) {
            const float4 e = *reinterpret_cast<const float4 *>(j.slot + k * j.stride + i * dp + c);
            sum.x += e.x, sum.y += e.y, sum.z += e.z, sum.w += e.w;
        }
        const float v[4] = {sum.x, sum.y, sum.z, sum.w};
        T *out = static_cast<T *>(j.out) + i * d + c;
#pragma unroll
        for (int y = 0; y < 4; ++y)
            if (c + y < d) out[y] = from_f<T>(v[y]);
    }
}

template <typename T>
__global__ void __launch_bounds__(1024) loss_finish_kernel(const __grid_constant__ FinishArgs p)
{
    __shared__ float s[1024];
    loss_kernel_begin();
    loss_kernel_wait();
    int b = (int)blockIdx.x;
    if (b < p.db_blocks) {   // db_lanes threads per column, each some of the row groups
        const int wide = 1024 / p.db_lanes, tx = threadIdx.x % wide, ty = threadIdx.x / wide;
        const long j = (long)b * wide + tx;
        float sum = 0.f;
        if (j < p.cols)
#pragma unroll 8
            for (int x = ty; x < p.parts; x += p.db_lanes) sum += p.dbpart[x * p.pitch + j];
        s[threadIdx.x] = sum;
        __syncthreads();
        if (ty == 0 && j < p.cols) {
            for (int x = 1; x < p.db_lanes; ++x) sum += s[x * wide + tx];
            p.db[j] = sum;
        }
        return;
    }
    b -= p.db_blocks;
    if (b < p.sum[0].blocks)
        sum_slots<T>(p.sum[0], p.d, p.dp, b);
    else
        sum_slots<T>(p.sum[1], p.d, p.dp, b - p.sum[0].blocks);
}

// Joins the strips of a row's softmax and its listed logits: kRows rows per
// block (coalesced over rows), 1024 / kRows threads share a row's slots, then
// a warp its entries.  8 rows where there are few, so that more SMs read.
// Hardly more than its launch: 6144 rows 6 us, 16384 rows with 64 entries
// each 15 us.
template <int kRows>
__global__ void __launch_bounds__(1024)
loss_merge_kernel(const float2 *part, int slots, const float *ysel, LossRows r, float t2, float *loss, float *lse,
                  int rows)
{
    constexpr int kLanes = 1024 / kRows;
    __shared__ float sm[kRows][kLanes + 1], sl[kRows][kLanes + 1];
    loss_kernel_begin();
    loss_kernel_wait();
    {
        const int tx = threadIdx.x % kRows, ty = threadIdx.x / kRows;
        const long i = (long)blockIdx.x * kRows + tx;
        float m = -INFINITY, l = 0.f;
        if (i < rows) {
#pragma unroll 4
            for (int x = ty; x < slots; x += kLanes) {
                const float2 e = part[(long)x * rows + i];
                const float mm = fmaxf(m, e.x), ref = mm == -INFINITY ? 0.f : mm;
                l = l * exp2f(m - ref) + e.y * exp2f(e.x - ref);
                m = mm;
            }
        }
        sm[tx][ty] = m;
        sl[tx][ty] = l;
    }
    __syncthreads();
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const long row = (long)blockIdx.x * kRows + ty;
    if (ty >= kRows || row >= rows) return;
    float mm = -INFINITY;
    for (int x = tx; x < kLanes; x += 32) mm = fmaxf(mm, sm[ty][x]);
#pragma unroll
    for (int o = 16; o; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
    const float ref = mm == -INFINITY ? 0.f : mm;
    float l = 0.f;
    for (int x = tx; x < kLanes; x += 32) l += sl[ty][x] * exp2f(sm[ty][x] - ref);
#pragma unroll
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    row_loss(r, ysel, ref, l, t2, row, tx, loss, lse);
}

// ---------------------------------------------------------------- host side
bool al(const void *p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

bool overlap(const void *a, size_t na, const void *b, size_t nb)
{
    if (!a || !b || na == 0 || nb == 0) return false;
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return x < y + nb && y < x + na;
}

// At most this for one piece of dz and of copied weights, where 256 columns take
// no more (rows are not divided: dz of 2^20 bf16 rows, a third of that in fp32).
// Smaller pieces would stay in L2, but each costs a launch and a drain: forward
// of fp32 20 x 1024 x 131072 with 64, 128, 256, 512 MB of weights 558, 545, 463,
// 410 us, bf16 128 x 769 x 131072 163, 141, 130, 130 us.
constexpr size_t kPieceBytes = (size_t)512 << 20;
constexpr int kMaxSize = 1 << 30;                  // rows and vocabulary
// d_model: the sum of a tile's products over it has to end well within the limit of the kernels'
// waits (2 s; one SM's share of HBM delivers 2^24 columns of a bf16 tile's 256 rows in about 0.2 s)
constexpr int kMaxWidth = 1 << 24;
constexpr int64_t kMaxElements = (int64_t)1 << 40; // of h and of w

long up(long a, long b) { return (a + b - 1) / b * b; }

// How a call is divided and where things lie in the workspace; from sizes,
// alignment and the number of SMs alone.
struct LossPlan {
    int dz_rows;            // rows of dz with its parts (dz_rows())
    int parts, dp;          // bf16 parts of an element; operand row pitch (d rounded up to 8)
    bool few;               // on the CUDA cores, ...
    FewShape shape;
    bool copy_h, copy_w;
    int piece;              // vocabulary columns per piece
    int slots;              // forward: partial softmaxes per row over all pieces
    bool joined;            // ... which the kernel that makes them joins itself
    bool dh_slots;          // dh of several pieces adds up in slots
    // backward, for a whole piece and for the last one
    struct Piece {
        LossTiling vocab, dh, dw;
    } whole, last;
    size_t col, even, p, ent, bias, ysel, part, h, ht, w, dz, dh_acc, dw_acc, dbpart, bytes;
};

// h_ok, w_ok: 16-byte aligned bases of h and w
// (K 0: cross entropy)
LossPlan make_plan(int rows, int d, int vocab, int K, txl_dtype dtype, bool backward, bool h_ok, bool w_ok)
{
    LossPlan q = {};
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t o = at;
        at += (n + 255) / 256 * 256;
        return o;
    };
    const size_t n = (size_t)rows;
    const bool distill = K > 0;
    q.parts = dtype == TXL_F32 ? 3 : 1;
    q.dp = (int)up(d, 8);
    const bool tma = dtype == TXL_BF16 && d % 8 == 0;
    q.few = few_shape(rows, d, vocab, dtype == TXL_F32, w_ok, backward, &q.shape);
    if (q.few) {
        q.col = take(distill ? n * K * 4 : 0);
        q.p = take(distill ? n * K * 4 : 0);
        q.even = take(distill ? n * 4 : 0);
        q.ent = take(distill ? n * 4 : 0);
        q.slots = q.shape.blocks;
        q.joined = q.shape.joined;
        if (backward) {
            q.dh_acc = take(n * q.shape.blocks * q.shape.groups * d * 4);
        } else {
            q.ysel = take(n * (distill ? K : 1) * 4);
            q.part = take(n * q.slots * 8);
        }
        q.bytes = at ? at : 256;
        return q;
    }
    q.copy_h = !tma || !h_ok;
    q.copy_w = !tma || !w_ok;
    // what a vocabulary column of a piece takes; pieces start at multiples of the widest tile
    q.dz_rows = backward ? dz_rows(rows, q.parts) : 0;
    const size_t per = ((size_t)q.dz_rows + (q.copy_w ? (size_t)q.dp : 0)) * q.parts * 2;
    size_t most = per ? kPieceBytes / per / kLossPieceUnit * kLossPieceUnit : (size_t)vocab;
    if (most < (size_t)kLossPieceUnit) most = kLossPieceUnit;
    if (backward)
        q.piece = gradient_piece(rows, d, vocab, q.parts, most < (size_t)kMaxSize ? (int)most : kMaxSize);
    else
        q.piece = most < (size_t)vocab ? (int)most : vocab;
    q.col = take(distill ? n * K * 4 : 0);
    q.p = take(distill ? n * K * 4 : 0);
    q.even = take(distill ? n * 4 : 0);
    q.ent = take(distill ? n * 4 : 0);
    q.bias = take((size_t)vocab * 4);
    q.h = take(q.copy_h ? n * q.dp * q.parts * 2 : 0);
    q.w = take(q.copy_w ? (size_t)q.piece * q.dp * q.parts * 2 : 0);
    if (!backward) {
        const int last = vocab % q.piece ? vocab % q.piece : q.piece;
        q.whole.vocab = vocab_tiling(rows, q.piece, d, q.parts);
        q.last.vocab = vocab_tiling(rows, last, d, q.parts);
        const long more = (vocab - last) / q.piece;   // whole pieces before the last one
        q.slots = kSlotsPerStrip * (int)(more * vocab_strips(q.whole.vocab) + vocab_strips(q.last.vocab));
        q.joined = !distill && more == 0 && q.slots == kSlotsPerStrip;
        q.ysel = take(n * (distill ? K : 1) * 4);
        q.part = take(n * q.slots * 8);
    } else {
        q.ht = take((size_t)d * up(q.dz_rows, 64) * q.parts * 2);
        q.dz = take((size_t)q.dz_rows * up(q.piece, 64) * q.parts * 2);
        q.dh_slots = q.piece < vocab || q.dz_rows != rows;
        // every piece splits dh alike, so that each adds to the same slots; the last, narrower one may split dW further
        const int last = vocab % q.piece ? vocab % q.piece : q.piece;
        gradient_tiling(q.dz_rows, d, q.piece, q.piece, q.parts, q.dh_slots, 0, &q.whole.dh, &q.whole.dw);
        gradient_tiling(q.dz_rows, d, last, q.piece, q.parts, q.dh_slots, q.whole.dh.splits, &q.last.dh, &q.last.dw);
        q.whole.vocab = vocab_tiling(rows, q.piece, d, q.parts);
        q.last.vocab = vocab_tiling(rows, last, d, q.parts);
        auto dw_slots = [&](const LossTiling &t, int cols) {
            return t.splits > 1 ? (size_t)t.splits * cols * q.dp * 4 : 0;
        };
        const size_t dw_whole = dw_slots(q.whole.dw, q.piece), dw_last = dw_slots(q.last.dw, last);
        q.dh_acc = take(q.dh_slots || q.whole.dh.splits > 1 ? (size_t)q.whole.dh.splits * q.dz_rows * q.dp * 4 : 0);
        q.dw_acc = take(dw_whole > dw_last ? dw_whole : dw_last);
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
    // alignment that makes no difference is left out of the key
    FewShape few;
    if (few_shape(rows, d, vocab, dtype == TXL_F32, w_ok, backward, &few))
        h_ok = false;
    else if (dtype != TXL_BF16 || d % 8)
        h_ok = w_ok = false;
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

// The bytes either direction may need whatever the buffers' alignment (a query
// has no buffers; a call checks for what its own need, which is less where
// weights of many tokens are read in place).
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
    const int64_t *idx;            // [rows][K], or [rows] targets
    const void *t_logits;
    txl_dtype t_dtype;
    float temp;
    int rows, d, vocab, K;         // K 0: cross entropy
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
    if (rows < 0 || d < 1 || vocab < 1 || K < 0) return TXL_ERR_INVALID;
    if (K > kMaxTopK || rows > kMaxSize || vocab > kMaxSize || d > kMaxWidth) return TXL_ERR_UNSUPPORTED;
    if ((int64_t)(rows > vocab ? rows : vocab) * d > kMaxElements) return TXL_ERR_UNSUPPORTED;
    return TXL_OK;
}

txl_status loss_workspace(int rows, int d, int vocab, int K, txl_dtype dtype, int backward, size_t *bytes)
{
    if (!bytes) return TXL_ERR_INVALID;
    const txl_status st = loss_sizes(rows, d, vocab, K, dtype);
    if (st != TXL_OK) return st;
    // (no rows: nothing is planned or launched, and nothing is needed)
    *bytes = rows ? loss_bytes(rows, d, vocab, K, dtype, backward != 0) : 256;
    return TXL_OK;
}

float alpha_of(const LossArgs &a) { return 1.f / (kLn2 * (a.temp != 0.f ? a.temp : 1.f)); }

// (fills *plan when there are rows)
txl_status loss_checks(const LossArgs &a, bool backward, LossPlan *plan)
{
    const txl_status st = loss_sizes(a.rows, a.d, a.vocab, a.K, a.dtype);
    if (st != TXL_OK) return st;
    const bool distill = a.K > 0;
    if (distill) {
        if (a.t_dtype != TXL_F32 && a.t_dtype != TXL_BF16) return TXL_ERR_UNSUPPORTED;
        // (the loss is scaled by t^2: outside, an infinite or vanished factor of whatever rounding left)
        if (!(a.temp >= 0x1p-63f && a.temp <= 0x1p63f)) return TXL_ERR_INVALID;
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
                       {a.idx, n * (distill ? a.K : 1) * 8, 8, true},
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
    if (a.rows == 0) return TXL_OK;
    *plan = loss_plan(a.rows, a.d, a.vocab, a.K, a.dtype, backward, al(a.h, 16), al(a.w, 16));
    return a.ws_bytes < plan->bytes ? TXL_ERR_INVALID : TXL_OK;
}

LossRows rows_at(const LossArgs &a, const LossPlan &q)
{
    unsigned char *ws = (unsigned char *)a.ws;
    LossRows r;
    r.target = a.K == 0 ? a.idx : nullptr;
    r.col = (int *)(ws + q.col);
    r.even = (int *)(ws + q.even);
    r.p = (float *)(ws + q.p);
    r.ent = (float *)(ws + q.ent);
    r.K = a.K ? a.K : 1;
    r.vocab = a.vocab;
    r.t = a.temp != 0.f ? a.temp : 1.f;
    r.lse = a.lse;
    r.dloss = a.dloss;
    return r;
}

// the biases as the kernels read them
const float *bias_of(const LossArgs &a, const LossPlan &q)
{
    return q.few || !a.bias || al(a.bias, 16) ? a.bias : (const float *)((unsigned char *)a.ws + q.bias);
}

// blocks of a pass over n threads' work that strides over its grid
int grid_of(long n, int threads)
{
    const long want = (n + threads - 1) / threads, most = 16L * device_sm_count() * 256 / threads;
    return (int)(want < most ? want : most);
}

int load_width(const LossArgs &a, const void *p) { return a.d % 8 == 0 && al(p, 16) ? 16 : a.d % 2 == 0 && al(p, 4) ? 4 : 1; }

CopyJob copy_job(const LossArgs &a, const LossPlan &q, const void *src, size_t at, int rows, long part_stride)
{
    CopyJob c;
    c.src = src;
    c.dst = (__nv_bfloat16 *)((unsigned char *)a.ws + at);
    c.rows = rows;
    c.blocks = grid_of((long)rows * (q.dp / 8), 256);
    c.part_stride = part_stride;
    c.vec = load_width(a, src);
    return c;
}

cudaError_t launch_prep(const LossArgs &a, const PrepArgs &p)
{
    const long blocks = (long)p.row_blocks + p.bias_blocks + p.t_blocks + p.copy[0].blocks + p.copy[1].blocks;
    if (blocks > INT32_MAX) return cudaErrorNotSupported;
    if (blocks == 0) return cudaSuccess;
    return loss_launch(a.dtype == TXL_F32 ? loss_prep_kernel<float> : loss_prep_kernel<__nv_bfloat16>, (unsigned)blocks,
                       256, 0, 1, a.s, p);
}

// columns v0 .. v0+cols of the vocabulary: where they lie, or where *copy puts them
LossMatrix w_operand(const LossArgs &a, const LossPlan &q, long v0, int cols, CopyJob *copy)
{
    const size_t esz = a.dtype == TXL_F32 ? 4 : 2;
    const void *src = (const unsigned char *)a.w + (size_t)v0 * a.d * esz;
    if (!q.copy_w) return {src, a.d, 0, cols, a.d, 1};
    const long stride = (long)q.piece * q.dp;
    *copy = copy_job(a, q, src, q.w, cols, stride);
    return {(unsigned char *)a.ws + q.w, q.dp, stride, cols, q.dp, q.parts};
}

// The first preparation: row lists, biases, h, the vocabulary's first piece
// and, for dW, h^T.
cudaError_t prepare(const LossArgs &a, const LossPlan &q, const LossRows &r, LossMatrix *h, LossMatrix *w, LossMatrix *ht)
{
    PrepArgs p;
    memset(&p, 0, sizeof(p));
    p.idx = a.idx;
    p.logits = a.t_logits;
    p.logits_f32 = a.t_dtype == TXL_F32;
    p.inv_t = 1.f / r.t;
    p.r = r;
    p.rows = a.rows;
    p.vocab = a.vocab;
    for (p.K2 = 2; p.K2 < a.K;) p.K2 <<= 1;
    p.row_blocks = a.K ? (a.rows + 7) / 8 : 0;
    p.bias = a.bias;
    p.bias_copy = (float *)((unsigned char *)a.ws + q.bias);
    p.bias_blocks = bias_of(a, q) != a.bias ? (a.vocab + 255) / 256 : 0;
    if (q.few) return launch_prep(a, p);
    p.d = a.d;
    p.dp = q.dp;
    if (q.copy_h) {
        const long stride = (long)a.rows * q.dp;
        p.copy[0] = copy_job(a, q, a.h, q.h, a.rows, stride);
        *h = {p.copy[0].dst, q.dp, stride, a.rows, q.dp, q.parts};
    } else {
        *h = {a.h, a.d, 0, a.rows, a.d, 1};
    }
    *w = w_operand(a, q, 0, a.vocab < q.piece ? a.vocab : q.piece, &p.copy[1]);
    if (ht) {
        p.h = a.h;
        p.h_vec = load_width(a, a.h);
        p.ht = (__nv_bfloat16 *)((unsigned char *)a.ws + q.ht);
        // few rows: a line of memory for each column's, else every SM asks for the same few lines
        // (2 x 1024 x 131072 tokens, both directions: rows of 16 bytes 266 us, of 128 219 us)
        p.rp = up(q.dz_rows, q.dz_rows != a.rows ? 64 : 8);
        p.twice = q.dz_rows != a.rows;
        p.ht_stride = a.d * p.rp;
        p.t_cols = (a.d + 63) / 64;
        const long blocks = (long)((a.rows + 63) / 64) * p.t_cols;
        if (blocks > INT32_MAX) return cudaErrorNotSupported;
        p.t_blocks = (int)blocks;
        *ht = {p.ht, p.rp, p.ht_stride, a.d, q.dz_rows, q.parts};
    }
    return launch_prep(a, p);
}

// a later piece of the vocabulary
cudaError_t next_weights(const LossArgs &a, const LossPlan &q, long v0, int cols, LossMatrix *w)
{
    PrepArgs p;
    memset(&p, 0, sizeof(p));
    p.d = a.d;
    p.dp = q.dp;
    *w = w_operand(a, q, v0, cols, &p.copy[0]);
    return q.copy_w ? launch_prep(a, p) : cudaSuccess;
}

float square_of(const LossArgs &a) { return a.temp != 0.f ? a.temp * a.temp : 1.f; }

FewCall few_call(const LossArgs &a, const LossPlan &q, const LossRows &r, bool backward)
{
    unsigned char *ws = (unsigned char *)a.ws;
    FewCall f;
    f.h = a.h;
    f.w = a.w;
    f.bias = a.bias;
    f.r = r;
    f.rows = a.rows;
    f.d = a.d;
    f.vocab = a.vocab;
    f.s = q.shape;
    f.f32 = a.dtype == TXL_F32;
    f.backward = backward;
    f.alpha = alpha_of(a);
    f.ysel = (float *)(ws + q.ysel);
    f.part = (float2 *)(ws + q.part);
    f.t2 = square_of(a);
    f.loss = a.loss;
    f.lse_out = a.lse_out;
    f.dh = backward ? a.dh : nullptr;
    f.dw = backward ? a.dw : nullptr;
    f.db = backward ? a.db : nullptr;
    f.dh_part = (float *)(ws + q.dh_acc);
    return f;
}

cudaError_t run_fwd(const LossArgs &a, const LossPlan &q)
{
    unsigned char *ws = (unsigned char *)a.ws;
    const LossRows r = rows_at(a, q);
    const float *bias = bias_of(a, q);
    float2 *part = (float2 *)(ws + q.part);
    LossMatrix h, w;
    cudaError_t e = prepare(a, q, r, &h, &w, nullptr);
    if (e == cudaSuccess && q.few) e = launch_loss_few(few_call(a, q, r, false), a.s);
    long slot = 0;
    for (long v0 = 0; e == cudaSuccess && !q.few && v0 < a.vocab; v0 += q.piece) {
        const int cols = (int)(a.vocab - v0 < q.piece ? a.vocab - v0 : q.piece);
        const LossTiling t = cols == q.piece ? q.whole.vocab : q.last.vocab;
        if (v0 > 0) e = next_weights(a, q, v0, cols, &w);
        if (e == cudaSuccess)
            e = launch_loss_lse(h, w, bias ? bias + v0 : nullptr, (int)v0, alpha_of(a), r, (float *)(ws + q.ysel),
                                part + slot * a.rows, q.joined ? a.loss : nullptr, q.joined ? a.lse_out : nullptr, t, a.s);
        slot += kSlotsPerStrip * vocab_strips(t);
    }
    if (e != cudaSuccess || q.joined) return e;
    const int per = a.rows <= 2048 ? 8 : 32;
    return loss_launch(per == 8 ? loss_merge_kernel<8> : loss_merge_kernel<32>, (unsigned)((a.rows + per - 1) / per), 1024,
                       0, 1, a.s, (const float2 *)part, q.slots, (const float *)(ws + q.ysel), r, square_of(a), a.loss,
                       a.lse_out, a.rows);
}

LossOutput direct_out(const LossArgs &a, void *p)
{
    LossOutput o;
    o.base = p;
    o.pitch = a.d;
    o.slot_stride = 0;
    o.f32 = a.dtype == TXL_F32;
    o.add = false;
    o.tma = (size_t)a.d * (o.f32 ? 4 : 2) % 16 == 0 && al(p, 16);
    return o;
}

SumJob sum_job(const LossArgs &a, const float *slot, int slots, long stride, void *out, int rows)
{
    SumJob j;
    j.slot = slot;
    j.out = out;
    j.slots = slots;
    j.rows = rows;
    j.blocks = grid_of((long)rows * ((a.d + 3) / 4), 1024);
    j.stride = stride;
    return j;
}

LossOutput slot_out(float *p, long pitch, long stride, bool add)
{
    LossOutput o;
    o.base = p;
    o.pitch = pitch;
    o.slot_stride = stride;
    o.f32 = true;
    o.add = add;
    o.tma = true;
    return o;
}

cudaError_t run_bwd(const LossArgs &a, const LossPlan &q)
{
    unsigned char *ws = (unsigned char *)a.ws;
    const LossRows r = rows_at(a, q);
    const float *bias = bias_of(a, q);
    const size_t esz = a.dtype == TXL_F32 ? 4 : 2;
    const long h_stride = (long)q.dz_rows * q.dp;
    float *acc_h = (float *)(ws + q.dh_acc), *acc_w = (float *)(ws + q.dw_acc);
    LossMatrix h, ht, w;
    cudaError_t e = prepare(a, q, r, &h, &w, a.dw ? &ht : nullptr);
    if (q.few) return e == cudaSuccess ? launch_loss_few(few_call(a, q, r, true), a.s) : e;
    for (long v0 = 0; e == cudaSuccess && v0 < a.vocab; v0 += q.piece) {
        const int cols = (int)(a.vocab - v0 < q.piece ? a.vocab - v0 : q.piece);
        const bool last = v0 + cols == a.vocab;
        const LossPlan::Piece &t = cols == q.piece ? q.whole : q.last;
        const long pitch = up(cols, 64), w_stride = (long)cols * q.dp;
        // its parts one behind another; to the products two of them are one matrix
        const LossMatrix dz_out = {ws + q.dz, pitch, (long)a.rows * pitch, a.rows, cols, dz_parts(a.rows, q.parts)};
        const LossMatrix dz = {ws + q.dz, pitch, (long)a.rows * pitch, q.dz_rows, cols, q.parts};
        float *dbp = a.db ? (float *)(ws + q.dbpart) : nullptr;
        if (v0 > 0) e = next_weights(a, q, v0, cols, &w);
        if (e == cudaSuccess)
            e = launch_loss_dz(h, w, bias ? bias + v0 : nullptr, (int)v0, alpha_of(a), r, dz_out, dbp, t.vocab, a.s);
        if (e != cudaSuccess) return e;
        // both gradients of the piece in one launch, the longer items first
        LossContraction job[2];
        int n = 0;
        const bool h_direct = !q.dh_slots && t.dh.splits == 1;
        void *dw_out = a.dw ? (unsigned char *)a.dw + (size_t)v0 * a.d * esz : nullptr;
        const bool w_direct = t.dw.splits == 1;
        if (a.dh) {
            LossContraction &j = job[a.dw && t.dw.first ? 1 : 0];
            ++n;
            j.a = t.dh.turned ? w : dz;
            j.b = t.dh.turned ? dz : w;
            j.a_t = j.b_t = j.out_t = t.dh.turned;
            j.m = t.dh.turned ? a.d : q.dz_rows;
            j.n = t.dh.turned ? q.dz_rows : a.d;
            j.k = cols;
            j.out = h_direct ? direct_out(a, a.dh) : slot_out(acc_h, q.dp, h_stride, v0 > 0);
            j.t = t.dh;
        }
        if (a.dw) {
            LossContraction &j = job[a.dh && !t.dw.first ? 1 : 0];
            ++n;
            j.a = dz;
            j.b = ht;
            j.a_t = j.b_t = true;
            j.out_t = false;
            j.m = cols;
            j.n = a.d;
            j.k = q.dz_rows;
            j.out = w_direct ? direct_out(a, dw_out) : slot_out(acc_w, q.dp, w_stride, false);
            j.t = t.dw;
        }
        if (n) e = launch_loss_gradients(job, n, q.parts, a.s);
        if (e != cudaSuccess) return e;
        FinishArgs f;
        memset(&f, 0, sizeof(f));
        f.d = a.d;
        f.dp = q.dp;
        if (a.db) {
            f.dbpart = dbp;
            f.db = a.db + v0;
            f.parts = (int)(up(a.rows, 32) / 32);
            f.cols = cols;
            f.pitch = pitch;
            // as many threads per column as leave each some row groups, in one round of
            // blocks (192 row groups of 32768 columns: 8 threads 11 us, 32 in four rounds 24)
            const long round = 2048L * device_sm_count();
            for (f.db_lanes = 1; f.db_lanes < 32 && 4 * f.db_lanes < f.parts && 2L * f.db_lanes * cols <= round;)
                f.db_lanes <<= 1;
            f.db_blocks = (int)((cols + 1024 / f.db_lanes - 1) / (1024 / f.db_lanes));
        }
        if (a.dw && !w_direct) f.sum[0] = sum_job(a, acc_w, t.dw.splits, w_stride, dw_out, cols);
        if (a.dh && !h_direct && last)
            f.sum[1] = sum_job(a, acc_h, t.dh.splits * (q.dz_rows / a.rows), (long)a.rows * q.dp, a.dh, a.rows);
        const int blocks = f.db_blocks + f.sum[0].blocks + f.sum[1].blocks;
        if (blocks)
            e = loss_launch(a.dtype == TXL_F32 ? loss_finish_kernel<float> : loss_finish_kernel<__nv_bfloat16>,
                            (unsigned)blocks, 1024, 0, 1, a.s, f);
    }
    return e;
}

txl_status loss_fwd(const LossArgs &a)
{
    LossPlan q;
    const txl_status st = loss_checks(a, false, &q);
    if (st != TXL_OK || a.rows == 0) return st;
    const cudaError_t e = run_fwd(a, q);
    if (e == cudaSuccess) return TXL_OK;
    note_cuda_error(e);
    return TXL_ERR_CUDA;
}

txl_status loss_bwd(const LossArgs &a)
{
    LossPlan q;
    const txl_status st = loss_checks(a, true, &q);
    if (st != TXL_OK) return st;
    cudaError_t e = cudaSuccess;
    if (a.rows == 0) {   // sums over no rows
        if (a.dw) e = cudaMemsetAsync(a.dw, 0, (size_t)a.vocab * a.d * (a.dtype == TXL_F32 ? 4 : 2), a.s);
        if (e == cudaSuccess && a.db) e = cudaMemsetAsync(a.db, 0, (size_t)a.vocab * 4, a.s);
    } else if (a.dh || a.dw || a.db) {
        e = run_bwd(a, q);
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
    return loss_workspace(rows, d_model, vocab, 0, dtype, backward, bytes);
}

txl_status txl_distill_workspace(int rows, int d_model, int vocab, int top_k, txl_dtype dtype, int backward,
                                 size_t *bytes)
{
    if (top_k < 1) return TXL_ERR_INVALID;
    return loss_workspace(rows, d_model, vocab, top_k, dtype, backward, bytes);
}

txl_status txl_softmax_xent_fwd(const void *h, const void *w, const float *bias, const int64_t *target, int rows,
                                int d_model, int vocab, txl_dtype dtype, float *loss, float *lse, void *workspace,
                                size_t workspace_bytes, void *stream)
{
    return loss_fwd({h, w, bias, target, nullptr, TXL_F32, 0.f, rows, d_model, vocab, 0, dtype, loss, lse, nullptr,
                     nullptr, nullptr, nullptr, nullptr, workspace, workspace_bytes, (cudaStream_t)stream});
}

txl_status txl_softmax_xent_bwd(const void *h, const void *w, const float *bias, const int64_t *target,
                                const float *lse, const float *dloss, int rows, int d_model, int vocab,
                                txl_dtype dtype, void *dh, void *dw, float *dbias, void *workspace,
                                size_t workspace_bytes, void *stream)
{
    return loss_bwd({h, w, bias, target, nullptr, TXL_F32, 0.f, rows, d_model, vocab, 0, dtype, nullptr, nullptr, lse,
                     dloss, dh, dw, dbias, workspace, workspace_bytes, (cudaStream_t)stream});
}

txl_status txl_distill_fwd(const void *h, const void *w, const float *bias, const int64_t *teacher_idx,
                           const void *teacher_logits, txl_dtype teacher_dtype, float temperature, int rows,
                           int d_model, int vocab, int top_k, txl_dtype dtype, float *loss, float *lse,
                           void *workspace, size_t workspace_bytes, void *stream)
{
    if (!(temperature > 0.f) || top_k < 1) return TXL_ERR_INVALID;
    return loss_fwd({h, w, bias, teacher_idx, teacher_logits, teacher_dtype, temperature, rows, d_model, vocab, top_k,
                     dtype, loss, lse, nullptr, nullptr, nullptr, nullptr, nullptr, workspace, workspace_bytes,
                     (cudaStream_t)stream});
}

txl_status txl_distill_bwd(const void *h, const void *w, const float *bias, const int64_t *teacher_idx,
                           const void *teacher_logits, txl_dtype teacher_dtype, float temperature, const float *lse,
                           const float *dloss, int rows, int d_model, int vocab, int top_k, txl_dtype dtype,
                           void *dh, void *dw, float *dbias, void *workspace, size_t workspace_bytes, void *stream)
{
    if (!(temperature > 0.f) || top_k < 1) return TXL_ERR_INVALID;
    return loss_bwd({h, w, bias, teacher_idx, teacher_logits, teacher_dtype, temperature, rows, d_model, vocab, top_k,
                     dtype, nullptr, nullptr, lse, dloss, dh, dw, dbias, workspace, workspace_bytes,
                     (cudaStream_t)stream});
}

}  // extern "C"

// loss_few.cu -- the output-layer losses for a handful of rows on the CUDA
// cores: where the tensor-core kernel could only read the weights through a
// copy (fp32 operands, which it takes as three bf16 parts, and bf16 rows that
// the TMA unit cannot address), and small vocabularies.
//
// With few rows both directions are bound by moving the weights: every element
// takes 2 * rows operations per product, below what the CUDA cores do while
// HBM delivers it, and the copies would move each element four to six times.
// A block walks a range of the vocabulary in chunks of 16 to 64 tokens, which lie
// contiguous in memory whatever d_model: bulk copies bring them into a ring in
// shared memory, and all products of a chunk read it there.
//   logits    a warp takes two tokens, its lanes lie along d_model; h in shared
//             memory, fp32 products and sums;
//   forward   each thread keeps the maximum and sum of some of the chunk's
//             tokens for one row; loss_merge_kernel joins the blocks, or they
//             do it themselves as a cluster;
//   backward  dz of the chunk in shared memory (fp32, not rounded); then the
//             threads take columns of d_model: dW = dz^T h is written once,
//             dh += dz W stays in registers.  few_finish_kernel adds the
//             blocks' parts of dh in order.
// fp32, 2 rows x 1024 x 131072 tokens: forward 89 us (537 MB of weights at
// 6.0 TB/s), both directions 297 us (1.6 GB at 5.4 TB/s); tensor-core kernel
// 560 and 1404 us.  With 16 rows the multiply-adds bound it: 195 and 637 us
// (561 and 1376).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "internal.h"
#include "loss_products.h"
#include "sm100.cuh"

namespace txl {

using namespace sm100;

namespace {

__device__ unsigned int g_few_err;      // read by txl_check once a launch was made or captured
std::atomic<bool> g_few_ran{false};

constexpr int kThreads = 256;
constexpr int kMaxSlots = 8;
constexpr int kCluster = 8;                           // blocks that join their parts themselves
constexpr int kFewSmem = 220 * 1024;                  // dynamic shared memory at most
constexpr uint64_t kFewWaitNs = 2000000000ull;        // 2 s per wait, then give up

__device__ __forceinline__ float as_f(float x) { return x; }
__device__ __forceinline__ float as_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T of_f(float x);
template <>
__device__ __forceinline__ float of_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 of_f<__nv_bfloat16>(float x) { return __float2bfloat16(x); }

// kV elements from an address aligned to them
template <int kV, typename T>
__device__ __forceinline__ void load_v(const T *p, float (&v)[kV])
{
    struct alignas(sizeof(T) * kV) Pack {
        T e[kV];
    };
    const Pack x = *reinterpret_cast<const Pack *>(p);
#pragma unroll
    for (int i = 0; i < kV; ++i) v[i] = as_f(x.e[i]);
}
template <int kV, typename T>
__device__ __forceinline__ void store_v(T *p, const float (&v)[kV])
{
    struct alignas(sizeof(T) * kV) Pack {
        T e[kV];
    };
    Pack x;
#pragma unroll
    for (int i = 0; i < kV; ++i) x.e[i] = of_f<T>(v[i]);
    *reinterpret_cast<Pack *>(p) = x;
}

// Sums over the warp of kN <= 32 values: lane l ends up with the sum of value
// l * kN / 32, in kN - 1 shuffles (and one per further halving of the lanes).
template <int kN>
__device__ __forceinline__ float warp_sums(float (&v)[kN], int lane)
{
    int n = kN;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        if (n > 1) {
            n >>= 1;
            const bool up = lane & o;
#pragma unroll
            for (int x = 0; x < kN / 2; ++x) {
                if (x >= n) break;
                const float send = up ? v[x] : v[x + n], keep = up ? v[x + n] : v[x];
                v[x] = keep + __shfl_xor_sync(0xffffffffu, send, o);
            }
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
        }
    }
    return v[0];
}

struct FewParams {
    const void *h, *w;
    const float *bias;
    LossRows r;
    int rows, d, dp, vocab;         // dp: d rounded up to 4
    FewShape s;
    uint32_t slot_bytes;
    float alpha;
    float *ysel;                    // forward
    float2 *part;                   // [block][rows]
    float t2, *loss, *lse;          // of a joined shape
    void *dw;                       // backward
    bool dw_vec;                    // dw is aligned to kV elements
    float *db, *dh_part;            // dh_part: [block][group][rows][d]
};

// The row lists, followed along the vocabulary by thread `row` < rows; the
// next entry of either half stays in a register, so that chunks without one
// cost no load.
struct FewCursor {
    int at[2], next[2];
    __device__ __forceinline__ int peek(const LossRows &r, int row, int half) const
    {
        return at[half] < (half ? r.K : r.even[row]) ? r.col[(long)row * r.K + at[half]] : kNoColumn;
    }
    __device__ __forceinline__ void seek(const LossRows &r, int row, int from)
    {
        at[0] = at[1] = 0;
        next[1] = kNoColumn;
        if (r.target) {
            next[0] = target_column(r, row);
            return;
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            int lo = half ? r.even[row] : 0, hi = half ? r.K : r.even[row];
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (r.col[(long)row * r.K + mid] < from)
                    lo = mid + 1;
                else
                    hi = mid;
            }
            at[half] = lo;
            next[half] = peek(r, row, half);
        }
    }
    // f(entry, token of the chunk) for the row's entries in tokens n0 .. n1 - 1
    // (of one half: chunks do not cross multiples of 64)
    template <typename F>
    __device__ __forceinline__ void chunk(const LossRows &r, int row, int n0, int n1, F f)
    {
        if (r.target) {
            if (next[0] >= n0 && next[0] < n1) f((long)row, next[0] - n0);
            return;
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            if (half != ((n0 >> 6) & 1)) continue;
            while (next[half] < n1) {
                f((long)row * r.K + at[half], next[half] - n0);
                ++at[half];
                next[half] = peek(r, row, half);
            }
        }
    }
};

// The block's tokens b0 .. b1 - 1 of W, chunk by chunk through the ring.
template <typename T>
struct FewRing {
    const FewParams &p;
    unsigned char *slots;
    uint32_t bars;
    int b0, b1, chunks;

    __device__ __forceinline__ void issue(int i) const      // one thread
    {
        const int n0 = b0 + i * p.s.tok, count = b1 - n0 < p.s.tok ? b1 - n0 : p.s.tok, slot = i % p.s.slots;
        const unsigned char *src = static_cast<const unsigned char *>(p.w) + (long)n0 * p.d * sizeof(T);
        unsigned char *dst = slots + slot * p.slot_bytes;
        // a chunk starts on a 16-byte boundary (its first token is a multiple
        // of 16); what the last one has behind its last boundary is copied here
        const uint32_t bytes = count * p.d * sizeof(T), bulk = bytes & ~15u;
        for (uint32_t x = bulk; x < bytes; x += sizeof(T))
            *reinterpret_cast<T *>(dst + x) = *reinterpret_cast<const T *>(src + x);
        mbar_arrive_expect_tx(bars + 8 * slot, bulk);
        if (bulk) bulk_load(smem_u32(dst), src, bulk, bars + 8 * slot);
    }
    __device__ __forceinline__ void start() const           // one thread
    {
        for (int i = 0; i < p.s.slots && i < chunks; ++i) issue(i);
    }
    // chunk i is in the ring, its predecessor's slot is refilled; false: gave up
    __device__ __forceinline__ bool next(int i) const
    {
        const bool ok = mbar_wait(bars + 8 * (i % p.s.slots), (i / p.s.slots) & 1, kFewWaitNs);
        if (__syncthreads_or(!ok)) {
            if (threadIdx.x == 0) {
                atomicOr(&g_few_err, 1u);
                // the block's memory stays until its copies are through
                for (int x = i; x < chunks && x < i + p.s.slots - (i > 0); ++x)
                    mbar_wait(bars + 8 * (x % p.s.slots), (x / p.s.slots) & 1, kFewWaitNs);
            }
            return false;
        }
        if (threadIdx.x == 0 && i > 0 && i - 1 + p.s.slots < chunks) issue(i - 1 + p.s.slots);
        return true;
    }
    __device__ __forceinline__ const T *chunk(int i) const
    {
        return reinterpret_cast<const T *>(slots + (i % p.s.slots) * p.slot_bytes);
    }
};

// h as fp32 in shared memory (rows of factor 0 as zeros with `coef`)
template <typename T, int kR>
__device__ __forceinline__ void few_load_h(const FewParams &p, float *hs, const float *coef)
{
    for (int x = threadIdx.x; x < kR * p.dp; x += kThreads) {
        const int r = x / p.dp, c = x - r * p.dp;
        float v = 0.f;
        if (r < p.rows && c < p.d && (!coef || coef[r] != 0.f)) v = as_f(static_cast<const T *>(p.h)[(long)r * p.d + c]);
        hs[x] = v;
    }
}

// zs[token][row] = f(y, row) of a chunk, y = alpha (h . w + bias), which is
// -infinity past the block's tokens
template <typename T, int kV, int kR, typename F>
__device__ __forceinline__ void few_logits(const FewParams &p, const T *w, const float *hs, float *zs, int n0, int n1, F f)
{
    constexpr int kN = 2 * kR;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int mine = lane * kN / 32, jm = mine / kR, rm = mine % kR;
    for (int g = warp * 2; g < p.s.tok; g += kThreads / 16) {
        const int n = n0 + g + jm;
        const float bias = p.bias && n < n1 ? p.bias[n] : 0.f;
        float acc[kN];
#pragma unroll
        for (int x = 0; x < kN; ++x) acc[x] = 0.f;
        const T *w0 = w + g * p.d, *w1 = w0 + p.d;
#pragma unroll 2
        for (int c = lane * kV; c < p.d; c += 32 * kV) {
            float a[kV], b[kV];
            load_v<kV>(w0 + c, a);
            load_v<kV>(w1 + c, b);
#pragma unroll
            for (int r = 0; r < kR; ++r) {
                float x[kV];
                load_v<kV>(hs + r * p.dp + c, x);
#pragma unroll
                for (int i = 0; i < kV; ++i) {
                    acc[r] = fmaf(a[i], x[i], acc[r]);
                    acc[kR + r] = fmaf(b[i], x[i], acc[kR + r]);
                }
            }
        }
        const float z = warp_sums(acc, lane);
        zs[(g + jm) * kR + rm] = f(n < n1 ? (z + bias) * p.alpha : -INFINITY);
    }
}

template <int kR>
struct FewMemory {
    float *hs, *zs;
    unsigned char *slots;
    uint32_t bars;
    __device__ __forceinline__ FewMemory(const FewParams &p, unsigned char *sm)
    {
        slots = sm;
        hs = reinterpret_cast<float *>(sm + p.s.slots * p.slot_bytes);
        zs = hs + kR * p.dp;
        bars = smem_u32(zs + 64 * kR);
        if (threadIdx.x == 0) {
            for (int x = 0; x < p.s.slots; ++x) mbar_init(bars + 8 * x, 1);
            fence_mbar_init();
        }
    }
};

template <typename T, int kV, int kR>
__global__ void __launch_bounds__(kThreads) few_lse_kernel(const __grid_constant__ FewParams p)
{
    extern __shared__ __align__(128) unsigned char few_sm[];
    __shared__ float2 state[kThreads];
    const FewMemory<kR> sm(p, few_sm);
    const int tid = threadIdx.x;
    const int b0 = blockIdx.x * p.s.per, b1 = p.vocab - b0 < p.s.per ? p.vocab : b0 + p.s.per;
    const FewRing<T> ring = {p, sm.slots, sm.bars, b0, b1, (b1 - b0 + p.s.tok - 1) / p.s.tok};
    loss_kernel_begin();
    loss_kernel_wait();
    if (tid == 0) ring.start();
    FewCursor cur;
    if (tid < p.rows) cur.seek(p.r, tid, b0);
    few_load_h<T, kR>(p, sm.hs, nullptr);
    float m = -INFINITY, l = 0.f;     // of row tid % kR
    __syncthreads();
    for (int i = 0; i < ring.chunks; ++i) {
        const int n0 = b0 + i * p.s.tok, n1 = b1 - n0 < p.s.tok ? b1 : n0 + p.s.tok;
        if (!ring.next(i)) return;
        few_logits<T, kV, kR>(p, ring.chunk(i), sm.hs, sm.zs, n0, n1, [](float y) { return y; });
        __syncthreads();
        if (tid < p.rows)
            cur.chunk(p.r, tid, n0, n1, [&](long at, int c) { p.ysel[at] = sm.zs[c * kR + tid]; });
        for (int x = tid; x < p.s.tok * kR; x += kThreads) {
            const float y = sm.zs[x], mm = fmaxf(m, y), ref = mm == -INFINITY ? 0.f : mm;
            l = l * exp2f(m - ref) + exp2f(y - ref);
            m = mm;
        }
    }
    state[tid] = make_float2(m, l);
    __syncthreads();
    auto join = [&](float2 e) {
        const float mm = fmaxf(m, e.x), ref = mm == -INFINITY ? 0.f : mm;
        l = l * exp2f(m - ref) + e.y * exp2f(e.x - ref);
        m = mm;
    };
    if (tid < p.rows) {
        for (int x = tid + kR; x < kThreads; x += kR) join(state[x]);
        p.part[(long)blockIdx.x * p.rows + tid] = make_float2(m, l);
    }
    if (!p.s.joined) return;
    // the cluster's first block takes what the others have left
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
    if (blockIdx.x) return;
    for (int row = tid >> 5; row < p.rows; row += kThreads / 32) {
        m = -INFINITY;
        l = 0.f;
        for (int x = 0; x < p.s.blocks; ++x) join(__ldcg(p.part + (long)x * p.rows + row));
        row_loss(p.r, p.ysel, m == -INFINITY ? 0.f : m, l, p.t2, row, tid & 31, p.loss, p.lse);
    }
}

template <typename T, int kV, int kR>
__global__ void __launch_bounds__(kThreads) few_bwd_kernel(const __grid_constant__ FewParams p)
{
    extern __shared__ __align__(128) unsigned char few_sm[];
    __shared__ float coef[kR], l2[kR];
    constexpr int kC = kFewColumns / kThreads;          // columns per thread, in accesses of kV
    const FewMemory<kR> sm(p, few_sm);
    const int tid = threadIdx.x;
    const int b0 = blockIdx.x * p.s.per, b1 = p.vocab - b0 < p.s.per ? p.vocab : b0 + p.s.per;
    const FewRing<T> ring = {p, sm.slots, sm.bars, b0, b1, (b1 - b0 + p.s.tok - 1) / p.s.tok};
    loss_kernel_begin();
    loss_kernel_wait();
    if (tid == 0) ring.start();
    if (tid < kR) {
        float c = 0.f, l = 0.f;
        if (tid < p.rows) {
            const bool any = (p.r.target ? target_column(p.r, tid) : p.r.col[(long)tid * p.r.K]) != kNoColumn;
            c = row_factor(p.r, tid, any);
            l = p.r.lse[tid] * (1.f / kLn2);
        }
        coef[tid] = c;
        l2[tid] = l;
    }
    FewCursor cur;
    if (tid < p.rows) cur.seek(p.r, tid, b0);
    __syncthreads();
    few_load_h<T, kR>(p, sm.hs, coef);
    // the row whose logits this lane gets from few_logits
    const int rl = ((tid & 31) * 2 * kR / 32) % kR;
    const float c_mine = coef[rl], l_mine = l2[rl];
    __syncthreads();
    // narrow rows leave room for groups of threads that take the tokens in turn
    // (fp32 8 x 64 x 65000, both directions: one group 106 us, 16 groups 58 us)
    float hr[kR][kC], dh[kR][kC];
    int col[kC];
    const int group = tid / (kThreads / p.s.groups), tx = tid % (kThreads / p.s.groups);
#pragma unroll
    for (int i = 0; i < kC; ++i) {
        col[i] = (i / kV * (kThreads / p.s.groups) + tx) * kV + i % kV;
#pragma unroll
        for (int r = 0; r < kR; ++r) {
            hr[r][i] = col[i] < p.d ? sm.hs[r * p.dp + col[i]] : 0.f;
            dh[r][i] = 0.f;
        }
    }
    for (int c = 0; c < ring.chunks; ++c) {
        const int n0 = b0 + c * p.s.tok, n1 = b1 - n0 < p.s.tok ? b1 : n0 + p.s.tok;
        if (!ring.next(c)) return;
        const T *w = ring.chunk(c);
        few_logits<T, kV, kR>(p, w, sm.hs, sm.zs, n0, n1,
                              [&](float y) { return c_mine != 0.f ? c_mine * exp2f(y - l_mine) : 0.f; });
        __syncthreads();
        if (tid < p.rows && coef[tid] != 0.f)
            cur.chunk(p.r, tid, n0, n1, [&](long at, int j) {
                sm.zs[j * kR + tid] -= coef[tid] * (p.r.target ? 1.f : p.r.p[at]);
            });
        __syncthreads();
        if (p.db && tid < n1 - n0) {
            float s = 0.f;
#pragma unroll
            for (int r = 0; r < kR; ++r) s += sm.zs[tid * kR + r];
            p.db[n0 + tid] = s;
        }
#pragma unroll 2
        for (int j = group; j < n1 - n0; j += p.s.groups) {
            float z[kR];
#pragma unroll
            for (int r = 0; r < kR; r += 2) {
                const float2 t = *reinterpret_cast<const float2 *>(sm.zs + j * kR + r);
                z[r] = t.x;
                z[r + 1] = t.y;
            }
#pragma unroll
            for (int i0 = 0; i0 < kC; i0 += kV) {
                if (col[i0] >= p.d) continue;
                if (p.dw) {
                    float o[kV];
#pragma unroll
                    for (int i = 0; i < kV; ++i) {
                        o[i] = 0.f;
#pragma unroll
                        for (int r = 0; r < kR; ++r) o[i] = fmaf(z[r], hr[r][i0 + i], o[i]);
                    }
                    T *to = static_cast<T *>(p.dw) + (long)(n0 + j) * p.d + col[i0];
                    if (p.dw_vec)
                        store_v<kV>(to, o);
                    else
#pragma unroll
                        for (int i = 0; i < kV; ++i) to[i] = of_f<T>(o[i]);
                }
                if (p.dh_part) {
                    float v[kV];
                    load_v<kV>(w + j * p.d + col[i0], v);
#pragma unroll
                    for (int i = 0; i < kV; ++i)
#pragma unroll
                        for (int r = 0; r < kR; ++r) dh[r][i0 + i] = fmaf(z[r], v[i], dh[r][i0 + i]);
                }
            }
        }
    }
    if (p.dh_part)
#pragma unroll
        for (int r = 0; r < kR; ++r)
#pragma unroll
            for (int i = 0; i < kC; ++i)
                if (r < p.rows && col[i] < p.d)
                    p.dh_part[(((long)blockIdx.x * p.s.groups + group) * p.rows + r) * p.d + col[i]] = dh[r][i];
}

// dh = the blocks' parts, added in order: 32 elements per block, 32 threads each.
// Hardly more than its launch: 2 x 1024 of 152 blocks (1.2 MB) in 4 us.
template <typename T>
__global__ void __launch_bounds__(1024)
few_finish_kernel(const float *part, int parts, int n, T *dh)
{
    __shared__ float s[32][33];
    loss_kernel_begin();
    loss_kernel_wait();
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, x = blockIdx.x * 32 + tx;
    float sum = 0.f;
    if (x < n)
        for (int b = ty; b < parts; b += 32) sum += part[(long)b * n + x];
    s[ty][tx] = sum;
    __syncthreads();
    if (ty || x >= n) return;
    float all = 0.f;
    for (int y = 0; y < 32; ++y) all += s[y][tx];
    dh[x] = of_f<T>(all);
}

// rows a kernel is built for: they are kept in registers
int few_height(int rows) { return rows <= 2 ? 2 : rows <= 8 ? 8 : 16; }

uint32_t slot_bytes(int tok, int d, bool f32) { return (uint32_t)(tok * d * (f32 ? 4 : 2) + 127) / 128 * 128; }
uint32_t fixed_bytes(int rows, int d)
{
    return (uint32_t)few_height(rows) * ((d + 3) / 4 * 4 + 64) * 4 + kMaxSlots * 8;
}

template <typename K>
cudaError_t few_start(K kern, const FewParams &p, size_t smem, std::atomic<uint64_t> &done, cudaStream_t s)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(done.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kFewSmem);
        if (e != cudaSuccess) return e;
        done.fetch_or(bit, std::memory_order_relaxed);
    }
    g_few_ran.store(true, std::memory_order_relaxed);
    return loss_launch(kern, (unsigned)p.s.blocks, kThreads, smem, p.s.joined ? (unsigned)p.s.blocks : 1, s, p);
}

template <typename T, int kV, int kR>
cudaError_t few_launch(bool backward, const FewParams &p, size_t smem, cudaStream_t s)
{
    static std::atomic<uint64_t> done_f{0}, done_b{0};
    return backward ? few_start(few_bwd_kernel<T, kV, kR>, p, smem, done_b, s)
                    : few_start(few_lse_kernel<T, kV, kR>, p, smem, done_f, s);
}

template <typename T, int kV>
cudaError_t few_rows_of(bool backward, const FewParams &p, size_t smem, cudaStream_t s)
{
    if (p.rows <= 2) return few_launch<T, kV, 2>(backward, p, smem, s);
    if constexpr (sizeof(T) == 4)
        if (p.rows > 8) return few_launch<T, kV, 16>(backward, p, smem, s);
    return few_launch<T, kV, 8>(backward, p, smem, s);
}

}  // namespace

bool few_shape(int rows, int d, int vocab, bool f32, bool w_ok, bool backward, FewShape *s)
{
    // Both directions, this kernel / the tensor-core kernel: fp32 16 x 768 x
    // 90326 406 / 677 us, 2 x 512 x 204 21 / 50 us; bf16 8 x 769 x 90326 377 /
    // 475 us, 8 x 410 x 20011 67 / 75 us.  bf16 rows that the tensor-core kernel
    // reads in place are this one's while launches are most of the time (two
    // less): 8 x 512 x 3000 28 / 34 us, 8 x 512 x 8000 37 / 44, but 8 x 64 x 40000
    // 56 / 48 and 8 x 768 x 90326 342 / 137.
    // w has to be aligned for the bulk copies, h and dh stay in registers.
    const bool in_place = !f32 && d % 8 == 0, small = vocab <= (16 << 10) && (int64_t)vocab * d <= (4 << 20);
    if (!w_ok || d > kFewColumns || rows > (f32 ? 16 : 8) || (in_place && !small)) return false;
    const uint32_t room = kFewSmem - fixed_bytes(rows, d);
    s->tok = 64;
    // a cluster covers a vocabulary that eight blocks are soon through: no launch to
    // join the blocks then (from Python: bf16 1 x 512 x 256 11.4 -> 9.3 us, 8 x 512 x
    // 256 11.0 -> 9.2; larger ones want more SMs: 8 x 1024 x 500 11.0 -> 14.8)
    s->joined = !backward && vocab <= 64 * kCluster && (int64_t)vocab * d * few_height(rows) <= (1 << 20);
    if (s->joined) {
        s->per = ((vocab + kCluster - 1) / kCluster + 15) / 16 * 16;
        while (s->per % s->tok || 2 * slot_bytes(s->tok, d, f32) > room) s->tok >>= 1;
        s->slots = (int)(room / slot_bytes(s->tok, d, f32));
        s->slots = s->slots < kMaxSlots ? s->slots : kMaxSlots;
        s->blocks = (vocab + s->per - 1) / s->per;
        s->groups = 1;
        return true;
    }
    // chunks as large as leave a ring of three, and a ring as deep as fits
    while (s->tok > 16 && 3 * slot_bytes(s->tok, d, f32) > room) s->tok >>= 1;
    // ... and no larger than gives every SM some
    const long sms = device_sm_count();
    while (s->tok > 16 && (long)s->tok * sms > vocab) s->tok >>= 1;
    const uint32_t slots = room / slot_bytes(s->tok, d, f32);
    s->slots = slots < (uint32_t)kMaxSlots ? (int)slots : kMaxSlots;
    const long chunks = ((long)vocab + s->tok - 1) / s->tok, each = (chunks + sms - 1) / sms;
    s->per = (int)each * s->tok;
    s->blocks = (int)((chunks + each - 1) / each);
    s->groups = 1;
    while (s->groups < 16 && 2 * s->groups * d <= kFewColumns) s->groups <<= 1;
    return true;
}

cudaError_t launch_loss_few(const FewCall &a, cudaStream_t s)
{
    FewParams p;
    p.h = a.h;
    p.w = a.w;
    p.bias = a.bias;
    p.r = a.r;
    p.rows = a.rows;
    p.d = a.d;
    p.dp = (a.d + 3) / 4 * 4;
    p.vocab = a.vocab;
    p.s = a.s;
    p.slot_bytes = slot_bytes(a.s.tok, a.d, a.f32);
    p.alpha = a.alpha;
    p.ysel = a.ysel;
    p.part = a.part;
    p.t2 = a.t2;
    p.loss = a.loss;
    p.lse = a.lse_out;
    p.dw = a.dw;
    p.db = a.db;
    p.dh_part = a.dh ? a.dh_part : nullptr;
    const size_t smem = (size_t)a.s.slots * p.slot_bytes + fixed_bytes(a.rows, a.d);
    // elements per access: as many as rows are aligned to (the sums' order and
    // with it the results depend on the sizes alone)
    const int esz = a.f32 ? 4 : 2, v = a.f32 ? (a.d % 4 == 0 ? 4 : a.d % 2 == 0 ? 2 : 1) : (a.d % 2 == 0 ? 2 : 1);
    p.dw_vec = (uintptr_t)a.dw % (v * esz) == 0;
    cudaError_t e;
    if (a.f32)
        e = v == 4   ? few_rows_of<float, 4>(a.backward, p, smem, s)
            : v == 2 ? few_rows_of<float, 2>(a.backward, p, smem, s)
                     : few_rows_of<float, 1>(a.backward, p, smem, s);
    else
        e = v == 2 ? few_rows_of<__nv_bfloat16, 2>(a.backward, p, smem, s)
                   : few_rows_of<__nv_bfloat16, 1>(a.backward, p, smem, s);
    if (e != cudaSuccess || !a.backward || !a.dh) return e;
    const int n = a.rows * a.d;
    const unsigned blocks = (unsigned)(n + 31) / 32;
    const float *part = a.dh_part;
    const int parts = a.s.blocks * a.s.groups;
    return a.f32 ? loss_launch(few_finish_kernel<float>, blocks, 1024, 0, 1, s, part, parts, n, (float *)a.dh)
                 : loss_launch(few_finish_kernel<__nv_bfloat16>, blocks, 1024, 0, 1, s, part, parts, n,
                               (__nv_bfloat16 *)a.dh);
}

cudaError_t read_and_clear_few_error(unsigned int *word, cudaStream_t s)
{
    if (!g_few_ran.load(std::memory_order_relaxed)) return cudaSuccess;
    return read_and_clear_word(g_few_err, word, s);
}

}  // namespace txl

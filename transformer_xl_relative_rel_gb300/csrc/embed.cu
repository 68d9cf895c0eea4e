// embed.cu -- the token embedding and its table's gradient.
//
//     out_i = scale table[tok_i]                          (0 for a token outside the vocabulary)
//     dtable_t (+)= scale sum_{i: tok_i = t} dout_i
//
// The gradient sums rows by token in a fixed order, so that the same call
// gives the same bits: tokens are sorted by a stable radix sort (digits of up
// to kDigitBits bits, a counting and a placing launch per digit), the sorted
// rows are cut into chunks of kChunk, and a warp adds up a chunk's columns,
// writing each token's sum as its last row passes.  A token whose rows lie in
// several chunks leaves a partial sum in each, which a last launch adds.
#include <cuda_runtime.h>
#include <stdint.h>

#include "buffers.h"
#include "chain.h"
#include "internal.h"
#include "rows.cuh"

namespace txl {
namespace {

constexpr int kMaxSize = 1 << 30;                  // rows and vocabulary
constexpr int kMaxWidth = 1 << 24;                 // d_model
constexpr int64_t kMaxElements = (int64_t)1 << 40; // of the table and of the rows
constexpr int NT = 256;
constexpr int kChunk = 32;                         // sorted rows a warp adds up
constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kDigitBits = 9;                      // a placing block's counters: 32 warps x 512 digits, 64 KB

// ---------------------------------------------------------------- forward
struct EmbedArgs {
    const int64_t *tokens;
    const void *table;
    void *out;
    float scale;
    long rows, vectors;      // vectors of V elements per row
    int d, vocab;
};

template <typename T, int V>
__global__ void __launch_bounds__(NT) embed_fwd_kernel(const __grid_constant__ EmbedArgs a)
{
    chain_begin();
    chain_wait();
    const long total = a.rows * a.vectors, stride = (long)gridDim.x * NT;
    for (long x = (long)blockIdx.x * NT + threadIdx.x; x < total; x += stride) {
        const long row = x / a.vectors;
        const int c = (int)(x - row * a.vectors) * V;
        const int64_t t = a.tokens[row];
        float v[V];
        if (t >= 0 && t < a.vocab) {
            unpack<T, V>(load_raw<T, V>((const T *)a.table + t * a.d + c), v);
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] *= a.scale;
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = 0.f;
        }
        store_vec<T, V>((T *)a.out + row * a.d + c, v);
    }
}

// ---------------------------------------------------------------- sorting
// One digit of the sort.  Keys are tokens; one outside the vocabulary gets the
// key `vocab`, behind all others.  Blocks take consecutive tiles of rows, a
// block's warps consecutive parts of its tile, so that ranks in that order
// keep equal keys in the order of their rows.
struct SortPass {
    const int64_t *tokens;           // the first pass reads these
    const int *key_in, *row_in;      // the others these
    int *key_out, *row_out;
    int *count;                      // [blocks][1 << bits]
    int n, vocab, tile, blocks, shift, bits;
};

struct ZeroJob {
    unsigned char *p;
    size_t bytes;
};

__device__ __forceinline__ int sort_key(const SortPass &a, int i)
{
    if (!a.tokens) return a.key_in[i];
    const int64_t t = a.tokens[i];
    return t >= 0 && t < a.vocab ? (int)t : a.vocab;
}

// the digit of row i, one past the digits for a lane behind the end
__device__ __forceinline__ int sort_digit(const SortPass &a, int key, bool in)
{
    return in ? (key >> a.shift) & ((1 << a.bits) - 1) : 1 << a.bits;
}

// counts the tile's digits; blocks behind the tiles set the table to zero
__global__ void __launch_bounds__(kSortThreads)
sort_count_kernel(const __grid_constant__ SortPass a, const __grid_constant__ ZeroJob z)
{
    chain_begin();
    __shared__ int count[1 << kDigitBits];
    const int digits = 1 << a.bits;
    for (int d = threadIdx.x; d < digits; d += kSortThreads) count[d] = 0;
    chain_wait();
    if ((int)blockIdx.x >= a.blocks) {
        const long stride = (long)(gridDim.x - a.blocks) * kSortThreads;
        const long first = (long)(blockIdx.x - a.blocks) * kSortThreads + threadIdx.x;
        const size_t head = z.bytes < (-(uintptr_t)z.p & 15) ? z.bytes : (-(uintptr_t)z.p & 15);
        const size_t n16 = (z.bytes - head) / 16, tail = z.bytes - head - 16 * n16;
        uint4 *v = (uint4 *)(z.p + head);
        for (long i = first; i < (long)n16; i += stride) v[i] = make_uint4(0, 0, 0, 0);
        if (first < (long)(head / 2)) ((uint16_t *)z.p)[first] = 0;
        if (first < (long)(tail / 2)) ((uint16_t *)(z.p + z.bytes - tail))[first] = 0;
        return;
    }
    __syncthreads();
    const int lane = threadIdx.x & 31, first = blockIdx.x * a.tile;
    const int end = min(first + a.tile, a.n);
    for (int i = first + (int)threadIdx.x; i - lane < end; i += kSortThreads) {
        const bool in = i < end;
        const int d = sort_digit(a, in ? sort_key(a, i) : 0, in);
        const unsigned same = __match_any_sync(0xffffffffu, d);
        if (in && (same & ((1u << lane) - 1)) == 0) atomicAdd(&count[d], __popc(same));
    }
    __syncthreads();
    for (int d = threadIdx.x; d < digits; d += kSortThreads) a.count[(size_t)blockIdx.x * digits + d] = count[d];
}

// places the tile's rows
__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(const __grid_constant__ SortPass a)
{
    chain_begin();
    extern __shared__ int smem[];
    const int digits = 1 << a.bits, t = threadIdx.x, lane = t & 31, w = t >> 5;
    int *mine = smem + w * digits;                    // this warp's counts, then its next places
    int *sums = smem + kSortWarps * digits;           // [kSortWarps]
    for (int d = t; d < kSortWarps * digits; d += kSortThreads) smem[d] = 0;
    __syncthreads();
    chain_wait();
    const int per = a.tile / kSortWarps, tile_end = min((int)(blockIdx.x + 1) * a.tile, a.n);
    const int first = blockIdx.x * a.tile + w * per, end = min(first + per, tile_end);
    for (int i = first + lane; i - lane < end; i += 32) {
        const bool in = i < end;
        const int d = sort_digit(a, in ? sort_key(a, i) : 0, in);
        const unsigned same = __match_any_sync(0xffffffffu, d);
        if (in && (same & ((1u << lane) - 1)) == 0) mine[d] += __popc(same);
        __syncwarp();
    }
    // a digit's rows in all blocks, and those in the blocks before this one
    int total = 0, before = 0;
    if (t < digits)
        for (int b = 0; b < a.blocks; ++b) {
            const int c = a.count[(size_t)b * digits + t];
            if (b < (int)blockIdx.x) before += c;
            total += c;
        }
    // sums over the digits below
    int run = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += v;
    }
    if (lane == 31) sums[w] = run;
    __syncthreads();
    int place = run - total + before;
    for (int x = 0; x < w; ++x) place += sums[x];
    if (t < digits)
        for (int x = 0; x < kSortWarps; ++x) {
            const int c = smem[x * digits + t];
            smem[x * digits + t] = place;
            place += c;
        }
    __syncthreads();
    for (int i = first + lane; i - lane < end; i += 32) {
        const bool in = i < end;
        const int key = in ? sort_key(a, i) : 0;
        const int d = sort_digit(a, key, in);
        const unsigned same = __match_any_sync(0xffffffffu, d), below = same & ((1u << lane) - 1);
        if (in) {
            const int to = mine[d] + __popc(below);
            a.key_out[to] = key;
            a.row_out[to] = a.tokens ? i : a.row_in[i];
        }
        __syncwarp();
        if (in && below == 0) mine[d] += __popc(same);
        __syncwarp();
    }
}

// ---------------------------------------------------------------- sums
struct SumArgs {
    const int *key, *row;    // sorted by token
    const void *dout;
    void *dtable;
    float *part;             // [chunks][2][pitch]: sums of a token that begins before the chunk (0), of one
                             // that begins in it and goes on behind it (1)
    float scale;
    int n, d, vocab, chunks, strips, accumulate;
    long pitch;
};

template <typename T, int V>
__device__ __forceinline__ void write_sum(const SumArgs &a, int token, int c, float (&acc)[V])
{
    T *to = (T *)a.dtable + (size_t)token * a.d + c;
    float old[V];
    if (a.accumulate) unpack<T, V>(load_raw<T, V>(to), old);
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = a.accumulate ? fmaf(a.scale, acc[i], old[i]) : a.scale * acc[i];
    store_vec<T, V>(to, acc);
}

template <typename T, int V>
__global__ void __launch_bounds__(NT) embed_sum_kernel(const __grid_constant__ SumArgs a)
{
    chain_begin();
    chain_wait();
    const int lane = threadIdx.x & 31;
    const long task = (long)blockIdx.x * (NT / 32) + (threadIdx.x >> 5);
    const int chunk = (int)(task / a.strips), c = (int)(task - (long)chunk * a.strips) * 32 * V + lane * V;
    if (chunk >= a.chunks) return;
    const int first = chunk * kChunk, n = min(kChunk, a.n - first);
    const int key = lane < n ? a.key[first + lane] : a.vocab;
    const int row = lane < n ? a.row[first + lane] : 0;
    const int before = first > 0 ? a.key[first - 1] : -1, after = first + n < a.n ? a.key[first + n] : a.vocab;
    const int live = __popc(__ballot_sync(0xffffffffu, key < a.vocab));
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    constexpr int U = 8;     // rows asked for at once
    for (int j = 0; j < live; j += U) {
        raw_t<T, V> raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long r = __shfl_sync(0xffffffffu, row, (j + u) & 31);
            if (j + u < live && c < a.d) raw[u] = load_raw<T, V>((const T *)a.dout + r * a.d + c);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (j + u >= live) break;
            const int k = __shfl_sync(0xffffffffu, key, j + u);
            const int next = __shfl_sync(0xffffffffu, key, (j + u + 1) & 31);
            float v[V];
            if (c < a.d) {
                unpack<T, V>(raw[u], v);
#pragma unroll
                for (int i = 0; i < V; ++i) acc[i] += v[i];
            }
            const bool end = j + u + 1 == n;
            if (!end && next == k) continue;
            // the token's last row in this chunk
            const int head = __shfl_sync(0xffffffffu, key, 0);
            const bool from_before = k == head && before == k, goes_on = end && after == k;
            if (c < a.d) {
                if (from_before || goes_on)
                    store_floats<V>(a.part + (2 * (size_t)chunk + !from_before) * a.pitch + c, acc);
                else
                    write_sum<T, V>(a, k, c, acc);
            }
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = 0.f;
        }
    }
}

// Adds the partial sums of a token that begins in this block's chunk and goes
// on behind it: 8 threads per column take every eighth chunk.
constexpr int kJoinColumns = 32, kJoinLanes = NT / kJoinColumns;

template <typename T>
__global__ void __launch_bounds__(NT) embed_join_kernel(const __grid_constant__ SumArgs a)
{
    chain_begin();
    chain_wait();
    const int strips = (a.d + kJoinColumns - 1) / kJoinColumns;
    const int chunk = blockIdx.x / strips, last = chunk * kChunk + kChunk - 1;
    if (last + 1 >= a.n) return;
    const int key = a.key[last];
    if (key >= a.vocab || a.key[last + 1] != key) return;
    const int first = chunk * kChunk;
    if (first > 0 && a.key[first] == key && a.key[first - 1] == key) return;   // begins before
    int lo = last + 1, hi = a.n;              // the first sorted row behind the token's
    while (lo < hi) {
        const int mid = lo + (hi - lo) / 2;
        if (a.key[mid] > key) hi = mid;
        else lo = mid + 1;
    }
    const int end = (lo - 1) / kChunk;        // the last chunk with rows of it
    const int x = threadIdx.x % kJoinColumns, y = threadIdx.x / kJoinColumns;
    const int c = (int)(blockIdx.x % strips) * kJoinColumns + x;
    float acc = 0.f;
    if (c < a.d)
        for (int k = chunk + y; k <= end; k += kJoinLanes)
            acc += a.part[(2 * (size_t)k + (k == chunk)) * a.pitch + c];
    __shared__ float sums[kJoinLanes][kJoinColumns];
    sums[y][x] = acc;
    __syncthreads();
    if (y == 0 && c < a.d) {
        float total[1] = {0.f};
#pragma unroll
        for (int k = 0; k < kJoinLanes; ++k) total[0] += sums[k][x];
        write_sum<T, 1>(a, key, c, total);
    }
}

// ---------------------------------------------------------------- host side
size_t up(size_t n) { return (n + 255) / 256 * 256; }

struct EmbedPlan {
    int passes, bits, tile, blocks, chunks;
    long pitch;
    size_t key[2], row[2], count, part, bytes;
};

EmbedPlan embed_plan(int rows, int d, int vocab)
{
    EmbedPlan q;
    int bits = 0;
    while (((int64_t)1 << bits) <= vocab) ++bits;      // keys 0 .. vocab
    q.passes = (bits + kDigitBits - 1) / kDigitBits;
    q.bits = (bits + q.passes - 1) / q.passes;
    // tiles of at least a row per thread, at most about one block per SM (every block reads all counts)
    long tile = ((long)rows + 151) / 152;
    tile = (tile + kSortThreads - 1) / kSortThreads * kSortThreads;
    q.tile = (int)tile;
    q.blocks = (int)((rows + tile - 1) / tile);
    q.chunks = (rows + kChunk - 1) / kChunk;
    q.pitch = (d + 3) / 4 * 4;
    size_t at = 0;
    auto take = [&](size_t bytes) { const size_t p = at; at += up(bytes); return p; };
    for (int x = 0; x < 2; ++x) {
        q.key[x] = take((size_t)rows * 4);
        q.row[x] = take((size_t)rows * 4);
    }
    q.count = take((size_t)q.blocks * ((size_t)1 << q.bits) * 4);
    q.part = take((size_t)q.chunks * 2 * q.pitch * 4);
    q.bytes = at;
    return q;
}

txl_status embed_sizes(int rows, int d, int vocab, txl_dtype dtype)
{
    if (dtype != TXL_F32 && dtype != TXL_BF16) return TXL_ERR_UNSUPPORTED;
    if (rows < 0 || d < 1 || vocab < 1) return TXL_ERR_INVALID;
    if (rows > kMaxSize || vocab > kMaxSize || d > kMaxWidth) return TXL_ERR_UNSUPPORTED;
    if ((int64_t)(rows > vocab ? rows : vocab) * d > kMaxElements) return TXL_ERR_UNSUPPORTED;
    return TXL_OK;
}

txl_status finish(cudaError_t e)
{
    if (e == cudaSuccess) return TXL_OK;
    note_cuda_error(e);
    return TXL_ERR_CUDA;
}

// the widest load that every row of both tensors can be read by
int load_bytes(int d, size_t esz, const void *p, const void *q)
{
    for (int n : {16, 4})
        if (d * esz % n == 0 && at_boundary(p, n) && at_boundary(q, n)) return n;
    return (int)esz;
}

template <typename T, int V>
cudaError_t run_fwd(EmbedArgs a, cudaStream_t s)
{
    a.vectors = a.d / V;
    const long want = (a.rows * a.vectors + NT - 1) / NT, most = 16L * device_sm_count();
    return chain_launch(embed_fwd_kernel<T, V>, (unsigned)(want < most ? want : most), NT, 0, 1, s, a);
}

template <typename T, int V>
cudaError_t run_sums(SumArgs a, cudaStream_t s)
{
    a.strips = (a.d + 32 * V - 1) / (32 * V);
    const long tasks = (long)a.chunks * a.strips;
    cudaError_t e = chain_launch(embed_sum_kernel<T, V>, (unsigned)((tasks + NT / 32 - 1) / (NT / 32)), NT, 0, 1, s, a);
    if (e != cudaSuccess || a.chunks == 1) return e;
    const long strips = (a.d + kJoinColumns - 1) / kJoinColumns;
    return chain_launch(embed_join_kernel<T>, (unsigned)((a.chunks - 1) * strips), NT, 0, 1, s, a);
}

cudaError_t run_bwd(const int64_t *tokens, const void *dout, float scale, int rows, int d, int vocab, txl_dtype dtype,
                    bool accumulate, void *dtable, unsigned char *ws, cudaStream_t s)
{
    const EmbedPlan q = embed_plan(rows, d, vocab);
    const size_t esz = dtype == TXL_F32 ? 4 : 2;
    const ZeroJob none = {nullptr, 0}, whole = {(unsigned char *)dtable, (size_t)vocab * d * esz};
    const size_t smem = (size_t)(kSortWarps << q.bits) * 4 + kSortWarps * 4;
    cudaError_t e = cudaFuncSetAttribute(sort_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    for (int x = 0; x < q.passes && e == cudaSuccess; ++x) {
        SortPass p;
        p.tokens = x == 0 ? tokens : nullptr;
        p.key_in = (int *)(ws + q.key[(x + 1) & 1]);
        p.row_in = (int *)(ws + q.row[(x + 1) & 1]);
        p.key_out = (int *)(ws + q.key[x & 1]);
        p.row_out = (int *)(ws + q.row[x & 1]);
        p.count = (int *)(ws + q.count);
        p.n = rows;
        p.vocab = vocab;
        p.tile = q.tile;
        p.blocks = q.blocks;
        p.shift = x * q.bits;
        p.bits = q.bits;
        const bool zero = x == 0 && !accumulate;
        const size_t rounds = whole.bytes / (16 * kSortThreads * 4) + 1, most = 2 * (size_t)device_sm_count();
        const unsigned extra = zero ? (unsigned)(rounds < most ? rounds : most) : 0;
        e = chain_launch(sort_count_kernel, (unsigned)q.blocks + extra, kSortThreads, 0, 1, s, p, zero ? whole : none);
        if (e == cudaSuccess) e = chain_launch(sort_place_kernel, (unsigned)q.blocks, kSortThreads, smem, 1, s, p);
    }
    if (e != cudaSuccess) return e;
    SumArgs a;
    a.key = (int *)(ws + q.key[(q.passes + 1) & 1]);
    a.row = (int *)(ws + q.row[(q.passes + 1) & 1]);
    a.dout = dout;
    a.dtable = dtable;
    a.part = (float *)(ws + q.part);
    a.scale = scale;
    a.n = rows;
    a.d = d;
    a.vocab = vocab;
    a.chunks = q.chunks;
    a.strips = 0;
    a.accumulate = accumulate;
    a.pitch = q.pitch;
    const int wide = load_bytes(d, esz, dout, dtable);
    if (dtype == TXL_F32) return wide == 16 ? run_sums<float, 4>(a, s) : run_sums<float, 1>(a, s);
    return wide == 16 ? run_sums<__nv_bfloat16, 8>(a, s)
           : wide == 4 ? run_sums<__nv_bfloat16, 2>(a, s) : run_sums<__nv_bfloat16, 1>(a, s);
}

}  // namespace
}  // namespace txl

using namespace txl;

extern "C" {

txl_status txl_embed_fwd(const int64_t *tokens, const void *table, float scale, int rows, int d_model, int vocab,
                         txl_dtype dtype, void *out, void *stream)
{
    txl_status st = embed_sizes(rows, d_model, vocab, dtype);
    if (st != TXL_OK) return st;
    const size_t esz = dtype == TXL_F32 ? 4 : 2, n = (size_t)rows;
    st = check_buffers({{tokens, n * 8, 8, true}, {table, rows ? (size_t)vocab * d_model * esz : 0, esz, true}},
                       {{out, n * d_model * esz, esz, true}});
    if (st != TXL_OK || rows == 0) return st;
    const EmbedArgs a = {tokens, table, out, scale, rows, 0, d_model, vocab};
    cudaStream_t s = (cudaStream_t)stream;
    const int wide = load_bytes(d_model, esz, table, out);
    if (dtype == TXL_F32) return finish(wide == 16 ? run_fwd<float, 4>(a, s) : run_fwd<float, 1>(a, s));
    return finish(wide == 16 ? run_fwd<__nv_bfloat16, 8>(a, s)
                  : wide == 4 ? run_fwd<__nv_bfloat16, 2>(a, s) : run_fwd<__nv_bfloat16, 1>(a, s));
}

txl_status txl_embed_bwd_workspace(int rows, int d_model, int vocab, txl_dtype dtype, size_t *bytes)
{
    if (!bytes) return TXL_ERR_INVALID;
    const txl_status st = embed_sizes(rows, d_model, vocab, dtype);
    if (st != TXL_OK) return st;
    *bytes = rows ? embed_plan(rows, d_model, vocab).bytes : 256;
    return TXL_OK;
}

txl_status txl_embed_bwd(const int64_t *tokens, const void *dout, float scale, int rows, int d_model, int vocab,
                         txl_dtype dtype, int accumulate, void *dtable, void *workspace, size_t workspace_bytes,
                         void *stream)
{
    txl_status st = embed_sizes(rows, d_model, vocab, dtype);
    if (st != TXL_OK) return st;
    const size_t esz = dtype == TXL_F32 ? 4 : 2, n = (size_t)rows, table = (size_t)vocab * d_model * esz;
    const bool touched = rows || !accumulate;
    st = check_buffers({{tokens, n * 8, 8, true}, {dout, n * d_model * esz, esz, true}},
                       {{dtable, touched ? table : 0, esz, true}, {workspace, rows ? workspace_bytes : 0, 256, rows > 0}});
    if (st != TXL_OK || !touched) return st;
    cudaStream_t s = (cudaStream_t)stream;
    if (rows == 0) return finish(cudaMemsetAsync(dtable, 0, table, s));
    if (!workspace || workspace_bytes < embed_plan(rows, d_model, vocab).bytes) return TXL_ERR_INVALID;
    return finish(run_bwd(tokens, dout, scale, rows, d_model, vocab, dtype, accumulate != 0, dtable,
                          (unsigned char *)workspace, s));
}

}  // extern "C"

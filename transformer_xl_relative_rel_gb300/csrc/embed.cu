// embed.cu -- the token embedding and its table's gradient.
//
//     out_i = scale table[tok_i]                          (0 for a token outside the vocabulary)
//     dtable_t (+)= scale sum_{i: tok_i = t} dout_i
//
// The gradient sums rows by token in a fixed order, so that the same call
// gives the same bits: tokens are sorted by a stable radix sort (digits of up
// to kDigitBits bits), the sorted rows are cut into chunks of kChunk, and a
// warp adds up a chunk's columns, writing each token's sum as its last row
// passes.  A token whose rows lie in several chunks leaves a partial sum in
// each, which a last launch adds (with kManyChunks or more, chunks inside one
// token's rows are joined by groups before, and those where a token begins
// that goes on are listed: 1048576 x 512 rows of one token 1730 -> 298 us).
//
// Up to kClusterRows rows are sorted by one cluster in its blocks' shared
// memory, while other clusters of the launch set the table to zero; more by a
// counting and a placing launch per digit.  (Counting and placing launches for
// all took 14 us per digit for 16896 rows, the cluster 10 for the first and 5
// for another; of 4, 8 and 16 blocks 16 are fastest: 15, 12 and 10 us.)
//
// What bounds it, forward and gradient of one call, under a profiler one by
// one: 16896 x 512 rows of 256 tokens, added to the table: gather 7 to 8, sort
// 10 to 12, sums 7, join 6 to 7 us, latencies of launches and of a handful of dependent loads
// in each (the bytes are worth 5 us); 6144 x 1024 rows, table of 131072 set
// to zero: 45 us for 268 MB (5.9 TB/s, the sort hidden in it), sums 8, join 4.
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
constexpr int kChunk = 16;                         // sorted rows a warp adds up
constexpr int kMostBlocks = 16;                    // of the sorting cluster
constexpr int kBlockRows = 8192;                   // of one of its blocks: two lists of 64 KB beside the counters
constexpr int kClusterRows = kMostBlocks * kBlockRows;
constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kDigitBits = 9;                      // a placing block's counters: 32 warps x 512 digits, 64 KB

// ---------------------------------------------------------------- forward
struct EmbedArgs {
    const int64_t *tokens;
    const void *table;
    void *out;
    float scale;
    int rows, d, vocab, shift;      // 1 << shift threads take a row
};

template <typename T, int V>
__global__ void __launch_bounds__(NT) embed_fwd_kernel(const __grid_constant__ EmbedArgs a)
{
    chain_begin();
    chain_wait();
    const long row = ((long)blockIdx.x * NT + threadIdx.x) >> a.shift;
    if (row >= a.rows) return;
    const int threads = 1 << a.shift, first = (threadIdx.x & (threads - 1)) * V, step = threads * V;
    const int64_t t = a.tokens[row];
    const bool in = t >= 0 && t < a.vocab;
    const T *from = (const T *)a.table + (in ? t : 0) * a.d;
    T *to = (T *)a.out + row * a.d;
    constexpr int U = 4;      // vectors asked for at once
    for (int c = first; c < a.d; c += U * step) {
        raw_t<T, V> raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (in && c + u * step < a.d) raw[u] = load_raw<T, V>(from + c + u * step);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float v[V] = {};
            if (in && c + u * step < a.d) {
                unpack<T, V>(raw[u], v);
#pragma unroll
                for (int i = 0; i < V; ++i) v[i] *= a.scale;
            }
            if (c + u * step < a.d) store_vec<T, V>(to + c + u * step, v);
        }
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

// what the sort's first launch sets to zero besides: the table, the work list's length
struct ZeroJob {
    unsigned char *p;
    size_t bytes;
    int *length;
};

__device__ __forceinline__ int sort_key(const SortPass &a, int i)
{
    if (!a.tokens) return a.key_in[i];
    const int64_t t = a.tokens[i];
    return t >= 0 && t < a.vocab ? (int)t : a.vocab;
}

// The lanes with the digit d, among those that have a row (in).  A ballot per
// bit: the instruction that matches whole values takes a turn per different
// value (131072 rows of as many tokens sorted in 51 us with it, 39 without).
__device__ __forceinline__ unsigned same_digit(int d, int bits, bool in)
{
    unsigned same = __ballot_sync(0xffffffffu, in);
#pragma unroll
    for (int b = 0; b < kDigitBits; ++b)
        if (b < bits) {
            const bool set = d >> b & 1;
            const unsigned with = __ballot_sync(0xffffffffu, set);
            same &= set ? with : ~with;
        }
    return same;
}

// sets the table to zero, as block `block` of `blocks` of kSortThreads threads
__device__ __forceinline__ void zero_table(const ZeroJob &z, long block, long blocks)
{
    const long stride = blocks * kSortThreads, first = block * kSortThreads + threadIdx.x;
    const size_t head = z.bytes < (-(uintptr_t)z.p & 15) ? z.bytes : (-(uintptr_t)z.p & 15);
    const size_t n16 = (z.bytes - head) / 16, tail = z.bytes - head - 16 * n16;
    uint4 *v = (uint4 *)(z.p + head);
    for (long i = first; i < (long)n16; i += stride) v[i] = make_uint4(0, 0, 0, 0);
    if (first < (long)(head / 2)) ((uint16_t *)z.p)[first] = 0;
    if (first < (long)(tail / 2)) ((uint16_t *)(z.p + z.bytes - tail))[first] = 0;
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
    if (z.length && blockIdx.x == 0 && threadIdx.x == 0) *z.length = 0;
    if ((int)blockIdx.x >= a.blocks) {
        zero_table(z, blockIdx.x - a.blocks, gridDim.x - a.blocks);
        return;
    }
    __syncthreads();
    const int lane = threadIdx.x & 31, first = blockIdx.x * a.tile;
    const int end = min(first + a.tile, a.n);
    for (int i = first + (int)threadIdx.x; i - lane < end; i += kSortThreads) {
        const bool in = i < end;
        const int d = (in ? sort_key(a, i) : 0) >> a.shift & (digits - 1);
        const unsigned same = same_digit(d, a.bits, in);
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
        const int d = (in ? sort_key(a, i) : 0) >> a.shift & (digits - 1);
        const unsigned same = same_digit(d, a.bits, in);
        if (in && (same & ((1u << lane) - 1)) == 0) mine[d] += __popc(same);
        __syncwarp();
    }
    // a digit's rows in all blocks, and those in the blocks before this one
    int total = 0, before = 0;
    if (t < digits)
        for (int b = 0; b < a.blocks; b += 16) {      // (16 asked for at once)
            int c[16];
#pragma unroll
            for (int u = 0; u < 16; ++u) c[u] = b + u < a.blocks ? a.count[(size_t)(b + u) * digits + t] : 0;
#pragma unroll
            for (int u = 0; u < 16; ++u) {
                if (b + u < (int)blockIdx.x) before += c[u];
                total += c[u];
            }
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
        const int d = key >> a.shift & (digits - 1);
        const unsigned same = same_digit(d, a.bits, in), below = same & ((1u << lane) - 1);
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

// ---------------------------------------------------------------- one cluster's sort
struct ClusterSort {
    const int64_t *tokens;
    int *key, *row;                  // [n] sorted
    int n, vocab, blocks, tile, bits, passes;
};

__device__ __forceinline__ uint32_t shared_address(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
// the address of another block's copy of what lies at `at` in this one's shared memory
__device__ __forceinline__ uint32_t in_block(uint32_t at, int block)
{
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(at), "r"(block));
    return r;
}
__device__ __forceinline__ void cluster_barrier()
{
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// The first cluster sorts, block b holding the sorted places b tile .. of every
// pass; the others set the table to zero.  A pass counts the digits of each
// warp's rows, adds up over warps, exchanges the blocks' totals, and sends
// each row to its place in its block (in the last pass, to memory).
__global__ void __launch_bounds__(kSortThreads)
embed_sort_kernel(const __grid_constant__ ClusterSort a, const __grid_constant__ ZeroJob z)
{
    chain_begin();
    if ((int)blockIdx.x >= a.blocks) {
        chain_wait();
        zero_table(z, blockIdx.x - a.blocks, gridDim.x - a.blocks);
        return;
    }
    extern __shared__ __align__(16) unsigned char dynamic[];
    const int digits = 1 << a.bits, t = threadIdx.x, lane = t & 31, w = t >> 5, rank = blockIdx.x;
    int *count = (int *)dynamic;                      // [kSortWarps][digits]
    int *total = count + kSortWarps * digits;         // [digits] of this block
    int *base = total + digits;                       // [digits]: the place of this block's first row of a digit
    int *sums = base + digits;                        // [kSortWarps]
    int2 *list[2] = {(int2 *)(sums + kSortWarps), (int2 *)(sums + kSortWarps) + a.tile};    // keys and rows
    int *mine = count + w * digits;
    const int first = rank * a.tile, n = max(0, min(a.tile, a.n - first));
    const int per = (a.tile + kSortWarps - 1) / kSortWarps, from = min(w * per, n), to = min(from + per, n);
    chain_wait();
    if (z.length && rank == 0 && t == 0) *z.length = 0;
    for (int i = t; i < n; i += kSortThreads) {
        const int64_t token = a.tokens[first + i];
        list[0][i] = make_int2(token >= 0 && token < a.vocab ? (int)token : a.vocab, first + i);
    }
    for (int pass = 0; pass < a.passes; ++pass) {
        const int2 *in = list[pass & 1];
        const int shift = pass * a.bits;
        for (int x = t; x < kSortWarps * digits / 4; x += kSortThreads) ((int4 *)count)[x] = make_int4(0, 0, 0, 0);
        __syncthreads();
        for (int i = from + lane; i - lane < to; i += 32) {
            const int d = (i < to ? in[i].x : 0) >> shift & (digits - 1);
            const unsigned same = same_digit(d, a.bits, i < to);
            if (i < to && (same & ((1u << lane) - 1)) == 0) mine[d] += __popc(same);
            __syncwarp();
        }
        __syncthreads();
        if (t < digits) {      // (loads before what depends on them: one wait, not 32)
            int c[kSortWarps], run = 0;
#pragma unroll
            for (int x = 0; x < kSortWarps; ++x) c[x] = count[x * digits + t];
#pragma unroll
            for (int x = 0; x < kSortWarps; ++x) {
                count[x * digits + t] = run;
                run += c[x];
            }
            total[t] = run;
        }
        cluster_barrier();
        int all = 0, before = 0;
        if (t < digits) {
            const uint32_t at = shared_address(total + t);
            int c[kMostBlocks];
#pragma unroll
            for (int b = 0; b < kMostBlocks; ++b) {
                c[b] = 0;
                if (b < a.blocks) asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(c[b]) : "r"(in_block(at, b)));
            }
#pragma unroll
            for (int b = 0; b < kMostBlocks; ++b) {
                all += c[b];
                before += b < rank ? c[b] : 0;
            }
        }
        int run = all;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, run, o);
            if (lane >= o) run += v;
        }
        if (lane == 31) sums[w] = run;
        __syncthreads();
        run += __reduce_add_sync(0xffffffffu, lane < w ? sums[lane] : 0);
        if (t < digits) base[t] = run - all + before;
        __syncthreads();
        const bool last = pass + 1 == a.passes;
        const uint32_t out = shared_address(list[(pass + 1) & 1]);
        for (int i = from + lane; i - lane < to; i += 32) {
            const int2 one = i < to ? in[i] : make_int2(0, 0);
            const int d = one.x >> shift & (digits - 1);
            const unsigned same = same_digit(d, a.bits, i < to), below = same & ((1u << lane) - 1);
            if (i < to) {
                const unsigned place = base[d] + mine[d] + __popc(below);
                if (last) {
                    a.key[place] = one.x;
                    a.row[place] = one.y;
                } else {
                    const unsigned block = place / (unsigned)a.tile;
                    const uint32_t at = in_block(out + (place - block * a.tile) * 8, (int)block);
                    asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(at), "r"(one.x), "r"(one.y) : "memory");
                }
            }
            __syncwarp();
            if (i < to && below == 0) mine[d] += __popc(same);
            __syncwarp();
        }
        // (after the last pass: no block ends while another reads its totals)
        cluster_barrier();
    }
}

// ---------------------------------------------------------------- sums
struct SumArgs {
    const int *key, *row;    // sorted by token
    const void *dout;
    void *dtable;
    float *part;             // [chunks][2][pitch]: sums of a token that begins before the chunk (0), of one
                             // that begins in it and goes on behind it (1)
    int *work;               // NULL, or the number of chunks in which a token begins that goes on, and these chunks
    float scale;
    int n, d, vocab, chunks, strips, accumulate;
    long pitch;
};

constexpr int kStrip = 256;      // columns of a warp: 32 K V

// A warp adds kStrip columns of a chunk's rows, of which U are asked for at
// once, as many as 64 registers hold.  ACC: with each token's last row the
// table's is asked for too (one after another they made forward and gradient
// of 6144 x 1024 rows of 3000 tokens take 64 us where it is 26).
template <typename T, int V, bool ACC>
__global__ void __launch_bounds__(NT) embed_sum_kernel(const __grid_constant__ SumArgs a)
{
    constexpr int K = kStrip / (32 * V), kRegs = K * (sizeof(raw_t<T, V>) >= 4 ? (int)sizeof(raw_t<T, V>) / 4 : 1);
    constexpr int U = (ACC ? 32 : 64) / kRegs;
    static_assert(kChunk % U == 0, "a chunk is so many whole batches");
    chain_begin();
    chain_wait();
    const int lane = threadIdx.x & 31;
    const long task = (long)blockIdx.x * (NT / 32) + (threadIdx.x >> 5);
    const int chunk = (int)(task / a.strips), c = (int)(task - (long)chunk * a.strips) * kStrip + lane * V;
    if (chunk >= a.chunks) return;
    const int first = chunk * kChunk, n = min(kChunk, a.n - first);
    const int key = lane < n ? a.key[first + lane] : a.vocab;
    const int row = lane < n ? a.row[first + lane] : 0;
    const int before = first > 0 ? a.key[first - 1] : -1, after = first + n < a.n ? a.key[first + n] : a.vocab;
    const int live = __popc(__ballot_sync(0xffffffffu, key < a.vocab)), head = __shfl_sync(0xffffffffu, key, 0);
    // a token's last row here, and whether others of it lie before or behind
    const int next = __shfl_down_sync(0xffffffffu, key, 1);
    const unsigned last = __ballot_sync(0xffffffffu, lane < live && (lane + 1 == n || next != key));
    const bool from_before = before == key, goes_on = lane + 1 == n && after == key;
    const unsigned whole = __ballot_sync(0xffffffffu, lane < live && !((key == head && from_before) || goes_on));
    // (the list's order does not matter: its entries are summed one by one)
    if (a.work && lane + 1 == kChunk && lane < live && goes_on && !(key == head && from_before) && c < kStrip)
        a.work[1 + atomicAdd(a.work, 1)] = chunk;
    float acc[K][V];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) acc[k][i] = 0.f;
    for (int j = 0; j < live; j += U) {
        raw_t<T, V> raw[U][K], old[ACC ? U : 1][K];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const T *from = (const T *)a.dout + (size_t)__shfl_sync(0xffffffffu, row, (j + u) & 31) * a.d;
            const T *to = (const T *)a.dtable + (size_t)__shfl_sync(0xffffffffu, key, (j + u) & 31) * a.d;
            const bool in = j + u < live, ends = ACC && (last & whole) >> ((j + u) & 31) & 1;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int at = c + 32 * k * V;
                if (in && at < a.d) raw[u][k] = load_raw<T, V>(from + at);
                if (ends && at < a.d) old[ACC ? u : 0][k] = load_raw<T, V>(to + at);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (j + u >= live) break;
            const int token = __shfl_sync(0xffffffffu, key, j + u);
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (c + 32 * k * V < a.d) {
                    float v[V];
                    unpack<T, V>(raw[u][k], v);
#pragma unroll
                    for (int i = 0; i < V; ++i) acc[k][i] += v[i];
                }
            if (!(last >> (j + u) & 1)) continue;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int at = c + 32 * k * V;
                if (at < a.d) {
                    if (!(whole >> (j + u) & 1)) {
                        // to the first place where rows of it lie in chunks before
                        const bool begins = !(token == head && before == token);
                        store_floats<V>(a.part + (2 * (size_t)chunk + begins) * a.pitch + at, acc[k]);
                    } else {
                        float x[V];
                        if (ACC) unpack<T, V>(old[ACC ? u : 0][k], x);
#pragma unroll
                        for (int i = 0; i < V; ++i) x[i] = ACC ? fmaf(a.scale, acc[k][i], x[i]) : a.scale * acc[k][i];
                        store_vec<T, V>((T *)a.dtable + (size_t)token * a.d + at, x);
                    }
                }
#pragma unroll
                for (int i = 0; i < V; ++i) acc[k][i] = 0.f;
            }
        }
    }
}

// Joining the partial sums of tokens that begin in a chunk and go on behind it.
constexpr int kJoinWarps = NT / 32, kJoinColumns = 128;
constexpr int kJoinAlone = 8;      // chunks behind the first that a warp adds by itself
constexpr int kGroup = 32;         // chunks whose sums are joined beforehand where one token fills them
constexpr int kManyChunks = 2048;  // from which on there are groups and a list of work

__device__ __forceinline__ void add_float4(float4 &acc, const float4 &v)
{
    acc.x += v.x;
    acc.y += v.y;
    acc.z += v.z;
    acc.w += v.w;
}

// the partial sums of a chunk's token from before (0) or going on (1), four columns
__device__ __forceinline__ float4 part_of(const SumArgs &a, int chunk, int which, int c)
{
    return *(const float4 *)(a.part + (2 * (size_t)chunk + which) * a.pitch + c);
}

template <typename T>
__device__ __forceinline__ void write_sum(const SumArgs &a, int token, int c, float sum)
{
    T *to = (T *)a.dtable + (size_t)token * a.d + c;
    float x[1] = {0.f};
    if (a.accumulate) unpack<T, 1>(load_raw<T, 1>(to), x);
    x[0] = a.accumulate ? fmaf(a.scale, sum, x[0]) : a.scale * sum;
    store_vec<T, 1>(to, x);
}

// The sums of the warps' `acc`, of kJoinColumns columns, in the first threads.
__device__ __forceinline__ float block_columns(const float4 &acc, float4 (&sums)[kJoinWarps][32])
{
    __syncthreads();             // (the places may still be read)
    sums[threadIdx.x >> 5][threadIdx.x & 31] = acc;
    __syncthreads();
    float all = 0.f;
    if (threadIdx.x < kJoinColumns)
#pragma unroll
        for (int k = 0; k < kJoinWarps; ++k) all += ((const float *)sums[k])[threadIdx.x];
    return all;
}

// Joins each group of chunks that lie inside one token's: their sum takes the
// place 1 of the first one's, which such chunks do not use.
__global__ void __launch_bounds__(NT) embed_group_kernel(const __grid_constant__ SumArgs a)
{
    chain_begin();
    __shared__ float4 sums[kJoinWarps][32];
    const int lane = threadIdx.x & 31, y = threadIdx.x >> 5, strips = (a.d + kJoinColumns - 1) / kJoinColumns;
    const int first = (int)(blockIdx.x / strips) * kGroup, c = (int)(blockIdx.x % strips) * kJoinColumns + 4 * lane;
    const long row = (long)first * kChunk, after = row + kGroup * kChunk;
    chain_wait();
    if (row == 0 || after >= a.n) return;
    const int key = a.key[row], before = a.key[row - 1], behind = a.key[after];
    if (key >= a.vocab || before != key || behind != key) return;
    constexpr int kEach = kGroup / kJoinWarps;
    float4 v[kEach];
#pragma unroll
    for (int u = 0; u < kEach; ++u) v[u] = c < a.d ? part_of(a, first + y + u * kJoinWarps, 0, c) : make_float4(0, 0, 0, 0);
#pragma unroll
    for (int u = 1; u < kEach; ++u) add_float4(v[0], v[u]);
    const float all = block_columns(v[0], sums);
    const int column = (int)(blockIdx.x % strips) * kJoinColumns + threadIdx.x;
    if (threadIdx.x < kJoinColumns && column < a.d) a.part[(2 * (size_t)first + 1) * a.pitch + column] = all;
}

// The last chunk with rows of the token `key`, which has the first row of
// `chunk` + 1 (a warp's search by 32 chunks' first rows at once).
__device__ __forceinline__ int last_chunk(const SumArgs &a, int chunk, int key)
{
    int lo = chunk, hi = a.chunks;      // lo has rows of it, hi has not
    while (hi - lo > 1) {
        const int step = (hi - lo + 32) / 33;
        const long at = lo + (long)step * ((threadIdx.x & 31) + 1);
        const int in = __popc(__ballot_sync(0xffffffffu, at < hi && a.key[at * kChunk] == key));
        if ((long)lo + (long)step * (in + 1) < hi) hi = lo + step * (in + 1);
        lo += step * in;
    }
    return lo;
}

// The sum of the token's chunks from `chunk` to `end` over the block's warps,
// warp y taking the y-th, (y + 8)-th, ... of them, groups (where there are) as one.
__device__ __forceinline__ float4 warp_share(const SumArgs &a, int chunk, int end, bool groups, int c, int y)
{
    // chunks before the first group inside, the groups, chunks behind them
    int g0 = chunk / kGroup + 1, g1 = end / kGroup;
    if (!groups || g1 < g0) g0 = g1 = end / kGroup + 1;
    const int head = min(end + 1, g0 * kGroup) - chunk, inside = g1 - g0;
    const int total = head + inside + (end + 1 > g1 * kGroup ? end + 1 - g1 * kGroup : 0);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (c < a.d)
        for (int i = y; i < total; i += 8 * kJoinWarps) {
            float4 v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int x = i + u * kJoinWarps;
                if (x < head) v[u] = part_of(a, chunk + x, x == 0, c);
                else if (x < head + inside) v[u] = part_of(a, (g0 + x - head) * kGroup, 1, c);
                else if (x < total) v[u] = part_of(a, g1 * kGroup + x - head - inside, 0, c);
            }
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (i + u * kJoinWarps < total) add_float4(acc, v[u]);
        }
    return acc;
}

// Warp y looks at the y-th of eight chunks and adds what begins there where
// that is in few chunks; a longer token's are shared out among the warps.  The
// chunks are a block's own, or, LIST, the listed ones, blocks taking eight of
// them and a strip in turn.
template <typename T, bool LIST>
__global__ void __launch_bounds__(NT) embed_join_kernel(const __grid_constant__ SumArgs a)
{
    chain_begin();
    __shared__ int token[kJoinWarps], begins[kJoinWarps], ends[kJoinWarps];
    __shared__ float4 sums[kJoinWarps][32];
    const int lane = threadIdx.x & 31, y = threadIdx.x >> 5, strips = (a.d + kJoinColumns - 1) / kJoinColumns;
    chain_wait();
    const int listed = LIST ? a.work[0] : 0;
    const long items = LIST ? ((long)listed + kJoinWarps - 1) / kJoinWarps * strips : (long)gridDim.x;
    for (long item = blockIdx.x; item < items; item += gridDim.x) {
        const int group = (int)(item / strips) * kJoinWarps, strip = (int)(item % strips) * kJoinColumns;
        const int c = strip + 4 * lane;
        {
            const bool there = !LIST || group + y < listed;
            const int chunk = LIST ? (there ? a.work[1 + group + y] : 0) : group + y;
            const int first = chunk * kChunk, next = first + kChunk;
            int key = -1, end = chunk;      // end: the last chunk with rows of it
            if (there && next < a.n) {
                const long at = (long)next + (long)lane * kChunk;      // (asked for at once with the others)
                const int begin = at < a.n ? a.key[at] : -1;
                const int before = first > 0 ? a.key[first - 1] : -1;
                key = a.key[next - 1];
                if (key >= a.vocab || before == key) key = -1;
                const unsigned same = __ballot_sync(0xffffffffu, begin == key);
                if (key >= 0) end = same == 0xffffffffu ? last_chunk(a, chunk + 32, key) : chunk + __ffs(~same) - 1;
                if (end == chunk) key = -1;
            }
            if (key >= 0 && end - chunk <= kJoinAlone) {
                if (c < a.d) {
                    float4 v[kJoinAlone + 1];
#pragma unroll
                    for (int k = 0; k <= kJoinAlone; ++k)
                        if (chunk + k <= end) v[k] = part_of(a, chunk + k, k == 0, c);
#pragma unroll
                    for (int k = 1; k <= kJoinAlone; ++k)
                        if (chunk + k <= end) add_float4(v[0], v[k]);
                    const float one[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (c + i < a.d) write_sum<T>(a, key, c + i, one[i]);
                }
                key = -1;
            }
            if (LIST) __syncthreads();      // (the places may still be read)
            if (lane == 0) {
                token[y] = key;
                begins[y] = chunk;
                ends[y] = end;
            }
        }
        __syncthreads();
        for (int x = 0; x < kJoinWarps; ++x) {
            if (token[x] < 0) continue;
            const float all = block_columns(warp_share(a, begins[x], ends[x], LIST, c, y), sums);
            if (threadIdx.x < kJoinColumns && strip + (int)threadIdx.x < a.d) write_sum<T>(a, token[x], strip + threadIdx.x, all);
        }
    }
}

// ---------------------------------------------------------------- host side
size_t up(size_t n) { return (n + 255) / 256 * 256; }

struct EmbedPlan {
    bool cluster;
    int passes, bits, tile, blocks, chunks;
    long pitch;
    size_t key[2], row[2], count, part, work, bytes;
};

EmbedPlan embed_plan(int rows, int d, int vocab)
{
    EmbedPlan q;
    int bits = 0;
    while (((int64_t)1 << bits) <= vocab) ++bits;      // keys 0 .. vocab
    q.passes = (bits + kDigitBits - 1) / kDigitBits;
    q.bits = (bits + q.passes - 1) / q.passes;
    q.cluster = rows <= kClusterRows;
    if (q.cluster) {     // as many blocks as leave each a row per thread
        for (q.blocks = 1; q.blocks < kMostBlocks && q.blocks * kSortThreads < rows;) q.blocks *= 2;
        q.tile = (rows + q.blocks - 1) / q.blocks;
    } else {             // at most about one block per SM: every block reads all counts
        const long tile = ((long)rows + 151) / 152;
        q.tile = (int)((tile + kSortThreads - 1) / kSortThreads * kSortThreads);
        q.blocks = (int)(((long)rows + q.tile - 1) / q.tile);
    }
    q.chunks = (rows + kChunk - 1) / kChunk;
    q.pitch = (d + 3) / 4 * 4;
    size_t at = 0;
    auto take = [&](size_t bytes) { const size_t p = at; at += up(bytes); return p; };
    for (int x = 0; x < (q.cluster ? 1 : 2); ++x) {
        q.key[x] = take((size_t)rows * 4);
        q.row[x] = take((size_t)rows * 4);
    }
    q.count = take(q.cluster ? 0 : (size_t)q.blocks * ((size_t)1 << q.bits) * 4);
    q.part = take((size_t)q.chunks * 2 * q.pitch * 4);
    q.work = take(q.chunks >= kManyChunks ? (size_t)(q.chunks + 1) * 4 : 0);
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
    for (a.shift = 0; a.shift < 5 && (V << a.shift) < a.d;) ++a.shift;      // a warp at most
    const long threads = (long)a.rows << a.shift;
    return chain_launch(embed_fwd_kernel<T, V>, (unsigned)((threads + NT - 1) / NT), NT, 0, 1, s, a);
}

template <typename T, int V>
cudaError_t run_sums(SumArgs a, cudaStream_t s)
{
    a.strips = (a.d + kStrip - 1) / kStrip;
    const long tasks = (long)a.chunks * a.strips;
    cudaError_t e = chain_launch(a.accumulate ? embed_sum_kernel<T, V, true> : embed_sum_kernel<T, V, false>,
                                 (unsigned)((tasks + NT / 32 - 1) / (NT / 32)), NT, 0, 1, s, a);
    if (e != cudaSuccess || a.chunks == 1) return e;
    const long strips = (a.d + kJoinColumns - 1) / kJoinColumns;
    if (a.work) {
        e = chain_launch(embed_group_kernel, (unsigned)((a.chunks + kGroup - 1) / kGroup * strips), NT, 0, 1, s, a);
        const long want = (a.chunks + kJoinWarps - 1) / kJoinWarps * strips, most = 4L * device_sm_count();
        if (e == cudaSuccess)
            e = chain_launch(embed_join_kernel<T, true>, (unsigned)(want < most ? want : most), NT, 0, 1, s, a);
        return e;
    }
    const long groups = (a.chunks + kJoinWarps - 2) / kJoinWarps;
    return chain_launch(embed_join_kernel<T, false>, (unsigned)(groups * strips), NT, 0, 1, s, a);
}

// blocks that set the table to zero: at most what fills the SMs
unsigned zero_blocks(const ZeroJob &z)
{
    const size_t want = (z.bytes + 16 * kSortThreads * 4 - 1) / (16 * kSortThreads * 4), most = 2 * (size_t)device_sm_count();
    return (unsigned)(want < most ? want : most);
}

cudaError_t sort_in_cluster(const EmbedPlan &q, const int64_t *tokens, int rows, int vocab, const ZeroJob &z, int *key,
                            int *row, cudaStream_t s)
{
    const ClusterSort a = {tokens, key, row, rows, vocab, q.blocks, q.tile, q.bits, q.passes};
    const size_t smem = ((size_t)(kSortWarps + 2) << q.bits) * 4 + kSortWarps * 4 + (size_t)q.tile * 16;
    // (of all calls: the largest list and the most digits)
    constexpr int kMost = ((kSortWarps + 2) << kDigitBits) * 4 + kSortWarps * 4 + kBlockRows * 16;
    static_assert(kMost <= 227 << 10, "shared memory of a block");
    cudaError_t e = cudaFuncSetAttribute(embed_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    if (e == cudaSuccess && q.blocks > 8)
        e = cudaFuncSetAttribute(embed_sort_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    const unsigned zero = zero_blocks(z), clusters = 1 + (zero + q.blocks - 1) / q.blocks;
    return chain_launch(embed_sort_kernel, clusters * q.blocks, kSortThreads, smem, (unsigned)q.blocks, s, a, z);
}

cudaError_t sort_by_launches(const EmbedPlan &q, const int64_t *tokens, int rows, int vocab, const ZeroJob &z,
                             unsigned char *ws, cudaStream_t s)
{
    const size_t smem = (size_t)(kSortWarps << q.bits) * 4 + kSortWarps * 4;
    cudaError_t e = cudaFuncSetAttribute(sort_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (kSortWarps << kDigitBits) * 4 + kSortWarps * 4);
    const ZeroJob none = {nullptr, 0, nullptr};
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
        const unsigned extra = x == 0 ? zero_blocks(z) : 0;
        e = chain_launch(sort_count_kernel, (unsigned)q.blocks + extra, kSortThreads, 0, 1, s, p, x == 0 ? z : none);
        if (e == cudaSuccess) e = chain_launch(sort_place_kernel, (unsigned)q.blocks, kSortThreads, smem, 1, s, p);
    }
    return e;
}

cudaError_t run_bwd(const int64_t *tokens, const void *dout, float scale, int rows, int d, int vocab, txl_dtype dtype,
                    bool accumulate, void *dtable, unsigned char *ws, cudaStream_t s)
{
    const EmbedPlan q = embed_plan(rows, d, vocab);
    const size_t esz = dtype == TXL_F32 ? 4 : 2;
    int *work = q.chunks >= kManyChunks ? (int *)(ws + q.work) : nullptr;
    const ZeroJob z = {(unsigned char *)dtable, accumulate ? 0 : (size_t)vocab * d * esz, work};
    const int sorted = q.cluster ? 0 : (q.passes + 1) & 1;
    int *key = (int *)(ws + q.key[sorted]), *row = (int *)(ws + q.row[sorted]);
    const cudaError_t e = q.cluster ? sort_in_cluster(q, tokens, rows, vocab, z, key, row, s)
                                    : sort_by_launches(q, tokens, rows, vocab, z, ws, s);
    if (e != cudaSuccess) return e;
    SumArgs a;
    a.key = key;
    a.row = row;
    a.dout = dout;
    a.dtable = dtable;
    a.part = (float *)(ws + q.part);
    a.work = work;
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
    const EmbedArgs a = {tokens, table, out, scale, rows, d_model, vocab, 0};
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

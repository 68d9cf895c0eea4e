// loss_products.cu -- the output-layer losses' products on the tensor cores.
//
// Three passes share one persistent tcgen05 kernel, D = A B^T with fp32
// accumulators in TMEM and a different epilogue each:
//   lse       A = h, B = W: the running maximum and sum of the softmax over a
//             strip of vocabulary tiles, the logits themselves never stored;
//   dz        A = h, B = W: dz = coef (softmax - listed weights) of one
//             vocabulary piece, in the bf16 parts that dz_parts() says;
//   contract  dW = dz^T h (A = dz^T read as it is stored, MN-major tiles; B =
//             h^T from a transposed copy of h) and dh = dz W, as its transpose
//             W^T dz^T (A = W^T as W is stored, B = dz), turned back on the
//             way out.  An MN-major A costs nothing, an MN-major B a quarter
//             of the rate (9728 x 1024 over 9728: 1803 against 1323
//             TFLOP/s), so B is MN-major only where d_model fills the rows of
//             the transposed tiles badly (dh = dz W directly).
// fp32 operands are held as three bf16 parts whose sum is exact (8 + 8 + 8
// bits of the 24-bit significand); the product keeps the six part products
// down to 2^-16 of the largest, dropping three of at most 2^-24, smallest
// first.  The tensor core truncates where it accumulates (measured: a chain of
// n additions comes out about n 2^-25 too small), so with fp32 operands an
// accumulator takes two 64-deep steps (8 additions of the largest products)
// and the epilogue warps add these in registers, rounding to nearest.
//
// What bounds them (GB300, device time of a launch, bf16): with many rows the
// tensor pipe.  6144 x 1024 over 131072 tokens: lse 888 us (1857 TFLOP/s), dz
// 257 us per 32768 of them (1604; it stores 403 MB meanwhile), both products
// of that piece in one launch 474 us (1739).  At d_model 512 a tile has half
// the products for the same epilogue: 16384 x 512 over 65536 tokens lse 653
// us (1683), dz 762 (1443), products 1372 (1603); 64 listed columns per row
// cost lse 6% and dz 18%, half of it the search at the start of a strip.
// A bias costs lse 7% and dz 12% there (9000 x 410 x 50021).  Up to 128 rows
// the weights' way from memory: 128 x 1024 over 65536 tokens 25 us (5.3 TB/s).
// fp32 operands take six part products and twice as many, narrower tiles:
// 1111 x 410 x 20011 lse 107 us (1020 TFLOP/s of part products).
//
// Roles (12 warps): warp 0 issues the TMA loads, warp 1 the MMAs, warps 4-11
// are two epilogue groups of four (a warp per 32 TMEM lanes), which share a
// tile's 64-column chunks alternately.  Two accumulators: a tile's epilogue
// runs beside the next tile's MMAs.  With more than 128 rows a pair of CTAs
// on neighbouring SMs works on a 256-row tile (cta_group::2): each holds its
// own 128 rows of A and half of the columns of B, so a stage is 32 KB per
// SM instead of 48 KB for the same products.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <atomic>

#include "internal.h"
#include "loss_products.h"
#include "sm100.cuh"

namespace txl {

// bounded waits of the kernel below that gave up (read by txl_check, a copy of
// some 10 us, once a launch was made or captured)
__device__ unsigned int g_loss_err;
static std::atomic<bool> g_loss_ran{false};

namespace {
using namespace sm100;

constexpr int LK = 64;                         // K elements per stage
constexpr int LNT = 384;
constexpr int kPartSteps = 2;                  // steps per accumulation of fp32 operands
constexpr int LEPI = 8;                        // epilogue warps
constexpr uint64_t LWAIT_NS = 2000000000ull;   // 2 s per wait, then give up

enum { MODE_LSE = 0, MODE_DZ = 1, MODE_CT = 2 };

// kParts: fp32 operands in three bf16 parts (128-wide tiles, one stage per
// part); else bf16 operands (256-wide tiles).  dz stores a whole tile from
// every accumulation, so its staging buffers are two per epilogue warp.
template <int CG, int MODE, bool kParts>
struct LSmem {
    static constexpr int BN = kParts ? 128 : 256;           // widest tile
    static constexpr int STG = MODE == MODE_LSE ? 0 : MODE == MODE_DZ ? 2 : 1;
    static constexpr uint32_t ASZ = 128 * 128;              // 128 rows of 64 elements
    static constexpr uint32_t BSZ = BN / CG * 128;
    static constexpr int ST = (int)((224u * 1024u - LEPI * 4096u * STG) / (ASZ + BSZ));
    static constexpr uint32_t A = 0, B = A + ST * ASZ, OST = B + ST * BSZ, BARS = OST + LEPI * 4096 * STG;
    static constexpr int FULL = 0, EMPTY = ST, AFULL = 2 * ST, AEMPTY = 2 * ST + 2, DONE = 2 * ST + 4,
                         JFULL = 2 * ST + 5, JEMPTY = JFULL + 4, NBAR = JEMPTY + 4;
    static constexpr uint32_t MISC = BARS + (NBAR + (NBAR & 1)) * 8, JOIN = MISC + 16;
    static constexpr uint32_t TOTAL = JOIN + (MODE == MODE_LSE ? 1024 : 0) + 1024;
    static_assert(TOTAL <= 232448 && ST >= 3, "shared memory");
};

// one output of a contraction launch
struct LJob {
    int M, N, bn, tiles_m, tiles_n, ksteps, splits, items;
    int a_mn, b_mn;           // operands stored with the output index innermost
    int bn_last;              // the last column tile's width
    int a_box;                // rows of K-major A that are loaded, a multiple of 8
    int f32, add, out_t;      // out_t: element (m, n) goes to row n, column m
    void *out;                // where TMA stores cannot write (else NULL)
    long pitch;
};
struct LMaps {
    CUtensorMap a[2], b[2], o[2];
};

struct LParams {
    int items;
    // vocabulary passes
    int M, N, bn, tiles_m, tiles_n, strip, ksteps, a_box;
    const float *bias;        // [columns]; -infinity takes a column out
    int v0;
    float alpha;
    LossRows r;
    float *ysel, *dbpart;
    float2 *part;
    float *loss, *lse;        // cross entropy whose rows are an item's alone; else NULL
    long dbpitch;
    // contraction: the pairs without a last item of job 0 do `ahead` items of
    // job 1 in the meantime
    LJob job[2];
    int ahead;
};

// ------------------------------------------------------------ cta_group forms
template <int CG>
__device__ __forceinline__ void l_alloc(uint32_t dst)
{
    if (CG == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(dst) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
        tmem_alloc(dst, 512);
        tmem_relinquish();
    }
}
template <int CG>
__device__ __forceinline__ void l_dealloc(uint32_t t)
{
    if (CG == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(t) : "memory");
    else
        tmem_dealloc(t, 512);
}
template <int CG>
__device__ __forceinline__ void l_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    if (CG == 2)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(acc)
            : "memory");
    else
        mma_bf16_ss(d, a, b, idesc, acc);
}
// arrives on a barrier of this CTA
__device__ __forceinline__ void l_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// arrives on the barrier of that offset in every CTA of the tile
template <int CG>
__device__ __forceinline__ void l_commit(uint32_t bar)
{
    if (CG == 2)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
            "h"((uint16_t)3)
            : "memory");
    else
        mma_commit(bar);
}
template <int CG>
__device__ __forceinline__ void l_load(uint32_t dst, const CUtensorMap *m, uint32_t bar, int x, int y, int z)
{
    if (CG == 2)
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2"
            " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "r"(y), "r"(z)
            : "memory");
    else
        tma_load_3d(dst, m, bar, x, y, z);
}
// arrives on this CTA's barrier alone
template <int CG>
__device__ __forceinline__ void l_commit_here(uint32_t bar)
{
    if (CG == 2)
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
                     : "memory");
    else
        mma_commit(bar);
}
// the address of `bar` in the pair's first CTA
template <int CG>
__device__ __forceinline__ uint32_t l_leader(uint32_t bar)
{
    if (CG == 1) return bar;
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(bar));
    return r;
}
template <int CG>
__device__ __forceinline__ void l_arrive_leader(uint32_t bar)
{
    if (CG == 2)
        asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(l_leader<CG>(bar)) : "memory");
    else
        asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
template <int CG>
__device__ __forceinline__ void l_cluster_sync()
{
    if (CG == 2) {
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
}
__device__ __forceinline__ void l_reduce_3d(const void *tmap, uint32_t src, int x, int y, int z)
{
    asm volatile(
        "cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
            reinterpret_cast<uint64_t>(tmap)),
        "r"(src), "r"(x), "r"(y), "r"(z)
        : "memory");
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&h);
}
// the leading 8 bits of x's significand (x - top_part(x) is exact)
__device__ __forceinline__ float top_part(float x) { return __bfloat162float(__float2bfloat16(x)); }
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void st_shared(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void st_shared32(uint32_t at, float x)
{
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(x) : "memory");
}
__device__ __forceinline__ void st_shared16(uint32_t at, float x)
{
    asm volatile("st.shared.b16 [%0], %1;" ::"r"(at), "h"(__bfloat16_as_ushort(__float2bfloat16(x))) : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// pairs of fp32 in one instruction
__device__ __forceinline__ uint64_t pair(float lo, float hi)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t x, float &lo, float &hi)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max32(const float (&v)[32], float m)
{
    float a[11];
#pragma unroll
    for (int j = 0; j < 10; ++j) a[j] = max3(v[3 * j], v[3 * j + 1], v[3 * j + 2]);
    a[10] = max3(v[30], v[31], m);
    const float x = max3(a[0], a[1], a[2]), y = max3(a[3], a[4], a[5]), z = max3(a[6], a[7], a[8]);
    return max3(max3(x, y, z), a[9], a[10]);
}

// 32 columns of a warp's 32 TMEM lanes; nothing reads v before l_tmem_wait(v)
__device__ __forceinline__ void l_tmem_issue(uint32_t taddr, float (&v)[32])
{
    uint32_t *r = reinterpret_cast<uint32_t *>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}
// The same 32 lanes x 32 columns as 8 x 8 blocks spread over the warp (the
// 16x256b shape): thread l holds rows l / 4 + 8 r and columns 8 i + 2 (l % 4)
// + e in v[16 (r / 2) + 4 i + 2 (r % 2) + e], r, i < 4.
__device__ __forceinline__ void l_tmem_issue_blocks(uint32_t taddr, float (&v)[32])
{
    uint32_t *r = reinterpret_cast<uint32_t *>(v);
#pragma unroll
    for (int h = 0; h < 2; ++h)
        asm volatile(
            "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
            "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
            : "=r"(r[16 * h + 0]), "=r"(r[16 * h + 1]), "=r"(r[16 * h + 2]), "=r"(r[16 * h + 3]), "=r"(r[16 * h + 4]),
              "=r"(r[16 * h + 5]), "=r"(r[16 * h + 6]), "=r"(r[16 * h + 7]), "=r"(r[16 * h + 8]), "=r"(r[16 * h + 9]),
              "=r"(r[16 * h + 10]), "=r"(r[16 * h + 11]), "=r"(r[16 * h + 12]), "=r"(r[16 * h + 13]),
              "=r"(r[16 * h + 14]), "=r"(r[16 * h + 15])
            : "r"(taddr + ((uint32_t)(16 * h) << 16))
            : "memory");
}
// four 8 x 8 blocks of bf16 to shared memory; thread l addresses row l % 8 of block l / 8
__device__ __forceinline__ void st_blocks(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c),
                 "r"(d)
                 : "memory");
}
__device__ __forceinline__ void l_tmem_wait(float (&v)[32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                   "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]),
                   "+f"(v[15]), "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]),
                   "+f"(v[22]), "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27])
                 :
                 : "memory");
    asm volatile("" : "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31])::"memory");
}

// ------------------------------------------------------------------- items
struct LItem {
    int m0, nt0, nt1, ks0, ks1, split, strip;
    int job, M, N, n0, bn, a_mn, b_mn, f32, add, out_t;
};
// The i-th item of tile slot c0 of G, or -1.  Items go round the slots; where
// job 0's do not come out even, the slots left without one (r .. G-1) take
// job 1's first items until the others are done.
template <int MODE>
__device__ __forceinline__ int l_next(const LParams &p, int c0, int G, int i)
{
    if (MODE != MODE_CT) {
        const long item = c0 + (long)i * G;
        return item < p.items ? (int)item : -1;
    }
    const int n0 = p.job[0].items, r = n0 % G, mine = n0 / G + (c0 < r);
    if (i < mine) return c0 + i * G;
    i -= mine;
    long x;
    if (c0 >= r)
        x = i < p.ahead ? (long)i * (G - r) + (c0 - r) : (long)p.ahead * (G - r) + (long)(i - p.ahead) * G + (c0 - r);
    else
        x = (long)p.ahead * (G - r) + (long)i * G + (G - r) + c0;
    return x < p.job[1].items ? (int)(n0 + x) : -1;
}
template <int CG, int MODE>
__device__ __forceinline__ LItem l_item(const LParams &p, int item)
{
    LItem t;
    if (MODE == MODE_CT) {
        t.job = item >= p.job[0].items;
        const LJob &j = t.job ? p.job[1] : p.job[0];
        if (t.job) item -= p.job[0].items;
        const int n = item % j.tiles_n, x = item / j.tiles_n;
        t.m0 = (x % j.tiles_m) * 128 * CG;
        t.split = x / j.tiles_m;
        t.nt0 = n;
        t.nt1 = n + 1;
        t.ks0 = (int)((long)t.split * j.ksteps / j.splits);
        t.ks1 = (int)((long)(t.split + 1) * j.ksteps / j.splits);
        if (t.ks0 == t.ks1) t.nt1 = t.nt0;   // nothing to add
        t.strip = 0;
        t.M = j.M;
        t.N = j.N;
        t.n0 = n * j.bn;
        t.bn = n + 1 < j.tiles_n ? j.bn : j.bn_last;
        t.a_mn = j.a_mn;
        t.b_mn = j.b_mn;
        t.out_t = j.out_t;
        t.f32 = j.f32;
        t.add = j.add;
    } else {
        // row blocks fastest: neighbours read the same vocabulary tiles at the same time
        t.m0 = (item % p.tiles_m) * 128 * CG;
        t.strip = item / p.tiles_m;
        t.nt0 = t.strip * p.strip;
        t.nt1 = t.nt0 + p.strip < p.tiles_n ? t.nt0 + p.strip : p.tiles_n;
        t.ks0 = 0;
        t.ks1 = p.ksteps;
        t.split = t.job = t.a_mn = t.b_mn = t.f32 = t.add = t.out_t = 0;
        t.M = p.M;
        t.N = p.N;
        t.n0 = t.nt0 * p.bn;
        t.bn = p.bn;
    }
    return t;
}

// A row's listed columns of one parity of 64-column chunks (an epilogue group
// works on one) in ascending order, the next two held in registers.
struct Cursor {
    const int *col;
    const float *p;
    int K, pos, c0, c1;
    float p0, p1;
    __device__ __forceinline__ void load(int at, int &c, float &w) const
    {
        const bool in = at < K;
        c = in ? col[at] : kNoColumn;
        w = in && p ? p[at] : 0.f;
    }
    // the row's first entry of a column >= from
    __device__ __forceinline__ void seek(const LossRows &r, long row, bool live, bool weights, int from, int half)
    {
        K = 0;
        pos = 0;
        c0 = c1 = kNoColumn;
        p0 = 1.f;
        if (!live) return;
        if (r.target) {
            const int y = target_column(r, row);
            if (y >= from && ((y >> 6) & 1) == half) c0 = y;
            return;
        }
        col = r.col + row * r.K;
        p = weights ? r.p + row * r.K : nullptr;
        const int even = r.even[row];
        K = half ? r.K : even;   // the end of this parity's entries
        // seven probes at once: the search waits for memory, not for instructions
        // (16384 x 512 x 65536 with 64 listed per row, both directions 3252 -> 3107 us)
        int lo = half ? even : 0, hi = K;
        while (lo < hi) {
            const int base = lo, end = hi, step = (end - base + 7) >> 3;
            int c[7];
#pragma unroll
            for (int x = 0; x < 7; ++x) {
                const int mid = base + (x + 1) * step - 1;
                c[x] = mid < end ? col[mid] : kNoColumn;
            }
#pragma unroll
            for (int x = 0; x < 7; ++x) {
                const int mid = base + (x + 1) * step - 1;
                if (c[x] < from)
                    lo = mid + 1;
                else if (mid < hi)
                    hi = mid;
            }
        }
        pos = lo;
        load(pos, c0, p0);
        load(pos + 1, c1, p1);
    }
    __device__ __forceinline__ void next()
    {
        ++pos;
        c0 = c1;
        p0 = p1;
        load(pos + 1, c1, p1);
    }
};

template <int CG, int MODE, bool kParts, bool kBias>
__global__ void __launch_bounds__(LNT, 1)
loss_product_kernel(const __grid_constant__ LMaps maps, const __grid_constant__ LParams p)
{
    using S = LSmem<CG, MODE, kParts>;
    constexpr int kDzParts = kParts ? 3 : CG == 1 ? 2 : 1;      // dz_parts()
    constexpr int ST = S::ST;
    loss_kernel_begin();
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = CG == 2 ? (int)(blockIdx.x & 1) : 0;
    const uint32_t sbase = smem_u32(smem);
    auto bar = [&](int i) { return sbase + S::BARS + 8u * (uint32_t)i; };
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(smem + S::MISC);
    volatile int *abort = reinterpret_cast<volatile int *>(smem + S::MISC + 8);
    // bounded wait; gives up when another role has given up
    auto wait = [&](int i, uint32_t parity) -> bool {
        const uint32_t b = bar(i);
        if (mbar_try_wait(b, parity)) return true;
        const uint64_t t0 = globaltimer_ns();
        while (true) {
            if (mbar_try_wait_sleep(b, parity, WAIT_SLEEP_NS)) return true;
            if (*abort) return false;
            if (globaltimer_ns() - t0 > LWAIT_NS) {
                *abort = 1;
                atomicOr(&g_loss_err, 1u);
                return false;
            }
        }
    };

    if (warp == 1) l_alloc<CG>(smem_u32(tmem_holder));
    if (tid == 0) {
        *abort = 0;
        for (int s = 0; s < ST; ++s) {
            mbar_init(bar(S::FULL + s), 1);
            mbar_init(bar(S::EMPTY + s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar(S::AFULL + b), 1);
            mbar_init(bar(S::AEMPTY + b), LEPI * CG);
        }
        mbar_init(bar(S::DONE), 1);
        for (int x = 0; MODE == MODE_LSE && x < 4; ++x) {
            mbar_init(bar(S::JFULL + x), 1);
            mbar_init(bar(S::JEMPTY + x), 1);
        }
        fence_mbar_init();
        for (int j = 0; j < (MODE == MODE_CT && p.job[1].items ? 2 : 1); ++j) {
            prefetch_tmap(&maps.a[j]);
            prefetch_tmap(&maps.b[j]);
            if (MODE != MODE_LSE) prefetch_tmap(&maps.o[j]);
        }
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    l_cluster_sync<CG>();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    loss_kernel_wait();
    const int G = (int)gridDim.x / CG, c0 = (int)blockIdx.x / CG;

    if (warp == 0) {
        // =================================================================== TMA producer
        if (lane == 0) {
            int it = 0;
            bool ok = true;
            for (int i = 0, item; ok && (item = l_next<MODE>(p, c0, G, i)) >= 0; ++i) {
                const LItem t = l_item<CG, MODE>(p, item);
                const CUtensorMap *ma = &maps.a[t.job], *mb = &maps.b[t.job];
                const int bcols = t.bn / CG;                          // this CTA's columns of B
                const int nb = (bcols + 63) / 64;                     // MN-major B: blocks of 64 columns
                // K-major B: a box as high as the widest tile's share, whatever this tile uses of it
                const int box = (MODE == MODE_CT ? (t.job ? p.job[1].bn : p.job[0].bn) : p.bn) / CG;
                const int a_box = MODE == MODE_CT ? (t.job ? p.job[1].a_box : p.job[0].a_box) : p.a_box;
                const uint32_t bytes = ((uint32_t)a_box * 128u + (t.b_mn ? (uint32_t)nb * 8192u : (uint32_t)box * 128u)) * CG;
                const int m0 = t.m0 + rank * 128;
                for (int nt = t.nt0; ok && nt < t.nt1; ++nt) {
                    const int n0 = t.n0 + (nt - t.nt0) * t.bn + rank * bcols;
                    for (int ks = t.ks0; ok && ks < t.ks1; ++ks) {
                        for (int part = 0; part < (kParts ? 3 : 1); ++part, ++it) {
                            const int s = it % ST;
                            if (it >= ST && !wait(S::EMPTY + s, ((it / ST) - 1) & 1)) {
                                ok = false;
                                break;
                            }
                            const uint32_t da = sbase + S::A + s * S::ASZ, db = sbase + S::B + s * S::BSZ;
                            const uint32_t full = l_leader<CG>(bar(S::FULL + s));
                            if (rank == 0) mbar_arrive_expect_tx(bar(S::FULL + s), bytes);
                            if (t.a_mn) {
                                l_load<CG>(da, ma, full, m0, ks * LK, part);
                                l_load<CG>(da + 8192u, ma, full, m0 + 64, ks * LK, part);
                            } else {
                                l_load<CG>(da, ma, full, ks * LK, m0, part);
                            }
                            if (t.b_mn) {
                                for (int b = 0; b < nb; ++b)
                                    l_load<CG>(db + 8192u * b, mb, full, n0 + 64 * b, ks * LK, part);
                            } else {
                                l_load<CG>(db, mb, full, ks * LK, n0, part);
                            }
                        }
                    }
                }
            }
            // the last stages' releases arrive here (from the pair's first CTA) before this CTA leaves
            for (int x = it > ST ? it - ST : 0; ok && x < it; ++x) ok = wait(S::EMPTY + x % ST, (x / ST) & 1);
            // after a wait that gave up: the copies still in flight land before the CTA leaves
            if (!ok && rank == 0)
                for (int x = it > ST ? it - ST : 0; x < it; ++x) {
                    const uint64_t t0 = globaltimer_ns();
                    while (!mbar_try_wait_sleep(bar(S::FULL + x % ST), (x / ST) & 1, WAIT_SLEEP_NS) &&
                           globaltimer_ns() - t0 < LWAIT_NS) {
                    }
                }
        }
        __syncwarp();
    } else if (warp == 1) {
        // =================================================================== MMA issuer
        if (lane == 0 && rank == 0) {
            int it = 0, lt = 0;
            bool ok = true;
            for (int i = 0, item; ok && (item = l_next<MODE>(p, c0, G, i)) >= 0; ++i) {
                const LItem t = l_item<CG, MODE>(p, item);
                const uint32_t idesc = idesc_bf16(128 * CG, t.bn, t.a_mn, t.b_mn);
                // K-major: K steps of 32 bytes along the swizzled row; MN-major:
                // K steps of 16 rows (2 KB), blocks of 64 outputs 8 KB apart
                const uint64_t da0 = smem_desc_sw128(sbase + S::A, t.a_mn ? 8192 : 16, 1024);
                const uint64_t db0 = smem_desc_sw128(sbase + S::B, t.b_mn ? 8192 : 16, 1024);
                const uint64_t sa = t.a_mn ? 128 : 2, sb = t.b_mn ? 128 : 2;
                for (int nt = t.nt0; ok && nt < t.nt1; ++nt) {
                    for (int ks = t.ks0; ok && ks < t.ks1; ++lt) {
                        // one accumulation: the whole K range, or some steps of three parts
                        const int buf = lt & 1, k1 = kParts && ks + kPartSteps < t.ks1 ? ks + kPartSteps : t.ks1;
                        if (lt >= 2 && !wait(S::AEMPTY + buf, ((lt >> 1) - 1) & 1)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t acc = tmem + (uint32_t)(buf * 256);
                        uint32_t more = 0u;
                        for (; ok && ks < k1; ++ks) {
                            constexpr int kStages = kParts ? 3 : 1;
                            uint64_t da[kStages], db[kStages];
#pragma unroll
                            for (int part = 0; part < kStages; ++part) {
                                const int s = (it + part) % ST;
                                if (ok && !wait(S::FULL + s, ((it + part) / ST) & 1)) ok = false;
                                da[part] = da0 + ((uint64_t)(s * S::ASZ) >> 4);
                                db[part] = db0 + ((uint64_t)(s * S::BSZ) >> 4);
                            }
                            if (!ok) break;
                            tc_fence_after();
#pragma unroll
                            for (int x = kParts ? 0 : 5; x < 6; ++x) {
                                constexpr int pa[6] = {2, 1, 0, 1, 0, 0}, pb[6] = {0, 1, 2, 0, 1, 0};
#pragma unroll
                                for (int k = 0; k < LK / 16; ++k) {
                                    l_mma<CG>(acc, da[pa[x]] + sa * k, db[pb[x]] + sb * k, idesc, more);
                                    more = 1u;
                                }
                            }
#pragma unroll
                            for (int part = 0; part < kStages; ++part, ++it) l_commit<CG>(bar(S::EMPTY + it % ST));
                        }
                        if (ok) l_commit<CG>(bar(S::AFULL + buf));
                    }
                }
            }
            // every MMA issued here has completed before the pair winds down
            l_commit_here<CG>(bar(S::DONE));
            wait(S::DONE, 0);
        }
        __syncwarp();
    } else if (warp >= 4) {
        // =================================================================== epilogue
        const int q = warp & 3, half = (warp - 4) >> 2;
        // staging: STG buffers of 32 rows x 128 bytes per warp, used in turn
        const uint32_t stg0 = sbase + S::OST + (uint32_t)(warp - 4) * 4096u;
        uint32_t stg_a = stg0;
        int nst = 0;
        int lt = 0;
        bool ok = true;
        // the next staging buffer, once the store that last used it has read it (every use of one
        // is followed by a store of its own)
        auto stage_wait = [&]() {
            if (S::STG == 2) {
                stg_a = stg0 + ((nst++ & 1) ? LEPI * 4096u : 0u);
                if (lane == 0) bulk_wait_read_1();
            } else if (lane == 0) {
                bulk_wait_read();
            }
            __syncwarp();
        };
        auto stage_bf16 = [&](const float (&v)[32], int at) {      // columns 32 at .. 32 at + 31 of the row
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                st_shared(stg_a + lane * 128 + (((4 * at + j) ^ (lane & 7)) << 4), pack2(v[8 * j + 0], v[8 * j + 1]),
                          pack2(v[8 * j + 2], v[8 * j + 3]), pack2(v[8 * j + 4], v[8 * j + 5]),
                          pack2(v[8 * j + 6], v[8 * j + 7]));
            }
        };
        auto store = [&](int job, int x, int y, int z, bool add) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                if (add)
                    l_reduce_3d(&maps.o[job], stg_a, x, y, z);
                else
                    tma_store_3d(&maps.o[job], stg_a, x, y, z);
                bulk_commit();
            }
        };
        auto release = [&](int buf) {      // this warp's part of the accumulator is in registers
            tc_fence_before();
            __syncwarp();
            if (lane == 0) l_arrive_leader<CG>(bar(S::AEMPTY + buf));
        };
        const uint64_t alpha2 = pair(p.alpha, p.alpha);
        for (int i = 0, item; ok && (item = l_next<MODE>(p, c0, G, i)) >= 0; ++i) {
            const LItem t = l_item<CG, MODE>(p, item);
            const int row0 = t.m0 + rank * 128 + 32 * q, row = row0 + lane;
            const bool live = row < t.M;
            const int nch = t.bn / 64;                                // 64-column chunks, alternately per half
            float m = -INFINITY, l = 0.f, coef = 0.f, l2 = 0.f;
            Cursor cur;
            bool dead = false;
            if (MODE != MODE_CT) {
                if (MODE == MODE_DZ && live) {
                    // (a list's valid entries come first)
                    const bool any = (p.r.target ? target_column(p.r, row) : p.r.col[(long)row * p.r.K]) != kNoColumn;
                    coef = row_factor(p.r, row, any);
                    l2 = p.r.lse[row] * (1.f / kLn2);
                }
                cur.seek(p.r, row, live, MODE == MODE_DZ, p.v0 + t.n0, half);
                if (MODE == MODE_DZ) dead = __any_sync(0xffffffffu, coef == 0.f);
            }
            // dz: a thread's four rows of the 8 x 8 blocks
            float bc[4], bl[4];
            if (MODE == MODE_DZ) {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    bc[r] = __shfl_sync(0xffffffffu, coef, (lane >> 2) + 8 * r);
                    bl[r] = __shfl_sync(0xffffffffu, l2, (lane >> 2) + 8 * r);
                }
            }
            auto process_dz = [&](float (&v)[32], const float2 (&bias)[4], int n0, int sub) {
                // a warp without rows stages nothing: a staging buffer is taken again by counting
                // the stores since, and it makes none
                if (n0 >= p.N || row0 >= p.M) return;
                const int col0 = p.v0 + n0, c2 = 2 * (lane & 3);   // columns n0 + 8 i + c2 + {0, 1}
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint64_t b2 = pair(bias[i].x, bias[i].y);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        float &x = v[16 * (r >> 1) + 4 * i + 2 * (r & 1)], &y = v[16 * (r >> 1) + 4 * i + 2 * (r & 1) + 1];
                        const uint64_t off = pair(-bl[r], -bl[r]);
                        float a, b;
                        unpair(fma2(kBias ? add2(pair(x, y), b2) : pair(x, y), alpha2, off), a, b);
                        unpair(mul2(pair(ex2(a), ex2(b)), pair(bc[r], bc[r])), x, y);
                    }
                }
                if (dead) {   // whatever an empty row holds
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (bc[r] == 0.f) {
#pragma unroll
                            for (int x = 0; x < 8; ++x) v[16 * (r >> 1) + 4 * (x >> 1) + 2 * (r & 1) + (x & 1)] = 0.f;
                        }
                }
                if (n0 + 32 > p.N) {   // columns past the vocabulary
#pragma unroll
                    for (int x = 0; x < 32; ++x)
                        if (n0 + 8 * ((x >> 2) & 3) + c2 + (x & 1) >= p.N) v[x] = 0.f;
                }
                // listed columns: every row's next one at once; a thread asks the
                // four lanes that follow its rows' lists
                while (const unsigned rows = __ballot_sync(0xffffffffu, cur.c0 < col0 + 32)) {
                    const bool hit = cur.c0 < col0 + 32;
                    const int mc = hit ? cur.c0 - col0 : 64;
                    const float mine = hit && coef != 0.f ? -coef * cur.p0 : 0.f;
                    if (hit) cur.next();
                    __syncwarp();
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        if (((rows >> (8 * r)) & 0xffu) == 0) continue;
                        const int c = __shfl_sync(0xffffffffu, mc, (lane >> 2) + 8 * r);
                        const float g = __shfl_sync(0xffffffffu, mine, (lane >> 2) + 8 * r);
                        const int at = ((c >> 1) & 3) == (lane & 3) ? c >> 3 : 8;
                        const uint64_t g2 = pair(c & 1 ? 0.f : g, c & 1 ? g : 0.f);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int e = 16 * (r >> 1) + 4 * i + 2 * (r & 1);
                            if (at == i) unpair(add2(pair(v[e], v[e + 1]), g2), v[e], v[e + 1]);
                        }
                    }
                }
                if (p.dbpart) {
                    // column sums over the warp's 32 rows: 4 in the thread, 8 by halving exchanges
                    // over the threads of a column, which leave one column in each thread
                    float s[8];
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        const int at = 4 * (x >> 1) + (x & 1);
                        s[x] = (v[at] + v[at + 2]) + (v[at + 16] + v[at + 18]);
                    }
#pragma unroll
                    for (int o = 4; o; o >>= 1) {
                        const bool up = lane & (4 * o);
#pragma unroll
                        for (int x = 0; x < o; ++x) {
                            const float send = up ? s[x] : s[x + o], keep = up ? s[x + o] : s[x];
                            s[x] = keep + __shfl_xor_sync(0xffffffffu, send, 4 * o);
                        }
                    }
                    // (columns past the last one lie in the row's padding)
                    p.dbpart[(long)(row0 >> 5) * p.dbpitch + n0 + 8 * (lane >> 3) + c2 + ((lane >> 2) & 1)] = s[0];
                }
#pragma unroll
                for (int part = 0; part < kDzParts; ++part) {
                    if (kDzParts > 1 || sub == 0) stage_wait();
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        uint32_t w4[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float &a = v[16 * (r >> 1) + 4 * i + 2 * (r & 1)], &b = v[16 * (r >> 1) + 4 * i + 2 * (r & 1) + 1];
                            w4[i] = pack2(a, b);
                            if (part + 1 < kDzParts) {
                                a -= top_part(a);
                                b -= top_part(b);
                            }
                        }
                        // rows of 128 bytes (64 per part of several) and their swizzles
                        const int y = 8 * r + (lane & 7), i = lane >> 3;
                        st_blocks(kDzParts > 1 ? stg_a + y * 64 + ((i ^ ((y >> 1) & 3)) << 4)
                                               : stg_a + y * 128 + (((4 * sub + i) ^ (y & 7)) << 4),
                                  w4[0], w4[1], w4[2], w4[3]);
                    }
                    if (kDzParts > 1) {
                        store(0, n0, row0, part, false);
                    } else if (sub == 1 || n0 + 32 >= p.N) {
                        // the second half of the chunk may lie past the last column
                        store(0, n0 - 32 * sub, row0, 0, false);
                    }
                }
            };
            // the staging buffer to rows that TMA stores cannot address: `high` rows of `wide` bytes
            // (128 swizzled, else as they are), to row y and column x on, within `cols` columns
            auto store_rows = [&](int x, int y, int high, int wide, int rows, int cols) {
                const LJob &j = t.job ? p.job[1] : p.job[0];
                const int esz = t.f32 ? 4 : 2, words = wide / 4, per = 32 / words;
                __syncwarp();
                for (int r0 = 0; r0 < high; r0 += per) {
                    const int r = r0 + lane / words, w = lane % words;
                    const bool sw = !t.out_t && wide == 128;
                    const uint32_t at = stg_a + r * wide + (sw ? (((w >> 2) ^ (r & 7)) << 4) + (w & 3) * 4 : w * 4);
                    uint32_t v;
                    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
                    if (y + r >= rows) continue;
                    unsigned char *row = static_cast<unsigned char *>(j.out) + ((long)(y + r) * j.pitch + x) * esz;
                    if (t.f32) {
                        if (x + w < cols) reinterpret_cast<uint32_t *>(row)[w] = v;
                    } else if (((j.pitch | (long)reinterpret_cast<uintptr_t>(j.out) / 2) & 1) == 0 && x + 2 * w + 1 < cols) {
                        reinterpret_cast<uint32_t *>(row)[w] = v;
                    } else {
                        if (x + 2 * w < cols) reinterpret_cast<uint16_t *>(row)[2 * w] = (uint16_t)v;
                        if (x + 2 * w + 1 < cols) reinterpret_cast<uint16_t *>(row)[2 * w + 1] = (uint16_t)(v >> 16);
                    }
                }
                __syncwarp();
            };
            const bool by_tma = MODE != MODE_CT || (t.job ? p.job[1].out : p.job[0].out) == nullptr;
            // 32 columns from n0 on (the second half of their 64-column chunk with sub = 1)
            auto process = [&](float (&v)[32], int n0, int sub) {
                if (MODE == MODE_CT) {
                    if (row0 >= t.M || n0 - 32 * sub >= t.N) return;
                    if (t.out_t) {
                        // lanes are columns of the output, v its rows
                        if (t.f32) {
                            if (n0 >= t.N) return;
                            stage_wait();
#pragma unroll
                            for (int j = 0; j < 32; ++j) st_shared32(stg_a + 128 * j + 4 * lane, v[j]);
                            if (by_tma)
                                store(t.job, row0, n0, t.split, t.add);
                            else
                                store_rows(row0, n0, 32, 128, t.N, t.M);
                        } else {
                            if (sub == 0) stage_wait();
#pragma unroll
                            for (int j = 0; j < 32; ++j) st_shared16(stg_a + 64 * (32 * sub + j) + 2 * lane, v[j]);
                            if (sub == 1) {
                                if (by_tma)
                                    store(t.job, row0, n0 - 32, 0, false);
                                else
                                    store_rows(row0, n0 - 32, 64, 64, t.N, t.M);
                            }
                        }
                        return;
                    }
                    if (t.f32) {
                        if (n0 >= t.N) return;
                        stage_wait();
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            st_shared(stg_a + lane * 128 + ((j ^ (lane & 7)) << 4), __float_as_uint(v[4 * j]),
                                      __float_as_uint(v[4 * j + 1]), __float_as_uint(v[4 * j + 2]),
                                      __float_as_uint(v[4 * j + 3]));
                        if (by_tma)
                            store(t.job, n0, row0, t.split, t.add);
                        else
                            store_rows(n0, row0, 32, 128, t.M, t.N);
                    } else {
                        if (sub == 0) stage_wait();
                        stage_bf16(v, sub);
                        if (sub == 1) {
                            if (by_tma)
                                store(t.job, n0 - 32, row0, 0, false);
                            else
                                store_rows(n0 - 32, row0, 32, 128, t.M, t.N);
                        }
                    }
                    return;
                }
                if (n0 >= p.N) return;
                const int col0 = p.v0 + n0;
                // logits; the running maximum is kept of these, unscaled
                if (kBias) {
                    if (n0 + 32 <= p.N) {
#pragma unroll
                        for (int j = 0; j < 32; j += 4) {
                            const float4 b4 = *reinterpret_cast<const float4 *>(p.bias + n0 + j);
                            unpair(add2(pair(v[j], v[j + 1]), pair(b4.x, b4.y)), v[j], v[j + 1]);
                            unpair(add2(pair(v[j + 2], v[j + 3]), pair(b4.z, b4.w)), v[j + 2], v[j + 3]);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (n0 + j < p.N) v[j] += p.bias[n0 + j];
                    }
                }
                if (n0 + 32 > p.N) {   // columns past the vocabulary
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (n0 + j >= p.N) v[j] = -INFINITY;
                }
                while (cur.c0 < col0 + 32) {
                    float y = 0.f;
#pragma unroll
                    for (int j = 0; j < 32; ++j) y = cur.c0 == col0 + j ? v[j] : y;
                    p.ysel[(long)row * p.r.K + cur.pos] = y * p.alpha;
                    cur.next();
                }
                __syncwarp();
                // (no reference of -infinity, nor one that scaling makes so: the type's lowest value)
                const float cm = max32(v, m), ref = cm * p.alpha == -INFINITY ? 0.f : cm;
                const uint64_t off = pair(-ref * p.alpha, -ref * p.alpha);
                uint64_t s[4] = {0, 0, 0, 0};
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    float a, b;
                    unpair(fma2(pair(v[2 * j], v[2 * j + 1]), alpha2, off), a, b);
                    s[j & 3] = add2(s[j & 3], pair(ex2(a), ex2(b)));
                }
                float a, b;
                unpair(add2(add2(s[0], s[1]), add2(s[2], s[3])), a, b);
                l = fmaf(l, ex2((m - ref) * p.alpha), a + b);
                m = cm;
            };
            auto issue = [&](uint32_t taddr, float (&v)[32]) {
                if (MODE == MODE_DZ)
                    l_tmem_issue_blocks(taddr, v);
                else
                    l_tmem_issue(taddr, v);
            };
            // dz: the biases of a thread's columns, asked for ahead of their use
            auto biases = [&](float2 (&b)[4], int n0) {
                if constexpr (MODE == MODE_DZ && kBias) {
                    const float2 *at = reinterpret_cast<const float2 *>(p.bias + n0 + 2 * (lane & 3));
                    if (n0 + 32 <= p.N) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) b[i] = at[4 * i];
                        return;
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int n = n0 + 8 * i + 2 * (lane & 3);
                        b[i] = n + 1 < p.N ? *reinterpret_cast<const float2 *>(p.bias + n)
                                           : make_float2(n < p.N ? p.bias[n] : 0.f, 0.f);
                    }
                }
            };
            auto work = [&](float (&v)[32], const float2 (&b)[4], int n0, int sub) {
                if (MODE == MODE_DZ)
                    process_dz(v, b, n0, sub);
                else
                    process(v, n0, sub);
            };
            const uint32_t tq = tmem + ((uint32_t)(32 * q) << 16);
            for (int nt = t.nt0; ok && nt < t.nt1; ++nt) {
                float v0[32], v1[32];
                float2 b0[4], b1[4];
                // the tile's columns, and the first of its chunks that is this group's (by its
                // parity in the vocabulary)
                const int first = t.n0 + (nt - t.nt0) * t.bn, mine = half ^ ((first >> 6) & 1);
                biases(b0, first + 64 * mine);
                if constexpr (kParts) {
                    // this half's 64 columns, summed over the steps
#pragma unroll
                    for (int j = 0; j < 32; ++j) v0[j] = v1[j] = 0.f;
                    for (int ks = t.ks0; ks < t.ks1; ks += kPartSteps, ++lt) {
                        if (!wait(S::AFULL + (lt & 1), (lt >> 1) & 1)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        if (mine < nch) {
                            const uint32_t at = tq + (uint32_t)((lt & 1) * 256 + 64 * mine);
                            float x[32];
                            issue(at, x);
                            l_tmem_wait(x);
#pragma unroll
                            for (int j = 0; j < 32; ++j) v0[j] += x[j];
                            issue(at + 32u, x);
                            l_tmem_wait(x);
#pragma unroll
                            for (int j = 0; j < 32; ++j) v1[j] += x[j];
                        }
                        release(lt & 1);
                    }
                    if (!ok) break;
                    if (mine < nch) {
                        biases(b1, first + 64 * mine + 32);
                        work(v0, b0, first + 64 * mine, 0);
                        work(v1, b1, first + 64 * mine + 32, 1);
                    }
                } else {
                    const int buf = lt & 1;
                    if (!wait(S::AFULL + buf, (lt >> 1) & 1)) {
                        ok = false;
                        break;
                    }
                    ++lt;
                    tc_fence_after();
                    if (MODE == MODE_LSE && kBias && nt + 1 < t.nt1 && 32 * lane < t.bn && (nt + 1) * t.bn + 32 * lane < t.N)   // the next tile's biases
                        asm volatile("prefetch.global.L1 [%0];" ::"l"(p.bias + (nt + 1) * t.bn + 32 * lane));
                    if (mine >= nch) {
                        release(buf);
                        continue;
                    }
                    // each load is in flight while the columns before it are worked on
                    const uint32_t tacc = tq + (uint32_t)(buf * 256);
                    issue(tacc + 64u * mine, v0);
                    l_tmem_wait(v0);
                    for (int c = mine; c < nch; c += 2) {
                        const int n0 = first + 64 * c;
                        issue(tacc + 64u * c + 32u, v1);
                        biases(b1, n0 + 32);
                        work(v0, b0, n0, 0);
                        l_tmem_wait(v1);
                        if (c + 2 < nch)
                            issue(tacc + 64u * (c + 2), v0);
                        else
                            release(buf);
                        if (c + 2 < nch) biases(b0, n0 + 128);
                        work(v1, b1, n0 + 32, 1);
                        if (c + 2 < nch) l_tmem_wait(v0);
                    }
                }
            }
            if (MODE == MODE_LSE && p.loss) {
                // the strip is the whole vocabulary: the second group's half of each row goes to the
                // first's warp for the same rows, which is done with the row then (no launch to join
                // them: 16896 x 512 x 256 forward 15.5 -> 11.0 us)
                float2 *join = reinterpret_cast<float2 *>(smem + S::JOIN) + 32 * q + lane;
                if (half) {
                    if (ok && i > 0) ok = wait(S::JEMPTY + q, (i - 1) & 1);
                    if (ok) {
                        *join = make_float2(m * p.alpha, l);
                        __syncwarp();
                        if (lane == 0) l_arrive(bar(S::JFULL + q));
                    }
                } else if (ok && (ok = wait(S::JFULL + q, i & 1))) {
                    const float2 e = *join;
                    __syncwarp();
                    if (lane == 0) l_arrive(bar(S::JEMPTY + q));
                    const float ms = m * p.alpha, top = fmaxf(ms, e.x), ref = top == -INFINITY ? 0.f : top;
                    const float y_lse = ref + log2f(l * exp2f(ms - ref) + e.y * exp2f(e.x - ref));
                    if (live) {
                        const bool any = target_column(p.r, row) != kNoColumn && y_lse != -INFINITY;
                        p.lse[row] = y_lse * kLn2;
                        p.loss[row] = any ? kLn2 * (y_lse - __ldcg(p.ysel + row)) : 0.f;
                    }
                }
            } else if (MODE == MODE_LSE && ok && live) {
                p.part[(long)(kSlotsPerStrip * t.strip + half) * p.M + row] = make_float2(m * p.alpha, l);
            }
        }
        if (lane == 0) bulk_wait_all();
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    l_cluster_sync<CG>();
    if (warp == 1) {
        tc_fence_after();
        l_dealloc<CG>(tmem);
    }
}

// ------------------------------------------------------------------ host side
PFN_cuTensorMapEncodeTiled_v12000 l_encode_fn()
{
    static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> found{nullptr};
    PFN_cuTensorMapEncodeTiled_v12000 fn = found.load(std::memory_order_relaxed);
    if (!fn) {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            found.store(fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr), std::memory_order_relaxed);
    }
    return fn;
}

cudaError_t l_map(CUtensorMap *m, CUtensorMapDataType type, int esz, const void *base, long cols, long rows,
                  long depth, long pitch, long depth_stride, int box_x, int box_y, CUtensorMapSwizzle swizzle)
{
    auto enc = l_encode_fn();
    if (!enc) return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)depth};
    const cuuint64_t strides[2] = {(cuuint64_t)(pitch * esz), (cuuint64_t)(depth > 1 ? depth_stride * esz : pitch * esz)};
    const cuuint32_t box[3] = {(cuuint32_t)box_x, (cuuint32_t)box_y, 1}, estr[3] = {1, 1, 1};
    return enc(m, type, 3, const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}
cudaError_t l_in_map(CUtensorMap *m, const LossMatrix &x, int box_y)
{
    return l_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, x.base, x.cols, x.rows, x.pieces, x.pitch, x.piece_stride, LK,
                 box_y, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int CG, int MODE, bool kParts, bool kBias>
cudaError_t l_launch(const LMaps &maps, const LParams &p, cudaStream_t s)
{
    auto kern = loss_product_kernel<CG, MODE, kParts, kBias>;
    static std::atomic<int> most[64];      // tiles that run at once, per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorNotSupported;
    const size_t smem = LSmem<CG, MODE, kParts>::TOTAL;
    int n = most[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        n = device_sm_count() / CG;
        if (CG == 2) {
            // an odd SM of a GPC takes no pair
            cudaLaunchAttribute at[1];
            at[0].id = cudaLaunchAttributeClusterDimension;
            at[0].val.clusterDim.x = CG;
            at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3((unsigned)(CG * n));
            cfg.blockDim = dim3(LNT);
            cfg.dynamicSmemBytes = smem;
            cfg.attrs = at;
            cfg.numAttrs = 1;
            int fit = 0;
            e = cudaOccupancyMaxActiveClusters(&fit, kern, &cfg);
            if (e != cudaSuccess) return e;
            if (fit > 0 && fit < n) n = fit;
        }
        most[dev].store(n, std::memory_order_relaxed);
    }
    g_loss_ran.store(true, std::memory_order_relaxed);
    return loss_launch(kern, (unsigned)(CG * (p.items < n ? p.items : n)), LNT, smem, CG, s, maps, p);
}

template <int MODE, bool kBias>
cudaError_t l_launch_cg(int cg, int parts, const LMaps &maps, const LParams &p, cudaStream_t s)
{
    if (parts == 3)
        return cg == 2 ? l_launch<2, MODE, true, kBias>(maps, p, s) : l_launch<1, MODE, true, kBias>(maps, p, s);
    return cg == 2 ? l_launch<2, MODE, false, kBias>(maps, p, s) : l_launch<1, MODE, false, kBias>(maps, p, s);
}

long cdiv(long a, long b) { return (a + b - 1) / b; }

// Rows of K-major A in a stage: those of a single tile that exist.  (What lies
// in the others' place reaches only rows of the accumulator that nobody reads.)
// 2 x 1024 x 131072 tokens, forward: 128 rows 65 us, 8 rows 52 us.
int a_box(int rows, int cg) { return cg == 1 && rows < 128 ? (int)(cdiv(rows, 8) * 8) : 128; }

// the fields the two vocabulary passes share
cudaError_t vocab_params(LParams &p, LMaps &maps, const LossMatrix &h, const LossMatrix &w, const float *bias, int v0,
                         float alpha, const LossRows &r, const LossTiling &t)
{
    memset(&p, 0, sizeof(p));
    p.M = h.rows;
    p.N = w.rows;
    p.bn = t.bn;
    p.tiles_m = t.tiles_m;
    p.tiles_n = t.tiles_n;
    p.strip = t.strip;
    const long items = (long)t.tiles_m * vocab_strips(t);
    if (items > INT32_MAX) return cudaErrorNotSupported;
    p.items = (int)items;
    p.ksteps = (int)cdiv(h.cols, LK);
    p.bias = bias;
    p.v0 = v0;
    p.alpha = alpha;
    p.r = r;
    p.a_box = a_box(h.rows, t.cg);
    cudaError_t e = l_in_map(&maps.a[0], h, p.a_box);
    if (e == cudaSuccess) e = l_in_map(&maps.b[0], w, t.bn / t.cg);
    return e;
}

// What the division rules below count with, measured on GB300 at 2 GHz: a
// 64-deep step of a 256-column tile (per SM 128 rows of it), what an item
// costs beside its steps, a vocabulary tile's epilogue, a launch with the
// drain before it, and HBM bytes per microsecond.
constexpr double kStepUs = 0.32, kItemUs = 1.0, kEpilogueUs = 2.4, kLaunchUs = 5.0, kHbmPerUs = 6.0e6;
constexpr double kMnB = 1.36;          // what an MN-major B takes longer
constexpr double kL2Bytes = 80e6;      // dz pieces up to this are read back from L2

double step_us(int bn, int parts) { return kStepUs * bn / 256 * (parts == 3 ? 6 : 1); }

// The longest of the tile slots when n0 items of a and n1 items of b go round
// them as l_next deals them out, with the best `ahead`.
double makespan(long slots, long n0, double a, long n1, double b, int *ahead)
{
    const long r = n0 % slots, q = n0 / slots;
    double best = 1e300;
    const long k0 = r ? (long)(a / b) : 0;
    for (long k = k0; k <= k0 + (r ? 1 : 0); ++k) {
        const long rest = n1 - k * (slots - r);                     // items dealt out to all
        const long late = rest > 0 ? cdiv(rest, slots) : 0;         // ... of them to the slots from r on
        const long early = rest > slots - r ? cdiv(rest - (slots - r), slots) : 0;
        const long kk = rest > 0 ? k : cdiv(n1, slots - r > 0 ? slots - r : 1);
        const double x = q * a + (kk + late) * b, y = r ? (q + 1) * a + early * b : 0.0;
        const double t = x > y ? x : y;
        if (t < best) {
            best = t;
            *ahead = (int)k;
        }
    }
    return best;
}

void job_tiles(LossTiling &t, int m, int n, int cg, int parts)
{
    t.cg = cg;
    t.tiles_m = (int)cdiv(m, 128 * cg);
    t.tiles_n = (int)cdiv(n, parts == 3 ? 128 : 256);
    const int widest = parts == 3 ? 128 : 256;
    t.bn = n >= widest ? widest : (int)(cdiv(n, 64) * 64);   // the last column tile may be narrower
    t.strip = 1;
    t.splits = 1;
    t.turned = t.first = false;
    t.ahead = 0;
}

}  // namespace

LossTiling vocab_tiling(int rows, int cols, int d, int parts, double *us)
{
    LossTiling t;
    t.cg = rows > 128 ? 2 : 1;
    t.tiles_m = (int)cdiv(rows, 128 * t.cg);
    t.splits = 1;
    t.turned = t.first = false;
    t.ahead = 0;
    // The widest tiles (narrower ones that would fill the last round of CTAs
    // better took longer: 2816 x 512 x 131072 in 192-wide tiles 321 us, in
    // 256-wide ones 272), in the strips that leave the last round fullest; of
    // equal ones the longest (fewest partial results).
    // Where even half as wide ones leave CTAs idle, those: every tile is then
    // a CTA's only one.
    const int widest = parts == 3 ? 128 : 256;
    const long slots = device_sm_count() / t.cg;
    t.bn = cols > widest - 64 ? widest : (int)(cdiv(cols, 64) * 64);
    while (t.bn >= 128 && t.bn % 128 == 0 && t.tiles_m * cdiv(cols, t.bn / 2) <= slots) t.bn /= 2;
    t.tiles_n = (int)cdiv(cols, t.bn);
    double best = 1e300;
    for (int s = 1; s <= t.tiles_n && s <= 64; ++s) {
        const double cost = (double)cdiv(t.tiles_m * cdiv(t.tiles_n, s), slots) * (s + 0.15);
        if (cost <= best) {
            best = cost;
            t.strip = s;
        }
    }
    if (t.tiles_m == 1) t.strip = 1;   // bound by reading the weights: every SM reads (2 x 768 x 90326: 36.7 -> 33.3 us)
    if (us) {
        const double main = cdiv(d, LK) * step_us(t.bn, parts), epi = kEpilogueUs * t.bn / 256;
        *us = best * (main > epi ? main : epi) + kLaunchUs;
    }
    return t;
}

double gradient_tiling(int rows, int d, int cols, int whole, int parts, bool dh_slots, int dh_splits, LossTiling *dh,
                       LossTiling *dw)
{
    const int cg = rows > 128 ? 2 : 1;
    // dh as the transpose of W^T dz^T unless that wastes more rows of its tiles
    // than an MN-major B costs, or reading the weights bounds it (few rows):
    // as B they come in twice the bytes per stage
    LossTiling turned;
    job_tiles(turned, d, rows, cg, parts);
    job_tiles(*dh, rows, d, cg, parts);
    turned.turned = true;
    if (cg == 2 && (double)turned.tiles_m * cdiv(rows, 64) <= kMnB * dh->tiles_m * cdiv(d, 64)) *dh = turned;
    job_tiles(*dw, cols, d, cg, parts);
    const long slots = device_sm_count() / cg;
    const long n0 = (long)dh->tiles_m * dh->tiles_n, n1 = (long)dw->tiles_m * dw->tiles_n;
    // a step of an average column tile
    auto wide = [](int n, const LossTiling &t) { return (int)(cdiv(n, 64) * 64 / t.tiles_n); };
    const double s0 = step_us(wide(dh->turned ? rows : d, *dh), parts) * (dh->turned ? 1.0 : kMnB);
    const double s1 = step_us(wide(d, *dw), parts);
    const long k0 = cdiv(cols, LK), k1 = cdiv(rows, LK), kw = cdiv(whole, LK);
    double best = 1e300;
    static const int cand[] = {1, 2, 3, 4, 5, 6, 8, 10, 12, 16, 20, 24, 32, 48, 64};
    for (int a : cand) {
        if (a > kw) break;
        if (dh_splits && a != dh_splits) continue;
        for (int b : cand) {
            if (b > k1) break;
            // a split costs a pass over its slot, written (added to) and read back
            int ahead;
            const double l0 = cdiv(k0, a) * s0 + kItemUs, l1 = cdiv(k1, b) * s1 + kItemUs;
            const bool w_first = l1 > l0;
            double us = w_first ? makespan(slots, n1 * b, l1, n0 * a, l0, &ahead)
                                : makespan(slots, n0 * a, l0, n1 * b, l1, &ahead);
            const double pass = (a > 1 || dh_slots ? 2.0 * a * rows * d * 4 : 0.0) + (b > 1 ? 2.0 * b * cols * d * 4 : 0.0);
            us += pass / kHbmPerUs + (b > 1 ? kLaunchUs : 0.0);
            if (us < best) {
                best = us;
                dh->splits = a;
                dw->splits = b;
                dh->first = !w_first;
                dw->first = w_first;
                dh->ahead = dw->ahead = ahead;
            }
        }
    }
    return best + kLaunchUs;
}

int gradient_piece(int rows, int d, int vocab, int parts, int most)
{
    if (vocab <= kLossPieceUnit) return vocab;
    const int n = dz_rows(rows, parts);
    int best_piece = 0;
    double best = 1e300;
    const long units = cdiv(vocab, kLossPieceUnit), least = cdiv(units, most / kLossPieceUnit);
    for (long x = least; x <= units && x < least + 12; ++x) {
        const long piece = cdiv(units, x) * kLossPieceUnit;
        const int cols = (int)(piece < vocab ? piece : vocab), last = vocab % cols;
        LossTiling a, b;
        auto cost = [&](int c) {
            double vus;
            vocab_tiling(rows, c, d, parts, &vus);
            const double dz = (double)n * c * 2 * parts, hbm = dz > kL2Bytes ? dz / kHbmPerUs : 0.0;
            const double g = gradient_tiling(n, d, c, cols, parts, cols < vocab || n != rows, 0, &a, &b);
            return (vus > hbm ? vus : hbm) + (g > 2 * hbm ? g : 2 * hbm);
        };
        const double us = vocab / cols * cost(cols) + (last ? cost(last) : 0.0);
        if (us < best || !best_piece) {
            best = us;
            best_piece = cols;
        }
    }
    return best_piece;
}

cudaError_t launch_loss_lse(const LossMatrix &h, const LossMatrix &w, const float *bias, int v0, float alpha,
                            const LossRows &r, float *ysel, float2 *part, float *loss, float *lse, const LossTiling &t, cudaStream_t s)
{
    LParams p;
    LMaps maps;
    memset(&maps, 0, sizeof(maps));
    cudaError_t e = vocab_params(p, maps, h, w, bias, v0, alpha, r, t);
    if (e != cudaSuccess) return e;
    p.ysel = ysel;
    p.part = part;
    p.loss = loss;
    p.lse = lse;
    return bias ? l_launch_cg<MODE_LSE, true>(t.cg, h.pieces, maps, p, s)
              : l_launch_cg<MODE_LSE, false>(t.cg, h.pieces, maps, p, s);
}

cudaError_t launch_loss_dz(const LossMatrix &h, const LossMatrix &w, const float *bias, int v0, float alpha,
                           const LossRows &r, const LossMatrix &dz, float *dbpart, const LossTiling &t,
                           cudaStream_t s)
{
    LParams p;
    LMaps maps;
    memset(&maps, 0, sizeof(maps));
    cudaError_t e = vocab_params(p, maps, h, w, bias, v0, alpha, r, t);
    if (e != cudaSuccess) return e;
    p.dbpart = dbpart;
    p.dbpitch = dz.pitch;
    const bool several = dz.pieces > 1;
    e = l_map(&maps.o[0], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, dz.base, dz.cols, dz.rows, dz.pieces, dz.pitch,
              dz.piece_stride, several ? 32 : 64, 32, several ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
    if (e != cudaSuccess) return e;
    return bias ? l_launch_cg<MODE_DZ, true>(t.cg, h.pieces, maps, p, s)
              : l_launch_cg<MODE_DZ, false>(t.cg, h.pieces, maps, p, s);
}

cudaError_t launch_loss_gradients(const LossContraction *jobs, int n, int parts, cudaStream_t s)
{
    LParams p;
    LMaps maps;
    memset(&p, 0, sizeof(p));
    memset(&maps, 0, sizeof(maps));
    long items = 0;
    for (int x = 0; x < n; ++x) {
        const LossContraction &c = jobs[x];
        LJob &j = p.job[x];
        j.M = c.m;
        j.N = c.n;
        j.bn = c.t.bn;
        j.bn_last = (int)(cdiv(c.n - (long)(c.t.tiles_n - 1) * c.t.bn, 64) * 64);
        j.tiles_m = c.t.tiles_m;
        j.tiles_n = c.t.tiles_n;
        j.ksteps = (int)cdiv(c.k, LK);
        j.splits = c.t.splits;
        j.a_mn = c.a_t;
        j.b_mn = !c.b_t;
        j.out_t = c.out_t;
        j.f32 = c.out.f32;
        j.add = c.out.add;
        const long mine = (long)j.tiles_m * j.tiles_n * j.splits;
        items += mine;
        if (items > INT32_MAX) return cudaErrorNotSupported;
        j.items = (int)mine;
        j.a_box = c.a_t ? 128 : a_box(c.m, c.t.cg);
        cudaError_t e = l_in_map(&maps.a[x], c.a, c.a_t ? 64 : j.a_box);
        if (e == cudaSuccess) e = l_in_map(&maps.b[x], c.b, c.b_t ? j.bn / c.t.cg : 64);
        if (!c.out.tma) {
            j.out = c.out.base;
            j.pitch = c.out.pitch;
        } else if (e == cudaSuccess)
            e = l_map(&maps.o[x], c.out.f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                      c.out.f32 ? 4 : 2, c.out.base, c.out_t ? c.m : c.n, c.out_t ? c.n : c.m, j.splits, c.out.pitch,
                      c.out.slot_stride, c.out.f32 || c.out_t ? 32 : 64, c.out_t && !c.out.f32 ? 64 : 32,
                      c.out_t ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B);
        if (e != cudaSuccess) return e;
    }
    p.items = (int)items;
    p.ahead = n == 2 ? jobs[0].t.ahead : 0;
    return l_launch_cg<MODE_CT, false>(jobs[0].t.cg, parts, maps, p, s);
}

cudaError_t read_and_clear_loss_error(unsigned int *word, cudaStream_t s)
{
    if (!g_loss_ran.load(std::memory_order_relaxed)) return cudaSuccess;
    return read_and_clear_word(g_loss_err, word, s);
}

}  // namespace txl

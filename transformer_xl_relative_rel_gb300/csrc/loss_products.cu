// loss_products.cu -- the output-layer losses' products on the tensor cores.
//
// Three passes share one persistent tcgen05 kernel, D = A B^T with fp32
// accumulators in TMEM and a different epilogue each:
//   lse       A = h, B = W: the running maximum and sum of the softmax over a
//             strip of vocabulary tiles, the logits themselves never stored;
//   dz        A = h, B = W: dz = coef (softmax - listed weights) of one
//             vocabulary piece, rounded to bf16 and stored;
//   contract  dh = dz W (A = dz, B = W^T) and dW = dz^T h (A = dz^T, B = h^T):
//             the transposed operands are read as they are stored
//             (MN-major tiles), nothing is transposed in memory.
// fp32 operands are held as three bf16 parts whose sum is exact (8 + 8 + 8
// bits of the 24-bit significand); the product keeps the six part products
// down to 2^-16 of the largest, dropping three of at most 2^-24, smallest
// first.  The tensor core truncates where it accumulates (measured: a chain
// of n additions comes out about n 2^-25 too small), so with fp32 operands an
// accumulator takes one 64-deep step and the epilogue warps add the steps in
// registers, rounding to nearest.
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

// bounded waits of the kernel below that gave up (read by txl_check)
__device__ unsigned int g_loss_err;

namespace {
using namespace sm100;

constexpr int LK = 64;                         // K elements per stage
constexpr int LNT = 384;
constexpr int LEPI = 8;                        // epilogue warps
constexpr uint64_t LWAIT_NS = 2000000000ull;   // 2 s per wait, then give up

// kParts: fp32 operands in three bf16 parts (128-wide tiles, one stage per
// part); else bf16 operands (256-wide tiles).
template <int CG, bool kParts>
struct LSmem {
    static constexpr int BN = kParts ? 128 : 256;           // widest tile
    static constexpr int ST = kParts ? (CG == 2 ? 8 : 6) : (CG == 2 ? 6 : 4);
    static constexpr uint32_t ASZ = 128 * 128;              // 128 rows of 64 elements
    static constexpr uint32_t BSZ = BN / CG * 128;
    static constexpr uint32_t A = 0, B = A + ST * ASZ, OST = B + ST * BSZ, BARS = OST + LEPI * 4096;
    static constexpr int FULL = 0, EMPTY = ST, AFULL = 2 * ST, AEMPTY = 2 * ST + 2, DONE = 2 * ST + 4,
                         NBAR = 2 * ST + 5;
    static constexpr uint32_t MISC = BARS + NBAR * 8 + 8;
    static constexpr uint32_t TOTAL = MISC + 16 + 1024;
};
static_assert(LSmem<1, false>::TOTAL <= 232448 && LSmem<2, false>::TOTAL <= 232448 &&
                  LSmem<1, true>::TOTAL <= 232448 && LSmem<2, true>::TOTAL <= 232448,
              "shared memory");

enum { MODE_LSE = 0, MODE_DZ = 1, MODE_CT = 2 };

struct LParams {
    int M, N;                 // output extent
    int bn, tiles_m, tiles_n, strip, strips, items;
    int ksteps, splits;
    int a_mn, b_mn;           // operands stored with the output index innermost
    // vocabulary passes
    const float *bz;          // [columns], biases in base-2 units; -infinity takes a column out
    int has_bz, v0;
    float alpha;
    LossRows r;
    float *ysel, *dbpart;
    float2 *part;
    long dbpitch;
    // contraction
    int f32, add;
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
};
template <int CG, int MODE>
__device__ __forceinline__ LItem l_item(const LParams &p, int item)
{
    LItem t;
    if (MODE == MODE_CT) {
        const int n = item % p.tiles_n, x = item / p.tiles_n;
        t.m0 = (x % p.tiles_m) * 128 * CG;
        t.split = x / p.tiles_m;
        t.nt0 = n;
        t.nt1 = n + 1;
        t.ks0 = (int)((long)t.split * p.ksteps / p.splits);
        t.ks1 = (int)((long)(t.split + 1) * p.ksteps / p.splits);
        if (t.ks0 == t.ks1) t.nt1 = t.nt0;   // nothing to add
        t.strip = 0;
    } else {
        // row blocks fastest: neighbours read the same vocabulary tiles at the same time
        t.m0 = (item % p.tiles_m) * 128 * CG;
        t.strip = item / p.tiles_m;
        t.nt0 = t.strip * p.strip;
        t.nt1 = t.nt0 + p.strip < p.tiles_n ? t.nt0 + p.strip : p.tiles_n;
        t.ks0 = 0;
        t.ks1 = p.ksteps;
        t.split = 0;
    }
    return t;
}

// A row's listed columns in ascending order, the next two held in registers.
struct Cursor {
    const int *col;
    const float *p;
    int K, pos, c0, c1;
    float p0, p1;
    __device__ __forceinline__ void load(int at, int &c, float &w) const
    {
        const bool in = at < K;
        c = in ? __ldg(col + at) : kNoColumn;
        w = in && p ? __ldg(p + at) : 0.f;
    }
    // the first entry of a column >= from
    __device__ __forceinline__ void seek(int from)
    {
        int lo = 0, hi = K;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (__ldg(col + mid) < from)
                lo = mid + 1;
            else
                hi = mid;
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

template <int CG, int MODE, bool kParts>
__global__ void __launch_bounds__(LNT, 1)
loss_product_kernel(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mb,
                    const __grid_constant__ CUtensorMap mo, const LParams p)
{
    using S = LSmem<CG, kParts>;
    constexpr int ST = S::ST;
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
        fence_mbar_init();
        prefetch_tmap(&ma);
        prefetch_tmap(&mb);
        if (MODE != MODE_LSE) prefetch_tmap(&mo);
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    l_cluster_sync<CG>();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    const int G = (int)gridDim.x / CG, c0 = (int)blockIdx.x / CG;
    const int bcols = p.bn / CG;                                  // this CTA's columns of B

    if (warp == 0) {
        // =================================================================== TMA producer
        if (lane == 0) {
            const int nb = (bcols + 63) / 64;                     // MN-major B: blocks of 64 columns
            const uint32_t bytes = (S::ASZ + (p.b_mn ? (uint32_t)nb * 8192u : (uint32_t)bcols * 128u)) * CG;
            int it = 0;
            bool ok = true;
            for (int item = c0; ok && item < p.items; item += G) {
                const LItem t = l_item<CG, MODE>(p, item);
                const int m0 = t.m0 + rank * 128;
                for (int nt = t.nt0; ok && nt < t.nt1; ++nt) {
                    const int n0 = nt * p.bn + rank * bcols;
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
                            if (p.a_mn) {
                                l_load<CG>(da, &ma, full, m0, ks * LK, part);
                                l_load<CG>(da + 8192u, &ma, full, m0 + 64, ks * LK, part);
                            } else {
                                l_load<CG>(da, &ma, full, ks * LK, m0, part);
                            }
                            if (p.b_mn) {
                                for (int b = 0; b < nb; ++b)
                                    l_load<CG>(db + 8192u * b, &mb, full, n0 + 64 * b, ks * LK, part);
                            } else {
                                l_load<CG>(db, &mb, full, ks * LK, n0, part);
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
            const uint32_t idesc = idesc_bf16(128 * CG, p.bn, p.a_mn, p.b_mn);
            // K-major: K steps of 32 bytes along the swizzled row; MN-major:
            // K steps of 16 rows (2 KB), blocks of 64 outputs 8 KB apart
            const uint64_t da0 = smem_desc_sw128(sbase + S::A, p.a_mn ? 8192 : 16, 1024);
            const uint64_t db0 = smem_desc_sw128(sbase + S::B, p.b_mn ? 8192 : 16, 1024);
            const uint64_t sa = p.a_mn ? 128 : 2, sb = p.b_mn ? 128 : 2;
            int it = 0, lt = 0;
            bool ok = true;
            for (int item = c0; ok && item < p.items; item += G) {
                const LItem t = l_item<CG, MODE>(p, item);
                for (int nt = t.nt0; ok && nt < t.nt1; ++nt) {
                    for (int ks = t.ks0; ok && ks < t.ks1; ++lt) {
                        // one accumulation: the whole K range, or one step of three parts
                        const int buf = lt & 1, k1 = kParts ? ks + 1 : t.ks1;
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
        unsigned char *stg = smem + S::OST + (uint32_t)(warp - 4) * 4096u;
        const uint32_t stg_a = sbase + S::OST + (uint32_t)(warp - 4) * 4096u;
        const int nch = p.bn / 64;                                // 64-column chunks, alternately per half
        int lt = 0;
        bool ok = true;
        // the staging buffer (32 rows x 128 bytes) is free once the previous store has read it
        auto stage_wait = [&]() {
            if (lane == 0) bulk_wait_read();
            __syncwarp();
        };
        auto stage_bf16 = [&](const float (&v)[32], int at) {      // columns 32 at .. 32 at + 31 of the row
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint4 pk;
                pk.x = pack2(v[8 * j + 0], v[8 * j + 1]);
                pk.y = pack2(v[8 * j + 2], v[8 * j + 3]);
                pk.z = pack2(v[8 * j + 4], v[8 * j + 5]);
                pk.w = pack2(v[8 * j + 6], v[8 * j + 7]);
                *reinterpret_cast<uint4 *>(stg + lane * 128 + (((4 * at + j) ^ (lane & 7)) << 4)) = pk;
            }
        };
        auto store = [&](int x, int y, int z, bool add) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                if (add)
                    l_reduce_3d(&mo, stg_a, x, y, z);
                else
                    tma_store_3d(&mo, stg_a, x, y, z);
                bulk_commit();
            }
        };
        auto release = [&](int buf) {      // this warp's part of the accumulator is in registers
            tc_fence_before();
            __syncwarp();
            if (lane == 0) l_arrive_leader<CG>(bar(S::AEMPTY + buf));
        };
        const uint64_t alpha2 = pair(p.alpha, p.alpha);
        // without biases the running maximum is kept of the unscaled logits
        const float mscale = p.has_bz ? 1.f : p.alpha;

        for (int item = c0; ok && item < p.items; item += G) {
            const LItem t = l_item<CG, MODE>(p, item);
            const int row0 = t.m0 + rank * 128 + 32 * q, row = row0 + lane;
            const bool live = row < p.M;
            float m = -INFINITY, l = 0.f, coef = 0.f, l2 = 0.f;
            Cursor cur;
            bool dead = false;
            if (MODE != MODE_CT) {
                cur.K = live ? p.r.K : 0;
                cur.col = p.r.col + (long)(live ? row : 0) * p.r.K;
                cur.p = MODE == MODE_DZ ? p.r.p + (long)(live ? row : 0) * p.r.K : nullptr;
                cur.seek(p.v0 + t.nt0 * p.bn);
                if (MODE == MODE_DZ) {
                    if (live) {
                        coef = p.r.coef[row];
                        l2 = p.r.l2[row];
                    }
                    dead = __any_sync(0xffffffffu, coef == 0.f);
                }
            }
            // 32 columns from n0 on (the second half of their 64-column chunk with sub = 1)
            auto process = [&](float (&v)[32], int n0, int sub) {
                if (MODE == MODE_CT) {
                    if (row0 >= p.M || n0 - 32 * sub >= p.N) return;
                    if (p.f32) {
                        if (n0 >= p.N) return;
                        stage_wait();
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            *reinterpret_cast<float4 *>(stg + lane * 128 + ((j ^ (lane & 7)) << 4)) =
                                make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                        store(n0, row0, t.split, p.add);
                    } else {
                        if (sub == 0) stage_wait();
                        stage_bf16(v, sub);
                        if (sub == 1) store(n0 - 32, row0, 0, false);
                    }
                    return;
                }
                if (n0 >= p.N) return;
                const int col0 = p.v0 + n0;
                // y = alpha z + bz in base-2 units (dz: less the row's lse)
                if (p.has_bz) {
                    const uint64_t off = pair(-l2, -l2);
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        const float4 b4 = __ldg(reinterpret_cast<const float4 *>(p.bz + n0 + j));
                        uint64_t b01 = pair(b4.x, b4.y), b23 = pair(b4.z, b4.w);
                        if (MODE == MODE_DZ) {
                            b01 = add2(b01, off);
                            b23 = add2(b23, off);
                        }
                        unpair(fma2(pair(v[j], v[j + 1]), alpha2, b01), v[j], v[j + 1]);
                        unpair(fma2(pair(v[j + 2], v[j + 3]), alpha2, b23), v[j + 2], v[j + 3]);
                    }
                }
                if (n0 + 32 > p.N) {   // columns past the vocabulary
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (n0 + j >= p.N) v[j] = -INFINITY;
                }
                if (MODE == MODE_LSE) {
                    while (cur.c0 < col0 + 32) {
                        if (cur.c0 >= col0) {
                            float y = 0.f;
#pragma unroll
                            for (int j = 0; j < 32; ++j) y = cur.c0 == col0 + j ? v[j] : y;
                            p.ysel[(long)row * p.r.K + cur.pos] = y * mscale;
                        }
                        cur.next();
                    }
                    __syncwarp();
                    const float cm = max32(v, m), ref = cm == -INFINITY ? 0.f : cm;
                    const uint64_t off = pair(-ref * mscale, -ref * mscale), one = pair(mscale, mscale);
                    uint64_t s[4] = {0, 0, 0, 0};
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        float a, b;
                        const uint64_t x = pair(v[2 * j], v[2 * j + 1]);
                        unpair(p.has_bz ? add2(x, off) : fma2(x, one, off), a, b);
                        s[j & 3] = add2(s[j & 3], pair(ex2(a), ex2(b)));
                    }
                    float a, b;
                    unpair(add2(add2(s[0], s[1]), add2(s[2], s[3])), a, b);
                    l = fmaf(l, ex2((m - ref) * mscale), a + b);
                    m = cm;
                } else {
                    const uint64_t off = pair(-l2, -l2), c2 = pair(coef, coef);
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        float a = v[j], b = v[j + 1];
                        if (!p.has_bz) unpair(fma2(pair(a, b), alpha2, off), a, b);
                        unpair(mul2(pair(ex2(a), ex2(b)), c2), v[j], v[j + 1]);
                    }
                    while (cur.c0 < col0 + 32) {
                        if (cur.c0 >= col0) {
                            const float g = coef * cur.p0;
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (cur.c0 == col0 + j) v[j] -= g;
                        }
                        cur.next();
                    }
                    __syncwarp();
                    if (dead) {   // whatever an empty row holds
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = coef == 0.f ? 0.f : v[j];
                    }
                    if (!kParts) {
                        if (sub == 0) stage_wait();
                        stage_bf16(v, sub);
                        // the second half of the chunk may lie past the last column
                        if ((sub == 1 || n0 + 32 >= p.N) && row0 < p.M) store(n0 - 32 * sub, row0, 0, false);
                    } else {
                        float rest[32];
#pragma unroll
                        for (int j = 0; j < 32; ++j) rest[j] = v[j];
#pragma unroll
                        for (int part = 0; part < 3; ++part) {
                            stage_wait();
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                uint32_t w4[4];
#pragma unroll
                                for (int x = 0; x < 4; ++x) {
                                    const float a = rest[8 * j + 2 * x], b = rest[8 * j + 2 * x + 1];
                                    const float ta = top_part(a), tb = top_part(b);
                                    w4[x] = pack2(ta, tb);
                                    rest[8 * j + 2 * x] = a - ta;
                                    rest[8 * j + 2 * x + 1] = b - tb;
                                }
                                // 64-byte rows, their swizzle: chunk c of row r at c ^ (r / 2 % 4)
                                *reinterpret_cast<uint4 *>(stg + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)) =
                                    make_uint4(w4[0], w4[1], w4[2], w4[3]);
                            }
                            if (row0 < p.M) store(n0, row0, part, false);
                        }
                    }
                    if (p.dbpart) {
                        // sums over the warp's 32 rows: halving exchanges leave column j in lane j
#pragma unroll
                        for (int o = 16; o; o >>= 1) {
                            const bool up = lane & o;
#pragma unroll
                            for (int j = 0; j < o; ++j) {
                                const float send = up ? v[j] : v[j + o];
                                const float keep = up ? v[j + o] : v[j];
                                v[j] = keep + __shfl_xor_sync(0xffffffffu, send, o);
                            }
                        }
                        if (row0 < p.M && n0 + lane < p.N)
                            p.dbpart[(long)(row0 >> 5) * p.dbpitch + n0 + lane] = v[0];
                    }
                }
            };
            const uint32_t tq = tmem + ((uint32_t)(32 * q) << 16);
            for (int nt = t.nt0; ok && nt < t.nt1; ++nt) {
                float v0[32], v1[32];
                if (kParts) {
                    // this half's 64 columns, summed over the steps
#pragma unroll
                    for (int j = 0; j < 32; ++j) v0[j] = v1[j] = 0.f;
                    for (int ks = t.ks0; ks < t.ks1; ++ks, ++lt) {
                        if (!wait(S::AFULL + (lt & 1), (lt >> 1) & 1)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        if (half < nch) {
                            const uint32_t at = tq + (uint32_t)((lt & 1) * 256 + 64 * half);
                            float x[32];
                            tmem_ld32(at, x);
#pragma unroll
                            for (int j = 0; j < 32; ++j) v0[j] += x[j];
                            tmem_ld32(at + 32u, x);
#pragma unroll
                            for (int j = 0; j < 32; ++j) v1[j] += x[j];
                        }
                        release(lt & 1);
                    }
                    if (!ok) break;
                    if (half < nch) {
                        process(v0, nt * p.bn + 64 * half, 0);
                        process(v1, nt * p.bn + 64 * half + 32, 1);
                    }
                    continue;
                }
                const int buf = lt & 1;
                if (!wait(S::AFULL + buf, (lt >> 1) & 1)) {
                    ok = false;
                    break;
                }
                ++lt;
                tc_fence_after();
                if (half >= nch) {
                    release(buf);
                    continue;
                }
                // each load is in flight while the columns before it are worked on
                const uint32_t tacc = tq + (uint32_t)(buf * 256);
                l_tmem_issue(tacc + 64u * half, v0);
                l_tmem_wait(v0);
                for (int c = half; c < nch; c += 2) {
                    const int n0 = nt * p.bn + 64 * c;
                    l_tmem_issue(tacc + 64u * c + 32u, v1);
                    process(v0, n0, 0);
                    l_tmem_wait(v1);
                    if (c + 2 < nch)
                        l_tmem_issue(tacc + 64u * (c + 2), v0);
                    else
                        release(buf);
                    process(v1, n0 + 32, 1);
                    if (c + 2 < nch) l_tmem_wait(v0);
                }
            }
            if (MODE == MODE_LSE && ok && live)
                p.part[(long)(kSlotsPerStrip * t.strip + half) * p.M + row] = make_float2(m * mscale, l);
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
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    if (!fn) {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
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

template <int CG, int MODE, bool kParts>
cudaError_t l_launch(const CUtensorMap &ma, const CUtensorMap &mb, const CUtensorMap &mo, const LParams &p,
                     cudaStream_t s)
{
    auto kern = loss_product_kernel<CG, MODE, kParts>;
    static std::atomic<int> most[64];      // tiles that run at once, per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorNotSupported;
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    cfg.blockDim = dim3(LNT);
    cfg.dynamicSmemBytes = LSmem<CG, kParts>::TOTAL;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = CG;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    int n = most[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)LSmem<CG, kParts>::TOTAL);
        if (e != cudaSuccess) return e;
        n = device_sm_count() / CG;
        if (CG == 2) {
            // an odd SM of a GPC takes no pair
            cfg.gridDim = dim3((unsigned)(CG * n));
            int fit = 0;
            e = cudaOccupancyMaxActiveClusters(&fit, kern, &cfg);
            if (e != cudaSuccess) return e;
            if (fit > 0 && fit < n) n = fit;
        }
        most[dev].store(n, std::memory_order_relaxed);
    }
    cfg.gridDim = dim3((unsigned)(CG * (p.items < n ? p.items : n)));
    return cudaLaunchKernelEx(&cfg, kern, ma, mb, mo, p);
}

template <int MODE>
cudaError_t l_launch_cg(int cg, int parts, const CUtensorMap &ma, const CUtensorMap &mb, const CUtensorMap &mo, const LParams &p,
                        cudaStream_t s)
{
    if (parts == 3) return cg == 2 ? l_launch<2, MODE, true>(ma, mb, mo, p, s) : l_launch<1, MODE, true>(ma, mb, mo, p, s);
    return cg == 2 ? l_launch<2, MODE, false>(ma, mb, mo, p, s) : l_launch<1, MODE, false>(ma, mb, mo, p, s);
}

// the fields the two vocabulary passes share
cudaError_t vocab_params(LParams &p, CUtensorMap &ma, CUtensorMap &mb, const LossMatrix &h, const LossMatrix &w,
                         const float *bz, int v0, float alpha, const LossRows &r, const LossTiling &t)
{
    memset(&p, 0, sizeof(p));
    p.M = h.rows;
    p.N = w.rows;
    p.bn = t.bn;
    p.tiles_m = t.tiles_m;
    p.tiles_n = t.tiles_n;
    p.strip = t.strip;
    p.strips = vocab_strips(t);
    const long items = (long)t.tiles_m * p.strips;
    if (items > INT32_MAX) return cudaErrorNotSupported;
    p.items = (int)items;
    p.ksteps = (h.cols + LK - 1) / LK;
    p.splits = 1;
    p.bz = bz;
    p.has_bz = bz != nullptr;
    p.v0 = v0;
    p.alpha = alpha;
    p.r = r;
    cudaError_t e = l_in_map(&ma, h, 128);
    if (e == cudaSuccess) e = l_in_map(&mb, w, t.bn / t.cg);
    return e;
}

long cdiv(long a, long b) { return (a + b - 1) / b; }

}  // namespace

LossTiling vocab_tiling(int rows, int cols, int d, int pieces)
{
    LossTiling t;
    t.cg = rows > 128 ? 2 : 1;
    const int widest = pieces == 3 ? 128 : 256;
    t.bn = cols > widest - 64 ? widest : (cols + 63) / 64 * 64;
    t.tiles_m = (int)cdiv(rows, 128 * t.cg);
    t.tiles_n = (int)cdiv(cols, t.bn);
    t.splits = 1;
    // strips: few enough partial results, and the last round of CTAs full
    const long slots = device_sm_count() / t.cg;
    double best = 1e300;
    t.strip = 1;
    for (int s = 1; s <= t.tiles_n && s <= 64; ++s) {
        const double cost = (double)cdiv(t.tiles_m * cdiv(t.tiles_n, s), slots) * (s + 0.15);
        if (cost <= best) {
            best = cost;
            t.strip = s;
        }
    }
    (void)d;
    return t;
}

LossTiling contract_tiling(int m, int n, int k, int pieces, bool always_slots)
{
    LossTiling t;
    t.cg = m > 128 ? 2 : 1;
    t.tiles_m = (int)cdiv(m, 128 * t.cg);
    t.tiles_n = (int)cdiv(n, pieces == 3 ? 128 : 256);
    t.bn = (int)(cdiv(cdiv(n, t.tiles_n), 64) * 64);
    t.strip = 1;
    const long slots = device_sm_count() / t.cg;
    const long ksteps = cdiv(k, LK) * (pieces == 3 ? 6 : 1);
    const double step_us = 0.27 * t.bn / 256;
    // splits of the long axis fill the SMs; each costs a pass over its slot
    // (0.27 us per 64-deep step of a 256-wide tile, 5 TB/s for the slots)
    double best = 1e300;
    t.splits = 1;
    for (int s = 1; s <= 64 && s <= cdiv(k, LK); ++s) {
        const double rounds = (double)cdiv((long)t.tiles_m * t.tiles_n * s, slots);
        const double passes = s > 1 || always_slots ? 2.0 * s * m * n * 4 / 5e6 : 0.0;
        const double cost = rounds * ((double)cdiv(ksteps, s) + 6) * step_us + passes + (s > 1 ? 3.0 : 0.0);
        if (cost < best) {
            best = cost;
            t.splits = s;
        }
    }
    return t;
}

cudaError_t launch_loss_lse(const LossMatrix &h, const LossMatrix &w, const float *bz, int v0, float alpha,
                            const LossRows &r, float *ysel, float2 *part, const LossTiling &t, cudaStream_t s)
{
    LParams p;
    CUtensorMap ma, mb;
    cudaError_t e = vocab_params(p, ma, mb, h, w, bz, v0, alpha, r, t);
    if (e != cudaSuccess) return e;
    p.ysel = ysel;
    p.part = part;
    return l_launch_cg<MODE_LSE>(t.cg, h.pieces, ma, mb, ma, p, s);
}

cudaError_t launch_loss_dz(const LossMatrix &h, const LossMatrix &w, const float *bz, int v0, float alpha,
                           const LossRows &r, const LossMatrix &dz, float *dbpart, const LossTiling &t,
                           cudaStream_t s)
{
    LParams p;
    CUtensorMap ma, mb, mo;
    cudaError_t e = vocab_params(p, ma, mb, h, w, bz, v0, alpha, r, t);
    if (e != cudaSuccess) return e;
    p.dbpart = dbpart;
    p.dbpitch = dz.pitch;
    const bool three = dz.pieces == 3;
    e = l_map(&mo, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, dz.base, dz.cols, dz.rows, dz.pieces, dz.pitch,
              dz.piece_stride, three ? 32 : 64, 32, three ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
    if (e != cudaSuccess) return e;
    return l_launch_cg<MODE_DZ>(t.cg, h.pieces, ma, mb, mo, p, s);
}

cudaError_t launch_loss_contract(const LossMatrix &a, bool a_t, const LossMatrix &b, int m, int n, int k,
                                 const LossOutput &out, const LossTiling &t, cudaStream_t s)
{
    LParams p;
    memset(&p, 0, sizeof(p));
    p.M = m;
    p.N = n;
    p.bn = t.bn;
    p.tiles_m = t.tiles_m;
    p.tiles_n = t.tiles_n;
    p.strip = 1;
    p.splits = t.splits;
    const long items = (long)t.tiles_m * t.tiles_n * t.splits;
    if (items > INT32_MAX) return cudaErrorNotSupported;
    p.items = (int)items;
    p.ksteps = (k + LK - 1) / LK;
    p.a_mn = a_t;
    p.b_mn = 1;
    p.f32 = out.f32;
    p.add = out.add;
    CUtensorMap ma, mb, mo;
    cudaError_t e = l_in_map(&ma, a, a_t ? 64 : 128);
    if (e == cudaSuccess) e = l_in_map(&mb, b, 64);
    if (e == cudaSuccess)
        e = l_map(&mo, out.f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, out.f32 ? 4 : 2,
                  out.base, n, m, t.splits, out.pitch, out.slot_stride, out.f32 ? 32 : 64, 32,
                  CU_TENSOR_MAP_SWIZZLE_128B);
    if (e != cudaSuccess) return e;
    return l_launch_cg<MODE_CT>(t.cg, a.pieces, ma, mb, mo, p, s);
}

cudaError_t read_and_clear_loss_error(unsigned int *word, cudaStream_t s)
{
    cudaError_t e = cudaMemcpyFromSymbolAsync(word, g_loss_err, sizeof(unsigned int), 0, cudaMemcpyDeviceToHost, s);
    if (e != cudaSuccess) return e;
    e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return e;
    if (*word) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbolAsync(g_loss_err, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, s);
        if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    }
    return e;
}

}  // namespace txl

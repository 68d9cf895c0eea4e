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
        asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(l_leader<CG>(bar)) : "memory");
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
        // 32 rows x 128 bytes from the staging buffer; the previous store has read it first
        auto stage_wait = [&]() {
            if (lane == 0) bulk_wait_read();
            __syncwarp();
        };
        for (int item = c0; ok && item < p.items; item += G) {
            const LItem t = l_item<CG, MODE>(p, item);
            const int row0 = t.m0 + rank * 128 + 32 * q, row = row0 + lane;
            const bool live = row < p.M;
            float m = -INFINITY, l = 0.f, coef = 0.f, l2 = 0.f;
            Cursor cur;
            if (MODE != MODE_CT) {
                cur.K = live ? p.r.K : 0;
                cur.col = p.r.col + (long)(live ? row : 0) * p.r.K;
                cur.p = MODE == MODE_DZ ? p.r.p + (long)(live ? row : 0) * p.r.K : nullptr;
                cur.seek(p.v0 + t.nt0 * p.bn);
                if (MODE == MODE_DZ && live) {
                    coef = p.r.coef[row];
                    l2 = p.r.l2[row];
                }
            }
            for (int nt = t.nt0; ok && nt < t.nt1; ++nt) {
                const uint32_t tq = tmem + ((uint32_t)(32 * q) << 16);
                float acc[kParts ? 64 : 1];
                if (kParts) {
                    // this half's 64 columns, summed over the steps
#pragma unroll
                    for (int j = 0; j < (kParts ? 64 : 1); ++j) acc[j] = 0.f;
                    for (int ks = t.ks0; ks < t.ks1; ++ks, ++lt) {
                        if (!wait(S::AFULL + (lt & 1), (lt >> 1) & 1)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        if (half < nch) {
#pragma unroll
                            for (int sub = 0; sub < 2; ++sub) {
                                float v[32];
                                tmem_ld32(tq + (uint32_t)((lt & 1) * 256 + 64 * half + 32 * sub), v);
#pragma unroll
                                for (int j = 0; j < 32; ++j) acc[kParts ? 32 * sub + j : 0] += v[j];
                            }
                        }
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) l_arrive_leader<CG>(bar(S::AEMPTY + (lt & 1)));
                    }
                    if (!ok) break;
                } else {
                    if (!wait(S::AFULL + (lt & 1), (lt >> 1) & 1)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                }
                const int buf = lt & 1;
                const uint32_t tacc = tq + (uint32_t)(buf * 256);
                for (int c = half; c < nch; c += 2) {
#pragma unroll
                    for (int sub = 0; sub < 2; ++sub) {
                        const int n0 = nt * p.bn + 64 * c + 32 * sub;   // first output column of these 32
                        float v[32];
                        if (kParts) {
#pragma unroll
                            for (int j = 0; j < 32; ++j) v[j] = acc[kParts ? 32 * sub + j : 0];
                        } else {
                            tmem_ld32(tacc + (uint32_t)(64 * c + 32 * sub), v);
                        }
                        if (MODE == MODE_CT) {
                            if (p.f32) {
                                if (row0 >= p.M || n0 >= p.N) continue;
                                stage_wait();
#pragma unroll
                                for (int j = 0; j < 8; ++j)
                                    *reinterpret_cast<float4 *>(stg + lane * 128 + ((j ^ (lane & 7)) << 4)) =
                                        make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                                fence_proxy_async_smem();
                                __syncwarp();
                                if (lane == 0) {
                                    if (p.add)
                                        l_reduce_3d(&mo, stg_a, n0, row0, t.split);
                                    else
                                        tma_store_3d(&mo, stg_a, n0, row0, t.split);
                                    bulk_commit();
                                }
                            } else {
                                if (row0 >= p.M || n0 - 32 * sub >= p.N) continue;
                                if (sub == 0) stage_wait();
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    uint4 pk;
                                    pk.x = pack2(v[8 * j + 0], v[8 * j + 1]);
                                    pk.y = pack2(v[8 * j + 2], v[8 * j + 3]);
                                    pk.z = pack2(v[8 * j + 4], v[8 * j + 5]);
                                    pk.w = pack2(v[8 * j + 6], v[8 * j + 7]);
                                    *reinterpret_cast<uint4 *>(stg + lane * 128 + (((4 * sub + j) ^ (lane & 7)) << 4)) = pk;
                                }
                                if (sub == 1) {
                                    fence_proxy_async_smem();
                                    __syncwarp();
                                    if (lane == 0) {
                                        tma_store_3d(&mo, stg_a, n0 - 32, row0, 0);
                                        bulk_commit();
                                    }
                                }
                            }
                            continue;
                        }
                        if (n0 >= p.N) continue;
                        // y in base-2 units; columns past the vocabulary are -infinity
                        const bool tail = n0 + 32 > p.N;
                        if (p.has_bz) {
                            if (!tail) {
#pragma unroll
                                for (int j = 0; j < 32; j += 4) {
                                    const float4 b4 = __ldg(reinterpret_cast<const float4 *>(p.bz + n0 + j));
                                    v[j] = fmaf(v[j], p.alpha, b4.x);
                                    v[j + 1] = fmaf(v[j + 1], p.alpha, b4.y);
                                    v[j + 2] = fmaf(v[j + 2], p.alpha, b4.z);
                                    v[j + 3] = fmaf(v[j + 3], p.alpha, b4.w);
                                }
                            } else {
#pragma unroll
                                for (int j = 0; j < 32; ++j)
                                    v[j] = n0 + j < p.N ? fmaf(v[j], p.alpha, __ldg(p.bz + n0 + j)) : -INFINITY;
                            }
                        } else {
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                v[j] = !tail || n0 + j < p.N ? v[j] * p.alpha : -INFINITY;
                        }
                        const int col0 = p.v0 + n0;
                        if (MODE == MODE_LSE) {
                            float cm = m;
#pragma unroll
                            for (int j = 0; j < 32; ++j) cm = fmaxf(cm, v[j]);
                            const float ref = cm == -INFINITY ? 0.f : cm;
                            float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
                            while (cur.c0 < col0 + 32) {
                                if (cur.c0 >= col0) {
                                    float y = 0.f;
#pragma unroll
                                    for (int j = 0; j < 32; ++j) y = cur.c0 == col0 + j ? v[j] : y;
                                    p.ysel[(long)row * p.r.K + cur.pos] = y;
                                }
                                cur.next();
                            }
                            __syncwarp();
#pragma unroll
                            for (int j = 0; j < 32; j += 4) {
                                s0 += ex2(v[j] - ref);
                                s1 += ex2(v[j + 1] - ref);
                                s2 += ex2(v[j + 2] - ref);
                                s3 += ex2(v[j + 3] - ref);
                            }
                            l = l * ex2(m - ref) + ((s0 + s1) + (s2 + s3));
                            m = cm;
                        } else {
#pragma unroll
                            for (int j = 0; j < 32; ++j) v[j] = coef * ex2(v[j] - l2);
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
                            if (coef == 0.f) {   // whatever the row holds
#pragma unroll
                                for (int j = 0; j < 32; ++j) v[j] = 0.f;
                            }
                            if (!kParts) {
                                if (sub == 0) stage_wait();
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    uint4 pk;
                                    pk.x = pack2(v[8 * j + 0], v[8 * j + 1]);
                                    pk.y = pack2(v[8 * j + 2], v[8 * j + 3]);
                                    pk.z = pack2(v[8 * j + 4], v[8 * j + 5]);
                                    pk.w = pack2(v[8 * j + 6], v[8 * j + 7]);
                                    *reinterpret_cast<uint4 *>(stg + lane * 128 + (((4 * sub + j) ^ (lane & 7)) << 4)) = pk;
                                }
                                // the second half of the chunk may lie past the last column
                                if (sub == 1 || n0 + 32 >= p.N) {
                                    fence_proxy_async_smem();
                                    __syncwarp();
                                    if (lane == 0 && row0 < p.M) {
                                        tma_store_3d(&mo, stg_a, n0 - 32 * sub, row0, 0);
                                        bulk_commit();
                                    }
                                }
                            } else {
                                // three parts, each 32 columns wide in its own half of the row
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
                                    fence_proxy_async_smem();
                                    __syncwarp();
                                    if (lane == 0 && row0 < p.M) {
                                        tma_store_3d(&mo, stg_a, n0, row0, part);
                                        bulk_commit();
                                    }
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
                    }
                }
                if (!kParts) {
                    // this warp's part of the accumulator is in registers
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) l_arrive_leader<CG>(bar(S::AEMPTY + buf));
                    ++lt;
                }
            }
            if (MODE == MODE_LSE && ok && live)
                p.part[(long)(kSlotsPerStrip * t.strip + half) * p.M + row] = make_float2(m, l);
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

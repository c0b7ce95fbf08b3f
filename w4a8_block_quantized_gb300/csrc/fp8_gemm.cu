// fp8_gemm.cu -- matrix product in 8-bit floating point (e4m3) with a scale for each block of 128.
//
// The mathematics:  y[m,n] = sum_b sa[b,m] sw[n / 128, b] P_b[m,n] (+ bias[n]),
//                   P_b[m,n] = sum over the 128 columns k of block b of a[m,k] w[n,k].
// A scale changes from block to block, so the tensor cores can sum only inside a block: each
// block's product P_b gets a TMEM accumulator of its own, and the epilogue warps fold it into
// fp32 sums in registers, one fma a block and output, y += (sa sw) P_b, while the tensor cores
// form the next block's product in another accumulator.
//
// Orientation: tokens are the MMA's M = 128 operand (TMEM lanes), weight rows its N operand, so a
// thread owns one token and the factor sa sw is one scalar per thread, block and 128 columns.
// Operand tiles come straight from the caller's row-major arrays by TMA: 128 rows x 128 columns
// = one scale block, 128-byte swizzled; rows past M or N and columns past K read as zeros, which
// add nothing to the products.
#include "fp8_ptx.cuh"
#include "ops_internal.h"

#include <cuda_bf16.h>

namespace w4a8 {
namespace {

constexpr uint32_t kLayoutSw128 = 2;
constexpr int kThreads = 256;

struct Fp8Params {
    CUtensorMap amap, wmap, ymap;
    const float* sa;
    const float* sw;
    const float* bias;
    void* y;
    int bf16, vec;  // vec: 16-byte stores fit every row of y
    int64_t M, N;
    int nb, tiles_m, tiles_n;
    uint32_t* status;
    uint64_t wait_limit_ns;
};

// Bounded wait that ignores the abort flag: used while unwinding, so that copies and MMAs in
// flight land before the CTA's shared memory and TMEM are released.
__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
    const uint32_t a = smem_u32(bar);
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(a, parity)) {
        if (globaltimer_ns() - t0 > limit_ns) return;
    }
}

namespace base {
constexpr int kBM = 128, kBN = 128, kStages = 4;
constexpr int kATile = kBM * 128, kStageBytes = kATile + kBN * 128;
constexpr int kOffBar = kStages * kStageBytes;
constexpr int kSmemBytes = kOffBar + 256 + 1024;
}  // namespace base

// Output columns n0 + 0 .. 31 of token m, with the bias where it is not in the sums already.
template <bool BIAS>
__device__ __forceinline__ void store_cols(const Fp8Params& p, int64_t m, int64_t n0, const float* y) {
    if (m >= p.M) return;
    if (p.vec && n0 + 32 <= p.N) {
        if (p.bf16) {
            uint4* d = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.y) + m * p.N + n0);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t u[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float v0 = y[8 * i + 2 * e], v1 = y[8 * i + 2 * e + 1];
                    if (BIAS && p.bias) v0 += p.bias[n0 + 8 * i + 2 * e], v1 += p.bias[n0 + 8 * i + 2 * e + 1];
                    const __nv_bfloat162 b = __floats2bfloat162_rn(v0, v1);
                    u[e] = *reinterpret_cast<const uint32_t*>(&b);
                }
                d[i] = make_uint4(u[0], u[1], u[2], u[3]);
            }
        } else {
            float4* d = reinterpret_cast<float4*>(static_cast<float*>(p.y) + m * p.N + n0);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float4 v = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
                if (BIAS && p.bias) {
                    const float* b = p.bias + n0 + 4 * i;
                    v.x += b[0], v.y += b[1], v.z += b[2], v.w += b[3];
                }
                d[i] = v;
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const int64_t n = n0 + i;
        if (n < p.N) {
            const float v = BIAS && p.bias ? y[i] + p.bias[n] : y[i];
            if (p.bf16) static_cast<__nv_bfloat16*>(p.y)[m * p.N + n] = __float2bfloat16_rn(v);
            else static_cast<float*>(p.y)[m * p.N + n] = v;
        }
    }
}

// 128 x 128 output tiles, one CTA each in turn (persistent).  Warp 0 copies, warp 1 issues the
// MMAs (4 of K = 32 a block), warps 4-7 drain: a thread holds its token's 128 sums.
__global__ void __launch_bounds__(kThreads, 1) fp8_gemm_kernel(const __grid_constant__ Fp8Params p) {
    using namespace base;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + kOffBar);
    uint64_t* empty = full + kStages;
    uint64_t* tfull = empty + kStages;
    uint64_t* tempty = tfull + 2;
    uint64_t* drain = tempty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile uint32_t* abort_flag = tmem_slot + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const WaitCtl ctl{abort_flag, p.status, p.wait_limit_ns};
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&tfull[i], 1);
            mbar_init(&tempty[i], 4);
        }
        mbar_init(drain, 1);
        *abort_flag = 0u;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, 2 * kBN);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    griddep_launch_dependents();
    griddep_wait();
    const int tiles = p.tiles_m * p.tiles_n;

    if (warp == 0) {
        if (lane == 0) {
            uint32_t j = 0, issued = 0;
            bool ok = true;
            for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
                const int m0 = (t % p.tiles_m) * kBM, n0 = (t / p.tiles_m) * kBN;
                for (int b = 0; b < p.nb; ++b, ++j) {
                    const uint32_t s = j % kStages, k = j / kStages;
                    if (k > 0 && !mbar_poll(&empty[s], (k - 1) & 1, ctl)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&full[s], kStageBytes);
                    tma_load_2d(smem + s * kStageBytes, &p.amap, b * 128, m0, &full[s]);
                    tma_load_2d(smem + s * kStageBytes + kATile, &p.wmap, b * 128, n0, &full[s]);
                    issued = j + 1;
                }
            }
            if (*abort_flag)
                for (uint32_t q = issued > kStages ? issued - kStages : 0; q < issued; ++q)
                    drain_wait(&full[q % kStages], (q / kStages) & 1, 100000000ull);
        }
        __syncwarp();
    } else if (warp == 1) {
        constexpr uint32_t idesc = idesc_e4m3_f32(kBM, kBN);
        uint32_t j = 0;
        bool ok = true;
        for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
            for (int b = 0; b < p.nb; ++b, ++j) {
                const uint32_t s = j % kStages, buf = j & 1u, u = j >> 1;
                ok = __all_sync(0xffffffffu, (u == 0 || mbar_poll(&tempty[buf], (u - 1) & 1, ctl)) &&
                                                 mbar_poll(&full[s], (j / kStages) & 1, ctl));
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t sa = smem_u32(smem + s * kStageBytes);
                    const uint64_t da = smem_desc(sa, 1024, kLayoutSw128);
                    const uint64_t dw = smem_desc(sa + kATile, 1024, kLayoutSw128);
#pragma unroll
                    for (int k = 0; k < 4; ++k) mma_f8f6f4(tmem + buf * kBN, da + 2 * k, dw + 2 * k, idesc, k > 0);
                    mma_commit(&empty[s]);
                    mma_commit(&tfull[buf]);
                }
                __syncwarp();
            }
        }
        if (elect_one()) mma_commit(drain);
        __syncwarp();
        drain_wait(drain, 0, 100000000ull);
    } else if (warp >= 4) {
        const int q = warp & 3;
        const uint32_t tl = tmem + (static_cast<uint32_t>(q * 32) << 16);
        uint32_t j = 0;
        bool ok = true;
        for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
            const int tn = t / p.tiles_m;
            const int64_t m = static_cast<int64_t>(t % p.tiles_m) * kBM + q * 32 + lane;
            const float* sa = p.sa + m;
            const float* sw = p.sw + static_cast<int64_t>(tn) * p.nb;
            float y[kBN];
#pragma unroll
            for (int c = 0; c < kBN; ++c) y[c] = 0.0f;
            for (int b = 0; b < p.nb; ++b, ++j) {
                const uint32_t buf = j & 1u;
                const float f = m < p.M ? __ldcg(sa + static_cast<int64_t>(b) * p.M) * __ldcg(sw + b) : 0.0f;
                if (!__all_sync(0xffffffffu, mbar_poll(&tfull[buf], (j >> 1) & 1, ctl))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < kBN; c += 32) {
                    uint32_t v[32];
                    tmem_ld_32x32b_x16(tl + buf * kBN + c, v);
                    tmem_ld_32x32b_x16(tl + buf * kBN + c + 16, v + 16);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e) y[c + e] = fmaf(f, __uint_as_float(v[e]), y[c + e]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&tempty[buf]);
            }
            if (!ok) break;
#pragma unroll
            for (int c = 0; c < kBN; c += 32) store_cols<true>(p, m, static_cast<int64_t>(tn) * kBN + c, y + c);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 2 * kBN);
    }
}

// ---------------------------------------------------------------- pairs of CTAs
// The large form: a cluster of two CTAs owns a 256 x 256 output tile.  One MMA covers 256 tokens
// x 128 weight rows over both SMs (cta_group::2): each CTA's shared memory holds its own 128
// tokens and half of the weight rows, so per SM and block 32 KB are copied and read where two
// lone 128 x 256 tiles would take 48.  The even CTA issues the MMAs; commits arrive on the barriers
// of both.
//   warp 0      copies: its tokens' and its half of the weights' boxes, four stages; both CTAs'
//               copies complete the even CTA's barrier
//   warps 1-2   (even CTA) every other block each: 2 x 4 MMAs of K = 32, one accumulator for each
//               half of the columns
//   warp 3      scales: eight blocks' sa and sw (and a tile's bias) at a time into shared memory,
//               one batch ahead
//   warps 4-19  drain, 4 lane quarters x 4 runs of 64 columns: a thread holds 64 sums
//
// Measured at 8192 x 4096 -> 14336 (bf16 out): 408 us, 2.36 PFLOP/s.  What bounds it is not the tensor
// pipe (206 us for the MMAs alone, 258 with the copies and the issue) but what surrounds each block:
// 32768 fmas a CTA and block (256 cycles of the fp32 pipes, against 512 of the tensor pipe), and the
// accumulators' way from a commit over the drain back to the issuer, during which their TMEM lies
// idle (350 us without the fmas).  So:
//   - four accumulators of 128 columns rather than two of 256: each is handed back as soon as
//     eight warps of each CTA have read it;
//   - sixteen draining warps: a warp spends most of a block waiting (barrier, TMEM load), and four
//     warps a scheduler fill that time with one another's fmas (eight warps of 128 sums: 416 us);
//   - one wait for an issuer: a stage's barrier counts its copies and the release of the
//     accumulators that its block overwrites (waits, MMAs and commits of a block cost a thread
//     about 700 cycles, so two issuers take turns).
// The outputs leave through a 4 KB staging box per warp and TMA stores (whole lines, rows past M
// and columns past N cut by the copy) while the tensor cores work on the next tile.
namespace pair {
constexpr int kThreads = 640, kEpiWarps = 16;
constexpr int kBM = 256, kBN = 256, kStages = 4;
constexpr int kABytes = 128 * 128, kWRows = 128;  // one CTA's boxes
constexpr int kStageBytes = kABytes + kWRows * 128;
constexpr int kOffOut = kStages * kStageBytes;    // staging: 32 rows x 128 bytes per epilogue warp
constexpr int kOutBox = 32 * 128;
constexpr int kChunk = 8;                         // blocks per batch of scales
constexpr int kOffScale = kOffOut + kEpiWarps * kOutBox;
constexpr int kScaleFloats = kChunk * 128 + 2 * kChunk;  // sa [block][row], sw [block][column half]
constexpr int kOffBias = kOffScale + 2 * kScaleFloats * 4;  // the tile's bias, two tiles
constexpr int kOffBar = kOffBias + 2 * kBN * 4;
constexpr int kSmemBytes = kOffBar + 256 + 1024;
static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
// Register split: launch = 640 x 96 (checked at build time); the first four warps drop to 32,
// the sixteen epilogue warps rise to 112: 128 * 32 + 512 * 112 = 640 * 96.
constexpr int kRegsLow = 32, kRegsHigh = 112;
static_assert(128 * kRegsLow + 512 * kRegsHigh == kThreads * 96, "register split");
// A wait on parity P returns at once while the phase before P is still open, so all phases of a
// stage must be waited for by one warp: the two issuers take the even and the odd stages.  And a
// stage's barrier may count a release only once its previous phase is over: a block's accumulators
// come free for the block two later, whose stage was last used two blocks before.
static_assert(kStages % 2 == 0 && kStages > 2, "stages of one issuer; releases after the previous phase");
}  // namespace pair

// Grouped raster: groups of eight row tiles, the row tile varying fastest inside a group, so the
// CTAs running at one time share operand tiles in L2.
__device__ __forceinline__ void tile_at(uint32_t t, uint32_t tiles_m, uint32_t tiles_n, uint32_t& tm, uint32_t& tn) {
    const uint32_t per = 8 * tiles_n, grp = t / per, r = t - grp * per, g0 = grp * 8;
    const uint32_t gsz = tiles_m - g0 < 8 ? tiles_m - g0 : 8;
    tn = r / gsz;
    tm = g0 + (r - tn * gsz);
}

// y[c] = fma(s, v[c], y[c]) for 32 columns, two per instruction (each element one fp32 fma).
__device__ __forceinline__ void fold32(float* y, float s, const uint32_t (&v)[32]) {
    uint64_t ss;
    asm("mov.b64 %0, {%1, %1};" : "=l"(ss) : "f"(s));
#pragma unroll
    for (int c = 0; c < 32; c += 2) {
        uint64_t yy, vv;
        asm("mov.b64 %0, {%1, %2};" : "=l"(yy) : "f"(y[c]), "f"(y[c + 1]));
        asm("mov.b64 %0, {%1, %2};" : "=l"(vv) : "r"(v[c]), "r"(v[c + 1]));
        asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(yy) : "l"(ss), "l"(vv));
        asm("mov.b64 {%0, %1}, %2;" : "=f"(y[c]), "=f"(y[c + 1]) : "l"(yy));
    }
}

// 32 rows (one a lane) x 128 bytes of columns from n0 of the warp's tokens from m0 into a staging
// box and out by a TMA store.  y: the lane's row.
template <bool BF16>
__device__ __forceinline__ void stage_out(const Fp8Params& p, uint8_t* box, int m0, int n0, const float* y, int lane) {
    if (lane == 0) bulk_wait_all<true>();  // the box's last store has read it
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        uint32_t u[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (BF16) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(y[8 * c + 2 * e], y[8 * c + 2 * e + 1]);
                u[e] = *reinterpret_cast<const uint32_t*>(&h);
            } else {
                u[e] = __float_as_uint(y[4 * c + e]);
            }
        }
        // the output map's 128-byte swizzle
        *reinterpret_cast<uint4*>(box + lane * 128 + ((c ^ (lane & 7)) << 4)) = make_uint4(u[0], u[1], u[2], u[3]);
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
        tma_store_2d(&p.ymap, n0, m0, box);
        bulk_commit();
    }
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(pair::kThreads, 1)
    fp8_pair_kernel(const __grid_constant__ Fp8Params p) {
    using namespace pair;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + kOffBar);
    uint64_t* empty = full + kStages;
    uint64_t* tfull = empty + kStages;  // [accumulator]: 2 (block parity) + half of the columns
    uint64_t* sfull = tfull + 4;
    uint64_t* sempty = sfull + 2;
    uint64_t* drain = sempty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 2);
    volatile uint32_t* abort_flag = tmem_slot + 1;
    float* scales = reinterpret_cast<float*>(smem + kOffScale);
    float* biases = reinterpret_cast<float*>(smem + kOffBias);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const WaitCtl ctl{abort_flag, p.status, p.wait_limit_ns};
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1 + 2 * kEpiWarps);  // the copies, and both CTAs' epilogue warps
            mbar_init(&empty[s], 1);
        }
        for (int i = 0; i < 4; ++i) mbar_init(&tfull[i], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sfull[i], 32);  // the copying warp's lanes
            mbar_init(&sempty[i], kEpiWarps);
            mbar_init(&drain[i], 1);
        }
        *abort_flag = 0u;
        fence_barrier_init();
    }
    if (warp == 1) tmem_alloc_pair(tmem_slot, 512);
    tc_fence_before();
    cluster_sync_all();  // both CTAs' barriers are ready before either signals the other
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    griddep_launch_dependents();
    griddep_wait();
    const uint32_t tiles = static_cast<uint32_t>(p.tiles_m) * static_cast<uint32_t>(p.tiles_n);
    const uint32_t first = blockIdx.x >> 1, step = gridDim.x >> 1;
    // blocks of this pair, over all its tiles
    const uint32_t total = tiles > first ? ((tiles - 1 - first) / step + 1) * static_cast<uint32_t>(p.nb) : 0u;

    if (warp < 4) {
        regs_dec<kRegsLow>();
        if (warp == 0 && lane == 0) {
            uint32_t j = 0, issued = 0;
            bool ok = true;
            for (uint32_t t = first; ok && t < tiles; t += step) {
                uint32_t tm, tn;
                tile_at(t, p.tiles_m, p.tiles_n, tm, tn);
                const int m0 = static_cast<int>(tm * kBM + rank * 128), n0 = static_cast<int>(tn * kBN + rank * kWRows);
#pragma unroll 1
                for (int b = 0; b < p.nb; ++b, ++j) {
                    const uint32_t s = j % kStages, k = j / kStages;
                    if (k > 0 && !mbar_poll(&empty[s], (k - 1) & 1, ctl)) {
                        ok = false;
                        break;
                    }
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * kStageBytes);
                    tma_load_2d_pair(smem + s * kStageBytes, &p.amap, b * 128, m0, &full[s]);
                    tma_load_2d_pair(smem + s * kStageBytes + kABytes, &p.wmap, b * 128, n0, &full[s]);
                    issued = j + 1;
                }
            }
            // after a wait gave up: both CTAs' copies land on the even CTA's barriers, which it
            // watches (for a bounded time) before the cluster's last barrier lets either leave
            if (*abort_flag && rank == 0)
                for (uint32_t q = issued > kStages ? issued - kStages : 0; q < issued; ++q)
                    drain_wait(&full[q % kStages], (q / kStages) & 1, 10000000ull);
        } else if ((warp == 1 || warp == 2) && rank == 0) {
            // An accumulator's 128 columns: 64 weight rows of each CTA's box.
            constexpr uint32_t idesc = idesc_e4m3_f32(kBM, kBN / 2);
            const uint32_t par = warp - 1;
            const uint64_t da0 = smem_desc(smem_u32(smem), 1024, kLayoutSw128);
            const uint64_t dw0 = smem_desc(smem_u32(smem + kABytes), 1024, kLayoutSw128);
            const uint32_t d = tmem + par * kBN;
#pragma unroll 1
            for (uint32_t j = par; j < total; j += 2) {
                if (*abort_flag) break;
                const uint32_t s = j % kStages;
                (void)mbar_poll(&full[s], (j / kStages) & 1, ctl);
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t o = static_cast<uint64_t>((s * kStageBytes) >> 4);
                    constexpr uint64_t half = (kWRows / 2) * 128 >> 4;
#pragma unroll
                    for (int k = 0; k < 4; ++k) mma_f8f6f4_pair(d, da0 + o + 2 * k, dw0 + o + 2 * k, idesc, k > 0);
                    mma_commit_pair(&tfull[2 * par]);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_f8f6f4_pair(d + kBN / 2, da0 + o + 2 * k, dw0 + o + half + 2 * k, idesc, k > 0);
                    mma_commit_pair(&tfull[2 * par + 1]);
                    mma_commit_pair(&empty[s]);
                }
                __syncwarp();
            }
            if (elect_one()) mma_commit_pair(&drain[par]);
            __syncwarp();
            drain_wait(&drain[par], 0, 100000000ull);
        } else if (warp == 3) {
            uint32_t j = 0, i = 0;  // batches staged, tiles
            for (uint32_t t = first; t < tiles && !*abort_flag; t += step, ++i) {
                uint32_t tm, tn;
                tile_at(t, p.tiles_m, p.tiles_n, tm, tn);
                const int64_t m0 = static_cast<int64_t>(tm) * kBM + rank * 128;
                // rows past M and columns past N are not stored; they take the last ones' values
                const int64_t w0 = 2 * static_cast<int64_t>(tn), wl = (p.N - 1) / 128;
                for (int b0 = 0; b0 < p.nb; b0 += kChunk, ++j) {
                    const uint32_t buf = j & 1u, u = j >> 1;
                    const int cnt = p.nb - b0 < kChunk ? p.nb - b0 : kChunk;
                    if (u > 0) (void)mbar_poll(&sempty[buf], (u - 1) & 1, ctl);
                    float* d = scales + buf * kScaleFloats;
#pragma unroll 1
                    for (int e = lane; e < 128; e += 32) {
                        const int64_t r = m0 + e;
                        const float* src = p.sa + b0 * p.M + (r < p.M ? r : p.M - 1);
#pragma unroll 1
                        for (int k = 0; k < cnt; ++k, src += p.M) cp_async4(d + k * 128 + e, src);
                    }
                    if (lane < 2 * cnt) {
                        const int64_t wt = w0 + (lane & 1) < wl ? w0 + (lane & 1) : wl;
                        cp_async4(d + kChunk * 128 + lane, p.sw + wt * p.nb + b0 + (lane >> 1));
                    }
                    if (b0 == 0 && p.bias) {  // with a tile's first batch: its bias
                        for (int c = lane; c < kBN; c += 32) {
                            const int64_t n = static_cast<int64_t>(tn) * kBN + c;
                            cp_async4(biases + (i & 1u) * kBN + c, p.bias + (n < p.N ? n : p.N - 1));
                        }
                    }
                    cp_async_arrive(&sfull[buf]);
                }
            }
        }
        __syncwarp();
    } else {
        regs_inc<kRegsHigh>();
        // TMEM lane quarter, column half (its accumulators), and which 64 columns of that
        const int q = warp & 3, h = ((warp - 4) >> 2) & 1, r = (warp - 4) >> 3;
        const uint32_t tl = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(h * (kBN / 2) + r * 64);
        // their first column in the tile (the run r of an accumulator comes from CTA r's weight rows)
        const int col = r * 128 + h * 64;
        const uint32_t release = map_rank(&full[0], 0);
        // the accumulators start free: release those of the first two blocks
        if (lane == 0)
            for (uint32_t b = 0; b < 2 && b < total; ++b) mbar_arrive_cluster(release + 8 * b);
        uint32_t j = 0, js = 0, it = 0;  // blocks drained, batches of scales used, tiles mod 2
        for (uint32_t t = first; t < tiles && !*abort_flag; t += step) {
            // the sums start from the bias, which arrives with the tile's first scales
            float y[64];
            (void)mbar_poll(&sfull[js & 1u], (js >> 1) & 1, ctl);
            if (p.bias) {
                const float* bs = biases + it * kBN + col;
#pragma unroll
                for (int c = 0; c < 64; c += 4) {
                    const float4 v = *reinterpret_cast<const float4*>(bs + c);
                    y[c] = v.x, y[c + 1] = v.y, y[c + 2] = v.z, y[c + 3] = v.w;
                }
            } else {
#pragma unroll
                for (int c = 0; c < 64; ++c) y[c] = 0.0f;
            }
            it ^= 1;
#pragma unroll 1
            for (int b = 0; b < p.nb; ++b, ++j) {
                const int i = b & (kChunk - 1);
                const float* sc = scales + (js & 1u) * kScaleFloats;
                if (i == 0 && b > 0) (void)mbar_poll(&sfull[js & 1u], (js >> 1) & 1, ctl);
                const float f = sc[i * 128 + q * 32 + lane] * sc[kChunk * 128 + 2 * i + r];
                if (i == kChunk - 1 || b == p.nb - 1) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sempty[js & 1u]);
                    ++js;
                }
                (void)mbar_poll(&tfull[2 * (j & 1u) + h], (j >> 1) & 1, ctl);
                tc_fence_after();
                const uint32_t ta = tl + (j & 1u) * kBN;
                uint32_t v[32];
                tmem_ld_32x32b_x32(ta, v);
                tmem_wait_ld32(v);
                fold32(y, f, v);
                tmem_ld_32x32b_x32(ta + 32, v);
                tmem_wait_ld32(v);
                // this warp's columns are read: its part of the accumulators is free for the block
                // two later
                tc_fence_before();
                __syncwarp();
                if (lane == 0 && j + 2 < total) mbar_arrive_cluster(release + 8 * ((j + 2) % kStages));
                fold32(y + 32, f, v);
            }
            uint32_t tm, tn;
            tile_at(t, p.tiles_m, p.tiles_n, tm, tn);
            const int64_t mw = static_cast<int64_t>(tm) * kBM + rank * 128 + q * 32;
            const int64_t n0 = static_cast<int64_t>(tn) * kBN + col;
            if (mw >= p.M || n0 >= p.N) continue;
            uint8_t* box = smem + kOffOut + (warp - 4) * kOutBox;
            if (!p.vec) {
                store_cols<false>(p, mw + lane, n0, y);
                store_cols<false>(p, mw + lane, n0 + 32, y + 32);
            } else if (p.bf16) {
                stage_out<true>(p, box, static_cast<int>(mw), static_cast<int>(n0), y, lane);
            } else {
                stage_out<false>(p, box, static_cast<int>(mw), static_cast<int>(n0), y, lane);
                if (n0 + 32 < p.N) stage_out<false>(p, box, static_cast<int>(mw), static_cast<int>(n0) + 32, y + 32, lane);
            }
        }
        if (lane == 0) bulk_wait_all<false>();
        __syncwarp();
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // neither CTA leaves while the other may still signal it or read its memory
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

// cuTensorMapEncodeTiled, resolved once through the runtime (no link-time dependence on the
// driver library).
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_tiled() {
    static const EncodeTiledFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return static_cast<EncodeTiledFn>(nullptr);
        return reinterpret_cast<EncodeTiledFn>(p);
    }();
    return fn;
}

// A map over y [M][N], boxes of 32 rows x 128 bytes, 128-byte swizzled as stage_out writes them.
bool make_out_map(CUtensorMap* map, void* y, int64_t M, int64_t N, bool bf16) {
    const EncodeTiledFn enc = encode_tiled();
    if (!enc) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(M)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(N) * (bf16 ? 2 : 4)};
    const cuuint32_t box[2] = {bf16 ? 64u : 32u, 32};
    const cuuint32_t estr[2] = {1, 1};
    return enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, y, dims, strides,
               box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A map over the bytes [rows][K], boxes of `box_rows` rows x 128 columns, 128-byte swizzled.
bool make_map(CUtensorMap* map, const uint8_t* p, int64_t rows, int64_t K, int box_rows) {
    const EncodeTiledFn enc = encode_tiled();
    if (!enc) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(K)};
    const cuuint32_t box[2] = {128, static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t estr[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(p), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename Kernel>
cudaError_t launch(Kernel kernel, int smem_bytes, bool* attr_done, int64_t grid, int threads, int cluster,
                   const Fp8Params& p, cudaStream_t s) {
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 64 && !attr_done[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes);
        if (e != cudaSuccess) return e;
        attr_done[dev] = true;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem_bytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_fp8_linear(const Fp8Args& a, int num_sms, cudaStream_t s) {
    static bool attr_done[2][64] = {};
    if (num_sms < 1) return cudaErrorInvalidValue;
    Fp8Params p;
    p.sa = a.sa;
    p.sw = a.sw;
    p.bias = a.bias;
    p.y = a.y;
    p.bf16 = a.bf16;
    p.vec = a.N % (a.bf16 ? 8 : 4) == 0;
    p.M = a.M;
    p.N = a.N;
    p.nb = static_cast<int>((a.K + kGroup8 - 1) / kGroup8);
    p.status = a.status;
    p.wait_limit_ns = a.wait_limit_ns;
    // 256 x 256 tiles where they fill the GPU, else 128 x 128 tiles.
    const int64_t pairs = ((a.M + pair::kBM - 1) / pair::kBM) * ((a.N + pair::kBN - 1) / pair::kBN);
    if (2 * pairs >= num_sms) {
        p.tiles_m = static_cast<int>((a.M + pair::kBM - 1) / pair::kBM);
        p.tiles_n = static_cast<int>((a.N + pair::kBN - 1) / pair::kBN);
        if (!make_map(&p.amap, a.a, a.M, a.K, 128) || !make_map(&p.wmap, a.w, a.N, a.K, pair::kWRows) ||
            (p.vec && !make_out_map(&p.ymap, a.y, a.M, a.N, a.bf16)))
            return cudaErrorInvalidValue;
        const int64_t most = num_sms / 2;
        return launch(fp8_pair_kernel, pair::kSmemBytes, attr_done[1], 2 * (pairs < most ? pairs : most), pair::kThreads, 1,
                      p, s);
    }
    p.tiles_m = static_cast<int>((a.M + base::kBM - 1) / base::kBM);
    p.tiles_n = static_cast<int>((a.N + base::kBN - 1) / base::kBN);
    if (!make_map(&p.amap, a.a, a.M, a.K, base::kBM) || !make_map(&p.wmap, a.w, a.N, a.K, base::kBN))
        return cudaErrorInvalidValue;
    const int64_t tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n;
    return launch(fp8_gemm_kernel, base::kSmemBytes, attr_done[0], tiles < num_sms ? tiles : num_sms, kThreads, 1, p, s);
}

}  // namespace w4a8

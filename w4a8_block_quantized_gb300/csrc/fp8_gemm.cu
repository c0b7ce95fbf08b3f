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
#include "sm103_ptx.cuh"
#include "ops_internal.h"

#include <cuda_bf16.h>

namespace w4a8 {
namespace {

constexpr uint32_t kLayoutSw128 = 2;
constexpr int kThreads = 256;

struct Fp8Params {
    CUtensorMap amap, wmap;
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

// Output columns n0 + 0 .. 31 of token m.
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
                    if (p.bias) v0 += p.bias[n0 + 8 * i + 2 * e], v1 += p.bias[n0 + 8 * i + 2 * e + 1];
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
                if (p.bias) {
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
            const float v = p.bias ? y[i] + p.bias[n] : y[i];
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
                    if (k > 0 && !mbar_wait(&empty[s], (k - 1) & 1, ctl)) {
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
                ok = __all_sync(0xffffffffu, (u == 0 || mbar_wait(&tempty[buf], (u - 1) & 1, ctl)) &&
                                                 mbar_wait(&full[s], (j / kStages) & 1, ctl));
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
                if (!__all_sync(0xffffffffu, mbar_wait(&tfull[buf], (j >> 1) & 1, ctl))) {
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
            for (int c = 0; c < kBN; c += 32) store_cols(p, m, static_cast<int64_t>(tn) * kBN + c, y + c);
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
    static bool attr_done[1][64] = {};
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
    p.tiles_m = static_cast<int>((a.M + base::kBM - 1) / base::kBM);
    p.tiles_n = static_cast<int>((a.N + base::kBN - 1) / base::kBN);
    p.status = a.status;
    p.wait_limit_ns = a.wait_limit_ns;
    if (!make_map(&p.amap, a.a, a.M, a.K, base::kBM) || !make_map(&p.wmap, a.w, a.N, a.K, base::kBN))
        return cudaErrorInvalidValue;
    const int64_t tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n;
    return launch(fp8_gemm_kernel, base::kSmemBytes, attr_done[0], tiles < num_sms ? tiles : num_sms, kThreads, 1, p, s);
}

}  // namespace w4a8

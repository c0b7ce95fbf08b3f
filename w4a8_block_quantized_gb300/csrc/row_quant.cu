// row_quant.cu -- rows of a decoder layer's hidden state brought into the 8-bit forms that the
// linears read: root-mean-square norm with the residual's addition, the gated activation
// silu(gate) * up, or the values as they are.
//
// The mathematics.  A row's values are t_k (kSrcNorm: h_k gamma_k with h = x + residual) times
// a factor r common to the row (kSrcNorm: 1 / sqrt(mean h^2 + eps); else 1).  A quantizer that
// divides by a multiple of the largest magnitude is blind to a common factor, so r goes into the
// scales and the codes are those of t:
//   INT8  s = max_k |t_k| / 127, code = clamp(round_half_away(t / s), +-127), a_scale = s r
//   e4m3  per 128 columns m = max |t_k|: code = e4m3(t * (448 / m)), a_scale = (m / 448) r;
//         a group with m < 2^-100 is stored as zeros with scale 0 (448 / m stays finite)
// Every step up to the codes is a single IEEE fp32 operation or a maximum, so the codes do not
// depend on how a row is split over threads, and the sum of squares is wanted only for the
// scales: the codes are formed and stored without waiting for it.  The sum is taken in fp32 in an
// order that depends on K alone.
//
// A row is read once.  `W` warps hold it in registers, C chunks of 8 values a lane: 16-byte
// loads, 8-byte stores of codes.  Rows past 32 warps x 4 chunks take the looping kernel, which
// reads twice (the second time from L2).  What bounds it: HBM bytes for many rows, the latency
// of one load -> reduce -> store chain for few.
#include "ops_internal.h"
#include "quant_math.cuh"
#include "sm103_ptx.cuh"
#include "token_records.cuh"

#include <cuda_bf16.h>

namespace w4a8 {
namespace {

// 8 consecutive values.
struct Chunk {
    float v[8];
};

template <bool BF16>
__device__ __forceinline__ Chunk load_chunk(const void* p, int64_t idx) {
    Chunk c;
    if constexpr (BF16) {
        const uint4 w = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + idx));
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            c.v[2 * i] = __uint_as_float(u[i] << 16);
            c.v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    } else {
        const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(p) + idx);
        const float4 a = __ldcs(f), b = __ldcs(f + 1);
        c.v[0] = a.x, c.v[1] = a.y, c.v[2] = a.z, c.v[3] = a.w;
        c.v[4] = b.x, c.v[5] = b.y, c.v[6] = b.z, c.v[7] = b.w;
    }
    return c;
}

// Stored in the inputs' type, one rounding to nearest even (none for fp32).
template <bool BF16>
__device__ __forceinline__ void store_chunk(void* p, int64_t idx, const Chunk& c) {
    if constexpr (BF16) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(c.v[2 * i], c.v[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + idx) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
        float4* f = reinterpret_cast<float4*>(static_cast<float*>(p) + idx);
        f[0] = make_float4(c.v[0], c.v[1], c.v[2], c.v[3]);
        f[1] = make_float4(c.v[4], c.v[5], c.v[6], c.v[7]);
    }
}

// The chunk at column k of row m: t in `t`, and its share of the sum of squares added to `sum`.
// STORE: the residual sum is stored too.
template <int SRC, bool BF16, bool STORE>
__device__ __forceinline__ void source(const RowArgs& a, int64_t m, int64_t k, Chunk& t, float& sum) {
    t = load_chunk<BF16>(a.x, m * a.ld + k);
    if constexpr (SRC == kSrcNorm) {
        if (a.residual) {
            const Chunk r = load_chunk<BF16>(a.residual, m * a.K + k);
#pragma unroll
            for (int i = 0; i < 8; ++i) t.v[i] = __fadd_rn(t.v[i], r.v[i]);
            if (STORE && a.residual_out) store_chunk<BF16>(a.residual_out, m * a.K + k, t);
        }
        const float4* gp = reinterpret_cast<const float4*>(a.gamma + k);
        const float4 g0 = gp[0], g1 = gp[1];
        const float g[8] = {g0.x, g0.y, g0.z, g0.w, g1.x, g1.y, g1.z, g1.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            sum = fmaf(t.v[i], t.v[i], sum);
            t.v[i] = __fmul_rn(t.v[i], g[i]);
        }
    } else if constexpr (SRC == kSrcSwiglu) {
        const Chunk u = load_chunk<BF16>(a.up, m * a.ld + k);
        // g / (1 + exp(-g)): for g below -88 exp(-g) is infinite and the quotient 0, its limit
#pragma unroll
        for (int i = 0; i < 8; ++i) t.v[i] = __fdividef(t.v[i], 1.0f + __expf(-t.v[i])) * u.v[i];
    }
}

__device__ __forceinline__ float chunk_max(const Chunk& t) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(t.v[i]));
    return m;
}

// 1 / sqrt(sum / K + eps), every step IEEE-rounded.
__device__ __forceinline__ float row_factor(float sum, int64_t K, float eps) {
    return __frcp_rn(__fsqrt_rn(__fdiv_rn(sum, static_cast<float>(K)) + eps));
}

// Codes of one e4m3 group held by 16 lanes (lanes of the other half warp: another group), and
// its scale before the factor r.  Chunks past the row hold zeros.
__device__ __forceinline__ float e4m3_group(const Chunk& t, uint2& codes) {
    float m = chunk_max(t);
#pragma unroll
    for (int o = 8; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const bool live = m >= 0x1p-100f;
    const float inv = live ? __fdiv_rn(448.0f, m) : 0.0f;
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = __fmul_rn(t.v[i], inv);
    codes.x = e4m3x2(q[0], q[1]) | (e4m3x2(q[2], q[3]) << 16);
    codes.y = e4m3x2(q[4], q[5]) | (e4m3x2(q[6], q[7]) << 16);
    return live ? __fdiv_rn(m, 448.0f) : 0.0f;
}

// INT8 codes of one chunk (q, as floats) into the API layout or a token record, and the sum of
// each 64-block's codes, taken over its 8 lanes (exact: small integers).  All lanes take part.
template <int FORM>
__device__ __forceinline__ void store_int8(const RowArgs& a, int64_t m, int64_t chunk, bool in, const float4& q0,
                                           const float4& q1, int lane) {
    float rs = ((q0.x + q0.y) + (q0.z + q0.w)) + ((q1.x + q1.y) + (q1.z + q1.w));
#pragma unroll
    for (int o = 4; o; o >>= 1) rs += __shfl_xor_sync(0xffffffffu, rs, o);
    if (!in) return;
    const int64_t nb = a.K / kBlock, b = chunk >> 3;
    if constexpr (FORM == kFormInt8) {
        *reinterpret_cast<uint2*>(a.a_q + m * a.K + 8 * chunk) = make_uint2(bytes4f(q0), bytes4f(q1));
        if ((lane & 7) == 0) a.rowsum[m * nb + b] = static_cast<int>(rs);
    } else {
        const int ts = a.tw == 256 ? 8 : 7;
        const int r = static_cast<int>(m & ((1 << ts) - 1)), j = 2 * static_cast<int>(chunk & 7);
        uint8_t* rec = token_rec(a.trec, m, b, nb, ts);
        uint2 hi, lo;
        planes4f(q0, hi.x, lo.x);
        planes4f(q1, hi.y, lo.y);
        // quads j and j + 1 share a 16-byte chunk of the record (j is even): 8-byte stores
        *reinterpret_cast<uint2*>(rec + plane_off(r, j, 0)) = hi;
        *reinterpret_cast<uint2*>(rec + plane_off(r, j, 1)) = lo;
        if ((lane & 7) == 0) *reinterpret_cast<uint4*>(rec + (128 << ts) + r * 16) = rx_entry(static_cast<int>(rs));
    }
}

// The maximum over the row's W warps.  Of the row's sum of squares, each warp holds C segment
// shares: sum[i] is its lanes' part of segment i W + wg, 256 columns of the row.  The total is
// taken over the segments' sums, segment j on lane j % 32, so it depends on the row alone and not
// on how its segments were dealt to warps: a row has the same bits in any batch.
// `red`: W maxima, then W C segment sums; only the row's warps meet.
template <int C, bool SUM, bool MAX>
__device__ __forceinline__ void row_reduce(float& amax, float (&sum)[C], float& total, float* red, int wg, int W,
                                           int bar, int lane) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        if (MAX) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
#pragma unroll
        for (int i = 0; i < C; ++i)
            if (SUM) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], o);
    }
    float v = 0.0f;
    if (W == 1) {
#pragma unroll
        for (int i = 0; i < C; ++i)
            if (lane == i) v = sum[i];
    } else {
        if (lane == 0) {
            if (MAX) red[wg] = amax;
#pragma unroll
            for (int i = 0; i < C; ++i)
                if (SUM) red[W + i * W + wg] = sum[i];
        }
        named_bar_sync(bar, W * 32);
        if (MAX) {
            amax = lane < W ? red[lane] : 0.0f;
#pragma unroll
            for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        }
        if (SUM)
            for (int j = lane; j < W * C; j += 32) v += red[W + j];
    }
    if (SUM) {
#pragma unroll
        for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    }
    total = v;
}

// One row per W warps, blockDim / (32 W) rows a block; C chunks a lane (K <= 256 W C).
template <int SRC, int FORM, bool BF16, int C>
__global__ void __launch_bounds__(1024) row_quant_kernel(const RowArgs a, int W) {
    griddep_launch_dependents();
    __shared__ float slots[32 * (1 + C)];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rsub = warp / W, wg = warp - rsub * W;
    float* red = slots + rsub * W * (1 + C);
    const int64_t m = static_cast<int64_t>(blockIdx.x) * ((blockDim.x >> 5) / W) + rsub;
    const int64_t n8 = a.K / 8;
    const bool row = m < a.M;  // the same for every warp of a row
    griddep_wait();
    Chunk t[C];
    float sum[C], amax = 0.0f, total = 0.0f;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int64_t c = static_cast<int64_t>(i * W + wg) * 32 + lane;
        sum[i] = 0.0f;
        if (row && c < n8) {
            source<SRC, BF16, true>(a, m, 8 * c, t[i], sum[i]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) t[i].v[e] = 0.0f;
        }
        if (FORM != kFormE4m3) amax = fmaxf(amax, chunk_max(t[i]));
    }
    if constexpr (FORM == kFormE4m3) {
        float s[C];
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int64_t c = static_cast<int64_t>(i * W + wg) * 32 + lane;
            uint2 codes;
            s[i] = e4m3_group(t[i], codes);
            if (row && c < n8) *reinterpret_cast<uint2*>(a.a_q + m * a.K + 8 * c) = codes;
        }
        float r = 1.0f;
        if constexpr (SRC == kSrcNorm) {
            row_reduce<C, true, false>(amax, sum, total, red, wg, W, 1 + rsub, lane);
            r = row_factor(total, a.K, a.eps);
        }
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int64_t c = static_cast<int64_t>(i * W + wg) * 32 + lane;
            if (row && c < n8 && (lane & 15) == 0) a.a_scale[(c >> 4) * a.M + m] = s[i] * r;
        }
    } else {
        row_reduce<C, SRC == kSrcNorm, true>(amax, sum, total, red, wg, W, 1 + rsub, lane);
        const float s = __fdiv_rn(amax, 127.0f);
        const float inv = __frcp_rn(s);
        if (row && wg == 0 && lane == 0)
            a.a_scale[m] = SRC == kSrcNorm ? s * row_factor(total, a.K, a.eps) : s;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int64_t c = static_cast<int64_t>(i * W + wg) * 32 + lane;
            const float4 x[2] = {make_float4(t[i].v[0], t[i].v[1], t[i].v[2], t[i].v[3]),
                                 make_float4(t[i].v[4], t[i].v[5], t[i].v[6], t[i].v[7])};
            float4 q[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
            if (s > 0.0f) quant_lane<2>(x, q, s, inv);
            store_int8<FORM>(a, m, c, row && c < n8, q[0], q[1], lane);
        }
    }
}

// Longer rows: a block of 32 warps walks its row twice, first for the maximum and the sum, then
// (from L2) for the codes.  The residual is stored on the second walk, after every read of it.
template <int SRC, int FORM, bool BF16>
__global__ void __launch_bounds__(1024) row_quant_long_kernel(const RowArgs a) {
    griddep_launch_dependents();
    __shared__ float red[64];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t m = blockIdx.x, n8 = a.K / 8;
    griddep_wait();
    float sum[1] = {0.0f}, amax = 0.0f, total = 0.0f;
    for (int64_t c = threadIdx.x; c < n8; c += 1024) {
        Chunk t;
        source<SRC, BF16, false>(a, m, 8 * c, t, sum[0]);
        if (FORM != kFormE4m3) amax = fmaxf(amax, chunk_max(t));
    }
    row_reduce<1, true, true>(amax, sum, total, red, warp, 32, 1, lane);
    const float r = SRC == kSrcNorm ? row_factor(total, a.K, a.eps) : 1.0f;
    const float s = __fdiv_rn(amax, 127.0f), inv = __frcp_rn(s);
    if (FORM != kFormE4m3 && threadIdx.x == 0) a.a_scale[m] = s * r;
    for (int64_t c0 = warp * 32; c0 < n8; c0 += 1024) {
        const int64_t c = c0 + lane;
        Chunk t;
        float unused = 0.0f;
        if (c < n8) {
            source<SRC, BF16, true>(a, m, 8 * c, t, unused);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) t.v[e] = 0.0f;
        }
        if constexpr (FORM == kFormE4m3) {
            uint2 codes;
            const float sg = e4m3_group(t, codes);
            if (c < n8) {
                *reinterpret_cast<uint2*>(a.a_q + m * a.K + 8 * c) = codes;
                if ((lane & 15) == 0) a.a_scale[(c >> 4) * a.M + m] = sg * r;
            }
        } else {
            const float4 x[2] = {make_float4(t.v[0], t.v[1], t.v[2], t.v[3]),
                                 make_float4(t.v[4], t.v[5], t.v[6], t.v[7])};
            float4 q[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
            if (s > 0.0f) quant_lane<2>(x, q, s, inv);
            store_int8<FORM>(a, m, c, c < n8, q[0], q[1], lane);
        }
    }
}

cudaError_t launch_pdl(void (*kernel)(RowArgs, int), int64_t grid, int threads, const RowArgs& a, int W, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a, W);
}

template <int SRC, int FORM, bool BF16>
cudaError_t run(const RowArgs& a, int num_sms, cudaStream_t s) {
    const int64_t n8 = a.K / 8;
    if (n8 > 32 * 32 * 4) {
        row_quant_long_kernel<SRC, FORM, BF16><<<static_cast<unsigned>(a.M), 1024, 0, s>>>(a);
        return cudaGetLastError();
    }
    auto warps = [&](int C) { return static_cast<int>((n8 + 32 * C - 1) / (32 * C)); };
    int C = 4;
    if (warps(1) <= 32 && a.M <= num_sms) C = 1;  // few rows: the shortest chain a lane
    else if (n8 <= 64 || (warps(2) <= 32 && a.M <= num_sms)) C = 2;
    const int W = warps(C);
    const int rpc = W >= 8 ? 1 : 8 / W;
    const int64_t grid = (a.M + rpc - 1) / rpc;
    switch (C) {
        case 1: return launch_pdl(row_quant_kernel<SRC, FORM, BF16, 1>, grid, rpc * W * 32, a, W, s);
        case 2: return launch_pdl(row_quant_kernel<SRC, FORM, BF16, 2>, grid, rpc * W * 32, a, W, s);
        default: return launch_pdl(row_quant_kernel<SRC, FORM, BF16, 4>, grid, rpc * W * 32, a, W, s);
    }
}

template <bool BF16>
cudaError_t pick(RowSource src, RowForm form, const RowArgs& a, int num_sms, cudaStream_t s) {
    switch (src) {
        case kSrcNorm:
            switch (form) {
                case kFormInt8: return run<kSrcNorm, kFormInt8, BF16>(a, num_sms, s);
                case kFormRecords: return run<kSrcNorm, kFormRecords, BF16>(a, num_sms, s);
                default: return run<kSrcNorm, kFormE4m3, BF16>(a, num_sms, s);
            }
        case kSrcSwiglu:
            switch (form) {
                case kFormInt8: return run<kSrcSwiglu, kFormInt8, BF16>(a, num_sms, s);
                case kFormRecords: return run<kSrcSwiglu, kFormRecords, BF16>(a, num_sms, s);
                default: return run<kSrcSwiglu, kFormE4m3, BF16>(a, num_sms, s);
            }
        default: return form == kFormE4m3 ? run<kSrcPlain, kFormE4m3, BF16>(a, num_sms, s) : cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_row_quant(RowSource src, RowForm form, bool bf16, const RowArgs& a, int num_sms, cudaStream_t s) {
    return bf16 ? pick<true>(src, form, a, num_sms, s) : pick<false>(src, form, a, num_sms, s);
}

}  // namespace w4a8

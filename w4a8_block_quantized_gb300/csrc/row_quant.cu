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
// A row is read once: `W` warps hold it in registers, C chunks of 8 values a lane (16-byte loads,
// 8-byte stores of codes), straight from memory or, for many rows, through a ring of rows in shared
// memory.  Rows past 16 warps x 4 chunks take the looping kernel, which reads twice (the second time
// from L2).  What bounds it: HBM bytes for many rows (16384 x 4096 bf16 norm to e4m3: 73 us, 6.4 TB/s,
// 96% of the copy rate; 8192 x 14336 bf16 gated activation 90 us, 6.6 TB/s, 98%), the latency of one
// load -> reduce -> store chain for few (1 x 4096: 2.5 us).
#include "ops_internal.h"
#include "quant_math.cuh"
#include "sm103_ptx.cuh"
#include "token_records.cuh"

#include <cuda_bf16.h>

namespace w4a8 {
namespace {

// 8 consecutive values, as loaded and as fp32.
template <bool BF16>
struct Raw {
    uint4 w[BF16 ? 1 : 2];
};
struct Chunk {
    float v[8];
};

template <bool BF16>
__device__ __forceinline__ Raw<BF16> load_raw(const void* p, int64_t idx) {
    Raw<BF16> r;
    if constexpr (BF16) {
        r.w[0] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + idx));
    } else {
        const uint4* f = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + idx);
        r.w[0] = __ldcs(f);
        r.w[1] = __ldcs(f + 1);
    }
    return r;
}

template <bool BF16>
__device__ __forceinline__ Chunk values(const Raw<BF16>& r) {
    Chunk c;
#pragma unroll
    for (int h = 0; h < (BF16 ? 1 : 2); ++h) {
        const uint32_t u[4] = {r.w[h].x, r.w[h].y, r.w[h].z, r.w[h].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (BF16) {
                c.v[2 * i] = __uint_as_float(u[i] << 16);
                c.v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
            } else {
                c.v[4 * h + i] = __uint_as_float(u[i]);
            }
        }
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

// What a chunk is computed from, loaded for all of a lane's chunks before any is worked on: the
// residual's stores would otherwise keep the next chunk's loads behind them (they may alias).
template <int SRC, bool BF16>
struct Inputs {
    Raw<BF16> x, y;  // y: the residual, or up
};

template <int SRC, bool BF16>
__device__ __forceinline__ void load_inputs(const RowArgs& a, int64_t m, int64_t k, Inputs<SRC, BF16>& in) {
    in.x = load_raw<BF16>(a.x, m * a.ld + k);
    if (SRC == kSrcNorm && a.residual) in.y = load_raw<BF16>(a.residual, m * a.K + k);
    if (SRC == kSrcSwiglu) in.y = load_raw<BF16>(a.up, m * a.ld + k);
}

template <int SRC>
__device__ __forceinline__ Chunk load_gamma(const RowArgs& a, int64_t k) {
    Chunk c = {};
    if constexpr (SRC == kSrcNorm) {
        const float4* gp = reinterpret_cast<const float4*>(a.gamma + k);
        const float4 g0 = gp[0], g1 = gp[1];
        c.v[0] = g0.x, c.v[1] = g0.y, c.v[2] = g0.z, c.v[3] = g0.w;
        c.v[4] = g1.x, c.v[5] = g1.y, c.v[6] = g1.z, c.v[7] = g1.w;
    }
    return c;
}

// The chunk at column k of row m: t in `t`, and its share of the sum of squares added to `sum`.
// STORE: the residual sum is stored too.
template <int SRC, bool BF16, bool STORE>
__device__ __forceinline__ void source(const RowArgs& a, int64_t m, int64_t k, const Inputs<SRC, BF16>& in,
                                       const Chunk& gamma, Chunk& t, float& sum) {
    t = values(in.x);
    if constexpr (SRC == kSrcNorm) {
        if (a.residual) {
            const Chunk r = values(in.y);
#pragma unroll
            for (int i = 0; i < 8; ++i) t.v[i] = __fadd_rn(t.v[i], r.v[i]);
            if (STORE && a.residual_out) store_chunk<BF16>(a.residual_out, m * a.K + k, t);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            sum = fmaf(t.v[i], t.v[i], sum);
            t.v[i] = __fmul_rn(t.v[i], gamma.v[i]);
        }
    } else if constexpr (SRC == kSrcSwiglu) {
        const Chunk u = values(in.y);
        // g u / (1 + 2^(-g log2 e)), two values per instruction but for the power and the reciprocal, which
        // flush subnormals: for g below -87.3 the power is infinite or its reciprocal 0, and the product 0,
        // its limit to within 1.1e-36 u (through __expf and __fdividef, which guard those ranges, the
        // kernel issued 25 instructions a value and took 101 us at 8192 x 14336 for 90).  The error, in
        // units U = 2^-24 of t and with e = 2^(-g log2 e): the constant is 0.224 U off and its product rounded,
        // so e is 1.224 |g| off; the power's own error is at most 2^-22, 4 U; both count e / (1 + e) in the
        // sum, which is rounded (1); the reciprocal's is at most 2^-23 (2); two products (2).
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const uint64_t g = pk2(t.v[i], t.v[i + 1]);
            float e0, e1, r0, r1;
            upk2(mul2(g, pk2(-1.44269504f, -1.44269504f)), e0, e1);
            asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e0));
            asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e1));
            upk2(add2(pk2(e0, e1), pk2(1.0f, 1.0f)), r0, r1);
            asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(r0));
            asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(r1));
            upk2(mul2(mul2(g, pk2(r0, r1)), pk2(u.v[i], u.v[i + 1])), t.v[i], t.v[i + 1]);
        }
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

// C values reduced over the lanes that differ in the bits below TOP (a power of two; C <= TOP), all at
// once: each of the first steps sends half of a lane's values to its partner and keeps the rest, so C
// values cost C - 1 + log2(TOP / C) + 1 shuffles rather than C log2(2 TOP).  The lane is left with value
// slot<C, TOP>(lane); lane lane_of<C, TOP>(i) (and others) with value i.  Each value's tree pairs lanes at
// distance TOP, then TOP / 2, ..., 1, whatever C.
template <int C, int TOP>
__device__ __forceinline__ int slot(int lane) {
    return C == 4 ? ((lane & TOP) ? 2 : 0) + ((lane & (TOP / 2)) ? 1 : 0) : C == 2 ? ((lane & TOP) ? 1 : 0) : 0;
}
template <int C, int TOP>
__device__ __forceinline__ int lane_of(int i) {
    return C == 4 ? (i >> 1) * TOP + (i & 1) * (TOP / 2) : C == 2 ? i * TOP : 0;
}
template <int C, int TOP, typename Op>
__device__ __forceinline__ float reduce(const float (&v)[C], int lane, Op&& op) {
    float r;
    int o = TOP;
    if constexpr (C == 4) {
        const bool u = lane & TOP, w = lane & (TOP / 2);
        const float a0 = op(u ? v[2] : v[0], __shfl_xor_sync(0xffffffffu, u ? v[0] : v[2], TOP));
        const float a1 = op(u ? v[3] : v[1], __shfl_xor_sync(0xffffffffu, u ? v[1] : v[3], TOP));
        r = op(w ? a1 : a0, __shfl_xor_sync(0xffffffffu, w ? a0 : a1, TOP / 2));
        o = TOP / 4;
    } else if constexpr (C == 2) {
        const bool u = lane & TOP;
        r = op(u ? v[1] : v[0], __shfl_xor_sync(0xffffffffu, u ? v[0] : v[1], TOP));
        o = TOP / 2;
    } else {
        r = v[0];
    }
#pragma unroll
    for (; o; o >>= 1) r = op(r, __shfl_xor_sync(0xffffffffu, r, o));
    return r;
}
struct Max {
    __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
struct Add {
    __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};

// e4m3 codes of the C groups that this half warp holds (16 lanes, 8 columns each; chunks past the row
// hold zeros).  The groups' largest magnitudes are reduced together, which leaves group
// slot<C, 8>(lane) with the lane: one pair of divisions for all C groups (a pair each, and C separate
// reductions, made the divisions a third of the kernel's instructions).  Returns that group's scale
// before the factor r.
template <int C>
__device__ __forceinline__ float e4m3_groups(const Chunk (&t)[C], uint2 (&codes)[C], int lane) {
    float m[C];
#pragma unroll
    for (int i = 0; i < C; ++i) m[i] = chunk_max(t[i]);
    const float mine = reduce<C, 8>(m, lane, Max());
    const bool live = mine >= 0x1p-100f;
    const float inv = live ? __fdiv_rn(448.0f, mine) : 0.0f;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const float f = __shfl_sync(0xffffffffu, inv, (lane & 16) | lane_of<C, 8>(i));
        float q[8];
#pragma unroll
        for (int e = 0; e < 8; e += 2) upk2(mul2(pk2(t[i].v[e], t[i].v[e + 1]), pk2(f, f)), q[e], q[e + 1]);
        codes[i].x = e4m3x2(q[0], q[1]) | (e4m3x2(q[2], q[3]) << 16);
        codes[i].y = e4m3x2(q[4], q[5]) | (e4m3x2(q[6], q[7]) << 16);
    }
    return live ? __fdiv_rn(mine, 448.0f) : 0.0f;
}

// INT8 codes of one chunk (as floats) into the API layout or a token record.
template <int FORM>
__device__ __forceinline__ void store_int8(const RowArgs& a, int64_t m, int64_t chunk, const float4& q0, const float4& q1) {
    if constexpr (FORM == kFormInt8) {
        *reinterpret_cast<uint2*>(a.a_q + m * a.K + 8 * chunk) = make_uint2(bytes4f(q0), bytes4f(q1));
    } else {
        const int ts = a.tw == 256 ? 8 : 7;
        const int r = static_cast<int>(m & ((1 << ts) - 1)), j = 2 * static_cast<int>(chunk & 7);
        uint8_t* rec = token_rec(a.trec, m, chunk >> 3, a.K / kBlock, ts);
        uint2 hi, lo;
        planes4f(q0, hi.x, lo.x);
        planes4f(q1, hi.y, lo.y);
        // quads j and j + 1 share a 16-byte chunk of the record (j is even): 8-byte stores
        *reinterpret_cast<uint2*>(rec + plane_off(r, j, 0)) = hi;
        *reinterpret_cast<uint2*>(rec + plane_off(r, j, 1)) = lo;
    }
}

// The sum of the codes of 64-block b of row m.
template <int FORM>
__device__ __forceinline__ void store_sum(const RowArgs& a, int64_t m, int64_t b, int rs) {
    const int64_t nb = a.K / kBlock;
    if constexpr (FORM == kFormInt8) {
        a.rowsum[m * nb + b] = rs;
    } else {
        const int ts = a.tw == 256 ? 8 : 7;
        *reinterpret_cast<uint4*>(token_rec(a.trec, m, b, nb, ts) + (128 << ts) + (m & ((1 << ts) - 1)) * 16) = rx_entry(rs);
    }
}

// The C chunks' INT8 codes and the sums of their 64-blocks (8 lanes each; exact: small integers).
template <int FORM, int C>
__device__ __forceinline__ void int8_codes(const RowArgs& a, int64_t m, bool row, int64_t c0, int64_t by, int lane,
                                           const Chunk (&t)[C], float s) {
    const float inv = __frcp_rn(s);
    const int64_t n8 = a.K / 8;
    float sums[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const float4 x[2] = {make_float4(t[i].v[0], t[i].v[1], t[i].v[2], t[i].v[3]),
                             make_float4(t[i].v[4], t[i].v[5], t[i].v[6], t[i].v[7])};
        float4 q[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
        if (s > 0.0f) quant_lane<2>(x, q, s, inv);
        const int64_t c = c0 + i * by;
        if (row && c < n8) store_int8<FORM>(a, m, c, q[0], q[1]);
        sums[i] = ((q[0].x + q[0].y) + (q[0].z + q[0].w)) + ((q[1].x + q[1].y) + (q[1].z + q[1].w));
    }
    const float rs = reduce<C, 4>(sums, lane, Add());
    const int64_t c = c0 + slot<C, 4>(lane) * by;  // a chunk of this lane's block
    if ((lane & (8 / C - 1)) == 0 && row && c < n8) store_sum<FORM>(a, m, c >> 3, static_cast<int>(rs));
}

// The maximum over the row's W warps.  Of the row's sum of squares, each warp holds C segment
// shares: sum[i] is its lanes' part of segment i W + wg, 256 columns of the row.  The total is
// taken over the segments' sums, segment j on lane j % 32, so it depends on the row alone and not
// on how its segments were dealt to warps: a row has the same bits in any batch.
// `red`: W maxima, then W C segment sums; only the row's warps meet.
template <int C, bool SUM, bool MAX>
__device__ __forceinline__ void row_reduce(float& amax, const float (&sum)[C], float& total, float* red, int wg, int W,
                                           int bar, int lane) {
    float seg = 0.0f, v = 0.0f;
    if (MAX) amax = reduce<1, 16>({amax}, lane, Max());
    if (SUM) seg = reduce<C, 16>(sum, lane, Add());  // of segment slot<C, 16>(lane)
    if (W == 1) {
        if (SUM) {
            v = __shfl_sync(0xffffffffu, seg, lane_of<C, 16>(lane & (C - 1)));
            if (lane >= C) v = 0.0f;
        }
    } else {
        if (MAX && lane == 0) red[wg] = amax;
        if (SUM && (lane & (32 / C - 1)) == 0) red[W + slot<C, 16>(lane) * W + wg] = seg;
        __syncwarp();  // named barriers take whole warps
        named_bar_sync(bar, W * 32);
        if (MAX) amax = reduce<1, 16>({lane < W ? red[lane] : 0.0f}, lane, Max());
        if (SUM)
            for (int j = lane; j < W * C; j += 32) v += red[W + j];
    }
    if (SUM) total = reduce<1, 16>({v}, lane, Add());
}

// One row (`row`: it exists), or its part from chunk `base` on, held by W warps, this one the wg-th:
// chunk base + (i W + wg) 32 + lane is input(i), its gamma gamma(i), i < C.  After `read()` the inputs
// are in registers (of every lane of this warp; the row's other warps meet in the reduction).
template <int SRC, int FORM, bool BF16, int C, typename Input, typename Gamma, typename Read>
__device__ __forceinline__ void work_row(const RowArgs& a, int64_t m, bool row, int64_t base, int W, int wg, int lane,
                                         float* red, int bar, Input&& input, Gamma&& gamma, Read&& read) {
    const int64_t n8 = a.K / 8, c0 = base + static_cast<int64_t>(wg) * 32 + lane, by = static_cast<int64_t>(W) * 32;
    Chunk t[C];
    float sum[C], amax = 0.0f, total = 0.0f;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int64_t c = c0 + i * by;
        sum[i] = 0.0f;
        if (row && c < n8) {
            source<SRC, BF16, true>(a, m, 8 * c, input(i), gamma(i), t[i], sum[i]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) t[i].v[e] = 0.0f;
        }
        if (FORM != kFormE4m3) amax = fmaxf(amax, chunk_max(t[i]));
    }
    if constexpr (FORM == kFormE4m3) {
        uint2 codes[C];
        const float s = e4m3_groups(t, codes, lane);
#pragma unroll
        for (int i = 0; i < C; ++i)
            if (row && c0 + i * by < n8) *reinterpret_cast<uint2*>(a.a_q + m * a.K + 8 * (c0 + i * by)) = codes[i];
        float r = 1.0f;
        if constexpr (SRC == kSrcNorm) {
            row_reduce<C, true, false>(amax, sum, total, red, wg, W, bar, lane);
            r = row_factor(total, a.K, a.eps);
        }
        read();
        const int64_t c = c0 - (lane & 15) + slot<C, 8>(lane) * by;  // the first chunk of this lane's group
        if ((lane & (16 / C - 1)) == 0 && row && c < n8) a.a_scale[(c >> 4) * a.M + m] = s * r;
    } else {
        row_reduce<C, SRC == kSrcNorm, true>(amax, sum, total, red, wg, W, bar, lane);
        read();
        const float s = __fdiv_rn(amax, 127.0f);
        if (row && wg == 0 && lane == 0) a.a_scale[m] = SRC == kSrcNorm ? s * row_factor(total, a.K, a.eps) : s;
        int8_codes<FORM, C>(a, m, row, c0, by, lane, t, s);
    }
}

// The forms whose scales do not span the row (e4m3 without a norm) are worked on in parts of 256 C
// columns, a warp each: blocks of any size then fit any row.
template <int SRC, int FORM>
constexpr bool kParts = SRC != kSrcNorm && FORM == kFormE4m3;

// Straight into registers: a row per W warps (or a part per warp, W = 1), blockDim / (32 W) of them a
// block; C chunks a lane (K <= 256 W C parts), all loaded before the first is worked on.
template <int SRC, int FORM, bool BF16, int C>
__global__ void __launch_bounds__(512) row_quant_kernel(const RowArgs a, int W, int parts) {
    griddep_launch_dependents();
    __shared__ float slots[16 * (1 + C)];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rsub = warp / W, wg = warp - rsub * W;
    int64_t m = static_cast<int64_t>(blockIdx.x) * ((blockDim.x >> 5) / W) + rsub, base = 0;
    if constexpr (kParts<SRC, FORM>) {
        const int64_t item = m;
        m = item / parts;
        base = (item - m * parts) * (32 * C);
    }
    const int64_t n8 = a.K / 8, c0 = base + static_cast<int64_t>(wg) * 32 + lane, by = static_cast<int64_t>(W) * 32;
    const bool row = m < a.M;  // the same for every warp of a row
    griddep_wait();
    Inputs<SRC, BF16> in[C];
#pragma unroll
    for (int i = 0; i < C; ++i)
        if (row && c0 + i * by < n8) load_inputs<SRC, BF16>(a, m, 8 * (c0 + i * by), in[i]);
    work_row<SRC, FORM, BF16, C>(
        a, m, row, base, W, wg, lane, slots + rsub * W * (1 + C), 1 + rsub, [&](int i) { return in[i]; },
        [&](int i) { return load_gamma<SRC>(a, 8 * (c0 + i * by)); }, [] {});
}

// Many bf16 rows of a norm: they come through shared memory, copied by the async engine `stages` rows ahead
// of each group of W warps, so that the bytes in flight neither cost registers nor stop while a row is worked
// on.  A group walks rows m, m + groups, ...; its first thread refills a stage once the group has read
// it.  gamma stays in registers.  Shared memory: [group][stage][x | residual][K], then a barrier per stage.
template <int FORM>
__global__ void __launch_bounds__(512) row_stream_kernel(const RowArgs a, int W, int stages) {
    griddep_launch_dependents();
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr int C = 4, kEl = 2;
    __shared__ float slots[2][16 * (1 + C)];
    __shared__ uint32_t abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rsub = warp / W, wg = warp - rsub * W, rpc = static_cast<int>(blockDim.x >> 5) / W;
    const bool two = a.residual != nullptr;
    const uint32_t bytes = static_cast<uint32_t>(a.K) * kEl, stage_bytes = bytes * (two ? 2 : 1);
    uint8_t* ring = smem + static_cast<uint32_t>(rsub * stages) * stage_bytes;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + static_cast<uint32_t>(rpc * stages) * stage_bytes) + rsub * stages;
    const WaitCtl ctl{&abort_flag, a.status, 1000000000ull};
    if (threadIdx.x == 0) {
        for (int i = 0; i < rpc * stages; ++i) mbar_init(full + i, 1);
        abort_flag = 0u;
        fence_barrier_init();
    }
    __syncthreads();
    griddep_wait();
    const int64_t first = static_cast<int64_t>(blockIdx.x) * rpc + rsub, step = static_cast<int64_t>(gridDim.x) * rpc;
    const int64_t n8 = a.K / 8;
    const bool leader = wg == 0 && lane == 0;
    auto fill = [&](int64_t m, int s) {
        mbar_arrive_expect_tx(full + s, stage_bytes);
        bulk_load(ring + s * stage_bytes, static_cast<const uint8_t*>(a.x) + m * a.ld * kEl, bytes, full + s);
        if (two)
            bulk_load(ring + s * stage_bytes + bytes, static_cast<const uint8_t*>(a.residual) + m * a.K * kEl, bytes, full + s);
    };
    if (leader)
        for (int s = 0; s < stages && first + s * step < a.M; ++s) fill(first + s * step, s);
    Chunk gamma[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int64_t c = static_cast<int64_t>(i * W + wg) * 32 + lane;
        if (c < n8) gamma[i] = load_gamma<kSrcNorm>(a, 8 * c);
    }
    // after a wait gave up the rest of the rows is worked on as it is (the status word says so); the
    // stages in flight are left to land below
    bool ok = true;
    int s = 0, par = 0;
    uint32_t phase = 0;
    for (int64_t m = first; m < a.M; m += step, par ^= 1) {
        if (ok) ok = mbar_wait(full + s, phase, ctl);
        __syncwarp();
        const uint8_t* st = ring + s * stage_bytes;
        work_row<kSrcNorm, FORM, true, C>(
            a, m, true, 0, W, wg, lane, slots[par] + rsub * W * (1 + C), 1 + rsub,
            [&](int i) {
                const uint32_t at = static_cast<uint32_t>((i * W + wg) * 32 + lane) * 8 * kEl;
                Inputs<kSrcNorm, true> in;
                in.x.w[0] = *reinterpret_cast<const uint4*>(st + at);
                if (two) in.y.w[0] = *reinterpret_cast<const uint4*>(st + bytes + at);
                return in;
            },
            [&](int i) { return gamma[i]; },
            [&] {
                // every warp of the row has read the stage (they met in the reduction): its next row may land
                if (W == 1) __syncwarp();
                if (leader && ok && m + stages * step < a.M) fill(m + stages * step, s);
            });
        if (++s == stages) s = 0, phase ^= 1u;
    }
    if (leader && !ok) {  // let what is in flight land (for a bounded time) before the block leaves
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 10000000ull) __nanosleep(1000);
    }
}

// Longer rows: a block of 32 warps walks its row twice, first for the maximum and the sum, then
// (from L2) for the codes.  The residual is stored on the second walk, after every read of it.  Bound by
// the second walk, which forms every value again: 4096 x 28672 bf16 gated activation to INT8 221 us, 40% of the
// copy rate on its bytes; 4096 x 20480 bf16 norm to e4m3 194 us, 45%.
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
        Inputs<SRC, BF16> in;
        load_inputs<SRC, BF16>(a, m, 8 * c, in);
        source<SRC, BF16, false>(a, m, 8 * c, in, load_gamma<SRC>(a, 8 * c), t, sum[0]);
        if (FORM != kFormE4m3) amax = fmaxf(amax, chunk_max(t));
    }
    row_reduce<1, true, true>(amax, sum, total, red, warp, 32, 1, lane);
    const float r = SRC == kSrcNorm ? row_factor(total, a.K, a.eps) : 1.0f;
    const float s = __fdiv_rn(amax, 127.0f);
    if (FORM != kFormE4m3 && threadIdx.x == 0) a.a_scale[m] = s * r;
    for (int64_t c0 = warp * 32; c0 < n8; c0 += 1024) {
        const int64_t c = c0 + lane;
        Chunk t;
        float unused = 0.0f;
        if (c < n8) {
            Inputs<SRC, BF16> in;
            load_inputs<SRC, BF16>(a, m, 8 * c, in);
            source<SRC, BF16, true>(a, m, 8 * c, in, load_gamma<SRC>(a, 8 * c), t, unused);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) t.v[e] = 0.0f;
        }
        const Chunk tt[1] = {t};
        if constexpr (FORM == kFormE4m3) {
            uint2 codes[1];
            const float sg = e4m3_groups(tt, codes, lane);
            if (c < n8) {
                *reinterpret_cast<uint2*>(a.a_q + m * a.K + 8 * c) = codes[0];
                if ((lane & 15) == 0) a.a_scale[(c >> 4) * a.M + m] = sg * r;
            }
        } else {
            int8_codes<FORM, 1>(a, m, true, c, 0, lane, tt, s);
        }
    }
}

template <typename... Args>
cudaError_t launch_pdl(void (*kernel)(Args...), int64_t grid, int threads, size_t smem, cudaStream_t s, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Blocks launched per SM of the streaming kernel (two are resident, by registers), and rows in flight a
// group.  Measured on 16384 x 4096 bf16 (us):
// two stages and 4 / 6 / 8 blocks 73.3 / 74.3 / 72.9, three stages (smaller blocks) 78.3, one 87.1; on
// 4096 x 14336 4 / 6 / 8 blocks 70.7 / 76.1 / 76.8.
constexpr int kStreamBlocks = 4, kStreamStages = 2;

template <int FORM>
cudaError_t run_stream(const RowArgs& a, int W, int rpc, int num_sms, cudaStream_t s) {
    static bool attr_done[64] = {};
    constexpr int kMost = 2 * 2 * 16384 * kStreamStages;  // the deepest row: bf16, two inputs, one row a block
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 64 && !attr_done[dev]) {
        const cudaError_t e =
            cudaFuncSetAttribute(row_stream_kernel<FORM>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost + 256);
        if (e != cudaSuccess) return e;
        attr_done[dev] = true;
    }
    const size_t stage = static_cast<size_t>(a.K) * 2 * (a.residual ? 2 : 1);
    const size_t smem = static_cast<size_t>(rpc * kStreamStages) * (stage + 8);
    const int64_t need = (a.M + rpc - 1) / rpc, cap = static_cast<int64_t>(num_sms) * kStreamBlocks;
    const int64_t rounds = (need + cap - 1) / cap;
    return launch_pdl(row_stream_kernel<FORM>, (need + rounds - 1) / rounds, rpc * W * 32, smem, s, a, W, kStreamStages);
}

template <int SRC, int FORM, bool BF16>
cudaError_t run(const RowArgs& a, int num_sms, cudaStream_t s) {
    const int64_t n8 = a.K / 8;
    if constexpr (!kParts<SRC, FORM>) {
        if (n8 > 16 * 32 * 4) {
            row_quant_long_kernel<SRC, FORM, BF16><<<static_cast<unsigned>(a.M), 1024, 0, s>>>(a);
            return cudaGetLastError();
        }
    }
    auto warps = [&](int C) { return static_cast<int>((n8 + 32 * C - 1) / (32 * C)); };
    // Chunks a lane.  One where its warps still fit the GPU at once (512 x 2048 bf16 to INT8: 3.5 us
    // against 4.5 with two and 5.4 with four).  Then, fp32: two (8192 x 4096 to e4m3: 66.5 us against
    // 70.9 with four), four where the row would need more than 16 warps; bf16: four (16384 x 4096:
    // 79.0 against 86.6 with two).
    constexpr bool any = kParts<SRC, FORM>;  // no limit of warps to a row
    const int64_t few = static_cast<int64_t>(num_sms) * 48;
    int C = 4;
    if ((any || warps(1) <= 16) && a.M * warps(1) <= few) C = 1;
    else if ((any || warps(2) <= 16) && (!BF16 || n8 <= 64 || a.M * warps(2) <= few)) C = 2;
    const int W = any ? 1 : warps(C), parts = any ? warps(C) : 1;
    const int rpc = W >= 8 ? 1 : 8 / W;
    if constexpr (SRC == kSrcNorm && BF16) {
        // Through shared memory where each group of warps has at least three rows of 2048 columns or
        // more: 16384 x 4096 to e4m3 79.0 -> 73.0 us, to INT8 86.1 -> 77.8, 16384 x 2048 42.0 -> 38.7,
        // 4096 x 14336 102 -> 70.8; but 16384 x 1024 22.7 -> 23.1, 4096 x 2048 14.6 -> 14.8, and fp32
        // (which registers already carry at the copy rate) 66.5 -> 68.5.
        if (C == 4 && a.K >= 2048 && a.M >= static_cast<int64_t>(3 * kStreamBlocks) * num_sms * rpc)
            return run_stream<FORM>(a, W, rpc, num_sms, s);
    }
    const int64_t grid = (a.M * parts + rpc - 1) / rpc;
    if (grid > 2147483647LL) return cudaErrorInvalidValue;
    switch (C) {
        case 1: return launch_pdl(row_quant_kernel<SRC, FORM, BF16, 1>, grid, rpc * W * 32, 0, s, a, W, parts);
        case 2: return launch_pdl(row_quant_kernel<SRC, FORM, BF16, 2>, grid, rpc * W * 32, 0, s, a, W, parts);
        default: return launch_pdl(row_quant_kernel<SRC, FORM, BF16, 4>, grid, rpc * W * 32, 0, s, a, W, parts);
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

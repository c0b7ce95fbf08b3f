// rope_kv.cu -- rotary positions, and the 8-bit cache of keys and values: written (keys rotated on the
// way) and read back.
//
// Rotary positions: pair i of a head is turned by positions[t] * f_i.  An fp32 product loses the angle of
// far positions (position 10^6 at one radian each: an error of 0.06), and fp64 runs at 1/64 of the
// rate here.  So the frequency is kept as a 64-bit fraction of a turn: position * turns modulo 2^64 is the
// angle's fraction of a turn, exactly, in one integer product; whole turns fall off the top.  The
// top two bits pick the quarter, the signed rest is at most 1/8 turn and goes through sincospi in fp32.
//
// The cache: each token's head is one row of 8-bit codes with one scale, so that a product over the head
// factors it out.  The largest magnitude is a maximum over the 4 or 8 threads that hold the row.
//
// What bounds them: HBM for long inputs, a chain of position -> angle -> sincospi -> rotation for one
// token.  Sines and cosines are shared by all heads of a token, so a block forms them once in shared
// memory, while its rows' loads are in flight.
//
// Measured (GPU time alone): 16384 tokens of 32 heads of 128 bf16 41 us, 6.5 TB/s, the copy rate; one token of 16 heads 1.7 us;
// 8191 tokens of 32 + 8 + 8 heads rotated and written as e4m3 50 us, 4.7 TB/s (issue slots 64 %, the rest waits at the block's
// barrier and for loads, with 30 warps an SM); 131071 tokens of 8 heads read back 138 us, 5.9 TB/s.  Not faster: one
// block working through tokens with the next one's loads ahead (the write 64 us, at 80 registers a thread for 64).
#include "attn_internal.h"
#include "quant_math.cuh"
#include "sm103_ptx.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

namespace w4a8 {
namespace {

constexpr int kThreads = 128;
constexpr int kMostThreads = 256;  // of the rotary kernel: 128 to 256, by a token's items
constexpr int kPerThread = 2;      // items of 16 values a thread holds

struct RotaryParams {
    RotaryArgs a;
    int per_head;      // items of a head: head_dim / 16
    int items;         // of a token: all heads
    int block_tokens;  // tokens of a block
    int page_shift;
    // 2^32 / per_head and, for blocks of several tokens, 2^32 / items, rounded up: a number below 2^20 times the first, below 2^16
    // times the second has the quotient in its upper half
    uint32_t head_inverse, token_inverse;
};

__device__ __forceinline__ int quotient(int v, int by, uint32_t inverse) {
    return by == 1 ? v : static_cast<int>(__umulhi(static_cast<uint32_t>(v), inverse));
}

// cos and sin of the turn fraction, times magnitude.
__device__ __forceinline__ float2 turn(int32_t position, uint64_t turns, float magnitude) {
    const uint64_t phase = static_cast<uint64_t>(static_cast<int64_t>(position)) * turns;
    const uint64_t quarter = (phase + (1ull << 61)) >> 62;  // nearest quarter turn (mod 4)
    const int64_t rest = static_cast<int64_t>(phase - (quarter << 62));  // within 1/8 turn
    float s, c;
    // the top 32 of the rest's bits, in half turns: exact but for fp32's own 24 bits
    sincospif(static_cast<float>(static_cast<int32_t>(rest >> 32)) * 0x1p-31f, &s, &c);
    if (quarter & 1) {
        const float t = c;
        c = -s;
        s = t;
    }
    if (quarter & 2) {
        c = -c;
        s = -s;
    }
    return make_float2(c * magnitude, s * magnitude);
}

// A pair turned; the roundings are spelt out, so that every form gives the same bits.
__device__ __forceinline__ void rotate(float& x0, float& x1, float c, float s) {
    const float y0 = __fmaf_rn(x0, c, -__fmul_rn(x1, s));
    x1 = __fmaf_rn(x1, c, __fmul_rn(x0, s));
    x0 = y0;
}

// 8 values as loaded: 16 bytes of bf16 or 32 of fp32.
template <bool BF16>
struct Chunk {
    uint4 r[BF16 ? 1 : 2];
    __device__ __forceinline__ void load(const char* p) {
        r[0] = *reinterpret_cast<const uint4*>(p);
        if constexpr (!BF16) r[1] = *reinterpret_cast<const uint4*>(p + 16);
    }
    __device__ __forceinline__ void get(float* x) const {
        if constexpr (BF16) {
            const uint32_t w[4] = {r[0].x, r[0].y, r[0].z, r[0].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        } else {
            const uint32_t w[8] = {r[0].x, r[0].y, r[0].z, r[0].w, r[1].x, r[1].y, r[1].z, r[1].w};
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
        }
    }
};

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

template <bool BF16>
__device__ __forceinline__ void put(char* p, const float* x) {
    if constexpr (BF16) {
        *reinterpret_cast<uint4*>(p) =
            make_uint4(bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]), bf16_pair(x[4], x[5]), bf16_pair(x[6], x[7]));
    } else {
        *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<float4*>(p + 16) = make_float4(x[4], x[5], x[6], x[7]);
    }
}

__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
    return d;
}

// The codes of 16 values of a row whose largest magnitude over its threads is `amax`, NaN if one is; all lanes of a warp.
// A row with an element that is no finite number has none that its codes could hold: codes 0 and scale NaN.
__device__ __forceinline__ void codes16(const float (&x)[16], float amax, int format, uint32_t (&code)[4], float& scale) {
    const bool live = amax >= 0x1p-100f && amax < INFINITY;
    scale = amax < INFINITY ? 0.0f : __int_as_float(0x7fffffff);
    if (format == W4A8_KV_E4M3) {
        if (live) scale = __fdiv_rn(amax, 448.0f);
        const float inv = live ? __fdiv_rn(448.0f, amax) : 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            code[i] = live ? e4m3_pair(x[4 * i] * inv, x[4 * i + 1] * inv) | e4m3_pair(x[4 * i + 2] * inv, x[4 * i + 3] * inv) << 16 : 0u;
        return;
    }
    if (live) scale = __fdiv_rn(amax, 127.0f);
    const float s = live ? scale : 1.0f;
    float4 v[4], q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
    quant_lane<4>(v, q, s, __frcp_rn(s));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        code[i] = (static_cast<uint32_t>(static_cast<int>(q[i].x)) & 0xffu) |
                  (static_cast<uint32_t>(static_cast<int>(q[i].y)) & 0xffu) << 8 |
                  (static_cast<uint32_t>(static_cast<int>(q[i].z)) & 0xffu) << 16 |
                  static_cast<uint32_t>(static_cast<int>(q[i].w)) << 24;
        if (!live) code[i] = 0;
    }
}

// One item: 16 values of a head, as two chunks of 8 that meet in the rotation: pairs of halves take chunk
// c and the one rot / 2 further on; neighbours, and values that pass, chunks side by side.
template <bool BF16, bool CACHE>
__global__ void __launch_bounds__(kMostThreads, BF16 ? 4 : 3) rotary_kernel(const RotaryParams p) {
    extern __shared__ float cs[];  // [block token][cos of rot / 2 pairs, sin of them]
    constexpr int EL = BF16 ? 2 : 4;
    const RotaryArgs& a = p.a;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.block_tokens;
    const int nt = static_cast<int>(min(static_cast<int64_t>(p.block_tokens), a.tokens - t0));
    const int threads = blockDim.x, held = threads * kPerThread;
    const int first = blockIdx.y * held;  // only where a token has more items than a block holds
    const int count = min(nt * p.items - first, held);
    const int pairs = a.turns ? a.rot / 2 : 0;

    Chunk<BF16> raw[kPerThread][2];
    int at[kPerThread][2], head[kPerThread], tok[kPerThread];
#pragma unroll
    for (int u = 0; u < kPerThread; ++u) {
        const int i = threadIdx.x + u * threads;
        head[u] = -1;
        if (i < count) {
            tok[u] = p.block_tokens == 1 ? 0 : quotient(i, p.items, p.token_inverse);
            const int j = (first + i) - tok[u] * p.items;
            head[u] = quotient(j, p.per_head, p.head_inverse);
            const int c = j - head[u] * p.per_head;
            const bool halves = pairs && !a.interleaved && 8 * c < pairs && head[u] < a.q_heads + (CACHE ? static_cast<int>(a.cache.heads) : 0);
            at[u][0] = halves ? 8 * c : 16 * c;
            at[u][1] = halves ? 8 * c + pairs : 16 * c + 8;
            const HeadRows* src = &a.q;
            int h = head[u];
            if (CACHE && h >= a.q_heads) {
                h -= a.q_heads;
                src = &a.k;
                if (h >= a.cache.heads) {
                    h -= static_cast<int>(a.cache.heads);
                    src = &a.v;
                }
            }
            const char* row = static_cast<const char*>(src->p) + ((t0 + tok[u]) * src->token + h * src->head) * EL;
            raw[u][0].load(row + at[u][0] * EL);
            raw[u][1].load(row + at[u][1] * EL);
        }
    }
    for (int i = threadIdx.x; i < nt * pairs; i += threads) {
        const int t = p.block_tokens == 1 ? 0 : i / pairs, f = i - t * pairs;
        const float2 v = turn(a.positions[t0 + t], a.turns[f], a.magnitude);
        cs[t * 2 * pairs + f] = v.x;
        cs[t * 2 * pairs + pairs + f] = v.y;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kPerThread; ++u) {
        const bool on = head[u] >= 0;
        float x[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = 0.0f;
        int h = head[u], kind = 0;  // 0 q, 1 k, 2 v
        if (on) {
            raw[u][0].get(x);
            raw[u][1].get(x + 8);
            if (CACHE && h >= a.q_heads) {
                h -= a.q_heads;
                kind = 1;
                if (h >= a.cache.heads) {
                    h -= static_cast<int>(a.cache.heads);
                    kind = 2;
                }
            }
            const int c = a.interleaved || at[u][1] == at[u][0] + 8 ? at[u][0] / 2 : at[u][0];  // its first pair
            if (kind != 2 && c < pairs) {
                const float* cosp = cs + tok[u] * 2 * pairs + c;
                const float* sinp = cosp + pairs;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (a.interleaved) rotate(x[2 * e], x[2 * e + 1], cosp[e], sinp[e]);
                    else rotate(x[e], x[e + 8], cosp[e], sinp[e]);
                }
            }
            if (kind == 0) {
                char* row = static_cast<char*>(const_cast<void*>(a.q_out.p)) +
                            ((t0 + tok[u]) * a.q_out.token + h * a.q_out.head) * EL;
                put<BF16>(row + at[u][0] * EL, x);
                put<BF16>(row + at[u][1] * EL, x + 8);
            }
        }
        if constexpr (CACHE) {
            if (!__any_sync(0xffffffffu, on && kind != 0)) continue;  // a warp of queries
            float amax = 0.0f;
#pragma unroll
            for (int e = 0; e < 16; ++e) amax = max_nan(amax, fabsf(x[e]));
            for (int d = p.per_head >> 1; d > 0; d >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, d));
            uint32_t code[4];
            float scale;
            codes16(x, amax, a.cache.format, code, scale);
            if (on && kind != 0) {
                const int64_t slot = a.slots[t0 + tok[u]];
                const int64_t all = a.cache.pages * a.cache.page;
                if (slot >= all) {
                    atomicOr(a.status, kStatusIndex);
                } else if (slot >= 0) {
                    const int64_t page = slot >> p.page_shift, off = slot - (page << p.page_shift);
                    const int64_t row = ((page * a.cache.heads + h) << p.page_shift) + off;
                    uint8_t* dst = (kind == 1 ? a.cache.k : a.cache.v) + row * a.head_dim;
                    *reinterpret_cast<uint2*>(dst + at[u][0]) = make_uint2(code[0], code[1]);
                    *reinterpret_cast<uint2*>(dst + at[u][1]) = make_uint2(code[2], code[3]);
                    if (at[u][0] == 0) (kind == 1 ? a.cache.k_scale : a.cache.v_scale)[row] = scale;
                }
            }
        }
    }
}

// Any layout: a thread turns one pair, or passes one value.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) rotary_pairs_kernel(const RotaryArgs a) {
    const int pairs = a.rot / 2, each = a.head_dim - pairs;  // pairs, then passing values, of a head
    const int i = blockIdx.y * kThreads + threadIdx.x;
    if (i >= a.q_heads * each) return;
    const int h = i / each, j = i - h * each;
    const int64_t t = blockIdx.x;
    using T = typename std::conditional<BF16, __nv_bfloat16, float>::type;
    const T* x = static_cast<const T*>(a.q.p) + t * a.q.token + h * a.q.head;
    T* y = static_cast<T*>(const_cast<void*>(a.q_out.p)) + t * a.q_out.token + h * a.q_out.head;
    if (j >= pairs) {
        y[pairs + j] = x[pairs + j];
        return;
    }
    const int e0 = a.interleaved ? 2 * j : j, e1 = a.interleaved ? 2 * j + 1 : j + pairs;
    const float2 cs = turn(a.positions[t], a.turns[j], a.magnitude);
    float x0 = static_cast<float>(x[e0]), x1 = static_cast<float>(x[e1]);
    rotate(x0, x1, cs.x, cs.y);
    y[e0] = static_cast<T>(x0);
    y[e1] = static_cast<T>(x1);
}

// ---------------------------------------------------------------- reading back
constexpr int kReadPerThread = 4;

// 16 codes a step: values code * scale in fp32, rounded once.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const w4a8_kv_cache c, int page_shift, const int64_t* slots, int64_t tokens,
                                                           void* k_out, void* v_out, uint32_t* status) {
    const bool is_v = k_out == nullptr || blockIdx.y == 1;
    char* out = static_cast<char*>(is_v ? v_out : k_out);
    const uint8_t* codes = is_v ? c.v : c.k;
    const float* scales = is_v ? c.v_scale : c.k_scale;
    const uint32_t per_head = static_cast<uint32_t>(c.head_dim) / 16, per_token = per_head * static_cast<uint32_t>(c.heads);
    const int64_t items = tokens * per_token, base = static_cast<int64_t>(blockIdx.x) * kReadPerThread * kThreads;
    const int64_t t0 = base / per_token;
    const uint32_t rest = static_cast<uint32_t>(base - t0 * per_token);
    uint4 raw[kReadPerThread];
    float scale[kReadPerThread];
    int64_t slot[kReadPerThread];
    uint32_t item[kReadPerThread];
#pragma unroll
    for (int u = 0; u < kReadPerThread; ++u) {
        const uint32_t v = rest + u * kThreads + threadIdx.x, t = v / per_token;
        item[u] = v - t * per_token;
        slot[u] = base + u * kThreads + threadIdx.x < items ? slots[t0 + t] : -1;
    }
#pragma unroll
    for (int u = 0; u < kReadPerThread; ++u) {
        raw[u] = make_uint4(0, 0, 0, 0);
        scale[u] = 0.0f;
        if (slot[u] >= c.pages << page_shift) {
            atomicOr(status, kStatusIndex);
        } else if (slot[u] >= 0) {
            const uint32_t h = per_head == 8 ? item[u] >> 3 : item[u] >> 2;
            const int64_t page = slot[u] >> page_shift;
            const int64_t row = ((page * c.heads + h) << page_shift) + (slot[u] - (page << page_shift));
            raw[u] = *reinterpret_cast<const uint4*>(codes + row * c.head_dim + 16 * (item[u] - h * per_head));
            scale[u] = scales[row];
        }
    }
#pragma unroll
    for (int u = 0; u < kReadPerThread; ++u) {
        const int64_t i = (static_cast<int64_t>(blockIdx.x) * kReadPerThread + u) * kThreads + threadIdx.x;
        if (i >= items) continue;
        const uint32_t w[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
        float x[16];
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
            const uint32_t two = (w[e / 4] >> (8 * (e % 4))) & 0xffffu;
            if (c.format == W4A8_KV_E4M3) {
                uint32_t h2;
                asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(two)));
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
                x[e] = f.x * scale[u];
                x[e + 1] = f.y * scale[u];
            } else {
                x[e] = static_cast<float>(static_cast<int8_t>(two & 0xffu)) * scale[u];
                x[e + 1] = static_cast<float>(static_cast<int8_t>(two >> 8)) * scale[u];
            }
        }
        char* dst = out + i * 16 * (BF16 ? 2 : 4);
        put<BF16>(dst, x);
        put<BF16>(dst + 8 * (BF16 ? 2 : 4), x + 8);
    }
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, int num_sms, cudaStream_t s) {
    RotaryParams p;
    p.a = a;
    p.per_head = a.head_dim / 16;
    p.items = (a.q_heads + 2 * static_cast<int>(a.cache.heads)) * p.per_head;
    // whole tokens for each block as long as every SM gets two of them
    const int64_t even = a.tokens / (2 * num_sms);
    // a token's items in one block where they fit: 32 + 16 heads of 128 values are 192 threads
    const int threads = std::min(kMostThreads, std::max(kThreads, (p.items / kPerThread + 31) / 32 * 32)), held = threads * kPerThread;
    p.block_tokens = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(held / p.items, even)));
    const int parts = p.items > held ? (p.items + held - 1) / held : 1;
    p.page_shift = 0;
    while ((1ll << p.page_shift) < a.cache.page) ++p.page_shift;
    p.head_inverse = 0xffffffffu / static_cast<uint32_t>(p.per_head) + 1;
    p.token_inverse = 0xffffffffu / static_cast<uint32_t>(p.items) + 1;
    const dim3 grid(static_cast<unsigned>((a.tokens + p.block_tokens - 1) / p.block_tokens), parts);
    const size_t smem = a.turns ? static_cast<size_t>(p.block_tokens) * a.rot * sizeof(float) : 0;
    const bool cache = a.cache.heads > 0;
    if (a.bf16) {
        if (cache) rotary_kernel<true, true><<<grid, threads, smem, s>>>(p);
        else rotary_kernel<true, false><<<grid, threads, smem, s>>>(p);
    } else {
        if (cache) rotary_kernel<false, true><<<grid, threads, smem, s>>>(p);
        else rotary_kernel<false, false><<<grid, threads, smem, s>>>(p);
    }
    return cudaGetLastError();
}

cudaError_t launch_rotary_pairs(const RotaryArgs& a, cudaStream_t s) {
    const int each = a.head_dim - a.rot / 2;
    const dim3 grid(static_cast<unsigned>(a.tokens), static_cast<unsigned>((a.q_heads * each + kThreads - 1) / kThreads));
    if (a.bf16) rotary_pairs_kernel<true><<<grid, kThreads, 0, s>>>(a);
    else rotary_pairs_kernel<false><<<grid, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_kv_read(const w4a8_kv_cache& c, const int64_t* slots, int64_t tokens, void* k_out, void* v_out,
                           bool bf16, uint32_t* status, cudaStream_t s) {
    const int64_t items = tokens * c.heads * (c.head_dim / 16);
    const dim3 grid(static_cast<unsigned>((items + kThreads * kReadPerThread - 1) / (kThreads * kReadPerThread)),
                    k_out && v_out ? 2 : 1);
    int shift = 0;
    while ((1ll << shift) < c.page) ++shift;
    if (bf16) kv_read_kernel<true><<<grid, kThreads, 0, s>>>(c, shift, slots, tokens, k_out, v_out, status);
    else kv_read_kernel<false><<<grid, kThreads, 0, s>>>(c, shift, slots, tokens, k_out, v_out, status);
    return cudaGetLastError();
}

}  // namespace w4a8

// attn_common.cuh -- what the attention kernels share: their arguments, a sequence's lengths and keys,
// number helpers.
#pragma once

#include "attn_internal.h"
#include "kv_codes.cuh"
#include "sm103_ptx.cuh"

namespace w4a8 {

struct AttnParams {
    // few rows: the code arrays as [pages * heads * page][head_dim] bytes; many rows, expanded ahead: k16 and v16
    CUtensorMap kmap, vmap;
    const uint8_t* k;
    const uint8_t* v;
    const void* q;
    void* out;
    int64_t q_token, q_head, out_token, out_head;
    const float* k_scale;
    const float* v_scale;
    const int32_t* page_table;
    const int32_t* kv_len;
    const int32_t* q_start;
    int64_t table_stride, total, pages;
    int heads, group, page_shift;
    int box;  // few rows: rows of a TMA box, 16 or 32
    int max_q, window, sinks;
    int q_bf16, out_bf16;
    float c;  // scale * log2(e)
    // many rows, expanded ahead: [batch][heads][step_cap][128][head_dim] fp16, and a step's 2^E of keys, E and 2^-E of values
    uint16_t* k16;
    uint16_t* v16;
    float4* step_info;
    int step_cap;  // 0: expanded inside
    int batch, max_kv;
    int row_tiles, splits;  // many rows: runs of an item's keys; few rows: CTAs
    int item_cost;          // few rows: what an item costs a CTA beside its keys, in units of keys
    int cluster;            // few rows: CTAs of an item, a cluster; 0: the items' keys are dealt out
    // what is left to join, [slot][rows][head_dim] sums and [slot][rows] references and sums of weights (m, l); a slot:
    // many rows: an item's run; few rows: a CTA's first or last run
    float* part;
    float2* part_ml;
    int4* info;  // few rows, [CTA]: its first run's sequence and head, its first unit in the item, the item's units; then units of a CTA
    uint32_t* status;
    uint64_t wait_limit_ns;
};

// One sequence as the kernels see it: lengths held to the arrays.
struct Seq {
    int first;  // row of q
    int n, kv;
    int pos;    // position of its first query
};

__device__ __forceinline__ Seq sequence(const AttnParams& p, int b) {
    Seq s;
    bool bad = false;
    const int64_t room = p.table_stride << p.page_shift;
    int64_t kv = __ldcg(p.kv_len + b);
    const int64_t most = p.max_kv < room ? p.max_kv : room;
    if (kv < 0 || kv > most) {
        bad = true;
        kv = kv < 0 ? 0 : most;
    }
    int64_t lo = b, hi = b + 1;
    if (p.q_start) {
        lo = __ldcg(p.q_start + b);
        hi = __ldcg(p.q_start + b + 1);
    }
    if (lo < 0 || hi < lo || hi > p.total) {
        bad = true;
        lo = hi = 0;
    }
    s.pos = static_cast<int>(kv - (hi - lo));
    if (hi - lo > p.max_q) {  // the last ones are left out
        bad = true;
        hi = lo + p.max_q;
    }
    if (bad) atomicOr(p.status, kStatusIndex);
    s.first = static_cast<int>(lo);
    s.n = static_cast<int>(hi - lo);
    s.kv = static_cast<int>(kv);
    return s;
}

__device__ __forceinline__ uint32_t half_pair(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ bool finite(float v) { return fabsf(v) < INFINITY; }
constexpr uint32_t kBitsInf = 0x7f800000u;  // bits of a number >= 0 from here on: infinity, NaN
__device__ __forceinline__ float not_a_number() { return __int_as_float(0x7fffffff); }

// The exponent e of v >= 0, and 2^-e; `none` where v has none (0, or past the normal numbers).
__device__ __forceinline__ void exponent_of(float v, int none, float& e, float& inv) {
    int ex = static_cast<int>(__float_as_uint(v) >> 23);
    if (ex <= 0 || ex >= 254) ex = 127 + none;
    e = static_cast<float>(ex - 127);
    inv = __uint_as_float(static_cast<uint32_t>(254 - ex) << 23);
}

// A row of q, of largest magnitude `most`, is multiplied by `up`, a power of two, and its logits by 2^e: the largest magnitude
// comes to [2^8, 2^9), where fp16 keeps what is 2^-33 of it and a dot product stays below 2^24.  Exponents are held to
// -119 .. 126, where `up` and its inverse's power are numbers: below, rows come to less than 2^8, at 2^127 to less than 2^10.  `up`
// is NaN for a row with an infinity, whose logits would otherwise all be -inf where the codes it meets are of the other sign,
// as if it saw nothing.
__device__ __forceinline__ void query_factor(float most, float& e, float& up) {
    const int ex = min(max(static_cast<int>(__float_as_uint(most) >> 23), 8), 253);
    e = static_cast<float>(ex - 127 - 8);
    up = most == INFINITY ? not_a_number() : __uint_as_float(static_cast<uint32_t>(254 + 8 - ex) << 23);
}

// A run's reference as its join reads it, which passes over runs that saw nothing (-inf): not over one whose weights are NaN.
__device__ __forceinline__ float held_reference(float m, float l) { return l == l ? m : l; }

// The keys of a row tile whose positions span p_min .. p_max: runs of `step` from 0 (the sinks') and from the
// window's start on.
struct Keys {
    int step, sink_steps, wide, steps;
    __device__ __forceinline__ int first(int i) const { return (i < sink_steps ? i : wide + i - sink_steps) * step; }
    // which of the steps begins at key run * step
    __device__ __forceinline__ int index(int run) const { return run < sink_steps ? run : sink_steps + run - wide; }
};

__device__ __forceinline__ Keys key_steps(const AttnParams& p, int p_min, int p_max, int step) {
    Keys k;
    k.step = step;
    const int end = p_max + 1;  // keys
    int lo = 0;
    if (p.window > 0 && p_min >= p.window) lo = p_min - p.window + 1;
    const int last = end > 0 ? (end + step - 1) / step : 0;
    k.wide = lo / step;
    k.sink_steps = min((min(p.sinks, lo) + step - 1) / step, k.wide);
    k.steps = max(0, last - k.wide) + k.sink_steps;
    return k;
}

// Whether every row at p_min .. p_max sees all of the keys j0 .. j0 + count - 1.
__device__ __forceinline__ bool all_see(const AttnParams& p, int p_min, int p_max, int j0, int count) {
    return j0 + count - 1 <= p_min && (p.window == 0 || j0 > p_max - p.window || j0 + count <= p.sinks);
}
// Whether some row does see key j: the cache's place of one that none sees may hold anything.
__device__ __forceinline__ bool some_see(const AttnParams& p, int p_min, int p_max, int j) {
    return j <= p_max && (p.window == 0 || j > p_min - p.window || j < p.sinks);
}

// The page of key j of sequence b, as the table has it; and the key's row in the cache's arrays, page 0's in the place of a
// page outside the cache, which is recorded.
__device__ __forceinline__ int page_of(const AttnParams& p, int b, int j) {
    return p.page_table[b * p.table_stride + (j >> p.page_shift)];
}
__device__ __forceinline__ int row_in(const AttnParams& p, int page, int kvh, int j) {
    if (page < 0 || page >= p.pages) {
        atomicOr(p.status, kStatusIndex);
        page = 0;
    }
    return ((page * p.heads + kvh) << p.page_shift) + (j & ((1 << p.page_shift) - 1));
}
__device__ __forceinline__ int cache_row(const AttnParams& p, int b, int kvh, int j) { return row_in(p, page_of(p, b, j), kvh, j); }

}  // namespace w4a8

// attn_internal.h -- declarations of the operators between the q/k/v projections and the output
// projection: rotary positions and the 8-bit cache (rope_kv.cu), attention (attn_plan.cu, attn_few.cu,
// attn_rows.cu), and what their C entry points (attn_api.cu) hand them.
#pragma once

#include "../../include/w4a8.h"
#include "ops_internal.h"

namespace w4a8 {

// ---------------------------------------------------------------- rotary positions and the cache
// Rows of heads in memory: element d of head h of token t at t * token + h * head + d.
struct HeadRows {
    const void* p = nullptr;
    int64_t token = 0, head = 0;
};

struct RotaryArgs {
    HeadRows q, k, v, q_out;  // w4a8_rope: q and q_out alone
    bool bf16 = false;
    const int32_t* positions = nullptr;
    const uint64_t* turns = nullptr;  // null: nothing is rotated
    int rot = 0;
    bool interleaved = false;
    float magnitude = 1.0f;
    int64_t tokens = 0;
    int q_heads = 0, head_dim = 0;
    const int64_t* slots = nullptr;
    w4a8_kv_cache cache{};  // heads == 0: no cache
    uint32_t* status = nullptr;
};

cudaError_t launch_rotary(const RotaryArgs& a, int num_sms, cudaStream_t s);        // 16-byte accesses, rot and head_dim of whole 16s
cudaError_t launch_rotary_pairs(const RotaryArgs& a, cudaStream_t s);               // any layout, q alone
cudaError_t launch_kv_read(const w4a8_kv_cache& c, const int64_t* slots, int64_t tokens, void* k_out, void* v_out,
                           bool bf16, uint32_t* status, cudaStream_t s);

// ---------------------------------------------------------------- attention
// How a call's work is cut: a CTA takes `rows` rows (query, head of a group) of a sequence and cache head.
// Many rows: `splits` CTAs share their keys; few: `splits` CTAs share all sequences' and heads' keys.
struct AttnPlan {
    int rows = 8;
    int row_tiles = 1;
    int splits = 1;
    int cluster = 0;       // few: CTAs (a cluster) for each sequence and cache head, nothing left to join (0: dealt out)
    int step_cap = 0;      // many rows: steps of 128 keys expanded ahead, of each sequence and head (0: inside)
    size_t expand_at = 0;  // where they begin in the workspace
    size_t bytes = 0;      // workspace
};

constexpr int kRowTile = 256;  // rows of a CTA of the form for many rows

AttnPlan plan_attention(const w4a8_kv_cache& c, const w4a8_attention_args& a);
// What suffices for every call within the bounds of `a`.
size_t bound_attention(const w4a8_kv_cache& c, const w4a8_attention_args& a);
cudaError_t launch_attention(const w4a8_kv_cache& c, const w4a8_attention_args& a, const AttnPlan& p, void* ws,
                             uint32_t* status, cudaStream_t s);

struct AttnParams;
// A map over rows of row_bytes (elements of 1 or 2 bytes), boxes of box_rows rows x box_bytes (128 or 64: the swizzle).
bool make_rows_map(CUtensorMap* map, const void* p, int64_t rows, int row_bytes, int box_bytes, int box_rows, int elem_bytes);
cudaError_t launch_attn_few(AttnParams& p, const w4a8_kv_cache& c, int rows, cudaStream_t s);
cudaError_t launch_attn_rows(AttnParams& p, const w4a8_kv_cache& c, int64_t batch, cudaStream_t s);

}  // namespace w4a8

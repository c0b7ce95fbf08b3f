// attn_api.cu -- C entry points of rotary positions, the 8-bit cache and attention over it
// (include/w4a8.h): argument checks and launches.  Nothing here allocates memory.
#include "attn_internal.h"

#include <algorithm>
#include <cmath>

namespace w4a8 {
namespace {

constexpr int64_t kMaxDim = 2147483647LL;
constexpr int64_t kMaxLen = 1LL << 30;  // keys of a sequence, rows of a call: differences of positions fit an int
constexpr int64_t kMaxRows = 1LL << 36;  // of all sequences as bounded: a CTA for each 256 of them, most of which find none

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int check_cache(const w4a8_kv_cache* c) {
    if (!c || (c->format != W4A8_KV_INT8 && c->format != W4A8_KV_E4M3) || c->pages < 0 || c->heads <= 0) return W4A8_ERR_ARG;
    if ((c->head_dim != 64 && c->head_dim != 128) || c->page < 16 || c->page > 1024 || (c->page & (c->page - 1)) != 0 ||
        c->heads > 65535 || c->pages > kMaxDim / (c->heads * c->page))
        return W4A8_ERR_SHAPE;
    return W4A8_OK;
}

int check_arrays(const w4a8_kv_cache* c) {
    if (!c->k || !c->v || !c->k_scale || !c->v_scale) return W4A8_ERR_ARG;
    return aligned(c->k, 16) && aligned(c->v, 16) && aligned(c->k_scale, 16) && aligned(c->v_scale, 16) ? W4A8_OK
                                                                                                        : W4A8_ERR_ALIGN;
}

// Strides of `heads` heads of `dim` values and `tokens` tokens: none negative.
bool strides_ok(int64_t token, int64_t head) { return token >= 0 && head >= 0; }

// Rows that a call writes have no memory in common: heads inside a token's, or tokens inside a head's.
bool rows_apart(int64_t token, int64_t head, int64_t tokens, int64_t heads, int64_t dim) {
    if (tokens <= 1) return heads <= 1 || head >= dim;
    if (heads <= 1) return token >= dim;
    const auto spans = [dim](int64_t inner, int64_t n, int64_t outer) {  // (n - 1) * inner + dim <= outer, without overflow
        return inner >= dim && outer >= dim && inner <= (outer - dim) / (n - 1);
    };
    return spans(head, heads, token) || spans(token, tokens, head);
}

bool fits16(const void* p, int64_t token, int64_t head, int el) {
    return aligned(p, 16) && token * el % 16 == 0 && head * el % 16 == 0;
}

}  // namespace
}  // namespace w4a8

using namespace w4a8;

extern "C" {

int w4a8_rope_turns(int64_t rot, double base, int scaling, double factor, double original_len, double low, double high,
                    uint64_t* turns) {
    if (rot <= 0 || rot % 2 != 0 || rot > 4096 || !(base > 1.0) || !std::isfinite(base) || !turns) return W4A8_ERR_ARG;
    if (scaling < W4A8_ROPE_PLAIN || scaling > W4A8_ROPE_BANDS) return W4A8_ERR_ARG;
    if (scaling != W4A8_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor))) return W4A8_ERR_ARG;
    if (scaling == W4A8_ROPE_BASE) {
        if (rot <= 2) return W4A8_ERR_ARG;
        base *= std::pow(factor, static_cast<double>(rot) / static_cast<double>(rot - 2));
        if (!std::isfinite(base)) return W4A8_ERR_ARG;
    }
    if (scaling == W4A8_ROPE_BANDS &&
        (!(original_len > 0.0) || !std::isfinite(original_len) || !(low < high) || !std::isfinite(low) || !std::isfinite(high)))
        return W4A8_ERR_ARG;
    const double two_pi = 6.283185307179586476925286766559;
    for (int64_t i = 0; i < rot / 2; ++i) {
        double f = std::pow(base, -2.0 * static_cast<double>(i) / static_cast<double>(rot));
        if (scaling == W4A8_ROPE_LINEAR) f /= factor;
        if (scaling == W4A8_ROPE_BANDS) {
            const double n = original_len * f / two_pi;
            double keep = (n - low) / (high - low);
            keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
            f = f / factor * (1.0 - keep) + f * keep;
        }
        // f <= 1, so the turn's fraction is below 0.16: 64 bits of it, rounded
        turns[i] = static_cast<uint64_t>(std::ldexp(f / two_pi, 64) + 0.5);
    }
    return W4A8_OK;
}

int w4a8_rope(const void* x, int64_t x_token, int64_t x_head, void* out, int64_t out_token, int64_t out_head, int dtype,
              const int32_t* positions, const uint64_t* turns, int64_t rot, int interleaved, float magnitude, int64_t tokens,
              int64_t heads, int64_t head_dim, void* stream) {
    if (tokens < 0 || heads < 0 || (dtype != W4A8_IN_F32 && dtype != W4A8_IN_BF16) || !std::isfinite(magnitude))
        return W4A8_ERR_ARG;
    if (head_dim <= 0 || head_dim > 4096 || rot <= 0 || rot % 2 != 0 || rot > head_dim || tokens > kMaxDim ||
        heads > (1 << 22) / head_dim)
        return W4A8_ERR_SHAPE;
    if (!strides_ok(x_token, x_head) || !strides_ok(out_token, out_head)) return W4A8_ERR_ARG;
    if (tokens == 0 || heads == 0) return W4A8_OK;
    if (!x || !out || !positions || !turns) return W4A8_ERR_ARG;
    if (!rows_apart(out_token, out_head, tokens, heads, head_dim)) return W4A8_ERR_SHAPE;
    const int el = dtype == W4A8_IN_BF16 ? 2 : 4;
    if (!aligned(x, el) || !aligned(out, el) || !aligned(positions, 4) || !aligned(turns, 8)) return W4A8_ERR_ALIGN;
    RotaryArgs a;
    a.q = {x, x_token, x_head};
    a.q_out = {out, out_token, out_head};
    a.bf16 = dtype == W4A8_IN_BF16;
    a.positions = positions;
    a.turns = turns;
    a.rot = static_cast<int>(rot);
    a.interleaved = interleaved != 0;
    a.magnitude = magnitude;
    a.tokens = tokens;
    a.q_heads = static_cast<int>(heads);
    a.head_dim = static_cast<int>(head_dim);
    int num_sms = 0;
    const int rc = device_info(&num_sms, &a.status);
    if (rc != W4A8_OK) return rc;
    const bool wide = rot % 16 == 0 && head_dim % 16 == 0 && fits16(x, x_token, x_head, el) && fits16(out, out_token, out_head, el);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return (wide ? launch_rotary(a, num_sms, s) : launch_rotary_pairs(a, s)) == cudaSuccess ? W4A8_OK : W4A8_ERR_CUDA;
}

int w4a8_kv_write(const w4a8_kv_cache* cache, const w4a8_kv_rows* r, void* stream) {
    int rc = check_cache(cache);
    if (rc != W4A8_OK) return rc;
    if (!r || r->tokens < 0 || r->q_heads < 0 || (r->dtype != W4A8_IN_F32 && r->dtype != W4A8_IN_BF16)) return W4A8_ERR_ARG;
    if (r->tokens > kMaxDim || cache->heads > (1 << 21) / cache->head_dim || r->q_heads > (1 << 21) / cache->head_dim)
        return W4A8_ERR_SHAPE;
    if (!strides_ok(r->k_token, r->k_head) || !strides_ok(r->v_token, r->v_head)) return W4A8_ERR_ARG;
    const bool q = r->q != nullptr;
    if (r->turns) {
        if (!std::isfinite(r->magnitude)) return W4A8_ERR_ARG;
        if (r->rot <= 0 || r->rot % 16 != 0 || r->rot > cache->head_dim) return W4A8_ERR_SHAPE;
    } else if (q) {
        return W4A8_ERR_ARG;
    }
    if (q && (!r->q_out || r->q_heads == 0 || !strides_ok(r->q_token, r->q_head) || !strides_ok(r->q_out_token, r->q_out_head)))
        return W4A8_ERR_ARG;
    if (r->tokens == 0) return W4A8_OK;
    if (!r->k || !r->v || !r->slots || (r->turns && !r->positions)) return W4A8_ERR_ARG;
    if ((rc = check_arrays(cache)) != W4A8_OK) return rc;
    const int el = r->dtype == W4A8_IN_BF16 ? 2 : 4;
    if (!fits16(r->k, r->k_token, r->k_head, el) || !fits16(r->v, r->v_token, r->v_head, el) || !aligned(r->slots, 8) ||
        (r->turns && (!aligned(r->turns, 8) || !aligned(r->positions, 4))) ||
        (q && (!fits16(r->q, r->q_token, r->q_head, el) || !fits16(r->q_out, r->q_out_token, r->q_out_head, el))))
        return W4A8_ERR_ALIGN;
    if (q && !rows_apart(r->q_out_token, r->q_out_head, r->tokens, r->q_heads, cache->head_dim)) return W4A8_ERR_SHAPE;
    RotaryArgs a;
    a.k = {r->k, r->k_token, r->k_head};
    a.v = {r->v, r->v_token, r->v_head};
    if (q) {
        a.q = {r->q, r->q_token, r->q_head};
        a.q_out = {r->q_out, r->q_out_token, r->q_out_head};
        a.q_heads = static_cast<int>(r->q_heads);
    }
    a.bf16 = r->dtype == W4A8_IN_BF16;
    a.positions = r->positions;
    a.turns = r->turns;
    a.rot = r->turns ? static_cast<int>(r->rot) : 0;
    a.interleaved = r->interleaved != 0;
    a.magnitude = r->magnitude;
    a.tokens = r->tokens;
    a.head_dim = static_cast<int>(cache->head_dim);
    a.slots = r->slots;
    a.cache = *cache;
    int num_sms = 0;
    if ((rc = device_info(&num_sms, &a.status)) != W4A8_OK) return rc;
    return launch_rotary(a, num_sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? W4A8_OK : W4A8_ERR_CUDA;
}

int w4a8_kv_read(const w4a8_kv_cache* cache, const int64_t* slots, int64_t tokens, void* k_out, void* v_out, int dtype,
                 void* stream) {
    int rc = check_cache(cache);
    if (rc != W4A8_OK) return rc;
    if (tokens < 0 || (dtype != W4A8_IN_F32 && dtype != W4A8_IN_BF16)) return W4A8_ERR_ARG;
    if (tokens > kMaxDim || cache->heads > (1 << 21) / cache->head_dim) return W4A8_ERR_SHAPE;
    if (tokens == 0 || (!k_out && !v_out)) return W4A8_OK;
    if (!slots) return W4A8_ERR_ARG;
    if ((rc = check_arrays(cache)) != W4A8_OK) return rc;
    if (!aligned(slots, 8) || !aligned(k_out, 16) || !aligned(v_out, 16)) return W4A8_ERR_ALIGN;
    int num_sms = 0;
    uint32_t* status = nullptr;
    if ((rc = device_info(&num_sms, &status)) != W4A8_OK) return rc;
    return launch_kv_read(*cache, slots, tokens, k_out, v_out, dtype == W4A8_IN_BF16, status,
                          static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? W4A8_OK
               : W4A8_ERR_CUDA;
}

// Sizes and bounds of an attention call.
static int check_attention(const w4a8_kv_cache* c, const w4a8_attention_args* a) {
    const int rc = check_cache(c);
    if (rc != W4A8_OK) return rc;
    if (!a || a->batch < 0 || a->total < 0 || a->q_heads <= 0 || a->max_q < 0 || a->max_kv < 0 || a->window < 0 || a->sinks < 0 ||
        a->table_stride < 0)
        return W4A8_ERR_ARG;
    if (a->q_heads % c->heads != 0 || a->q_heads > 32768 || a->batch > 65535 || a->total > kMaxLen || a->max_q > kMaxLen / a->q_heads ||
        a->batch * (std::min(a->max_q, a->total) * a->q_heads) > kMaxRows || a->max_kv > kMaxDim || a->window > kMaxDim || a->sinks > kMaxDim || a->table_stride > kMaxLen / c->page)
        return W4A8_ERR_SHAPE;
    return W4A8_OK;
}

size_t w4a8_attention_workspace_bytes(const w4a8_kv_cache* cache, const w4a8_attention_args* a) {
    if (check_attention(cache, a) != W4A8_OK) return static_cast<size_t>(-1);
    if (a->batch == 0 || a->total == 0 || a->max_q == 0) return 0;
    return plan_attention(*cache, *a).bytes;
}

size_t w4a8_attention_workspace_bound(const w4a8_kv_cache* cache, const w4a8_attention_args* a) {
    if (check_attention(cache, a) != W4A8_OK) return static_cast<size_t>(-1);
    if (a->batch == 0 || a->total == 0 || a->max_q == 0) return 0;
    return bound_attention(*cache, *a);
}

int w4a8_attention(const w4a8_kv_cache* cache, const w4a8_attention_args* a, void* workspace, size_t workspace_bytes,
                   void* stream) {
    int rc = check_attention(cache, a);
    if (rc != W4A8_OK) return rc;
    if ((a->q_dtype != W4A8_IN_F32 && a->q_dtype != W4A8_IN_BF16) ||
        (a->out_dtype != W4A8_OUT_F32 && a->out_dtype != W4A8_OUT_BF16) || !(a->scale > 0.0f) || !std::isfinite(a->scale) ||
        !strides_ok(a->q_token, a->q_head) || !strides_ok(a->out_token, a->out_head))
        return W4A8_ERR_ARG;
    if (!a->q_start && a->max_q != 1) return W4A8_ERR_ARG;
    if (!a->q_start && a->batch > a->total) return W4A8_ERR_SHAPE;
    if (a->batch == 0 || a->total == 0 || a->max_q == 0) return W4A8_OK;
    if (!a->q || !a->out || (!a->page_table && a->table_stride > 0) || !a->kv_len) return W4A8_ERR_ARG;
    if (cache->pages == 0) return W4A8_ERR_SHAPE;
    if ((rc = check_arrays(cache)) != W4A8_OK) return rc;
    if (!fits16(a->q, a->q_token, a->q_head, a->q_dtype == W4A8_IN_BF16 ? 2 : 4) ||
        !fits16(a->out, a->out_token, a->out_head, a->out_dtype == W4A8_OUT_BF16 ? 2 : 4) || !aligned(a->page_table, 4) ||
        !aligned(a->kv_len, 4) || !aligned(a->q_start, 4))
        return W4A8_ERR_ALIGN;
    if (!rows_apart(a->out_token, a->out_head, a->total, a->q_heads, cache->head_dim)) return W4A8_ERR_SHAPE;
    int num_sms = 0;
    uint32_t* status = nullptr;
    if ((rc = device_info(&num_sms, &status)) != W4A8_OK) return rc;
    const AttnPlan p = plan_attention(*cache, *a);
    if (p.bytes > 0) {
        if (!workspace || workspace_bytes < p.bytes) return W4A8_ERR_WORKSPACE;
        if (!aligned(workspace, 16)) return W4A8_ERR_ALIGN;
    }
    return launch_attention(*cache, *a, p, workspace, status, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? W4A8_OK
               : W4A8_ERR_CUDA;
}

}  // extern "C"

// attn_plan.cu -- how an attention call is cut into work, its launches, and the join of key runs.
#include "attn_common.cuh"

#include <cuda_bf16.h>

#include <algorithm>

namespace w4a8 {
namespace {

constexpr int kJoinWarps = 4;
constexpr int kJoinRows = 16;  // rows of a block of the join, many rows
constexpr int kPlanSms = 152;  // SMs that work is cut for; a constant, so that a plan needs no device

// Joins the runs of rows in their order: slots `first`, then `next`, next + stride, ... (count - 1 of them).  A row is
// `share` of the block's warps', each with every share-th run; their sums meet in the warps' order: one order, whatever
// comes first.
template <int D, typename RowOut>
__device__ __forceinline__ void join_rows(const AttnParams& p, int64_t first, int64_t next, int64_t stride, int count, int R, int row0,
                                          int rows, RowOut&& out_at) {
    constexpr int V = D / 32;
    constexpr int U = 8;  // runs in flight
    __shared__ float sums[kJoinWarps][D];
    __shared__ float weights[kJoinWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int share = rows >= kJoinWarps ? 1 : kJoinWarps / rows, each = kJoinWarps / share;
    const int part = warp % share;
    for (int base = 0; base < rows; base += each) {
        const int row = base + warp / share;
        const bool on = row < rows && warp / share < each;
        float x[V], sum = 0.0f, top = -INFINITY;
#pragma unroll
        for (int e = 0; e < V; ++e) x[e] = 0.0f;
        if (on) {
            auto slot = [&](int i) { return (i == 0 ? first : next + (i - 1) * stride) * R + row0 + row; };
            float2 ml[U];
            float v[U][V];
            auto load = [&](int i0) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int i = i0 + u * share;
                    ml[u] = make_float2(-INFINITY, 0.0f);
                    if (i >= count) continue;
                    ml[u] = __ldcg(&p.part_ml[slot(i)]);
                    const float* src = p.part + slot(i) * D + lane * V;
                    if constexpr (V == 4) {
                        const float4 w = __ldcg(reinterpret_cast<const float4*>(src));
                        v[u][0] = w.x;
                        v[u][1] = w.y;
                        v[u][2] = w.z;
                        v[u][3] = w.w;
                    } else {
                        const float2 w = __ldcg(reinterpret_cast<const float2*>(src));
                        v[u][0] = w.x;
                        v[u][1] = w.y;
                    }
                }
            };
            load(part);  // on their way beside what the largest reference is found from
            for (int i = lane; i < count; i += 32) top = fmaxf(top, __ldcg(&p.part_ml[slot(i)]).x);
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            for (int i0 = part; i0 < count; i0 += U * share) {
                if (i0 != part) load(i0);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (ml[u].x == -INFINITY) continue;
                    const float f = exp2_fast(ml[u].x - top);
                    sum = fmaf(ml[u].y, f, sum);
#pragma unroll
                    for (int e = 0; e < V; ++e) x[e] = fmaf(v[u][e], f, x[e]);
                }
            }
        }
        if (share > 1) {
            if (base > 0) __syncthreads();
#pragma unroll
            for (int e = 0; e < V; ++e) sums[warp][lane * V + e] = x[e];
            if (lane == 0) weights[warp] = sum;
            __syncthreads();
            if (on && part == 0) {  // (warps past the last whole row have no one to add)
                for (int w = 1; w < share; ++w) {
                    sum += weights[warp + w];
#pragma unroll
                    for (int e = 0; e < V; ++e) x[e] += sums[warp + w][lane * V + e];
                }
            }
        }
        if (!on || part != 0) continue;
        const float f = top == -INFINITY ? 0.0f : 1.0f / sum;
        const int64_t at = out_at(row) + lane * V;
        if (p.out_bf16) {
            uint32_t h[V / 2];
#pragma unroll
            for (int e = 0; e < V / 2; ++e) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h[e]) : "f"(x[2 * e + 1] * f), "f"(x[2 * e] * f));
            __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + at;
            if constexpr (V == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(h[0], h[1]);
            else *reinterpret_cast<uint32_t*>(dst) = h[0];
        } else {
            float* dst = static_cast<float*>(p.out) + at;
            if constexpr (V == 4) *reinterpret_cast<float4*>(dst) = make_float4(x[0] * f, x[1] * f, x[2] * f, x[3] * f);
            else *reinterpret_cast<float2*>(dst) = make_float2(x[0] * f, x[1] * f);
        }
    }
}

__device__ __forceinline__ int64_t out_row(const AttnParams& p, const Seq& s, int kvh, int r) {
    return (s.first + r / p.group) * p.out_token + (kvh * p.group + r % p.group) * p.out_head;
}

// Many rows: a block for each kJoinRows rows of a tile.
template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps) join_rows_kernel(const __grid_constant__ AttnParams p) {
    griddep_wait();
    constexpr int kParts = kRowTile / kJoinRows;
    const int it = blockIdx.x / kParts, row0 = blockIdx.x % kParts * kJoinRows, kvh = it / p.row_tiles, tile = it % p.row_tiles;
    const int b = blockIdx.y;
    const Seq s = sequence(p, b);
    const int r0 = tile * kRowTile + row0, rows = min(kJoinRows, s.n * p.group - r0);
    if (rows <= 0) return;
    const int64_t first = ((static_cast<int64_t>(b) * p.heads + kvh) * p.row_tiles + tile) * p.splits;
    join_rows<D>(p, first, first + 1, 1, p.splits, kRowTile, row0, rows, [&](int r) { return out_row(p, s, kvh, r0 + r); });
}

// Few rows: blocks (c, *) join the item that CTA c was the second to work on, if there is one, each some of its rows.
// (A block a row costs more in blocks than it gains, 32 sequences of four queries 83 us for 71; one for all rows
// takes too long over them, 16 sequences with a window 40.1 us for 37.1.)
template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps) join_few_kernel(const __grid_constant__ AttnParams p, int R) {
    griddep_wait();
    const int c = blockIdx.x, per = __ldcg(&p.info[2 * gridDim.x]).x;
    const int4 run = __ldcg(&p.info[2 * c]);       // sequence, head, first unit in the item, the item's units
    const int4 where = __ldcg(&p.info[2 * c + 1]);  // first row of q, rows
    if (run.z <= 0 || run.z > per) return;
    Seq s;
    s.first = where.x;
    const int all = where.y, each = (all + gridDim.y - 1) / gridDim.y, row0 = blockIdx.y * each;
    const int rows = min(each, all - row0);
    if (rows <= 0) return;
    const int count = 1 + (run.w - run.z + per - 1) / per;
    join_rows<D>(p, 2 * static_cast<int64_t>(c - 1) + 1, 2 * static_cast<int64_t>(c), 2, count, R, row0, rows,
                 [&](int r) { return out_row(p, s, run.y, row0 + r); });
}

template <typename Kernel, typename... A>
cudaError_t launch_join(Kernel kernel, dim3 grid, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(32 * kJoinWarps);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// cuTensorMapEncodeTiled, resolved once through the runtime (no link-time dependence on the driver library).
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

}  // namespace

bool make_rows_map(CUtensorMap* map, const void* p, int64_t rows, int row_bytes, int box_bytes, int box_rows, int elem_bytes) {
    const EncodeTiledFn enc = encode_tiled();
    if (!enc) return false;
    const int el = elem_bytes;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(row_bytes / el), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(row_bytes)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_bytes / el), static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t estr[2] = {1, 1};
    return enc(map, el == 2 ? CU_TENSOR_MAP_DATA_TYPE_UINT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(p), dims, strides, box,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE, box_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace {

int rows_of_form(int64_t rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : kRowTile; }
// Keys that a sequence's rows see, as bounded.
int64_t most_seen(const w4a8_attention_args& a, int64_t max_q) {
    return a.window > 0 ? std::min(a.max_kv, a.window + max_q + a.sinks) : a.max_kv;
}
// Few rows: CTAs that fit on the SMs; what they leave to join.
int64_t few_places(int rows) { return (rows <= 16 ? 3 : 2) * kPlanSms; }
size_t few_bytes(int64_t ctas, int rows, int64_t dim) {
    return ctas > 1 ? static_cast<size_t>(ctas) * 2 * rows * (dim + 2) * sizeof(float) + (2 * ctas + 1) * sizeof(int4) : 0;
}
// Many rows: what `runs` CTAs leave to join; steps of 128 keys of a sequence, expanded; their bytes and the most of them.
size_t run_bytes(int64_t runs, int64_t dim) { return static_cast<size_t>(runs) * kRowTile * (dim + 2) * sizeof(float); }
int64_t steps_of(const w4a8_attention_args& a, int64_t max_q) {
    const int64_t cap = (a.max_kv + 127) / 128;
    return a.window > 0 ? std::min(cap, (a.window + max_q + 126) / 128 + 1 + (a.sinks + 127) / 128) : cap;
}
int64_t step_bytes(int64_t dim) { return 128 * dim * 2 * 2 + static_cast<int64_t>(sizeof(float4)); }
constexpr int64_t kMostExpanded = 8LL << 30;

}  // namespace

AttnPlan plan_attention(const w4a8_kv_cache& c, const w4a8_attention_args& a) {
    AttnPlan p;
    const int64_t max_q = std::min(a.max_q, a.total);
    const int64_t rows = max_q * (a.q_heads / c.heads);
    p.rows = rows_of_form(rows);
    p.row_tiles = static_cast<int>((rows + p.rows - 1) / p.rows);
    const int64_t seen = most_seen(a, max_q);
    const int64_t ctas = a.batch * c.heads * p.row_tiles;
    if (p.rows < kRowTile) {
        // Short keys: a cluster of up to eight CTAs for each sequence and head (item), which joins its sums itself: one launch.
        // Measured, so and dealt out: one sequence, 8 items of 512, 1024, 2048 and 4096 keys 6.9 and 9.3 us, 7.2 and 9.8,
        // 8.7 and 10.3, 11.6 and 10.7 (but a launch less to issue); 32 items of up to 512, 2048 and 4096 keys 7.3 and 12.3,
        // 10.3 and 13.0, 14.0 and 15.2; 64 items of 512 keys and 32 rows 14.8 and 21.2; 256 items of up to 512, 1024 and 2048
        // keys 12.7 and 15.9, 20.0 and 18.8, 34.9 and 28.9 (dealt out, by the rule); 512 items of up to 256, 512 and 1024 keys
        // 14.9 and 14.7, 19.1 and 21.0, 30.8 and 29.3; 1024 items 22.4 and 20.3, 31.6 and 33.9, 44.8 and 44.2.
        // Otherwise as many CTAs as fit on the SMs share the keys of all items; below 128 keys each, fewer of them.
        const int64_t item = std::max<int64_t>(1, (seen + 127) / 128), units = ctas * item;
        const int64_t places = few_places(p.rows);
        int cluster = 1;
        while (cluster < 8 && 2 * cluster <= item && 2 * cluster * ctas <= 2 * kPlanSms) cluster *= 2;
        int64_t each = (item + cluster - 1) / cluster;
        // (past 2^20 items, most of them of empty sequences then, a CTA each would take longer than their keys)
        bool clustered = ctas <= (1 << 20) && (each <= 4 || (each <= 8 && ctas >= kPlanSms));
        if (!clustered && seen < a.max_kv) {
            // A window, which keeps most sequences' keys equally many: as many CTAs as clusters fill seven eighths of the
            // SMs' places with (64 items, 33 units: clusters of 6 and 7, 21.4 and 30.6 us).  So and dealt out, for windows of
            // 2048, 4096, 6000 and 8192 keys: 64 items of up to 8 rows 13.5 and 17.2 us, 21.8 and 24.8, 26.1 and 29.6, 32.3 and
            // 36.0; of 16 rows 21.1 and 24.6, 32.6 and 34.1, 38.8 and 43.3, 47.6 and 52.4; of 32 rows, up to 6000 keys, 28.5 and
            // 32.1, 42.2 and 44.5, 51.7 and 54.7; 128 items of 8 rows, up to 6000 keys, 21.8 and 27.0, 32.3 and 36.0, 42.6 and
            // 45.4; of 16 rows 32.5 and 38.7, 47.8 and 52.5, 62.4 and 66.0.
            const int64_t fit = places * 7 / 8;
            cluster = static_cast<int>(std::min<int64_t>(8, fit / ctas));
            each = cluster > 0 ? (item + cluster - 1) / cluster : item;
            clustered = cluster > 0 && each <= 16 && 8 * ctas >= fit * 3 / 4;
        }
        if (clustered) {
            p.cluster = cluster;
            p.splits = static_cast<int>(ctas * cluster);
            return p;
        }
        p.splits = static_cast<int>(std::min<int64_t>(places, units));
        p.bytes = few_bytes(p.splits, p.rows, c.head_dim);
        return p;
    }
    // One CTA an SM: as many runs of an item's keys as fill the SMs, of at least four steps of 128 keys each.  Up to eight steps
    // in one run (64 rows of 32 heads, 1024 keys: one run 22.7 us, two 24.3; 2048 keys: two runs 29.9, four 25.8).
    p.splits = static_cast<int>(std::min<int64_t>({std::max<int64_t>(1, kPlanSms / ctas), seen <= 1024 ? 1 : (seen + 511) / 512, 256}));
    if (p.splits > 1) p.bytes = run_bytes(ctas * p.splits, c.head_dim);
    // Keys and values expanded once, ahead, unless that takes more than 8 GB of workspace.  Measured, ahead and inside: prompts
    // of 128, 512 and 2048 tokens 12.3 and 13.8 us, 16.7 and 22.9, 48 and 75; 16 prompts of 512 tokens 67 and 88; 64 tokens
    // over 2048 keys 25.8 and 31.1; 32 sequences of 16 tokens over 4096 keys 169 and 173.
    const int64_t cap = steps_of(a, max_q), steps = a.batch * c.heads * cap;
    if (cap > 0 && steps <= kMostExpanded / step_bytes(c.head_dim)) {
        p.step_cap = static_cast<int>(cap);
        p.expand_at = (p.bytes + 1023) & ~static_cast<size_t>(1023);
        p.bytes = p.expand_at + static_cast<size_t>(steps * step_bytes(c.head_dim));
    }
    return p;
}

size_t bound_attention(const w4a8_kv_cache& c, const w4a8_attention_args& a) {
    const int64_t max_q = std::min(a.max_q, a.total), group = a.q_heads / c.heads, rows = max_q * group;
    const int64_t seen = most_seen(a, max_q), items = a.batch * c.heads, units = items * std::max<int64_t>(1, (seen + 127) / 128);
    size_t most = 0;
    for (int r = rows_of_form(group); r <= 32 && r <= rows_of_form(rows); r *= 2)
        most = std::max(most, few_bytes(std::min(few_places(r), units), r, c.head_dim));
    if (rows > 32) {
        // more than one run an item only where all runs fit the SMs; the expansion begins on a whole 1024 bytes
        const size_t runs = seen > 1024 ? run_bytes(kPlanSms, c.head_dim) : 0;
        const int64_t steps = std::min(items * steps_of(a, max_q), kMostExpanded / step_bytes(c.head_dim));
        most = std::max(most, runs + 1023 + static_cast<size_t>(steps * step_bytes(c.head_dim)));
    }
    return most;
}

cudaError_t launch_attention(const w4a8_kv_cache& c, const w4a8_attention_args& a, const AttnPlan& plan, void* ws,
                             uint32_t* status, cudaStream_t s) {
    AttnParams p;
    int shift = 0;
    while ((1 << shift) < c.page) ++shift;
    p.k = c.k;
    p.v = c.v;
    p.q = a.q;
    p.out = a.out;
    p.q_token = a.q_token;
    p.q_head = a.q_head;
    p.out_token = a.out_token;
    p.out_head = a.out_head;
    p.k_scale = c.k_scale;
    p.v_scale = c.v_scale;
    p.page_table = a.page_table;
    p.kv_len = a.kv_len;
    p.q_start = a.q_start;
    p.table_stride = a.table_stride;
    p.total = a.total;
    p.pages = c.pages;
    p.heads = static_cast<int>(c.heads);
    p.group = static_cast<int>(a.q_heads / c.heads);
    p.page_shift = shift;
    p.max_q = static_cast<int>(a.max_q);
    const int64_t room = a.table_stride << shift;  // a window that holds every key hides none
    p.window = a.window < room ? static_cast<int>(a.window) : 0;
    p.sinks = p.window > 0 ? static_cast<int>(std::min(a.sinks, room)) : 0;
    p.q_bf16 = a.q_dtype == W4A8_IN_BF16;
    p.out_bf16 = a.out_dtype == W4A8_OUT_BF16;
    p.c = a.scale * 1.4426950408889634f;
    p.row_tiles = plan.row_tiles;
    p.splits = plan.splits;
    // Measured without, and with 1, 2, 3 and 4: 8 rows, 128 sequences of up to 4096 keys 114, 110, 105, 107 and 108 us; 32 rows, 32
    // sequences of up to 4096 keys 107, 96, 90, 88 and 90.
    p.item_cost = plan.rows <= 16 ? 2 : 3;
    p.cluster = plan.cluster;
    p.batch = static_cast<int>(a.batch);
    const size_t slots = plan.rows == kRowTile ? static_cast<size_t>(a.batch) * c.heads * plan.row_tiles * plan.splits : 2 * static_cast<size_t>(plan.splits);
    p.max_kv = static_cast<int>(a.max_kv);
    p.info = nullptr;
    p.part = static_cast<float*>(ws);
    p.part_ml = nullptr;
    p.step_cap = plan.step_cap;
    if (plan.step_cap > 0) {
        const size_t values = static_cast<size_t>(a.batch) * c.heads * plan.step_cap * 128 * c.head_dim;
        p.k16 = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(ws) + plan.expand_at);
        p.v16 = p.k16 + values;
        p.step_info = reinterpret_cast<float4*>(p.v16 + values);
    }
    if (plan.splits > 1 && plan.cluster == 0) {
        p.part_ml = reinterpret_cast<float2*>(p.part + slots * plan.rows * c.head_dim);
        if (plan.rows < kRowTile) p.info = reinterpret_cast<int4*>(p.part_ml + slots * plan.rows);
    }
    p.status = status;
    p.wait_limit_ns = 1000000000ull;
    cudaError_t e = plan.rows == kRowTile ? launch_attn_rows(p, c, a.batch, s) : launch_attn_few(p, c, plan.rows, s);
    if (e != cudaSuccess || p.splits == 1 || plan.cluster > 0) return e;
    if (plan.rows == kRowTile) {
        const dim3 grid(kRowTile / kJoinRows * p.heads * p.row_tiles, static_cast<unsigned>(a.batch));
        return c.head_dim == 128 ? launch_join(join_rows_kernel<128>, grid, s, p) : launch_join(join_rows_kernel<64>, grid, s, p);
    }
    const dim3 grid(p.splits, static_cast<unsigned>(std::min<int64_t>(4, a.max_q * p.group)));
    return c.head_dim == 128 ? launch_join(join_few_kernel<128>, grid, s, p, plan.rows)
                             : launch_join(join_few_kernel<64>, grid, s, p, plan.rows);
}

}  // namespace w4a8

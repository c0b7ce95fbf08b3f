// attn_few.cu -- attention over the 8-bit cache for few rows: one or some new tokens a sequence.
//
// The mathematics, for a row r (query, head of the group that shares a cache head) with factor c_r =
// scale * log2(e) and key j with code rows K_j, V_j and scales a_j, b_j:
//   x_rj = c_r a_j (q_r . K_j),  out_r = sum_j 2^(x_rj - m) b_j V_j / sum_j 2^(x_rj - m)
// in one pass with a running reference m: when it rises, what was summed is multiplied by a power of two.
//
// What bounds it: the cache's bytes from HBM; a key's codes are used for at most 8 rows a pass.  So the
// codes come by TMA into a ring in shared memory that each warp keeps for itself (no warp waits for
// another before the end), and meet the rows on warp-level tensor instructions (m16n8k16, fp16 operands,
// fp32 sums): with keys as their M and rows as their N, 8 rows fill an instruction that the tcgen05 form
// would leave empty from 128 lanes down to 8.  Both products take the codes straight out of 16-byte
// shared-memory reads, with no transposition: the order of a contraction's indices is free, so a
// lane takes 32 (keys) or 16 (values) neighbouring codes as its share of every instruction.
//
// fp16 weights: w = 2^(x - m) b 2^-E, E the exponent of the largest value scale of the step's 32 keys,
// so w stays in range whatever the scales are; m is kept for x + E, which makes sums of
// steps with different E agree without another multiplication.
//
// Measured (GPU time alone): 64 sequences of up to 16384 keys, e4m3, 195 us, 6.1 TB/s of the cache's bytes; one of 131072 keys 54 us,
// 4.9 TB/s, some 10 us of them start, the CTAs' own join and the join of 57 runs a head; one of 512 keys 6.5 us, a chain of
// lengths -> pages -> codes -> products -> join.  Issue slots 46 %, of which the codes' conversion is the largest part.
#include "attn_common.cuh"
#include "fp8_ptx.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

namespace w4a8 {
namespace {

constexpr int kStep = 32;    // keys a warp takes at a time
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kStages = 2;   // steps in a warp's ring
constexpr float kBoost = 11.0f, kLag = 3.0f;  // weights are kept 2^11 up in fp16's range: below 2^(11 + 3 + 1)

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose_8x8(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ float lds_f32(uint32_t a) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}

template <int D, int NT>
struct Few {
    static constexpr int kCodes = kStep * D;               // bytes of a step's keys (or values)
    static constexpr int kScales = 2 * kStep * 4;          // of its scales
    static constexpr int kStageBytes = 2 * kCodes + kScales;
    // shared memory: every warp's stages of codes (swizzle atoms whole), every warp's scales, two warps' sums on their
    // way to another warp, barriers
    static constexpr int kOffScales = kWarps * kStages * 2 * kCodes;
    static constexpr int kOffJoin = kOffScales + kWarps * kStages * kScales;
    static constexpr int kJoinRow = D + 4;                 // floats of a row, padded
    static constexpr int kJoinBytes = 8 * (kJoinRow + 2) * 4;  // eight rows at a time
    // 32 rows: the queries' fragments too, [tile][lane], which would not fit in registers beside the sums (632 bytes of spills a
    // thread, 126 us for 32 sequences of eight queries), and the rows' factors
    static constexpr bool kQueriesShared = NT > 2;
    static constexpr int kOffQueries = kOffJoin + 2 * kJoinBytes;
    static constexpr int kQueryBytes = kQueriesShared ? NT * 32 * (D / 8) * 4 + NT * 8 * 4 : 0;
    static constexpr int kOffBar = kOffQueries + kQueryBytes;
    static constexpr int kSmem = kOffBar + kWarps * kStages * 8 + 128;
    static_assert((NT > 2 ? 2 : 3) * (kSmem + 1024) <= 228 * 1024, "CTAs an SM");
};

// The lane's share of a row of q as loaded (values c D / 4 on), and in fp16 times a power of two.
template <int D, bool BF16>
struct QueryShare {
    static constexpr int N = D / 4, W = N * (BF16 ? 2 : 4) / 16;
    uint4 raw[W];
    __device__ __forceinline__ void load(const char* row, int c) {
#pragma unroll
        for (int i = 0; i < W; ++i) raw[i] = *reinterpret_cast<const uint4*>(row + 16 * (c * W + i));
    }
    // the power's exponent; the row's four lanes agree on it
    __device__ __forceinline__ float convert(uint32_t (&frag)[D / 8]) const {
        float v[N];
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const uint32_t u[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if constexpr (BF16) {
                    v[8 * i + 2 * k] = __uint_as_float(u[k] << 16);
                    v[8 * i + 2 * k + 1] = __uint_as_float(u[k] & 0xffff0000u);
                } else {
                    v[4 * i + k] = __uint_as_float(u[k]);
                }
            }
        }
        float most = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) most = fmaxf(most, fabsf(v[i]));
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
        float e, up;
        query_factor(most, e, up);
#pragma unroll
        for (int i = 0; i < N / 2; ++i) frag[i] = half_pair(v[2 * i] * up, v[2 * i + 1] * up);
        return e;
    }
};

// The work: each sequence and cache head is an item of so many units, a unit a step of keys for each of a
// CTA's warps; all items' units in a row, before each item's some for its queries and joins (`cost`), are dealt out
// evenly, whatever the sequences' lengths are.  (Dealt out by single steps, 128 sequences of up to 1024 keys took 64 us
// for 54: more items cut, and cut into crumbs.)
struct Item {
    int b, kvh, units;
    int first;  // where its units begin, counted from where the CTA's share does; its cost lies before them
};

__device__ __forceinline__ int units_of(const AttnParams& p, int b) {
    const Seq s = sequence(p, b);
    return s.n == 0 ? 0 : (key_steps(p, s.pos, s.pos + s.n - 1, kStep).steps + kWarps - 1) / kWarps;
}

// A sequence with queries and no keys: zeros.
__device__ __noinline__ void write_zeros(const AttnParams& p, int b, int dim) {
    const Seq s = sequence(p, b);
    for (int r = 0; r < s.n; ++r)
        for (int h = 0; h < p.heads * p.group; ++h)
            for (int d = 0; d < dim; d += 8) {
                const int64_t at = (s.first + r) * p.out_token + h * p.out_head + d;
                if (p.out_bf16) {
                    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + at) = make_uint4(0, 0, 0, 0);
                } else {
                    float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.out) + at);
                    dst[0] = dst[1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                }
            }
}

// The CTA's share: `count` of what is dealt out, `per` for most CTAs, of which the first lies in `item` (or its cost).
struct Share {
    int count, per, cost;
    Item item;
    __device__ __forceinline__ int from(const Item& it) const { return max(-it.first, 0); }
    __device__ __forceinline__ int to(const Item& it) const { return min(count - it.first, it.units); }  // 0 and less: none of it
    // whether some of the next item's units are the CTA's: then there is one, and it.units > 0
    __device__ __forceinline__ bool next(const AttnParams& p, Item& it) const;
};

// Every CTA adds up the lengths for itself, 128 sequences at a time: all of them, then (more than 128 sequences)
// again up to the one where its share begins.  `scan`: shared memory.
template <int D>
__device__ __forceinline__ Share find_share(const AttnParams& p, int* scan) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (p.cluster > 0) {
        const int which = blockIdx.x / p.cluster, part = blockIdx.x % p.cluster, b = which / p.heads, units = units_of(p, b);
        if (units == 0 && blockIdx.x % (p.cluster * p.heads) == 0 && threadIdx.x == 0) write_zeros(p, b, D);
        const int per = (units + p.cluster - 1) / p.cluster, unit = min(part * per, units);
        return Share{min(per, units - unit), per, 0, Item{b, which % p.heads, units, -unit}};
    }
    int mine = 0, before = 0, all = 0;  // of a group of 128: below 2^31
    int least = 0x7fffffff, most = 0;   // of all sequences, thread by thread, then over the block
    auto group = [&](int b0, bool zeros) {
        const int b = b0 + threadIdx.x;
        mine = b < p.batch ? units_of(p, b) : 0;
        if (zeros && mine == 0 && b < p.batch && b % gridDim.x == blockIdx.x) write_zeros(p, b, D);
        if (b < p.batch) {
            least = min(least, mine);
            most = max(most, mine);
        }
        if (mine > 0) mine += p.item_cost;
        int v = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, v, d);
            if (lane >= d) v += x;
        }
        __syncthreads();
        if (lane == 31) scan[warp] = v;
        __syncthreads();
        before = v - mine;
        all = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) before += scan[w];
            all += scan[w];
        }
    };
    int64_t total = 0;
    for (int b0 = 0; b0 < p.batch; b0 += kThreads) {
        group(b0, true);
        total += all;
    }
    total *= p.heads;
    Share sh;
    least = __reduce_min_sync(0xffffffffu, least);
    most = __reduce_max_sync(0xffffffffu, most);
    int* ends = scan + kWarps + 3;
    if (lane == 0) {
        ends[warp] = least;
        ends[kWarps + warp] = most;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        least = min(least, ends[w]);
        most = max(most, ends[kWarps + w]);
    }
    const int64_t items = static_cast<int64_t>(p.batch) * p.heads;
    if (least == most && most > 0 && items <= gridDim.x) {
        // Items of one length: the same number of CTAs for each, so that no CTA works on two, whose sums it would stop to join
        // in between.
        const int each = gridDim.x / static_cast<int>(items);
        sh.per = (most + each - 1) / each;
        const int used = (most + sh.per - 1) / sh.per, which = blockIdx.x / used, part = blockIdx.x % used;
        sh.cost = 0;
        if (which >= items) {  // a CTA too many: no item, and none that it could be the second to work on
            sh.count = 0;
            sh.item = Item{0, 0, 0, 0};
            return sh;
        }
        sh.item = Item{which / p.heads, which % p.heads, most, -part * sh.per};
        sh.count = min(most - part * sh.per, sh.per);
        return sh;
    }
    const int64_t per = (total + gridDim.x - 1) / gridDim.x;
    sh.per = static_cast<int>(min(per, static_cast<int64_t>(0x7fffffff)));  // the plan's grid keeps it far below
    sh.cost = p.item_cost;
    const int64_t unit = blockIdx.x * per;
    sh.count = static_cast<int>(max(min(per, total - unit), int64_t{0}));
    sh.item = Item{0, 0, 0, 0};
    if (sh.count == 0) return sh;
    int64_t base = 0;
    for (int b0 = 0; b0 < p.batch; b0 += kThreads) {
        if (p.batch > kThreads) group(b0, false);
        if (unit < (base + all) * p.heads) {
            const int64_t first = (base + before) * p.heads;
            if (unit >= first && unit < first + static_cast<int64_t>(mine) * p.heads) {
                scan[kWarps] = b0 + threadIdx.x;
                scan[kWarps + 1] = mine;
                scan[kWarps + 2] = before;
            }
            __syncthreads();
            sh.item.b = scan[kWarps];
            const int whole = scan[kWarps + 1];
            const int64_t at = (base + scan[kWarps + 2]) * p.heads;
            sh.item.units = whole - sh.cost;
            sh.item.kvh = static_cast<int>((unit - at) / whole);
            sh.item.first = static_cast<int>(at + static_cast<int64_t>(sh.item.kvh) * whole - unit) + sh.cost;
            return sh;
        }
        base += all;
    }
    return sh;
}

__device__ __forceinline__ bool Share::next(const AttnParams& p, Item& it) const {
    it.first += it.units + cost;
    if (it.first >= count) return false;
    if (++it.kvh < p.heads) return true;
    it.kvh = 0;
    do {
        it.units = units_of(p, ++it.b);
    } while (it.units == 0);  // there is another: the share reaches past its cost
    return true;
}

// The sums of a cluster's CTAs meet: each leaves its own in its shared memory, where the ring was (of which nothing is
// in flight any more), then each warp of each CTA takes some of the rows and reads them from all CTAs, in their order.
template <int D, int NT>
__device__ __forceinline__ void join_cluster(const AttnParams& p, uint8_t* base, const Seq& s, int kvh, const float (&m)[NT][2],
                                             const float (&l)[NT][2], const float (&o)[NT][D / 16][4]) {
    constexpr int kRow = D + 4, V = D / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3, rows = s.n * p.group;
    float* sums = reinterpret_cast<float*>(base);
    float2* ml = reinterpret_cast<float2*>(sums + NT * 8 * kRow);
    if (warp == 0) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = t * 8 + 2 * c + r;
                float* dst = sums + row * kRow + g * (D / 8);
#pragma unroll
                for (int q = 0; q < D / 16; q += 2)
                    *reinterpret_cast<float4*>(dst + 2 * q) = make_float4(o[t][q][r], o[t][q][2 + r], o[t][q + 1][r], o[t][q + 1][2 + r]);
                if (g == 0) ml[row] = make_float2(held_reference(m[t][r], l[t][r]), l[t][r]);
            }
    }
    cluster_sync_all();
    for (int row = warp * p.cluster + static_cast<int>(cluster_ctarank()); row < rows; row += kWarps * p.cluster) {
        float2 at[8];
        float x[8][V], top = -INFINITY;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (k >= p.cluster) break;
            at[k].x = ld_shared_cluster_f32(&ml[row].x, k);
            at[k].y = ld_shared_cluster_f32(&ml[row].y, k);
#pragma unroll
            for (int e = 0; e < V; ++e) x[k][e] = ld_shared_cluster_f32(sums + row * kRow + lane + 32 * e, k);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < p.cluster) top = fmaxf(top, at[k].x);
        float sum = 0.0f, y[V] = {};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (k >= p.cluster || at[k].x == -INFINITY) continue;
            const float f = exp2_fast(at[k].x - top);
            sum = fmaf(at[k].y, f, sum);
#pragma unroll
            for (int e = 0; e < V; ++e) y[e] = fmaf(x[k][e], f, y[e]);
        }
        const float f = top == -INFINITY ? 0.0f : 1.0f / sum;
        const int64_t to = (s.first + row / p.group) * p.out_token + (kvh * p.group + row % p.group) * p.out_head + lane;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            if (p.out_bf16) static_cast<__nv_bfloat16*>(p.out)[to + 32 * e] = __float2bfloat16(y[e] * f);
            else static_cast<float*>(p.out)[to + 32 * e] = y[e] * f;
        }
    }
    cluster_sync_all();  // no CTA leaves while another may still read its sums
}

template <int D, int NT, int FMT, bool BF16>
__global__ void __launch_bounds__(kThreads, NT <= 2 ? 3 : 2) few_kernel(const __grid_constant__ AttnParams p) {
    using F = Few<D, NT>;
    using C = Codes<FMT>;
    constexpr int KS = D / 16;  // instructions over the head
    constexpr int MT = D / 16;  // of 16 output values
    extern __shared__ __align__(1024) uint8_t base[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    uint64_t* full = reinterpret_cast<uint64_t*>(base + F::kOffBar) + warp * kStages;
    uint32_t* abort_flag = reinterpret_cast<uint32_t*>(base + F::kOffBar + kWarps * kStages * 8);
    int* scan = reinterpret_cast<int*>(abort_flag + 2);
    const WaitCtl ctl{abort_flag, p.status, p.wait_limit_ns};
    uint8_t* ring = base + warp * kStages * 2 * F::kCodes;
    uint8_t* scales = base + F::kOffScales + warp * kStages * F::kScales;

    if (lane == 0) {
        for (int i = 0; i < kStages; ++i) mbar_init(&full[i], 1);
        fence_barrier_init();
        if (warp == 0) *abort_flag = 0;
    }
    if (threadIdx.x < 2) tma_prefetch_map(threadIdx.x ? &p.vmap : &p.kmap);
    // A warp's copies complete barriers that its first lane set up, and every wait reads the flag; a cluster's CTA of up to 16
    // rows comes to no other barrier before them.
    __syncthreads();
    griddep_wait();
    griddep_launch_dependents();  // the join's blocks may come in, and wait for this grid
    const Share share = find_share<D>(p, scan);
    if (threadIdx.x == 0 && p.info) {
        p.info[2 * blockIdx.x] = make_int4(share.item.b, share.item.kvh, share.from(share.item), share.item.units);
        if (blockIdx.x == 0) p.info[2 * gridDim.x] = make_int4(share.per, 0, 0, 0);
    }
    // the whole CTA, a cluster as one: nothing, or no more than an item's cost
    if (p.cluster > 1 ? share.item.units == 0 : share.count == 0 || share.to(share.item) <= 0) return;

    // Copies run ahead of the sums, across items: the next step of this warp, its pages looked up one step before.
    Item a_item = share.item;
    int a_in = share.from(share.item), a_end = share.to(share.item);
    bool a_more = true;
    Keys a_keys;
    int a_last = 0, a_key = -1, a_page = 0;
    // a lane's copy: box `a_box` of the step, of keys or of values; as many lanes as that makes
    const int a_box = (lane >> 1) * 16;
    const bool a_on = lane < (p.box < kStep ? 4 : 2), a_value = lane & 1;
    const CUtensorMap* a_map = a_value ? &p.vmap : &p.kmap;
    const float* a_scale = a_value ? p.v_scale : p.k_scale;
    uint8_t* a_codes_to = ring + (a_value ? F::kCodes : 0) + a_box * D;
    uint8_t* a_scales_to = scales + (a_value ? kStep * 4 : 0) + a_box * 4;
    auto a_enter = [&] {
        const Seq s = sequence(p, a_item.b);
        a_last = s.pos + s.n - 1;
        a_keys = key_steps(p, s.pos, a_last, kStep);
    };
    auto a_next = [&] {
        a_key = -1;
        while (a_more) {
            if (a_in >= a_end) {
                a_more = a_end == a_item.units && share.next(p, a_item);
                if (!a_more) break;
                a_enter();
                a_in = 0;
                a_end = share.to(a_item);
            }
            const int step = a_in * kWarps + warp;
            ++a_in;
            if (step >= a_keys.steps) continue;
            a_key = a_keys.first(step);
            // a second box past the keys repeats the first one: its table entry may not exist
            const int j = a_key + a_box;
            a_page = page_of(p, a_item.b, a_on && j <= a_last ? j : a_key);
            return;
        }
    };
    int issued = 0, done = 0;  // steps of this warp
    auto issue = [&] {
        if (a_key < 0) return;
        const int stage = issued % kStages;
        ++issued;
        if (lane == 0) mbar_arrive_expect_tx(&full[stage], F::kStageBytes);
        if (a_on) {
            const int row = row_in(p, a_page, a_item.kvh, a_key + a_box <= a_last ? a_key + a_box : a_key);
            tma_load_2d(a_codes_to + stage * 2 * F::kCodes, a_map, 0, row, &full[stage]);
            bulk_load(a_scales_to + stage * F::kScales, a_scale + row, p.box * 4, &full[stage]);
        }
        __syncwarp();
        a_next();
    };
    a_enter();
    a_next();
    for (int i = 0; i < kStages; ++i) issue();

    auto query_row = [&](const Seq& s, int kvh, int r) {
        r = min(r, s.n * p.group - 1);
        return static_cast<const char*>(p.q) +
               ((s.first + r / p.group) * p.q_token + (kvh * p.group + r % p.group) * p.q_head) * (BF16 ? 2 : 4);
    };
    Item item = share.item;
    Seq s = sequence(p, item.b);
    if (threadIdx.x == 0 && p.info) p.info[2 * blockIdx.x + 1] = make_int4(s.first, s.n * p.group, 0, 0);
    QueryShare<D, BF16> qs;  // NT == 1: the next item's, loaded ahead
    if constexpr (NT == 1) qs.load(query_row(s, item.kvh, g), c);
    bool ok = true;

    for (;;) {
        const int rows = s.n * p.group, p_min = s.pos, p_max = s.pos + s.n - 1;
        const Keys keys = key_steps(p, p_min, p_max, kStep);
        const int lo = share.from(item), hi = share.to(item);
        // queries: row 8 t + g in this lane's fragments; rows 8 t + 2 c and 8 t + 2 c + 1 in its sums
        uint32_t qf[F::kQueriesShared ? 1 : NT][D / 8];
        float cr[NT][2];
        int pos[NT][2];
        const uint32_t queries = smem_u32(base + F::kOffQueries), factors = queries + NT * 32 * (D / 8) * 4;
        if constexpr (F::kQueriesShared) {  // a tile to a warp (the last join's barriers stand between this and earlier reads)
            static_assert(NT == kWarps, "a tile to a warp");
            qs.load(query_row(s, item.kvh, warp * 8 + g), c);
            const float f = p.c * exp2f(qs.convert(qf[0]));
#pragma unroll
            for (int i = 0; i < D / 8; i += 4)
                asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(queries + ((warp * (D / 32) + i / 4) * 32 + lane) * 16), "r"(qf[0][i]),
                             "r"(qf[0][i + 1]), "r"(qf[0][i + 2]), "r"(qf[0][i + 3]) : "memory");
            if (c == 0) asm volatile("st.shared.f32 [%0], %1;" ::"r"(factors + (warp * 8 + g) * 4), "f"(f) : "memory");
            __syncthreads();
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if constexpr (F::kQueriesShared) {
                cr[t][0] = lds_f32(factors + (t * 8 + 2 * c) * 4);
                cr[t][1] = lds_f32(factors + (t * 8 + 2 * c + 1) * 4);
            } else {
                if constexpr (NT > 1) qs.load(query_row(s, item.kvh, t * 8 + g), c);
                const float f = p.c * exp2f(qs.convert(qf[t]));
                cr[t][0] = __shfl_sync(0xffffffffu, f, 8 * c);
                cr[t][1] = __shfl_sync(0xffffffffu, f, 8 * c + 4);
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) pos[t][k] = s.pos + min(t * 8 + 2 * c + k, rows - 1) / p.group;
        }
        float o[NT][MT][4];
        float m[NT][2], l[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) o[t][i][k] = 0.0f;
            m[t][0] = m[t][1] = -INFINITY;
            l[t][0] = l[t][1] = 0.0f;
        }

        for (int i = lo * kWarps + warp; i < min(hi * kWarps, keys.steps); i += kWarps) {
            const int stage = done % kStages;
            // a wait that gave up: on without waiting, because the warps meet below
            ok = ok && __all_sync(0xffffffffu, mbar_poll(&full[stage], (done / kStages) & 1, ctl));
            ++done;
            if (!ok) continue;
            const uint32_t st = smem_u32(ring + stage * 2 * F::kCodes), sca = smem_u32(scales + stage * F::kScales);
            const int j0 = keys.first(i);
            float sc[NT][2][4];  // [16 keys][key g: rows 2c, 2c+1; key g + 8: the same]
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t k0[D / 16], k1[D / 16];  // this lane's codes of keys 16 h + g and 16 h + g + 8
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int row = 16 * h + 8 * e + g;
                    uint32_t(&k)[D / 16] = e ? k1 : k0;
#pragma unroll
                    for (int q = 0; q < D / 64; ++q) {
                        // 16-byte chunk of the row, swizzled as TMA wrote it: 128 bytes by row % 8, 64 by (row / 2) % 4
                        const int chunk = D == 128 ? ((2 * c + q) ^ (row & 7)) : (c ^ ((row >> 1) & 3));
                        const uint4 w = lds128(st + row * D + chunk * 16);
                        k[4 * q] = w.x;
                        k[4 * q + 1] = w.y;
                        k[4 * q + 2] = w.z;
                        k[4 * q + 3] = w.w;
                    }
                }
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int k = 0; k < 4; ++k) sc[t][h][k] = 0.0f;
                if constexpr (F::kQueriesShared) {
                    uint32_t ka[KS][4];
#pragma unroll
                    for (int q = 0; q < KS; ++q) {
                        const uint32_t w0 = C::ready(k0[q]), w1 = C::ready(k1[q]);
                        ka[q][0] = C::value(C::template raw<0, 1>(w0));
                        ka[q][1] = C::value(C::template raw<0, 1>(w1));
                        ka[q][2] = C::value(C::template raw<2, 3>(w0));
                        ka[q][3] = C::value(C::template raw<2, 3>(w1));
                    }
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int q = 0; q < KS; q += 2) {
                            const uint4 w = lds128(queries + ((t * (D / 32) + q / 2) * 32 + lane) * 16);
                            mma_16816(sc[t][h], ka[q][0], ka[q][1], ka[q][2], ka[q][3], w.x, w.y);
                            mma_16816(sc[t][h], ka[q + 1][0], ka[q + 1][1], ka[q + 1][2], ka[q + 1][3], w.z, w.w);
                        }
                } else {
#pragma unroll
                    for (int q = 0; q < KS; ++q) {
                        const uint32_t w0 = C::ready(k0[q]), w1 = C::ready(k1[q]);
                        const uint32_t a0 = C::value(C::template raw<0, 1>(w0)), a2 = C::value(C::template raw<2, 3>(w0));
                        const uint32_t a1 = C::value(C::template raw<0, 1>(w1)), a3 = C::value(C::template raw<2, 3>(w1));
#pragma unroll
                        for (int t = 0; t < NT; ++t) mma_16816(sc[t][h], a0, a1, a2, a3, qf[t][2 * q], qf[t][2 * q + 1]);
                    }
                }
            }
            // scales of keys g, g + 8, g + 16, g + 24
            const bool all_seen = all_see(p, p_min, p_max, j0, kStep);
            float ks[4], vs[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                ks[k] = lds_f32(sca + (g + 8 * k) * 4);
                vs[k] = lds_f32(sca + kStep * 4 + (g + 8 * k) * 4);
            }
            if (!all_seen) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (!some_see(p, p_min, p_max, j0 + g + 8 * k)) vs[k] = 0.0f;
            }
            // keys whose values are all zero add to l alone: their weights stay small beside other steps'
            float ev, iv;
            uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(max_nan(max_nan(vs[0], vs[1]), max_nan(vs[2], vs[3]))));
            if (most >= kBitsInf) {
                // a value that is no number: its key's logits are NaN, for the rows that see it, and it meets no weight of 0
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (finite(vs[k])) continue;
                    ks[k] = not_a_number();
                    vs[k] = 0.0f;
                }
                most = __reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(fmaxf(vs[0], vs[1]), fmaxf(vs[2], vs[3]))));
            }
            exponent_of(__uint_as_float(most), -24, ev, iv);
            uint32_t wf[NT][2][2];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                float top[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float& x = sc[t][k >> 1][(k & 1) * 2 + r];
                        x = fmaf(x, ks[k] * cr[t][r], ev);
                        if (!all_seen) {
                            const int j = j0 + g + 8 * k, at = pos[t][r];
                            const bool see = j <= at && (p.window == 0 || j > at - p.window || j < p.sinks);
                            if (!see) x = -INFINITY;
                        }
                    }
                    top[r] = fmaxf(fmaxf(sc[t][0][r], sc[t][0][2 + r]), fmaxf(sc[t][1][r], sc[t][1][2 + r]));
                }
                // m may lag the largest x by kLag: most steps need no reduction over the keys' lanes
                if (__any_sync(0xffffffffu, top[0] > m[t][0] + kLag || top[1] > m[t][1] + kLag)) {
                    float f[2];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 4));
                        top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 8));
                        top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 16));
                        const float n = fmaxf(m[t][r], top[r]);
                        f[r] = m[t][r] == n ? 1.0f : exp2_fast(m[t][r] - n);  // 0 from the start's -inf on
                        m[t][r] = n;
                        l[t][r] *= f[r];
                    }
#pragma unroll
                    for (int q = 0; q < MT; ++q) {
                        o[t][q][0] *= f[0];
                        o[t][q][1] *= f[1];
                        o[t][q][2] *= f[0];
                        o[t][q][3] *= f[1];
                    }
                }
                float sum[2] = {0.0f, 0.0f};
                float w[2][4];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float ref = m[t][r] == -INFINITY ? 0.0f : m[t][r] - kBoost;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float e = exp2_fast(sc[t][k >> 1][(k & 1) * 2 + r] - ref);
                        sum[r] += e;
                        w[r][k] = e * (vs[k] * iv);
                    }
                    l[t][r] = fmaf(sum[r], iv, l[t][r]);
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    wf[t][h][0] = transpose_8x8(half_pair(w[0][2 * h], w[1][2 * h]));
                    wf[t][h][1] = transpose_8x8(half_pair(w[0][2 * h + 1], w[1][2 * h + 1]));
                }
            }
            // values: the lane's codes 16 g .. (8 g .. for 64) of keys 2c, 2c + 1, 2c + 8, 2c + 9 of each 16
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                constexpr int VW = D / 32;  // registers of a lane's codes of one key
                uint32_t v[4][VW];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int row = 16 * h + 2 * c + (k & 1) + (k >> 1) * 8;
                    const uint32_t a = st + F::kCodes + row * D;
                    if constexpr (D == 128) {
                        const uint4 w = lds128(a + ((g ^ (row & 7)) * 16));
                        v[k][0] = w.x;
                        v[k][1] = w.y;
                        v[k][2] = w.z;
                        v[k][3] = w.w;
                    } else {
                        const uint2 w = lds64(a + (((g >> 1) ^ ((row >> 1) & 3)) * 16) + (g & 1) * 8);
                        v[k][0] = w.x;
                        v[k][1] = w.y;
                    }
                    if (!all_seen && !some_see(p, p_min, p_max, j0 + row)) {  // any code may lie there, NaN too
#pragma unroll
                        for (int q = 0; q < VW; ++q) v[k][q] = 0;
                    }
                }
#pragma unroll
                for (int q = 0; q < VW; ++q) {
                    const uint32_t u0 = C::ready(v[0][q]), u1 = C::ready(v[1][q]), u2 = C::ready(v[2][q]), u3 = C::ready(v[3][q]);
                    // [key 0 byte i, key 1 byte i, key 0 byte i + 1, key 1 byte i + 1]
                    const uint32_t lo01 = byte_perm(u0, u1, 0x5140), hi01 = byte_perm(u0, u1, 0x7362);
                    const uint32_t lo23 = byte_perm(u2, u3, 0x5140), hi23 = byte_perm(u2, u3, 0x7362);
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        mma_16816(o[t][2 * q], C::value(C::template raw<0, 1>(lo01)), C::value(C::template raw<2, 3>(lo01)),
                                  C::value(C::template raw<0, 1>(lo23)), C::value(C::template raw<2, 3>(lo23)), wf[t][h][0],
                                  wf[t][h][1]);
                        mma_16816(o[t][2 * q + 1], C::value(C::template raw<0, 1>(hi01)), C::value(C::template raw<2, 3>(hi01)),
                                  C::value(C::template raw<0, 1>(hi23)), C::value(C::template raw<2, 3>(hi23)), wf[t][h][0],
                                  wf[t][h][1]);
                    }
                }
            }
            __syncwarp();  // every lane has read the stage
            issue();
        }

        // the item's next in line: its queries come in while the warps' sums meet
        const Item was = item;
        const Seq ws = s;
        const bool more = hi == item.units && share.next(p, item);
        if (more) {
            s = sequence(p, item.b);
            if constexpr (NT == 1) qs.load(query_row(s, item.kvh, g), c);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                l[t][r] += __shfl_xor_sync(0xffffffffu, l[t][r], 4);
                l[t][r] += __shfl_xor_sync(0xffffffffu, l[t][r], 8);
                l[t][r] += __shfl_xor_sync(0xffffffffu, l[t][r], 16);
            }
        // warps 2 and 3 hand their sums to 0 and 1, then 1 to 0; eight rows at a time
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int half = kWarps / 2; half > 0; half >>= 1) {
                __syncthreads();
                if (warp >= half && warp < 2 * half) {
                    float* to = reinterpret_cast<float*>(base + F::kOffJoin + (warp - half) * F::kJoinBytes);
                    float2* ml = reinterpret_cast<float2*>(to + 8 * F::kJoinRow);
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int row = 2 * c + r;
                        float* dst = to + row * F::kJoinRow + g * (D / 8);
#pragma unroll
                        for (int q = 0; q < MT; q += 2)  // values 2 q .. 2 q + 3 of the lane's D / 8
                            *reinterpret_cast<float4*>(dst + 2 * q) = make_float4(o[t][q][r], o[t][q][2 + r], o[t][q + 1][r], o[t][q + 1][2 + r]);
                        if (g == 0) ml[row] = make_float2(m[t][r], l[t][r]);
                    }
                }
                __syncthreads();
                if (warp < half) {
                    const float* from = reinterpret_cast<const float*>(base + F::kOffJoin + warp * F::kJoinBytes);
                    const float2* ml = reinterpret_cast<const float2*>(from + 8 * F::kJoinRow);
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int row = 2 * c + r;
                        const float2 v = ml[row];
                        const float top = fmaxf(m[t][r], v.x);
                        const float f0 = m[t][r] == -INFINITY ? 0.0f : exp2_fast(m[t][r] - top);
                        const float f1 = v.x == -INFINITY ? 0.0f : exp2_fast(v.x - top);
                        m[t][r] = top;
                        l[t][r] = fmaf(l[t][r], f0, v.y * f1);
                        const float* src = from + row * F::kJoinRow + g * (D / 8);
#pragma unroll
                        for (int q = 0; q < MT; q += 2) {
                            const float4 x = *reinterpret_cast<const float4*>(src + 2 * q);
                            o[t][q][r] = fmaf(o[t][q][r], f0, x.x * f1);
                            o[t][q][2 + r] = fmaf(o[t][q][2 + r], f0, x.y * f1);
                            o[t][q + 1][r] = fmaf(o[t][q + 1][r], f0, x.z * f1);
                            o[t][q + 1][2 + r] = fmaf(o[t][q + 1][2 + r], f0, x.w * f1);
                        }
                    }
                }
            }
        }
        if (p.cluster > 1) {
            join_cluster<D, NT>(p, base, ws, was.kvh, m, l, o);
            break;
        }
        if (warp == 0) {
            const bool whole = lo == 0 && hi == was.units;
            // a run that another CTA began takes slot 2c, one that the next CTA goes on with 2c + 1
            const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (lo == 0);
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int row = t * 8 + 2 * c + r;
                    if (row >= rows) continue;
                    if (!whole && g == 0) p.part_ml[slot * (NT * 8) + row] = make_float2(held_reference(m[t][r], l[t][r]), l[t][r]);
                    const float f = !whole ? 1.0f : m[t][r] == -INFINITY ? 0.0f : 1.0f / l[t][r];
                    const int64_t at = (ws.first + row / p.group) * p.out_token + (was.kvh * p.group + row % p.group) * p.out_head + g * (D / 8);
                    if (whole && p.out_bf16) {
                        uint32_t h[D / 16];
#pragma unroll
                        for (int q = 0; q < MT; ++q)
                            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h[q]) : "f"(o[t][q][2 + r] * f), "f"(o[t][q][r] * f));
                        uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + at);
#pragma unroll
                        for (int q = 0; q < MT; q += 4) dst[q / 4] = make_uint4(h[q], h[q + 1], h[q + 2], h[q + 3]);
                    } else {
                        float4* dst = reinterpret_cast<float4*>(whole ? static_cast<float*>(p.out) + at
                                                                      : p.part + (slot * (NT * 8) + row) * D + g * (D / 8));
#pragma unroll
                        for (int q = 0; q < MT; q += 2)
                            dst[q / 2] = make_float4(o[t][q][r] * f, o[t][q][2 + r] * f, o[t][q + 1][r] * f, o[t][q + 1][2 + r] * f);
                    }
                }
        }
        if (!more) break;
    }
    // after a wait that gave up: what is still in flight lands before the CTA leaves
    for (int q = max(0, issued - kStages); !ok && q < issued; ++q) {
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(smem_u32(&full[q % kStages]), (q / kStages) & 1))
            if (globaltimer_ns() - t0 > 10000000ull) break;
    }
}

template <int D, int NT, int FMT, bool BF16>
cudaError_t launch_few(const AttnParams& p, cudaStream_t s) {
    static bool attr_done[64] = {};
    const auto kernel = few_kernel<D, NT, FMT, BF16>;
    constexpr int smem = Few<D, NT>::kSmem;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !attr_done[dev]) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        if (dev < 64) attr_done[dev] = true;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.splits);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(p.cluster);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int D, int NT>
cudaError_t launch_fmt(const AttnParams& p, int format, cudaStream_t s) {
    if (format == W4A8_KV_INT8)
        return p.q_bf16 ? launch_few<D, NT, W4A8_KV_INT8, true>(p, s) : launch_few<D, NT, W4A8_KV_INT8, false>(p, s);
    return p.q_bf16 ? launch_few<D, NT, W4A8_KV_E4M3, true>(p, s) : launch_few<D, NT, W4A8_KV_E4M3, false>(p, s);
}

template <int D>
cudaError_t launch_dim(const AttnParams& p, int rows, int format, cudaStream_t s) {
    return rows <= 8 ? launch_fmt<D, 1>(p, format, s)
                     : rows <= 16 ? launch_fmt<D, 2>(p, format, s) : launch_fmt<D, 4>(p, format, s);
}

}  // namespace

cudaError_t launch_attn_few(AttnParams& p, const w4a8_kv_cache& c, int rows, cudaStream_t s) {
    p.box = c.page >= kStep ? kStep : 16;
    const int64_t slots = c.pages * c.heads * c.page;
    const int dim = static_cast<int>(c.head_dim);
    if (!make_rows_map(&p.kmap, c.k, slots, dim, dim, p.box, 1) || !make_rows_map(&p.vmap, c.v, slots, dim, dim, p.box, 1))
        return cudaErrorInvalidValue;
    return c.head_dim == 128 ? launch_dim<128>(p, rows, c.format, s) : launch_dim<64>(p, rows, c.format, s);
}

}  // namespace w4a8

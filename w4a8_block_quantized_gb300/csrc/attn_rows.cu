// attn_rows.cu -- attention over the 8-bit cache for many rows: prompts, and chunks of them.
//
// The mathematics is that of attn_few.cu; rows are (query, head of a group) pairs, so that the heads that
// share a cache head share its keys too.  A CTA takes two tiles of 128 rows and walks the keys 128 at a time:
//   S = Q K^T        tcgen05 fp16, Q and the keys in shared memory, S in TMEM
//   P = 2^(c_r S + E - m)  by softmax threads, one a row: no exchange between threads; back to TMEM as fp16
//   O += P V         tcgen05 fp16, P from TMEM, the values in shared memory
// The tensor cores work for one tile while the other tile's softmax runs, and take P in two halves.
//
// Keys and values come to the tensor cores in fp16, in one of two ways:
//   ahead    expand_kernel writes the sequence's keys and values to the workspace once, code * scale * 2^-E in fp32
//            rounded once to fp16 (E: a step's largest scale), and the steps come by TMA.
//   inside   warps of the CTA turn codes into fp16 a step ahead: the codes exactly, the key's scale applied to S, the value's
//            scale rounded to fp16 and multiplied in.  Where the workspace would be too large: 4 bytes a code.  (The warps are
//            the slower way even for one row tile: pages, scales and codes are loads that wait for one another, 3 us a step
//            of 128 keys, where the tensor cores and the softmax take 1.2.)
// Rows of 64 values, 128-byte swizzle, are a K-major operand of the first product and the MN-major operand of
// the second, so nothing is transposed.
//
// Roles (512 threads):
//   warps 0-3, 4-7       softmax of tile 0, 1: thread = row = TMEM lane
//   warp 12              issues the MMAs
//   warp 8 (ahead)       copies;  warps 8-11, 14 and 15 (inside)  codes to fp16
//
// m is kept up to 8 (a factor of 256) behind the largest x + E seen: multiplying O by a power of two takes the sums out of
// TMEM and back, 600 cycles or more of a step's 2500, for all 32 rows of a warp where one needs it.
//
// Measured (GPU time alone): 8192 tokens of 32 heads of 128 over themselves 387 us, 1420 TFLOP/s of the products that the mask leaves
// (the tensor cores' measured rate is 1965; an MMA lasts 90 cycles beside the copies and queries in shared memory, 69 alone);
// 2048 tokens 48 us; 512 tokens of 16 heads 16.8 us: expansion 4, queries 2, four steps of 1.2, output 2, launches.
#include "attn_common.cuh"
#include "fp8_ptx.cuh"
#include "quant_math.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace w4a8 {
namespace {

constexpr int kStep = 128;    // keys of a step
constexpr int kThreads = 512;
constexpr int kMeta = 4;      // steps whose scales are kept: a softmax is at most two steps behind the expansion
constexpr float kBoost = 7.0f, kLag = 8.0f;  // weights stay below 2^(7 + 8) of fp16's 2^16
// Register split: launch 512 x 128 (checked at build time); softmax up, the rest down.
template <bool AHEAD>
struct Regs {
    static constexpr int kSoftmax = AHEAD ? 200 : 168, kThird = AHEAD ? 48 : 96, kLast = AHEAD ? 64 : 80;
    static_assert(256 * kSoftmax + 128 * kThird + 128 * kLast == kThreads * 128, "register split");
};
constexpr int kExpandWarps = 6, kExpandThreads = 32 * kExpandWarps;

template <int D, bool AHEAD>
struct Rows {
    static constexpr int kKeys = AHEAD ? 3 : 2;          // steps of keys in shared memory; two of values

    static constexpr int kHalf = 128 * 128;              // bytes of 128 rows of 64 fp16
    static constexpr int kTileBytes = 128 * D * 2;       // of a Q tile, a key or a value step
    static constexpr int kOffK = 2 * kTileBytes, kOffV = kOffK + kKeys * kTileBytes, kOffMeta = kOffV + 2 * kTileBytes;
    static constexpr int kMetaBytes = 2 * kStep * 4 + 16;  // inside: key scales, value scales, E, 2^-E
    static constexpr int kSmem = kOffMeta + (AHEAD ? 0 : kMeta * kMetaBytes) + 1024;
    static constexpr uint32_t kColO = 256;               // TMEM columns: S (and P) 0 and 128, O from here
    static_assert(kSmem <= 227 * 1024 - 1536, "shared memory budget");
};

// D[tmem] (+)= A[tmem] * B[smem], kind::f16.
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// Waits, up to 10 ms, for a copy that was begun.
__device__ __forceinline__ void land(uint32_t bar, uint32_t parity) {
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity))
        if (globaltimer_ns() - t0 > 10000000ull) break;
}

// A wait that gave up is decided for the whole warp: what follows wants all its lanes.
__device__ __forceinline__ bool all_ok_warp(bool ok) { return __all_sync(0xffffffffu, ok); }

__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// Where 16-byte chunk `c` (8 fp16) of row `r` of a tile lies: halves of 64 values, rows of 128 bytes, swizzled.
__device__ __forceinline__ uint32_t tile_chunk(int r, int c) {
    return static_cast<uint32_t>((c >> 3) * (128 * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}

// Bits 0 .. n - 1 of 32, none for n <= 0.
__device__ __forceinline__ uint32_t bits_below(int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u; }

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Rows row0 + i (i < 256) of an item as query and head of the group, without a division: i + row0 % group is below
// 2^17, where the product with 2^32 / group, rounded up, has the quotient in its upper half (group <= 2^15).
struct RowMap {
    int query0, rest, group;
    uint32_t inverse;
    __device__ __forceinline__ RowMap(int row0, int g) : query0(row0 / g), rest(row0 % g), group(g), inverse(0xffffffffu / g + 1) {}
    __device__ __forceinline__ void at(int i, int& query, int& head) const {
        const int v = rest + i, q = group == 1 ? v : static_cast<int>(__umulhi(static_cast<uint32_t>(v), inverse));
        query = query0 + q;
        head = v - q * group;
    }
};

// The 256 rows of q of a CTA (row_at: where the row of a tile index is, null past the rows) as fp16 times a power of two in two
// tiles, by all threads.  bf16 rows are first copied as they are to their places (copy_rows: whole rows, 8 or 16 lanes each,
// asynchronously, before the CTA's barriers are set up), then converted in place, a half row a thread; fp32 rows are
// read twice.  The exponents of the powers go to `exponent`.  Loops, not straight-line code: a CTA comes by here once,
// and unrolled this took 9 us of instruction fetches.
template <int D>
__device__ __forceinline__ void copy_rows(const char* first, int head, int group, int64_t token_step, int64_t head_step, int rows, uint32_t tiles) {
    constexpr int CH = D / 8, RPI = 32 / CH;  // 16-byte chunks of a row, rows an instruction of a warp
    const int lane = threadIdx.x & 31, r0 = (threadIdx.x >> 5) * 16 + lane / CH;
    first += 16 * (lane % CH);
#pragma unroll 1
    for (int i = 0; i < 16; i += RPI) {
        const int r = r0 + i;
        const uint32_t to = tiles + (r >> 7) * (256 * D) + tile_chunk(r & 127, lane % CH);
        if (r < rows) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(first) : "memory");
        else sts128(to, 0, 0, 0, 0);
        // the row RPI further on, from pointer to pointer: multiplied out, 16 warps' rows took 2 us
        first += RPI * head_step;
        for (head += RPI; head >= group; head -= group) first += token_step - group * head_step;
    }
}

template <int D, bool BF16, typename RowAt>
__device__ __forceinline__ void convert_rows(RowAt&& row_at, uint32_t tiles, float* exponent) {
    constexpr int CH = D / 8, HALF = CH / 2;
    const int lane = threadIdx.x & 31, r = (threadIdx.x >> 5) * 16 + (lane >> 1), c0 = (lane & 1) * HALF;  // 16 rows a warp
    const uint32_t tile = tiles + (r >> 7) * (256 * D);
    const float4* row = BF16 ? nullptr : reinterpret_cast<const float4*>(row_at(r));
    const float4 z = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float most = 0.0f, e, up;
#pragma unroll 4
    for (int i = c0; i < c0 + HALF; ++i) {
        if constexpr (BF16) {
            const uint4 w = lds128(tile + tile_chunk(r & 127, i));
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
                most = max3(most, fabsf(__uint_as_float(u[k] << 16)), fabsf(__uint_as_float(u[k] & 0xffff0000u)));
        } else {
            const float4 x = row ? row[2 * i] : z, y = row ? row[2 * i + 1] : z;
            most = max3(max3(most, fabsf(x.x), fabsf(x.y)), fabsf(x.z), fabsf(x.w));
            most = max3(max3(most, fabsf(y.x), fabsf(y.y)), fabsf(y.z), fabsf(y.w));
        }
    }
    most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
    query_factor(most, e, up);
#pragma unroll 2
    for (int i = c0; i < c0 + HALF; ++i) {
        const uint32_t at = tile + tile_chunk(r & 127, i);
        if constexpr (BF16) {
            const uint4 w = lds128(at);
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
            uint32_t h[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) h[k] = half_pair(__uint_as_float(u[k] << 16) * up, __uint_as_float(u[k] & 0xffff0000u) * up);
            sts128(at, h[0], h[1], h[2], h[3]);
        } else {
            const float4 x = row ? row[2 * i] : z, y = row ? row[2 * i + 1] : z;
            sts128(at, half_pair(x.x * up, x.y * up), half_pair(x.z * up, x.w * up), half_pair(y.x * up, y.y * up), half_pair(y.z * up, y.w * up));
        }
    }
    if ((lane & 1) == 0) exponent[r] = e;
    fence_proxy_async_smem();
}

// Codes of the step's keys and values in registers, a step ahead, and their way into shared memory (the form that expands
// inside).  Thread `tid` of 192 has chunk tid % (D / 16) of rows tid / (D / 16) + i * 192 / (D / 16).
template <int D, int FMT>
struct Expander {
    using C = Codes<FMT>;
    static constexpr int CH = D / 16, RS = kExpandThreads / CH, RPT = (128 + RS - 1) / RS;
    const AttnParams& p;
    const int b, kvh, p_min, p_max, ch, r0;
    int page[RPT], row[RPT];
    uint4 k[RPT], v[RPT];

    __device__ __forceinline__ Expander(const AttnParams& p_, int b_, int kvh_, int lo, int hi, int tid)
        : p(p_), b(b_), kvh(kvh_), p_min(lo), p_max(hi), ch(tid % CH), r0(tid / CH) {}
    __device__ __forceinline__ bool seen(int j0, int i) const {
        return r0 + i * RS < 128 && some_see(p, p_min, p_max, j0 + r0 + i * RS);
    }
    __device__ __forceinline__ void look_up(int j0) {  // the pages of a step's rows
#pragma unroll
        for (int i = 0; i < RPT; ++i) page[i] = seen(j0, i) ? page_of(p, b, j0 + r0 + i * RS) : 0;
    }
    __device__ __forceinline__ void rows(int j0) {  // unseen: -1, zeros
#pragma unroll
        for (int i = 0; i < RPT; ++i) row[i] = seen(j0, i) ? row_in(p, page[i], kvh, j0 + r0 + i * RS) : -1;
    }
    __device__ __forceinline__ void load(const uint8_t* codes, uint4 (&raw)[RPT]) {
#pragma unroll
        for (int i = 0; i < RPT; ++i)
            raw[i] = row[i] >= 0 ? __ldg(reinterpret_cast<const uint4*>(codes + static_cast<int64_t>(row[i]) * D) + ch) : make_uint4(0, 0, 0, 0);
    }
    // `scales`: shared memory, fp32 [128], of values; 0: the codes as they are
    __device__ __forceinline__ void store(uint32_t tile_at, const uint4 (&raw)[RPT], uint32_t scales, float inv) {
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const int r = r0 + i * RS;
            if (RPT * RS > 128 && r >= 128) break;
            const uint32_t w[4] = {C::ready(raw[i].x), C::ready(raw[i].y), C::ready(raw[i].z), C::ready(raw[i].w)};
            uint32_t h[8];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                h[2 * q] = C::value(C::template raw<0, 1>(w[q]));
                h[2 * q + 1] = C::value(C::template raw<2, 3>(w[q]));
            }
            if (scales) {
                float s;
                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(s) : "r"(scales + r * 4));
                const uint32_t s2 = half_pair(s * inv, s * inv);
#pragma unroll
                for (int q = 0; q < 8; ++q) h[q] = hmul2(h[q], s2);
            }
            // lanes of the second half store their chunks the other way round: no two of eight lanes share banks
            const uint32_t a = tile_at + tile_chunk(r, 2 * ch), z = tile_at + tile_chunk(r, 2 * ch + 1);
            if (ch < 4) {
                sts128(a, h[0], h[1], h[2], h[3]);
                sts128(z, h[4], h[5], h[6], h[7]);
            } else {
                sts128(z, h[4], h[5], h[6], h[7]);
                sts128(a, h[0], h[1], h[2], h[3]);
            }
        }
        fence_proxy_async_smem();
        __syncwarp();
    }
};

template <int D, int FMT, bool AHEAD>
__global__ void __launch_bounds__(kThreads, 1) rows_kernel(const __grid_constant__ AttnParams p) {
    using L = Rows<D, AHEAD>;
    extern __shared__ uint8_t dyn[];
    __shared__ __align__(8) uint64_t k_full[L::kKeys], k_empty[L::kKeys], v_full[2], v_empty[2], s_full[2], p_ready[2][2], o_done[2], drained;
    __shared__ uint32_t tmem_slot, abort_flag, scale_max[2][4];
    __shared__ float exponent[kRowTile];  // of the powers of two that the rows were multiplied by
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, wg = warp >> 2;
    const WaitCtl ctl{&abort_flag, p.status, p.wait_limit_ns};
    const uint32_t base = (smem_u32(dyn) + 1023u) & ~1023u;

    // the last row tiles see the most keys: they go first
    const int split = blockIdx.x % p.splits, it = blockIdx.x / p.splits;
    const int kvh = it % p.heads, tile = p.row_tiles - 1 - it / p.heads, b = blockIdx.y;
    if (AHEAD && threadIdx.x < 2) tma_prefetch_map(threadIdx.x ? &p.vmap : &p.kmap);
    // Ahead: what a CTA reads before it waits for the expansion -- lengths and bf16 queries, both by way of L2 -- comes from
    // grids that had ended before this one could begin: the expansion's blocks let it in after their own wait.  (No CTA
    // leaves without the wait, or the grid could end before the expansion does.)
    const bool early = AHEAD && p.q_bf16;
    auto begin = [&] {
        griddep_wait();
        griddep_launch_dependents();
    };
    if (!early) begin();
    const Seq s = sequence(p, b);
    const int rows = s.n * p.group, row0 = tile * kRowTile;
    if (row0 >= rows) {  // the whole CTA
        if (early) begin();
        return;
    }
    const int row_end = min(rows, row0 + kRowTile), tiles = row_end - row0 > 128 ? 2 : 1;
    const int p_min = s.pos + row0 / p.group, p_max = s.pos + (row_end - 1) / p.group;
    const Keys keys = key_steps(p, p_min, p_max, kStep);
    const int per = (keys.steps + p.splits - 1) / p.splits;
    const int s0 = min(split * per, keys.steps), n = min(s0 + per, keys.steps) - s0;
    // ahead: where step i of this CTA is among the sequence's expanded steps
    const Keys all = AHEAD ? key_steps(p, s.pos, s.pos + s.n - 1, kStep) : keys;
    const int64_t expanded = (static_cast<int64_t>(b) * p.heads + kvh) * p.step_cap;
    auto step_at = [&](int i) { return expanded + all.index(keys.first(s0 + i) / kStep); };

    // a step's keys or values into shared memory, by one thread
    auto copy_step = [&](int j, uint64_t& bar, const CUtensorMap& from, int to) {
        const int row = static_cast<int>(step_at(j) * kStep);
        mbar_arrive_expect_tx(&bar, L::kTileBytes);
        for (int h = 0; h < D / 64; ++h) tma_load_2d(dyn + (base - smem_u32(dyn)) + to + h * L::kHalf, &from, 64 * h, row, &bar);
    };
    if (threadIdx.x == 256) {
        abort_flag = 0;
        mbar_init(&drained, 1);
        for (int i = 0; i < L::kKeys; ++i) {
            mbar_init(&k_full[i], AHEAD ? 1 : kExpandWarps);
            mbar_init(&k_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&v_full[i], AHEAD ? 1 : kExpandWarps);
            mbar_init(&v_empty[i], 1);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_ready[i][0], 4);
            mbar_init(&p_ready[i][1], 4);
            mbar_init(&o_done[i], 1);
        }
        fence_barrier_init();
    }
    const RowMap map(row0, p.group);
    auto q_at = [&](int i) -> const char* {
        if (row0 + i >= row_end) return nullptr;
        int query, head;
        map.at(i, query, head);
        return static_cast<const char*>(p.q) + ((s.first + query) * p.q_token + (kvh * p.group + head) * p.q_head) * (p.q_bf16 ? 2 : 4);
    };
    if (p.q_bf16) {
        const int i = warp * 16 + lane / (D / 8);
        int query, head;
        map.at(i, query, head);
        copy_rows<D>(static_cast<const char*>(p.q) + ((s.first + query) * p.q_token + (kvh * p.group + head) * p.q_head) * 2, head, p.group,
                     2 * p.q_token, 2 * p.q_head, row_end - row0, base);
    }
    if (warp == 12) {
        tmem_alloc(&tmem_slot, 512);
        tmem_relinquish();
    }
    if (early) begin();
    if (AHEAD && threadIdx.x == 256) {  // the first steps' copies, before the CTA meets
        for (int j = 0; j < min(n, 2); ++j) {
            copy_step(j, k_full[j], p.kmap, L::kOffK + j * L::kTileBytes);
            copy_step(j, v_full[j], p.vmap, L::kOffV + j * L::kTileBytes);
        }
    }
    if (p.q_bf16) {
        cp_async_wait_all();
        __syncwarp();
        convert_rows<D, true>(q_at, base, exponent);
    } else {
        convert_rows<D, false>(q_at, base, exponent);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;

    // codes to fp16, by the warps of two warpgroups
    auto expand_all = [&](int tid) {
        if (n == 0) return;
        Expander<D, FMT> x(p, b, kvh, p_min, p_max, tid);
        constexpr int kVs = kExpandThreads - 128;
        // key scales by threads 0 .. 127, value scales by 64 .. 191, the thread of key i its number + 64
        float ks = 0.0f, vs = 0.0f;
        auto scales = [&](int j0) {
            ks = vs = 0.0f;
            // a key or value that is no number makes its key's logits NaN, for the rows that see it, and meets no weight of 0
            if (tid < 128 && some_see(p, p_min, p_max, j0 + tid)) {
                const int at = cache_row(p, b, kvh, j0 + tid);
                ks = __ldg(p.k_scale + at);
                if (!finite(__ldg(p.v_scale + at))) ks = not_a_number();
            }
            if (tid >= kVs && some_see(p, p_min, p_max, j0 + tid - kVs)) {
                vs = __ldg(p.v_scale + cache_row(p, b, kvh, j0 + tid - kVs));
                if (!finite(vs)) vs = 0.0f;
            }
        };
        int j0 = keys.first(s0);
        x.look_up(j0);
        x.rows(j0);
        x.load(p.k, x.k);
        x.load(p.v, x.v);
        scales(j0);
        if (n > 1) x.look_up(keys.first(s0 + 1));
        // a wait that gave up: its warp goes on without waiting, because the six meet at a named barrier
        bool ok = true;
        for (int j = 0; j < n; ++j) {
            const int slot = j & 1, use = j >> 1;
            const uint32_t meta = base + L::kOffMeta + (j % kMeta) * L::kMetaBytes;
            // E of the step: the largest value scale, which the last four of the six warps have
            const uint32_t big = __reduce_max_sync(0xffffffffu, __float_as_uint(vs));
            if (tid >= kVs && lane == 0) scale_max[slot][(tid - kVs) >> 5] = big;
            if (tid < 128) asm volatile("st.shared.f32 [%0], %1;" ::"r"(meta + tid * 4), "f"(ks) : "memory");
            if (tid >= kVs) asm volatile("st.shared.f32 [%0], %1;" ::"r"(meta + (kStep + tid - kVs) * 4), "f"(vs) : "memory");
            named_bar_sync(1, kExpandThreads);
            const uint32_t most = max(max(scale_max[slot][0], scale_max[slot][1]), max(scale_max[slot][2], scale_max[slot][3]));
            float ev, iv;
            exponent_of(__uint_as_float(most), -24, ev, iv);
            if (tid == 0) asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(meta + 2 * kStep * 4), "f"(ev), "f"(iv) : "memory");
            ok = ok && all_ok_warp(mbar_poll(&k_empty[slot], (use & 1) ^ 1, ctl));
            x.store(base + L::kOffK + slot * L::kTileBytes, x.k, 0u, 0.0f);
            if (lane == 0) mbar_arrive(&k_full[slot]);
            if (j + 1 < n) {
                j0 = keys.first(s0 + j + 1);
                x.rows(j0);
                x.load(p.k, x.k);
                scales(j0);
                if (j + 2 < n) x.look_up(keys.first(s0 + j + 2));
            }
            ok = ok && all_ok_warp(mbar_poll(&v_empty[slot], (use & 1) ^ 1, ctl));
            x.store(base + L::kOffV + slot * L::kTileBytes, x.v, meta + kStep * 4, iv);
            if (lane == 0) mbar_arrive(&v_full[slot]);
            if (j + 1 < n) x.load(p.v, x.v);
        }
    };

    if (wg < 2) {
        regs_inc<Regs<AHEAD>::kSoftmax>();
        if (wg < tiles) {
            const int t = wg, local = t * 128 + (threadIdx.x & 127), r = row0 + local;
            const bool live = r < row_end;
            const int at = live ? s.pos + r / p.group : -1;
            const float c = p.c * exp2f(exponent[local]);
            const int w_min = s.pos + (row0 + t * 128) / p.group, w_max = s.pos + (min(row_end, row0 + t * 128 + 128) - 1) / p.group;
            const uint32_t quarter = static_cast<uint32_t>(warp & 3) << 21;  // 32 lanes, in the address's upper half
            const uint32_t ts = tmem + quarter + t * 128, to = tmem + quarter + L::kColO + t * D;

            float m = -INFINITY, l = 0.0f;
            bool ok = true;
            float4 next = make_float4(1.0f, 0.0f, 1.0f, 0.0f);  // ahead: a step's 2^E of keys, E and 2^-E of values
            if (AHEAD && n > 0) next = __ldcg(p.step_info + step_at(0));
            for (int j = 0; j < n; ++j) {
                const float4 info = next;
                if (AHEAD && j + 1 < n) next = __ldcg(p.step_info + step_at(j + 1));
                ok = all_ok_warp(mbar_poll(&s_full[t], j & 1, ctl));
                if (!ok) break;
                tc_fence_after();
                uint32_t x[4][32];
#pragma unroll
                for (int i = 0; i < 4; ++i) tmem_ld_32x32b_x32(ts + 32 * i, x[i]);
                const uint32_t meta = base + L::kOffMeta + (j % kMeta) * L::kMetaBytes;
                const int j0 = keys.first(s0 + j);
                float ev = info.y, iv = info.z;
                if constexpr (!AHEAD)
                    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(ev), "=f"(iv) : "r"(meta + 2 * kStep * 4) : "memory");
                // not 0, which would make NaN of the -inf of hidden keys (a NaN stays one)
                const float cj = c * info.x < 0x1p-126f ? 0x1p-126f : c * info.x;
#pragma unroll
                for (int i = 0; i < 4; ++i) tmem_wait_ld32(x[i]);
                if constexpr (!AHEAD) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int k = 0; k < 32; k += 4) {
                            uint64_t a0, a1;
                            asm volatile("ld.shared.v2.u64 {%0, %1}, [%2];" : "=l"(a0), "=l"(a1) : "r"(meta + (32 * i + k) * 4));
                            float u, v;
                            upk2(mul2(pk2(__uint_as_float(x[i][k]), __uint_as_float(x[i][k + 1])), a0), u, v);
                            x[i][k] = __float_as_uint(u);
                            x[i][k + 1] = __float_as_uint(v);
                            upk2(mul2(pk2(__uint_as_float(x[i][k + 2]), __uint_as_float(x[i][k + 3])), a1), u, v);
                            x[i][k + 2] = __float_as_uint(u);
                            x[i][k + 3] = __float_as_uint(v);
                        }
                }
                if (!all_see(p, w_min, w_max, j0, kStep)) {
                    // the keys that the row sees, a bit each (comparisons key by key took 12000 cycles a step)
                    const int hi = at - j0, lo = p.window > 0 ? hi - p.window : -1, first = p.sinks - j0;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t see = bits_below(hi + 1 - 32 * i) & (~bits_below(lo + 1 - 32 * i) | bits_below(first - 32 * i));
#pragma unroll
                        for (int k = 0; k < 32; ++k) x[i][k] = see & (1u << k) ? x[i][k] : 0xff800000u;
                    }
                }
                float top4[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    top4[i] = max3(__uint_as_float(x[i][0]), __uint_as_float(x[i][1]), __uint_as_float(x[i][2]));
#pragma unroll
                    for (int k = 3; k < 31; k += 2) top4[i] = max3(top4[i], __uint_as_float(x[i][k]), __uint_as_float(x[i][k + 1]));
                    top4[i] = fmaxf(top4[i], __uint_as_float(x[i][31]));
                }
                const float top = fmaf(fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3])), cj, ev);
                if (__any_sync(0xffffffffu, top > m + kLag)) {
                    const float now = top > m + kLag ? top : m;
                    const float f = m == now ? 1.0f : exp2_fast(m - now);
                    m = now;
                    l *= f;
                    if (j > 0) {  // the sums so far, out of TMEM and back
                        ok = all_ok_warp(mbar_poll(&o_done[t], (j - 1) & 1, ctl));
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int d = 0; d < D; d += 32) {
                            uint32_t o[32];
                            tmem_ld_32x32b_x32(to + d, o);
                            tmem_wait_ld32(o);
                            const uint64_t f2 = pk2(f, f);
#pragma unroll
                            for (int k = 0; k < 32; k += 2) {
                                float u, v;
                                upk2(mul2(pk2(__uint_as_float(o[k]), __uint_as_float(o[k + 1])), f2), u, v);
                                o[k] = __float_as_uint(u);
                                o[k + 1] = __float_as_uint(v);
                            }
                            tmem_st_32x32b_x16(to + d, o);
                            tmem_st_32x32b_x16(to + d + 16, o + 16);
                        }
                    }
                }
                const float ref = ev + kBoost - (m == -INFINITY ? 0.0f : m);
                const uint64_t c2 = pk2(cj, cj), r2 = pk2(ref, ref);
                uint64_t sum = 0, sum1 = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t h[16];
#pragma unroll
                    for (int k = 0; k < 32; k += 4) {
                        float u, v;
                        upk2(fma2(pk2(__uint_as_float(x[i][k]), __uint_as_float(x[i][k + 1])), c2, r2), u, v);
                        u = exp2_fast(u);
                        v = exp2_fast(v);
                        sum = add2(sum, pk2(u, v));
                        h[k / 2] = half_pair(u, v);
                        upk2(fma2(pk2(__uint_as_float(x[i][k + 2]), __uint_as_float(x[i][k + 3])), c2, r2), u, v);
                        u = exp2_fast(u);
                        v = exp2_fast(v);
                        sum1 = add2(sum1, pk2(u, v));
                        h[k / 2 + 1] = half_pair(u, v);
                    }
                    tmem_st_32x32b_x16(ts + 16 * i, h);
                    if (i & 1) {  // half of the keys: the tensor cores may begin
                        tmem_wait_st();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&p_ready[t][i >> 1]);
                    }
                }
                float u, v;
                upk2(add2(sum, sum1), u, v);
                l = fmaf(u + v, iv, l);
            }
            if (ok && n > 0) {
                ok = all_ok_warp(mbar_poll(&o_done[t], (n - 1) & 1, ctl));
                tc_fence_after();
            }
            // out: a thread writes its row, 32 values at a time (by way of shared memory, rows whole, took twice as long)
            const int64_t item = (static_cast<int64_t>(b) * p.heads + kvh) * p.row_tiles + tile;
            // nothing seen: no weight (a NaN among the logits leaves m as it was, but l NaN)
            const bool none = n == 0 || !ok || l == 0.0f, partial = p.splits > 1;
            const float f = none ? 0.0f : partial ? 1.0f : 1.0f / l;
            const int64_t slot = (item * p.splits + split) * kRowTile + local;
            if (partial && live) p.part_ml[slot] = make_float2(none ? -INFINITY : held_reference(m, l), l);
            int query, head;
            map.at(local, query, head);
            const int64_t row = (s.first + query) * p.out_token + (kvh * p.group + head) * p.out_head;
            const bool narrow = !partial && p.out_bf16;
            float* dst = partial ? p.part + slot * D : static_cast<float*>(p.out) + row;
            __nv_bfloat16* dst16 = static_cast<__nv_bfloat16*>(p.out) + row;
#pragma unroll 1
            for (int d = 0; d < D; d += 32) {
                uint32_t o[32];
                if (n > 0) {
                    tmem_ld_32x32b_x32(to + d, o);
                    tmem_wait_ld32(o);
                }
                if (!live) continue;
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(none ? 0.0f : __uint_as_float(o[k]) * f);
                if (narrow) {
                    uint32_t h[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h[k]) : "f"(__uint_as_float(o[2 * k + 1])), "f"(__uint_as_float(o[2 * k])));
#pragma unroll
                    for (int k = 0; k < 16; k += 4) *reinterpret_cast<uint4*>(dst16 + d + 2 * k) = make_uint4(h[k], h[k + 1], h[k + 2], h[k + 3]);
                } else {
#pragma unroll
                    for (int k = 0; k < 32; k += 4) *reinterpret_cast<uint4*>(dst + d + k) = make_uint4(o[k], o[k + 1], o[k + 2], o[k + 3]);
                }
            }
            tc_fence_before();
        }
    } else if (wg == 2) {
        regs_dec<Regs<AHEAD>::kThird>();
        if constexpr (AHEAD) {
            if (warp == 8) {
                bool ok = true;
                int keys_done = min(n, 2), values_done = keys_done;
                for (int j = keys_done; j < n; ++j) {
                    const int kslot = j % L::kKeys, vslot = j & 1;
                    ok = all_ok_warp(mbar_poll(&k_empty[kslot], ((j / L::kKeys) & 1) ^ 1, ctl));
                    if (!ok) break;
                    if (lane == 0) copy_step(j, k_full[kslot], p.kmap, L::kOffK + kslot * L::kTileBytes);
                    __syncwarp();
                    keys_done = j + 1;
                    ok = all_ok_warp(mbar_poll(&v_empty[vslot], ((j >> 1) & 1) ^ 1, ctl));
                    if (!ok) break;
                    if (lane == 0) copy_step(j, v_full[vslot], p.vmap, L::kOffV + vslot * L::kTileBytes);
                    __syncwarp();
                    values_done = j + 1;
                }
                // what is still in flight lands before the CTA leaves
                for (int j = max(0, keys_done - L::kKeys); j < keys_done; ++j) land(smem_u32(&k_full[j % L::kKeys]), (j / L::kKeys) & 1);
                for (int j = max(0, values_done - 2); j < values_done; ++j) land(smem_u32(&v_full[j & 1]), (j >> 1) & 1);
            }
        } else {
            expand_all(threadIdx.x - 256);
        }
    } else {
        regs_dec<Regs<AHEAD>::kLast>();
        if (warp >= 14) {  // (13 has nothing to do)
            if constexpr (!AHEAD) expand_all(threadIdx.x - 448 + 128);  // warps 14, 15: threads 128 .. 191 of them
        } else if (warp == 12) {
            // One thread runs the whole loop, over values that the compiler knows to be the warp's: with a lane's branch around
            // each group of MMAs an MMA took 108 cycles to issue, for 69 that it lasts.  The tiles take turns, each with its whole
            // step (the second product, then the next step's first): interleaved, both tiles' scores come at once, and the
            // tensor cores rest while both softmaxes run.
            const int un = __shfl_sync(0xffffffffu, n, 0), utiles = __shfl_sync(0xffffffffu, tiles, 0);
            const uint32_t utmem = __shfl_sync(0xffffffffu, tmem, 0), ubase = __shfl_sync(0xffffffffu, base, 0);
            if (un > 0 && elect_one()) {
                constexpr uint32_t kIdS = (1u << 4) | ((128u >> 3) << 17) | ((128u >> 4) << 24);               // fp16, fp16 -> fp32
                constexpr uint32_t kIdO = (1u << 4) | (1u << 16) | ((D >> 3) << 17) | ((128u >> 4) << 24);  // B MN-major
                // an address in a descriptor counts 16 bytes: steps are added to it
                const uint64_t q_desc = smem_desc(ubase, 1024, 2), k_desc = smem_desc(ubase + L::kOffK, 1024, 2);
                const uint64_t v_desc = smem_desc(ubase + L::kOffV, 1024, 2, L::kHalf);
                constexpr uint32_t kStride = L::kTileBytes >> 4;
                auto score = [&](uint32_t t, uint32_t slot) {
                    const uint64_t qd = q_desc + t * kStride, kd = k_desc + slot * kStride;
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint32_t off = ((k / 4) * L::kHalf + (k % 4) * 32) >> 4;
                        mma_f16(utmem + t * 128, qd + off, kd + off, kIdS, k > 0);
                    }
                    mma_commit(&s_full[t]);
                };
                bool ok = mbar_poll(&k_full[0], 0, ctl);
                if (ok) {
                    tc_fence_after();
                    for (int t = 0; t < utiles; ++t) score(t, 0);
                    mma_commit(&k_empty[0]);
                    ok = mbar_poll(&v_full[0], 0, ctl) && (un < 2 || mbar_poll(&k_full[1], 0, ctl));
                }
#pragma unroll 1
                for (int j = 0; ok && j < un; ++j) {
                    const uint32_t slot = j & 1, after = (j + 1) % L::kKeys;
#pragma unroll 1
                    for (int t = 0; ok && t < utiles; ++t) {
                        const uint64_t vd = v_desc + slot * kStride;
                        const uint32_t od = utmem + L::kColO + t * D, pd = utmem + t * 128;
                        if (!(ok = mbar_poll(&p_ready[t][0], j & 1, ctl))) break;
                        tc_fence_after();
#pragma unroll
                        for (int k = 0; k < 4; ++k) mma_f16_ts(od, pd + k * 8, vd + k * (2048 >> 4), kIdO, j > 0 || k > 0);
                        if (!(ok = mbar_poll(&p_ready[t][1], j & 1, ctl))) break;
                        tc_fence_after();
#pragma unroll
                        for (int k = 4; k < 8; ++k) mma_f16_ts(od, pd + k * 8, vd + k * (2048 >> 4), kIdO, 1);
                        mma_commit(&o_done[t]);
                        if (t == utiles - 1) mma_commit(&v_empty[slot]);
                        if (j + 1 < un) {
                            score(t, after);
                            if (t == utiles - 1) mma_commit(&k_empty[after]);
                            // the next step's copies; with three steps of keys here, where MMAs are queued behind this thread: a
                            // look at a barrier takes some 160 cycles even where the phase is long complete
                            if (t == (AHEAD ? 0 : utiles - 1))
                                ok = mbar_poll(&v_full[slot ^ 1], ((j + 1) >> 1) & 1, ctl) &&
                                     (j + 2 >= un || mbar_poll(&k_full[(j + 2) % L::kKeys], ((j + 2) / L::kKeys) & 1, ctl));
                        }
                    }
                }
                // nothing leaves while an MMA is in flight
                mma_commit(&drained);
                const uint64_t t0 = globaltimer_ns();
                while (!mbar_try_wait(smem_u32(&drained), 0))
                    if (globaltimer_ns() - t0 > 100000000ull) break;
            }
            __syncwarp();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 12) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// The sequence's seen keys and values as fp16, code * scale * 2^-E, in the order of its steps: block (step, head) of
// sequence blockIdx.y.  Bound by memory at long prompts (a code read, two bytes written for it), by three loads one
// after the other (lengths, pages, codes and scales) at short ones.
template <int D, int FMT>
__global__ void __launch_bounds__(256) expand_kernel(const __grid_constant__ AttnParams p) {
    griddep_wait();
    griddep_launch_dependents();
    __shared__ float scale[2][kStep];
    __shared__ uint32_t most[2][4];
    const int step = blockIdx.x / p.heads, kvh = blockIdx.x % p.heads, b = blockIdx.y;
    const Seq s = sequence(p, b);
    if (s.n == 0) return;
    const int p_min = s.pos, p_max = s.pos + s.n - 1;
    const Keys keys = key_steps(p, p_min, p_max, kStep);
    if (step >= keys.steps || step >= p.step_cap) return;
    const int j0 = keys.first(step), tid = threadIdx.x;
    constexpr int CH = D / 16, RS = 256 / CH, N = kStep / RS;  // a thread: chunk tid % CH of rows tid / CH + i RS
    const int ch = tid % CH, r0 = tid / CH;
    int page[N], row[N];
    const int which = tid >> 7, key = tid & 127;  // and the scale of a key, or of a value
    const bool seen = some_see(p, p_min, p_max, j0 + key);
    const int my_page = seen ? page_of(p, b, j0 + key) : 0;
#pragma unroll
    for (int i = 0; i < N; ++i) page[i] = some_see(p, p_min, p_max, j0 + r0 + i * RS) ? page_of(p, b, j0 + r0 + i * RS) : 0;
    uint4 raw[2][N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int j = j0 + r0 + i * RS;
        row[i] = some_see(p, p_min, p_max, j) ? row_in(p, page[i], kvh, j) : -1;
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int w = 0; w < 2; ++w)
            raw[w][i] = row[i] >= 0 ? __ldg(reinterpret_cast<const uint4*>((w ? p.v : p.k) + static_cast<int64_t>(row[i]) * D) + ch)
                                    : make_uint4(0, 0, 0, 0);
    const float sc = seen ? __ldg((which ? p.v_scale : p.k_scale) + row_in(p, my_page, kvh, j0 + key)) : 0.0f;
    scale[which][key] = sc;
    const uint32_t big = __reduce_max_sync(0xffffffffu, finite(sc) ? __float_as_uint(sc) : 0u);
    if ((tid & 31) == 0) most[which][(tid >> 5) & 3] = big;
    __syncthreads();
    const int64_t out = (static_cast<int64_t>(b) * p.heads + kvh) * p.step_cap + step;
    float e[2], inv[2];
#pragma unroll
    for (int w = 0; w < 2; ++w)
        exponent_of(__uint_as_float(max(max(most[w][0], most[w][1]), max(most[w][2], most[w][3]))), w ? -24 : 0, e[w], inv[w]);
    if (tid == 0) p.step_info[out] = make_float4(exp2f(e[0]), e[1], inv[1], 0.0f);
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        uint4* dst = reinterpret_cast<uint4*>((w ? p.v16 : p.k16) + out * kStep * D);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int r = r0 + i * RS;
            // a key or value that is no number makes its key's logits NaN, for the rows that see it, and meets no weight of 0
            const float f = w ? (finite(scale[1][r]) ? scale[1][r] * inv[1] : 0.0f)
                              : (finite(scale[1][r]) ? scale[0][r] * inv[0] : not_a_number());
            const uint32_t u[4] = {raw[w][i].x, raw[w][i].y, raw[w][i].z, raw[w][i].w};
            uint32_t h[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const uint32_t two = (u[q / 2] >> (16 * (q % 2))) & 0xffffu;
                float x, y;
                if constexpr (FMT == W4A8_KV_E4M3) {
                    uint32_t v2;
                    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(v2) : "h"(static_cast<uint16_t>(two)));
                    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&v2));
                    x = v.x;
                    y = v.y;
                } else {
                    x = static_cast<float>(static_cast<int8_t>(two & 0xffu));
                    y = static_cast<float>(static_cast<int8_t>(two >> 8));
                }
                h[q] = half_pair(x * f, y * f);
            }
            dst[2 * (r * CH + ch)] = make_uint4(h[0], h[1], h[2], h[3]);
            dst[2 * (r * CH + ch) + 1] = make_uint4(h[4], h[5], h[6], h[7]);
        }
    }
}

template <typename Kernel>
cudaError_t launch_dependent(Kernel kernel, dim3 grid, int threads, int smem, const AttnParams& p, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int D, int FMT, bool AHEAD>
cudaError_t launch(const AttnParams& p, int64_t batch, cudaStream_t s) {
    static bool attr_done[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !attr_done[dev]) {
        e = cudaFuncSetAttribute(rows_kernel<D, FMT, AHEAD>, cudaFuncAttributeMaxDynamicSharedMemorySize, (Rows<D, AHEAD>::kSmem));
        if (e != cudaSuccess) return e;
        if (dev < 64) attr_done[dev] = true;
    }
    if (AHEAD) {
        e = launch_dependent(expand_kernel<D, FMT>, dim3(p.step_cap * p.heads, static_cast<unsigned>(batch)), 256, 0, p, s);
        if (e != cudaSuccess) return e;
    }
    return launch_dependent(rows_kernel<D, FMT, AHEAD>, dim3(p.splits * p.heads * p.row_tiles, static_cast<unsigned>(batch)), kThreads,
                            (Rows<D, AHEAD>::kSmem), p, s);
}

template <int D, bool AHEAD>
cudaError_t launch_fmt(const AttnParams& p, int format, int64_t batch, cudaStream_t s) {
    return format == W4A8_KV_INT8 ? launch<D, W4A8_KV_INT8, AHEAD>(p, batch, s) : launch<D, W4A8_KV_E4M3, AHEAD>(p, batch, s);
}

}  // namespace

cudaError_t launch_attn_rows(AttnParams& p, const w4a8_kv_cache& c, int64_t batch, cudaStream_t s) {
    const int dim = static_cast<int>(c.head_dim);
    if (p.step_cap > 0) {
        const int64_t rows = batch * c.heads * p.step_cap * kStep;
        if (!make_rows_map(&p.kmap, p.k16, rows, 2 * dim, 128, kStep, 2) || !make_rows_map(&p.vmap, p.v16, rows, 2 * dim, 128, kStep, 2))
            return cudaErrorInvalidValue;
        return dim == 128 ? launch_fmt<128, true>(p, c.format, batch, s) : launch_fmt<64, true>(p, c.format, batch, s);
    }
    return dim == 128 ? launch_fmt<128, false>(p, c.format, batch, s) : launch_fmt<64, false>(p, c.format, batch, s);
}

}  // namespace w4a8

// fp8_gemm.cu -- matrix product in 8-bit floating point (e4m3) with a scale for each block of 128.
//
// The mathematics:  y[m,n] = sum_b sa[b,m] sw[n / 128, b] P_b[m,n] (+ bias[n]),
//                   P_b[m,n] = sum over the 128 columns k of block b of a[m,k] w[n,k].
// A scale changes from block to block, so the tensor cores can sum only inside a block: each
// block's product P_b gets a TMEM accumulator of its own, and the epilogue warps fold it into
// fp32 sums in registers, one fma a block and output, y += (sa sw) P_b, while the tensor cores
// form the next block's product in another accumulator.
//
// Two forms.  For large problems tokens are the MMA's M operand (TMEM lanes) and weight rows its N
// operand: a thread owns one token, and the factor sa sw is one scalar per thread, block and 128
// columns (pairs of CTAs, below).  For few tokens the roles are swapped.  Operand tiles come straight
// from the caller's row-major arrays by TMA, 128 columns = one scale block wide, 128-byte swizzled;
// rows past M or N and columns past K read as zeros, which add nothing to the products.
#include "device_memo.h"
#include "fp8_ptx.cuh"
#include "ops_internal.h"

#include <cuda_bf16.h>

namespace w4a8 {
namespace {

constexpr uint32_t kLayoutSw128 = 2;
// Register split of the 640-thread kernels: launch = 640 x 96 (checked at build time); the first four
// warps drop to 32, the sixteen draining warps rise to 112: 128 * 32 + 512 * 112 = 640 * 96.
constexpr int kRegsLow = 32, kRegsHigh = 112, kSplitThreads = 640;
// The 112 do not quite hold what a draining thread keeps beside its 64 sums and 32 loaded columns: the pair
// kernel spills 64 bytes a thread and loads 92, the 128-token form 92 and 112 (-Xptxas -v).
static_assert(128 * kRegsLow + 512 * kRegsHigh == kSplitThreads * 96, "register split");

struct Fp8Params {
    CUtensorMap amap, wmap, ymap;
    const float* sa;
    const float* sw;
    const float* bias;
    void* y;
    int bf16, vec;  // vec: 16-byte stores fit every row of y
    int64_t M, N;
    int nb, tiles_m, tiles_n;
    int split;  // CTAs (a cluster) sharing a tile's K
    uint32_t* status;
    uint64_t wait_limit_ns;
    uint32_t copy_blocks;  // a CTA's copies stop before this block (none: the last one's number is smaller)
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

// What follows a wait that gave up.  The flag that says so can rise between two lanes' reads of it, so
// no lane leaves a loop on its own: a warp decides for all its lanes together (all_ok), because the
// instructions ahead (TMEM loads, named barriers, __syncwarp) want the whole warp.
__device__ __forceinline__ bool all_ok(bool ok) { return __all_sync(0xffffffffu, ok); }

// The copies of blocks 0 .. issued - 1 that may still be in flight land (for a bounded time) before the
// CTA leaves; for one thread, once every role has ended.
template <int STAGES>
__device__ __forceinline__ void land_copies(uint64_t* full, uint32_t issued) {
    for (uint32_t q = issued > STAGES ? issued - STAGES : 0; q < issued; ++q)
        drain_wait(&full[q % STAGES], (q / STAGES) & 1, 10000000ull);
}

// ---------------------------------------------------------------- one CTA, weights on the lanes
// The form for few tokens and for problems that 256 x 256 tiles would not fill the GPU with.  Roles
// are swapped: 128 weight rows are the MMA's M operand (TMEM lanes) and TN tokens its N operand, so
// a tile is as narrow as the tokens ask for and a warp's stores run along a row of y.  A thread
// owns one weight row; the factor sa sw then differs from column to column and comes from shared
// memory, as products formed by a loader warp eight blocks at a time.
//   warp 0      copies      warps 1-2  every other block's 4 MMAs      warp 3  factors
//   warps 4..   drain, two sets: one takes the even blocks, one the odd
// What bounds it: few tokens, the weights' stream from HBM (stages in flight, and K split over a
// cluster of `split` CTAs so that every SM has some of it); more tokens, the drain.  Reading one
// accumulator costs a warp about 700 cycles of waits in a row (barrier, factors, TMEM) however few
// its columns, so the two sets work on two blocks at a time, each with sums of its own that are
// added at the end of a tile (8 x 4096 -> 14336 12.3 us, 13.6 with one set; 512 x 2048 -> 6144 with
// 128-token tiles 17.5 and 27, of which generic loads were part).  A split sums each output's parts in
// the order of the ranks, each CTA for its share of the columns, read from the others' shared memory.
template <int TN_>
struct Tok {
    static constexpr int TN = TN_;
    static constexpr int kSetWarps = TN <= 32 ? 4 : 8;  // warps of one set
    static constexpr int kCols = TN * 4 / kSetWarps;    // columns a thread sums
    static constexpr int kThreads = 128 + 64 * kSetWarps;
    static constexpr int kNBuf = 4;                     // TMEM accumulators
    static constexpr int kStages = TN <= 32 ? 10 : TN <= 64 ? 6 : 4;
    static constexpr int kWBytes = 128 * 128, kStageBytes = kWBytes + TN * 128;
    static constexpr uint32_t kTmemCols = TN * kNBuf;
    static constexpr int kChunk = 8;                    // blocks per batch of factors
    static constexpr int kOffPart = kStages * kStageBytes;  // the sets' exchange area [column][weight row]
    static constexpr int kOffScale = kOffPart + TN * 512;
    static constexpr int kScaleBytes = kChunk * TN * 4;
    static constexpr int kRawFloats = kChunk * TN + kChunk;  // the scales they are formed from: sa, then sw
    static constexpr int kOffRaw = kOffScale + 2 * kScaleBytes;
    static constexpr int kOffBar = kOffRaw + 2 * kRawFloats * 4;
    static constexpr int kSmemBytes = kOffBar + 512 + 1024;
    // The 640-thread form with 64 sums a thread re-splits its registers.
    static constexpr bool kResplit = kCols == 64;
    static_assert(!kResplit || kThreads == kSplitThreads, "register split");
    static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
    static_assert((kTmemCols & (kTmemCols - 1)) == 0 && kTmemCols >= 32 && kTmemCols <= 512, "TMEM allocation");
    // Each stage and each accumulator has one issuer and one set at every phase (their counts are
    // even); an accumulator's release for the block kNBuf later reaches that block's stage only
    // after the stage's previous phase.
    static_assert(kStages % 2 == 0 && kNBuf == 4 && kStages >= kNBuf, "phases");
    static_assert(TN % 16 == 0 && kCols % 16 == 0, "MMA N; TMEM loads of 16 columns");
};

// y[c] = fma(f[c], v[c], y[c]) for 16 columns, two per instruction; f from shared memory, the same
// for every lane.
__device__ __forceinline__ void fold16(float* y, const float* f, const uint32_t* v) {
#pragma unroll
    for (int c = 0; c < 16; c += 4) {
        const ulonglong2 ff = *reinterpret_cast<const ulonglong2*>(f + c);
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
            uint64_t yy, vv;
            asm("mov.b64 %0, {%1, %2};" : "=l"(yy) : "f"(y[c + e]), "f"(y[c + e + 1]));
            asm("mov.b64 %0, {%1, %2};" : "=l"(vv) : "r"(v[c + e]), "r"(v[c + e + 1]));
            asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(yy) : "l"(e ? ff.y : ff.x), "l"(vv));
            asm("mov.b64 {%0, %1}, %2;" : "=f"(y[c + e]), "=f"(y[c + e + 1]) : "l"(yy));
        }
    }
}

// The end of a tile: this thread's sums y of C columns (tokens m0 ..) of weight row n, of which it
// keeps the half from column K0 on.  `part`: the tile's exchange area [column][weight row], at this
// thread's first column and row; `threads`: of both sets.  Then the outputs, or, for a split tile, the
// CTA's sums into the area.
template <int C, int K0, int THREADS>
__device__ __forceinline__ void finish_cols(const Fp8Params& p, float* part, const float (&y)[C], int64_t m0, int64_t n,
                                            bool split, bool first) {
    constexpr int G0 = C / 2 - K0;  // the half it hands over
    __syncwarp();  // named barriers take whole warps
    if (!first) named_bar_sync(1, THREADS);  // the last tile's have been read
#pragma unroll
    for (int c = 0; c < C / 2; ++c) part[(G0 + c) * 128] = y[G0 + c];
    named_bar_sync(1, THREADS);
    if (split) {
#pragma unroll
        for (int c = 0; c < C / 2; ++c) part[(K0 + c) * 128] += y[K0 + c];
        return;
    }
    if (n >= p.N) return;
    const float bn = p.bias ? __ldcg(p.bias + n) : 0.0f;
    const int live = p.M - m0 < C ? static_cast<int>(p.M - m0) : C;
    if (p.bf16) {
        __nv_bfloat16* d = static_cast<__nv_bfloat16*>(p.y) + (m0 + K0) * p.N + n;
#pragma unroll
        for (int c = 0; c < C / 2; ++c, d += p.N)
            if (K0 + c < live) *d = __float2bfloat16_rn(y[K0 + c] + part[(K0 + c) * 128] + bn);
    } else {
        float* d = static_cast<float*>(p.y) + (m0 + K0) * p.N + n;
#pragma unroll
        for (int c = 0; c < C / 2; ++c, d += p.N)
            if (K0 + c < live) *d = y[K0 + c] + part[(K0 + c) * 128] + bn;
    }
}

// Columns c0 .. c1 - 1 (tokens) of a split tile: the sums [column][weight row] of `split` CTAs added
// in rank order; the draining warps' threads, G groups of 128.
template <int TN, int G>
__device__ __forceinline__ void store_share(const Fp8Params& p, const float* sums, uint32_t t, int c0, int c1,
                                            uint32_t split) {
    const int row = threadIdx.x & 127, g = (threadIdx.x - 128) >> 7;
    const int64_t n = static_cast<int64_t>(t / p.tiles_m) * 128 + row, m0 = static_cast<int64_t>(t % p.tiles_m) * TN;
    if (n >= p.N) return;
    if (p.M - m0 < c1) c1 = static_cast<int>(p.M - m0);
    const float bn = p.bias ? __ldcg(p.bias + n) : 0.0f;
    // eight columns' remote reads in flight (one at a time, 128 columns of two CTAs took 5 us)
    for (int c = c0 + g; c < c1; c += 8 * G) {
        float v[8] = {};
        for (uint32_t k = 0; k < split; ++k) {
            float r[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                r[e] = c + e * G < c1 ? ld_shared_cluster_f32(sums + (c + e * G) * 128 + row, k) : 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += r[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (c + e * G >= c1) break;
            const int64_t at = (m0 + c + e * G) * p.N + n;
            if (p.bf16) static_cast<__nv_bfloat16*>(p.y)[at] = __float2bfloat16_rn(v[e] + bn);
            else static_cast<float*>(p.y)[at] = v[e] + bn;
        }
    }
}

template <int TN>
__global__ void __launch_bounds__(Tok<TN>::kThreads, 1) fp8_tok_kernel(const __grid_constant__ Fp8Params p) {
    using T = Tok<TN>;
    constexpr int kStages = T::kStages, kStageBytes = T::kStageBytes, kNBuf = T::kNBuf, kCols = T::kCols,
                  kChunk = T::kChunk, kSetWarps = T::kSetWarps;
    extern __shared__ uint8_t smem_raw[];
    // by an offset, not by a cast of the address: the compiler then knows it for shared memory (through
    // generic loads the factors cost 512 x 8192 -> 2048 35 us for 31)
    uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + T::kOffBar);
    uint64_t* empty = full + kStages;
    uint64_t* tfull = empty + kStages;
    uint64_t* sfull = tfull + kNBuf;
    uint64_t* sempty = sfull + 2;
    uint64_t* drain = sempty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 2);
    volatile uint32_t* abort_flag = tmem_slot + 1;
    uint32_t* issued = tmem_slot + 2;  // blocks whose copies were issued; read after an abort
    float* factors = reinterpret_cast<float*>(smem + T::kOffScale);
    float* raw = reinterpret_cast<float*>(smem + T::kOffRaw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const WaitCtl ctl{abort_flag, p.status, p.wait_limit_ns};
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1 + kSetWarps);  // the copies, and a set's release of the accumulator
            mbar_init(&empty[s], 1);
        }
        for (int i = 0; i < kNBuf; ++i) mbar_init(&tfull[i], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sfull[i], 1);
            mbar_init(&sempty[i], 2 * kSetWarps);
            mbar_init(&drain[i], 1);
        }
        *abort_flag = 0u;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, T::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    griddep_launch_dependents();
    griddep_wait();
    // this CTA's share of K, and its tiles (one for a cluster that splits K)
    const uint32_t split = static_cast<uint32_t>(p.split), rank = blockIdx.x % split;
    const int per = (p.nb + p.split - 1) / p.split, kb0 = static_cast<int>(rank) * per;
    const int nb = p.nb - kb0 < per ? (p.nb - kb0 > 0 ? p.nb - kb0 : 0) : per;
    const uint32_t tiles = static_cast<uint32_t>(p.tiles_m) * static_cast<uint32_t>(p.tiles_n);
    const uint32_t first = blockIdx.x / split, step = gridDim.x / split;
    const uint32_t total = tiles > first ? ((tiles - 1 - first) / step + 1) * static_cast<uint32_t>(nb) : 0u;

    if (warp < 4) {
        if constexpr (T::kResplit) regs_dec<kRegsLow>();
        if (warp == 0) {
            if (lane == 0) {
                uint32_t j = 0;
                bool ok = true;
                for (uint32_t t = first; ok && t < tiles; t += step) {
                    const int m0 = static_cast<int>(t % p.tiles_m) * TN, n0 = static_cast<int>(t / p.tiles_m) * 128;
#pragma unroll 1
                    for (int b = 0; b < nb; ++b, ++j) {
                        const uint32_t s = j % kStages, k = j / kStages;
                        if (j >= p.copy_blocks || (k > 0 && !mbar_poll(&empty[s], (k - 1) & 1, ctl))) {
                            ok = false;
                            break;
                        }
                        mbar_arrive_expect_tx(&full[s], kStageBytes);
                        tma_load_2d(smem + s * kStageBytes, &p.wmap, (kb0 + b) * 128, n0, &full[s]);
                        tma_load_2d(smem + s * kStageBytes + T::kWBytes, &p.amap, (kb0 + b) * 128, m0, &full[s]);
                    }
                }
                *issued = j;
            }
            __syncwarp();
        } else if (warp <= 2) {
            constexpr uint32_t idesc = idesc_e4m3_f32(128, TN);
            const uint32_t par = warp - 1;
            const uint64_t dw0 = smem_desc(smem_u32(smem), 1024, kLayoutSw128);
            const uint64_t dt0 = smem_desc(smem_u32(smem + T::kWBytes), 1024, kLayoutSw128);
            if (elect_one()) {  // one thread runs the whole loop
                uint32_t s = par, phase = 0, buf = par;
#pragma unroll 1
                for (uint32_t j = par; j < total; j += 2) {
                    if (!mbar_poll(&full[s], phase, ctl)) break;
                    tc_fence_after();
                    const uint64_t o = static_cast<uint64_t>((s * kStageBytes) >> 4);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_f8f6f4(tmem + buf * TN, dw0 + o + 2 * k, dt0 + o + 2 * k, idesc, k > 0);
                    mma_commit(&tfull[buf]);
                    mma_commit(&empty[s]);
                    buf ^= 2u;
                    if ((s += 2) >= kStages) s -= kStages, phase ^= 1u;
                }
                mma_commit(&drain[par]);
            }
            __syncwarp();
            drain_wait(&drain[par], 0, 100000000ull);
        } else {
            // the scales of a batch are copied while the factors of the one before are formed (a loader
            // that waited for its loads held the drain up: 512 x 2048 -> 6144 took 30 us with one)
            uint32_t j = 0;  // batches
            uint32_t tn = first, bn = 0;  // the next batch to copy: tile, block
            auto copy = [&](uint32_t buf) {
                if (tn < tiles && nb > 0) {
                    const int64_t m0 = static_cast<int64_t>(tn % p.tiles_m) * TN;
                    const float* sw = p.sw + static_cast<int64_t>(tn / p.tiles_m) * p.nb + kb0 + bn;
                    const float* sa = p.sa + (kb0 + bn) * p.M + m0;
                    const int last = p.M - m0 < TN ? static_cast<int>(p.M - m0) - 1 : TN - 1;  // columns past M: unused
                    const int cnt = nb - static_cast<int>(bn) < kChunk ? nb - static_cast<int>(bn) : kChunk;
                    float* d = raw + buf * T::kRawFloats;
#pragma unroll 1
                    for (int c = lane; c < TN; c += 32) {
                        const float* src = sa + (c < last ? c : last);
#pragma unroll 1
                        for (int k = 0; k < cnt; ++k, src += p.M) cp_async4(d + k * TN + c, src);
                    }
                    if (lane < cnt) cp_async4(d + kChunk * TN + lane, sw + lane);
                    bn += kChunk;
                    if (static_cast<int>(bn) >= nb) bn = 0, tn += step;
                }
                cp_async_commit();
            };
            copy(0);
            bool ok = true;
            for (uint32_t t = first; ok && t < tiles; t += step) {
                for (int b0 = 0; b0 < nb; b0 += kChunk, ++j) {
                    const uint32_t buf = j & 1u, u = j >> 1;
                    const int cnt = nb - b0 < kChunk ? nb - b0 : kChunk;
                    copy(buf ^ 1u);
                    cp_async_wait<1>();
                    __syncwarp();
                    if (u > 0 && !(ok = all_ok(mbar_poll(&sempty[buf], (u - 1) & 1, ctl)))) break;
                    float* d = factors + buf * (kChunk * TN);
                    const float* r = raw + buf * T::kRawFloats;
#pragma unroll 1
                    for (int k = 0; k < cnt; ++k) {
                        const float w = r[kChunk * TN + k];
#pragma unroll
                        for (int c = 0; c < TN; c += 32)
                            if (TN >= 32 || lane < TN) d[k * TN + c + lane] = r[k * TN + c + lane] * w;
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sfull[buf]);
                }
            }
            cp_async_wait<0>();
            __syncwarp();
        }
    } else {
        if constexpr (T::kResplit) regs_inc<kRegsHigh>();
        // set, lane quarter, column group
        const uint32_t set = (warp - 4) / kSetWarps;
        const int q = warp & 3, g = ((warp - 4) % kSetWarps) >> 2;
        const uint32_t tl = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(g * kCols);
        float* part = reinterpret_cast<float*>(smem + T::kOffPart) + g * kCols * 128 + q * 32 + lane;
        // the accumulators start free
        if (lane == 0)
            for (uint32_t b = set; b < kNBuf && b < total; b += 2) mbar_arrive(&full[b]);
        uint32_t js = 0, odd = 0;  // batches of factors used; the parity of the batch's first block
        // of this set's next block: its accumulator (and, times 8, its barrier), that barrier's phase, and
        // the stage (times 8) that its release counts towards
        uint32_t buf = set, phase = 0, rel = (set + kNBuf) % kStages * 8;
        const uint32_t bars = smem_u32(tfull), release = smem_u32(full);
        // after a wait gave up this warp waits no more: its sums are then undefined (the status word
        // says so), but it still meets every barrier of the sets and of the cluster
        bool ok = true;
        for (uint32_t t = first; t < tiles; t += step) {
            float y[kCols];
#pragma unroll
            for (int c = 0; c < kCols; ++c) y[c] = 0.0f;
#pragma unroll 1
            for (int b0 = 0; b0 < nb; b0 += kChunk, ++js) {
                if (ok) ok = mbar_poll(&sfull[js & 1u], (js >> 1) & 1, ctl);
                const int cnt = nb - b0 < kChunk ? nb - b0 : kChunk;
                const float* f = factors + (js & 1u) * (kChunk * TN) + g * kCols;
                const float* end = f + cnt * TN;
                f += (set ^ odd) * TN;
                odd ^= cnt & 1;
#pragma unroll 1
                for (; f < end; f += 2 * TN) {
                    if (ok && __builtin_expect(!mbar_try_wait_long(bars + 8 * buf, phase), 0))
                        ok = mbar_wait_on(bars + 8 * buf, phase, ctl);
                    __syncwarp();
                    tc_fence_after();
                    const uint32_t ta = tl + buf * TN;
                    constexpr int kAt = kCols == 32 ? 32 : 16;  // columns read at a time
#pragma unroll
                    for (int c0 = 0; c0 < kCols; c0 += kAt) {
                        uint32_t v[kAt];
#pragma unroll
                        for (int c = 0; c < kAt; c += 16) tmem_ld_32x32b_x16(ta + c0 + c, v + c);
                        tmem_wait_ld();
#pragma unroll
                        for (int c = 0; c < kAt; ++c) asm volatile("" : "+r"(v[c]));  // uses stay behind the wait
                        if (c0 + kAt == kCols) {
                            // released for the block kNBuf later (past the last block: a barrier nobody waits for)
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive_on(release + rel);
                        }
#pragma unroll
                        for (int c = 0; c < kAt; c += 16) fold16(y + c0 + c, f + c0 + c, v + c);
                    }
                    phase ^= buf >> 1;
                    buf ^= 2u;
                    rel = rel + 16 >= 8 * kStages ? rel + 16 - 8 * kStages : rel + 16;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sempty[js & 1u]);
            }
            // each set hands half of its columns to the other, adds the half it is handed and stores it
            const int64_t m0 = static_cast<int64_t>(t % p.tiles_m) * TN + g * kCols;
            const int64_t n = static_cast<int64_t>(t / p.tiles_m) * 128 + q * 32 + lane;
            if (set == 0) finish_cols<kCols, 0, 64 * kSetWarps>(p, part, y, m0, n, split > 1, t == first);
            else finish_cols<kCols, kCols / 2, 64 * kSetWarps>(p, part, y, m0, n, split > 1, t == first);
        }
    }
    __syncwarp();
    if (split > 1) {
        cluster_sync_all();
        const int share = TN / static_cast<int>(split);
        if (warp >= 4)
            store_share<TN, 2 * kSetWarps / 4>(p, reinterpret_cast<const float*>(smem + T::kOffPart), first,
                                               static_cast<int>(rank) * share, (static_cast<int>(rank) + 1) * share, split);
        cluster_sync_all();  // no CTA leaves while another may still read its sums
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && *abort_flag) land_copies<kStages>(full, *issued);
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, T::kTmemCols);
    }
}

// ---------------------------------------------------------------- pairs of CTAs
// The large form: a cluster of two CTAs owns a 256 x 256 output tile.  One MMA covers 256 tokens
// x 128 weight rows over both SMs (cta_group::2): each CTA's shared memory holds its own 128
// tokens and half of the weight rows, so per SM and block 32 KB are copied and read where two
// lone 128 x 256 tiles would take 48.  The even CTA issues the MMAs; commits arrive on the barriers
// of both.
//   warp 0      copies: its tokens' and its half of the weights' boxes, four stages; both CTAs'
//               copies complete the even CTA's barrier
//   warps 1-2   (even CTA) every other block each: 2 x 4 MMAs of K = 32, one accumulator for each
//               half of the columns
//   warp 3      scales: eight blocks' sa and sw (and a tile's bias) at a time into shared memory,
//               one batch ahead
//   warps 4-19  drain, 4 lane quarters x 4 runs of 64 columns: a thread holds 64 sums
//
// Measured at 8192 x 4096 -> 14336 (bf16 out) on several GPUs: 333 to 347 us, 2.8 PFLOP/s, in short runs;
// 368 to 386 us, 2.5 PFLOP/s, in long ones, where the power limit holds the clock at 1.7 to 1.8 GHz.  What
// bounds it is not the tensor pipe (206 us for the MMAs alone, 258 with the copies and the issue) but what
// surrounds each block:
// 32768 fmas a CTA and block (256 cycles of the fp32 pipes, against 512 of the tensor pipe), and the
// accumulators' way from a commit over the drain back to the issuer, during which their TMEM lies
// idle (323 us without the fmas).  So:
//   - four accumulators of 128 columns rather than two of 256: each is handed back as soon as
//     eight warps of each CTA have read it;
//   - sixteen draining warps: a warp spends most of a block waiting (barrier, TMEM load), and four
//     warps a scheduler fill that time with one another's fmas (eight warps of 128 sums: 416 us
//     against 408 at that step);
//   - the halves of a block are released and waited for one by one: with one wait for both, the
//     first half's MMAs waited for the second half's drain (350 us, then 341); waits, MMAs and
//     commits of a block cost a thread about 700 cycles, so two issuers take turns.
// The outputs leave through a 4 KB staging box per warp and TMA stores (whole lines, rows past M
// and columns past N cut by the copy) while the tensor cores work on the next tile.
namespace pair {
constexpr int kThreads = 640, kEpiWarps = 16;
constexpr int kBM = 256, kBN = 256, kStages = 4;
constexpr int kABytes = 128 * 128, kWRows = 128;  // one CTA's boxes
constexpr int kStageBytes = kABytes + kWRows * 128;
constexpr int kOffOut = kStages * kStageBytes;    // staging: 32 rows x 128 bytes per epilogue warp
constexpr int kOutBox = 32 * 128;
constexpr int kChunk = 8;                         // blocks per batch of scales
constexpr int kOffScale = kOffOut + kEpiWarps * kOutBox;
constexpr int kScaleFloats = kChunk * 128 + 2 * kChunk;  // sa [block][row], sw [block][column half]
constexpr int kOffBias = kOffScale + 2 * kScaleFloats * 4;  // the tile's bias, two tiles
constexpr int kOffBar = kOffBias + 2 * kBN * 4;
constexpr int kSmemBytes = kOffBar + 256 + 1024;
static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
static_assert(kThreads == kSplitThreads, "register split");
// A wait on parity P returns at once while the phase before P is still open, so all phases of a
// stage must be waited for by one warp: the two issuers take the even and the odd stages.
static_assert(kStages % 2 == 0, "stages of one issuer");
}  // namespace pair

// Grouped raster: groups of eight row tiles, the row tile varying fastest inside a group, so the
// CTAs running at one time share operand tiles in L2.
__device__ __forceinline__ void tile_at(uint32_t t, uint32_t tiles_m, uint32_t tiles_n, uint32_t& tm, uint32_t& tn) {
    const uint32_t per = 8 * tiles_n, grp = t / per, r = t - grp * per, g0 = grp * 8;
    const uint32_t gsz = tiles_m - g0 < 8 ? tiles_m - g0 : 8;
    tn = r / gsz;
    tm = g0 + (r - tn * gsz);
}

// y[c] = fma(s, v[c], y[c]) for 32 columns, two per instruction (each element one fp32 fma).
__device__ __forceinline__ void fold32(float* y, float s, const uint32_t (&v)[32]) {
    uint64_t ss;
    asm("mov.b64 %0, {%1, %1};" : "=l"(ss) : "f"(s));
#pragma unroll
    for (int c = 0; c < 32; c += 2) {
        uint64_t yy, vv;
        asm("mov.b64 %0, {%1, %2};" : "=l"(yy) : "f"(y[c]), "f"(y[c + 1]));
        asm("mov.b64 %0, {%1, %2};" : "=l"(vv) : "r"(v[c]), "r"(v[c + 1]));
        asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(yy) : "l"(ss), "l"(vv));
        asm("mov.b64 {%0, %1}, %2;" : "=f"(y[c]), "=f"(y[c + 1]) : "l"(yy));
    }
}

// 32 rows (one a lane) x 128 bytes of columns from n0 of the warp's tokens from m0 into a staging
// box and out by a TMA store.  y: the lane's row.
template <bool BF16>
__device__ __forceinline__ void stage_out(const Fp8Params& p, uint8_t* box, int m0, int n0, const float* y, int lane) {
    if (lane == 0) bulk_wait_all<true>();  // the box's last store has read it
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        uint32_t u[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (BF16) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(y[8 * c + 2 * e], y[8 * c + 2 * e + 1]);
                u[e] = *reinterpret_cast<const uint32_t*>(&h);
            } else {
                u[e] = __float_as_uint(y[4 * c + e]);
            }
        }
        // the output map's 128-byte swizzle
        *reinterpret_cast<uint4*>(box + lane * 128 + ((c ^ (lane & 7)) << 4)) = make_uint4(u[0], u[1], u[2], u[3]);
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
        tma_store_2d(&p.ymap, n0, m0, box);
        bulk_commit();
    }
}

// The same 32 x 32 outputs for rows of y that no 16-byte store fits: turned in the staging box, so that a
// warp's stores run along a row.
__device__ __forceinline__ void store_rows(const Fp8Params& p, uint8_t* box, int64_t m0, int64_t n0, const float* y,
                                           int lane) {
    float* b = reinterpret_cast<float*>(box);
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 32; ++c) b[lane * 32 + (c ^ lane)] = y[c];  // the exclusive or keeps the banks apart
    __syncwarp();
    const int64_t n = n0 + lane;
    const int rows = p.M - m0 < 32 ? static_cast<int>(p.M - m0) : 32;
    if (n >= p.N) return;
    for (int r = 0; r < rows; ++r) {
        const float v = b[r * 32 + (lane ^ r)];
        if (p.bf16) static_cast<__nv_bfloat16*>(p.y)[(m0 + r) * p.N + n] = __float2bfloat16_rn(v);
        else static_cast<float*>(p.y)[(m0 + r) * p.N + n] = v;
    }
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(pair::kThreads, 1)
    fp8_pair_kernel(const __grid_constant__ Fp8Params p) {
    using namespace pair;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + kOffBar);
    uint64_t* empty = full + kStages;
    uint64_t* tfull = empty + kStages;  // [accumulator]: 2 (block parity) + half of the columns
    static_assert((kOffBar + 2 * kStages * 8) % 64 == 0, "the two parities' barriers differ in one address bit");
    uint64_t* tempty = tfull + 4;       // the even CTA's, as arrivals go
    uint64_t* sfull = tempty + 4;
    uint64_t* sempty = sfull + 2;
    uint64_t* drain = sempty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 2);
    volatile uint32_t* abort_flag = tmem_slot + 1;
    uint32_t* issued = tmem_slot + 2;  // blocks whose copies were issued; read after an abort
    float* scales = reinterpret_cast<float*>(smem + kOffScale);
    float* biases = reinterpret_cast<float*>(smem + kOffBias);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const WaitCtl ctl{abort_flag, p.status, p.wait_limit_ns};
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&tfull[i], 1);
            mbar_init(&tempty[i], kEpiWarps);  // half of the warps of both CTAs
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sfull[i], 32);  // the copying warp's lanes
            mbar_init(&sempty[i], kEpiWarps);
            mbar_init(&drain[i], 1);
        }
        *abort_flag = 0u;
        fence_barrier_init();
    }
    if (warp == 1) tmem_alloc_pair(tmem_slot, 512);
    tc_fence_before();
    cluster_sync_all();  // both CTAs' barriers are ready before either signals the other
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    griddep_launch_dependents();
    griddep_wait();
    const uint32_t tiles = static_cast<uint32_t>(p.tiles_m) * static_cast<uint32_t>(p.tiles_n);
    const uint32_t first = blockIdx.x >> 1, step = gridDim.x >> 1;
    // blocks of this pair, over all its tiles
    const uint32_t total = tiles > first ? ((tiles - 1 - first) / step + 1) * static_cast<uint32_t>(p.nb) : 0u;

    if (warp < 4) {
        regs_dec<kRegsLow>();
        if (warp == 0 && lane == 0) {
            uint32_t j = 0;
            bool ok = true;
            for (uint32_t t = first; ok && t < tiles; t += step) {
                uint32_t tm, tn;
                tile_at(t, p.tiles_m, p.tiles_n, tm, tn);
                const int m0 = static_cast<int>(tm * kBM + rank * 128), n0 = static_cast<int>(tn * kBN + rank * kWRows);
#pragma unroll 1
                for (int b = 0; b < p.nb; ++b, ++j) {
                    const uint32_t s = j % kStages, k = j / kStages;
                    if (j >= p.copy_blocks || (k > 0 && !mbar_poll(&empty[s], (k - 1) & 1, ctl))) {
                        ok = false;
                        break;
                    }
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * kStageBytes);
                    tma_load_2d_pair(smem + s * kStageBytes, &p.amap, b * 128, m0, &full[s]);
                    tma_load_2d_pair(smem + s * kStageBytes + kABytes, &p.wmap, b * 128, n0, &full[s]);
                }
            }
            *issued = j;
        } else if ((warp == 1 || warp == 2) && rank == 0) {
            // An accumulator's 128 columns: 64 weight rows of each CTA's box.
            constexpr uint32_t idesc = idesc_e4m3_f32(kBM, kBN / 2);
            const uint32_t par = warp - 1;
            const uint64_t da0 = smem_desc(smem_u32(smem), 1024, kLayoutSw128);
            const uint64_t dw0 = smem_desc(smem_u32(smem + kABytes), 1024, kLayoutSw128);
            const uint32_t d = tmem + par * kBN;
            if (elect_one()) {  // one thread runs the whole loop
                uint32_t s = par, phase = 0, free = 1;  // waiting for phase 1 of a fresh barrier returns at once
#pragma unroll 1
                for (uint32_t j = par; j < total; j += 2) {
                    if (!mbar_poll(&full[s], phase, ctl) || !mbar_poll(&tempty[2 * par], free, ctl)) break;
                    tc_fence_after();
                    const uint64_t o = static_cast<uint64_t>((s * kStageBytes) >> 4);
                    constexpr uint64_t half = (kWRows / 2) * 128 >> 4;
#pragma unroll
                    for (int k = 0; k < 4; ++k) mma_f8f6f4_pair(d, da0 + o + 2 * k, dw0 + o + 2 * k, idesc, k > 0);
                    mma_commit_pair(&tfull[2 * par]);
                    if (!mbar_poll(&tempty[2 * par + 1], free, ctl)) break;
                    tc_fence_after();
                    free ^= 1u;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_f8f6f4_pair(d + kBN / 2, da0 + o + 2 * k, dw0 + o + half + 2 * k, idesc, k > 0);
                    mma_commit_pair(&tfull[2 * par + 1]);
                    mma_commit_pair(&empty[s]);
                    if ((s += 2) >= kStages) s -= kStages, phase ^= 1u;
                }
                mma_commit_pair(&drain[par]);
            }
            __syncwarp();
            drain_wait(&drain[par], 0, 100000000ull);
        } else if (warp == 3) {
            uint32_t j = 0, i = 0;  // batches staged, tiles
            bool ok = true;
            for (uint32_t t = first; ok && t < tiles; t += step, ++i) {
                uint32_t tm, tn;
                tile_at(t, p.tiles_m, p.tiles_n, tm, tn);
                const int64_t m0 = static_cast<int64_t>(tm) * kBM + rank * 128;
                // rows past M and columns past N are not stored; they take the last ones' values
                const int64_t w0 = 2 * static_cast<int64_t>(tn), wl = (p.N - 1) / 128;
                for (int b0 = 0; b0 < p.nb; b0 += kChunk, ++j) {
                    const uint32_t buf = j & 1u, u = j >> 1;
                    const int cnt = p.nb - b0 < kChunk ? p.nb - b0 : kChunk;
                    if (u > 0 && !(ok = all_ok(mbar_poll(&sempty[buf], (u - 1) & 1, ctl)))) break;
                    float* d = scales + buf * kScaleFloats;
#pragma unroll 1
                    for (int e = lane; e < 128; e += 32) {
                        const int64_t r = m0 + e;
                        const float* src = p.sa + b0 * p.M + (r < p.M ? r : p.M - 1);
#pragma unroll 1
                        for (int k = 0; k < cnt; ++k, src += p.M) cp_async4(d + k * 128 + e, src);
                    }
                    if (lane < 2 * cnt) {
                        const int64_t wt = w0 + (lane & 1) < wl ? w0 + (lane & 1) : wl;
                        cp_async4(d + kChunk * 128 + lane, p.sw + wt * p.nb + b0 + (lane >> 1));
                    }
                    if (b0 == 0 && p.bias) {  // with a tile's first batch: its bias
                        for (int c = lane; c < kBN; c += 32) {
                            const int64_t n = static_cast<int64_t>(tn) * kBN + c;
                            cp_async4(biases + (i & 1u) * kBN + c, p.bias + (n < p.N ? n : p.N - 1));
                        }
                    }
                    cp_async_arrive(&sfull[buf]);
                }
            }
            cp_async_wait_all();
        }
        __syncwarp();
    } else {
        regs_inc<kRegsHigh>();
        // TMEM lane quarter, column half (its accumulators), and which 64 columns of that
        const int q = warp & 3, h = ((warp - 4) >> 2) & 1, r = (warp - 4) >> 3;
        const uint32_t tl = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(h * (kBN / 2) + r * 64);
        // their first column in the tile (the run r of an accumulator comes from CTA r's weight rows)
        const int col = r * 128 + h * 64;
        uint32_t release = map_rank(&tempty[h], 0);
        uint32_t js = 0, it = 0;  // batches of scales used, tiles mod 2
        // of the next block: its accumulator's barrier, that barrier's phase, the accumulator, and the
        // barrier that its release counts towards.  The loop's own instructions matter: with the index
        // arithmetic, the batch's bounds and the end of the pair's blocks tested for every block, a warp
        // spent 148 instructions on a block's 32 fmas (then 110; 8192 x 4096 -> 14336 379 -> 344 us).
        uint32_t bar = smem_u32(&tfull[h]), phase = 0, ta = tl;
        constexpr uint32_t kBarStep = 16, kTmemStep = kBN;
        // after a wait gave up the warp ends with its tile, whose sums are undefined (the status word says so)
        for (uint32_t t = first; t < tiles && all_ok(!*abort_flag); t += step) {
            // the sums start from the bias, which arrives with the tile's first scales
            float y[64];
            (void)mbar_poll(&sfull[js & 1u], (js >> 1) & 1, ctl);
            if (p.bias) {
                const float* bs = biases + it * kBN + col;
#pragma unroll
                for (int c = 0; c < 64; c += 4) {
                    const float4 v = *reinterpret_cast<const float4*>(bs + c);
                    y[c] = v.x, y[c + 1] = v.y, y[c + 2] = v.z, y[c + 3] = v.w;
                }
            } else {
#pragma unroll
                for (int c = 0; c < 64; ++c) y[c] = 0.0f;
            }
            it ^= 1;
#pragma unroll 1
            for (int b0 = 0; b0 < p.nb; b0 += kChunk) {
                if (b0 > 0) (void)mbar_poll(&sfull[js & 1u], (js >> 1) & 1, ctl);
                const float* sa = scales + (js & 1u) * kScaleFloats + q * 32 + lane;
                const float* sw = scales + (js & 1u) * kScaleFloats + kChunk * 128 + r;
                const float* end = sw + 2 * (p.nb - b0 < kChunk ? p.nb - b0 : kChunk);
#pragma unroll 1
                for (; sw != end; sa += 128, sw += 2) {
                    const float f = *sa * *sw;
                    // the TMEM loads take the whole warp: it votes on its first try, so that the branch is one for all
                    // lanes (a branch lane by lane and a __syncwarp after it cost five instructions a block, 341 us)
                    if (__builtin_expect(!all_ok(mbar_try_wait_long(bar, phase)), 0)) {
                        (void)mbar_wait_on(bar, phase, ctl);
                        __syncwarp();
                    }
                    tc_fence_after();
                    uint32_t v[32];
                    tmem_ld_32x32b_x32(ta, v);
                    tmem_wait_ld32(v);
                    fold32(y, f, v);
                    tmem_ld_32x32b_x32(ta + 32, v);
                    tmem_wait_ld32(v);
                    // this warp's columns are read: its part of the accumulator is free for the block two later
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(release);
                    fold32(y + 32, f, v);
                    phase ^= ta != tl;
                    bar ^= kBarStep;
                    ta ^= kTmemStep;
                    release ^= kBarStep;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sempty[js & 1u]);
                ++js;
            }
            uint32_t tm, tn;
            tile_at(t, p.tiles_m, p.tiles_n, tm, tn);
            const int64_t mw = static_cast<int64_t>(tm) * kBM + rank * 128 + q * 32;
            const int64_t n0 = static_cast<int64_t>(tn) * kBN + col;
            if (mw >= p.M || n0 >= p.N) continue;
            uint8_t* box = smem + kOffOut + (warp - 4) * kOutBox;
            if (!p.vec) {
                store_rows(p, box, mw, n0, y, lane);
                store_rows(p, box, mw, n0 + 32, y + 32, lane);
            } else if (p.bf16) {
                stage_out<true>(p, box, static_cast<int>(mw), static_cast<int>(n0), y, lane);
            } else {
                stage_out<false>(p, box, static_cast<int>(mw), static_cast<int>(n0), y, lane);
                if (n0 + 32 < p.N) stage_out<false>(p, box, static_cast<int>(mw), static_cast<int>(n0) + 32, y + 32, lane);
            }
        }
        if (lane == 0) bulk_wait_all<false>();
        __syncwarp();
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && *abort_flag) {
        // both CTAs' copies land on the even CTA's barriers; the odd one has only the time to go by
        if (rank == 0) land_copies<kStages>(full, *issued);
        else drain_wait(&full[0], 0, 10000000ull);
    }
    // the issuers' last commits arrive on this CTA's barriers too: it may not leave before they have
    if (rank == 1 && threadIdx.x < 2) drain_wait(&drain[threadIdx.x], 0, 100000000ull);
    cluster_sync_all();  // neither CTA leaves while the other may still signal it or read its memory
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
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

// A map over y [M][N], boxes of 32 rows x 128 bytes, 128-byte swizzled as stage_out writes them.
bool make_out_map(CUtensorMap* map, void* y, int64_t M, int64_t N, bool bf16) {
    const EncodeTiledFn enc = encode_tiled();
    if (!enc) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(M)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(N) * (bf16 ? 2 : 4)};
    const cuuint32_t box[2] = {bf16 ? 64u : 32u, 32};
    const cuuint32_t estr[2] = {1, 1};
    return enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, y, dims, strides,
               box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
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

// How many clusters of `split` CTAs of the one-CTA kernel run at once on device `dev`, the current one (one
// CTA to an SM, clusters within a GPC, so not num_sms / split: of eight CTAs fewer than 16).  Asked once a
// device; minus a cudaError_t where the driver could not say.
constexpr int kMaxSplit = 8;
template <int TN>
int tok_clusters(int dev, int split) {
    using T = Tok<TN>;
    static DeviceMemo<64, kMaxSplit + 1> memo;
    return memo.get(dev, split, [split] {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(split));
        cfg.blockDim = dim3(T::kThreads);
        cfg.dynamicSmemBytes = T::kSmemBytes;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = static_cast<unsigned>(split);
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        cudaError_t e = cudaFuncSetAttribute(fp8_tok_kernel<TN>, cudaFuncAttributeMaxDynamicSharedMemorySize, T::kSmemBytes);
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&n, fp8_tok_kernel<TN>, &cfg);
        if (e != cudaSuccess) (void)cudaGetLastError();
        return e == cudaSuccess ? n : -static_cast<int>(e);
    });
}

template <int TN>
cudaError_t run_tok(Fp8Params& p, const Fp8Args& a, int num_sms, cudaStream_t s) {
    using T = Tok<TN>;
    static bool attr_done[64] = {};
    p.tiles_m = static_cast<int>((a.M + TN - 1) / TN);
    p.tiles_n = static_cast<int>((a.N + 127) / 128);
    if (!make_map(&p.amap, a.a, a.M, a.K, TN) || !make_map(&p.wmap, a.w, a.N, a.K, 128)) return cudaErrorInvalidValue;
    const int64_t tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n;
    const int64_t grid = p.split > 1 ? tiles * p.split : (tiles < num_sms ? tiles : num_sms);
    return launch(fp8_tok_kernel<TN>, T::kSmemBytes, attr_done, grid, T::kThreads, p.split, p, s);
}

cudaError_t run_pair(Fp8Params& p, const Fp8Args& a, int num_sms, cudaStream_t s) {
    static bool attr_done[64] = {};
    p.tiles_m = static_cast<int>((a.M + pair::kBM - 1) / pair::kBM);
    p.tiles_n = static_cast<int>((a.N + pair::kBN - 1) / pair::kBN);
    if (!make_map(&p.amap, a.a, a.M, a.K, 128) || !make_map(&p.wmap, a.w, a.N, a.K, pair::kWRows) ||
        (p.vec && !make_out_map(&p.ymap, a.y, a.M, a.N, a.bf16)))
        return cudaErrorInvalidValue;
    const int64_t tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n, most = num_sms / 2;
    return launch(fp8_pair_kernel, pair::kSmemBytes, attr_done, 2 * (tiles < most ? tiles : most), pair::kThreads, 1, p, s);
}

// Estimated time in us of a form: start, then waves of tiles, each of `blocks` K-blocks and an end.
// Fitted to measurements (bf16 out, back-to-back launches, us), in the order pairs, 16-, 32-, 64- and
// 128-token tiles: 512 x 2048 -> 2048 11.0, 12.8, 8.5, 7.0, 10.2; 512 x 8192 -> 2048 31.2, 40.4, 22.8,
// 16.8, 26.2; 256 x 2048 -> 2048 10.9, 7.7, 5.3, 6.8, 10.0; 512 x 2048 -> 6144 12.3, 31.3, 21.0, 16.0,
// 17.5; 4096 x 1024 -> 2048 13.7, 45.2, 30.2, 21.5, 20.5; 8 x 4096 -> 14336 22.3, 12.3, 12.7, 17.4, 25.2.
// Outputs of another type or width, pairs against 128-token tiles: rows of y that no 16-byte store fits cost
// pairs 3.4 us a tile (512 x 2048 -> 6143 15.9 and 18.1, 4096 x 1024 -> 2047 20.9 and 21.5, but 2048 x 512 ->
// 14335 46.3 and 43.2, against 22.8 and 40.9 at 14336), which counts for any N that is no multiple of 8, so
// that the order of the sums does not depend on y's type; fp32 rows cost them 1.2 (512 x 2048 -> 6144 13.8 and
// 18.2, 2048 x 512 -> 14336 29.7 and 42.3), which changed no choice and is not counted.
double form_us(double start, double block, double end, int64_t tiles, int64_t slots, int64_t blocks) {
    const int64_t waves = (tiles + slots - 1) / slots;
    return start + static_cast<double>(waves) * (block * static_cast<double>(blocks) + end);
}

// The form a problem takes: 0 (pairs) or the token tile, and the CTAs that share a tile's K.
struct Form {
    int tn, split;
};
int clusters(int dev, int tn, int split) {
    return tn == 16   ? tok_clusters<16>(dev, split)
           : tn == 32 ? tok_clusters<32>(dev, split)
           : tn == 64 ? tok_clusters<64>(dev, split)
                      : tok_clusters<128>(dev, split);
}

// `fit(tn, split)`: how many of a split's clusters run at once.  Where that fails (a negative answer) no form
// is picked but that answer returned as `split`, with tn -1: a form picked without it would sum in another
// order than the same call's next.
template <typename Fit>
Form pick_form(int64_t M, int64_t N, int64_t nb, int num_sms, Fit&& fit) {
    const int64_t n128 = (N + 127) / 128;
    Form best{0, 1};
    double us = form_us(1.5, 0.418, N % 8 == 0 ? 2.7 : 6.1, ((M + 255) / 256) * ((N + 255) / 256), num_sms / 2, nb);
    const int tns[4] = {16, 32, 64, 128};
    const double start[4] = {2.35, 1.9, 2.1, 2.4}, block[4] = {0.153, 0.16, 0.205, 0.335}, end[4] = {0.2, 0.75, 1.33, 2.2};
    for (int i = 0; i < 4; ++i) {
        const int tn = tns[i];
        const int64_t tiles = ((M + tn - 1) / tn) * n128;
        for (int split = 1, log = 0; split <= kMaxSplit && split <= nb; split *= 2, ++log) {
            // a split has one tile to a cluster, all of them running at once (with eight CTAs a tile and 16
            // tiles, two waves of clusters, 16 x 6144 -> 2048 took 11.4 us against 6.3 with four)
            if (split > 1 && tiles * split > num_sms) break;
            const int most = split > 1 ? fit(tn, split) : 1;
            if (most < 0) return Form{-1, most};
            if (split > 1 && tiles > most) break;
            // handing the parts over: 1 x 6144 -> 1024 took 8.9, 6.7, 5.4 and 4.9 us on one, two, four and
            // eight CTAs a tile, 1 x 1024 -> 1024 3.6, 3.8, 3.7 and 4.1; with 64-token tiles 128 x 6144 ->
            // 1024 9.7 on two and 8.0 on four
            const double t = form_us(start[i] + (split > 1 ? 0.4 + 0.32 * log + 0.012 * tn : 0.0), block[i], end[i], tiles,
                                     num_sms, (nb + split - 1) / split);
            if (t < us) us = t, best = Form{tn, split};
        }
    }
    return best;
}

cudaError_t launch_form(const Fp8Args& a, Form f, int num_sms, cudaStream_t s) {
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
    p.split = f.split;
    p.status = a.status;
    p.wait_limit_ns = a.wait_limit_ns;
    p.copy_blocks = a.copy_blocks;
    switch (f.tn) {
        case 0: return run_pair(p, a, num_sms, s);
        case 16: return run_tok<16>(p, a, num_sms, s);
        case 32: return run_tok<32>(p, a, num_sms, s);
        case 64: return run_tok<64>(p, a, num_sms, s);
        default: return run_tok<128>(p, a, num_sms, s);
    }
}

}  // namespace

cudaError_t launch_fp8_linear(const Fp8Args& a, int num_sms, cudaStream_t s) {
    if (num_sms < 1) return cudaErrorInvalidValue;
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const Form f = pick_form(a.M, a.N, (a.K + kGroup8 - 1) / kGroup8, num_sms,
                             [dev](int tn, int split) { return clusters(dev, tn, split); });
    if (f.tn < 0) return static_cast<cudaError_t>(-f.split);
    return launch_form(a, f, num_sms, s);
}

}  // namespace w4a8

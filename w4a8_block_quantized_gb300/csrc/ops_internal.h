// ops_internal.h -- declarations of the operators around the linears (row_quant.cu,
// fp8_gemm.cu) and of what their C entry points (ops_api.cu) share with api.cu.
#pragma once

#include "w4a8_internal.h"

namespace w4a8 {

// The current device, checked once to be an sm_103 part: its SM count and the address of its
// status word.  A w4a8_status (defined in api.cu).
int device_info(int* num_sms, uint32_t** status);

constexpr int kGroup8 = 128;  // columns per e4m3 scale

// ---------------------------------------------------------------- row quantizers
// What a row's values t are computed from.
enum RowSource : int {
    kSrcPlain = 0,   // t = x
    kSrcNorm = 1,    // t = (x + residual) * gamma, common factor r = 1 / sqrt(mean((x + residual)^2) + eps)
    kSrcSwiglu = 2,  // t = x / (1 + exp(-x)) * up
};
// How they are stored.
enum RowForm : int {
    kFormInt8 = 0,     // a_q int8 [M][K], a_scale [M], rowsum [M][K/64]
    kFormRecords = 1,  // token records and s_a (w4a8_internal.h)
    kFormE4m3 = 2,     // a_q e4m3 [M][K], a_scale [ceil(K/128)][M]
};

struct RowArgs {
    const void* x = nullptr;    // [M] rows of K, ld elements apart (the gate for kSrcSwiglu)
    const void* up = nullptr;   // kSrcSwiglu: [M] rows of K, ld elements apart
    int64_t ld = 0;
    const float* gamma = nullptr;
    const void* residual = nullptr;   // [M][K] or null
    void* residual_out = nullptr;     // [M][K] or null; may be `residual`
    float eps = 0.0f;
    int64_t M = 0, K = 0;
    uint8_t* a_q = nullptr;
    float* a_scale = nullptr;
    int32_t* rowsum = nullptr;
    uint8_t* trec = nullptr;
    int tw = 128;
    uint32_t* status = nullptr;
};

// bf16: the type of x, up, residual and residual_out (fp32 otherwise).
cudaError_t launch_row_quant(RowSource src, RowForm form, bool bf16, const RowArgs& a, int num_sms, cudaStream_t s);

// ---------------------------------------------------------------- e4m3 linear
struct Fp8Args {
    const uint8_t* a = nullptr;     // e4m3 [M][K]
    const float* sa = nullptr;      // [ceil(K/128)][M]
    const uint8_t* w = nullptr;     // e4m3 [N][K]
    const float* sw = nullptr;      // [ceil(N/128)][ceil(K/128)]
    const float* bias = nullptr;    // [N] or null
    void* y = nullptr;              // [M][N]
    int bf16 = 0;
    int64_t M = 0, N = 0, K = 0;
    uint32_t* status = nullptr;
    uint64_t wait_limit_ns = 1000000000ull;
    uint32_t copy_blocks = 0xffffffffu;  // fewer than a CTA has: its waits run out (tests of the bounded waits)
};

cudaError_t launch_fp8_linear(const Fp8Args& a, int num_sms, cudaStream_t s);

}  // namespace w4a8

// ops_api.cu -- C entry points of the operators around the linears (include/w4a8.h): argument
// checks and launches.  Nothing here allocates memory.
#include "../../include/w4a8.h"
#include "ops_internal.h"

#include <cmath>

namespace w4a8 {
namespace {

constexpr int64_t kMaxDim = 2147483647LL;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Sizes of a row quantizer: `unit` divides K.
int check_rows(int64_t M, int64_t K, int64_t unit, int in_dtype) {
    if (M < 0 || (in_dtype != W4A8_IN_F32 && in_dtype != W4A8_IN_BF16)) return W4A8_ERR_ARG;
    if (K <= 0 || K % unit != 0 || M > kMaxDim || K > kMaxDim) return W4A8_ERR_SHAPE;
    return W4A8_OK;
}

int check_norm(const RowArgs& a) {
    if (!a.x || !a.gamma || !(a.eps > 0.0f) || !std::isfinite(a.eps) || (a.residual_out && !a.residual))
        return W4A8_ERR_ARG;
    if (!aligned(a.x, 16) || !aligned(a.gamma, 16) || !aligned(a.residual, 16) || !aligned(a.residual_out, 16))
        return W4A8_ERR_ALIGN;
    return W4A8_OK;
}

int check_swiglu(const RowArgs& a, int in_dtype) {
    if (!a.x || !a.up) return W4A8_ERR_ARG;
    if (a.ld < a.K || a.ld > kMaxDim) return W4A8_ERR_SHAPE;
    if (!aligned(a.x, 16) || !aligned(a.up, 16) || a.ld % (in_dtype == W4A8_IN_BF16 ? 8 : 4) != 0)
        return W4A8_ERR_ALIGN;
    return W4A8_OK;
}

int check_codes(const void* a_q, const float* a_scale) {
    if (!a_q || !a_scale) return W4A8_ERR_ARG;
    return aligned(a_q, 16) && aligned(a_scale, 4) ? W4A8_OK : W4A8_ERR_ALIGN;
}

// The opaque buffer `act` as the outputs of the operand form.
int set_act(RowArgs* a, void* act, size_t act_bytes) {
    if (!act) return W4A8_ERR_ARG;
    if (!aligned(act, 16)) return W4A8_ERR_ALIGN;
    const ActLayout L = act_layout(a->M, a->K, true, token_tile(a->M));
    if (act_bytes < L.total) return W4A8_ERR_WORKSPACE;
    a->trec = static_cast<uint8_t*>(act) + L.rec;
    a->a_scale = reinterpret_cast<float*>(static_cast<uint8_t*>(act) + L.s_a);
    a->tw = L.tw;
    return W4A8_OK;
}

int run_rows(RowSource src, RowForm form, int in_dtype, RowArgs a, void* stream) {
    int num_sms = 0;
    const int rc = device_info(&num_sms, &a.status);
    if (rc != W4A8_OK) return rc;
    return launch_row_quant(src, form, in_dtype == W4A8_IN_BF16, a, num_sms, static_cast<cudaStream_t>(stream)) ==
                   cudaSuccess
               ? W4A8_OK
               : W4A8_ERR_CUDA;
}

RowArgs norm_args(const void* x, const void* residual, const float* gamma, float eps, void* residual_out, int64_t M,
                  int64_t K) {
    RowArgs a;
    a.x = x;
    a.ld = K;
    a.residual = residual;
    a.gamma = gamma;
    a.eps = eps;
    a.residual_out = residual_out;
    a.M = M;
    a.K = K;
    return a;
}

RowArgs swiglu_args(const void* gate, const void* up, int64_t ld, int64_t M, int64_t K) {
    RowArgs a;
    a.x = gate;
    a.up = up;
    a.ld = ld;
    a.M = M;
    a.K = K;
    return a;
}

}  // namespace
}  // namespace w4a8

using namespace w4a8;

extern "C" {

int w4a8_rmsnorm_quant(const void* x, const void* residual, const float* gamma, float eps, int in_dtype,
                       void* residual_out, int8_t* a_q, float* a_scale, int32_t* rowsum, int64_t M, int64_t K,
                       void* stream) {
    int rc = check_rows(M, K, kBlock, in_dtype);
    if (rc != W4A8_OK || M == 0) return rc;
    RowArgs a = norm_args(x, residual, gamma, eps, residual_out, M, K);
    if ((rc = check_norm(a)) != W4A8_OK || (rc = check_codes(a_q, a_scale)) != W4A8_OK) return rc;
    if (!rowsum) return W4A8_ERR_ARG;
    if (!aligned(rowsum, 4)) return W4A8_ERR_ALIGN;
    a.a_q = reinterpret_cast<uint8_t*>(a_q);
    a.a_scale = a_scale;
    a.rowsum = rowsum;
    return run_rows(kSrcNorm, kFormInt8, in_dtype, a, stream);
}

int w4a8_rmsnorm_prepare(const void* x, const void* residual, const float* gamma, float eps, int in_dtype,
                         void* residual_out, void* act, size_t act_bytes, int64_t M, int64_t K, void* stream) {
    int rc = check_rows(M, K, kBlock, in_dtype);
    if (rc != W4A8_OK || M == 0) return rc;
    RowArgs a = norm_args(x, residual, gamma, eps, residual_out, M, K);
    if ((rc = check_norm(a)) != W4A8_OK || (rc = set_act(&a, act, act_bytes)) != W4A8_OK) return rc;
    return run_rows(kSrcNorm, kFormRecords, in_dtype, a, stream);
}

int w4a8_rmsnorm_quant_fp8(const void* x, const void* residual, const float* gamma, float eps, int in_dtype,
                           void* residual_out, uint8_t* a_q, float* a_scale, int64_t M, int64_t K, void* stream) {
    int rc = check_rows(M, K, 16, in_dtype);
    if (rc != W4A8_OK || M == 0) return rc;
    RowArgs a = norm_args(x, residual, gamma, eps, residual_out, M, K);
    if ((rc = check_norm(a)) != W4A8_OK || (rc = check_codes(a_q, a_scale)) != W4A8_OK) return rc;
    a.a_q = a_q;
    a.a_scale = a_scale;
    return run_rows(kSrcNorm, kFormE4m3, in_dtype, a, stream);
}

int w4a8_swiglu_quant(const void* gate, const void* up, int64_t ld, int in_dtype, int8_t* a_q, float* a_scale,
                      int32_t* rowsum, int64_t M, int64_t K, void* stream) {
    int rc = check_rows(M, K, kBlock, in_dtype);
    if (rc != W4A8_OK || M == 0) return rc;
    RowArgs a = swiglu_args(gate, up, ld, M, K);
    if ((rc = check_swiglu(a, in_dtype)) != W4A8_OK || (rc = check_codes(a_q, a_scale)) != W4A8_OK) return rc;
    if (!rowsum) return W4A8_ERR_ARG;
    if (!aligned(rowsum, 4)) return W4A8_ERR_ALIGN;
    a.a_q = reinterpret_cast<uint8_t*>(a_q);
    a.a_scale = a_scale;
    a.rowsum = rowsum;
    return run_rows(kSrcSwiglu, kFormInt8, in_dtype, a, stream);
}

int w4a8_swiglu_prepare(const void* gate, const void* up, int64_t ld, int in_dtype, void* act, size_t act_bytes,
                        int64_t M, int64_t K, void* stream) {
    int rc = check_rows(M, K, kBlock, in_dtype);
    if (rc != W4A8_OK || M == 0) return rc;
    RowArgs a = swiglu_args(gate, up, ld, M, K);
    if ((rc = check_swiglu(a, in_dtype)) != W4A8_OK || (rc = set_act(&a, act, act_bytes)) != W4A8_OK) return rc;
    return run_rows(kSrcSwiglu, kFormRecords, in_dtype, a, stream);
}

int w4a8_swiglu_quant_fp8(const void* gate, const void* up, int64_t ld, int in_dtype, uint8_t* a_q, float* a_scale,
                          int64_t M, int64_t K, void* stream) {
    int rc = check_rows(M, K, 16, in_dtype);
    if (rc != W4A8_OK || M == 0) return rc;
    RowArgs a = swiglu_args(gate, up, ld, M, K);
    if ((rc = check_swiglu(a, in_dtype)) != W4A8_OK || (rc = check_codes(a_q, a_scale)) != W4A8_OK) return rc;
    a.a_q = a_q;
    a.a_scale = a_scale;
    return run_rows(kSrcSwiglu, kFormE4m3, in_dtype, a, stream);
}

int w4a8_quant_fp8(const void* x, int in_dtype, uint8_t* a_q, float* a_scale, int64_t M, int64_t K, void* stream) {
    int rc = check_rows(M, K, 16, in_dtype);
    if (rc != W4A8_OK || M == 0) return rc;
    if (!x) return W4A8_ERR_ARG;
    if (!aligned(x, 16)) return W4A8_ERR_ALIGN;
    if ((rc = check_codes(a_q, a_scale)) != W4A8_OK) return rc;
    RowArgs a;
    a.x = x;
    a.ld = K;
    a.M = M;
    a.K = K;
    a.a_q = a_q;
    a.a_scale = a_scale;
    return run_rows(kSrcPlain, kFormE4m3, in_dtype, a, stream);
}

int w4a8_fp8_linear(const uint8_t* a_q, const float* a_scale, const uint8_t* w_q, const float* w_scale,
                    const float* bias, void* y, int out_dtype, int64_t M, int64_t N, int64_t K, void* stream) {
    if (M < 0 || N < 0 || (out_dtype != W4A8_OUT_F32 && out_dtype != W4A8_OUT_BF16)) return W4A8_ERR_ARG;
    if (K <= 0 || K % 16 != 0 || M > kMaxDim || N > kMaxDim || K > kMaxDim) return W4A8_ERR_SHAPE;
    // the kernels count tiles and a CTA's blocks (tiles x K/128) in 32 unsigned bits; the smallest tile, 128 x 16,
    // has at most twice the number counted here
    const int64_t tiles = ((M + 31) / 32) * ((N + kGroup8 - 1) / kGroup8);
    if (tiles > kMaxDim / ((K + kGroup8 - 1) / kGroup8)) return W4A8_ERR_SHAPE;
    if (M == 0 || N == 0) return W4A8_OK;
    if (!a_q || !a_scale || !w_q || !w_scale || !y) return W4A8_ERR_ARG;
    if (!aligned(a_q, 16) || !aligned(w_q, 16) || !aligned(y, 16) || !aligned(a_scale, 4) || !aligned(w_scale, 4) ||
        !aligned(bias, 4))
        return W4A8_ERR_ALIGN;
    Fp8Args a;
    a.a = a_q;
    a.sa = a_scale;
    a.w = w_q;
    a.sw = w_scale;
    a.bias = bias;
    a.y = y;
    a.bf16 = out_dtype == W4A8_OUT_BF16;
    a.M = M;
    a.N = N;
    a.K = K;
    int num_sms = 0;
    const int rc = device_info(&num_sms, &a.status);
    if (rc != W4A8_OK) return rc;
    return launch_fp8_linear(a, num_sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? W4A8_OK : W4A8_ERR_CUDA;
}

}  // extern "C"

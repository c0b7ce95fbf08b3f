// fp8_forms.cu -- the e4m3 linear's forms called by name, for the tests: which kernel, how many CTAs
// share a tile's K, and how long its waits last.  Compiled together with the product's source, so that
// the kernels are the product's own.
#include "../w4a8_block_quantized_gb300/csrc/fp8_gemm.cu"

using namespace w4a8;

extern "C" {

// Clusters of `split` CTAs of the tile `tn` (16, 32, 64, 128) that the current device runs at once.
int forms_clusters(int tn, int split) {
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess ? clusters(dev, tn, split) : -1;
}

// The form that a problem takes on a GPU of num_sms SMs where fit[4 i + j] clusters of 2^j CTAs of the i-th token
// tile (16, 32, 64, 128) run at once (negative: the driver could not say): tile and split.
void forms_pick(int64_t M, int64_t N, int64_t K, int num_sms, const int* fit, int* tn, int* split) {
    const Form f = pick_form(M, N, (K + kGroup8 - 1) / kGroup8, num_sms, [fit](int t, int s) {
        return fit[4 * (t == 16 ? 0 : t == 32 ? 1 : t == 64 ? 2 : 3) + (s == 1 ? 0 : s == 2 ? 1 : s == 4 ? 2 : 3)];
    });
    *tn = f.tn;
    *split = f.split;
}

// One launch of a form: tn 0 (pairs of CTAs) or the token tile, on at most num_sms SMs.  copy_blocks: a
// CTA's copies stop before this block of its own (-1: none).
int forms_run(int tn, int split, const uint8_t* a_q, const float* a_scale, const uint8_t* w_q, const float* w_scale,
              const float* bias, void* y, int bf16, int64_t M, int64_t N, int64_t K, uint32_t* status,
              int64_t limit_us, int64_t copy_blocks, int num_sms, void* stream) {
    Fp8Args a;
    a.a = a_q;
    a.sa = a_scale;
    a.w = w_q;
    a.sw = w_scale;
    a.bias = bias;
    a.y = y;
    a.bf16 = bf16;
    a.M = M;
    a.N = N;
    a.K = K;
    a.status = status;
    a.wait_limit_ns = static_cast<uint64_t>(limit_us) * 1000u;
    if (copy_blocks >= 0) a.copy_blocks = static_cast<uint32_t>(copy_blocks);
    return launch_form(a, Form{tn, split}, num_sms, static_cast<cudaStream_t>(stream));
}

}  // extern "C"

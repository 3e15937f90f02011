// fp8.h -- host-side interfaces of the 8-bit block-scaled operators (the
// quantizer, the product and the few-token mixture-of-experts layer), shared
// by their translation units and api.cu (not installed, not part of the C ABI).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

#include "internal.h"

namespace gemm11 {

constexpr int kScaleBlock = 128;  // elements that share one scale along the contraction
// 8-bit types, the codes of the C ABI's gemm_dtype.
constexpr int kTypeE4M3 = 3;
constexpr int kTypeE5M2 = 4;

// Tensor map of a row-major matrix of `outer` rows of `inner` elements, rows
// row_bytes apart; false when the encoder is missing or refuses.
bool encode_matrix_map(CUtensorMap *map, CUtensorMapDataType dt, const void *base, uint64_t inner, uint64_t outer,
                       uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer, CUtensorMapSwizzle swizzle);
// The same with a third dimension (rows row_bytes, its steps step_bytes apart)
// and the 128-byte swizzle.
bool encode_box_map(CUtensorMap *map, CUtensorMapDataType dt, const void *base, uint64_t inner, uint64_t rows, uint64_t steps,
                    uint64_t row_bytes, uint64_t step_bytes, uint32_t box_inner, uint32_t box_rows, uint32_t box_steps);

// ---- quantizer (fp8_quant.cu) ----
struct Fp8Quant {
    int rows = 0, cols = 0;
    const void *X = nullptr;
    int x_type = 0;
    long long ldx = 0;
    void *Q = nullptr;
    int q_type = kTypeE4M3;
    long long ldq = 0;
    float *S = nullptr;
    long long lds = 0;
    int layout = 0;  // the codes of gemm_fp8_layout
};
cudaError_t run_fp8_quantize(const Fp8Quant &q, cudaStream_t stream, CallInfo *info);

// ---- product (fp8_gemm.cu) ----
// C = act(alpha * sum over k blocks of sa sb (A_kb op(B)_kb) + beta * C + bias).
// A: M x K, its scales SA[kb * ldsa + m].  B: N x K (b_trans) or K x N; its
// scales one for each 128 x 128 block of B as stored, SB[row / 128 * ldsb +
// col / 128], or (b_rows, N x K only) SB[kb * ldsb + n].
struct Fp8Gemm {
    int M = 0, N = 0, K = 0;
    float alpha = 1.f, beta = 0.f;
    const void *A = nullptr;
    int a_type = kTypeE4M3;
    long long lda = 0;
    const float *SA = nullptr;
    long long ldsa = 0;
    const void *B = nullptr;
    int b_type = kTypeE4M3;
    long long ldb = 0;
    const float *SB = nullptr;
    long long ldsb = 0;
    int b_trans = 1;
    int b_rows = 0;
    void *C = nullptr;
    int c_type = 0;
    long long ldc = 0;
    const float *bias = nullptr;
    int act = 0;
};
// K > 0 and alpha != 0.
cudaError_t run_fp8_gemm(const Fp8Gemm &g, cudaStream_t stream, CallInfo *info);
// The same with no product (K == 0 or alpha == 0): C = act(beta * C + bias).
cudaError_t run_fp8_scale_c(const Fp8Gemm &g, cudaStream_t stream, CallInfo *info);

// ---- mixture of experts for a few tokens (moe.cu) ----
constexpr int kMoeMaxTokens = 128, kMoeMaxExperts = 512, kMoeMaxTopK = 16, kMoeMaxSlots = 1024, kMoeMaxWidth = 32768;
constexpr int kActSilu = 4;  // the C ABI's GEMM_ACT_SILU
struct Moe {
    int T = 0, E = 0, top_k = 0, H = 0, I = 0;
    const void *X = nullptr;  // T x H
    int x_type = 0;
    long long ldx = 0;
    const void *router = nullptr;  // E x H
    int router_type = 0;
    const void *gate = nullptr, *up = nullptr, *down = nullptr;  // E x I x H, E x I x H (or NULL), E x H x I
    int w_type = 0;
    const float *s_gate = nullptr, *s_up = nullptr, *s_down = nullptr;  // 128 x 128 scales of 8-bit weights
    void *Y = nullptr;  // T x H
    int y_type = 0;
    long long ldy = 0;
    int act = 0, renorm = 0;
    int *ids = nullptr;  // T x top_k, or NULL
    float *weights = nullptr;
};
cudaError_t run_moe(const Moe &m, cudaStream_t stream, CallInfo *info);

}  // namespace gemm11

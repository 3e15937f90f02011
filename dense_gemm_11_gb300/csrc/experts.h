// experts.h -- host-side interfaces of the mixture-of-experts operators for
// many tokens (sorted rows and back, the experts' products, the gated
// activation with 8-bit copies), shared by their translation units and api.cu
// (not installed, not part of the C ABI).
#pragma once

#include <cuda_runtime.h>

#include "internal.h"

namespace gemm11 {

constexpr int kDispatchMaxExperts = 4096;

// ---- rows of the tokens in the order of the experts, and back (moe_rows.cu) ----
struct MoeDispatch {
    int T = 0, E = 0, top_k = 0, H = 0;  // H = 0: the order alone
    const int *ids = nullptr;            // T x top_k
    const void *X = nullptr;             // T x H
    int x_type = 0;
    long long ldx = 0;
    void *Xs = nullptr;  // at least T * top_k rows
    long long ldxs = 0;
    int *offsets = nullptr;  // E + 1
    int *rows = nullptr;     // T x top_k
};
cudaError_t run_moe_dispatch(const MoeDispatch &d, cudaStream_t stream, CallInfo *info);

struct MoeCombine {
    int T = 0, top_k = 0, H = 0, R = 0;
    const void *Ys = nullptr;  // R x H
    int type = 0;              // of Ys, Y, dY and dYs
    long long ldys = 0;
    const int *rows = nullptr;       // T x top_k
    const float *weights = nullptr;  // T x top_k, or NULL: ones (the sum only)
    void *Y = nullptr;               // T x H: the sum; or, for the gradient, dY
    long long ldy = 0;
    void *dYs = nullptr;  // R x H (gradient)
    long long lddys = 0;
    float *dweights = nullptr;  // T x top_k (gradient)
};
cudaError_t run_moe_combine(const MoeCombine &c, cudaStream_t stream, CallInfo *info);
cudaError_t run_moe_combine_grad(const MoeCombine &c, cudaStream_t stream, CallInfo *info);

// ---- products over the sorted rows (grouped.cu) ----
// wgrad = 0: C[r] = alpha A[r] op(B[e]) + beta C[r] for the rows r of expert e,
//            A R x K, B E x N x K (b_trans) or E x K x N, C R x N;
// wgrad = 1: C[e] = alpha A[rows of e]^T B[rows of e] + beta C[e],
//            A R x M, B R x N, C E x M x N.
struct Grouped {
    int wgrad = 0, E = 0, R = 0, M = 0, N = 0, K = 0;
    float alpha = 1.f, beta = 0.f;
    const void *A = nullptr;
    long long lda = 0;
    const void *B = nullptr;
    long long ldb = 0, stride_b = 0;
    int b_trans = 1;
    bool bf16 = false;
    void *C = nullptr;
    int c_type = 0;
    long long ldc = 0, stride_c = 0;
    const int *offsets = nullptr;  // E + 1
};
cudaError_t run_grouped(const Grouped &g, cudaStream_t stream, CallInfo *info);

// ---- gated activation with 8-bit copies of its inputs (gated_act.cu) ----
struct GatedAct {
    int rows = 0, cols = 0;
    const void *G = nullptr, *U = nullptr;  // U NULL: no gate
    int type = 0;                           // of G, U, H, dH, dG and dU
    long long ldg = 0, ldu = 0;
    void *H = nullptr;
    long long ldh = 0;
    void *GQ = nullptr, *UQ = nullptr;
    int q_type = 0;
    long long ldgq = 0, lduq = 0;
    float *GS = nullptr, *US = nullptr;
    long long ldgs = 0, ldus = 0;
    const void *dH = nullptr;
    long long lddh = 0;
    void *dG = nullptr, *dU = nullptr;
    long long lddg = 0, lddu = 0;
    int act = 0;
};
cudaError_t run_gated_act(const GatedAct &a, cudaStream_t stream, CallInfo *info);
cudaError_t run_gated_act_grad(const GatedAct &a, cudaStream_t stream, CallInfo *info);

}  // namespace gemm11

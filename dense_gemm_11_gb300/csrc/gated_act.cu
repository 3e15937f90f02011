// gated_act.cu -- the gated activation h = act(g) u of a feed-forward layer whose
// inputs are kept for the backward pass in 8 bits, and that backward pass:
//
//   forward    h = act(g) u, and g and u each as q = round8(x F / a), s = a / F
//              with a the largest |x| of a block of 128 of a row (the scales and
//              rounding of the quantizer, its layout "rows");
//   backward   with g' = gq gs and u' = uq us:
//              dg = dh u' act'(g'),  du = dh act(g'),  and, if asked for, h' =
//              act(g') u' again for the gradient of the weights that follow.
//
// Kept in 16 bits, g, u and h of a row of I columns are 6 I bytes; the 8-bit
// copies are 2.06 I.  The derivative is that of act at g', which the backward
// pass knows exactly: the copies' rounding is the only thing that is lost.
//
// Bound: memory.  One pass: 16 lanes hold 128 columns of a row, eight each, so
// that the maximum is four shuffles; everything is computed in FP32 and rounded
// once.
#include <algorithm>
#include <cstdint>

#include <cuda_fp8.h>

#include "experts.h"
#include "fp8.h"
#include "rows8.cuh"

namespace gemm11 {
namespace {

struct GatedArgs {
    int rows, cols;
    const void *G, *U;
    long long ldg, ldu;
    void *H;
    long long ldh;
    uint8_t *GQ, *UQ;
    long long ldgq, lduq;
    float *GS, *US;
    long long ldgs, ldus;
    const void *dH;
    long long lddh;
    void *dG, *dU;
    long long lddg, lddu;
    int act, e5m2;
    int per_cta;  // column blocks of a CTA
    int nx;       // CTAs along the columns
    int q_vec;    // rows of GQ and UQ take aligned 8-byte accesses
    unsigned *err;
    size_t h_extent, q_extent, s_extent;  // elements, checked by GEMM11_DEBUG builds (the smallest of the results written)
};

// act(x) and its derivative.  One exponential and one approximate reciprocal
// each, as the epilogues' forms, whose polynomial for the normal distribution's
// tail they share.
template <int ACT>
__device__ __forceinline__ void act_slope(float x, float &a, float &slope) {
    if constexpr (ACT == 0) {
        a = x;
        slope = 1.f;
    } else if constexpr (ACT == 1) {
        // Phi(x) + x phi(x); the tail's exponential is phi(x) sqrt(2 pi)
        const float e = __expf(-0.5f * x * x);
        const float t = rcp_approx(fmaf(0.3275911f * 0.70710678118654752f, fabsf(x), 1.f));
        float poly = fmaf(1.061405429f, t, -1.453152027f);
        poly = fmaf(poly, t, 1.421413741f);
        poly = fmaf(poly, t, -0.284496736f);
        poly = fmaf(poly, t, 0.254829592f);
        const float q = 0.5f * poly * t * e;
        const float cdf = x >= 0.f ? 1.f - q : q;
        a = x * cdf;
        slope = fmaf(0.39894228040143268f * x, e, cdf);
    } else if constexpr (ACT == 2) {
        a = x < 0.f ? 0.f : x;  // a NaN stays one
        slope = x > 0.f ? 1.f : 0.f;
    } else if constexpr (ACT == 3) {
        // x p and p + x p (1 - p) 2 u', p = 1 / (1 + exp(-2 u))
        const float u2 = 2.f * 0.79788456080286536f * fmaf(0.044715f * x, x * x, x);
        const float p = rcp_approx(1.f + __expf(-u2));
        a = x * p;
        const float w = p * (1.f - p);  // 0 where x * x could overflow
        slope = w > 0.f ? fmaf(x * w, 2.f * 0.79788456080286536f * fmaf(3.f * 0.044715f * x, x, 1.f), p) : p;
    } else {
        const float p = rcp_approx(1.f + __expf(-x));
        a = x * p;
        slope = fmaf(x, p * (1.f - p), p);
    }
}

__device__ __forceinline__ float fp8_top(int e5m2) { return e5m2 ? 57344.f : 448.f; }
__device__ __forceinline__ float fp8_floor(int e5m2) { return e5m2 ? 0x1p-110f : 0x1p-117f; }

__device__ __forceinline__ uint32_t to_fp8x4(float a, float b, float c, float d, int e5m2) {
    const __nv_fp8_interpretation_t t = e5m2 ? __NV_E5M2 : __NV_E4M3;
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, t);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, t);
    return lo | (hi << 16);
}
__device__ __forceinline__ float2 from_fp8x2(uint32_t w, int e5m2) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w & 0xFFFFu), e5m2 ? __NV_E5M2 : __NV_E4M3);
    return __half22float2(__half2(h));
}

// A block's scale and its eight elements of this lane in 8 bits.
__device__ __forceinline__ void keep8(const GatedArgs &p, const float (&v)[8], uint8_t *Q, long long ldq, float *S, long long lds, long long row, int c,
                                      int block, int sub, bool live) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
#pragma unroll
    for (int d = 8; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    m = fmaxf(m, fp8_floor(p.e5m2));
    const float top = fp8_top(p.e5m2), inv = top / m;
    if (!live) return;
    const long long at = static_cast<long long>(block) * lds + row;
    if (sub == 0 && debug_in_bounds(static_cast<size_t>(at) < p.s_extent, p.err)) S[at] = m / top;
    if (c >= p.cols) return;
    uint2 w;
    w.x = to_fp8x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv, p.e5m2);
    w.y = to_fp8x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv, p.e5m2);
    uint8_t *q = Q + row * ldq + c;
    const int left = p.cols - c;
    if (!debug_in_bounds(static_cast<size_t>(q - Q) + min(8, left) <= p.q_extent, p.err)) return;
    if (p.q_vec && left >= 8) {
        *reinterpret_cast<uint2 *>(q) = w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) q[i] = static_cast<uint8_t>((i < 4 ? w.x >> (8 * i) : w.y >> (8 * (i - 4))) & 0xFFu);
    }
}

template <int XT, bool VEC, int ACT>
__global__ void __launch_bounds__(256) gated_act_kernel(const GatedArgs p) {
    pdl_wait();
    pdl_launch_dependents();
    const int sub = threadIdx.x & 15;
    const int bx = blockIdx.x % p.nx, by = blockIdx.x / p.nx;
    const long long row = static_cast<long long>(by) * 16 + (threadIdx.x >> 4);
    const int nb = (p.cols + kScaleBlock - 1) / kScaleBlock;
    const int b0 = bx * p.per_cta, b1 = min(nb, b0 + p.per_cta);
    const bool inside = row < p.rows;
    constexpr int kDeep = 2;  // blocks in flight
    for (int b = b0; b < b1; b += kDeep) {
        Row8<XT> g[kDeep], u[kDeep];
#pragma unroll
        for (int d = 0; d < kDeep; ++d) {
            const int c = (b + d) * kScaleBlock + sub * 8;
            g[d].clear();
            u[d].clear();
            if (inside && b + d < b1 && c < p.cols) {
                g[d].template load<VEC>(p.G, row * p.ldg + c, p.cols - c);
                if (p.U) u[d].template load<VEC>(p.U, row * p.ldu + c, p.cols - c);
            }
        }
#pragma unroll
        for (int d = 0; d < kDeep; ++d) {
            const int c = (b + d) * kScaleBlock + sub * 8;
            const bool live = inside && b + d < b1;
            float vg[8], vu[8], h[8];
            g[d].widen(vg);
            u[d].widen(vu);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float slope;
                act_slope<ACT>(vg[i], h[i], slope);
                if (p.U) h[i] *= vu[i];
            }
            if (live && c < p.cols && debug_in_bounds(static_cast<size_t>(row * p.ldh + min(c + 8, p.cols)) <= p.h_extent, p.err)) {
                Row8<XT> out;
                out.round(h);
                out.template store<VEC>(p.H, row * p.ldh + c, p.cols - c);
            }
            keep8(p, vg, p.GQ, p.ldgq, p.GS, p.ldgs, row, c, b + d, sub, live);
            if (p.U) keep8(p, vu, p.UQ, p.lduq, p.US, p.ldus, row, c, b + d, sub, live);
        }
    }
}

// Eight 8-bit values times their scale.
__device__ __forceinline__ uint2 load_kept(const GatedArgs &p, const uint8_t *Q, long long at, int left) {
    if (p.q_vec && left >= 8) return __ldg(reinterpret_cast<const uint2 *>(Q + at));
    uint2 w = make_uint2(0, 0);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < left) (i < 4 ? w.x : w.y) |= static_cast<uint32_t>(Q[at + i]) << (8 * (i & 3));
    return w;
}
__device__ __forceinline__ void widen_kept(uint2 w, float s, int e5m2, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = from_fp8x2((i < 2 ? w.x : w.y) >> (16 * (i & 1)), e5m2);
        v[2 * i] = f.x * s;
        v[2 * i + 1] = f.y * s;
    }
}

template <int XT, bool VEC, int ACT>
__global__ void __launch_bounds__(256) gated_act_grad_kernel(const GatedArgs p) {
    pdl_wait();
    pdl_launch_dependents();
    const int sub = threadIdx.x & 15;
    const int bx = blockIdx.x % p.nx, by = blockIdx.x / p.nx;
    const long long row = static_cast<long long>(by) * 16 + (threadIdx.x >> 4);
    const int nb = (p.cols + kScaleBlock - 1) / kScaleBlock;
    const int b0 = bx * p.per_cta, b1 = min(nb, b0 + p.per_cta);
    if (row >= p.rows) return;
    constexpr int kDeep = 2;
    for (int b = b0; b < b1; b += kDeep) {
        Row8<XT> dh[kDeep];
        uint2 gq[kDeep], uq[kDeep];
        float gs[kDeep], us[kDeep];
#pragma unroll
        for (int d = 0; d < kDeep; ++d) {
            const int c = (b + d) * kScaleBlock + sub * 8;
            if (b + d >= b1 || c >= p.cols) continue;
            dh[d].template load<VEC>(p.dH, row * p.lddh + c, p.cols - c);
            gq[d] = load_kept(p, p.GQ, row * p.ldgq + c, p.cols - c);
            gs[d] = __ldg(p.GS + static_cast<long long>(b + d) * p.ldgs + row);
            if (p.UQ) {
                uq[d] = load_kept(p, p.UQ, row * p.lduq + c, p.cols - c);
                us[d] = __ldg(p.US + static_cast<long long>(b + d) * p.ldus + row);
            }
        }
#pragma unroll
        for (int d = 0; d < kDeep; ++d) {
            const int c = (b + d) * kScaleBlock + sub * 8;
            if (b + d >= b1 || c >= p.cols) continue;
            float vh[8], vg[8], vu[8], a[8];
            dh[d].widen(vh);
            widen_kept(gq[d], gs[d], p.e5m2, vg);
            if (p.UQ) widen_kept(uq[d], us[d], p.e5m2, vu);
            Row8<XT> out;
            const bool in = debug_in_bounds(static_cast<size_t>(row) * p.lddg + min(c + 8, p.cols) <= p.h_extent, p.err);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float slope;
                act_slope<ACT>(vg[i], a[i], slope);
                vg[i] = vh[i] * slope;
                if (p.UQ) vg[i] *= vu[i];
            }
            if (in) {
                out.round(vg);
                out.template store<VEC>(p.dG, row * p.lddg + c, p.cols - c);
            }
            if (p.dU && in) {
#pragma unroll
                for (int i = 0; i < 8; ++i) vg[i] = vh[i] * a[i];
                out.round(vg);
                out.template store<VEC>(p.dU, row * p.lddu + c, p.cols - c);
            }
            if (p.H && in) {
#pragma unroll
                for (int i = 0; i < 8; ++i) vg[i] = p.UQ ? a[i] * vu[i] : a[i];
                out.round(vg);
                out.template store<VEC>(p.H, row * p.ldh + c, p.cols - c);
            }
        }
    }
}

template <int XT, bool VEC, int ACT>
cudaError_t launch_gated(const GatedArgs &a, bool grad, cudaStream_t stream) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(a.nx) * ((a.rows + 15) / 16));
    const cudaError_t e = grad ? cudaLaunchKernelEx(&cfg, gated_act_grad_kernel<XT, VEC, ACT>, a) : cudaLaunchKernelEx(&cfg, gated_act_kernel<XT, VEC, ACT>, a);
    return e != cudaSuccess ? e : cudaPeekAtLastError();
}

template <int XT, bool VEC>
cudaError_t launch_gated(const GatedArgs &a, bool grad, cudaStream_t stream) {
    switch (a.act) {
        case 0: return launch_gated<XT, VEC, 0>(a, grad, stream);
        case 1: return launch_gated<XT, VEC, 1>(a, grad, stream);
        case 2: return launch_gated<XT, VEC, 2>(a, grad, stream);
        case 3: return launch_gated<XT, VEC, 3>(a, grad, stream);
        default: return launch_gated<XT, VEC, kActSilu>(a, grad, stream);
    }
}

cudaError_t gated(const GatedAct &g, bool grad, cudaStream_t stream) {
    GatedArgs a = {};
    a.rows = g.rows;
    a.cols = g.cols;
    a.G = g.G;
    a.U = g.U;
    a.ldg = g.ldg;
    a.ldu = g.ldu;
    a.H = g.H;
    a.ldh = g.ldh;
    a.GQ = static_cast<uint8_t *>(g.GQ);
    a.UQ = static_cast<uint8_t *>(g.UQ);
    a.ldgq = g.ldgq;
    a.lduq = g.lduq;
    a.GS = g.GS;
    a.US = g.US;
    a.ldgs = g.ldgs;
    a.ldus = g.ldus;
    a.dH = g.dH;
    a.lddh = g.lddh;
    a.dG = g.dG;
    a.dU = g.dU;
    a.lddg = g.lddg;
    a.lddu = g.lddu;
    a.act = g.act;
    a.e5m2 = g.q_type == kTypeE5M2;
    a.err = watchdog_word();
    const int b = g.type == kOutF32 ? 4 : 2;
    auto fits = [&](const void *p, long long ld) { return !p || rows_aligned(p, ld, b, g.rows); };
    const bool vec = fits(g.G, g.ldg) && fits(g.U, g.ldu) && fits(g.H, g.ldh) && fits(g.dH, g.lddh) && fits(g.dG, g.lddg) && fits(g.dU, g.lddu);
    auto q_fits = [&](const void *p, long long ld) { return reinterpret_cast<uintptr_t>(p) % 8 == 0 && (g.rows == 1 || ld % 8 == 0); };
    a.q_vec = q_fits(g.GQ, g.ldgq) && (!g.UQ || q_fits(g.UQ, g.lduq));
    const int nb = (g.cols + kScaleBlock - 1) / kScaleBlock;
    if (kDebugBuild) {
        const long long ld = grad ? g.lddg : g.ldh;
        a.h_extent = static_cast<size_t>((g.rows - 1LL) * ld + g.cols);
        a.h_extent -= std::min(a.h_extent, debug_shrink_c());
        a.q_extent = static_cast<size_t>((g.rows - 1LL) * (g.UQ ? std::max(g.ldgq, g.lduq) : g.ldgq) + g.cols);
        a.s_extent = static_cast<size_t>((nb - 1LL) * (g.US ? std::max(g.ldgs, g.ldus) : g.ldgs) + g.rows);
    }
    // Two column blocks a CTA (kDeep) once that leaves every SM several CTAs.
    const long long ctas = static_cast<long long>((g.rows + 15) / 16) * nb;
    a.per_cta = ctas >= 16LL * device_sm_count() ? 2 : 1;
    a.nx = (nb + a.per_cta - 1) / a.per_cta;
    switch (g.type * 2 + (vec ? 1 : 0)) {
        case 0: return launch_gated<kOutF32, false>(a, grad, stream);
        case 1: return launch_gated<kOutF32, true>(a, grad, stream);
        case 2: return launch_gated<kOutF16, false>(a, grad, stream);
        case 3: return launch_gated<kOutF16, true>(a, grad, stream);
        case 4: return launch_gated<kOutBF16, false>(a, grad, stream);
        default: return launch_gated<kOutBF16, true>(a, grad, stream);
    }
}

}  // namespace

cudaError_t run_gated_act(const GatedAct &a, cudaStream_t stream, CallInfo *info) {
    info->plan = "fp8_gated_act";
    info->launches = 1;
    return gated(a, false, stream);
}

cudaError_t run_gated_act_grad(const GatedAct &a, cudaStream_t stream, CallInfo *info) {
    info->plan = "fp8_gated_act_grad";
    info->launches = 1;
    return gated(a, true, stream);
}

}  // namespace gemm11

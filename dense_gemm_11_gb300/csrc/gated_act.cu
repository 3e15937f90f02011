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
// pass knows exactly: the copies' rounding is the only thing that is lost.  As in the
// quantizer, a NaN leaves the rest of its block alone and an infinity makes its
// block's scale infinite: what the backward pass computes from those 128 columns is NaN.
//
// Bound: memory.  One pass: 16 lanes hold 128 columns of a row, eight each, so
// that the maximum is four shuffles; everything is computed in FP32 and rounded
// once.  Measured on BF16 and e4m3 of 8192 x 11008: forward 108 us (727 MB, 6.7
// TB/s), backward with h 133 (908 MB, 6.8 TB/s); with GELU, whose polynomial adds
// to the arithmetic, 122 and 140.  32 x 11008 2.4 us in a graph.
#include <algorithm>
#include <cstdint>

#include <cuda_fp8.h>

#include "experts.h"
#include "fp8.cuh"
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

// Two FP32 values at a time: the additions and products of a pair are one
// instruction (PTX f32x2), which counts here, where a block's arithmetic is close
// to what its bytes take.
using f2 = uint64_t;
__device__ __forceinline__ f2 both(float v) { return pack_f32x2(v, v); }
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) { return mul_f32x2(a, b); }
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
// 2^x and 1 / x of both (PTX approximations, 2 ulp; results below 2^-126 are 0).
__device__ __forceinline__ f2 exp2_2(f2 x) {
    float a, b;
    unpack_f32x2(x, a, b);
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(a));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(b));
    return pack_f32x2(a, b);
}
__device__ __forceinline__ f2 rcp2(f2 x) {
    float a, b;
    unpack_f32x2(x, a, b);
    return pack_f32x2(rcp_approx(a), rcp_approx(b));
}

// act(x) and its derivative, one exponential and one reciprocal each.  GELU takes
// the normal distribution's tail Q(|x|) from the polynomial of the epilogues'
// gelu_erf; the exponential of that is phi(x) sqrt(2 pi), which the derivative
// Phi(x) + x phi(x) needs too.
template <int ACT, bool SLOPE>
__device__ __forceinline__ void act2(f2 x, f2 &a, f2 &slope) {
    constexpr float kLog2e = 1.4426950408889634f;
    if constexpr (ACT == 0) {
        a = x;
        slope = both(1.f);
    } else if constexpr (ACT == 1) {
        float x0, x1, q0, q1;
        unpack_f32x2(x, x0, x1);
        const f2 e = exp2_2(mul2(mul2(x, both(-0.5f * kLog2e)), x));
        const f2 t = rcp2(fma2(pack_f32x2(fabsf(x0), fabsf(x1)), both(0.3275911f * 0.70710678118654752f), both(1.f)));
        f2 poly = fma2(both(1.061405429f), t, both(-1.453152027f));
        poly = fma2(poly, t, both(1.421413741f));
        poly = fma2(poly, t, both(-0.284496736f));
        poly = fma2(poly, t, both(0.254829592f));
        const f2 q = mul2(mul2(poly, both(0.5f)), mul2(t, e));
        unpack_f32x2(q, q0, q1);
        const f2 cdf = pack_f32x2(x0 >= 0.f ? 1.f - q0 : q0, x1 >= 0.f ? 1.f - q1 : q1);
        a = mul2(x, cdf);
        if (SLOPE) slope = fma2(mul2(x, both(0.39894228040143268f)), e, cdf);
    } else if constexpr (ACT == 2) {
        float x0, x1;
        unpack_f32x2(x, x0, x1);
        a = pack_f32x2(x0 < 0.f ? 0.f : x0, x1 < 0.f ? 0.f : x1);  // a NaN stays one
        if (SLOPE) slope = pack_f32x2(x0 > 0.f ? 1.f : 0.f, x1 > 0.f ? 1.f : 0.f);
    } else {
        // p = 1 / (1 + exp(-z)), z = x for SiLU and 2 sqrt(2 / pi) (x + 0.044715 x^3)
        // for the tanh form: x p and p + x p (1 - p) z'
        constexpr float kC = ACT == 3 ? 2.f * 0.79788456080286536f : 1.f;
        f2 z = mul2(x, both(-kC * kLog2e));
        if (ACT == 3) z = mul2(z, fma2(mul2(x, both(0.044715f)), x, both(1.f)));
        const f2 p = rcp2(add2(exp2_2(z), both(1.f)));
        a = mul2(x, p);
        if (SLOPE) {
            const f2 w = fma2(mul2(p, both(-1.f)), p, p);
            if (ACT == 3) {
                // where w is 0, x^2 could be an infinity
                float w0, w1, s0, s1, p0, p1;
                unpack_f32x2(w, w0, w1);
                unpack_f32x2(p, p0, p1);
                unpack_f32x2(fma2(mul2(x, w), mul2(fma2(mul2(x, both(3.f * 0.044715f)), x, both(1.f)), both(kC)), p), s0, s1);
                slope = pack_f32x2(w0 > 0.f ? s0 : p0, w1 > 0.f ? s1 : p1);
            } else {
                slope = fma2(x, w, p);
            }
        }
    }
}
template <bool SLOPE>
__device__ __forceinline__ void act8(int act, const f2 (&x)[4], f2 (&a)[4], f2 (&slope)[4]) {
    switch (act) {
        case 0:
#pragma unroll
            for (int i = 0; i < 4; ++i) act2<0, SLOPE>(x[i], a[i], slope[i]);
            break;
        case 1:
#pragma unroll
            for (int i = 0; i < 4; ++i) act2<1, SLOPE>(x[i], a[i], slope[i]);
            break;
        case 2:
#pragma unroll
            for (int i = 0; i < 4; ++i) act2<2, SLOPE>(x[i], a[i], slope[i]);
            break;
        case 3:
#pragma unroll
            for (int i = 0; i < 4; ++i) act2<3, SLOPE>(x[i], a[i], slope[i]);
            break;
        default:
#pragma unroll
            for (int i = 0; i < 4; ++i) act2<kActSilu, SLOPE>(x[i], a[i], slope[i]);
    }
}

template <int XT>
__device__ __forceinline__ void widen2(const Row8<XT> &r, f2 (&v)[4]) {
    float f[8];
    r.widen(f);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = pack_f32x2(f[2 * i], f[2 * i + 1]);
}
template <int XT>
__device__ __forceinline__ Row8<XT> round2(const f2 (&v)[4]) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) unpack_f32x2(v[i], f[2 * i], f[2 * i + 1]);
    Row8<XT> r;
    r.round(f);
    return r;
}

// The larger magnitudes of two rows' eight elements, NaN left out: (a's, b's) in
// the type's own pair, or as floats.
template <int XT>
struct Maxima;
template <>
struct Maxima<kOutF32> {
    float a, b;
    __device__ __forceinline__ void take(const Row8<kOutF32> &ra, const Row8<kOutF32> &rb) {
        float v[8], w[8];
        ra.widen(v);
        rb.widen(w);
        a = b = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(v[i])), b = fmaxf(b, fabsf(w[i]));
    }
    __device__ __forceinline__ void join(int lanes) {
        a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, lanes));
        b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, lanes));
    }
    __device__ __forceinline__ float first() const { return a; }
    __device__ __forceinline__ float second() const { return b; }
};
template <typename T2, typename T1>
struct Maxima16 {
    T2 m;
    static __device__ __forceinline__ T2 pair(uint32_t w) {
        w &= 0x7FFF7FFFu;
        return *reinterpret_cast<const T2 *>(&w);
    }
    static __device__ __forceinline__ T2 of(uint4 w) { return __hmax2(__hmax2(pair(w.x), pair(w.y)), __hmax2(pair(w.z), pair(w.w))); }
    __device__ __forceinline__ void take(uint4 wa, uint4 wb) {
        const T2 a = of(wa), b = of(wb);
        m.x = __hmax(a.x, a.y), m.y = __hmax(b.x, b.y);
    }
    __device__ __forceinline__ void join(int lanes) {
        const uint32_t o = __shfl_xor_sync(0xffffffffu, *reinterpret_cast<const uint32_t *>(&m), lanes);
        m = __hmax2(m, *reinterpret_cast<const T2 *>(&o));
    }
};
template <>
struct Maxima<kOutF16> : Maxima16<__half2, __half> {
    __device__ __forceinline__ void take(const Row8<kOutF16> &a, const Row8<kOutF16> &b) { Maxima16::take(a.w[0], b.w[0]); }
    __device__ __forceinline__ float first() const { return __half2float(m.x); }
    __device__ __forceinline__ float second() const { return __half2float(m.y); }
};
template <>
struct Maxima<kOutBF16> : Maxima16<__nv_bfloat162, __nv_bfloat16> {
    __device__ __forceinline__ void take(const Row8<kOutBF16> &a, const Row8<kOutBF16> &b) { Maxima16::take(a.w[0], b.w[0]); }
    __device__ __forceinline__ float first() const { return __bfloat162float(m.x); }
    __device__ __forceinline__ float second() const { return __bfloat162float(m.y); }
};

template <bool E5M2>
__device__ __forceinline__ uint32_t to_fp8x2(f2 v) {
    float a, b;
    unpack_f32x2(v, a, b);
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, E5M2 ? __NV_E5M2 : __NV_E4M3);
}
template <bool E5M2>
__device__ __forceinline__ f2 from_fp8x2(uint32_t w) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w & 0xFFFFu), E5M2 ? __NV_E5M2 : __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    return pack_f32x2(f.x, f.y);
}

// Eight elements in 8 bits, `inv` the reciprocal of their scale.
template <bool E5M2>
__device__ __forceinline__ void keep8(const GatedArgs &p, const f2 (&v)[4], float inv, uint8_t *Q, long long at, int left) {
    const f2 i2 = both(inv);
    uint2 w;
    w.x = to_fp8x2<E5M2>(mul2(v[0], i2)) | to_fp8x2<E5M2>(mul2(v[1], i2)) << 16;
    w.y = to_fp8x2<E5M2>(mul2(v[2], i2)) | to_fp8x2<E5M2>(mul2(v[3], i2)) << 16;
    if (!debug_in_bounds(static_cast<size_t>(at) + min(8, left) <= p.q_extent, p.err)) return;
    if (p.q_vec && left >= 8) {
        *reinterpret_cast<uint2 *>(Q + at) = w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) Q[at + i] = static_cast<uint8_t>((i < 4 ? w.x >> (8 * i) : w.y >> (8 * (i - 4))) & 0xFFu);
    }
}

constexpr int kDeep = 2;  // blocks of a row in flight

template <int XT, bool VEC, bool E5M2, bool GATED>
__global__ void __launch_bounds__(256, XT == kOutF32 ? 1 : 5) gated_act_kernel(const GatedArgs p) {
    pdl_wait();
    pdl_launch_dependents();
    const int sub = threadIdx.x & 15, group = threadIdx.x & 16;
    const int bx = blockIdx.x % p.nx, by = blockIdx.x / p.nx;
    const long long row = static_cast<long long>(by) * 16 + (threadIdx.x >> 4);
    const int nb = (p.cols + kScaleBlock - 1) / kScaleBlock;
    const int b0 = bx * p.per_cta, b1 = min(nb, b0 + p.per_cta);
    const bool inside = row < p.rows;
    constexpr float kTop = E5M2 ? 57344.f : 448.f, kFloor = E5M2 ? 0x1p-110f : 0x1p-117f;
    for (int b = b0; b < b1; b += kDeep) {
        Row8<XT> g[kDeep], u[kDeep];
#pragma unroll
        for (int d = 0; d < kDeep; ++d) {
            const int c = (b + d) * kScaleBlock + sub * 8;
            g[d].clear();
            u[d].clear();
            if (inside && b + d < b1 && c < p.cols) {
                g[d].template load<VEC>(p.G, row * p.ldg + c, p.cols - c);
                if (GATED) u[d].template load<VEC>(p.U, row * p.ldu + c, p.cols - c);
            }
        }
        Maxima<XT> m[kDeep];
#pragma unroll
        for (int d = 0; d < kDeep; ++d) m[d].take(g[d], u[d]);
#pragma unroll
        for (int lanes = 8; lanes >= 1; lanes >>= 1)
#pragma unroll
            for (int d = 0; d < kDeep; ++d) m[d].join(lanes);
        // The divisions, one a lane: lanes 0 .. 3 of the sixteen have F / a of (block
        // 0, g), (block 0, u), (block 1, g), (block 1, u), lanes 4 .. 7 a / F.
        static_assert(kDeep == 2, "lanes of the divisions");
        const float a = fmaxf((sub & 2) ? ((sub & 1) ? m[1].second() : m[1].first()) : ((sub & 1) ? m[0].second() : m[0].first()), kFloor);
        const bool scale = sub & 4;
        const float quotient = (scale ? a : kTop) / (scale ? kTop : a);
        if (scale && sub < 8 && inside && (GATED || !(sub & 1))) {
            const int block = b + ((sub >> 1) & 1);
            const long long at = static_cast<long long>(block) * ((sub & 1) ? p.ldus : p.ldgs) + row;
            if (block < b1 && debug_in_bounds(static_cast<size_t>(at) < p.s_extent, p.err)) ((sub & 1) ? p.US : p.GS)[at] = quotient;
        }
#pragma unroll
        for (int d = 0; d < kDeep; ++d) {
            const int c = (b + d) * kScaleBlock + sub * 8;
            const float inv_g = __shfl_sync(0xffffffffu, quotient, group + 2 * d), inv_u = GATED ? __shfl_sync(0xffffffffu, quotient, group + 2 * d + 1) : 0.f;
            if (!inside || b + d >= b1 || c >= p.cols) continue;
            f2 vg[4], vu[4], h[4], slope[4];
            widen2(g[d], vg);
            act8<false>(p.act, vg, h, slope);
            if (GATED) {
                widen2(u[d], vu);
#pragma unroll
                for (int i = 0; i < 4; ++i) h[i] = mul2(h[i], vu[i]);
            }
            if (debug_in_bounds(static_cast<size_t>(row * p.ldh + min(c + 8, p.cols)) <= p.h_extent, p.err))
                round2<XT>(h).template store<VEC>(p.H, row * p.ldh + c, p.cols - c);
            keep8<E5M2>(p, vg, inv_g, p.GQ, row * p.ldgq + c, p.cols - c);
            if (GATED) keep8<E5M2>(p, vu, inv_u, p.UQ, row * p.lduq + c, p.cols - c);
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
template <bool E5M2>
__device__ __forceinline__ void widen_kept(uint2 w, float s, f2 (&v)[4]) {
    const f2 s2 = both(s);
    v[0] = mul2(from_fp8x2<E5M2>(w.x), s2);
    v[1] = mul2(from_fp8x2<E5M2>(w.x >> 16), s2);
    v[2] = mul2(from_fp8x2<E5M2>(w.y), s2);
    v[3] = mul2(from_fp8x2<E5M2>(w.y >> 16), s2);
}

template <int XT, bool VEC, bool E5M2, bool GATED>
__global__ void __launch_bounds__(256, XT == kOutF32 ? 1 : 4) gated_act_grad_kernel(const GatedArgs p) {
    pdl_wait();
    pdl_launch_dependents();
    const int sub = threadIdx.x & 15;
    const int bx = blockIdx.x % p.nx, by = blockIdx.x / p.nx;
    const long long row = static_cast<long long>(by) * 16 + (threadIdx.x >> 4);
    const int nb = (p.cols + kScaleBlock - 1) / kScaleBlock;
    const int b0 = bx * p.per_cta, b1 = min(nb, b0 + p.per_cta);
    if (row >= p.rows) return;
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
            if (GATED) {
                uq[d] = load_kept(p, p.UQ, row * p.lduq + c, p.cols - c);
                us[d] = __ldg(p.US + static_cast<long long>(b + d) * p.ldus + row);
            }
        }
#pragma unroll
        for (int d = 0; d < kDeep; ++d) {
            const int c = (b + d) * kScaleBlock + sub * 8;
            if (b + d >= b1 || c >= p.cols) continue;
            if (!debug_in_bounds(static_cast<size_t>(row) * p.lddg + min(c + 8, p.cols) <= p.h_extent, p.err)) continue;
            f2 vh[4], vg[4], vu[4], a[4], slope[4];
            widen2(dh[d], vh);
            widen_kept<E5M2>(gq[d], gs[d], vg);
            act8<true>(p.act, vg, a, slope);
#pragma unroll
            for (int i = 0; i < 4; ++i) slope[i] = mul2(vh[i], slope[i]);
            if (GATED) {
                widen_kept<E5M2>(uq[d], us[d], vu);
#pragma unroll
                for (int i = 0; i < 4; ++i) slope[i] = mul2(slope[i], vu[i]), vh[i] = mul2(vh[i], a[i]);
                round2<XT>(vh).template store<VEC>(p.dU, row * p.lddu + c, p.cols - c);
            }
            round2<XT>(slope).template store<VEC>(p.dG, row * p.lddg + c, p.cols - c);
            if (p.H) {
                if (GATED) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) a[i] = mul2(a[i], vu[i]);
                }
                round2<XT>(a).template store<VEC>(p.H, row * p.ldh + c, p.cols - c);
            }
        }
    }
}

template <int XT, bool VEC, bool E5M2, bool GATED>
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
    const cudaError_t e = grad ? cudaLaunchKernelEx(&cfg, gated_act_grad_kernel<XT, VEC, E5M2, GATED>, a) : cudaLaunchKernelEx(&cfg, gated_act_kernel<XT, VEC, E5M2, GATED>, a);
    return e != cudaSuccess ? e : cudaPeekAtLastError();
}

template <int XT, bool VEC>
cudaError_t launch_gated(const GatedArgs &a, bool grad, cudaStream_t stream) {
    if (grad ? a.UQ != nullptr : a.U != nullptr)
        return a.e5m2 ? launch_gated<XT, VEC, true, true>(a, grad, stream) : launch_gated<XT, VEC, false, true>(a, grad, stream);
    return a.e5m2 ? launch_gated<XT, VEC, true, false>(a, grad, stream) : launch_gated<XT, VEC, false, false>(a, grad, stream);
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
    // Column blocks of a CTA: one while that leaves SMs without work, then four
    // (8192 x 11008 BF16: 112 us in twos, 109 in fours, 110 in eights; backward 148,
    // 145, 143), or two in FP32 forwards (4096 x 11008: 90.6, 92.4 in fours).  The
    // launch bounds of the 16-bit kernels add to that: 115 -> 109 and 145 -> 134.
    const long long ctas = static_cast<long long>((g.rows + 15) / 16) * nb;
    a.per_cta = ctas < 16LL * device_sm_count() ? 1 : !grad && g.type == kOutF32 ? 2 : 4;
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

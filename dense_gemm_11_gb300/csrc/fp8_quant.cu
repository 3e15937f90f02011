// fp8_quant.cu -- FP32 / FP16 / BF16 matrices to 8-bit floating point with one
// FP32 scale for each block of 128.
//
// A block's scale is s = a / F with a = max(max |x|, floor) and F the 8-bit
// type's largest value (448 for e4m3, 57344 for e5m2); an element becomes
// q = round8(x * (F / a)), one IEEE division for the block and one FP32
// multiplication for the element, to nearest even.  The floor, F 2^-126 rounded
// up to a power of two (2^-117 and 2^-110), keeps both quotients normal numbers
// (s = 2^-126 / 0.875 and F / a = 1.75 * 2^125 at the floor), so that a block of
// zeros needs no case of its own.  |x| (F / a) exceeds F by at most
// an ulp, which rounds to F.  A NaN becomes the NaN code and leaves the rest
// of its block alone (fmaxf skips it); an infinity makes its block's scale
// infinite and with it every product of the block NaN or infinite.
//
// Bound: memory.  Every element is read once, as 16-byte loads where rows
// allow it, kept in registers between the maximum and the rounding, and
// written once.  Three kernels, one for each direction of the blocks:
//   rows    16 lanes hold one 1 x 128 block (8 elements each); a CTA covers
//           16 rows so that its scales, which lie along the rows, share sectors;
//   cols    a CTA holds a tile of 128 rows x 64 columns, takes the maxima down
//           its columns and turns the tile round in shared memory (bytes, rows
//           of 33 words: neither side has bank conflicts);
//   blocks  a CTA holds one 128 x 128 block.
// Measured on BF16 of 4096 x 11008 (135 MB read and written, several such
// matrices in turn): rows 28.7 us, cols 30.1, blocks 28.5, 4.5 to 4.7 TB/s; on
// FP32 of 11008 x 4096, 225 MB, blocks takes 36.6 us, 6.2 TB/s; rows of 16 x
// 4096, one wave of small CTAs, 1.5 us.
#include <algorithm>

#include <cuda_fp8.h>

#include "fp8.h"
#include "ptx.cuh"

namespace gemm11 {
namespace {


struct QuantArgs {
    const void *X;
    long long ldx;
    uint8_t *Q;
    long long ldq;
    float *S;
    long long lds;
    int rows, cols;
    int e5m2;
    int per_cta;  // rows kernel: column blocks of a CTA
    int nx;       // CTAs along the columns (the grid is one-dimensional: rows may be many)
    int q_vec;    // Q rows take aligned 8-byte (rows, blocks) or 4-byte (cols) stores
    unsigned *err;
    size_t q_extent, s_extent;  // checked by GEMM11_DEBUG builds
};

__device__ __forceinline__ bool scale_inside(const QuantArgs &p, long long at) {
    return debug_in_bounds(static_cast<size_t>(at) < p.s_extent, p.err);
}

template <int XT>
struct XElem;
template <>
struct XElem<kOutF32> {
    using T = float;
};
template <>
struct XElem<kOutF16> {
    using T = __half;
};
template <>
struct XElem<kOutBF16> {
    using T = __nv_bfloat16;
};

// Eight elements of a row as they are in memory: 16-bit types take half the
// registers that their FP32 values would.
template <int XT>
struct Eight {
    uint4 w[XT == kOutF32 ? 2 : 1];
    __device__ __forceinline__ void clear() {
        w[0] = make_uint4(0, 0, 0, 0);
        if (XT == kOutF32) w[XT == kOutF32 ? 1 : 0] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void widen(float (&v)[8]) const {
        if constexpr (XT == kOutF32) {
            v[0] = __uint_as_float(w[0].x), v[1] = __uint_as_float(w[0].y), v[2] = __uint_as_float(w[0].z), v[3] = __uint_as_float(w[0].w);
            v[4] = __uint_as_float(w[1].x), v[5] = __uint_as_float(w[1].y), v[6] = __uint_as_float(w[1].z), v[7] = __uint_as_float(w[1].w);
        } else {
            unpack8_out16(w[0], XT, v);
        }
    }
    // Elements [c, c + 8) of row `row`, zeros from `cols` on.  VEC: rows start
    // on 16-byte boundaries and c is a multiple of 8.
    template <bool VEC>
    __device__ __forceinline__ void load(const QuantArgs &p, long long row, int c) {
        using T = typename XElem<XT>::T;
        const T *x = static_cast<const T *>(p.X) + row * p.ldx + c;
        if (VEC && c + 8 <= p.cols) {
            w[0] = __ldg(reinterpret_cast<const uint4 *>(x));
            if constexpr (XT == kOutF32) w[1] = __ldg(reinterpret_cast<const uint4 *>(x) + 1);
        } else {
            clear();
            T *e = reinterpret_cast<T *>(w);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c + i < p.cols) e[i] = x[i];
        }
    }
};

template <int XT>
__device__ __forceinline__ float max8(const Eight<XT> &x) {
    float v[8], m = 0.f;
    x.widen(v);
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
    return m;
}

__device__ __forceinline__ float type_max(int e5m2) { return e5m2 ? 57344.f : 448.f; }
__device__ __forceinline__ float type_floor(int e5m2) { return e5m2 ? 0x1p-110f : 0x1p-117f; }

// Four values, scaled and rounded, as packed bytes (the first lowest).
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d, int e5m2) {
    const __nv_fp8_interpretation_t t = e5m2 ? __NV_E5M2 : __NV_E4M3;
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, t);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, t);
    return lo | (hi << 16);
}

template <int XT>
__device__ __forceinline__ void store8(const QuantArgs &p, long long row, int c, const Eight<XT> &x, float inv) {
    float v[8];
    x.widen(v);
    uint2 w;
    w.x = pack4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv, p.e5m2);
    w.y = pack4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv, p.e5m2);
    uint8_t *q = p.Q + row * p.ldq + c;
    if (!debug_in_bounds(c >= p.cols || static_cast<size_t>(q - p.Q) + min(8, p.cols - c) <= p.q_extent, p.err)) return;
    if (p.q_vec && c + 8 <= p.cols) {
        *reinterpret_cast<uint2 *>(q) = w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < p.cols) q[i] = static_cast<uint8_t>((i < 4 ? w.x >> (8 * i) : w.y >> (8 * (i - 4))) & 0xFFu);
    }
}

// 1 x 128 blocks: half-warp h of the CTA has row 16 by + h, and the CTA column
// blocks [bx * per_cta, + per_cta).
template <int XT, bool VEC>
__global__ void __launch_bounds__(256) quant_rows_kernel(const QuantArgs p) {
    pdl_wait();
    pdl_launch_dependents();
    const int sub = threadIdx.x & 15;
    const int bx = blockIdx.x % p.nx, by = blockIdx.x / p.nx;
    const long long row = static_cast<long long>(by) * 16 + (threadIdx.x >> 4);
    const int nb = (p.cols + kScaleBlock - 1) / kScaleBlock;
    const int b0 = bx * p.per_cta, b1 = min(nb, b0 + p.per_cta);
    const bool live = row < p.rows;
    constexpr int kDeep = 4;  // blocks in flight
    for (int b = b0; b < b1; b += kDeep) {
        Eight<XT> v[kDeep];
#pragma unroll
        for (int u = 0; u < kDeep; ++u) {
            if (live && b + u < b1)
                v[u].template load<VEC>(p, row, (b + u) * kScaleBlock + sub * 8);
            else
                v[u].clear();
        }
#pragma unroll
        for (int u = 0; u < kDeep; ++u) {
            float m = max8(v[u]);
#pragma unroll
            for (int d = 8; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
            m = fmaxf(m, type_floor(p.e5m2));
            const float top = type_max(p.e5m2);
            if (live && b + u < b1) {
                store8(p, row, (b + u) * kScaleBlock + sub * 8, v[u], top / m);
                if (sub == 0 && scale_inside(p, static_cast<long long>(b + u) * p.lds + row)) p.S[static_cast<long long>(b + u) * p.lds + row] = m / top;
            }
        }
    }
}

// 128 x 128 blocks, one for each CTA: 16 lanes x 8 elements along a row, 16
// rows at a time.
template <int XT, bool VEC>
__global__ void __launch_bounds__(256, 3) quant_blocks_kernel(const QuantArgs p) {
    pdl_wait();
    pdl_launch_dependents();
    __shared__ float warp_max[8];
    const int bx = blockIdx.x % p.nx, by = blockIdx.x / p.nx;
    const int c = bx * kScaleBlock + (threadIdx.x & 15) * 8;
    const long long r0 = static_cast<long long>(by) * kScaleBlock + (threadIdx.x >> 4);
    Eight<XT> v[8];
    float m = 0.f;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        if (r0 + 16 * u < p.rows)
            v[u].template load<VEC>(p, r0 + 16 * u, c);
        else
            v[u].clear();
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) m = fmaxf(m, max8(v[u]));
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = m;
    __syncthreads();
    m = type_floor(p.e5m2);
#pragma unroll
    for (int w = 0; w < 8; ++w) m = fmaxf(m, warp_max[w]);
    const float top = type_max(p.e5m2), inv = top / m;
    if (threadIdx.x == 0 && scale_inside(p, static_cast<long long>(by) * p.lds + bx)) p.S[static_cast<long long>(by) * p.lds + bx] = m / top;
#pragma unroll
    for (int u = 0; u < 8; ++u)
        if (r0 + 16 * u < p.rows) store8(p, r0 + 16 * u, c, v[u], inv);
}

// 128 x 1 blocks, the result transposed: a CTA has rows [128 by, +128) of
// X and columns [64 bx, +64); thread t has 8 columns (t % 8) and
// the 4 rows 4 (t / 8) + i, whose bytes become one word of the turned tile.
template <int XT, bool VEC>
__global__ void __launch_bounds__(256, 6) quant_cols_kernel(const QuantArgs p) {
    pdl_wait();
    pdl_launch_dependents();
    __shared__ float part[8][64];
    __shared__ uint32_t turned[64][33];
    const int cg = threadIdx.x & 7, rg = threadIdx.x >> 3, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int bx = blockIdx.x % p.nx, by = blockIdx.x / p.nx;
    const int c0 = bx * 64;
    const long long r0 = static_cast<long long>(by) * kScaleBlock;
    Eight<XT> v[4];
    float m[8], f[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const long long r = r0 + rg * 4 + i;
        if (r < p.rows)
            v[i].template load<VEC>(p, r, c0 + cg * 8);
        else
            v[i].clear();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i].widen(f[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        m[j] = fmaxf(fmaxf(fabsf(f[0][j]), fabsf(f[1][j])), fmaxf(fabsf(f[2][j]), fabsf(f[3][j])));
        m[j] = fmaxf(m[j], __shfl_xor_sync(0xffffffffu, m[j], 8));
        m[j] = fmaxf(m[j], __shfl_xor_sync(0xffffffffu, m[j], 16));
    }
    if (lane < 8) {
#pragma unroll
        for (int j = 0; j < 8; ++j) part[warp][cg * 8 + j] = m[j];
    }
    __syncthreads();
    const float top = type_max(p.e5m2);
    if (threadIdx.x < 64) {
        float a = type_floor(p.e5m2);
#pragma unroll
        for (int w = 0; w < 8; ++w) a = fmaxf(a, part[w][threadIdx.x]);
        part[0][threadIdx.x] = top / a;
        if (c0 + static_cast<int>(threadIdx.x) < p.cols && scale_inside(p, static_cast<long long>(by) * p.lds + c0 + threadIdx.x))
            p.S[static_cast<long long>(by) * p.lds + c0 + threadIdx.x] = a / top;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i].widen(f[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float inv = part[0][cg * 8 + j];
        turned[cg * 8 + j][rg] = pack4(f[0][j] * inv, f[1][j] * inv, f[2][j] * inv, f[3][j] * inv, p.e5m2);
    }
    __syncthreads();
    const long long left = p.rows - r0;  // bytes of a turned row that exist
    for (int c = warp; c < 64 && c0 + c < p.cols; c += 8) {
        uint8_t *q = p.Q + static_cast<long long>(c0 + c) * p.ldq + r0 + lane * 4;
        const uint32_t w = turned[c][lane];
        if (!debug_in_bounds(lane * 4 >= left || static_cast<size_t>(q - p.Q) + min(4LL, left - lane * 4) <= p.q_extent, p.err)) continue;
        if (p.q_vec && lane * 4 + 4 <= left) {
            *reinterpret_cast<uint32_t *>(q) = w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (lane * 4 + i < left) q[i] = static_cast<uint8_t>((w >> (8 * i)) & 0xFFu);
        }
    }
}

template <int XT, bool VEC>
cudaError_t launch_quant(const QuantArgs &a, int layout, cudaStream_t stream, CallInfo *info) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    QuantArgs args = a;
    const int nb = (a.cols + kScaleBlock - 1) / kScaleBlock, rb = (a.rows + kScaleBlock - 1) / kScaleBlock;
    cudaError_t e;
    info->launches = 1;
    if (layout == 0) {
        // One column block a CTA while that leaves SMs without work, else up to four (kDeep).
        const long long ctas = static_cast<long long>((a.rows + 15) / 16) * nb;
        args.per_cta = ctas >= 16LL * device_sm_count() ? 4 : 1;
        args.nx = (nb + args.per_cta - 1) / args.per_cta;
        cfg.gridDim = dim3(static_cast<unsigned>(args.nx) * ((a.rows + 15) / 16));
        info->plan = "fp8_quant_rows";
        e = cudaLaunchKernelEx(&cfg, quant_rows_kernel<XT, VEC>, args);
    } else if (layout == 1) {
        args.nx = (a.cols + 63) / 64;
        cfg.gridDim = dim3(static_cast<unsigned>(args.nx) * rb);
        info->plan = "fp8_quant_cols";
        e = cudaLaunchKernelEx(&cfg, quant_cols_kernel<XT, VEC>, args);
    } else {
        args.nx = nb;
        cfg.gridDim = dim3(static_cast<unsigned>(nb) * rb);
        info->plan = "fp8_quant_blocks";
        e = cudaLaunchKernelEx(&cfg, quant_blocks_kernel<XT, VEC>, args);
    }
    return e != cudaSuccess ? e : cudaPeekAtLastError();
}

}  // namespace

cudaError_t run_fp8_quantize(const Fp8Quant &q, cudaStream_t stream, CallInfo *info) {
    QuantArgs a = {};
    a.X = q.X;
    a.ldx = q.ldx;
    a.Q = static_cast<uint8_t *>(q.Q);
    a.ldq = q.ldq;
    a.S = q.S;
    a.lds = q.lds;
    a.rows = q.rows;
    a.cols = q.cols;
    a.e5m2 = q.q_type == kTypeE5M2;
    const int xb = q.x_type == kOutF32 ? 4 : 2;
    const bool vec = (reinterpret_cast<uintptr_t>(q.X) & 15u) == 0 && (q.rows == 1 || (q.ldx * xb) % 16 == 0);
    const uintptr_t qa = q.layout == 1 ? 3u : 7u;
    const int q_rows = q.layout == 1 ? q.cols : q.rows;
    a.err = watchdog_word();
    if (kDebugBuild) {
        const long long q_cols = q.layout == 1 ? q.rows : q.cols, kb = (q_cols + kScaleBlock - 1) / kScaleBlock;
        a.q_extent = static_cast<size_t>((q_rows - 1LL) * q.ldq + q_cols);
        a.s_extent = static_cast<size_t>(q.layout == 2 ? ((q_rows + kScaleBlock - 1LL) / kScaleBlock - 1) * q.lds + kb : (kb - 1) * q.lds + q_rows);
        a.q_extent -= std::min(a.q_extent, debug_shrink_c());
    }
    a.q_vec = (reinterpret_cast<uintptr_t>(q.Q) & qa) == 0 && (q_rows == 1 || (q.ldq & static_cast<long long>(qa)) == 0);
    switch (q.x_type * 2 + (vec ? 1 : 0)) {
        case 0: return launch_quant<kOutF32, false>(a, q.layout, stream, info);
        case 1: return launch_quant<kOutF32, true>(a, q.layout, stream, info);
        case 2: return launch_quant<kOutF16, false>(a, q.layout, stream, info);
        case 3: return launch_quant<kOutF16, true>(a, q.layout, stream, info);
        case 4: return launch_quant<kOutBF16, false>(a, q.layout, stream, info);
        default: return launch_quant<kOutBF16, true>(a, q.layout, stream, info);
    }
}

}  // namespace gemm11

// rows8.cuh -- eight neighbouring elements of a row of FP32, FP16 or BF16, as
// the kernels that pass once over rows hold them.
#pragma once

#include "ptx.cuh"

namespace gemm11 {

template <int XT>
struct Elem8;
template <>
struct Elem8<kOutF32> {
    using T = float;
};
template <>
struct Elem8<kOutF16> {
    using T = __half;
};
template <>
struct Elem8<kOutBF16> {
    using T = __nv_bfloat16;
};

// The elements as they are in memory: 16-bit types take half the registers that
// their FP32 values would.  VEC: x starts on a 16-byte boundary; `left` is the
// number of elements from x to the end of the row.
template <int XT>
struct Row8 {
    using T = typename Elem8<XT>::T;
    static constexpr int kWords = XT == kOutF32 ? 2 : 1;
    uint4 w[kWords];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = make_uint4(0, 0, 0, 0);
    }
    template <bool VEC>
    __device__ __forceinline__ void load(const void *base, long long at, int left) {
        const T *x = static_cast<const T *>(base) + at;
        if (VEC && left >= 8) {
#pragma unroll
            for (int i = 0; i < kWords; ++i) w[i] = __ldg(reinterpret_cast<const uint4 *>(x) + i);
        } else {
            clear();
            T *e = reinterpret_cast<T *>(w);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < left) e[i] = x[i];
        }
    }
    __device__ __forceinline__ void widen(float (&v)[8]) const {
        if constexpr (XT == kOutF32) {
            v[0] = __uint_as_float(w[0].x), v[1] = __uint_as_float(w[0].y), v[2] = __uint_as_float(w[0].z), v[3] = __uint_as_float(w[0].w);
            v[4] = __uint_as_float(w[1].x), v[5] = __uint_as_float(w[1].y), v[6] = __uint_as_float(w[1].z), v[7] = __uint_as_float(w[1].w);
        } else {
            unpack8_out16(w[0], XT, v);
        }
    }
    // Rounded once, to nearest even.
    __device__ __forceinline__ void round(const float (&v)[8]) {
        if constexpr (XT == kOutF32) {
            w[0] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
            w[1] = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
        } else {
            w[0] = make_uint4(pack2_out16(v[0], v[1], XT), pack2_out16(v[2], v[3], XT), pack2_out16(v[4], v[5], XT), pack2_out16(v[6], v[7], XT));
        }
    }
    template <bool VEC>
    __device__ __forceinline__ void store(void *base, long long at, int left) const {
        T *x = static_cast<T *>(base) + at;
        if (VEC && left >= 8) {
#pragma unroll
            for (int i = 0; i < kWords; ++i) reinterpret_cast<uint4 *>(x)[i] = w[i];
        } else {
            const T *e = reinterpret_cast<const T *>(w);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < left) x[i] = e[i];
        }
    }
};

// Rows of elements of `bytes` bytes that start on 16-byte boundaries.
inline bool rows_aligned(const void *p, long long ld, int bytes, long long rows) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (rows <= 1 || ld * bytes % 16 == 0);
}

}  // namespace gemm11

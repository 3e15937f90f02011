// fp8.cuh -- device helpers of the 8-bit block-scaled product: the
// tcgen05.mma of kind::f8f6f4 (e4m3 / e5m2 operands, FP32 accumulator).
#pragma once

#include "ptx.cuh"

namespace gemm11 {

// mbar_wait whose tries may suspend the warp for up to a millisecond (the
// barrier wakes it), and which reads the clock only where the first tries
// fail.  A warp that polls takes issue slots from the others of its scheduler:
// beside the MMA warp's polling two of the product's eight epilogue warps ran
// 400 cycles a block late.
__device__ __forceinline__ bool mbar_try_wait_long(uint32_t bar_addr, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n"
        " .reg .pred p;\n"
        " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
        " selp.u32 %0, 1, 0, p;\n"
        "}\n"
        : "=r"(ok)
        : "r"(bar_addr), "r"(parity), "r"(1000000u)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool mbar_test_wait(uint32_t bar_addr, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n"
        " .reg .pred p;\n"
        " mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n"
        "}\n"
        : "=r"(ok)
        : "r"(bar_addr), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool mbar_wait_patient(uint64_t *bar, uint32_t parity, unsigned long long limit_ns = kWaitLimitNs) {
    const uint32_t a = smem_u32(bar);
    if (mbar_test_wait(a, parity)) return true;
    for (int i = 0; i < 4; ++i)
        if (mbar_try_wait_long(a, parity)) return true;
    const unsigned long long t0 = globaltimer_ns();
    for (;;) {
        if (mbar_try_wait_long(a, parity)) return true;
        if (globaltimer_ns() - t0 > limit_ns) return false;
    }
}

// 16 or 32 columns of a warp's 32 tensor-memory lanes.
template <int COLS>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[COLS]) {
    static_assert(COLS == 16 || COLS == 32, "columns");
    if constexpr (COLS == 32)
        tmem_ld_32x32b_x32(taddr, r);
    else
        tmem_ld_32x32b_x16(taddr, r);
}

// Two FP32 values in one 64-bit register, and acc = a * b + acc, a * b on both
// (PTX f32x2; one rounding each, as fmaf).  Held as 64-bit values so that the
// pairs stay in place.
__device__ __forceinline__ uint64_t pack_f32x2(float lo, float hi) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
    return v;
}
__device__ __forceinline__ uint64_t pack_b32x2(uint32_t lo, uint32_t hi) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(lo), "r"(hi));
    return v;
}
__device__ __forceinline__ void unpack_f32x2(uint64_t v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ void fma_f32x2(uint64_t &acc, uint64_t a, uint64_t b) {
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(a), "l"(b));
}
// acc = (a * f) * (lo, hi) + acc, in order (volatile), so that the products do
// not pile up in registers.
__device__ __forceinline__ void fma_scaled_f32x2(uint64_t &acc, uint64_t a, uint64_t f, uint32_t lo, uint32_t hi) {
    asm volatile(
        "{\n"
        " .reg .b64 d, t;\n"
        " mov.b64 d, {%3, %4};\n"
        " mul.rn.f32x2 t, %1, %2;\n"
        " fma.rn.f32x2 %0, t, d, %0;\n"
        "}\n"
        : "+l"(acc)
        : "l"(a), "l"(f), "r"(lo), "r"(hi));
}
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
    uint64_t v;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
    return v;
}

// True in one lane of a warp that runs together.  A warp whose loop is uniform
// and only guards its tcgen05 and TMA instructions with this keeps their
// operands (descriptors, addresses) in uniform registers; a loop inside a
// one-lane branch moves them there for every instruction, which took 125
// cycles an MMA, as long as the MMA itself.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n"
        " .reg .pred p;\n"
        " elect.sync _|p, 0xffffffff;\n"
        " selp.u32 %0, 1, 0, p;\n"
        "}\n"
        : "=r"(p));
    return p != 0;
}

// Arrive on an mbarrier of another CTA of the cluster, releasing at CTA scope:
// for a consumer's "I have read it" whose reads have completed (their values
// were used).  The cluster-scope release of mbar_arrive_cluster waits for every
// earlier memory operation of the thread: 1,500 cycles in the product's loop.
__device__ __forceinline__ void mbar_arrive_remote(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// D(tmem) (+)= A(smem desc) x B(smem desc), 8-bit operands, K = 32 per
// instruction (32 bytes of each K-major row).
__device__ __forceinline__ void umma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                        uint32_t accumulate) {
    asm volatile(
        "{\n"
        " .reg .pred p;\n"
        " setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n"
        "}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// The pair form: issued by one thread of the even CTA, as umma_f16_pair.
__device__ __forceinline__ void umma_f8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
    asm volatile(
        "{\n"
        " .reg .pred p;\n"
        " setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n"
        "}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Instruction descriptor for kind::f8f6f4: operand formats E4M3 = 0, E5M2 = 1
// (they may differ), FP32 accumulator, a_mn / b_mn = operand stored MN-major.
constexpr uint32_t umma_idesc_f8(int M, int N, int a_e5m2, int b_e5m2, int a_mn, int b_mn) {
    return (1u << 4)                                     // D format: F32
           | (static_cast<uint32_t>(a_e5m2) << 7)        // A format
           | (static_cast<uint32_t>(b_e5m2) << 10)       // B format
           | (static_cast<uint32_t>(a_mn) << 15)         // A major
           | (static_cast<uint32_t>(b_mn) << 16)         // B major
           | (static_cast<uint32_t>(N >> 3) << 17)       // N >> 3
           | (static_cast<uint32_t>(M >> 4) << 24);      // M >> 4
}

// act(alpha * v + beta * cold + b) for four values, the activation's branch
// taken once for all four so that their chains interleave.
__device__ __forceinline__ void epilogue4(float (&v)[4], float alpha, float beta, const float (&cold)[4],
                                          const float (&b)[4], int act) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] *= alpha;
        if (beta != 0.f) v[i] = fmaf(beta, cold[i], v[i]);
        v[i] += b[i];
    }
    if (act == 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = gelu_erf(v[i]);
    } else if (act == 3) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = gelu_tanh(v[i]);
    } else if (act == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = fmaxf(v[i], 0.f);
    }
}

}  // namespace gemm11

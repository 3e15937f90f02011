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

// A read that is in flight where a loop comes round.  The compiler may copy a
// variable there, which would read it before it has landed; registers that only
// PTX knows it cannot.  A kernel declares them once, before their first use.
#define GEMM11_TMEM_AHEAD_REGISTERS() asm volatile(".reg .b32 ahead<32>;")
template <int COLS>
__device__ __forceinline__ void tmem_ld_ahead(uint32_t taddr) {
    static_assert(COLS == 16 || COLS == 32, "columns");
    if constexpr (COLS == 32)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {ahead0, ahead1, ahead2, ahead3, ahead4, ahead5, ahead6, ahead7, ahead8, ahead9, ahead10, ahead11, ahead12, ahead13, ahead14, ahead15, "
                     "ahead16, ahead17, ahead18, ahead19, ahead20, ahead21, ahead22, ahead23, ahead24, ahead25, ahead26, ahead27, ahead28, ahead29, ahead30, ahead31}, [%0];" ::"r"(taddr) : "memory");
    else
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {ahead0, ahead1, ahead2, ahead3, ahead4, ahead5, ahead6, ahead7, ahead8, ahead9, ahead10, ahead11, ahead12, ahead13, ahead14, ahead15}, [%0];" ::"r"(taddr) : "memory");
}
// Wait for it, and for this thread's other reads.
template <int COLS>
__device__ __forceinline__ void tmem_wait_ahead(uint32_t (&r)[COLS]) {
    tmem_wait_ld();
    if constexpr (COLS == 32)
        asm volatile(
            "mov.b32 %0, ahead0; mov.b32 %1, ahead1; mov.b32 %2, ahead2; mov.b32 %3, ahead3; mov.b32 %4, ahead4; mov.b32 %5, ahead5; mov.b32 %6, ahead6; mov.b32 %7, ahead7;"
            "mov.b32 %8, ahead8; mov.b32 %9, ahead9; mov.b32 %10, ahead10; mov.b32 %11, ahead11; mov.b32 %12, ahead12; mov.b32 %13, ahead13; mov.b32 %14, ahead14; mov.b32 %15, ahead15;"
            "mov.b32 %16, ahead16; mov.b32 %17, ahead17; mov.b32 %18, ahead18; mov.b32 %19, ahead19; mov.b32 %20, ahead20; mov.b32 %21, ahead21; mov.b32 %22, ahead22; mov.b32 %23, ahead23;"
            "mov.b32 %24, ahead24; mov.b32 %25, ahead25; mov.b32 %26, ahead26; mov.b32 %27, ahead27; mov.b32 %28, ahead28; mov.b32 %29, ahead29; mov.b32 %30, ahead30; mov.b32 %31, ahead31;"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
              "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
              "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
              "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]));
    else
        asm volatile(
            "mov.b32 %0, ahead0; mov.b32 %1, ahead1; mov.b32 %2, ahead2; mov.b32 %3, ahead3; mov.b32 %4, ahead4; mov.b32 %5, ahead5; mov.b32 %6, ahead6; mov.b32 %7, ahead7;"
            "mov.b32 %8, ahead8; mov.b32 %9, ahead9; mov.b32 %10, ahead10; mov.b32 %11, ahead11; mov.b32 %12, ahead12; mov.b32 %13, ahead13; mov.b32 %14, ahead14; mov.b32 %15, ahead15;"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
              "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]));
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

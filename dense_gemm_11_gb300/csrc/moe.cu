// moe.cu -- a whole mixture-of-experts layer for a few tokens in one kernel:
//
//   logits = X Wr^T,  p = softmax(logits),  the top_k experts e_1.. of a token
//   (ties: the lower index),  w_j = p[e_j]  or  p[e_j] / sum_j p[e_j],
//   h_j = act(Wgate[e_j] x) * (Wup[e_j] x)      (or act(Wgate[e_j] x)),
//   y   = sum_j w_j Wdown[e_j] h_j.
//
// Bound: memory.  With a few tokens the matrices of the chosen experts are
// read once and used for one to a few products each, so the layer takes as
// long as those bytes do.  The kernel is persistent (one CTA per SM, launched
// cooperatively) and built as one stream of weight bytes:
//   * work is cut into units of 16 WR matrix rows (gate rows with the up rows
//     they meet, or rows of the down projection) for one expert and up to 8 NT
//     of its tokens.  A unit goes through its k in stages of 32 KB of weights:
//     16 WR rows x 16 / WR boxes of 128 bytes, one TMA copy (two with a gate).
//     Issuing a copy costs the producer about 100 cycles, so stages are large:
//     with 16 KB it, not memory, set the pace (130 us against 116 at 1 token, 8
//     experts of 4096 x 11008, 2 each)
//   * one warp fills a ring of stages with weights.  It runs ahead of the
//     arithmetic across units, and into the down projection while other CTAs
//     still finish the first half.  One or two more bring the tokens' rows of
//     the same k, a copy each (by the weights' warp, 6 of them a stage held the
//     weights back: 138 us against 134 at 64 tokens, 64 experts);
//   * sixteen warps take a stage's WR row groups x 16 / WR boxes, one each, and
//     multiply their 16 rows x 128 bytes by the tokens with mma.sync; warps that
//     share rows add their sums in warp order in shared memory at the unit's
//     end.  The matrix instruction is the warp-level one: a unit has 1 to 8 NT
//     columns of a 128-column tcgen05 tile and is bound by memory, and
//     fragments come straight from the row-major rows (the k of a fragment may
//     be any permutation that both operands share, so that a thread's k's are
//     neighbours, one 16-byte load).
// Few row groups (WR = 1) make many small units, which spread evenly over the
// SMs; many (WR = 16) read a token's activations once for 256 rows and leave no
// sums to add and no warp to wait for.  The host takes the largest WR whose
// units still spread well.
// Between the phases (router, first half, down projection, sum over a token's
// experts) CTAs meet at grid barriers; every sum has a fixed order, so results
// do not depend on timing.  Every wait is bounded.
//
// Numbers.  Every product is a 16-bit x 16-bit mma.sync with FP32 sums; what
// the activations are held in depends on the types:
//   BF16 weights   X as it is; h as the sum of three BF16 numbers, all of its
//                  FP32 bits, three products each;
//   FP16 weights   X as it is; h as the sum of two FP16 numbers (22 bits);
//   e4m3 weights   widened to FP16 (exact), one conversion for two elements
//                  (TF32 products took two more each, and twice the matrix
//                  instructions: 165 us against 149 at 16 tokens, 32 experts).
//                  h as with FP16 weights.  An FP16 X as it is; a BF16 X in FP16
//                  after scaling a token by the power of two that brings its
//                  largest element to [2^14, 2^15) (its 8 bits are exact down to
//                  2^-31 of that).
// h in one 16-bit number would leave an FP32 Y with 11 or 8 bits, and a BF16 Y
// with last bits that differ from those of FP32 sums in a tenth of its elements.
// Where h is held in FP16 it is written in FP32 too.  If some slot's largest
// |h| turns out to be outside [2^-4, 65504] (inside, what two numbers drop is
// 2^-21 of the largest at most), all are fitted as a BF16 X is, between two grid barriers
// (3 us), else nothing is.  The e4m3 scale of a 128 x 128 block multiplies that
// block's FP32 sum.
#include <algorithm>
#include <cstdint>

#include <cmath>

#include <cuda_fp8.h>

#include "fp8.cuh"
#include "fp8.h"

namespace gemm11 {
namespace {

constexpr int kStageWeights = 32768;            // bytes of weights in a stage
constexpr int kWarps = 16;                      // that multiply
constexpr int kBoxes = kWarps;                  // of 16 rows x 128 bytes in a stage, one for each of them
constexpr int kMaxStages = 12;
constexpr int kMaxSplits = 4;                   // units that share a row group's k in the down projection
constexpr int kTokensOfTheirOwn = 32;           // from so many on a CTA routes a token by itself

struct MoeArgs {
    int T, E, top_k, H, I;
    const void *X;
    long long ldx;
    const void *router;
    int router_f32;
    const void *gate, *up, *down;
    const float *s_gate, *s_up, *s_down;
    void *Y;
    long long ldy;
    int y_type, act, renorm;
    int *ids;
    float *weights;
    // Scratch: T x E logits; h in FP32 (slots x I) and as 16-bit numbers, two or
    // three, these in runs of 64 by turns; X in FP16, scaled; the largest |h| of
    // a slot, and the scale of a token; k_splits x slots x H partial results.
    float *logits, *hidden, *part;
    uint8_t *hidden16;
    __half *x16;
    unsigned *h_max;
    float *x_scale;
    uint16_t *chosen;  // T x top_k, and their weights
    float *chosen_weight;
    unsigned *counters;  // four barriers and the exit
    unsigned *err;
    int lw1, lw2;    // log2 of WR, the row groups (of 16 rows) of a unit, in the first half and in the down projection
    int k_splits;    // units of the down projection that share a row group's k
    int by_token;    // the routing takes a CTA for each token
    int flat_h, flat_i;  // elements of a row up to which one copy takes a stage's boxes (whole 128-byte ones)
    int stages, stage_bytes;
    // Elements (hidden16: bytes) of each part of the scratch, and of Y, checked by GEMM11_DEBUG builds.
    size_t n_logits, n_hidden, n_hidden16, n_x16, n_part, n_y;
};

// Whether element `at` of a buffer of n may be accessed.
__device__ __forceinline__ bool inside(long long at, size_t n, const MoeArgs &p) {
    return debug_in_bounds(at >= 0 && static_cast<size_t>(at) < n, p.err);
}

// Shared-memory tables of the routing, the same in every CTA.
struct Routing {
    float weight[kMoeMaxSlots];
    float x_scale[kMoeMaxTokens];   // what a token's sums are multiplied by
    uint16_t expert[kMoeMaxSlots];  // of slot t * top_k + j
    uint16_t order[kMoeMaxSlots];   // slots, grouped by expert, ascending
    uint16_t pair_expert[kMoeMaxSlots], pair_first[kMoeMaxSlots], pair_start[kMoeMaxSlots];
    uint8_t pair_groups[kMoeMaxSlots], pair_count[kMoeMaxSlots];
    int offset[kMoeMaxExperts + 1];
    int pairs;
    uint32_t per_token;  // 65536 / top_k, rounded up
    // Token of a slot: slot / top_k, exact for slots < 1024 and top_k <= 16.
    __device__ __forceinline__ int token(int slot) const { return static_cast<int>(slot * per_token >> 16); }
};

template <int XT>
__device__ __forceinline__ void mma_16bit(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
    if constexpr (XT == kOutBF16)
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Contiguous bytes, a multiple of 16 at 16-byte aligned addresses.
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}
// Arrive on `bar` when this thread's cp.async copies so far are complete.
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }
__device__ __forceinline__ void consumer_sync() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory"); }
__device__ __forceinline__ unsigned load_acquire(const unsigned *p) {
    unsigned v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
// Wait (bounded) until `*c` has reached `want`.
__device__ __forceinline__ bool wait_count(const unsigned *c, unsigned want) {
    if (load_acquire(c) >= want) return true;
    const unsigned long long t0 = globaltimer_ns();
    for (uint32_t it = 1;; ++it) {
        if (load_acquire(c) >= want) return true;
        if ((it & 63u) == 0u && globaltimer_ns() - t0 > kWaitLimitNs) return false;
    }
}

// SiLU by the approximate exponential and reciprocal: each is within 2^-22 of
// its value, and v log2(e) is rounded to FP32 before, so the result is within
// (4 + |v| / 2) 2^-23 of its value, below what the FP32 sums v comes from err by.
__device__ __forceinline__ float moe_act(int act, float v) {
    return act == kActSilu ? v * rcp_approx(1.f + __expf(-v)) : apply_activation(act, v);
}

// Eight neighbouring values of a row as floats.
__device__ __forceinline__ void widen8(const uint4 &w, int type, float (&v)[8]) { unpack8_out16(w, type, v); }
// Four e4m3 values of a word as two FP16 pairs.
__device__ __forceinline__ void widen_e4m3(uint32_t w, uint32_t &lo, uint32_t &hi) {
    const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w & 0xFFFFu), __NV_E4M3);
    const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> 16), __NV_E4M3);
    lo = *reinterpret_cast<const uint32_t *>(&a);
    hi = *reinterpret_cast<const uint32_t *>(&b);
}
// Four 8 x 16-byte matrices, whose rows' addresses the lanes give in turn:
// word i of thread (g, t) is bytes [4 t, 4 t + 4) of row g of matrix i.
__device__ __forceinline__ void load_matrices(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// h as a sum of N 16-bit numbers, each the rest of the one before it.  One that
// overflows to infinity leaves no rest.
template <int TYPE, int N>
__device__ __forceinline__ void split_parts(float h, uint16_t (&part)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float back;
        if constexpr (TYPE == kOutF16) {
            const __half a = __float2half_rn(h);
            part[i] = __half_as_ushort(a);
            back = __half2float(a);
        } else {
            const __nv_bfloat16 a = __float2bfloat16_rn(h);
            part[i] = __bfloat16_as_ushort(a);
            back = __bfloat162float(a);
        }
        h = fabsf(back) < INFINITY ? h - back : 0.f;
    }
}
// 2^e that brings a largest magnitude into [2^14, 2^15), and 2^-e.  Normal
// numbers both (a maximum below 2^-112 stays smaller); 1 for zero.
__device__ __forceinline__ int fit_exponent(float largest) {
    const int field = static_cast<int>(__float_as_uint(largest) >> 23) & 0xFF;
    return largest == 0.f ? 0 : min(126, 14 + 127 - field);
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<unsigned>(127 + e) << 23); }

// ---------------------------------------------------------------- routing
constexpr int kRouterTokens = 4;  // of one unit

// Sum of w x over `threads` threads' share of H for one expert and 4 tokens,
// two steps' loads in flight.
template <int XT>
__device__ __forceinline__ void router_dot(const MoeArgs &p, int e, int t0, int thread, int threads, float (&acc)[kRouterTokens]) {
#pragma unroll
    for (int i = 0; i < kRouterTokens; ++i) acc[i] = 0.f;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    const int step = threads * 8;
    for (int k0 = thread * 8; k0 < p.H; k0 += 2 * step) {
        uint4 x[2][kRouterTokens], w16[2];
        float w[2][8];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int k = k0 + u * step;
            const bool in = k < p.H;
            const long long at = static_cast<long long>(e) * p.H + k;
            if (p.router_f32) {
                const float4 *r = reinterpret_cast<const float4 *>(static_cast<const float *>(p.router) + at);
                const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
                const float4 a = in ? __ldg(r) : z, b = in ? __ldg(r + 1) : z;
                w[u][0] = a.x, w[u][1] = a.y, w[u][2] = a.z, w[u][3] = a.w, w[u][4] = b.x, w[u][5] = b.y, w[u][6] = b.z, w[u][7] = b.w;
            } else {
                w16[u] = in ? __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.router) + at)) : zero;
            }
#pragma unroll
            for (int i = 0; i < kRouterTokens; ++i)
                x[u][i] = in && t0 + i < p.T
                              ? __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.X) + (t0 + i) * p.ldx + k))
                              : zero;
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            if (!p.router_f32) widen8(w16[u], XT, w[u]);
#pragma unroll
            for (int i = 0; i < kRouterTokens; ++i) {
                float f[8];
                widen8(x[u][i], XT, f);
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[i] = fmaf(w[u][j], f[j], acc[i]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kRouterTokens; ++i)
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], d);
}

// All logits, in units of one expert and 4 tokens: a CTA takes a unit while
// there are no more units than CTAs (its warps share H), else each warp does.
template <int XT>
__device__ void router_logits(const MoeArgs &p, float *red) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int groups = (p.T + kRouterTokens - 1) / kRouterTokens, units = p.E * groups;
    float acc[kRouterTokens];
    if (units > static_cast<int>(gridDim.x)) {
        for (int u = warp * gridDim.x + blockIdx.x; u < units; u += gridDim.x * kWarps) {
            const int e = u / groups, t0 = (u % groups) * kRouterTokens;
            router_dot<XT>(p, e, t0, lane, 32, acc);
#pragma unroll
            for (int i = 0; i < kRouterTokens; ++i)
                if (lane == i && t0 + i < p.T && inside((t0 + i) * p.E + e, p.n_logits, p)) p.logits[(t0 + i) * p.E + e] = acc[i];
        }
    } else if (static_cast<int>(blockIdx.x) < units) {
        const int e = blockIdx.x / groups, t0 = (blockIdx.x % groups) * kRouterTokens;
        router_dot<XT>(p, e, t0, threadIdx.x, 32 * kWarps, acc);
#pragma unroll
        for (int i = 0; i < kRouterTokens; ++i)
            if (lane == i) red[warp * kRouterTokens + i] = acc[i];
        consumer_sync();
        if (threadIdx.x < kRouterTokens && t0 + threadIdx.x < p.T) {
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) v += red[w * kRouterTokens + threadIdx.x];
            if (inside((t0 + threadIdx.x) * p.E + e, p.n_logits, p)) p.logits[(t0 + threadIdx.x) * p.E + e] = v;
        }
    }
}

// Order-preserving key of a logit: -0 equals +0, NaN comes first; 0 is below
// every key.
__device__ __forceinline__ uint32_t logit_key(float v) {
    if (v != v) return 0xFFFFFFFFu;
    const uint32_t b = __float_as_uint(v + 0.f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ float key_logit(uint32_t k) { return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k); }

// The keys of one token's logits, by a whole CTA: a warp takes 4 experts at a
// time, with the token in shared memory (xs) and the experts' rows of 4 steps
// (2 of FP32) in flight.
template <int XT>
__device__ void router_token(const MoeArgs &p, int t, uint32_t *keys, uint4 *xs) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint4 *x = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.X) + t * p.ldx);
    for (int k = threadIdx.x; k < p.H / 8; k += 32 * kWarps) xs[k] = __ldg(x + k);
    consumer_sync();
    for (int e0 = warp * 4; e0 < p.E; e0 += kWarps * 4) {
        float acc[4] = {};
        auto rows = [&](auto wide) {  // wide: an FP32 router, 16 bytes are 4 elements
            constexpr bool kWide = decltype(wide)::value;
            constexpr int kDeep = kWide ? 2 : 4, kParts = kWide ? 2 : 1;
            for (int k0 = lane; k0 < p.H / 8; k0 += 32 * kDeep) {
                uint4 w[kDeep][4][kParts];
#pragma unroll
                for (int u = 0; u < kDeep; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int k = min(k0 + 32 * u, p.H / 8 - 1), e = min(e0 + i, p.E - 1);
                        const uint4 *r = static_cast<const uint4 *>(p.router) + (static_cast<long long>(e) * (p.H / 8) + k) * kParts;
#pragma unroll
                        for (int h = 0; h < kParts; ++h) w[u][i][h] = __ldg(r + h);
                    }
#pragma unroll
                for (int u = 0; u < kDeep; ++u) {
                    if (k0 + 32 * u >= p.H / 8) break;
                    float f[8];
                    widen8(xs[k0 + 32 * u], XT, f);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float v[8];
                        if constexpr (kWide) {
                            const uint4 a = w[u][i][0], b = w[u][i][kParts - 1];
                            v[0] = __uint_as_float(a.x), v[1] = __uint_as_float(a.y), v[2] = __uint_as_float(a.z), v[3] = __uint_as_float(a.w);
                            v[4] = __uint_as_float(b.x), v[5] = __uint_as_float(b.y), v[6] = __uint_as_float(b.z), v[7] = __uint_as_float(b.w);
                        } else {
                            widen8(w[u][i][0], XT, v);
                        }
#pragma unroll
                        for (int j = 0; j < 8; ++j) acc[i] = fmaf(v[j], f[j], acc[i]);
                    }
                }
            }
        };
        if (p.router_f32)
            rows(std::true_type{});
        else
            rows(std::false_type{});
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int d = 16; d >= 1; d >>= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], d);
            if (lane == i && e0 + i < p.E) keys[e0 + i] = logit_key(acc[i]);
        }
    }
}

// One token's X in FP16, scaled, by a whole CTA.
template <int XT>
__device__ void scale_token(const MoeArgs &p, int t, float *red) {
    const uint16_t *x = static_cast<const uint16_t *>(p.X) + t * p.ldx;
    float m = 0.f;
    for (int k = threadIdx.x * 8; k < p.H; k += 32 * kWarps * 8) {
        float v[8];
        widen8(__ldg(reinterpret_cast<const uint4 *>(x + k)), XT, v);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (fabsf(v[i]) < INFINITY) m = fmaxf(m, fabsf(v[i]));
    }
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
    consumer_sync();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, red[w]);
    consumer_sync();
    const int e = fit_exponent(m);
    const float f = pow2(e);
    for (int k = threadIdx.x * 8; k < p.H; k += 32 * kWarps * 8) {
        float v[8];
        widen8(__ldg(reinterpret_cast<const uint4 *>(x + k)), XT, v);
        if (!inside(static_cast<long long>(t) * p.H + k + 7, p.n_x16, p)) continue;
        *reinterpret_cast<uint4 *>(p.x16 + static_cast<long long>(t) * p.H + k) =
            make_uint4(pack2_out16(v[0] * f, v[1] * f, kOutF16), pack2_out16(v[2] * f, v[3] * f, kOutF16),
                       pack2_out16(v[4] * f, v[5] * f, kOutF16), pack2_out16(v[6] * f, v[7] * f, kOutF16));
    }
    if (threadIdx.x == 0) p.x_scale[t] = pow2(-e);
}

// One warp, one token: softmax and its top_k largest, by repeated maximum over
// the logits' keys (shared memory; taken ones are set to 0).  Lane j keeps the
// j-th choice.
__device__ void choose_experts(const MoeArgs &p, uint32_t *keys, uint16_t *experts, float *weights) {
    const int lane = threadIdx.x & 31;
    uint32_t mine = 0, first = 0;
    int my_expert = 0;
    float sum = 0.f;
    for (int j = 0; j < p.top_k; ++j) {
        uint32_t best = 0;
        int at = 0;
#pragma unroll 2
        for (int e = lane; e < p.E; e += 32) {
            const uint32_t k = keys[e];
            if (k > best) best = k, at = e;
        }
        const uint32_t m = __reduce_max_sync(0xffffffffu, best);
        const int e = static_cast<int>(__reduce_min_sync(0xffffffffu, best == m ? static_cast<unsigned>(at) : 0xFFFFFFFFu));
        if (j == 0) {
            first = m;
            if (!p.renorm)
                for (int i = lane; i < p.E; i += 32) sum += expf(key_logit(keys[i]) - key_logit(m));
        }
        if (lane == j) mine = m, my_expert = e;
        if (lane == (e & 31)) keys[e] = 0;
    }
    const float v = lane < p.top_k ? expf(key_logit(mine) - key_logit(first)) : 0.f;
    if (p.renorm) sum = v;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (lane < p.top_k) {
        weights[lane] = v / sum;
        experts[lane] = static_cast<uint16_t>(my_expert);
    }
}

// Slots grouped by expert, in ascending order, and the (expert, token group)
// pairs that the units go over.  A token has an expert once at most, so an
// expert's slots are a mask over the tokens (4 words each, in `mask`), and a
// slot's place among them the bits below its own.
__device__ void group_slots(const MoeArgs &p, Routing &r, uint32_t *mask, int group) {
    static_assert(kMoeMaxTokens == 128, "four words of a mask");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, slots = p.T * p.top_k;
    for (int i = threadIdx.x; i < p.E * 4; i += 32 * kWarps) mask[i] = 0;
    consumer_sync();
    for (int s = threadIdx.x; s < slots; s += 32 * kWarps) {
        const int t = s / p.top_k;
        atomicOr(&mask[r.expert[s] * 4 + (t >> 5)], 1u << (t & 31));
    }
    consumer_sync();
    if (warp == 0) {
        int before = 0, pairs_before = 0;
        for (int e0 = 0; e0 < p.E; e0 += 32) {
            const int e = e0 + lane;
            int n = 0;
            if (e < p.E) {
                const uint4 m = *reinterpret_cast<const uint4 *>(mask + e * 4);
                n = __popc(m.x) + __popc(m.y) + __popc(m.z) + __popc(m.w);
            }
            const int np = (n + group - 1) / group;
            int sum = n | (np << 16);  // both sums at once
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int a = __shfl_up_sync(0xffffffffu, sum, d);
                if (lane >= d) sum += a;
            }
            if (e < p.E) {
                const int first = pairs_before + (sum >> 16) - np, start = before + (sum & 0xFFFF) - n;
                r.offset[e] = start;
                for (int i = 0; i < np; ++i) {
                    r.pair_expert[first + i] = static_cast<uint16_t>(e);
                    r.pair_first[first + i] = static_cast<uint16_t>(first);
                    r.pair_groups[first + i] = static_cast<uint8_t>(np);
                    r.pair_start[first + i] = static_cast<uint16_t>(start + i * group);
                    r.pair_count[first + i] = static_cast<uint8_t>(min(group, n - i * group));
                }
            }
            const int all = __shfl_sync(0xffffffffu, sum, 31);
            before += all & 0xFFFF;
            pairs_before += all >> 16;
        }
        if (lane == 0) r.pairs = pairs_before;
    }
    consumer_sync();
    for (int s = threadIdx.x; s < slots; s += 32 * kWarps) {
        const int e = r.expert[s], t = s / p.top_k;
        int rank = __popc(mask[e * 4 + (t >> 5)] & ((1u << (t & 31)) - 1u));
        for (int i = 0; i < (t >> 5); ++i) rank += __popc(mask[e * 4 + i]);
        r.order[r.offset[e] + rank] = static_cast<uint16_t>(s);
    }
}

// Whether every slot's largest |h| is inside FP16's comfortable range.  Each
// warp looks for itself (after the first half's barrier).
__device__ __forceinline__ bool slots_fit(const MoeArgs &p) {
    bool fits = true;
    for (int i = threadIdx.x & 31; i < p.T * p.top_k; i += 32) {
        const float m = __uint_as_float(__ldcg(p.h_max + i));
        fits = fits && (m == 0.f || (m >= 0.0625f && m <= 65504.f));
    }
    return __all_sync(0xffffffffu, fits);
}

// ---------------------------------------------------------------- units
// Bytes of a slot's h as `parts` 16-bit numbers an element.
__host__ __device__ constexpr long long parts_bytes(int I, int parts) { return (I + 63ll) / 64 * 128 * parts; }

struct Unit {
    int expert, row, start, count;  // first matrix row (of the expert), first slot in `order`, tokens
    int ch0, ch1, split;            // stages
};
// Unit u of the first half: the token groups of an expert next to each other
// for the same rows, so that they share the rows' bytes in L2.
__device__ __forceinline__ Unit first_unit(const Routing &r, int u, int row_groups, int rows, int stages) {
    Unit n;
    const int p0 = u / row_groups, first = r.pair_first[p0], groups = r.pair_groups[p0];
    const int i = u - first * row_groups;
    const int pair = first + i % groups;
    n.row = i / groups * rows;
    n.expert = r.pair_expert[pair];
    n.start = r.pair_start[pair];
    n.count = r.pair_count[pair];
    n.ch0 = 0;
    n.ch1 = stages;
    n.split = 0;
    return n;
}
// Unit u of the down projection: row group by row group.
__device__ __forceinline__ Unit down_unit(const Routing &r, int u, int rows, int stages, int splits) {
    Unit n;
    n.split = u % splits;
    u /= splits;
    const int pair = u % r.pairs;
    n.row = u / r.pairs * rows;
    n.expert = r.pair_expert[pair];
    n.start = r.pair_start[pair];
    n.count = r.pair_count[pair];
    n.ch0 = stages * n.split / splits;
    n.ch1 = stages * (n.split + 1) / splits;
    return n;
}

template <int XT, bool FP8>
struct MoeCfg {
    static constexpr int kWBytes = FP8 ? 1 : 2;
    static constexpr int kBoxK = 128 / kWBytes;  // k of a box: 128 (one scale block) or 64
    static constexpr bool kFit = FP8 || XT == kOutF16;         // h in FP16
    static constexpr int kParts = kFit ? 2 : 3;                // numbers that h is the sum of
    static constexpr bool kScaledX = FP8 && XT == kOutBF16;    // X as scaled FP16
    static constexpr int kMma = FP8 ? kOutF16 : XT;
    static constexpr int kXBytes = 2, kHBytes = 2 * kParts;
    static constexpr int kScaleBytes = FP8 ? kBoxes * 2 * 4 : 0;
    static constexpr int kActOffset = kStageWeights + kScaleBytes;
    // Row strides of the activations: the 8 threads of a quarter warp (16 of
    // half a warp with 8-byte loads) fall on different banks.
    static constexpr int kPad = FP8 ? 32 : 16;
    __host__ __device__ static constexpr int act_stride(int lw, bool first) {
        return (kBoxes >> lw) * kBoxK * (first ? kXBytes : kHBytes) + kPad;
    }
};

// This warp's 16 rows x one box of k times the tokens, added to c (a box's own
// sums: the matrix instruction's additions truncate, and 11008 k in one chain
// of them left 7e-6 of the result, boxes added to nearest 4e-7).  Thread
// (g, t) holds rows g and g + 8, token 8 n + g and the same k's of both; w0 and
// w1 are the first of each 8 rows (16-byte chunk c of row g at c ^ g, by the
// copy's swizzle), act[n] its token's k's of this box; USED of the NT groups of
// 8 tokens exist.  PARTS: activations are sums of so many numbers, 64 k's of
// the next one 128 bytes after those of the one before.  TAIL: only `valid` k's exist; the
// weights past them are zeros, the activations are left over from other stages.
template <int XT, bool FP8, int NT, int USED, int PARTS, bool TAIL>
__device__ __forceinline__ void multiply_box(const uint8_t *w0, const uint8_t *w1, const uint8_t *const (&act)[NT], int valid,
                                             float (&c)[NT][4]) {
    using Cfg = MoeCfg<XT, FP8>;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    if constexpr (FP8) {
        // Lanes 0-7 and 8-15 give the two groups' rows of one chunk, 16-31 of the next.
        const uint32_t row = smem_u32((lane & 8) ? w1 : w0) + (lane & 7) * 128;
#pragma unroll
        for (int ch = 0; ch < 8; ch += 2) {
            uint32_t w[4];
            load_matrices(row + (((ch + (lane >> 4)) ^ (lane & 7)) << 4), w);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t a0, a1, a2, a3;
                widen_e4m3(w[2 * h], a0, a2);
                widen_e4m3(w[2 * h + 1], a1, a3);
                const int k = (ch + h) * 16 + t * 4;
                const int at = (ch / 4) * (128 * PARTS) + ((ch + h) % 4 * 16 + t * 4) * 2;
#pragma unroll
                for (int part = 0; part < PARTS; ++part)
#pragma unroll
                    for (int n = 0; n < USED; ++n) {
                        uint2 x = *reinterpret_cast<const uint2 *>(act[n] + at + part * 128);
                        if (TAIL && k >= valid) x = make_uint2(0, 0);
                        mma_16bit<Cfg::kMma>(c[n], a0, a1, a2, a3, x.x, x.y);
                    }
            }
        }
    } else {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int chunk = 2 * t + s;
            const uint4 a = *reinterpret_cast<const uint4 *>(w0 + g * 128 + ((chunk ^ g) << 4));
            const uint4 b = *reinterpret_cast<const uint4 *>(w1 + g * 128 + ((chunk ^ g) << 4));
#pragma unroll
            for (int part = 0; part < PARTS; ++part)
#pragma unroll
                for (int n = 0; n < USED; ++n) {
                    uint4 x = *reinterpret_cast<const uint4 *>(act[n] + part * 128 + chunk * 16);
                    if (TAIL && chunk * 8 >= valid) x = make_uint4(0, 0, 0, 0);
                    mma_16bit<Cfg::kMma>(c[n], a.x, b.x, a.y, b.y, x.x, x.y);
                    mma_16bit<Cfg::kMma>(c[n], a.z, b.z, a.w, b.w, x.z, x.w);
                }
        }
    }
}

// Of each matrix: boxes by the stage, and single boxes for a ragged end.
struct MoeMaps {
    CUtensorMap gate, up, down, gate1, up1, down1;
};

// One token warp brings the 8 tokens of a unit, two 16.  (Units of 32 tokens
// were slower than two of 16 at 13 tokens an expert and more: their registers
// leave room for half the warps.)
constexpr int moe_threads(int nt) { return 32 * (kWarps + 1 + nt); }

template <int XT, bool FP8, int NT>
__global__ void __launch_bounds__(moe_threads(NT), 1)
    moe_kernel(const __grid_constant__ MoeMaps maps, const MoeArgs p) {
    using Cfg = MoeCfg<XT, FP8>;
    static_assert(NT == 1 || NT == 2, "8 or 16 tokens a unit");
    constexpr int kThreads = moe_threads(NT);
    extern __shared__ uint8_t ring_raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(ring_raw) + 1023) & ~uintptr_t(1023));
    __shared__ Routing r;
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages];
    __shared__ float red[2][kWarps][NT][4][32];
    __shared__ volatile int abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool gated = p.up != nullptr;
    const int rows1 = (gated ? 8 : 16) << p.lw1, rows2 = 16 << p.lw2;  // rows of h and of y of a unit
    const int rg1 = (p.I + rows1 - 1) / rows1, rg2 = (p.H + rows2 - 1) / rows2;
    const int kc1 = (kBoxes >> p.lw1) * Cfg::kBoxK, kc2 = (kBoxes >> p.lw2) * Cfg::kBoxK;  // k of a stage
    const int nch1 = (p.H + kc1 - 1) / kc1, nch2 = (p.I + kc2 - 1) / kc2;

    auto give_up = [&] {
        abort_flag = 1;
        atomicOr(p.err, kWatchdogTimeout);
    };
    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(&full[s], (FP8 ? 33 : 1) + NT);
            mbar_init(&empty[s], kWarps);
        }
        abort_flag = 0;
        fence_mbarrier_init();
        tma_prefetch_desc(&maps.gate);
        tma_prefetch_desc(&maps.up);
        tma_prefetch_desc(&maps.down);
    }
    __syncthreads();

    // ---------------------------------------------------- router
    if (warp < kWarps) {
        if (blockIdx.x == 0)
            for (int i = threadIdx.x; i < p.T * p.top_k; i += 32 * kWarps) p.h_max[i] = 0u;
        if constexpr (Cfg::kScaledX) {
            for (int t = gridDim.x - 1 - blockIdx.x; t < p.T; t += gridDim.x) scale_token<XT>(p, t, &red[0][0][0][0][0]);
            fence_proxy_async_all();  // x16 is read by bulk copies
        }
        // Few tokens: the logits are dealt out over the CTAs, and after the
        // barrier every CTA makes the same choice.  Many: a CTA takes a token,
        // logits and choice, and the barrier is for the choices.
        uint32_t *keys = reinterpret_cast<uint32_t *>(ring);
        const bool by_token = p.by_token;
        const int slots = p.T * p.top_k;
        if (by_token) {
            for (int t = blockIdx.x; t < p.T; t += gridDim.x) {
                router_token<XT>(p, t, keys, reinterpret_cast<uint4 *>(ring + 4096));
                consumer_sync();
                if (warp == 0) choose_experts(p, keys, p.chosen + t * p.top_k, p.chosen_weight + t * p.top_k);
                consumer_sync();
            }
        } else {
            router_logits<XT>(p, &red[0][0][0][0][0]);
        }
        __threadfence();
        consumer_sync();
        if (threadIdx.x == 0) {
            atomicAdd(&p.counters[0], 1u);
            if (!wait_count(&p.counters[0], gridDim.x)) give_up();
        }
        consumer_sync();
        if (by_token) {
            for (int i = threadIdx.x; i < slots; i += 32 * kWarps) {
                r.expert[i] = __ldcg(p.chosen + i);
                if (abort_flag) r.expert[i] = 0;  // never written
                r.weight[i] = __ldcg(p.chosen_weight + i);
            }
        } else {
            for (int i = threadIdx.x; i < p.T * p.E; i += 32 * kWarps) keys[i] = logit_key(__ldcg(p.logits + i));
            consumer_sync();
            for (int t = warp; t < p.T; t += kWarps) choose_experts(p, keys + t * p.E, r.expert + t * p.top_k, r.weight + t * p.top_k);
        }
        consumer_sync();
        group_slots(p, r, keys, 8 * NT);
        if (threadIdx.x == 0) r.per_token = (65536u + p.top_k - 1) / p.top_k;
        if (threadIdx.x == 0 && abort_flag) r.pairs = 0;
        for (int t = threadIdx.x; t < p.T; t += 32 * kWarps) r.x_scale[t] = Cfg::kScaledX ? __ldcg(p.x_scale + t) : 1.f;
    }
    fence_proxy_async_all();  // the ring held the keys; x16 of other CTAs is read by bulk copies
    __syncthreads();
    const int units1 = r.pairs * rg1, units2 = r.pairs * rg2 * p.k_splits;
    if (blockIdx.x == 0)
        for (int s = threadIdx.x; s < p.T * p.top_k && r.pairs; s += kThreads) {
            if (p.ids) p.ids[s] = r.expert[s];
            if (p.weights) p.weights[s] = r.weight[s];
        }
    // CTAs that had one unit less in the first half begin the second.
    const int grid = gridDim.x;
    const int shift = (static_cast<int>(blockIdx.x) + grid - units1 % grid) % grid;
    bool h_fits = true;  // h is used as the first half wrote it

    if (warp == kWarps) {
        // ------------------------------------------------ weights
        int stage = 0;
        uint32_t phase = 0, armed = 0, armed_parity = 0;
        bool ok = true;
        int y = 0;                     // matrix row of the unit
        const float *scale = nullptr;  // 8-bit weights: this lane's scale of a stage, of box lane % 16, its rows g or g + 8
        auto begin_unit = [&](bool first, const Unit &n) {
            const int rows = first ? p.I : p.H, width = first ? p.H : p.I, lw = first ? p.lw1 : p.lw2;
            y = n.expert * rows + n.row;
            if constexpr (FP8) {
                const int wrow = lane & ((1 << lw) - 1), box = (lane & 15) >> lw, upper = lane >> 4;
                const int row = min(rows - 1, n.row + (first && gated ? wrow * 8 : wrow * 16 + upper * 8));
                const long long kbs = (width + kScaleBlock - 1) / kScaleBlock, nbs = (rows + kScaleBlock - 1) / kScaleBlock;
                const float *base = !first ? p.s_down : gated && upper ? p.s_up : p.s_gate;
                scale = base + (n.expert * nbs + row / kScaleBlock) * kbs + box;
            }
        };
        auto load_stage = [&](bool first, int ch) {
            if (!__all_sync(0xffffffffu, mbar_wait_patient(&empty[stage], phase ^ 1u))) {
                if (lane == 0) give_up();
                ok = false;
                return;
            }
            uint8_t *dst = ring + stage * p.stage_bytes;
            const int lw = first ? p.lw1 : p.lw2, boxes = kBoxes >> lw, width = first ? p.H : p.I, k0 = ch * boxes * Cfg::kBoxK;
            if (lane == 0) {
                // Gate rows in the first half of the stage, up rows in the second.
                const int half = first && gated ? kStageWeights / 2 : 0, box_bytes = (half ? 1024 : 2048) << lw;
                if (k0 + boxes * Cfg::kBoxK <= (first ? p.flat_h : p.flat_i)) {
                    mbar_arrive_expect_tx(&full[stage], kStageWeights);
                    tma_load_3d(first ? &maps.gate : &maps.down, &full[stage], dst, 0, y, ch * boxes);
                    if (half) tma_load_3d(&maps.up, &full[stage], dst + half, 0, y, ch * boxes);
                } else {
                    // the row's end: the boxes that have any of it, one by one
                    const int some = min(boxes, (width - k0 + Cfg::kBoxK - 1) / Cfg::kBoxK);
                    mbar_arrive_expect_tx(&full[stage], some * box_bytes * (half ? 2 : 1));
                    for (int b = 0; b < some; ++b) {
                        tma_load_3d(first ? &maps.gate1 : &maps.down1, &full[stage], dst + b * box_bytes, k0 + b * Cfg::kBoxK, y, 0);
                        if (half) tma_load_3d(&maps.up1, &full[stage], dst + half + b * box_bytes, k0 + b * Cfg::kBoxK, y, 0);
                    }
                }
            }
            __syncwarp();
            if constexpr (FP8) {
                if (k0 + ((lane & 15) >> lw) * Cfg::kBoxK < width) cp_async_4(dst + kStageWeights + lane * 4, scale + ch * boxes, 4);
                cp_async_arrive(&full[stage]);
            }
            armed |= 1u << stage;
            armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
            if (kDebugBuild && !__all_sync(0xffffffffu, mbar_wait(&empty[stage], phase))) {  // one stage in flight
                if (lane == 0) give_up();
                ok = false;
                return;
            }
            if (++stage == p.stages) stage = 0, phase ^= 1u;
        };
        for (int u = blockIdx.x; ok && u < units1; u += grid) {
            begin_unit(true, first_unit(r, u, rg1, rows1, nch1));
            for (int ch = 0; ok && ch < nch1; ++ch) load_stage(true, ch);
        }
        for (int u = shift; ok && u < units2; u += grid) {
            const Unit n = down_unit(r, u, rows2, nch2, p.k_splits);
            begin_unit(false, n);
            for (int ch = n.ch0; ok && ch < n.ch1; ++ch) load_stage(false, ch);
        }
        __syncwarp();
        // No copy may be in flight when the CTA ends.  After a time-out a stage
        // may lack its tokens and never complete; its weights get 10 ms.
        if (lane == 0)
            for (int s = 0; s < p.stages; ++s)
                if ((armed & (1u << s)) && !mbar_wait(&full[s], (armed_parity >> s) & 1u, abort_flag ? 10000000ull : kWaitLimitNs)) give_up();
        __syncwarp();
    } else if (warp > kWarps) {
        // ------------------------------------------------ tokens
        const int first_token = (warp - kWarps - 1) * 8;
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        auto load_unit = [&](bool first, const Unit &n) {
            const int width = first ? p.H : p.I, lw = first ? p.lw1 : p.lw2, kc = (kBoxes >> lw) * Cfg::kBoxK;
            const int count = max(0, min(n.count - first_token, 8));  // of this warp
            const int offset = Cfg::kActOffset + (first_token + lane) * Cfg::act_stride(lw, first);
            const uint8_t *token = nullptr;
            if (lane < count) {
                const int slot = r.order[n.start + first_token + lane], t = r.token(slot);
                if (first)
                    token = Cfg::kScaledX ? reinterpret_cast<const uint8_t *>(p.x16 + static_cast<long long>(t) * p.H)
                                          : static_cast<const uint8_t *>(p.X) + 2 * (t * p.ldx);
                else
                    token = p.hidden16 + slot * parts_bytes(p.I, Cfg::kParts);
            }
            for (int ch = n.ch0; ok && ch < n.ch1; ++ch) {
                if (!__all_sync(0xffffffffu, mbar_wait_patient(&empty[stage], phase ^ 1u))) {
                    if (lane == 0) give_up();
                    ok = false;
                    break;
                }
                // Bytes of a token's k's (those of h come in whole runs of 64).
                const int k0 = ch * kc, k = min(kc, width - k0);
                const int bytes = first ? k * Cfg::kXBytes : static_cast<int>(parts_bytes(k, Cfg::kParts));
                if (lane == 0) mbar_arrive_expect_tx(&full[stage], count * bytes);
                __syncwarp();
                if (lane < count)
                    bulk_load(ring + stage * p.stage_bytes + offset, token + k0 * (first ? Cfg::kXBytes : Cfg::kHBytes), bytes, &full[stage]);
                if (++stage == p.stages) stage = 0, phase ^= 1u;
            }
        };
        for (int u = blockIdx.x; ok && u < units1; u += grid) load_unit(true, first_unit(r, u, rg1, rows1, nch1));
        // h of every CTA has to be there (and fitted, if need be).
        if (ok && shift < units2) {
            ok = __all_sync(0xffffffffu, wait_count(&p.counters[1], grid));
            if (ok && Cfg::kFit && !slots_fit(p)) ok = __all_sync(0xffffffffu, wait_count(&p.counters[2], grid));
            if (!ok && lane == 0) give_up();
            fence_proxy_async_all();
        }
        for (int u = shift; ok && u < units2; u += grid) load_unit(false, down_unit(r, u, rows2, nch2, p.k_splits));
    } else {
        // ------------------------------------------------ arithmetic
        int stage = 0, buf = 0;
        uint32_t phase = 0;
        const int g = lane >> 2;
        // One unit's sums for this warp's row group and box column.
        auto unit_sums = [&](auto first_c, const Unit &n, float(&acc)[NT][4]) {
            constexpr bool kFirst = decltype(first_c)::value;
            const int lw = kFirst ? p.lw1 : p.lw2, sharers = kWarps >> lw, my_row = warp & ((1 << lw) - 1), my_box = warp >> lw;
            const bool halves = kFirst && gated;
            const int w_box = halves ? 1024 : 2048, row8 = halves ? kStageWeights / 2 : 1024;
            const int width = kFirst ? p.H : p.I;
            constexpr int kParts = kFirst ? 1 : Cfg::kParts;
            constexpr int kBoxBytes = Cfg::kBoxK * (kFirst ? Cfg::kXBytes : Cfg::kHBytes);  // of a token's k's of a box
            // Token of this thread in each group of 8 (past the last: the last one, whose sums nobody takes).
            int token_at[NT];
#pragma unroll
            for (int i = 0; i < NT; ++i)
                token_at[i] = Cfg::kActOffset + my_box * kBoxBytes + min(i * 8 + g, n.count - 1) * Cfg::act_stride(lw, kFirst);
#pragma unroll
            for (int i = 0; i < NT; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
            for (int ch = n.ch0; ch < n.ch1; ++ch) {
                // after a time-out everything runs through without waiting
                if (!abort_flag && !mbar_wait_patient(&full[stage], phase)) give_up();
                const uint8_t *st = ring + stage * p.stage_bytes, *w = st + warp * w_box;
                const int valid = width - (ch * sharers + my_box) * Cfg::kBoxK;
                if (valid > 0) {
                    const uint8_t *act[NT];
#pragma unroll
                    for (int i = 0; i < NT; ++i) act[i] = st + token_at[i];
                    float sum[NT][4] = {};
                    if (valid < Cfg::kBoxK)
                        multiply_box<XT, FP8, NT, NT, kParts, true>(w, w + row8, act, valid, sum);
                    else if (NT > 1 && n.count <= 8)
                        multiply_box<XT, FP8, NT, 1, kParts, false>(w, w + row8, act, valid, sum);
                    else
                        multiply_box<XT, FP8, NT, NT, kParts, false>(w, w + row8, act, valid, sum);
                    // the scales of a box's rows
                    float s0 = 1.f, s1 = 1.f;
                    if constexpr (FP8) {
                        const float *sc = reinterpret_cast<const float *>(st + kStageWeights) + warp;
                        s0 = sc[0], s1 = sc[kBoxes];
                    }
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        acc[i][0] = fmaf(s0, sum[i][0], acc[i][0]);
                        acc[i][1] = fmaf(s0, sum[i][1], acc[i][1]);
                        acc[i][2] = fmaf(s1, sum[i][2], acc[i][2]);
                        acc[i][3] = fmaf(s1, sum[i][3], acc[i][3]);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[stage]);
                if (++stage == p.stages) stage = 0, phase ^= 1u;
            }
            // Warps of the same rows add their sums, in the order of their
            // boxes: the first one for the even tokens, the second for the odd.
            if (sharers == 1) return 3;
#pragma unroll
            for (int i = 0; i < NT; ++i)
                if (i * 8 < n.count)
#pragma unroll
                    for (int j = 0; j < 4; ++j) red[buf][warp][i][j][lane] = acc[i][j];
            consumer_sync();
            if (my_box < 2) {
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    if (i * 8 >= n.count) break;
                    float lo = 0.f, hi = 0.f;
                    for (int b = 0; b < sharers; ++b) {
                        lo += red[buf][(b << lw) + my_row][i][my_box][lane];
                        hi += red[buf][(b << lw) + my_row][i][my_box + 2][lane];
                    }
                    if (my_box == 0)
                        acc[i][0] = lo, acc[i][2] = hi;
                    else
                        acc[i][1] = lo, acc[i][3] = hi;
                }
            }
            buf ^= 1;
            return my_box == 0 ? 1 : my_box == 1 ? 2 : 0;
        };
        // Element i of a fragment: row g + 8 (i / 2), token 2 (lane % 4) + i % 2;
        // bit j of what unit_sums returns says that this warp has tokens of
        // i % 2 == j.
        float acc[NT][4];
        for (int u = blockIdx.x; u < units1; u += grid) {
            const Unit n = first_unit(r, u, rg1, rows1, nch1);
            const int mine = unit_sums(std::true_type{}, n, acc);
            const int row = n.row + (warp & ((1 << p.lw1) - 1)) * (gated ? 8 : 16) + g;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    if (!(mine & (1 << j)) || nt * 8 + j >= n.count) continue;
                    const int tok = nt * 8 + 2 * (lane & 3) + j;
                    const bool in = tok < n.count;
                    const int slot = r.order[n.start + min(tok, n.count - 1)];
                    const float xs = Cfg::kScaledX ? r.x_scale[r.token(slot)] : 1.f;
                    float largest = 0.f;
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        if (gated && half) break;
                        const int at = row + 8 * half;
                        float h = moe_act(p.act, acc[nt][j + 2 * half] * xs);
                        if (gated) h *= acc[nt][j + 2] * xs;
                        if (!in || at >= p.I) continue;
                        uint16_t part[Cfg::kParts];
                        split_parts<Cfg::kMma>(h, part);
                        uint16_t *to = reinterpret_cast<uint16_t *>(p.hidden16 + slot * parts_bytes(p.I, Cfg::kParts)) + at / 64 * (64 * Cfg::kParts) + at % 64;
                        if (!inside(reinterpret_cast<uint8_t *>(to + 64 * (Cfg::kParts - 1)) + 1 - p.hidden16, p.n_hidden16, p)) continue;
#pragma unroll
                        for (int i = 0; i < Cfg::kParts; ++i) to[64 * i] = part[i];
                        if constexpr (Cfg::kFit) {
                            if (!inside(static_cast<long long>(slot) * p.I + at, p.n_hidden, p)) continue;
                            p.hidden[static_cast<long long>(slot) * p.I + at] = h;
                            if (fabsf(h) < INFINITY) largest = fmaxf(largest, fabsf(h));
                        }
                    }
                    if constexpr (Cfg::kFit) {
#pragma unroll
                        for (int d = 16; d >= 4; d >>= 1) largest = fmaxf(largest, __shfl_xor_sync(0xffffffffu, largest, d));
                        if (in && lane < 4) atomicMax(p.h_max + slot, __float_as_uint(largest));
                    }
                }
        }
        fence_proxy_async_all();  // h is read by bulk copies
        __threadfence();
        consumer_sync();
        if (threadIdx.x == 0) atomicAdd(&p.counters[1], 1u);
        if constexpr (Cfg::kFit) {
            // h to FP16, now that every slot's largest element is known
            if (threadIdx.x == 0 && !wait_count(&p.counters[1], grid)) give_up();
            consumer_sync();
            h_fits = slots_fit(p);
        }
        if (!h_fits) {
            const int per = p.I / 8, all = p.T * p.top_k * per;
            for (int x = blockIdx.x * 32 * kWarps + threadIdx.x; x < all; x += grid * 32 * kWarps) {
                const float f = pow2(fit_exponent(__uint_as_float(__ldcg(p.h_max + x / per))));
                const float4 *h = reinterpret_cast<const float4 *>(p.hidden) + 2ll * x;
                const float4 a = __ldcg(h), b = __ldcg(h + 1);
                const float v[8] = {a.x * f, a.y * f, a.z * f, a.w * f, b.x * f, b.y * f, b.z * f, b.w * f};
                const int at = x % per * 8;
                uint16_t part[8][Cfg::kParts];
#pragma unroll
                for (int i = 0; i < 8; ++i) split_parts<Cfg::kMma>(v[i], part[i]);
                uint8_t *to = p.hidden16 + x / per * parts_bytes(p.I, Cfg::kParts) + at / 64 * (128 * Cfg::kParts) + at % 64 * 2;
                if (!inside(to + 128 * (Cfg::kParts - 1) + 15 - p.hidden16, p.n_hidden16, p)) continue;
#pragma unroll
                for (int j = 0; j < Cfg::kParts; ++j) {
                    auto two = [&](int i) { return part[i][j] | static_cast<uint32_t>(part[i + 1][j]) << 16; };
                    *reinterpret_cast<uint4 *>(to + 128 * j) = make_uint4(two(0), two(2), two(4), two(6));
                }
            }
            fence_proxy_async_all();  // read by bulk copies
            __threadfence();
            consumer_sync();
            if (threadIdx.x == 0) atomicAdd(&p.counters[2], 1u);
        }
        const long long slots = static_cast<long long>(p.T) * p.top_k;
        for (int u = shift; u < units2; u += grid) {
            const Unit n = down_unit(r, u, rows2, nch2, p.k_splits);
            const int mine = unit_sums(std::false_type{}, n, acc);
            const int row = n.row + (warp & ((1 << p.lw2) - 1)) * 16 + g;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int tok = nt * 8 + 2 * (lane & 3) + (i & 1), at = row + 8 * (i >> 1);
                    if (!(mine & (1 << (i & 1))) || tok >= n.count || at >= p.H) continue;
                    const long long to = (n.split * slots + r.order[n.start + tok]) * p.H + at;
                    if (inside(to, p.n_part, p)) p.part[to] = acc[nt][i];
                }
        }
        // ------------------------------------------------ sum over a token's experts
        __threadfence();
        consumer_sync();
        if (threadIdx.x == 0) {
            atomicAdd(&p.counters[3], 1u);
            if (!wait_count(&p.counters[3], grid)) give_up();
        }
        consumer_sync();
        if (!abort_flag) {
            const int groups = p.H / 4;
            for (int x = blockIdx.x * 32 * kWarps + threadIdx.x; x < p.T * groups; x += grid * 32 * kWarps) {
                const int t = x / groups, c = x % groups * 4;
                float y[4] = {0.f, 0.f, 0.f, 0.f};
                for (int j = 0; j < p.top_k; ++j) {
                    const long long slot = static_cast<long long>(t) * p.top_k + j;
                    float4 v = __ldcg(reinterpret_cast<const float4 *>(p.part + slot * p.H + c));
                    for (int s = 1; s < p.k_splits; ++s) {
                        const float4 w = __ldcg(reinterpret_cast<const float4 *>(p.part + (s * slots + slot) * p.H + c));
                        v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
                    }
                    float f = r.weight[slot];
                    if (!h_fits) f *= pow2(-fit_exponent(__uint_as_float(__ldcg(p.h_max + slot))));
                    y[0] = fmaf(f, v.x, y[0]), y[1] = fmaf(f, v.y, y[1]), y[2] = fmaf(f, v.z, y[2]), y[3] = fmaf(f, v.w, y[3]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (inside(static_cast<long long>(t) * p.ldy + c + i, p.n_y, p)) store_out(p.Y, static_cast<size_t>(t) * p.ldy + c + i, p.y_type, y[i]);
            }
        }
    }
    __syncthreads();
    // The last CTA to leave clears the barriers for the next call.
    if (threadIdx.x == 0 && atomicAdd(&p.counters[4], 1u) == gridDim.x - 1)
        p.counters[0] = p.counters[1] = p.counters[2] = p.counters[3] = p.counters[4] = 0u;
}

// Tensor maps of all experts' `rows` rows of `width` elements: `many` with boxes
// of `boxes` 128-byte pieces of `box_rows` rows (dimensions: piece, row, number
// of the whole piece), `one` with single pieces, where the row's ragged end reads
// as zeros.  *flat: elements of a row that `many` reaches.  A map that no stage
// takes is the other one again.
bool encode_expert_maps(CUtensorMap *many, CUtensorMap *one, int *flat, const void *base, int elem_bytes, CUtensorMapDataType dt,
                        uint64_t rows, uint64_t width, uint32_t box_rows, uint32_t boxes) {
    const uint64_t piece = 128 / elem_bytes, whole = width / piece, stage = boxes * piece;
    const bool use_many = whole >= boxes, use_one = !use_many || width % stage != 0;
    *flat = use_many ? static_cast<int>(whole * piece) : 0;
    bool ok = true;
    if (use_many) ok = encode_box_map(many, dt, base, piece, rows, whole, width * elem_bytes, 128, piece, box_rows, boxes);
    if (ok && use_one) ok = encode_box_map(one, dt, base, width, rows, 1, width * elem_bytes, width * elem_bytes, piece, box_rows, 1);
    if (!use_many) *many = *one;
    if (!use_one) *one = *many;
    return ok;
}

// How a phase is cut into units: log2 of WR, and of the down projection also
// how many units share a row group's k.  `groups` row groups of 16 (one of each
// expert that is used), `k` long; `act_bytes` of activations in a stage with
// WR = 1.  Preferred is the largest WR, then the fewest splits, whose units
// fill whole rounds over the SMs to 80 %; failing that, what fills them best.
// (64 tokens, 64 experts of 2048 x 1024, 6 each: 104 us with WR = 16 at 84 %, 110
// with WR = 8 at 96 %; 52 tokens, 23 experts of 352 x 880, 7 each: 41 at 83 %, 56
// with WR = 1 at 95 %; one token over 8 experts: 104 us at 75 %, 98 at 91 %.)
// WR is at least what keeps a stage's activations within its weights (the ring
// would hold too few stages) and a stage's k below the whole length; 16 only
// where a unit of 8 would have fewer than 12 stages, over which to hide its end.
struct Cut {
    int lw = 0, splits = 1;
};
Cut pick_cut(double groups, int k, int box_k, int act_bytes, int max_splits, int sms) {
    int least = 0;
    while (least < 4 && ((act_bytes >> least) > kStageWeights || (kBoxes >> least) * box_k >= 2 * k)) ++least;
    Cut best;
    double best_fill = -1.0;
    const int most = k < 12 * (kBoxes >> 3) * box_k ? 4 : 3;
    for (int lw = std::max(most, least); lw >= least; --lw)
        for (int splits = 1; splits <= max_splits; splits *= 2) {
            if (splits > 1 && (kBoxes >> lw) * box_k * splits * 2 > k) break;  // two stages at least
            const double units = std::max(1.0, groups / (1 << lw) * splits);
            const double fill = units / (std::ceil(units / sms - 1e-9) * sms);
            if (fill > best_fill + 1e-9) best_fill = fill, best.lw = lw, best.splits = splits;
            if (fill >= 0.8) return best;
        }
    return best;
}

template <int XT, bool FP8, int NT>
cudaError_t launch_moe(const Moe &m, MoeArgs a, double active, cudaStream_t stream) {
    using Cfg = MoeCfg<XT, FP8>;
    auto kern = moe_kernel<XT, FP8, NT>;
    const int sms = device_sm_count(), act = std::min(m.T, 8 * NT) * kBoxes * Cfg::kBoxK;  // elements of a stage with WR = 1
    const Cut c1 = pick_cut(active * m.I / (m.up ? 8 : 16), m.H, Cfg::kBoxK, act * Cfg::kXBytes, 1, sms);
    const Cut c2 = pick_cut(active * m.H / 16, m.I, Cfg::kBoxK, act * Cfg::kHBytes, kMaxSplits, sms);
    a.lw1 = c1.lw;
    a.lw2 = c2.lw;
    a.k_splits = c2.splits;
    // a stage holds the weights, their scales and either kind of activations
    const int act_bytes = std::min(m.T, 8 * NT) * std::max(Cfg::act_stride(a.lw1, true), Cfg::act_stride(a.lw2, false));
    a.stage_bytes = (Cfg::kActOffset + act_bytes + 1023) / 1024 * 1024;
    constexpr int kRing = 226 * 1024 - static_cast<int>(sizeof(Routing) + 2 * kWarps * NT * 4 * 32 * 4 + 16 * kMaxStages + 128);
    static_assert(kRing >= 1024 + kTokensOfTheirOwn * kMoeMaxExperts * 4 && kRing >= 1024 + 4096 + kMoeMaxWidth * 2,
                  "the ring holds the keys of the choice, or one token and its keys");
    a.stages = std::min(kMaxStages, (kRing - 1024) / a.stage_bytes);  // two at least: 2 x (32 + 32) KB and paddings
    const int wb = Cfg::kWBytes;
    const auto dt = FP8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16;
    a.by_token = m.T >= kTokensOfTheirOwn;
    MoeMaps maps;
    const uint64_t rows_i = static_cast<uint64_t>(m.E) * m.I, rows_h = static_cast<uint64_t>(m.E) * m.H;
    const uint32_t rows1 = (m.up ? 8 : 16) << a.lw1, boxes1 = kBoxes >> a.lw1, rows2 = 16 << a.lw2, boxes2 = kBoxes >> a.lw2;
    bool ok = encode_expert_maps(&maps.gate, &maps.gate1, &a.flat_h, m.gate, wb, dt, rows_i, m.H, rows1, boxes1) &&
              encode_expert_maps(&maps.down, &maps.down1, &a.flat_i, m.down, wb, dt, rows_h, m.I, rows2, boxes2);
    if (ok && m.up)
        ok = encode_expert_maps(&maps.up, &maps.up1, &a.flat_h, m.up, wb, dt, rows_i, m.H, rows1, boxes1);
    else
        maps.up = maps.up1 = maps.gate;  // not used
    if (!ok) return cudaErrorNotSupported;
    static unsigned long long smem_set = 0;
    cudaError_t e = ensure_dynamic_smem(kern, kRing, smem_set);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeCooperative;
    attr.val.cooperative = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(device_sm_count());
    cfg.blockDim = dim3(moe_threads(NT));
    cfg.dynamicSmemBytes = kRing;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kern, maps, a);
    return e != cudaSuccess ? e : cudaPeekAtLastError();
}

// 8 tokens a unit up to 6.5 tokens an expert, where a second unit for an expert
// with more costs less than accumulators that mostly stay empty (64 tokens over
// 64 experts, 6 each: 104 us against 114 with 16 a unit), else 16 (52 tokens over
// 23 experts, 7 each, 15.8 an expert: 41.0 us against 42.6 with 8, and with BF16
// weights 40.3 against 47.0).
template <int XT, bool FP8>
cudaError_t launch_moe_tokens(const Moe &m, const MoeArgs &a, double active, double tokens, cudaStream_t stream) {
    return tokens <= 6.5 ? launch_moe<XT, FP8, 1>(m, a, active, stream) : launch_moe<XT, FP8, 2>(m, a, active, stream);
}

}  // namespace

cudaError_t run_moe(const Moe &m, cudaStream_t stream, CallInfo *info) {
    MoeArgs a = {};
    a.T = m.T;
    a.E = m.E;
    a.top_k = m.top_k;
    a.H = m.H;
    a.I = m.I;
    a.X = m.X;
    a.ldx = m.ldx;
    a.router = m.router;
    a.router_f32 = m.router_type == kOutF32;
    a.gate = m.gate;
    a.up = m.up;
    a.down = m.down;
    a.s_gate = m.s_gate;
    a.s_up = m.s_up;
    a.s_down = m.s_down;
    a.Y = m.Y;
    a.ldy = m.ldy;
    a.y_type = m.y_type;
    a.act = m.act;
    a.renorm = m.renorm;
    a.ids = m.ids;
    a.weights = m.weights;
    a.err = watchdog_word();
    // Experts with any token if the router chose evenly, and tokens of one.
    const double slots = static_cast<double>(m.T) * m.top_k;
    const double active = m.E * (1.0 - std::pow(1.0 - static_cast<double>(m.top_k) / m.E, m.T)), tokens = slots / active;
    // Scratch, in floats, each part on 256 bytes.
    auto up64 = [](size_t n) { return (n + 63) / 64 * 64; };
    const size_t n_slots = static_cast<size_t>(m.T) * m.top_k;
    const size_t n_logits = up64(static_cast<size_t>(m.T) * m.E), n_hidden = up64(n_slots * m.I);
    const size_t n_h16 = up64(n_slots * parts_bytes(m.I, 3) / 4), n_x16 = up64(static_cast<size_t>(m.T) * m.H / 2), n_max = up64(n_slots);
    Scratch s;
    const cudaError_t e =
        acquire_scratch(stream, n_logits + n_hidden + n_h16 + n_x16 + 3 * n_max + up64(m.T) + n_slots * m.H * kMaxSplits, 5, &s);
    if (e != cudaSuccess) return e;
    a.logits = s.partials;
    a.hidden = a.logits + n_logits;
    a.hidden16 = reinterpret_cast<uint8_t *>(a.hidden + n_hidden);
    a.x16 = reinterpret_cast<__half *>(a.hidden + n_hidden + n_h16);
    a.h_max = reinterpret_cast<unsigned *>(a.hidden + n_hidden + n_h16 + n_x16);
    a.x_scale = a.hidden + n_hidden + n_h16 + n_x16 + n_max;
    a.chosen_weight = a.x_scale + up64(m.T);
    a.chosen = reinterpret_cast<uint16_t *>(a.chosen_weight + n_max);
    a.part = a.chosen_weight + 2 * n_max;
    a.counters = s.counters;
    if (kDebugBuild) {
        a.n_logits = n_logits;
        a.n_hidden = n_hidden;
        a.n_hidden16 = n_h16 * 4;
        a.n_x16 = n_x16 * 2;
        a.n_part = n_slots * m.H * kMaxSplits;
        a.n_y = static_cast<size_t>(m.T - 1) * static_cast<size_t>(m.ldy) + m.H;
        a.n_y -= std::min(a.n_y, debug_shrink_c());
    }
    info->launches = 1;
    info->plan = "moe_few_tokens";
    const bool fp8 = m.w_type == kTypeE4M3;
    if (m.x_type == kOutF16)
        return fp8 ? launch_moe_tokens<kOutF16, true>(m, a, active, tokens, stream) : launch_moe_tokens<kOutF16, false>(m, a, active, tokens, stream);
    return fp8 ? launch_moe_tokens<kOutBF16, true>(m, a, active, tokens, stream) : launch_moe_tokens<kOutBF16, false>(m, a, active, tokens, stream);
}

}  // namespace gemm11

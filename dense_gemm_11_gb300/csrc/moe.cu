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
//   * work is cut into units of 16 matrix rows (8 gate rows with the 8 up rows
//     they meet, or 16 rows of the down projection) for one expert and up to
//     8 NT of its tokens.  Units are small so that they spread evenly;
//   * a producer warp copies each unit's rows and its tokens' activations in
//     chunks (1 KB of every row) into a ring of stages with bulk copies.  It
//     runs ahead of the arithmetic across units, and into the down projection
//     while the other CTAs still finish the first half;
//   * eight warps share a chunk's k; each multiplies its 16 x (K / 8) slice by
//     the tokens with mma.sync and the eight partial tiles are added in warp
//     order in shared memory.  The matrix instruction is the warp-level one:
//     a unit has 1 to 8 NT columns of 128-column tcgen05 tiles and is bound by
//     memory, and fragments come straight from the row-major chunk (the k of a
//     fragment may be any permutation that both operands share, so that a
//     thread's k's are 8 neighbours, one 16-byte load).
// Between the phases (router, first half, down projection) CTAs meet at two
// grid barriers; the last unit of a row group to finish adds the experts'
// contributions of its 16 columns in slot order, so results do not depend on
// timing.  Every wait is bounded.
//
// Numbers: weights and tokens of the same 16-bit type multiply exactly in
// mma.sync's native type; 8-bit weights and the down projection use TF32,
// which holds every 16- and 8-bit value exactly.  Sums are FP32.  h is rounded
// once, to TF32 (11 significant bits, FP32's range: a 16-bit type would lose
// either bits or range).
#include <algorithm>
#include <cstdint>

#include <cuda_fp8.h>

#include "fp8.h"
#include "ptx.cuh"

namespace gemm11 {
namespace {

constexpr int kWarps = 8;                       // consumer warps
constexpr int kMoeThreads = 32 * (kWarps + 1);  // and the producer warp
constexpr int kRows = 16;                       // matrix rows of a unit
constexpr int kMaxStages = 16;

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
    float *logits, *hidden, *part;  // scratch: T x E, slots x I, slots x H
    unsigned *counters;             // 0..2: barriers and exit; 4..: row groups of the down projection
    unsigned *err;
    int stages, stage_bytes, tok_rows;
};

// Shared-memory tables of the routing, the same in every CTA.
struct Routing {
    float weight[kMoeMaxSlots];
    uint16_t expert[kMoeMaxSlots];  // of slot t * top_k + j
    uint16_t order[kMoeMaxSlots];   // slots, grouped by expert, ascending
    uint16_t pair_expert[kMoeMaxSlots], pair_first[kMoeMaxSlots], pair_start[kMoeMaxSlots];
    uint8_t pair_groups[kMoeMaxSlots], pair_count[kMoeMaxSlots];
    int offset[kMoeMaxExperts + 1];
    int pairs;
};

__device__ __forceinline__ void mma_tf32(float (&c)[4], const float (&a)[4], float b0, float b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(__float_as_uint(a[0])), "r"(__float_as_uint(a[1])), "r"(__float_as_uint(a[2])), "r"(__float_as_uint(a[3])),
          "r"(__float_as_uint(b0)), "r"(__float_as_uint(b1)));
}
template <int XT>
__device__ __forceinline__ void mma_16bit(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
    if constexpr (XT == kOutBF16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile(
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

__device__ __forceinline__ float moe_act(int act, float v) {
    return act == kActSilu ? v * rcp_approx(1.f + __expf(-v)) : apply_activation(act, v);
}

// Eight neighbouring values of a row as floats.
__device__ __forceinline__ void widen8(const uint4 &w, int type, float (&v)[8]) { unpack8_out16(w, type, v); }
__device__ __forceinline__ void widen8_e4m3(const uint2 &w, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t u = i < 2 ? w.x : w.y;
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(u >> (16 * (i & 1))), __NV_E4M3);
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

// ---------------------------------------------------------------- routing
// Logits of expert e for 8 tokens at a time, one (expert, token group) a CTA;
// the consumer warps share H.
template <int XT>
__device__ void router_logits(const MoeArgs &p, float *red) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int groups = (p.T + 7) / 8;
    for (int u = blockIdx.x; u < p.E * groups; u += gridDim.x) {
        const int e = u / groups, t0 = (u % groups) * 8;
        float acc[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = 0.f;
        for (int k = threadIdx.x * 8; k < p.H; k += 32 * kWarps * 8) {
            float w[8];
            const long long at = static_cast<long long>(e) * p.H + k;
            if (p.router_f32) {
                const float4 *r = reinterpret_cast<const float4 *>(static_cast<const float *>(p.router) + at);
                const float4 a = __ldg(r), b = __ldg(r + 1);
                w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
            } else {
                widen8(__ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.router) + at)), XT, w);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (t0 + i >= p.T) break;
                float x[8];
                widen8(__ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.X) + (t0 + i) * p.ldx + k)), XT, x);
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[i] = fmaf(w[j], x[j], acc[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
#pragma unroll
            for (int d = 16; d >= 1; d >>= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], d);
            if (lane == 0) red[warp * 8 + i] = acc[i];
        }
        consumer_sync();
        if (threadIdx.x < 8 && t0 + threadIdx.x < p.T) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) s += red[w * 8 + threadIdx.x];
            p.logits[static_cast<long long>(t0 + threadIdx.x) * p.E + e] = s;
        }
        consumer_sync();
    }
}

// Order-preserving key of a logit: -0 equals +0, NaN comes first; 0 is below
// every key.
__device__ __forceinline__ uint32_t logit_key(float v) {
    if (v != v) return 0xFFFFFFFFu;
    const uint32_t b = __float_as_uint(v + 0.f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// One warp, one token: softmax and its top_k largest, by repeated maximum
// (keys in shared memory, taken ones set to 0).
__device__ void choose_experts(const MoeArgs &p, int t, uint32_t *keys, Routing &r) {
    const int lane = threadIdx.x & 31;
    const float *logits = p.logits + static_cast<long long>(t) * p.E;
    for (int e = lane; e < p.E; e += 32) keys[e] = logit_key(__ldcg(logits + e));
    float top = 0.f, chosen = 0.f;
    float mine[(kMoeMaxTopK + 31) / 32];
    mine[0] = 0.f;
    for (int j = 0; j < p.top_k; ++j) {
        uint32_t best = 0;
        int at = 0;
        for (int e = lane; e < p.E; e += 32)
            if (keys[e] > best) best = keys[e], at = e;
        const uint32_t m = __reduce_max_sync(0xffffffffu, best);
        const int e = static_cast<int>(__reduce_min_sync(0xffffffffu, best == m ? static_cast<unsigned>(at) : 0xFFFFFFFFu));
        const float l = __ldcg(logits + e);
        if (j == 0) top = l;
        const float v = expf(l - top);
        chosen += v;
        if (lane == j) mine[0] = v;
        if (lane == 0) r.expert[t * p.top_k + j] = static_cast<uint16_t>(e);
        if (lane == (e & 31)) keys[e] = 0;
        __syncwarp();
    }
    float sum = chosen;
    if (!p.renorm) {
        sum = 0.f;
        for (int e = lane; e < p.E; e += 32) sum += expf(__ldcg(logits + e) - top);
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    }
    if (lane < p.top_k) r.weight[t * p.top_k + lane] = mine[0] / sum;
    __syncwarp();
}

// One warp: slots grouped by expert (a counting sort that keeps their order),
// and the (expert, token group) pairs that the units go over.
__device__ void group_slots(const MoeArgs &p, Routing &r, int group) {
    const int lane = threadIdx.x & 31, slots = p.T * p.top_k;
    for (int e = lane; e <= p.E; e += 32) r.offset[e] = 0;
    __syncwarp();
    for (int s = lane; s < slots; s += 32) atomicAdd(&r.offset[r.expert[s]], 1);
    __syncwarp();
    int before = 0, pairs_before = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
        const int e = e0 + lane;
        const int n = e < p.E ? r.offset[e] : 0;
        const int np = (n + group - 1) / group;
        int sum = n, psum = np;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int a = __shfl_up_sync(0xffffffffu, sum, d), b = __shfl_up_sync(0xffffffffu, psum, d);
            if (lane >= d) sum += a, psum += b;
        }
        if (e < p.E) {
            const int first = pairs_before + psum - np, start = before + sum - n;
            r.offset[e] = start;
            for (int i = 0; i < np; ++i) {
                r.pair_expert[first + i] = static_cast<uint16_t>(e);
                r.pair_first[first + i] = static_cast<uint16_t>(first);
                r.pair_groups[first + i] = static_cast<uint8_t>(np);
                r.pair_start[first + i] = static_cast<uint16_t>(start + i * group);
                r.pair_count[first + i] = static_cast<uint8_t>(min(group, n - i * group));
            }
        }
        before += __shfl_sync(0xffffffffu, sum, 31);
        pairs_before += __shfl_sync(0xffffffffu, psum, 31);
    }
    if (lane == 0) r.pairs = pairs_before;
    __syncwarp();
    for (int s0 = 0; s0 < slots; s0 += 32) {
        const int s = s0 + lane;
        const int e = s < slots ? r.expert[s] : -1 - lane;
        const unsigned same = __match_any_sync(0xffffffffu, e);
        const int rank = __popc(same & ((1u << lane) - 1u));
        const int base = s < slots ? r.offset[e] : 0;
        __syncwarp();
        if (s < slots) {
            r.order[base + rank] = static_cast<uint16_t>(s);
            if (rank == 0) r.offset[e] = base + __popc(same);
        }
        __syncwarp();
    }
}

// ---------------------------------------------------------------- units
struct Unit {
    int expert, rg, pair, start, count;
};
// Unit u of the first half: the token groups of an expert next to each other
// for the same rows, so that they share the rows' bytes in L2.
__device__ __forceinline__ Unit first_unit(const Routing &r, int u, int row_groups) {
    Unit n;
    const int p0 = u / row_groups, first = r.pair_first[p0], groups = r.pair_groups[p0];
    const int i = u - first * row_groups;
    n.rg = i / groups;
    n.pair = first + i % groups;
    n.expert = r.pair_expert[n.pair];
    n.start = r.pair_start[n.pair];
    n.count = r.pair_count[n.pair];
    return n;
}
// Unit u of the down projection: row group by row group.
__device__ __forceinline__ Unit down_unit(const Routing &r, int u) {
    Unit n;
    n.rg = u / r.pairs;
    n.pair = u % r.pairs;
    n.expert = r.pair_expert[n.pair];
    n.start = r.pair_start[n.pair];
    n.count = r.pair_count[n.pair];
    return n;
}

template <bool FP8>
struct MoeCfg {
    static constexpr int kWBytes = FP8 ? 1 : 2;
    static constexpr int kKC = 1024 / kWBytes;         // k of a chunk
    static constexpr int kKW = kKC / kWarps;           // of one warp: 128 (one scale block) or 64
    // Row strides in shared memory that keep the fragment loads free of bank
    // conflicts: a quarter warp reads 2 rows x 64 bytes (16-bit weights and
    // tokens) or 4 x 16 bytes of 2 rows (FP32 activations), half a warp 4 rows
    // x 32 bytes (8-bit weights).
    static constexpr int kWStride = 1024 + (FP8 ? 32 : 64);
    static constexpr int kXStride = kKC * 2 + 64;
    static constexpr int kHStride = kKC * 4 + 16;
    static constexpr int kScaleBytes = FP8 ? 2 * kWarps * 4 : 0;
    static constexpr int kActOffset = kRows * kWStride + kScaleBytes;
};

// The 16 rows x this warp's k of one chunk times the tokens, added to acc.
// FIRST: tokens are X rows of 16 bits, else FP32 h rows.  valid: k's of the
// chunk that exist.
template <int XT, bool FP8, int NT, bool FIRST>
__device__ __forceinline__ void multiply_chunk(const uint8_t *stage, int valid, int count, float (&acc)[NT][4]) {
    using Cfg = MoeCfg<FP8>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int k_warp = warp * Cfg::kKW;
    if (k_warp >= valid) return;
    float sum[NT][4];
    float(&c)[NT][4] = FP8 ? sum : acc;
    if (FP8) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[n][i] = 0.f;
    }
#pragma unroll
    for (int s = 0; s < Cfg::kKW / 32; ++s) {
        const int k = k_warp + s * 32 + t * 8;
        const bool in = k < valid;
        const uint8_t *w0 = stage + g * Cfg::kWStride + k * Cfg::kWBytes, *w1 = w0 + 8 * Cfg::kWStride;
        const uint4 zero = make_uint4(0, 0, 0, 0);
        if constexpr (!FP8 && FIRST) {
            const uint4 a = in ? *reinterpret_cast<const uint4 *>(w0) : zero;
            const uint4 b = in ? *reinterpret_cast<const uint4 *>(w1) : zero;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if (n * 8 >= count) break;
                const uint4 x = in && n * 8 + g < count ? *reinterpret_cast<const uint4 *>(stage + Cfg::kActOffset + (n * 8 + g) * Cfg::kXStride + k * 2) : zero;
                mma_16bit<XT>(c[n], a.x, b.x, a.y, b.y, x.x, x.y);
                mma_16bit<XT>(c[n], a.z, b.z, a.w, b.w, x.z, x.w);
            }
        } else {
            float wa[8], wb[8];
            if constexpr (FP8) {
                const uint2 z2 = make_uint2(0, 0);
                widen8_e4m3(in ? *reinterpret_cast<const uint2 *>(w0) : z2, wa);
                widen8_e4m3(in ? *reinterpret_cast<const uint2 *>(w1) : z2, wb);
            } else {
                widen8(in ? *reinterpret_cast<const uint4 *>(w0) : zero, XT, wa);
                widen8(in ? *reinterpret_cast<const uint4 *>(w1) : zero, XT, wb);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if (n * 8 >= count) break;
                const bool tok = in && n * 8 + g < count;
                float x[8];
                if constexpr (FIRST) {
                    widen8(tok ? *reinterpret_cast<const uint4 *>(stage + Cfg::kActOffset + (n * 8 + g) * Cfg::kXStride + k * 2) : zero, XT, x);
                } else {
                    const float4 *h = reinterpret_cast<const float4 *>(stage + Cfg::kActOffset + (n * 8 + g) * Cfg::kHStride + k * 4);
                    const float4 z4 = make_float4(0.f, 0.f, 0.f, 0.f);
                    const float4 h0 = tok ? h[0] : z4, h1 = tok ? h[1] : z4;
                    x[0] = h0.x, x[1] = h0.y, x[2] = h0.z, x[3] = h0.w, x[4] = h1.x, x[5] = h1.y, x[6] = h1.z, x[7] = h1.w;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float a[4] = {wa[2 * i], wb[2 * i], wa[2 * i + 1], wb[2 * i + 1]};
                    mma_tf32(c[n], a, x[2 * i], x[2 * i + 1]);
                }
            }
        }
    }
    if (FP8) {
        const float *sc = reinterpret_cast<const float *>(stage + kRows * Cfg::kWStride);
        const float s0 = sc[warp], s1 = sc[kWarps + warp];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            acc[n][0] = fmaf(s0, sum[n][0], acc[n][0]);
            acc[n][1] = fmaf(s0, sum[n][1], acc[n][1]);
            acc[n][2] = fmaf(s1, sum[n][2], acc[n][2]);
            acc[n][3] = fmaf(s1, sum[n][3], acc[n][3]);
        }
    }
}

template <int XT, bool FP8, int NT, bool GATED>
__global__ void __launch_bounds__(kMoeThreads, 1) moe_kernel(const MoeArgs p) {
    using Cfg = MoeCfg<FP8>;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ Routing r;
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages];
    __shared__ float red[2][kWarps][NT][4][32];
    __shared__ volatile int abort_flag;
    __shared__ int last;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kUnitRows1 = GATED ? 8 : 16;  // rows of h of a unit
    const int rg1 = p.I / kUnitRows1, rg2 = p.H / kRows;
    const int nch1 = (p.H + Cfg::kKC - 1) / Cfg::kKC, nch2 = (p.I + Cfg::kKC - 1) / Cfg::kKC;

    auto give_up = [&] {
        abort_flag = 1;
        atomicOr(p.err, kWatchdogTimeout);
    };
    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(&full[s], FP8 ? 33 : 1);
            mbar_init(&empty[s], kWarps);
        }
        abort_flag = 0;
        fence_mbarrier_init();
    }
    __syncthreads();

    // ---------------------------------------------------- router
    if (warp < kWarps) {
        router_logits<XT>(p, &red[0][0][0][0][0]);
        __threadfence();
        consumer_sync();
        if (threadIdx.x == 0) {
            atomicAdd(&p.counters[0], 1u);
            if (!wait_count(&p.counters[0], gridDim.x)) give_up();
        }
        consumer_sync();
        if (!abort_flag)
            for (int t = warp; t < p.T; t += kWarps)
                choose_experts(p, t, reinterpret_cast<uint32_t *>(ring) + warp * kMoeMaxExperts, r);
        consumer_sync();
        if (warp == 0 && !abort_flag) group_slots(p, r, 8 * NT);
        if (threadIdx.x == 0 && abort_flag) r.pairs = 0;
    }
    fence_proxy_async_smem();  // the ring held the keys
    __syncthreads();
    const int units1 = r.pairs * rg1, units2 = r.pairs * rg2;
    if (blockIdx.x == 0)
        for (int s = threadIdx.x; s < p.T * p.top_k && r.pairs; s += kMoeThreads) {
            if (p.ids) p.ids[s] = r.expert[s];
            if (p.weights) p.weights[s] = r.weight[s];
        }
    // CTAs that had one unit less in the first half begin the second.
    const int shift = (blockIdx.x + gridDim.x - units1 % gridDim.x) % gridDim.x;

    if (warp == kWarps) {
        // ------------------------------------------------ producer
        int stage = 0;
        uint32_t phase = 0, armed = 0, armed_parity = 0;
        bool ok = true;
        const long long hi_bytes = static_cast<long long>(p.H) * Cfg::kWBytes, i_bytes = static_cast<long long>(p.I) * Cfg::kWBytes;
        // Takes a free stage and starts the copies of a chunk's weight rows.
        auto load_rows = [&](bool first, const Unit &n, int ch) {
            if (!__all_sync(0xffffffffu, mbar_wait(&empty[stage], phase ^ 1u))) {
                if (lane == 0) give_up();
                ok = false;
                return;
            }
            uint8_t *dst = ring + static_cast<size_t>(stage) * p.stage_bytes;
            const int k0 = ch * Cfg::kKC, k = min(Cfg::kKC, (first ? p.H : p.I) - k0);
            if (lane == 0)
                mbar_arrive_expect_tx(&full[stage], kRows * k * Cfg::kWBytes + n.count * k * (first ? 2 : 4));
            __syncwarp();
            if (lane < kRows) {
                const uint8_t *base;
                long long row;
                if (first) {
                    const bool is_up = GATED && lane >= 8;
                    base = static_cast<const uint8_t *>(is_up ? p.up : p.gate);
                    row = static_cast<long long>(n.expert) * p.I + n.rg * kUnitRows1 + (GATED ? lane & 7 : lane);
                    base += row * hi_bytes;
                } else {
                    row = static_cast<long long>(n.expert) * p.H + n.rg * kRows + lane;
                    base = static_cast<const uint8_t *>(p.down) + row * i_bytes;
                }
                bulk_load(dst + lane * Cfg::kWStride, base + static_cast<long long>(k0) * Cfg::kWBytes, k * Cfg::kWBytes, &full[stage]);
            }
            if constexpr (FP8) {
                // scales of the chunk's 8 k blocks, for rows 0..7 and rows 8..15
                const int kbs = ((first ? p.H : p.I) + kScaleBlock - 1) / kScaleBlock;
                const int nbs = ((first ? p.I : p.H) + kScaleBlock - 1) / kScaleBlock;
                const int kb = ch * kWarps + (lane & 7);
                if (lane < 2 * kWarps && kb < kbs) {
                    const int row = first ? n.rg * kUnitRows1 + (GATED ? 0 : lane & 8) : n.rg * kRows + (lane & 8);
                    const float *s = first ? (GATED && lane >= 8 ? p.s_up : p.s_gate) : p.s_down;
                    cp_async_4(dst + kRows * Cfg::kWStride + lane * 4,
                               s + (static_cast<long long>(n.expert) * nbs + row / kScaleBlock) * kbs + kb, 4);
                }
                cp_async_arrive(&full[stage]);
            }
            armed |= 1u << stage;
            armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
        };
        // The activations of the same chunk.
        auto load_tokens = [&](bool first, const Unit &n, int ch, int at) {
            uint8_t *dst = ring + static_cast<size_t>(at) * p.stage_bytes + Cfg::kActOffset;
            const int k0 = ch * Cfg::kKC, k = min(Cfg::kKC, (first ? p.H : p.I) - k0);
            for (int i = lane; i < n.count; i += 32) {
                const int slot = r.order[n.start + i];
                if (first)
                    bulk_load(dst + i * Cfg::kXStride, static_cast<const uint16_t *>(p.X) + (slot / p.top_k) * p.ldx + k0, k * 2, &full[at]);
                else
                    bulk_load(dst + i * Cfg::kHStride, p.hidden + static_cast<long long>(slot) * p.I + k0, k * 4, &full[at]);
            }
        };
        auto next = [&] {
            if (++stage == p.stages) stage = 0, phase ^= 1u;
        };
        for (int u = blockIdx.x; ok && u < units1; u += gridDim.x) {
            const Unit n = first_unit(r, u, rg1);
            for (int ch = 0; ch < nch1; ++ch) {
                load_rows(true, n, ch);
                if (!ok) break;
                load_tokens(true, n, ch, stage);
                next();
            }
        }
        // Down projection: fill the ring with weights, wait for every CTA's h,
        // then hand the h rows of those stages in and go on.
        const int mine2 = shift < units2 ? (units2 - shift + static_cast<int>(gridDim.x) - 1) / gridDim.x : 0;
        const int total = mine2 * nch2, ahead = min(total, p.stages), stage0 = stage;
        for (int i = 0; ok && i < ahead; ++i) {
            load_rows(false, down_unit(r, shift + (i / nch2) * gridDim.x), i % nch2);
            if (ok) next();
        }
        if (ok && total > 0) {
            if (!__all_sync(0xffffffffu, wait_count(&p.counters[1], gridDim.x))) {
                if (lane == 0) give_up();
                ok = false;
            }
            fence_proxy_async_all();
        }
        for (int i = 0; ok && i < total; ++i) {
            const Unit n = down_unit(r, shift + (i / nch2) * gridDim.x);
            if (i < ahead) {
                load_tokens(false, n, i % nch2, (stage0 + i) % p.stages);
            } else {
                load_rows(false, n, i % nch2);
                if (!ok) break;
                load_tokens(false, n, i % nch2, stage);
                next();
            }
        }
        __syncwarp();
        // A stage whose h rows were never asked for cannot complete; its weight
        // copies are in flight all the same: give them the time of a bounded wait.
        if (lane == 0)
            for (int s = 0; s < p.stages; ++s)
                if ((armed & (1u << s)) && !mbar_wait(&full[s], (armed_parity >> s) & 1u, ok ? kWaitLimitNs : 10000000ull)) give_up();
        __syncwarp();
    } else {
        // ------------------------------------------------ arithmetic
        int stage = 0, buf = 0;
        uint32_t phase = 0;
        auto take = [&] {  // after a time-out everything runs through without waiting
            if (!abort_flag && !mbar_wait(&full[stage], phase)) give_up();
        };
        auto release = [&] {
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[stage]);
            if (++stage == p.stages) stage = 0, phase ^= 1u;
        };
        auto put = [&](const float (&acc)[NT][4]) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) red[buf][warp][n][i][lane] = acc[n][i];
        };
        auto total = [&](int n, int i, int l) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) s += red[buf][w][n][i][l];
            return s;
        };
        for (int u = blockIdx.x; u < units1; u += gridDim.x) {
            const Unit n = first_unit(r, u, rg1);
            float acc[NT][4] = {};
            for (int ch = 0; ch < nch1; ++ch) {
                take();
                multiply_chunk<XT, FP8, NT, true>(ring + static_cast<size_t>(stage) * p.stage_bytes, p.H - ch * Cfg::kKC, n.count, acc);
                release();
            }
            put(acc);
            consumer_sync();
            // fragment element i of lane l: row l / 4 + 8 (i / 2), token 2 (l % 4) + i % 2
            for (int x = threadIdx.x; x < NT * (GATED ? 64 : 128); x += 32 * kWarps) {
                const int i = GATED ? x & 1 : x & 3, l = (x >> (GATED ? 1 : 2)) & 31, nt = x / (GATED ? 64 : 128);
                const int tok = nt * 8 + 2 * (l & 3) + (i & 1);
                if (tok < n.count) {
                    float h = moe_act(p.act, total(nt, i, l));
                    if (GATED) h *= total(nt, i + 2, l);
                    const int row = n.rg * kUnitRows1 + (l >> 2) + (GATED ? 0 : 8 * (i >> 1));
                    p.hidden[static_cast<long long>(r.order[n.start + tok]) * p.I + row] = tf32_round(h);
                }
            }
            buf ^= 1;
        }
        fence_proxy_async_all();  // h is read by bulk copies
        __threadfence();
        consumer_sync();
        if (threadIdx.x == 0) atomicAdd(&p.counters[1], 1u);
        for (int u = shift; u < units2; u += gridDim.x) {
            const Unit n = down_unit(r, u);
            float acc[NT][4] = {};
            for (int ch = 0; ch < nch2; ++ch) {
                take();
                multiply_chunk<XT, FP8, NT, false>(ring + static_cast<size_t>(stage) * p.stage_bytes, p.I - ch * Cfg::kKC, n.count, acc);
                release();
            }
            put(acc);
            consumer_sync();
            for (int x = threadIdx.x; x < NT * 128; x += 32 * kWarps) {
                const int i = x & 3, l = (x >> 2) & 31, nt = x >> 7;
                const int tok = nt * 8 + 2 * (l & 3) + (i & 1);
                if (tok < n.count)
                    p.part[static_cast<long long>(r.order[n.start + tok]) * p.H + n.rg * kRows + (l >> 2) + 8 * (i >> 1)] = total(nt, i, l);
            }
            buf ^= 1;
            __threadfence();
            consumer_sync();
            if (threadIdx.x == 0) last = atomicAdd(&p.counters[4 + n.rg], 1u) == static_cast<unsigned>(r.pairs - 1);
            consumer_sync();
            if (last) {
                __threadfence();
                if (threadIdx.x == 0) p.counters[4 + n.rg] = 0u;
                if (!abort_flag)
                    for (int x = threadIdx.x; x < p.T * kRows; x += 32 * kWarps) {
                        const int t = x / kRows, c = n.rg * kRows + x % kRows;
                        float y = 0.f;
                        for (int j = 0; j < p.top_k; ++j) {
                            const int slot = t * p.top_k + j;
                            y = fmaf(r.weight[slot], __ldcg(p.part + static_cast<long long>(slot) * p.H + c), y);
                        }
                        store_out(p.Y, static_cast<size_t>(t) * p.ldy + c, p.y_type, y);
                    }
            }
        }
    }
    __syncthreads();
    // The last CTA to leave clears the barriers for the next call.
    if (threadIdx.x == 0 && atomicAdd(&p.counters[2], 1u) == gridDim.x - 1) p.counters[0] = p.counters[1] = p.counters[2] = 0u;
}

template <int XT, bool FP8, int NT, bool GATED>
cudaError_t launch_moe(MoeArgs a, cudaStream_t stream) {
    using Cfg = MoeCfg<FP8>;
    auto kern = moe_kernel<XT, FP8, NT, GATED>;
    a.tok_rows = std::min(a.T, 8 * NT);
    // a stage holds the rows and either kind of activations
    const int act_bytes = a.tok_rows * std::max(Cfg::kXStride, Cfg::kHStride);
    a.stage_bytes = (Cfg::kActOffset + act_bytes + 127) / 128 * 128;
    constexpr int kRing = 227 * 1024 - 1024 - static_cast<int>(sizeof(Routing) + 2 * kWarps * NT * 4 * 32 * 4 + 16 * kMaxStages + 64);
    static_assert(kRing >= kWarps * kMoeMaxExperts * 4, "the ring holds the keys of the choice");
    a.stages = std::min(kMaxStages, kRing / a.stage_bytes);
    static unsigned long long smem_set = 0;
    cudaError_t e = ensure_dynamic_smem(kern, kRing, smem_set);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeCooperative;
    attr.val.cooperative = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(device_sm_count());
    cfg.blockDim = dim3(kMoeThreads);
    cfg.dynamicSmemBytes = kRing;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kern, a);
    return e != cudaSuccess ? e : cudaPeekAtLastError();
}

template <int XT, bool FP8>
cudaError_t launch_moe_types(const MoeArgs &a, cudaStream_t stream) {
    return a.up ? launch_moe<XT, FP8, 1, true>(a, stream) : launch_moe<XT, FP8, 1, false>(a, stream);
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
    const size_t slots = static_cast<size_t>(m.T) * m.top_k;
    const size_t n_logits = (static_cast<size_t>(m.T) * m.E + 63) / 64 * 64, n_hidden = slots * m.I, n_part = slots * m.H;
    Scratch s;
    cudaError_t e = acquire_scratch(stream, n_logits + n_hidden + n_part, 4 + m.H / kRows, &s);
    if (e != cudaSuccess) return e;
    a.logits = s.partials;
    a.hidden = s.partials + n_logits;
    a.part = a.hidden + n_hidden;
    a.counters = s.counters;
    info->launches = 1;
    info->plan = "moe_few_tokens";
    const bool fp8 = m.w_type == kTypeE4M3;
    if (m.x_type == kOutF16)
        return fp8 ? launch_moe_types<kOutF16, true>(a, stream) : launch_moe_types<kOutF16, false>(a, stream);
    return fp8 ? launch_moe_types<kOutBF16, true>(a, stream) : launch_moe_types<kOutBF16, false>(a, stream);
}

}  // namespace gemm11

// fp8_gemm.cu -- the product of two matrices held in 8 bits with one FP32
// scale for each 128 of the contraction:
//
//   C[m, n] = act(alpha * sum_kb sa[kb, m] sb[kb, n] D_kb[m, n] + beta C + bias[n]),
//   D_kb[m, n] = sum over the 128 k of block kb of A[m, k] op(B)[k, n].
//
// D_kb has no scales in it, so the tensor core forms it (tcgen05.mma of
// kind::f8f6f4, FP32 accumulator in tensor memory) and the epilogue warps
// multiply it by sa sb and add it to running sums in FP32 registers.  That
// also keeps the tensor core's sums, which truncate, 128 long.  Two
// accumulators in tensor memory alternate: while the warps take one block's
// sums out, the tensor core forms the next.
//
// Two kernels, and a small one after the second:
//   fp8_tile_kernel   one CTA a tile, computed transposed, C^T = op(B)^T A^T:
//                     128 columns n of C on the MMA's row side (tensor-memory
//                     lanes), BN rows m on its column side, so that a few rows
//                     of A cost no more than BN >= M columns of accumulator and
//                     a warp stores 32 consecutive elements of a row of C.
//                     Bound by op(B)'s bytes and, with the matrices in the L2
//                     or the product short, by the call: 1 x 4096 x 4096 6.9 us,
//                     16 x 11008 x 4096 11.6 us, 4.0 TB/s, 64 rows 13.8 us;
//   fp8_pair_kernel   two CTAs (tcgen05 cta_group::2) a tile of 256 x 256,
//                     persistent, for many rows: 4096 x 11008 x 4096 148 us,
//                     2.5 PFLOP/s, its figures at the kernel.  Tiles that would
//                     leave most SMs idle are cut along k; fp8_join_kernel adds.
//
// Roles of a CTA: warp 0 issues the TMA loads (operand tiles with the 128-byte
// swizzle, and the BN scales of A for the block), warp 1 the MMAs, the others
// are the epilogue.  Too few tiles for the SMs: the k blocks of a tile are
// shared out over the CTAs of a cluster, whose partial sums are added in rank
// order through distributed shared memory.  Every wait is bounded.
#include <algorithm>
#include <cstdint>
#include <cmath>
#include <mutex>

#include <cudaTypedefs.h>

#include "fp8.cuh"
#include "fp8.h"

namespace gemm11 {
namespace {

constexpr int kPR = 128;                 // columns n of a tile: the MMA's row side
constexpr int kPBytes = kPR * kScaleBlock;  // 16 KB of op(B) for one k block

struct Fp8Args {
    int M, N, K, kb_total;
    float alpha, beta;
    const float *SB;
    long long sb_n, sb_kb;  // scale of B: SB[n index * sb_n + kb * sb_kb], n index = n or n / 128
    int b_rows;
    const float *bias;
    int act;
    void *C;
    long long ldc;
    int c_type;
    int c_vec;  // rows of C take aligned stores of 4 elements
    int tiles_m, splits;
    int p_mn;   // op(B)'s tile is MN-major (B stored K x N)
    uint32_t idesc;
    unsigned *err;
    unsigned long long wait_ns;
    size_t c_extent;  // checked by GEMM11_DEBUG builds
};

constexpr int tmem_cols_fp8(int n) { return n <= 32 ? 32 : n <= 64 ? 64 : n <= 128 ? 128 : n <= 256 ? 256 : 512; }

template <int BN, int STAGES>
struct Fp8Cfg {
    static constexpr int kEpi = BN < 64 ? 4 : 8;  // epilogue warps
    static constexpr int kPerSm = BN <= 64 ? 2 : 1;  // CTAs that an SM holds
    static constexpr int kThreads = 64 + 32 * kEpi;
    static constexpr int kCols = BN / (kEpi / 4);  // accumulator columns of a warp
    static constexpr int kQBytes = BN * kScaleBlock;
    static constexpr int kStageBytes = kPBytes + kQBytes;
    // Scales of A, one slot for each k block in flight.  The producer refills
    // block i's slot only after the MMA of block i - STAGES is complete, which
    // was issued after the epilogue had released block i - STAGES - 2, so
    // STAGES + 2 slots are never overwritten while in use.
    static constexpr int kSlots = STAGES + 2;
    static constexpr int kSlotFloats = BN < 32 ? 32 : BN;  // TMA writes start on 128 bytes
    static constexpr int kSmemBytes = 1024 + STAGES * kStageBytes + kSlots * kSlotFloats * 4 + (2 * STAGES + 5) * 8 + 16;
    static constexpr int kTmemCols = tmem_cols_fp8(2 * BN);
    static_assert(BN % 16 == 0 && BN >= 16 && BN <= 128, "MMA N, two accumulators");
    static_assert(STAGES * kStageBytes >= kPR * BN * 4, "the partial tile fits in the operand ring");
};

__device__ __forceinline__ void fp8_timeout(volatile int *abort_flag, unsigned *err) {
    *abort_flag = 1;
    atomicOr(err, kWatchdogTimeout);
}

// Four consecutive columns n.. of row m of C from their sums.
__device__ __forceinline__ void store4(const Fp8Args &p, int m, int n, float (&v)[4]) {
    const size_t ci = static_cast<size_t>(m) * static_cast<size_t>(p.ldc) + n;
    float cold[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool in = n + i < p.N;
        cold[i] = (p.beta != 0.f && in) ? load_out(p.C, ci + i, p.c_type) : 0.f;
        b[i] = (p.bias && in) ? __ldg(p.bias + n + i) : 0.f;
    }
    epilogue4(v, p.alpha, p.beta, cold, b, p.act);
    if (!debug_in_bounds(p.c_extent == 0 || ci + min(3, p.N - 1 - n) < p.c_extent, p.err)) return;
    if (p.c_vec && n + 4 <= p.N) {
        if (p.c_type == kOutF32)
            *reinterpret_cast<float4 *>(static_cast<float *>(p.C) + ci) = make_float4(v[0], v[1], v[2], v[3]);
        else
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.C) + ci) =
                make_uint2(pack2_out16(v[0], v[1], p.c_type), pack2_out16(v[2], v[3], p.c_type));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (n + i < p.N) store_out(p.C, ci + i, p.c_type, v[i]);
    }
}

template <int BN, int STAGES>
__global__ void __launch_bounds__(Fp8Cfg<BN, STAGES>::kThreads, Fp8Cfg<BN, STAGES>::kPerSm)
    fp8_tile_kernel(const __grid_constant__ CUtensorMap tm_p, const __grid_constant__ CUtensorMap tm_q,
                    const __grid_constant__ CUtensorMap tm_sq, const Fp8Args p) {
    using Cfg = Fp8Cfg<BN, STAGES>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sP = smem;
    uint8_t *sQ = smem + STAGES * kPBytes;
    float *sS = reinterpret_cast<float *>(sQ + STAGES * Cfg::kQBytes);
    uint64_t *full = reinterpret_cast<uint64_t *>(sS + Cfg::kSlots * Cfg::kSlotFloats);
    uint64_t *empty = full + STAGES;
    uint64_t *tfull = empty + STAGES;
    uint64_t *tempty = tfull + 2;
    uint64_t *mma_done = tempty + 2;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(mma_done + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], Cfg::kEpi);
        }
        mbar_init(mma_done, 1);
        *abort_flag = 0;
        fence_mbarrier_init();
        tma_prefetch_desc(&tm_p);
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_sq);
    }
    if (warp == 1) {
        tmem_alloc(tmem_holder, Cfg::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;
    pdl_wait();
    pdl_launch_dependents();

    // The M tiles of one 128-column panel of op(B) run next to each other.
    const int tile = blockIdx.x / p.splits, split = blockIdx.x % p.splits;
    const int n0 = (tile / p.tiles_m) * kPR, m0 = (tile % p.tiles_m) * BN;
    const int kb0 = static_cast<int>(static_cast<long long>(p.kb_total) * split / p.splits);
    const int kb1 = static_cast<int>(static_cast<long long>(p.kb_total) * (split + 1) / p.splits);
    const int q = warp & 3;                               // tensor-memory lane quarter
    const int col0 = ((warp - 2) >> 2) * Cfg::kCols;      // first accumulator column (epilogue warps)
    const int n = n0 + q * 32 + lane;
    uint64_t acc[Cfg::kCols / 2];  // pairs of accumulator columns (rows m of C)
    uint32_t armed = 0, armed_parity = 0;

    if (warp == 0) {
        // ------------------------------------------------ TMA producer
        int stage = 0, slot = 0;
        uint32_t phase = 0;
        for (int kb = kb0; kb < kb1 && !*abort_flag; ++kb) {
            if (!__all_sync(0xffffffffu, mbar_wait_patient(&empty[stage], phase ^ 1u, p.wait_ns))) {
                fp8_timeout(abort_flag, p.err);
                break;
            }
            const int k0 = kb * kScaleBlock;
            if (elect_one()) {
                mbar_arrive_expect_tx(&full[stage], Cfg::kStageBytes + BN * 4);
                if (p.p_mn)
                    tma_load_2d(&tm_p, &full[stage], sP + stage * kPBytes, n0, k0);
                else
                    tma_load_2d(&tm_p, &full[stage], sP + stage * kPBytes, k0, n0);
                tma_load_2d(&tm_q, &full[stage], sQ + stage * Cfg::kQBytes, k0, m0);
                tma_load_2d(&tm_sq, &full[stage], sS + slot * Cfg::kSlotFloats, m0, kb);
            }
            __syncwarp();
            armed |= 1u << stage;
            armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
            if (kDebugBuild && !__all_sync(0xffffffffu, mbar_wait(&empty[stage], phase, p.wait_ns))) {  // one stage in flight
                fp8_timeout(abort_flag, p.err);
                break;
            }
            if (++stage == STAGES) stage = 0, phase ^= 1u;
            if (++slot == Cfg::kSlots) slot = 0;
        }
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer
        // K-major: 128-byte rows, 8-row groups 1024 bytes apart, 32 k = 32
        // bytes along the row.  MN-major: 128 n bytes for each k, 8-k groups
        // 1024 bytes apart, 32 k = 4 groups.
        const uint64_t p_desc0 = umma_desc_sw128(smem_u32(sP), 16, 1024);
        const uint64_t q_desc0 = umma_desc_sw128(smem_u32(sQ), 16, 1024);
        const uint32_t p_step = p.p_mn ? 4096u >> 4 : 32u >> 4;
        int stage = 0;
        uint32_t phase = 0;
        for (int i = 0; i < kb1 - kb0; ++i) {
            const int buf = i & 1;
            if (!__all_sync(0xffffffffu, mbar_wait_patient(&full[stage], phase, p.wait_ns) &&
                                             mbar_wait_patient(&tempty[buf], ((i >> 1) & 1) ^ 1u, p.wait_ns))) {
                fp8_timeout(abort_flag, p.err);
                break;
            }
            tc_fence_after();
            const uint64_t pd = p_desc0 + static_cast<uint64_t>(stage * (kPBytes >> 4));
            const uint64_t qd = q_desc0 + static_cast<uint64_t>(stage * (Cfg::kQBytes >> 4));
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < kScaleBlock / 32; ++kk)
                    umma_f8(tmem_base + buf * BN, pd + p_step * kk, qd + 2u * kk, p.idesc, kk > 0 ? 1u : 0u);
                umma_commit(&tfull[buf]);
                umma_commit(&empty[stage]);
            }
            __syncwarp();
            if (++stage == STAGES) stage = 0, phase ^= 1u;
        }
    } else if (warp >= 2) {
        // ------------------------------------------------ epilogue: scale and add
#pragma unroll
        for (int j = 0; j < Cfg::kCols / 2; ++j) acc[j] = 0;
        // B's scale: of this lane's column, one block ahead; or, one for the
        // whole tile, of 32 blocks at once (lane l has block kb0 + l, + 32, ..).
        const float *sb = p.SB + (p.b_rows ? min(n, p.N - 1) : n0 / kScaleBlock) * p.sb_n + kb0 * p.sb_kb;
        const int blocks = kb1 - kb0;
        float s_next = p.b_rows ? (blocks > 0 ? __ldg(sb) : 0.f) : (lane < blocks ? __ldg(sb + lane * p.sb_kb) : 0.f), s_lane = 0.f;
        int slot = 0;
        for (int kb = kb0; kb < kb1; ++kb) {
            const int i = kb - kb0, buf = i & 1;
            float s;
            if (p.b_rows) {
                s = s_next;
                if (i + 1 < blocks) s_next = __ldg(sb + (i + 1) * p.sb_kb);
            } else {
                if ((i & 31) == 0) {
                    s_lane = s_next;
                    if (i + 32 + lane < blocks) s_next = __ldg(sb + (i + 32 + lane) * p.sb_kb);
                }
                s = __shfl_sync(0xffffffffu, s_lane, i & 31);
            }
            if (!mbar_wait_patient(&tfull[buf], (i >> 1) & 1, p.wait_ns)) {
                fp8_timeout(abort_flag, p.err);
                break;
            }
            tc_fence_after();
            const uint32_t t = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + buf * BN + col0;
            const uint32_t sa = smem_u32(sS + slot * Cfg::kSlotFloats + col0);
            const uint64_t ss = pack_f32x2(s, s);
            constexpr int kDeep = Cfg::kCols >= 32 ? 2 : 1;  // reads of 16 columns in flight
#pragma unroll
            for (int c = 0; c < Cfg::kCols / 16; c += kDeep) {
                uint32_t r[kDeep][16];
#pragma unroll
                for (int u = 0; u < kDeep; ++u) tmem_ld_32x32b_x16(t + (c + u) * 16, r[u]);
                tmem_wait_ld();
#pragma unroll
                for (int u = 0; u < kDeep; ++u) {
                    tmem_landed(r[u]);
                    uint64_t f[8];  // volatile: 16 columns' scales at a time
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(f[2 * j]), "=l"(f[2 * j + 1]) : "r"(sa + ((c + u) * 16 + 4 * j) * 4));
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        fma_f32x2(acc[(c + u) * 8 + j], mul_f32x2(ss, f[j]), pack_b32x2(r[u][2 * j], r[u][2 * j + 1]));
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tempty[buf]);
            if (++slot == Cfg::kSlots) slot = 0;
        }
        if (p.splits == 1 && !*abort_flag && n < p.N) {
            const float b_n = p.bias ? __ldg(p.bias + n) : 0.f;
            const float b4[4] = {b_n, b_n, b_n, b_n};
#pragma unroll
            for (int j = 0; j < Cfg::kCols; j += 4) {
                if (m0 + col0 + j >= p.M) break;
                float w[4], cold[4];
                unpack_f32x2(acc[j / 2], w[0], w[1]);
                unpack_f32x2(acc[j / 2 + 1], w[2], w[3]);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int m = m0 + col0 + j + k;
                    cold[k] = (p.beta != 0.f && m < p.M) ? load_out(p.C, static_cast<size_t>(m) * p.ldc + n, p.c_type) : 0.f;
                }
                epilogue4(w, p.alpha, p.beta, cold, b4, p.act);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const size_t ci = static_cast<size_t>(m0 + col0 + j + k) * p.ldc + n;
                    if (m0 + col0 + j + k < p.M && debug_in_bounds(p.c_extent == 0 || ci < p.c_extent, p.err))
                        store_out(p.C, ci, p.c_type, w[k]);
                }
            }
        }
    }

    // ---------------------------------------------------- drain: copies and MMAs of this CTA
    if (warp == 0 && lane == 0) {
        for (int s = 0; s < STAGES; ++s)
            if ((armed & (1u << s)) && !mbar_wait(&full[s], (armed_parity >> s) & 1u)) fp8_timeout(abort_flag, p.err);
    }
    if (warp == 1) {
        if (elect_one()) umma_commit(mma_done);  // by the lane that issued the MMAs
        __syncwarp();
        if (!mbar_wait_patient(mma_done, 0)) fp8_timeout(abort_flag, p.err);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem_base, Cfg::kTmemCols);
    }
    if (p.splits == 1) return;

    // ---------------------------------------------------- cluster split: add the partial tiles
    // The operand ring is idle now; each CTA's partial goes over it, row m of
    // C at m * 128 floats, and the CTAs take groups of four columns in turn.
    float *part = reinterpret_cast<float *>(smem);
    const int rows = min(BN, p.M - m0);
    if (warp >= 2) {
#pragma unroll
        for (int j = 0; j < Cfg::kCols; j += 2) {
            float lo, hi;
            unpack_f32x2(acc[j / 2], lo, hi);
            if (col0 + j < rows) part[(col0 + j) * kPR + q * 32 + lane] = lo;
            if (col0 + j + 1 < rows) part[(col0 + j + 1) * kPR + q * 32 + lane] = hi;
        }
    }
    cluster_sync();
    const uint32_t part_addr = smem_u32(part);
    if (!*abort_flag) {
        for (int i = split * Cfg::kThreads + threadIdx.x; i < rows * (kPR / 4); i += p.splits * Cfg::kThreads) {
            float v[4] = {0.f, 0.f, 0.f, 0.f};
            for (int r = 0; r < p.splits; ++r) {
                const float4 w = ld_shared_cluster_v4(mapa_shared(part_addr + i * 16, r));
                v[0] += w.x, v[1] += w.y, v[2] += w.z, v[3] += w.w;
            }
            const int nn = n0 + (i % (kPR / 4)) * 4;
            if (nn < p.N) store4(p, m0 + i / (kPR / 4), nn, v);
        }
    }
    __syncwarp();
    cluster_sync();  // a CTA's partial stays until every CTA has read it
}

// ------------------------------------------------------------------ CTA pairs
// A cluster of two CTAs computes 256 x 256 tiles of C: CTA r stages rows
// [m0 + 128 r, + 128) of A and columns [n0 + 128 r, + 128) of op(B), 32 KB for a
// k block; the even CTA's MMA thread multiplies the pair, and each CTA's own
// tensor memory receives the block's sums of its 128 rows x 256 columns, twice
// buffered (all 512 columns).  Eight epilogue warps hold the running sums, 128
// a thread: warp w has lane quarter w % 4 and one half of the columns.
//
// A block's columns are two MMA groups, each handed over by barriers of its
// own: group h multiplies columns [64 h, + 64) of both CTAs' parts of op(B), so
// its columns of C are n0 + 64 h + j and n0 + 128 + 64 h + j, j < 64.  From the
// last MMA of a group to the first of the same group two blocks later pass the
// commit (290 clocks), the epilogue's reads (300 - 400) and its answer (360);
// two groups in turn keep the tensor core busy meanwhile.
//
// Bound: what the TMA unit brings in and the tensor core reads from shared
// memory.  TMA delivers 43.6 bytes a clock to an SM, 750 clocks for a block; the
// groups read 64 KB and TMA writes 32 KB, 750 clocks at 128 bytes each; the
// multiplication itself takes 512 and the scaling 300.  Measured a block, from
// a tile's first to its last: 789 clocks (4096 x 11008 x 4096, 148 us), 776 with
// B stored K x N (1000 x 4096 x 11008, 40.5 us).  With a scale for each column
// 1,161 (4096 x 4096 x 4095, 91 us), and the epilogue is the bound: of 1,340
// clocks, counted with the tiles' ends, the second multiplication costs 150,
// reading the columns' scales 290, both 420.
constexpr int kPairStages = 5;
constexpr int kPairEpi = 8;
constexpr int kPairN = 256;
constexpr int kPairCols = kPairN * 4 / kPairEpi;  // of an epilogue warp, and of an MMA group
// Registers: the launch gives each of the 384 threads 168, 64,512 in all; the
// first warpgroup (TMA, MMA) keeps 56 and the epilogue takes 224 each:
// 128 * 56 + 256 * 224 = 64,512.
constexpr int kPairRegsFew = 56, kPairRegsMany = 224;

template <bool B_ROWS>
struct Fp8PairCfg {
    static constexpr int kThreads = 128 + 32 * kPairEpi;
    static constexpr int kHalfBytes = 128 * kScaleBlock;  // this CTA's rows of A, and columns of op(B)
    static constexpr int kStageBytes = 2 * kHalfBytes;
    static constexpr int kSlots = kPairStages + 3;  // as in Fp8Cfg, and one for reads after a block's release
    static constexpr int kSlotFloats = 128 + (B_ROWS ? kPairN : 0);
    static constexpr int kCStage = kPairEpi * 4096;  // staging of C, 4 KB a warp
    static constexpr int kSmemBytes =
        1024 + kPairStages * kStageBytes + kCStage + kSlots * kSlotFloats * 4 + (2 * kPairStages + 9) * 8 + 16;
};

struct Fp8PairArgs {
    Fp8Args a;
    int tiles_m, tiles_n, c_tma;
    // Units of work: `whole` tiles, then the k blocks of each remaining tile in
    // `parts` units, whose sums fp8_join_kernel adds.
    int units, whole, parts;
    int part_blocks;     // of a unit but the tile's last
    uint32_t per_tile;   // 65536 / parts, rounded up
    float *partials;  // 256 x 256 sums of each such unit
    size_t partial_floats;  // of them all, checked by GEMM11_DEBUG builds
};

// Unit t: its tile and its blocks of k (v is below 256, so that the product
// divides it exactly).
struct Fp8PairUnit {
    int tile, kb0, blocks;
};
template <bool PARTS>
__device__ __forceinline__ Fp8PairUnit fp8_pair_unit(const Fp8PairArgs &p, int t) {
    if (!PARTS || t < p.whole) return {t, 0, p.a.kb_total};
    const int v = t - p.whole, tile = static_cast<int>(static_cast<uint32_t>(v) * p.per_tile >> 16);
    const int kb0 = (v - tile * p.parts) * p.part_blocks;
    return {p.whole + tile, kb0, min(p.part_blocks, p.a.kb_total - kb0)};
}

// Tile t: groups of 8 pair rows, so that a wave of tiles shares its rows of A
// and columns of op(B) in L2.
__device__ __forceinline__ void fp8_pair_origin(const Fp8PairArgs &p, int t, int &m0, int &n0) {
    const int group = 8 * p.tiles_n;
    const int first = t / group * 8, rows = min(p.tiles_m - first, 8);
    m0 = (first + t % group % rows) * 256;
    n0 = t % group / rows * kPairN;
}

// act(alpha * v + beta * C + bias) of columns n .. n + 31 of row m; the whole
// warp together.  The GELU forms run as a rolled loop that rotates v by 8 a
// trip: a quarter of the code beside the main loop.
__device__ __forceinline__ void epilogue32(const Fp8Args &p, float (&v)[32], int m, int n, int lane) {
    const float bias = p.bias && n + lane < p.N ? __ldg(p.bias + n + lane) : 0.f;
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] *= p.alpha;
    if (p.beta != 0.f && m < p.M) {
        const size_t ci = static_cast<size_t>(m) * static_cast<size_t>(p.ldc) + n;
        if (p.c_type == kOutF32) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (n + j < p.N) v[j] = fmaf(p.beta, static_cast<const float *>(p.C)[ci + j], v[j]);
        } else {
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (n + j < p.N) v[j] = fmaf(p.beta, load_out(p.C, ci + j, p.c_type), v[j]);
        }
    }
    if (p.bias) {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] += __shfl_sync(0xffffffffu, bias, j);
    }
    if (p.act == 2) {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = fmaxf(v[j], 0.f);
    } else if (p.act != 0) {
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
            float t[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) t[i] = p.act == 1 ? gelu_erf(v[i]) : gelu_tanh(v[i]);
#pragma unroll
            for (int i = 0; i < 24; ++i) v[i] = v[i + 8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[24 + i] = t[i];
        }
    }
}

// 32 columns of this lane's row through the warp's staging buffer (128-byte
// rows, 128-byte swizzle): 32 columns of FP32, or 64 of a 16-bit type, of which
// `second` is the upper half.  A full buffer goes out by a TMA store, or, where
// the rows of C are not aligned for one, row by row with neighbouring lanes on
// neighbouring elements.
__device__ __forceinline__ void stage32(const Fp8Args &p, const float (&v)[32], const CUtensorMap *tm_c, bool wide, bool by_tma, uint8_t *staged,
                                        int lane, int row, int n, int n_end, int second) {
    if (wide || !second) {  // the buffer's last store has read it
        if (lane == 0) bulk_wait_read_all();
        __syncwarp();
    }
    uint8_t *mine = staged + lane * 128;
    if (wide) {
#pragma unroll
        for (int c = 0; c < 8; ++c)
            *reinterpret_cast<float4 *>(mine + ((c ^ (lane & 7)) << 4)) = make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
    } else {
#pragma unroll
        for (int c = 0; c < 4; ++c)
            *reinterpret_cast<uint4 *>(mine + (((c + 4 * second) ^ (lane & 7)) << 4)) =
                make_uint4(pack2_out16(v[8 * c], v[8 * c + 1], p.c_type), pack2_out16(v[8 * c + 2], v[8 * c + 3], p.c_type),
                           pack2_out16(v[8 * c + 4], v[8 * c + 5], p.c_type), pack2_out16(v[8 * c + 6], v[8 * c + 7], p.c_type));
    }
    if (!wide && !second) return;
    const int first = wide ? n : n - 32, esize = wide ? 4 : 2;
    if (by_tma) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            if (first < n_end) tma_store_2d(tm_c, staged, first, row);
            bulk_commit();
        }
        return;
    }
    __syncwarp();
    constexpr int kRowsAtOnce = 8;  // reads of so many rows before their stores
    for (int r0 = 0; r0 < 32 && row + r0 < p.M; r0 += kRowsAtOnce) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int j = u * 32 + lane;
            if (j * esize >= 128 || first + j >= p.N) continue;
            float w[kRowsAtOnce];
#pragma unroll
            for (int k = 0; k < kRowsAtOnce; ++k) {
                const uint8_t *at = staged + (r0 + k) * 128 + ((((j * esize) >> 4) ^ k) << 4) + (j * esize & 15);
                w[k] = wide ? *reinterpret_cast<const float *>(at) : __uint_as_float(*reinterpret_cast<const uint16_t *>(at));
            }
#pragma unroll
            for (int k = 0; k < kRowsAtOnce; ++k) {
                if (row + r0 + k >= p.M) break;
                const size_t ci = static_cast<size_t>(row + r0 + k) * static_cast<size_t>(p.ldc) + first + j;
                if (!debug_in_bounds(p.c_extent == 0 || ci < p.c_extent, p.err)) continue;
                if (wide)
                    static_cast<float *>(p.C)[ci] = w[k];
                else
                    static_cast<uint16_t *>(p.C)[ci] = static_cast<uint16_t>(__float_as_uint(w[k]));
            }
        }
    }
    __syncwarp();
}

// acc[col ..] += s * r, 32 columns.
__device__ __forceinline__ void add_scaled(uint64_t (&acc)[kPairCols / 2], int col, const uint32_t (&r)[32], uint64_t ss) {
#pragma unroll
    for (int u = 0; u < 16; ++u) fma_f32x2(acc[col / 2 + u], ss, pack_b32x2(r[2 * u], r[2 * u + 1]));
}
// acc[col ..] += s * f * r, 16 columns, f their scales.
__device__ __forceinline__ void add_scaled(uint64_t (&acc)[kPairCols / 2], int col, const uint32_t (&r)[16], uint64_t ss,
                                           const uint64_t (&f)[8]) {
#pragma unroll
    for (int u = 0; u < 8; ++u) fma_scaled_f32x2(acc[col / 2 + u], ss, f[u], r[2 * u], r[2 * u + 1]);
}
// The scales of 16 columns (volatile: in order with the sums).
__device__ __forceinline__ void load_col_scales(uint64_t (&f)[8], uint32_t at) {
#pragma unroll
    for (int u = 0; u < 4; ++u)
        asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(f[2 * u]), "=l"(f[2 * u + 1]) : "r"(at + 16 * u));
}

template <bool B_ROWS, bool PARTS>
__global__ void __launch_bounds__(Fp8PairCfg<B_ROWS>::kThreads, 1)
    fp8_pair_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                    const __grid_constant__ CUtensorMap tm_sa, const __grid_constant__ CUtensorMap tm_sb,
                    const __grid_constant__ CUtensorMap tm_c, const __grid_constant__ CUtensorMap tm_parts,
                    const Fp8PairArgs pp) {
    using Cfg = Fp8PairCfg<B_ROWS>;
    const Fp8Args &p = pp.a;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sA = smem, *sB = smem + kPairStages * Cfg::kHalfBytes, *sC = sB + kPairStages * Cfg::kHalfBytes;
    float *sS = reinterpret_cast<float *>(sC + Cfg::kCStage);
    uint64_t *full = reinterpret_cast<uint64_t *>(sS + Cfg::kSlots * Cfg::kSlotFloats);
    uint64_t *empty = full + kPairStages;
    uint64_t *tfull = empty + kPairStages;
    uint64_t *tempty = tfull + 4;  // [buffer][group], as tfull
    uint64_t *mma_done = tempty + 4;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(mma_done + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int cid = blockIdx.x >> 1, ncl = gridDim.x >> 1;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kPairStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 2);  // both MMA warps
        }
        for (int b = 0; b < 4; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], kPairEpi);  // half the warps of both CTAs
        }
        mbar_init(mma_done, 2);
        *abort_flag = 0;
        fence_mbarrier_init();
        tma_prefetch_desc(&tm_a);
        tma_prefetch_desc(&tm_b);
        tma_prefetch_desc(&tm_sa);
        tma_prefetch_desc(&tm_c);
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_holder, 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;
    pdl_wait();
    pdl_launch_dependents();
    uint32_t armed = 0, armed_parity = 0;
    if (warp < 4) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPairRegsFew));
      if (warp == 0) {
        // ------------------------------------------------ TMA producer (both CTAs)
        const uint32_t tx = Cfg::kStageBytes + 512 + (B_ROWS ? kPairN * 4 : 0);
        int stage = 0, slot = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int t = cid; ok && t < pp.units && !*abort_flag; t += ncl) {
            const Fp8PairUnit unit = fp8_pair_unit<PARTS>(pp, t);
            int m0, n0;
            fp8_pair_origin(pp, unit.tile, m0, n0);
            const int my_m = m0 + static_cast<int>(rank) * 128, my_n = n0 + static_cast<int>(rank) * 128;
            for (int kb = unit.kb0; kb < unit.kb0 + unit.blocks; ++kb) {
                ok = __all_sync(0xffffffffu, mbar_wait_patient(&empty[stage], phase ^ 1u, p.wait_ns));
                if (!ok) {
                    fp8_timeout(abort_flag, p.err);
                    break;
                }
                const uint32_t bar = mapa_shared(smem_u32(&full[stage]), 0);
                const int k0 = kb * kScaleBlock;
                if (elect_one()) {
                    float *sc = sS + slot * Cfg::kSlotFloats;
                    if (leader) mbar_arrive_expect_tx(&full[stage], 2 * tx);
                    tma_load_2d_pair(&tm_a, bar, sA + stage * Cfg::kHalfBytes, k0, my_m);
                    if (p.p_mn)
                        tma_load_2d_pair(&tm_b, bar, sB + stage * Cfg::kHalfBytes, my_n, k0);
                    else
                        tma_load_2d_pair(&tm_b, bar, sB + stage * Cfg::kHalfBytes, k0, my_n);
                    tma_load_2d_pair(&tm_sa, bar, sc, my_m, kb);
                    if (B_ROWS) tma_load_2d_pair(&tm_sb, bar, sc + 128, n0, kb);
                }
                __syncwarp();
                armed |= 1u << stage;
                armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
                if (kDebugBuild) {  // one stage in flight
                    ok = __all_sync(0xffffffffu, mbar_wait(&empty[stage], phase, p.wait_ns));
                    if (!ok) {
                        fp8_timeout(abort_flag, p.err);
                        break;
                    }
                }
                if (++stage == kPairStages) stage = 0, phase ^= 1u;
                if (++slot == Cfg::kSlots) slot = 0;
            }
        }
      } else if (warp < 3 && leader) {
        // ------------------------------------------------ MMA issuers (even CTA), one for each group
        // A warp's waits and instructions for a group take 500 - 600 clocks a
        // block beside the epilogue's arithmetic, so one warp for both groups
        // would set the pace (920 clocks a block).
        const int h = warp - 1;
        const uint32_t b_step = p.p_mn ? 4096u >> 4 : 32u >> 4;
        const uint32_t b_group = h * (p.p_mn ? 64 : 64 * 128);  // bytes to the group's columns
        const uint64_t a_desc0 = umma_desc_sw128(smem_u32(sA), 16, 1024);
        const uint64_t b_desc0 = umma_desc_sw128(smem_u32(sB) + b_group, 16, 1024);
        const uint32_t d0 = tmem_base + h * kPairCols;
        int stage = 0, i = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int t = cid; ok && t < pp.units && !*abort_flag; t += ncl) {
            const int blocks = fp8_pair_unit<PARTS>(pp, t).blocks;
            for (int kb = 0; kb < blocks; ++kb, ++i) {
                const int buf = i & 1;
                ok = __all_sync(0xffffffffu, mbar_wait_patient(&full[stage], phase, p.wait_ns) &&
                                                 mbar_wait_patient(&tempty[buf * 2 + h], ((i >> 1) & 1) ^ 1u, p.wait_ns));
                if (!ok) {
                    fp8_timeout(abort_flag, p.err);
                    break;
                }
                tc_fence_after();
                const uint64_t ad = a_desc0 + static_cast<uint64_t>(stage * (Cfg::kHalfBytes >> 4));
                const uint64_t bd = b_desc0 + static_cast<uint64_t>(stage * (Cfg::kHalfBytes >> 4));
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < kScaleBlock / 32; ++kk)
                        umma_f8_pair(d0 + buf * kPairN, ad + 2u * kk, bd + b_step * kk, p.idesc, kk > 0 ? 1u : 0u);
                    umma_commit_pair_mc(&tfull[buf * 2 + h], 0x3);
                    umma_commit_pair_mc(&empty[stage], 0x3);
                }
                __syncwarp();
                if (++stage == kPairStages) stage = 0, phase ^= 1u;
            }
        }
      }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPairRegsMany));
        // ------------------------------------------------ epilogue (both CTAs)
        const int q = warp & 3, part = (warp - 4) >> 2;
        const uint32_t t_row = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + part * kPairCols;
        const uint32_t release[2] = {mapa_shared(smem_u32(&tempty[part]), 0), mapa_shared(smem_u32(&tempty[2 + part]), 0)};
        uint8_t *const staged = sC + (warp - 4) * 4096;
        int i = 0, slot = 0;
        bool ok = true;
        GEMM11_TMEM_AHEAD_REGISTERS();
        for (int t = cid; ok && t < pp.units && !*abort_flag; t += ncl) {
            const Fp8PairUnit unit = fp8_pair_unit<PARTS>(pp, t);
            // The shuffle keeps the compiler from carrying the unit's choice into
            // the loop below (1,000 clocks a block without it, 815 with, counted
            // with the tiles' ends).
            const int blocks = PARTS ? __shfl_sync(0xffffffffu, unit.blocks, 0) : p.kb_total;
            int m0, n0;
            fp8_pair_origin(pp, unit.tile, m0, n0);
            // Columns col + j and col + 128 + j, j < 64.
            int row = m0 + static_cast<int>(rank) * 128 + q * 32, col = n0 + part * 64;
            uint64_t acc[kPairCols / 2];  // pairs of columns
#pragma unroll
            for (int j = 0; j < kPairCols / 2; ++j) acc[j] = 0;
            // B's scales of the two 128-column blocks: lane l has those of k
            // blocks l, l + 32, .., and the next 32 are on their way.
            const float *sb = p.SB + unit.kb0 * p.sb_kb;
            const float *sb0 = sb + (B_ROWS ? 0 : min(col, p.N - 1) / kScaleBlock * p.sb_n);
            const float *sb1 = sb + (B_ROWS ? 0 : min(col + 128, p.N - 1) / kScaleBlock * p.sb_n);
            float lane0 = 1.f, lane1 = 1.f, next0 = 1.f, next1 = 1.f;
            if (!B_ROWS && lane < blocks) next0 = __ldg(sb0 + lane * p.sb_kb), next1 = __ldg(sb1 + lane * p.sb_kb);
            // While the sums of one read (32 columns, 16 with a scale for each
            // column) are added the next is on its way, over the end of a block
            // too, there in registers of its own (GEMM11_TMEM_AHEAD_REGISTERS).
            // A wait is for every read, so only one is in flight: with two
            // each wait paid for the later one (3 % for 4096 x 11008 x 4096).
            // The accumulator goes back as soon as the block's last read is in.
            // The registers of its own cost 3.5 % there (148 us against 143 with
            // a variable), turning the loop so that none is in flight where it
            // comes round 20 %.
            constexpr int kStep = B_ROWS ? 16 : 32;
            uint32_t r0[kStep], r1[kStep];
            uint64_t fa[8], fb[8];
            auto take = [&] {  // the next block's accumulator
                ok = mbar_wait_patient(&tfull[(i & 1) * 2 + part], (i >> 1) & 1, p.wait_ns);
                if (!ok) fp8_timeout(abort_flag, p.err);
                tc_fence_after();
            };
            take();
            tmem_ld_ahead<kStep>(t_row + (i & 1) * kPairN);
            for (int kb = 0; kb < blocks; ++kb) {
                const uint32_t from = t_row + (i & 1) * kPairN, answer = release[i & 1];
                float s0 = 1.f, s1 = 1.f;
                if (!B_ROWS) {
                    if ((kb & 31) == 0) {
                        lane0 = next0, lane1 = next1;
                        if (kb + 32 + lane < blocks)
                            next0 = __ldg(sb0 + (kb + 32 + lane) * p.sb_kb), next1 = __ldg(sb1 + (kb + 32 + lane) * p.sb_kb);
                    }
                    s0 = __shfl_sync(0xffffffffu, lane0, kb & 31), s1 = __shfl_sync(0xffffffffu, lane1, kb & 31);
                }
                const float *sc = sS + slot * Cfg::kSlotFloats;
                s0 *= sc[q * 32 + lane], s1 *= sc[q * 32 + lane];
                const uint64_t ss0 = pack_f32x2(s0, s0), ss1 = pack_f32x2(s1, s1);
                // columns from 64 on are 64 further in C's tile
                const uint32_t sbv = smem_u32(sc + 128 + part * 64), sbw = sbv + 64 * 4;
                if constexpr (B_ROWS) {
                    // each step's scales are read during the step before
                    load_col_scales(fa, sbv);
                    tmem_wait_ahead(r0);
                    tmem_ld<kStep>(from + 16, r1);
                    load_col_scales(fb, sbv + 16 * 4);
                    add_scaled(acc, 0, r0, ss0, fa);
                    tmem_wait_ld(r1);
                    tmem_ld<kStep>(from + 32, r0);
                    load_col_scales(fa, sbv + 32 * 4);
                    add_scaled(acc, 16, r1, ss0, fb);
                    tmem_wait_ld(r0);
                    tmem_ld<kStep>(from + 48, r1);
                    load_col_scales(fb, sbv + 48 * 4);
                    add_scaled(acc, 32, r0, ss0, fa);
                    tmem_wait_ld(r1);
                    tmem_ld<kStep>(from + 64, r0);
                    load_col_scales(fa, sbw + 64 * 4);
                    add_scaled(acc, 48, r1, ss0, fb);
                    tmem_wait_ld(r0);
                    tmem_ld<kStep>(from + 80, r1);
                    load_col_scales(fb, sbw + 80 * 4);
                    add_scaled(acc, 64, r0, ss0, fa);
                    tmem_wait_ld(r1);
                    tmem_ld<kStep>(from + 96, r0);
                    load_col_scales(fa, sbw + 96 * 4);
                    add_scaled(acc, 80, r1, ss0, fb);
                    tmem_wait_ld(r0);
                    tmem_ld<kStep>(from + 112, r1);
                    load_col_scales(fb, sbw + 112 * 4);
                    add_scaled(acc, 96, r0, ss0, fa);
                } else {
                    tmem_wait_ahead(r0);
                    tmem_ld<kStep>(from + 32, r1);
                    add_scaled(acc, 0, r0, ss0);
                    tmem_wait_ld(r1);
                    tmem_ld<kStep>(from + 64, r0);
                    add_scaled(acc, 32, r1, ss0);
                    tmem_wait_ld(r0);
                    tmem_ld<kStep>(from + 96, r1);
                    add_scaled(acc, 64, r0, ss1);
                }
                tmem_wait_ld(r1);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote(answer);
                ++i;
                const bool more = kb + 1 < blocks;
                if (more) {
                    take();
                    if (!ok) break;
                    tmem_ld_ahead<kStep>(t_row + (i & 1) * kPairN);
                }
                if constexpr (B_ROWS)
                    add_scaled(acc, 112, r1, ss0, fb);
                else
                    add_scaled(acc, 96, r1, ss1);
                if (++slot == Cfg::kSlots) slot = 0;
            }
            tmem_wait_ld();
            if (!ok || row >= p.M) continue;
            // The unit is done: 32 columns at a time to the epilogue and out, or
            // as they are to the partial sums.
            const bool some = PARTS && t >= pp.whole;
            if (some) row = (t - pp.whole) * 256 + static_cast<int>(rank) * 128 + q * 32, col = part * 64;
            if (some && !debug_in_bounds((row + 32u) * static_cast<size_t>(kPairN) <= pp.partial_floats, p.err)) continue;
            const int m = row + lane;
#pragma unroll
            for (int gr = 0; gr < kPairCols / 32; ++gr) {
                const int n = col + (gr & 1) * 32 + (gr >> 1) * 128;
                float v[32];
#pragma unroll
                for (int j = 0; j < 16; ++j) unpack_f32x2(acc[gr * 16 + j], v[2 * j], v[2 * j + 1]);
                if (!some) epilogue32(p, v, m, n, lane);
                stage32(p, v, some ? &tm_parts : &tm_c, some || p.c_type == kOutF32, some || pp.c_tma, staged, lane, row, n,
                        some ? kPairN : p.N, gr & 1);
            }
        }
        if (lane == 0) bulk_wait_all();
        __syncwarp();
    }

    // ---------------------------------------------------- drain and unwind
    if (warp == 0 && lane == 0 && leader) {
        // the even CTA's full barriers count the copies of both CTAs
        for (int s = 0; s < kPairStages; ++s)
            if ((armed & (1u << s)) && !mbar_wait(&full[s], (armed_parity >> s) & 1u)) fp8_timeout(abort_flag, p.err);
    }
    if ((warp == 1 || warp == 2) && leader) {
        // the electing lane issued the MMAs that the commit waits for
        if (elect_one()) umma_commit_pair_mc(mma_done, 0x1);
        __syncwarp();
        if (!mbar_wait(mma_done, 0)) fp8_timeout(abort_flag, p.err);
    }
    tc_fence_before();
    __syncwarp();
    cluster_sync();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, 512);
    }
}

// The tiles whose k the pair kernel's units shared: the parts' sums added in the
// order of k, and the epilogue.  Four columns a thread.
__global__ void __launch_bounds__(256) fp8_join_kernel(const Fp8PairArgs pp) {
    pdl_wait();
    pdl_launch_dependents();
    constexpr int kPieces = 256 * kPairN / 4;  // of a tile
    const int left = blockIdx.x / (kPieces / 256), at = blockIdx.x % (kPieces / 256) * 256 + threadIdx.x;
    int m, n;
    fp8_pair_origin(pp, pp.whole + left, m, n);
    m += at / (kPairN / 4), n += at % (kPairN / 4) * 4;
    if (m >= pp.a.M || n >= pp.a.N) return;
    const float4 *from = reinterpret_cast<const float4 *>(pp.partials) + static_cast<size_t>(left) * pp.parts * kPieces + at;
    if (!debug_in_bounds((static_cast<size_t>(left + 1) * pp.parts - 1) * kPieces + at < pp.partial_floats / 4, pp.a.err)) return;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int part = 0; part < pp.parts; ++part) {
        const float4 w = __ldcg(from + static_cast<size_t>(part) * kPieces);
        v[0] += w.x, v[1] += w.y, v[2] += w.z, v[3] += w.w;
    }
    store4(pp.a, m, n, v);
}

// C = act(beta * C + bias), where there is no product.
__global__ void __launch_bounds__(256) fp8_scale_c_kernel(const Fp8Args p) {
    pdl_wait();
    pdl_launch_dependents();
    const long long groups = (p.N + 3) / 4, total = groups * p.M;
    for (long long i = blockIdx.x * 256LL + threadIdx.x; i < total; i += gridDim.x * 256LL) {
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        store4(p, static_cast<int>(i / groups), static_cast<int>(i % groups) * 4, v);
    }
}

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &r) == cudaSuccess &&
            r == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    });
    return fn;
}

Fp8Args fp8_args(const Fp8Gemm &g) {
    Fp8Args a = {};
    a.M = g.M;
    a.N = g.N;
    a.K = g.K;
    a.kb_total = (g.K + kScaleBlock - 1) / kScaleBlock;
    a.alpha = g.alpha;
    a.beta = g.beta;
    a.SB = g.SB;
    a.b_rows = g.b_rows;
    a.sb_n = g.b_rows ? 1 : (g.b_trans ? g.ldsb : 1);
    a.sb_kb = g.b_rows ? g.ldsb : (g.b_trans ? 1 : g.ldsb);
    a.bias = g.bias;
    a.act = g.act;
    a.C = g.C;
    a.ldc = g.ldc;
    a.c_type = g.c_type;
    const int cb = g.c_type == kOutF32 ? 4 : 2;
    a.c_vec = reinterpret_cast<uintptr_t>(g.C) % (4 * cb) == 0 && (g.M == 1 || g.ldc % 4 == 0);
    a.p_mn = g.b_trans ? 0 : 1;
    a.err = watchdog_word();
    a.wait_ns = kWaitLimitNs;
    a.splits = 1;
    if (kDebugBuild) {
        a.c_extent = static_cast<size_t>(g.M - 1) * static_cast<size_t>(g.ldc) + g.N;
        a.c_extent -= std::min(a.c_extent - 1, debug_shrink_c());
    }
    return a;
}

template <int BN, int STAGES>
cudaError_t launch_fp8_tile(const Fp8Gemm &g, Fp8Args a, cudaStream_t stream) {
    using Cfg = Fp8Cfg<BN, STAGES>;
    auto kern = fp8_tile_kernel<BN, STAGES>;
    static unsigned long long smem_set = 0;
    cudaError_t e = ensure_dynamic_smem(kern, Cfg::kSmemBytes, smem_set);
    if (e != cudaSuccess) return e;
    CUtensorMap tp, tq, ts;
    const auto sw = CU_TENSOR_MAP_SWIZZLE_128B;
    const auto u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    const bool ok =
        (g.b_trans ? encode_matrix_map(&tp, u8, g.B, g.K, g.N, g.ldb, kScaleBlock, kPR, sw)
                   : encode_matrix_map(&tp, u8, g.B, g.N, g.K, g.ldb, kPR, kScaleBlock, sw)) &&
        encode_matrix_map(&tq, u8, g.A, g.K, g.M, g.lda, kScaleBlock, BN, sw) &&
        encode_matrix_map(&ts, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, g.SA, g.M, a.kb_total, g.ldsa * 4, BN, 1,
                          CU_TENSOR_MAP_SWIZZLE_NONE);
    if (!ok) return cudaErrorNotSupported;
    a.idesc = umma_idesc_f8(kPR, BN, g.b_type == kTypeE5M2, g.a_type == kTypeE5M2, a.p_mn, 0);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(a.splits);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((g.N + kPR - 1) / kPR) * a.tiles_m * a.splits);
    cfg.blockDim = dim3(Cfg::kThreads);
    cfg.dynamicSmemBytes = Cfg::kSmemBytes;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = a.splits > 1 ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, kern, tp, tq, ts, a);
    return e != cudaSuccess ? e : cudaPeekAtLastError();
}

// Clusters of `splits` CTAs of fp8_tile_kernel<BN, STAGES> that the GPU holds
// at once (cached; one device type per process).
template <int BN, int STAGES>
int tile_clusters(int splits) {
    static int cap[9] = {-1, -1, -1, -1, -1, -1, -1, -1, -1};  // atomic accesses: planners may run concurrently
    const int known = __atomic_load_n(&cap[splits], __ATOMIC_ACQUIRE);
    if (known >= 0) return known;
    using Cfg = Fp8Cfg<BN, STAGES>;
    auto kern = fp8_tile_kernel<BN, STAGES>;
    static unsigned long long smem_set = 0;
    int n = 0;
    if (ensure_dynamic_smem(kern, Cfg::kSmemBytes, smem_set) == cudaSuccess) {
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = static_cast<unsigned>(splits);
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(splits * 2 * device_sm_count());
        cfg.blockDim = dim3(Cfg::kThreads);
        cfg.dynamicSmemBytes = Cfg::kSmemBytes;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
            (void)cudaGetLastError();
            n = 0;
        }
    }
    __atomic_store_n(&cap[splits], n, __ATOMIC_RELEASE);
    return n;
}

// K splits of single-CTA tiles.  A model of measured times, in us: 4.5 for the
// call, a block in every wave of CTAs (0.47 with 128 columns of accumulator,
// where its scaling counts; 0.25 with up to 64, two CTAs an SM), and for a split
// 1.5 and the partial tile's bytes from the other CTAs at 32 GB/s.  Measured /
// modelled: 128 x 4096 x 4096 in 4 splits 9.9 / 10.3, 256 x 4096 x 4096 in 2
// 14.0 / 14.5, 128 x 19456 x 11008 whole 44.7 / 44.9.  With 128 columns all
// clusters have to fit at once: 512 x 512 x 11008 in 16 clusters of 8 CTAs, of
// which some had to wait, took 20.4 us, as long as two waves (12.8 in fewer
// splits).  Smaller tiles are bound by memory and do not mind: 16 x 11008 x 4096
// takes 8.3 us in 3 splits, not all of them at once, and 10.7 in 2.
int pick_splits(int bn, int tiles, int blocks, int rows, int sms, double *time_us) {
    const int room = sms * (bn <= 64 ? 2 : 1);  // CTAs at a time
    const double block_us = bn <= 64 ? 0.25 : 0.47;
    int best = 1;
    double best_t = 4.5 + std::ceil(static_cast<double>(tiles) / room) * blocks * block_us;
    for (int s = 2; s <= 8 && s <= blocks; ++s) {
        if (static_cast<long long>(tiles) * s > room || (bn > 64 && tiles > tile_clusters<128, 6>(s))) break;
        const double t = 4.5 + (blocks + s - 1) / s * block_us + 1.5 + rows * kPR * 4.0 * (s - 1) / s / 32e3;
        if (t < best_t) best_t = t, best = s;
    }
    *time_us = best_t;
    return best;
}

// Pair tiles on `clusters`: whole waves, and what they leave over, whose tiles may
// be cut into units along k (a second kernel adds them).  A block of k takes 0.44
// us, 0.70 with a scale for each column; a cut the second launch and the way
// through memory, 4.5 us where it is all there is, 12 after a wave (whose last
// tiles run faster than a full wave, and whose end the next launch fills in
// part), and 0.16 for each part.  Measured, whole tiles / cut: 2560 x 2048 x 8192
// (80 tiles) 56.3 / 42.9 us, with a scale for each column 84.4 / 60.6; 1024 x
// 1024 x 8192 (16) 20.3 in single-CTA tiles / 17.6, and 22.9 / 21.4; left whole
// 4096 x 11008 x 4096 (688) 148.0 / 149.5, 4096 x 4096 x 4096 (256) 62.1 / 64.6.
// The two models are off by a microsecond or so: 512 x 512 x 11008 (4) takes 13.1
// in single-CTA tiles and 14.7 cut, which is taken where clusters of 7 CTAs do
// not all fit at once.
struct PairPlan {
    int left, parts;  // tiles to cut, units of each
    double time_us;
};
PairPlan pair_plan(double tiles, int clusters, int blocks, bool b_rows) {
    const double block_us = b_rows ? 0.70 : 0.44, waves = std::floor(tiles / clusters);
    const int left = static_cast<int>(tiles - waves * clusters);
    PairPlan best = {0, 1, left ? blocks * block_us : 0.0};
    for (int s = 2; left && s <= blocks && s * left <= clusters; ++s) {
        const int each = (blocks + s - 1) / s;
        const double t = each * block_us + (waves > 0 ? 12.0 : 4.5) + 0.16 * s;
        if (t < best.time_us) best = {left, (blocks + each - 1) / each, t};
    }
    best.time_us += 4.5 + waves * blocks * block_us;
    return best;
}

template <bool B_ROWS, bool PARTS>
cudaError_t launch_fp8_pair(const Fp8Gemm &g, const Fp8Args &a, const PairPlan &plan, cudaStream_t stream, CallInfo *info) {
    using Cfg = Fp8PairCfg<B_ROWS>;
    auto kern = fp8_pair_kernel<B_ROWS, PARTS>;
    static int max_clusters = -1;  // one device type per process; atomic accesses
    static unsigned long long smem_set = 0;
    cudaError_t e = ensure_dynamic_smem(kern, Cfg::kSmemBytes, smem_set);
    if (e != cudaSuccess) return e;
    Fp8PairArgs args = {};
    args.a = a;
    args.tiles_m = (g.M + 255) / 256;
    args.tiles_n = (g.N + kPairN - 1) / kPairN;
    const int cb = g.c_type == kOutF32 ? 4 : 2;
    // TMA stores of C need aligned rows; any other C is stored element by element.
    args.c_tma = reinterpret_cast<uintptr_t>(g.C) % 16 == 0 && g.ldc * cb % 16 == 0;
    args.a.idesc = umma_idesc_f8(256, kPairCols, g.a_type == kTypeE5M2, g.b_type == kTypeE5M2, 0, a.p_mn);
    CUtensorMap ta, tb, tsa, tsb, tc;
    const auto sw = CU_TENSOR_MAP_SWIZZLE_128B, none = CU_TENSOR_MAP_SWIZZLE_NONE;
    const auto u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8, f32 = CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
    const auto ct = g.c_type == kOutF32 ? f32 : g.c_type == kOutF16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    bool ok = encode_matrix_map(&ta, u8, g.A, g.K, g.M, g.lda, kScaleBlock, 128, sw) &&
              (g.b_trans ? encode_matrix_map(&tb, u8, g.B, g.K, g.N, g.ldb, kScaleBlock, 128, sw)
                         : encode_matrix_map(&tb, u8, g.B, g.N, g.K, g.ldb, 128, kScaleBlock, sw)) &&
              encode_matrix_map(&tsa, f32, g.SA, g.M, a.kb_total, g.ldsa * 4, 128, 1, none);
    tsb = tsa;
    tc = ta;  // not used without TMA stores
    if (ok && B_ROWS) ok = encode_matrix_map(&tsb, f32, g.SB, g.N, a.kb_total, g.ldsb * 4, kPairN, 1, none);
    if (ok && args.c_tma) ok = encode_matrix_map(&tc, ct, g.C, g.N, g.M, g.ldc * cb, 128 / cb, 32, sw);
    if (!ok) return cudaErrorNotSupported;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(Cfg::kThreads);
    cfg.dynamicSmemBytes = Cfg::kSmemBytes;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int clusters = __atomic_load_n(&max_clusters, __ATOMIC_ACQUIRE);
    if (clusters < 0) {
        cfg.gridDim = dim3(2 * device_sm_count());
        e = cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg);
        if (e != cudaSuccess) return e;
        __atomic_store_n(&max_clusters, clusters, __ATOMIC_RELEASE);
    }
    if (clusters < 1) return cudaErrorNotSupported;
    args.parts = plan.parts;
    args.whole = args.tiles_m * args.tiles_n - plan.left;
    args.part_blocks = (a.kb_total + args.parts - 1) / args.parts;
    args.per_tile = (65536 + args.parts - 1) / args.parts;
    args.units = args.whole + plan.left * args.parts;
    CUtensorMap tp = ta;  // not used without parts
    if (PARTS) {
        const int rows = plan.left * args.parts * 256;
        Scratch sc;
        e = acquire_scratch(stream, static_cast<size_t>(rows) * kPairN, 0, info, &sc);
        if (e != cudaSuccess) return e;
        args.partials = sc.partials;
        args.partial_floats = static_cast<size_t>(rows) * kPairN;
        if (!encode_matrix_map(&tp, f32, sc.partials, kPairN, rows, kPairN * 4, 32, 32, sw)) return cudaErrorNotSupported;
    }
    cfg.gridDim = dim3(2 * std::min(clusters, args.units));
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, kern, ta, tb, tsa, tsb, tc, tp, args);
    if (e == cudaSuccess) e = cudaPeekAtLastError();
    if (e != cudaSuccess || !PARTS) return e;
    info->launches = 2;
    cfg.gridDim = dim3(plan.left * 64);
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    cfg.attrs = attr + 1;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, fp8_join_kernel, args);
    return e != cudaSuccess ? e : cudaPeekAtLastError();
}

}  // namespace

bool encode_matrix_map(CUtensorMap *map, CUtensorMapDataType dt, const void *base, uint64_t inner, uint64_t outer,
                       uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer, CUtensorMapSwizzle swizzle) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t dims[2] = {inner, outer};
    cuuint64_t strides[1] = {(row_bytes + 15) / 16 * 16};  // a single row has no stride of its own
    cuuint32_t box[2] = {box_inner, box_outer};
    cuuint32_t estr[2] = {1, 1};
    return enc(map, dt, 2, const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_box_map(CUtensorMap *map, CUtensorMapDataType dt, const void *base, uint64_t inner, uint64_t rows, uint64_t steps,
                    uint64_t row_bytes, uint64_t step_bytes, uint32_t box_inner, uint32_t box_rows, uint32_t box_steps) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {inner, rows, steps};
    cuuint64_t strides[2] = {row_bytes, step_bytes};
    cuuint32_t box[3] = {box_inner, box_rows, box_steps};
    cuuint32_t estr[3] = {1, 1, 1};
    return enc(map, dt, 3, const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t run_fp8_gemm(const Fp8Gemm &g, cudaStream_t stream, CallInfo *info) {
    Fp8Args a = fp8_args(g);
    const int bn = g.M <= 16 ? 16 : g.M <= 32 ? 32 : g.M <= 64 ? 64 : 128;
    a.tiles_m = (g.M + bn - 1) / bn;
    const long long tiles = static_cast<long long>((g.N + kPR - 1) / kPR) * a.tiles_m;
    const int sms = device_sm_count();
    double t_tile = 0.0;
    a.splits = pick_splits(bn, static_cast<int>(std::min<long long>(tiles, 1 << 30)), a.kb_total, std::min(bn, g.M), sms, &t_tile);
    info->launches = 1;
    const double pair_tiles = static_cast<double>((g.M + 255) / 256) * ((g.N + kPairN - 1) / kPairN);
    const PairPlan pairs = pair_plan(pair_tiles, sms / 2, a.kb_total, g.b_rows);
    if (g.M > 128 && pairs.time_us <= t_tile) {
        info->plan = pairs.left ? "fp8_pair_256x256_splitk" : "fp8_pair_256x256";
        a.splits = pairs.parts;
        if (pairs.left)
            return g.b_rows ? launch_fp8_pair<true, true>(g, a, pairs, stream, info) : launch_fp8_pair<false, true>(g, a, pairs, stream, info);
        return g.b_rows ? launch_fp8_pair<true, false>(g, a, pairs, stream, info) : launch_fp8_pair<false, false>(g, a, pairs, stream, info);
    }
    switch (bn) {
        case 16: info->plan = "fp8_tile_n16"; return launch_fp8_tile<16, 5>(g, a, stream);
        case 32: info->plan = "fp8_tile_n32"; return launch_fp8_tile<32, 5>(g, a, stream);
        case 64: info->plan = "fp8_tile_n64"; return launch_fp8_tile<64, 4>(g, a, stream);
        default: info->plan = "fp8_tile_n128"; return launch_fp8_tile<128, 6>(g, a, stream);
    }
}

cudaError_t run_fp8_scale_c(const Fp8Gemm &g, cudaStream_t stream, CallInfo *info) {
    const Fp8Args a = fp8_args(g);
    const long long groups = static_cast<long long>((g.N + 3) / 4) * g.M;
    const unsigned grid = static_cast<unsigned>(std::min<long long>((groups + 255) / 256, 8LL * device_sm_count()));
    info->plan = "fp8_scale_c";
    info->launches = 1;
    return launch_kernel(fp8_scale_c_kernel, dim3(grid), dim3(256), 0, stream, a);
}

}  // namespace gemm11

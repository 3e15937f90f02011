// grouped.cu -- the products of a mixture-of-experts layer over rows that are
// sorted by expert, rows offsets[e] .. offsets[e + 1] - 1 belonging to expert e:
//
//   rows     C[r] = alpha A[r] op(B[e]) + beta C[r]       (the forward product, with
//            B[e] stored N x K, and the gradient of the rows, with B[e] K x N),
//   weights  C[e] = alpha A[rows of e]^T B[rows of e] + beta C[e].
//
// FP16 or BF16 operands, FP32 sums.  The offsets are on the device and the host
// does not know them: a CTA pair takes every ncl-th tile of a list that each warp
// works out for itself, 32 experts at a time, one a lane.
#include <algorithm>
#include <cstdint>

#include "experts.h"
#include "fp8.cuh"
#include "fp8.h"

namespace gemm11 {
namespace {

constexpr int kKB = 64;                   // of the contraction a block: 128 bytes
constexpr int kHalf = 128 * kKB * 2;      // this CTA's 128 rows (or columns) of one operand, 16 KB
constexpr int kBox = 64 * kKB * 2;        // 64 columns of an operand stored along the tile
constexpr int kStages = 6;
constexpr int kTile = 256;
constexpr int kEpi = 8;                   // epilogue warps
constexpr int kCols = kTile * 4 / kEpi;   // accumulator columns of one
// The tensor core's sums truncate; so many blocks (512 of the contraction) are
// summed there, and these sums are added to nearest in FP32 registers.
constexpr int kChunk = 8;
// Registers: 384 threads of 168 at launch, 64,512; 128 x 56 + 256 x 224 = 64,512.
constexpr int kRegsFew = 56, kRegsMany = 224;
constexpr int kThreads = 128 + 32 * kEpi;
constexpr int kBars = 2 * kStages + 4 + 3;
constexpr int kSmemBytes = 1024 + kStages * 2 * kHalf + kEpi * 4096 + kBars * 8 + 16;
static_assert(kSmemBytes <= 232448, "shared memory of a CTA");

enum Mode { kRowsNT, kRowsNN, kWeights };

struct GroupedArgs {
    int E, R;
    int m, n, k;  // weights: C[e] is m x n; rows: n columns, contraction k
    const int *offsets;
    float alpha, beta;
    void *C;
    long long ldc, stride_c;
    int c_type, c_tma;
    int tiles_m, tiles_n;  // weights: of every expert; rows: tiles_n
    int product;           // 0: C = beta C
    uint32_t idesc;
    unsigned *err;
    unsigned long long wait_ns;
    size_t c_extent;  // checked by GEMM11_DEBUG builds
};

// A tile of C: rows [m0, row_end) of expert e from column n0, and its contraction.
struct Tile {
    int e, m0, n0, row_end;
    int k0, k1;  // rows of the contraction (weights), or 0 and k
};

// Groups of 8 tile rows, so that a wave of tiles shares its rows and columns in L2.
__device__ __forceinline__ void tile_origin(int i, int tiles_m, int tiles_n, int &m0, int &n0) {
    const int group = 8 * tiles_n;
    const int first = i / group * 8, rows = min(tiles_m - first, 8);
    m0 = (first + i % group % rows) * kTile;
    n0 = i % group / rows * kTile;
}

// The list of tiles, walked forwards by a whole warp: lane l has expert e0 + l.
template <int MODE>
struct TileList {
    int e0 = 0, base = 0;  // tiles before expert e0
    int start = 0, end = 0, tiles = 0, incl = 0;

    __device__ __forceinline__ void window(const GroupedArgs &p, int lane) {
        start = end = tiles = 0;
        if (e0 + lane < p.E) {
            start = min(max(__ldg(p.offsets + e0 + lane), 0), p.R);
            end = min(max(__ldg(p.offsets + e0 + lane + 1), start), p.R);
            tiles = MODE == kWeights ? p.tiles_m * p.tiles_n : ((end - start + kTile - 1) / kTile) * p.tiles_n;
        }
        incl = tiles;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += o;
        }
    }
    // Tile t; false behind the last.
    __device__ __forceinline__ bool find(const GroupedArgs &p, int t, int lane, Tile &tile) {
        for (;;) {
            const int total = __shfl_sync(0xffffffffu, incl, 31);
            if (t - base < total) break;
            base += total;
            e0 += 32;
            if (e0 >= p.E) return false;
            window(p, lane);
        }
        const int src = __ffs(__ballot_sync(0xffffffffu, incl > t - base)) - 1;
        const int before = __shfl_sync(0xffffffffu, incl - tiles, src);
        const int s = __shfl_sync(0xffffffffu, start, src), e = __shfl_sync(0xffffffffu, end, src);
        tile.e = e0 + src;
        if (MODE == kWeights) {
            tile_origin(t - base - before, p.tiles_m, p.tiles_n, tile.m0, tile.n0);
            tile.row_end = p.m;
            tile.k0 = s, tile.k1 = e;
        } else {
            tile_origin(t - base - before, (e - s + kTile - 1) / kTile, p.tiles_n, tile.m0, tile.n0);
            tile.m0 += s;
            tile.row_end = e;
            tile.k0 = 0, tile.k1 = p.k;
        }
        if (!p.product) tile.k1 = tile.k0;
        return true;
    }
};

__device__ __forceinline__ int tile_blocks(const Tile &t) { return (t.k1 - t.k0 + kKB - 1) / kKB; }

__device__ __forceinline__ void grouped_timeout(volatile int *abort_flag, unsigned *err) {
    *abort_flag = 1;
    atomicOr(err, kWatchdogTimeout);
}

// 32 columns of this lane's row through the warp's staging buffer (128-byte
// rows, 128-byte swizzle): 32 columns of FP32, or 64 of a 16-bit type, of which
// `second` is the upper half.  A full buffer goes out by a TMA store, or, where
// C's rows are not aligned for one or some of the 32 rows are another expert's,
// row by row with neighbouring lanes on neighbouring elements.
__device__ __forceinline__ void store32(const GroupedArgs &p, const float (&v)[32], const CUtensorMap *tm_c, bool by_tma, uint8_t *staged, int lane,
                                        int e, int row, int row_end, int n, int second) {
    const bool wide = p.c_type == kOutF32;
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
            if (first < p.n) tma_store_3d(tm_c, staged, first, row, e);
            bulk_commit();
        }
        return;
    }
    __syncwarp();
    constexpr int kRowsAtOnce = 8;  // reads of so many rows before their stores
    for (int r0 = 0; r0 < 32 && row + r0 < row_end; r0 += kRowsAtOnce) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int j = u * 32 + lane;
            if (j * esize >= 128 || first + j >= p.n) continue;
            float w[kRowsAtOnce];
#pragma unroll
            for (int k = 0; k < kRowsAtOnce; ++k) {
                const uint8_t *at = staged + (r0 + k) * 128 + ((((j * esize) >> 4) ^ k) << 4) + (j * esize & 15);
                w[k] = wide ? *reinterpret_cast<const float *>(at) : __uint_as_float(*reinterpret_cast<const uint16_t *>(at));
            }
#pragma unroll
            for (int k = 0; k < kRowsAtOnce; ++k) {
                if (row + r0 + k >= row_end) break;
                const size_t ci = static_cast<size_t>(e * p.stride_c) + static_cast<size_t>(row + r0 + k) * static_cast<size_t>(p.ldc) + first + j;
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

// CTA pairs (clusters of two) on tiles of 256 x 256: CTA r stages 128 rows of
// the tile and 128 of its columns, 32 KB a block of 64; the even CTA's MMA warp
// multiplies the pair, and each CTA's tensor memory receives its 128 rows x 256
// columns, twice buffered.  Warp 0 issues the copies, warp 1 the MMAs, warps 4 to
// 11 are the epilogue: warp w has lane quarter w % 4 and half of the columns,
// whose sums over the chunks it holds in registers.
//
// The contraction of the weights' gradient ends at any row of A and B, and
// behind it are the next expert's.  Both CTAs take the last block of 64 rows to a
// barrier of their own, zero what is behind the end in shared memory (a row is
// 128 bytes there, the swizzle moves bytes within it) and hand the block on.
template <int MODE>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_pair_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b, const __grid_constant__ CUtensorMap tm_c,
                        const GroupedArgs p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sA = smem, *sB = smem + kStages * kHalf, *sC = sB + kStages * kHalf;
    uint64_t *full = reinterpret_cast<uint64_t *>(sC + kEpi * 4096);
    uint64_t *empty = full + kStages;
    uint64_t *tfull = empty + kStages;
    uint64_t *tempty = tfull + 2;
    uint64_t *mma_done = tempty + 2;
    uint64_t *tail = mma_done + 1, *tail_peer = tail + 1;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(tail_peer + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int cid = blockIdx.x >> 1, ncl = gridDim.x >> 1;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], 2 * kEpi);  // the warps of both CTAs
        }
        mbar_init(mma_done, 1);
        mbar_init(tail, 1);
        mbar_init(tail_peer, 1);
        *abort_flag = 0;
        fence_mbarrier_init();
        if (p.product) {
            tma_prefetch_desc(&tm_a);
            tma_prefetch_desc(&tm_b);
        }
        if (p.c_tma) tma_prefetch_desc(&tm_c);
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
    uint32_t armed = 0, armed_parity = 0, tails = 0;
    TileList<MODE> list;
    Tile tile;
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsFew));
        if (warp == 0) {
            // ------------------------------------------------ TMA producer (both CTAs)
            list.window(p, lane);
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int t = cid; ok && !*abort_flag && list.find(p, t, lane, tile); t += ncl) {
                const int my_m = tile.m0 + static_cast<int>(rank) * 128, my_n = tile.n0 + static_cast<int>(rank) * 128;
                const int blocks = tile_blocks(tile);
                for (int kb = 0; kb < blocks; ++kb) {
                    ok = __all_sync(0xffffffffu, mbar_wait_patient(&empty[stage], phase ^ 1u, p.wait_ns));
                    if (!ok) {
                        grouped_timeout(abort_flag, p.err);
                        break;
                    }
                    const int k0 = tile.k0 + kb * kKB;
                    uint8_t *a = sA + stage * kHalf, *b = sB + stage * kHalf;
                    const int valid = tile.k1 - k0;
                    if (MODE == kWeights && valid < kKB) {
                        if (elect_one()) {
                            mbar_arrive_expect_tx(tail, 2 * kHalf);
                            tma_load_2d(&tm_a, tail, a, my_m, k0);
                            tma_load_2d(&tm_a, tail, a + kBox, my_m + 64, k0);
                            tma_load_2d(&tm_b, tail, b, my_n, k0);
                            tma_load_2d(&tm_b, tail, b + kBox, my_n + 64, k0);
                        }
                        __syncwarp();
                        ++tails;
                        ok = __all_sync(0xffffffffu, mbar_wait_patient(tail, (tails - 1) & 1u, p.wait_ns));
                        if (!ok) {
                            grouped_timeout(abort_flag, p.err);
                            break;
                        }
                        for (int i = valid * 8 + lane; i < kKB * 8; i += 32) {
                            const uint4 zero = make_uint4(0, 0, 0, 0);
                            reinterpret_cast<uint4 *>(a)[i] = zero;
                            reinterpret_cast<uint4 *>(a + kBox)[i] = zero;
                            reinterpret_cast<uint4 *>(b)[i] = zero;
                            reinterpret_cast<uint4 *>(b + kBox)[i] = zero;
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (leader) {
                            ok = __all_sync(0xffffffffu, mbar_wait_cluster(tail_peer, (tails - 1) & 1u, p.wait_ns));
                            if (!ok) {
                                grouped_timeout(abort_flag, p.err);
                                break;
                            }
                            if (elect_one()) mbar_arrive(&full[stage]);
                        } else if (elect_one()) {
                            mbar_arrive_cluster(mapa_shared(smem_u32(tail_peer), 0));
                        }
                        __syncwarp();
                    } else {
                        const uint32_t bar = mapa_shared(smem_u32(&full[stage]), 0);
                        if (elect_one()) {
                            if (leader) mbar_arrive_expect_tx(&full[stage], 4 * kHalf);
                            if (MODE == kWeights) {
                                tma_load_2d_pair(&tm_a, bar, a, my_m, k0);
                                tma_load_2d_pair(&tm_a, bar, a + kBox, my_m + 64, k0);
                                tma_load_2d_pair(&tm_b, bar, b, my_n, k0);
                                tma_load_2d_pair(&tm_b, bar, b + kBox, my_n + 64, k0);
                            } else {
                                tma_load_2d_pair(&tm_a, bar, a, k0, my_m);
                                if (MODE == kRowsNT) {
                                    tma_load_3d_pair(&tm_b, bar, b, k0, my_n, tile.e);
                                } else {
                                    tma_load_3d_pair(&tm_b, bar, b, my_n, k0, tile.e);
                                    tma_load_3d_pair(&tm_b, bar, b + kBox, my_n + 64, k0, tile.e);
                                }
                            }
                        }
                        __syncwarp();
                    }
                    armed |= 1u << stage;
                    armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
                    if (kDebugBuild) {  // one stage in flight
                        ok = __all_sync(0xffffffffu, mbar_wait(&empty[stage], phase, p.wait_ns));
                        if (!ok) {
                            grouped_timeout(abort_flag, p.err);
                            break;
                        }
                    }
                    if (++stage == kStages) stage = 0, phase ^= 1u;
                }
            }
        } else if (warp == 1 && leader) {
            // ------------------------------------------------ MMA issuer (even CTA)
            // K-major: 128-byte rows, 8-row groups 1024 bytes apart, 16 k = 32
            // bytes along the row.  Stored along the tile: 128 bytes (64
            // columns) for each k, boxes of 64 columns kBox apart, 16 k = 2048
            // bytes.
            constexpr bool kAmn = MODE == kWeights, kBmn = MODE != kRowsNT;
            const uint64_t a_desc0 = umma_desc_sw128(smem_u32(sA), kAmn ? kBox : 16, 1024);
            const uint64_t b_desc0 = umma_desc_sw128(smem_u32(sB), kBmn ? kBox : 16, 1024);
            constexpr uint32_t kAstep = kAmn ? 2048 >> 4 : 32 >> 4, kBstep = kBmn ? 2048 >> 4 : 32 >> 4;
            list.window(p, lane);
            int stage = 0, i = 0;  // i: chunk
            uint32_t phase = 0;
            bool ok = true;
            for (int t = cid; ok && !*abort_flag && list.find(p, t, lane, tile); t += ncl) {
                const int blocks = tile_blocks(tile);
                for (int kb0 = 0; ok && kb0 < blocks; kb0 += kChunk, ++i) {
                    const int buf = i & 1, some = min(kChunk, blocks - kb0);
                    ok = __all_sync(0xffffffffu, mbar_wait_patient(&tempty[buf], ((i >> 1) & 1) ^ 1u, p.wait_ns));
                    if (!ok) {
                        grouped_timeout(abort_flag, p.err);
                        break;
                    }
                    tc_fence_after();
                    for (int kb = 0; kb < some; ++kb) {
                        ok = __all_sync(0xffffffffu, mbar_wait_patient(&full[stage], phase, p.wait_ns));
                        if (!ok) {
                            grouped_timeout(abort_flag, p.err);
                            break;
                        }
                        tc_fence_after();
                        const uint64_t ad = a_desc0 + static_cast<uint64_t>(stage * (kHalf >> 4));
                        const uint64_t bd = b_desc0 + static_cast<uint64_t>(stage * (kHalf >> 4));
                        if (elect_one()) {
#pragma unroll
                            for (int kk = 0; kk < kKB / 16; ++kk)
                                umma_f16_pair(tmem_base + buf * kTile, ad + kAstep * kk, bd + kBstep * kk, p.idesc, kb > 0 || kk > 0 ? 1u : 0u);
                            umma_commit_pair_mc(&empty[stage], 0x3);
                            if (kb == some - 1) umma_commit_pair_mc(&tfull[buf], 0x3);
                        }
                        __syncwarp();
                        if (++stage == kStages) stage = 0, phase ^= 1u;
                    }
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsMany));
        // ------------------------------------------------ epilogue (both CTAs)
        const int q = warp & 3, part = (warp - 4) >> 2;
        const uint32_t t_row = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + part * kCols;
        const uint32_t release[2] = {mapa_shared(smem_u32(&tempty[0]), 0), mapa_shared(smem_u32(&tempty[1]), 0)};
        uint8_t *const staged = sC + (warp - 4) * 4096;
        list.window(p, lane);
        int i = 0;
        bool ok = true;
        for (int t = cid; ok && !*abort_flag && list.find(p, t, lane, tile); t += ncl) {
            const int chunks = (tile_blocks(tile) + kChunk - 1) / kChunk;
            const int row = tile.m0 + static_cast<int>(rank) * 128 + q * 32, col = tile.n0 + part * kCols;
            float acc[kCols];
#pragma unroll
            for (int j = 0; j < kCols; ++j) acc[j] = 0.f;
            for (int c = 0; c < chunks; ++c, ++i) {
                const int buf = i & 1;
                ok = __all_sync(0xffffffffu, mbar_wait_patient(&tfull[buf], (i >> 1) & 1, p.wait_ns));
                if (!ok) {
                    grouped_timeout(abort_flag, p.err);
                    break;
                }
                tc_fence_after();
                const uint32_t from = t_row + buf * kTile;
#pragma unroll
                for (int g = 0; g < kCols / 32; ++g) {
                    uint32_t r[32];
                    tmem_ld_32x32b_x32(from + g * 32, r);
                    tmem_wait_ld(r);
#pragma unroll
                    for (int j = 0; j < 32; ++j) acc[g * 32 + j] += __uint_as_float(r[j]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote(release[buf]);
            }
            if (!ok || row >= tile.row_end) continue;
            const int m = row + lane;
            const bool by_tma = p.c_tma && (MODE == kWeights || row + 32 <= tile.row_end);
            const int e = MODE == kWeights ? tile.e : 0;
#pragma unroll
            for (int g = 0; g < kCols / 32; ++g) {
                const int n = col + g * 32;
                float v[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = p.alpha * acc[g * 32 + j];
                if (p.beta != 0.f && m < tile.row_end) {
                    const size_t ci = static_cast<size_t>(e * p.stride_c) + static_cast<size_t>(m) * static_cast<size_t>(p.ldc) + n;
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (n + j < p.n) v[j] = fmaf(p.beta, load_out(p.C, ci + j, p.c_type), v[j]);
                }
                store32(p, v, &tm_c, by_tma, staged, lane, e, row, tile.row_end, n, g & 1);
            }
        }
        if (lane == 0) bulk_wait_all();
        __syncwarp();
    }

    // ---------------------------------------------------- drain and unwind
    if (warp == 0 && lane == 0) {
        if (MODE == kWeights && tails > 0 && !mbar_wait(tail, (tails - 1) & 1u)) grouped_timeout(abort_flag, p.err);
        // the even CTA's full barriers count the copies of both CTAs
        for (int s = 0; s < kStages; ++s)
            if (leader && (armed & (1u << s)) && !mbar_wait(&full[s], (armed_parity >> s) & 1u)) grouped_timeout(abort_flag, p.err);
    }
    if (warp == 1 && leader) {
        // the electing lane issued the MMAs that the commit waits for
        if (elect_one()) umma_commit_pair_mc(mma_done, 0x1);
        __syncwarp();
        if (!mbar_wait(mma_done, 0)) grouped_timeout(abort_flag, p.err);
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

template <int MODE>
cudaError_t launch_grouped_pair(const Grouped &g, GroupedArgs a, cudaStream_t stream) {
    auto kern = grouped_pair_kernel<MODE>;
    static int max_clusters = -1;  // one device type per process; atomic accesses
    static unsigned long long smem_set = 0;
    cudaError_t e = ensure_dynamic_smem(kern, kSmemBytes, smem_set);
    if (e != cudaSuccess) return e;
    const auto sw = CU_TENSOR_MAP_SWIZZLE_128B;
    const auto t16 = g.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const auto ct = g.c_type == kOutF32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : g.c_type == kOutF16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    // Strides that nothing has (of a single row, of a single expert) may be any.
    auto stride = [](long long elements, int bytes) { return static_cast<uint64_t>((elements * bytes + 15) / 16 * 16); };
    CUtensorMap ta = {}, tb = {}, tc = {};
    bool ok = true;
    if (a.product) {
        if (MODE == kWeights) {
            ok = encode_matrix_map(&ta, t16, g.A, g.M, g.R, stride(g.lda, 2), 64, kKB, sw) && encode_matrix_map(&tb, t16, g.B, g.N, g.R, stride(g.ldb, 2), 64, kKB, sw);
        } else {
            const uint64_t step = stride(g.stride_b, 2);
            ok = encode_matrix_map(&ta, t16, g.A, g.K, g.R, stride(g.lda, 2), kKB, 128, sw) &&
                 (MODE == kRowsNT ? encode_box_map(&tb, t16, g.B, g.K, g.N, g.E, stride(g.ldb, 2), step, kKB, 128, 1)
                                  : encode_box_map(&tb, t16, g.B, g.N, g.K, g.E, stride(g.ldb, 2), step, 64, kKB, 1));
        }
    }
    const int cb = g.c_type == kOutF32 ? 4 : 2;
    a.c_tma = reinterpret_cast<uintptr_t>(g.C) % 16 == 0 && g.ldc * cb % 16 == 0 && g.ldc < (1LL << 38) &&
              (MODE != kWeights || g.E == 1 || (g.stride_c * cb % 16 == 0 && g.stride_c < (1LL << 38)));
    if (ok && a.c_tma)
        ok = MODE == kWeights ? encode_box_map(&tc, ct, g.C, g.N, g.M, g.E, stride(g.ldc, cb), stride(g.stride_c, cb), 128 / cb, 32, 1)
                              : encode_box_map(&tc, ct, g.C, g.N, g.R, 1, stride(g.ldc, cb), stride(g.ldc, cb), 128 / cb, 32, 1);
    if (!ok) return cudaErrorNotSupported;
    a.tiles_m = (g.M + kTile - 1) / kTile;
    a.tiles_n = (g.N + kTile - 1) / kTile;
    a.idesc = umma_idesc_f16_f32(256, kTile, MODE == kWeights, MODE != kRowsNT) | (g.bf16 ? kIdescBf16Operands : 0u);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
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
    const long long most = MODE == kWeights ? static_cast<long long>(g.E) * a.tiles_m * a.tiles_n : (g.R / kTile + static_cast<long long>(std::min(g.E, g.R))) * a.tiles_n;
    cfg.gridDim = dim3(2 * static_cast<unsigned>(std::min<long long>(clusters, most)));
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, kern, ta, tb, tc, a);
    return e != cudaSuccess ? e : cudaPeekAtLastError();
}

}  // namespace

cudaError_t run_grouped(const Grouped &g, cudaStream_t stream, CallInfo *info) {
    GroupedArgs a = {};
    a.E = g.E;
    a.R = g.R;
    a.m = g.M;
    a.n = g.N;
    a.k = g.K;
    a.offsets = g.offsets;
    a.alpha = g.alpha;
    a.beta = g.beta;
    a.C = g.C;
    a.ldc = g.ldc;
    a.stride_c = g.wgrad ? g.stride_c : 0;
    a.c_type = g.c_type;
    a.product = g.alpha != 0.f && (g.wgrad ? g.R > 0 : g.K > 0);
    a.err = watchdog_word();
    a.wait_ns = kWaitLimitNs;
    if (kDebugBuild) {
        a.c_extent = g.wgrad ? static_cast<size_t>((g.E - 1LL) * g.stride_c + (g.M - 1LL) * g.ldc + g.N) : static_cast<size_t>((g.R - 1LL) * g.ldc + g.N);
        a.c_extent -= std::min(a.c_extent - 1, debug_shrink_c());
    }
    info->launches = 1;
    if (g.wgrad) {
        info->plan = "grouped_wgrad_pair_256x256";
        return launch_grouped_pair<kWeights>(g, a, stream);
    }
    info->plan = "grouped_pair_256x256";
    return g.b_trans ? launch_grouped_pair<kRowsNT>(g, a, stream) : launch_grouped_pair<kRowsNN>(g, a, stream);
}

}  // namespace gemm11

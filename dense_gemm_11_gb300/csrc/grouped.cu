// grouped.cu -- the products of a mixture-of-experts layer over rows that are
// sorted by expert, rows offsets[e] .. offsets[e + 1] - 1 belonging to expert e:
//
//   rows     C[r] = alpha A[r] op(B[e]) + beta C[r]       (the forward product, with
//            B[e] stored N x K, and the gradient of the rows, with B[e] K x N),
//   weights  C[e] = alpha A[rows of e]^T B[rows of e] + beta C[e].
//
// FP16 or BF16 operands, FP32 sums.  The offsets are on the device and the host
// does not know them: a CTA pair takes every ncl-th tile of a list that one warp of
// each CTA works out, 32 experts at a time, one a lane, ahead of the others.
//
// Bound: the tensor core at the clock that the power limit leaves, for long
// contractions (8192 rows over 8 experts of 4096 x 4096 158 us, 1.74 PFLOP/s; the
// weights' gradient with 4096 rows an expert 590 us for 32768 rows, 1.86); the
// weights' bytes for few rows (2400 rows over 64 experts of 2048 x 2048 88.3 us,
// 6.3 TB/s); both at once between (24,570 rows over 64 experts of 2048 x 1024 82
// us: 54 of multiplication, 62 of memory).  Results in FP32 beside a contraction of
// 1000 rows are bound by neither: 8 experts of 4096 x 4096 with 8192 rows take 202
// us, in BF16 175, without stores as long as their multiplication; the MMAs wait
// for operands, whose copies wait while the results are on their way to memory.
#include <algorithm>
#include <cstdint>

#include "experts.h"
#include "fp8.cuh"
#include "fp8.h"
#include "rows8.cuh"

namespace gemm11 {
namespace {

constexpr int kKB = 64;                   // of the contraction a block: 128 bytes
constexpr int kHalf = 128 * kKB * 2;      // one CTA's part of an operand, 16 KB
constexpr int kBox = 64 * kKB * 2;        // 64 columns of an operand stored along the tile
constexpr int kStages = 7;                // 5: 64 experts, 6 rows each 47.5 -> 49.3 us
constexpr int kTile = 256;
constexpr int kEpi = 8;                   // epilogue warps
constexpr int kCols = kTile * 4 / kEpi;   // accumulator columns of one
// The tensor core's sums truncate; so many blocks (512 of the contraction) are
// summed there, and these sums are added to nearest in FP32 registers.  In a row of
// calls that takes 8192 rows over 8 experts of 11008 x 4096 from 444 us, with all of a
// contraction summed there, to 448 (weights of some 2^-6), and the error of an FP32
// result over 11008 from 1.2e-5 of its norm to 4.8e-7 (4 blocks: 478 us, 2.5e-7).
constexpr int kChunk = 8;
// Registers: 384 threads of 168 at launch, 64,512; 128 x 56 + 256 x 224 = 64,512.
constexpr int kRegsFew = 56, kRegsMany = 224;
constexpr int kThreads = 128 + 32 * kEpi;
constexpr int kTiles = 4;                 // found ahead
constexpr int kBars = 3 * kStages + 4 + 1 + 2 * kTiles;
static_assert(kBars % 2 == 0, "the tiles behind them start on 16 bytes");
constexpr int kTurnRows = 192;            // of a contraction, on average
constexpr int kOutRows = 64, kOut = kOutRows * 32 * 2;  // results that a warp turns in shared memory at a time
static_assert(4 * kOut <= kHalf, "four warps turn theirs in one operand's part of a stage");
constexpr int kSmemBytes = 1024 + kStages * 2 * kHalf + kBars * 8 + 16 + kTiles * 32;
static_assert(kSmemBytes <= 232448, "shared memory of a CTA");
// Rows of A that one copy brings in: 32, once or twice, for a CTA's half of a tile
// of up to 128 rows, otherwise 128.  With 128 always, 2 rows of 2 experts of 11008 x
// 4096 took 45.7 us instead of 39.8; from 6 rows an expert on there is no difference.
constexpr int kBoxSome = 32, kBoxMany = 128;

// forward: C[r] = A[r] B[e]^T, dgrad: C[r] = A[r] B[e], wgrad: C[e] = A^T B.
enum Mode { kForward, kDgrad, kWgrad };

struct GroupedArgs {
    int E, R;
    int m, n, k;  // wgrad: C[e] is m x n; otherwise n columns, contraction k
    const int *offsets;
    float alpha, beta;
    void *C;
    long long ldc, stride_c;
    int c_type;
    int turn;    // C by store_turned, which has the memory of the last stage
    int stages;  // in the ring: without that one
    int tiles_m, tiles_n;  // tiles_m: of every expert (wgrad)
    int product;           // 0: C = beta C
    // A tile is `split` units, which share the blocks of its contraction; unit u
    // leaves its sums at partials + u * part_stride, laid out as C without gaps, and
    // grouped_join_kernel adds them in the order of the contraction.
    int split;
    float *partials;
    size_t part_stride;
    uint32_t idesc;
    unsigned *err;
    unsigned long long wait_ns;
    size_t c_extent;  // checked by GEMM11_DEBUG builds
};

// A tile of C: rows [m0, row_end) of expert e, `span` of them when rounded up to
// 16, from column n0; and its contraction k0 .. k1 (wgrad: rows of A and B).
struct alignas(16) Tile {
    int e, m0, n0, row_end, span;
    int k0, k1;
    int unit;  // of the tile (SPLIT)
};
static_assert(sizeof(Tile) == 32, "two words of 16 bytes");

// Tile i of tiles_m x tiles_n: groups of 8 tile rows, so that a wave of tiles
// shares its rows and columns in L2.
__device__ __forceinline__ void tile_place(int i, int tiles_m, int tiles_n, int &m, int &n) {
    const int group = 8 * tiles_n;
    const int first = i / group * 8, rows = min(tiles_m - first, 8);
    m = first + i % group % rows;
    n = i % group / rows;
}

// The list of tiles, walked forwards by a whole warp: lane l has expert e0 + l.
template <bool WGRAD, bool SPLIT>
struct TileList {
    int e0 = 0, base = 0;  // tiles before expert e0
    int start = 0, end = 0, tiles = 0, incl = 0;

    __device__ __forceinline__ void window(const GroupedArgs &p, int lane) {
        start = end = tiles = 0;
        if (e0 + lane < p.E) {
            start = min(max(__ldg(p.offsets + e0 + lane), 0), p.R);
            end = min(max(__ldg(p.offsets + e0 + lane + 1), start), p.R);
            tiles = WGRAD ? p.tiles_m * p.tiles_n : ((end - start + kTile - 1) / kTile) * p.tiles_n;
            if (SPLIT) tiles *= p.split;
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
        // The rows in as few tiles as hold them, all alike (to 16 rows), so that
        // the last is not nearly empty.
        const int first = WGRAD ? 0 : s, rows = WGRAD ? p.m : e - s;
        const int tiles_m = (rows + kTile - 1) / kTile;
        const unsigned even = (static_cast<unsigned>(rows) + static_cast<unsigned>(tiles_m) - 1) / static_cast<unsigned>(tiles_m);  // the sum may pass 2^31
        const int each = static_cast<int>(even + 15) & ~15;
        int i = t - base - before;
        tile.unit = 0;
        if (SPLIT) tile.unit = i % p.split, i /= p.split;
        tile_place(i, tiles_m, p.tiles_n, tile.m0, tile.n0);
        tile.m0 = first + tile.m0 * each;
        tile.row_end = min(first + rows, tile.m0 + each);
        tile.span = (tile.row_end - tile.m0 + 15) & ~15;
        tile.k0 = WGRAD ? s : 0, tile.k1 = WGRAD ? e : p.k;
        if (SPLIT) {
            const long long blocks = (tile.k1 - tile.k0 + kKB - 1) / kKB;
            const int from = static_cast<int>(blocks * tile.unit / p.split), to = static_cast<int>(blocks * (tile.unit + 1) / p.split);
            tile.k1 = min(tile.k1, tile.k0 + to * kKB);
            tile.k0 = min(tile.k1, tile.k0 + from * kKB);
        }
        tile.n0 *= kTile;
        if (!p.product) tile.k1 = tile.k0;
        return true;
    }
};

// The tiles that one warp of a CTA finds, kTiles ahead, for the others: some 700
// clocks of dependent shuffles and divisions each, which every warp spent by itself
// before (24,576 rows over 64 experts of 2048 x 256 47.9 -> 42.8 us, of 2048 x 1024
// 83.7 -> 81.6; the weights' gradient of 16,384 over 16 of 2048 x 4096 184 -> 179).
struct TileRing {
    uint64_t *found, *taken;
    Tile *tiles;
    int slot = 0;
    uint32_t phase = 0;

    __device__ __forceinline__ void step() {
        if (++slot == kTiles) slot = 0, phase ^= 1u;
    }
    // A whole warp's; 0: behind the last tile, -1: the wait ran out.
    __device__ __forceinline__ int take(Tile &tile, int lane, unsigned long long wait_ns) {
        if (!__all_sync(0xffffffffu, mbar_wait_patient(&found[slot], phase, wait_ns))) return -1;
        const int4 *from = reinterpret_cast<const int4 *>(tiles + slot);
        const int4 a = from[0], b = from[1];
        __syncwarp();
        if (lane == 0) mbar_arrive(&taken[slot]);
        step();
        tile.e = a.x, tile.m0 = a.y, tile.n0 = a.z, tile.row_end = a.w;
        tile.span = b.x, tile.k0 = b.y, tile.k1 = b.z, tile.unit = b.w;
        // The same in every lane: told so, the compiler keeps what depends on these
        // in uniform registers, which the copies and MMAs take.
        tile.e = __shfl_sync(0xffffffffu, tile.e, 0);
        tile.m0 = __shfl_sync(0xffffffffu, tile.m0, 0);
        tile.n0 = __shfl_sync(0xffffffffu, tile.n0, 0);
        tile.row_end = __shfl_sync(0xffffffffu, tile.row_end, 0);
        tile.span = __shfl_sync(0xffffffffu, tile.span, 0);
        tile.k0 = __shfl_sync(0xffffffffu, tile.k0, 0);
        tile.k1 = __shfl_sync(0xffffffffu, tile.k1, 0);
        return tile.e >= 0;
    }
};

__device__ __forceinline__ int tile_blocks(const Tile &t) { return (t.k1 - t.k0 + kKB - 1) / kKB; }

__device__ __forceinline__ void grouped_timeout(volatile int *abort_flag, unsigned *err) {
    *abort_flag = 1;
    atomicOr(err, kWatchdogTimeout);
}

// A lane's column of C down the rows of the tile that the warp has, from its sums.
// BETA = false: C is not read.  What the tile does not have is passed over by 16 rows
// (384 rows over 64 experts of 2048 x 128 21 -> 14 us).
template <int CT, bool BETA>
__device__ __forceinline__ void store_rows(const GroupedArgs &p, const float (&acc)[kCols], size_t at, int rows) {
    using T = typename Elem8<CT>::T;
    T *c = static_cast<T *>(p.C) + at;
    const long long ld = p.ldc;
    const float alpha = p.alpha, beta = p.beta;
#pragma unroll
    for (int j0 = 0; j0 < kCols; j0 += 16) {
        if (j0 >= rows) break;
#pragma unroll
        for (int j = j0; j < j0 + 16; ++j) {
            if (j < rows) {
                float v = alpha * acc[j];
                if (BETA) v = fmaf(beta, load_out(c, 0, CT), v);
                if (debug_in_bounds(p.c_extent == 0 || at + static_cast<size_t>(j) * static_cast<size_t>(ld) < p.c_extent, p.err)) store_out(c, 0, CT, v);
            }
            c += ld;
        }
    }
}

// The same for 16 bits through shared memory, 16 bytes a lane.  A lane puts 8 rows of
// its column there as 16 bytes, and takes eight columns of a row: 8 x 8 matrices, of
// which it gets two neighbouring elements of the transpose, four of them for columns
// 2 i, 2 i + 1 of each eight.  Column c of eight rows is at 16 bytes c, the eight that
// it is in turned by 2 (c / 8), so that none of the accesses meets a bank twice.
//
// For the weights' gradient from few rows, whose time is its stores: 256 rows over 16
// experts of 2048 x 4096 92 -> 79.5 us, 632 over 23 of 5120 x 2560 201 -> 169.  At 256
// rows an expert either takes 90, and behind that the ring's last stage, whose memory
// this has, is worth more.  Rows (of which a tile seldom has 256) gained nothing: 24,576
// over 64 experts of 2048 x 256 42.1 us, 42.8 stored singly, of 2048 x 512 52.6, 51.3.
// A copy of 256 bytes for each row out of shared memory took twice as long as single
// stores, full lines by four warps together a quarter longer.
// at: of the warp's first column; cols: that it has.
template <int CT>
__device__ __forceinline__ void store_turned(const GroupedArgs &p, const float (&acc)[kCols], size_t at, int rows, int cols, uint32_t smem, int lane) {
    const float alpha = p.alpha;
    const uint32_t put = smem + ((lane ^ (lane >> 3 << 1)) << 4);
    const int m = lane & 7, c = (m >> 1) * 8 + (lane >> 3) * 2 + (m & 1);  // of this lane's row of a matrix
    const uint32_t take = smem + ((c ^ (c >> 3 << 1)) << 4);
    const int col = (lane & 3) * 8, left = cols - col;
    uint16_t *to = static_cast<uint16_t *>(p.C) + at + static_cast<size_t>(lane >> 2) * static_cast<size_t>(p.ldc) + col;
    const long long step = 8 * p.ldc;
#pragma unroll
    for (int j0 = 0; j0 < kCols; j0 += kOutRows) {
        if (j0 < rows) {
#pragma unroll
            for (int j = j0; j < j0 + kOutRows; j += 8) {
                if (j >= rows) break;
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) w[k] = pack2_out16(alpha * acc[j + 2 * k], alpha * acc[j + 2 * k + 1], CT);
                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(put + (j - j0) * 64), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
            }
            __syncwarp();
#pragma unroll
            for (int j4 = j0; j4 < j0 + kOutRows; j4 += 32) {
                if (j4 >= rows) break;
                uint32_t w[4][4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];" : "=r"(w[k][0]), "=r"(w[k][1]), "=r"(w[k][2]), "=r"(w[k][3]) : "r"(take + (j4 - j0 + 8 * k) * 64) : "memory");
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int r = j4 + 8 * k + (lane >> 2);
                    if (r < rows && left > 0 && debug_in_bounds(p.c_extent == 0 || at + static_cast<size_t>(r) * static_cast<size_t>(p.ldc) + min(cols, col + 8) <= p.c_extent, p.err)) {
                        if (left >= 8) {
                            *reinterpret_cast<uint4 *>(to) = make_uint4(w[k][0], w[k][1], w[k][2], w[k][3]);
                        } else {
#pragma unroll
                            for (int i = 0; i < 7; ++i)
                                if (i < left) to[i] = static_cast<uint16_t>(w[k][i >> 1] >> (i & 1) * 16);
                        }
                    }
                    to += step;
                }
            }
            __syncwarp();
        }
    }
}

// The same of a unit's sums, to memory as they are.
__device__ __forceinline__ void store_sums(float *at, const float (&acc)[kCols], int ld, int rows) {
#pragma unroll
    for (int j0 = 0; j0 < kCols; j0 += 16) {
        if (j0 >= rows) break;
#pragma unroll
        for (int j = j0; j < j0 + 16; ++j) {
            if (j < rows) *at = acc[j];
            at += ld;
        }
    }
}

// CTA pairs (clusters of two), computed transposed: C^T = op(B)^T A^T, 256 columns
// n of C on the MMA's row side (128 of each CTA: tensor-memory lanes) and up to
// 256 rows on its column side, of which an MMA takes any multiple of 16.  So an
// expert's last rows cost what they are, a few rows cost little beside their
// expert's weights, and a warp stores 32 neighbouring elements of a row,
// whatever C's alignment.
//
// Tiles of 512 columns (both accumulators a tile's, a quarter less to bring in) were
// no faster (24,570 rows over 64 experts 85 -> 96 us), nor were copies of the next
// tile's operands into the L2 ahead of time (98 - 112), a second warp for the copies
// of A or one copy for two boxes (the same).
//
// CTA r stages columns [n0 + 128 r, + 128) and its half of the rows, up to 32 KB
// for a block of 64; the even CTA's MMA warp multiplies the pair, and each CTA's
// tensor memory receives the sums of its 128 columns, twice buffered.  Warp 0
// issues the copies, warp 1 the MMAs, warps 4 to 11 are the epilogue: warp w has
// lane quarter w % 4 and half of the rows, whose sums over the chunks it holds in
// registers.
//
// wgrad: the contraction ends at any row of A and B, and behind it are the next
// expert's.  The copies of the last block of 64 rows signal barriers of the CTA's
// own; warp 2 then zeroes what is behind the end in shared memory (a row is 128
// bytes there, the swizzle moves bytes within it) and hands the block on, while
// warp 0 is already at the next tile's (8192 rows, 8 experts of 11008 x 4096 618 ->
// 580 us against warp 0 doing it).
template <int MODE, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_kernel(const __grid_constant__ CUtensorMap tm_b, const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_a_some,
                   const GroupedArgs p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sB = smem, *sA = smem + kStages * kHalf;
    uint64_t *full = reinterpret_cast<uint64_t *>(sA + kStages * kHalf);
    uint64_t *empty = full + kStages;
    uint64_t *tfull = empty + kStages;
    uint64_t *tempty = tfull + 2;
    uint64_t *mma_done = tempty + 2;
    uint64_t *landed = mma_done + 1;  // last blocks of a contraction that ends in them
    uint64_t *found = landed + kStages;
    Tile *tiles = reinterpret_cast<Tile *>(found + 2 * kTiles);
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(tiles + kTiles);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int rank = static_cast<int>(cluster_ctarank());
    const bool leader = rank == 0;
    const int cid = blockIdx.x >> 1, ncl = gridDim.x >> 1;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], MODE == kWgrad ? 2 : 1);
            mbar_init(&empty[s], 1);
            mbar_init(&landed[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], 2 * kEpi);  // the warps of both CTAs
        }
        for (int b = 0; b < kTiles; ++b) {
            mbar_init(&found[b], 1);
            mbar_init(&found[kTiles + b], 1 + (leader ? 1 : 0) + (MODE == kWgrad ? 1 : 0) + kEpi);  // warps 0, 1, 2 and the epilogue
        }
        mbar_init(mma_done, 1);
        *abort_flag = 0;
        fence_mbarrier_init();
        if (p.product) {
            tma_prefetch_desc(&tm_b);
            tma_prefetch_desc(&tm_a);
            if (MODE != kWgrad) tma_prefetch_desc(&tm_a_some);
        }
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
    uint32_t ends = 0, ends_parity = 0;  // stages that had such a block, and the parity of the last
    TileRing ring = {found, found + kTiles, tiles};
    Tile tile;
    auto next = [&] {
        const int got = ring.take(tile, lane, p.wait_ns);
        if (got < 0) grouped_timeout(abort_flag, p.err);
        return got > 0;
    };
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsFew));
        if (warp == 0) {
            // ------------------------------------------------ TMA producer (both CTAs)
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            const uint32_t full_even = mapa_shared(smem_u32(full), 0), at_b = smem_u32(sB), at_a = smem_u32(sA);
            while (ok && !*abort_flag && next()) {
                const int half = tile.span >> 1, my_m = tile.m0 + rank * half, my_n = tile.n0 + rank * 128;
                // rows of A (wgrad: columns) come in boxes
                const int box = MODE == kWgrad ? 64 : half <= 2 * kBoxSome ? kBoxSome : kBoxMany;
                const int boxes = (half + box - 1) / box, box_bytes = box * kKB * 2;
                const uint32_t tx = kHalf + boxes * box_bytes;
                const int blocks = tile_blocks(tile);
                for (int kb = 0; kb < blocks; ++kb) {
                    ok = __all_sync(0xffffffffu, mbar_wait_patient(&empty[stage], phase ^ 1u, p.wait_ns));
                    if (!ok) {
                        grouped_timeout(abort_flag, p.err);
                        break;
                    }
                    const int k0 = tile.k0 + kb * kKB;
                    uint8_t *b = sB + stage * kHalf, *a = sA + stage * kHalf;
                    const int valid = tile.k1 - k0;
                    if (MODE == kWgrad && valid < kKB) {
                        if (elect_one()) {
                            mbar_arrive_expect_tx(&landed[stage], tx);
                            tma_load_2d(&tm_b, &landed[stage], b, my_n, k0);
                            tma_load_2d(&tm_b, &landed[stage], b + kBox, my_n + 64, k0);
                            for (int i = 0; i < boxes; ++i) tma_load_2d(&tm_a, &landed[stage], a + i * kBox, my_m + i * 64, k0);
                        }
                        __syncwarp();
                        if (ends & (1u << stage)) ends_parity ^= 1u << stage;
                        ends |= 1u << stage;
                    } else {
                        const uint32_t bar = full_even + stage * 8, b0 = at_b + stage * kHalf, a0 = at_a + stage * kHalf;
                        if (elect_one()) {
                            if (leader) mbar_arrive_expect_tx(&full[stage], 2 * tx);
                            if (MODE == kWgrad) {
                                if (leader) mbar_arrive(&full[stage]);
                                tma_load_2d_pair_at(&tm_b, bar, b0, my_n, k0);
                                tma_load_2d_pair_at(&tm_b, bar, b0 + kBox, my_n + 64, k0);
                                tma_load_2d_pair_at(&tm_a, bar, a0, my_m, k0);
                                if (half > 64) tma_load_2d_pair_at(&tm_a, bar, a0 + kBox, my_m + 64, k0);
                            } else {
                                if (MODE == kDgrad) {
                                    tma_load_3d_pair_at(&tm_b, bar, b0, my_n, k0, tile.e);
                                    tma_load_3d_pair_at(&tm_b, bar, b0 + kBox, my_n + 64, k0, tile.e);
                                } else {
                                    tma_load_3d_pair_at(&tm_b, bar, b0, k0, my_n, tile.e);
                                }
                                if (half > 2 * kBoxSome) {
                                    tma_load_2d_pair_at(&tm_a, bar, a0, k0, my_m);
                                } else {
                                    tma_load_2d_pair_at(&tm_a_some, bar, a0, k0, my_m);
                                    if (half > kBoxSome) tma_load_2d_pair_at(&tm_a_some, bar, a0 + kBoxSome * kKB * 2, k0, my_m + kBoxSome);
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
                    if (++stage == p.stages) stage = 0, phase ^= 1u;
                }
            }
        } else if (MODE == kWgrad && warp == 2) {
            // ------------------------------------------------ ends of contractions (both CTAs)
            int stage = 0;
            bool ok = true;
            while (ok && !*abort_flag && next()) {
                const int blocks = tile_blocks(tile), valid = tile.k1 - tile.k0 - (blocks - 1) * kKB;
                if (blocks == 0) continue;
                stage = (stage + blocks - 1) % p.stages;
                if (valid < kKB) {
                    ok = __all_sync(0xffffffffu, mbar_wait_patient(&landed[stage], ends_parity >> stage & 1u, p.wait_ns));
                    if (!ok) {
                        grouped_timeout(abort_flag, p.err);
                        break;
                    }
                    ends_parity ^= 1u << stage;
                    uint8_t *b = sB + stage * kHalf, *a = sA + stage * kHalf;
                    const uint4 zero = make_uint4(0, 0, 0, 0);
                    const int reached = (valid + 15) / 16 * 16;  // by the MMAs
                    for (int i = valid * 8 + lane; i < reached * 8; i += 32) {
                        reinterpret_cast<uint4 *>(b)[i] = zero;
                        reinterpret_cast<uint4 *>(b + kBox)[i] = zero;
                        reinterpret_cast<uint4 *>(a)[i] = zero;
                        reinterpret_cast<uint4 *>(a + kBox)[i] = zero;
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (elect_one()) mbar_arrive_cluster(mapa_shared(smem_u32(&full[stage]), 0));
                    __syncwarp();
                }
                stage = stage + 1 == p.stages ? 0 : stage + 1;
            }
        } else if (warp == 3) {
            // ------------------------------------------------ tiles (both CTAs)
            TileList<MODE == kWgrad, SPLIT> list;
            list.window(p, lane);
            for (int t = cid; !*abort_flag; t += ncl) {
                const bool more = list.find(p, t, lane, tile);
                if (!more) tile.e = -1;
                if (!__all_sync(0xffffffffu, mbar_wait_patient(&ring.taken[ring.slot], ring.phase ^ 1u, p.wait_ns))) {
                    grouped_timeout(abort_flag, p.err);
                    break;
                }
                if (lane == 0) {
                    int4 *to = reinterpret_cast<int4 *>(tiles + ring.slot);
                    to[0] = make_int4(tile.e, tile.m0, tile.n0, tile.row_end);
                    to[1] = make_int4(tile.span, tile.k0, tile.k1, tile.unit);
                    mbar_arrive(&found[ring.slot]);
                }
                __syncwarp();
                if (!more) break;
                ring.step();
            }
        } else if (warp == 1 && leader) {
            // ------------------------------------------------ MMA issuer (even CTA)
            // K-major: 128-byte rows, 8-row groups 1024 bytes apart, 16 k = 32
            // bytes along the row.  Stored along the tile: 128 bytes (64
            // columns) for each k, boxes of 64 columns kBox apart, 16 k = 2048
            // bytes.
            const uint64_t b_desc0 = umma_desc_sw128(smem_u32(sB), MODE != kForward ? kBox : 16, 1024);
            const uint64_t a_desc0 = umma_desc_sw128(smem_u32(sA), MODE == kWgrad ? kBox : 16, 1024);
            constexpr uint32_t kBstep = MODE != kForward ? 2048 >> 4 : 32 >> 4, kAstep = MODE == kWgrad ? 2048 >> 4 : 32 >> 4;
            int stage = 0, i = 0;  // i: chunk
            uint32_t phase = 0;
            bool ok = true;
            while (ok && !*abort_flag && next()) {
                const int blocks = tile_blocks(tile);
                const uint32_t idesc = p.idesc | static_cast<uint32_t>(tile.span >> 3) << 17;
                for (int kb0 = 0; ok && kb0 < blocks; kb0 += kChunk, ++i) {
                    const int buf = i & 1, some = min(kChunk, blocks - kb0);
                    ok = __all_sync(0xffffffffu, mbar_wait_patient(&tempty[buf], ((i >> 1) & 1) ^ 1u, p.wait_ns));
                    if (!ok) {
                        grouped_timeout(abort_flag, p.err);
                        break;
                    }
                    tc_fence_after();
                    for (int kb = 0; kb < some; ++kb) {
                        const int left = tile.k1 - tile.k0 - (kb0 + kb) * kKB;
                        // the end of a contraction comes from both CTAs' threads
                        ok = __all_sync(0xffffffffu, MODE == kWgrad && left < kKB ? mbar_wait_cluster(&full[stage], phase, p.wait_ns)
                                                                                  : mbar_wait_patient(&full[stage], phase, p.wait_ns));
                        if (!ok) {
                            grouped_timeout(abort_flag, p.err);
                            break;
                        }
                        tc_fence_after();
                        const uint64_t bd = b_desc0 + static_cast<uint64_t>(stage * (kHalf >> 4));
                        const uint64_t ad = a_desc0 + static_cast<uint64_t>(stage * (kHalf >> 4));
                        // of the last block only the 16 k that it reaches into
                        const int steps = (min(kKB, left) + 15) / 16;
                        if (elect_one()) {
#pragma unroll
                            for (int kk = 0; kk < kKB / 16; ++kk)
                                if (kk < steps)
                                    umma_f16_pair(tmem_base + buf * kTile, bd + kBstep * kk, ad + kAstep * kk, idesc, kb > 0 || kk > 0 ? 1u : 0u);
                            umma_commit_pair_mc(&empty[stage], 0x3);
                            if (kb == some - 1) umma_commit_pair_mc(&tfull[buf], 0x3);
                        }
                        __syncwarp();
                        if (++stage == p.stages) stage = 0, phase ^= 1u;
                    }
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsMany));
        // ------------------------------------------------ epilogue (both CTAs)
        // Lane l of quarter q has column n0 + 128 rank + 32 q + l of C, and the
        // warp one half of the tile's rows.
        const int q = warp & 3, part = (warp - 4) >> 2;
        const uint32_t t_row = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
        const uint32_t release[2] = {mapa_shared(smem_u32(&tempty[0]), 0), mapa_shared(smem_u32(&tempty[1]), 0)};
        const uint32_t turned = smem_u32((part ? sA : sB) + (kStages - 1) * kHalf) + q * kOut;
        int i = 0;
        bool ok = true;
        while (ok && !*abort_flag && next()) {
            const int chunks = (tile_blocks(tile) + kChunk - 1) / kChunk;
            const int half = tile.span >> 1;
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
                const uint32_t from = t_row + buf * kTile + part * half;
#pragma unroll
                for (int g = 0; g < kCols / 64; ++g) {
                    if (g * 64 < half) {
                        uint32_t r0[32], r1[32];
                        tmem_ld_32x32b_x32(from + g * 64, r0);
                        tmem_ld_32x32b_x32(from + g * 64 + 32, r1);
                        tmem_wait_ld(r0);
                        tmem_landed(r1);
#pragma unroll
                        for (int j = 0; j < 32; ++j) acc[g * 64 + j] += __uint_as_float(r0[j]), acc[g * 64 + 32 + j] += __uint_as_float(r1[j]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote(release[buf]);
            }
            if (!ok) continue;
            const int n = tile.n0 + rank * 128 + q * 32 + lane, row = tile.m0 + part * half;
            const int rows = n < p.n ? min(half, tile.row_end - row) : 0;
            if constexpr (SPLIT) {
                const size_t first = (MODE == kWgrad ? static_cast<size_t>(tile.e) * p.m : 0) + row;
                if (first + max(rows, 0) <= p.part_stride / p.n) store_sums(p.partials + tile.unit * p.part_stride + first * p.n + n, acc, p.n, rows);
                continue;
            }
            const size_t at = (MODE == kWgrad ? static_cast<size_t>(tile.e * p.stride_c) : 0) + static_cast<size_t>(row) * static_cast<size_t>(p.ldc) + n;
            if (MODE == kWgrad && p.turn) {
                const int first = n - lane, cols = min(p.n - first, 32), all = min(half, tile.row_end - row);
                if (cols > 0) {
                    if (p.c_type == kOutF16)
                        store_turned<kOutF16>(p, acc, at - lane, all, cols, turned, lane);
                    else
                        store_turned<kOutBF16>(p, acc, at - lane, all, cols, turned, lane);
                }
            } else if (p.beta != 0.f) {
                if (p.c_type == kOutF32)
                    store_rows<kOutF32, true>(p, acc, at, rows);
                else if (p.c_type == kOutF16)
                    store_rows<kOutF16, true>(p, acc, at, rows);
                else
                    store_rows<kOutBF16, true>(p, acc, at, rows);
            } else if (p.c_type == kOutF32) {
                store_rows<kOutF32, false>(p, acc, at, rows);
            } else if (p.c_type == kOutF16) {
                store_rows<kOutF16, false>(p, acc, at, rows);
            } else {
                store_rows<kOutBF16, false>(p, acc, at, rows);
            }
        }
    }

    // ---------------------------------------------------- drain and unwind
    if (warp == 0 && lane == 0) {
        // the even CTA's full barriers count the copies of both CTAs, except of the ends
        for (int s = 0; s < kStages; ++s) {
            if ((ends & (1u << s)) && !mbar_wait(&landed[s], (ends_parity >> s) & 1u)) grouped_timeout(abort_flag, p.err);
            if (leader && (armed & (1u << s)) && !mbar_wait(&full[s], (armed_parity >> s) & 1u)) grouped_timeout(abort_flag, p.err);
        }
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

// C = alpha times the units' sums + beta C, for the rows that an expert has (wgrad:
// all): four columns a thread, whose sums of four units are in flight together.
__global__ void __launch_bounds__(256) grouped_join_kernel(const GroupedArgs p, int wgrad) {
    pdl_wait();
    pdl_launch_dependents();
    const int quads = (p.n + 3) / 4;
    const long long r0 = wgrad ? 0 : min(max(__ldg(p.offsets), 0), p.R), r1 = wgrad ? static_cast<long long>(p.E) * p.m : min(max(__ldg(p.offsets + p.E), 0), p.R);
    for (long long i = blockIdx.x * 256LL + threadIdx.x; i < (r1 - r0) * quads; i += gridDim.x * 256LL) {
        const long long row = r0 + i / quads;
        const int n = static_cast<int>(i % quads) * 4, left = min(4, p.n - n);
        const float *from = p.partials + row * p.n + n;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
        for (int u = 0; u < p.split; u += 4) {
            float v[4][4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int j = 0; j < 4; ++j) v[k][j] = u + k < p.split && j < left ? __ldcg(from + (u + k) * p.part_stride + j) : 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int j = 0; j < 4; ++j) sum[j] += v[k][j];
        }
        const size_t at = wgrad ? static_cast<size_t>(row / p.m * p.stride_c + row % p.m * p.ldc) + n : static_cast<size_t>(row * p.ldc) + n;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (j >= left) break;
            float v = p.alpha * sum[j];
            if (p.beta != 0.f) v = fmaf(p.beta, load_out(p.C, at + j, p.c_type), v);
            if (debug_in_bounds(p.c_extent == 0 || at + j < p.c_extent, p.err)) store_out(p.C, at + j, p.c_type, v);
        }
    }
}

// Tiles that there are at most.
long long most_tiles(const Grouped &g) {
    const long long tiles_n = (g.N + kTile - 1) / kTile;
    return g.wgrad ? static_cast<long long>(g.E) * ((g.M + kTile - 1) / kTile) * tiles_n : (g.R / kTile + static_cast<long long>(std::min(g.E, g.R))) * tiles_n;
}

// Units of a tile where the tiles would leave pairs without work: a model, in us.
// A block of 64 takes a pair 0.37 (its 32 KB of weights at a 76th of the memory's
// rate), 0.2 at least where few pairs are at work; each unit 0.5 beside its
// blocks, and the sums' way through memory 3 and their bytes.  Measured, whole /
// shared: 2 rows over 2 experts of 1024 x 8192 (8 tiles) 33.9 / 12.5 us in 9 units, of
// 11008 x 4096 (86 tiles) 45.6 / 39.8 in 3; 400 rows over 4 experts of 1024 x 8192
// 36.2 / 26.6; the weights' gradient of 4 experts of 256 x 512 over 8192 rows 18.5 /
// 15.7 in 3, which the model leaves whole.  Left whole: 384 rows over 64 experts of
// 1024 x 2048 (256 tiles) 47.5 / 51.0 in 2, 1136 over 19 of 1445 x 6884 76.0 / 80.3.
int pick_split(const Grouped &g, int pairs) {
    const double tiles = static_cast<double>(most_tiles(g)), cells = g.wgrad ? static_cast<double>(g.E) * g.M * g.N : static_cast<double>(g.R) * g.N;
    const double blocks = std::floor(g.wgrad ? static_cast<double>(g.R) / g.E / kKB : (g.K + kKB - 1) / kKB);
    auto time = [&](int s) {
        const double units = tiles * s, each = std::ceil(blocks / s), waves = std::floor(units / pairs), left = units - waves * pairs, more = s > 1 ? 0.5 : 0.0;
        return waves * (each * 0.37 + more) + (left > 0 ? each * std::max(0.2, 0.37 * left / pairs) + more : 0.0) + (s > 1 ? 3.0 + cells * (8 * s + 4) / 6e6 : 0.0);
    };
    int best = 1;
    double t = time(1);
    for (int s = 2; s <= 16 && 2 * s <= blocks && cells * s <= 16e6; ++s) {  // 64 MB of sums
        const double with = time(s);
        if (with < t) t = with, best = s;
    }
    return best;
}

// Strides that nothing has (of a single row, of a single expert) may be any.
uint64_t map_stride(long long elements) { return static_cast<uint64_t>((elements * 2 + 15) / 16 * 16); }

template <int MODE, bool SPLIT>
cudaError_t launch_grouped(const Grouped &g, GroupedArgs a, cudaStream_t stream, CallInfo *info) {
    auto kern = grouped_kernel<MODE, SPLIT>;
    static int max_clusters = -1;  // one device type per process; atomic accesses
    static unsigned long long smem_set = 0;
    cudaError_t e = ensure_dynamic_smem(kern, kSmemBytes, smem_set);
    if (e != cudaSuccess) return e;
    const auto sw = CU_TENSOR_MAP_SWIZZLE_128B;
    const auto t16 = g.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    CUtensorMap tb = {}, ta = {}, some = {};
    if (a.product) {
        const uint64_t lda = map_stride(g.lda), ldb = map_stride(g.ldb), step = map_stride(g.stride_b);
        bool ok;
        if (MODE == kWgrad) {
            ok = encode_matrix_map(&ta, t16, g.A, g.M, g.R, lda, 64, kKB, sw) && encode_matrix_map(&tb, t16, g.B, g.N, g.R, ldb, 64, kKB, sw);
        } else {
            ok = encode_matrix_map(&ta, t16, g.A, g.K, g.R, lda, kKB, kBoxMany, sw) && encode_matrix_map(&some, t16, g.A, g.K, g.R, lda, kKB, kBoxSome, sw) &&
                 (MODE == kForward ? encode_box_map(&tb, t16, g.B, g.K, g.N, g.E, ldb, step, kKB, 128, 1) : encode_box_map(&tb, t16, g.B, g.N, g.K, g.E, ldb, step, 64, kKB, 1));
        }
        if (!ok) return cudaErrorNotSupported;
    }
    // The MMA's columns (rows of C) are set tile by tile.
    a.idesc = umma_idesc_f16_f32(256, 0, MODE != kForward, MODE == kWgrad) | (g.bf16 ? kIdescBf16Operands : 0u);
    a.tiles_m = (g.M + kTile - 1) / kTile;
    a.tiles_n = (g.N + kTile - 1) / kTile;
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
    const long long most = most_tiles(g) * a.split;
    if (SPLIT) {
        Scratch sc;
        a.part_stride = g.wgrad ? static_cast<size_t>(g.E) * g.M * g.N : static_cast<size_t>(g.R) * g.N;
        e = acquire_scratch(stream, a.part_stride * a.split, 0, info, &sc);
        if (e != cudaSuccess) return e;
        a.partials = sc.partials;
    }
    cfg.gridDim = dim3(2 * static_cast<unsigned>(std::min<long long>(clusters, most)));
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, kern, tb, ta, some, a);
    if (e == cudaSuccess) e = cudaPeekAtLastError();
    if (e != cudaSuccess || !SPLIT) return e;
    info->launches = 2;
    const long long quads = static_cast<long long>(a.part_stride / g.N) * ((g.N + 3) / 4);
    cfg.gridDim = dim3(static_cast<unsigned>(std::min<long long>((quads + 255) / 256, 8LL * device_sm_count())));
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    cfg.attrs = attr + 1;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, grouped_join_kernel, a, g.wgrad);
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
    // A warp may have to wait while another walks the offsets of experts without rows
    // (32 in 0.6 us: 2^28 experts of which the last alone has rows take 4 to 5 s), and for
    // all of a tile's contraction (a block in 0.2 to 0.8 us: 3.0 s for a pair alone with
    // 3 * 2^28 rows of an expert), which the host knows no better than as R.
    a.wait_ns = kWaitLimitNs + 2000ull * static_cast<unsigned long long>(g.E / 32) + 4000ull * static_cast<unsigned long long>((g.wgrad ? g.R : g.K) / kKB);
    if (kDebugBuild) {
        a.c_extent = g.wgrad ? static_cast<size_t>((g.E - 1LL) * g.stride_c + (g.M - 1LL) * g.ldc + g.N) : static_cast<size_t>((g.R - 1LL) * g.ldc + g.N);
        a.c_extent -= std::min(a.c_extent - 1, debug_shrink_c());
    }
    info->launches = 1;
    a.split = a.product ? pick_split(g, std::max(1, device_sm_count() / 2)) : 1;
    a.turn = g.wgrad && a.split == 1 && g.c_type != kOutF32 && g.beta == 0.f && g.R <= static_cast<long long>(kTurnRows) * g.E && reinterpret_cast<uintptr_t>(g.C) % 16 == 0 &&
             g.ldc % 8 == 0 && g.stride_c % 8 == 0;
    a.stages = kStages - a.turn;
    const bool split = a.split > 1;
    info->plan = g.wgrad ? (split ? "grouped_wgrad_pair_splitk" : "grouped_wgrad_pair") : split ? "grouped_pair_splitk" : "grouped_pair";
    if (g.wgrad) return split ? launch_grouped<kWgrad, true>(g, a, stream, info) : launch_grouped<kWgrad, false>(g, a, stream, info);
    if (g.b_trans) return split ? launch_grouped<kForward, true>(g, a, stream, info) : launch_grouped<kForward, false>(g, a, stream, info);
    return split ? launch_grouped<kDgrad, true>(g, a, stream, info) : launch_grouped<kDgrad, false>(g, a, stream, info);
}

}  // namespace gemm11

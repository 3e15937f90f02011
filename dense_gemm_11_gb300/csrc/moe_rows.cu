// moe_rows.cu -- the rows of a mixture-of-experts layer's tokens in the order
// of the experts, and back:
//
//   dispatch      offsets[e] = number of slots (t, j) whose expert is below e,
//                 rows[t, j] = offsets[e] + number of earlier slots of expert
//                 e = ids[t, j] (the sort is stable), -1 for an id outside
//                 0 .. E - 1, and Xs[rows[t, j]] = X[t];
//   combine       Y[t] = sum over j of w[t, j] Ys[rows[t, j]];
//   combine grad  dYs[rows[t, j]] = w[t, j] dY[t] and
//                 dw[t, j] = sum over h of dY[t, h] Ys[rows[t, j], h].
//
// Bound: memory.  Every row is read once and written once; a token's row is
// read once for its k copies, and the k rows of a token are gathered where they
// are summed, so no inverse of the order is stored.  No sum of floating-point
// numbers is made with atomics, so the results do not depend on the order in which
// CTAs run.  Measured on BF16, 8192 tokens, 6 slots of 64 experts, 2048 columns:
// dispatch 42.1 us, 7.1 of them for the order (235 MB, 5.6 TB/s), combine 40.6 (5.8
// TB/s), its gradient 68.6 (437 MB, 6.4 TB/s).  For few tokens a launch: 16 tokens, 2
// slots, 4096 columns 3.5 us in a graph.
#include <algorithm>
#include <cstdint>

#include "experts.h"
#include "rows8.cuh"

namespace gemm11 {
namespace {

constexpr int kSortThreads = 1024;
// Rows that go through shared memory: they are on their way while the slots are
// counted, and a copy of one is an instruction.  8192 tokens, 6 slots, in registers /
// so: rows of 1 KB 14.2 / 15.7 us, 2 KB 23.5 / 24.5, 4 KB 46.7 / 42.1; 2000 tokens with
// rows of 16 KB 43.3 / 38.9, of 32 KB 83.0 / 77.5, of 64 KB, of which 3 fit, 158.4 / 158.7.
constexpr int kBulkBytes = 4096;          // of a row, at least
constexpr int kMinBuffers = 4, kMaxBuffers = 64;
constexpr int kBulkSmem = 232448 - 5120;  // 5120: the kernel's own
constexpr int kSortBatch = 1024;  // slots that are ranked and then copied together
static_assert(kDispatchMaxExperts <= 8192, "an expert and its slots among 32 in one word");

struct DispatchArgs {
    int T, E, k, n;  // n = T k
    const int *ids;
    const uint8_t *X;
    long long x_bytes;  // from one row to the next
    uint8_t *Xs;
    long long xs_bytes;
    int row_bytes, esize;
    int *offsets, *rows;
    int per_cta;  // tokens
    int copies;   // of the counters, a power of two
    int warps, depth;  // that copy rows through shared memory (kBulk), and the buffers of each
    int pitch;         // bytes from one buffer to the next
    unsigned *err;
    size_t xs_extent;  // bytes, checked by GEMM11_DEBUG builds
};

// A segment of a row: U times 16 bytes a lane.
template <int U>
struct Segment {
    uint4 v[U];
    __device__ __forceinline__ void load(const DispatchArgs &p, const uint8_t *from, int c0, int lane) {
        const int full = p.row_bytes >> 4;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + u * 32 + lane;
            if (c < full) v[u] = __ldg(reinterpret_cast<const uint4 *>(from) + c);
        }
    }
    __device__ __forceinline__ void store(const DispatchArgs &p, const int *pos, int c0, int lane) const {
        const int full = p.row_bytes >> 4;
        for (int j = 0; j < p.k; ++j) {
            const int r = pos[j];
            if (r < 0) continue;
            uint8_t *to = p.Xs + r * p.xs_bytes;
            if (!debug_in_bounds(static_cast<size_t>(r * p.xs_bytes + p.row_bytes) <= p.xs_extent, p.err)) continue;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = c0 + u * 32 + lane;
                if (c < full) __stcs(reinterpret_cast<uint4 *>(to) + c, v[u]);
            }
        }
    }
};
constexpr int kSegment = 4;                        // 16-byte pieces of a lane: 46.7 us, 2: 47.4, 1: 49.4 (8192 tokens, 6 slots, 2048 columns, without kBulk)
constexpr int kSegmentPieces = 32 * kSegment;      // of a warp
constexpr int kSegmentElements = 128;              // of a warp, where rows are not aligned

// Elements [first, last) of a row to its copies, one a lane.
template <typename T>
__device__ __forceinline__ void copy_elements(const DispatchArgs &p, const uint8_t *from, const int *pos, int first, int last, int lane) {
    for (int i = first + lane; i < last; i += 32) {
        const T v = reinterpret_cast<const T *>(from)[i];
        for (int j = 0; j < p.k; ++j) {
            const int r = pos[j];
            if (r < 0) continue;
            if (!debug_in_bounds(static_cast<size_t>(r * p.xs_bytes + p.row_bytes) <= p.xs_extent, p.err)) continue;
            reinterpret_cast<T *>(p.Xs + r * p.xs_bytes)[i] = v;
        }
    }
}

// Every CTA counts all the slots itself, those before its own tokens apart, so
// that it knows where its slots go without waiting for another CTA: 49,152 slots
// over 64 experts take 3.5 us.  (Clusters of eight that share the counting save 1
// us of that and lose it again: of the 152 SMs they fill 128.)
enum Rows { kElements, kVectors, kBulk };  // in pieces of one element, 16 bytes, a row through shared memory
template <Rows ROWS>
__global__ void __launch_bounds__(kSortThreads) dispatch_kernel(const DispatchArgs p) {
    constexpr bool VEC = ROWS == kVectors;
    extern __shared__ __align__(128) int counts[];  // of each expert: slots before this CTA's, then the others
    __shared__ int warp_sum[32];
    __shared__ int pos[kSortBatch];
    __shared__ uint64_t full[ROWS == kBulk ? kMaxBuffers : 1];
    const int copies = p.copies, E = p.E;  // neighbouring lanes count in counters of their own: fewer of a warp's additions meet
    int *const before = counts, *const rest = counts + E * copies;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t0 = blockIdx.x * p.per_cta, t1 = t0 + min(p.T - t0, p.per_cta);
    for (int e = threadIdx.x; e < 2 * E * copies; e += kSortThreads) counts[e] = 0;
    const uint32_t rows_at = smem_u32(counts) + ((2 * E * copies * 4 + 127) & ~127);
    if (ROWS == kBulk && threadIdx.x == 0) {
        for (int b = 0; b < p.warps * p.depth; ++b) mbar_init(&full[b], 1);
        fence_mbarrier_init();
    }
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();
    // Warp 31 - w takes the CTA's tokens w, w + warps, ..; the m-th of them is in its
    // buffer m % depth.  (Few slots are counted by the lowest warps, which copy last.)
    const int worker = kSortThreads / 32 - 1 - warp;
    int next_row = worker, fetched = 0;
    auto fetch = [&] {
        if (next_row < t1 - t0 && lane == 0) {
            const int b = worker * p.depth + fetched % p.depth;
            mbar_arrive_expect_tx(&full[b], p.row_bytes);
            bulk_load(rows_at + b * p.pitch, p.X + static_cast<long long>(t0 + next_row) * p.x_bytes, p.row_bytes, &full[b]);
        }
        if (next_row < t1 - t0) ++fetched;
        next_row += p.warps;
    };
    if (ROWS == kBulk && worker < p.warps)
        for (int m = 0; m < p.depth; ++m) fetch();
    const int mine = t0 * p.k, my_copy = lane & (copies - 1);
    auto count = [&](int e, int i) {
        if (static_cast<unsigned>(e) < static_cast<unsigned>(E)) atomicAdd((i < mine ? before : rest) + e * copies + my_copy, 1);
    };
    int done = 0;
    if (reinterpret_cast<uintptr_t>(p.ids) % 16 == 0) {
        const int4 *ids4 = reinterpret_cast<const int4 *>(p.ids);
        const int quads = p.n >> 2;
        constexpr int kAhead = 4;
        for (int q0 = threadIdx.x; q0 < quads; q0 += kAhead * kSortThreads) {
            int4 e[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                e[u] = q0 + u * kSortThreads < quads ? __ldg(ids4 + q0 + u * kSortThreads) : make_int4(-1, -1, -1, -1);
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int i = (q0 + u * kSortThreads) * 4;
                count(e[u].x, i);
                count(e[u].y, i + 1);
                count(e[u].z, i + 2);
                count(e[u].w, i + 3);
            }
        }
        done = quads * 4;
    }
    for (int i = done + threadIdx.x; i < p.n; i += kSortThreads) count(__ldg(p.ids + i), i);
    __syncthreads();

    // before[e] becomes next[e], the row of this CTA's first slot of expert e.
    int *const next = before;
    constexpr int kPer = kDispatchMaxExperts / kSortThreads;
    const int per = (E + kSortThreads - 1) / kSortThreads;  // experts of a thread
    int total[kPer], ahead[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = threadIdx.x * per + i;
        total[i] = ahead[i] = 0;
        if (i < per && e < E) {
            for (int c = 0; c < copies; ++c) {
                ahead[i] += before[e * copies + c];
                total[i] += rest[e * copies + c];
            }
            total[i] += ahead[i];
        }
        sum += total[i];
    }
    int incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += o;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        int s = warp_sum[lane];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, s, d);
            if (lane >= d) s += o;
        }
        warp_sum[lane] = s;
    }
    __syncthreads();
    int start = incl - sum + (warp > 0 ? warp_sum[warp - 1] : 0);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = threadIdx.x * per + i;
        if (i < per && e < E) {
            next[e] = ahead[i] + start;
            if (blockIdx.x == 0) p.offsets[e] = start;
        }
        start += total[i];
    }
    if (blockIdx.x == 0 && threadIdx.x == kSortThreads - 1) p.offsets[E] = start;

    const int batch = kSortBatch / p.k;  // tokens
    int my_row = worker, read = 0;
    bool late = false;
    const int segments = VEC ? ((p.row_bytes >> 4) + kSegmentPieces - 1) / kSegmentPieces : (p.row_bytes / p.esize + kSegmentElements - 1) / kSegmentElements;
    const int elements = p.row_bytes / p.esize, whole = (p.row_bytes >> 4) * (16 / p.esize);
    for (int t = t0; t < t1; t += batch) {
        const int tokens = min(batch, t1 - t), slots = tokens * p.k, units = tokens * segments;
        auto source = [&](int u) { return p.X + static_cast<long long>(t + u / segments) * p.x_bytes; };
        Segment<kSegment> now;
        if (VEC && warp < units) now.load(p, source(warp), warp % segments * kSegmentPieces, lane);
        // Slots of one expert among the 32 of a warp (a match takes 400 clocks: all
        // warps at once), then, 32 after 32, where the expert's rows have come to.
        __syncthreads();  // the last batch's rows are written, and the first's counts
        static_assert(kSortBatch <= kSortThreads, "a slot a thread");
        if (warp * 32 < slots) {
            const int i = threadIdx.x;
            int e = i < slots ? __ldg(p.ids + t * p.k + i) : -1;
            if (static_cast<unsigned>(e) >= static_cast<unsigned>(E)) e = -1;
            const unsigned same = __match_any_sync(0xffffffffu, e);
            const int rank = __popc(same & ((1u << lane) - 1u)), alike = lane == __ffs(same) - 1 ? __popc(same) : 0;
            if (i < slots) pos[i] = e < 0 ? -1 : e | rank << 13 | alike << 18;
        }
        __syncthreads();
        if (warp == 0) {
            for (int i0 = 0; i0 < slots; i0 += 32) {
                const int i = i0 + lane, packed = i < slots ? pos[i] : -1, e = packed & 0x1FFF;
                const int r = packed >= 0 ? next[e] : 0;
                __syncwarp();
                if (packed >= 0) {
                    pos[i] = r + (packed >> 13 & 31);
                    if (packed >> 18) next[e] = r + (packed >> 18);
                }
                __syncwarp();
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < slots; i += kSortThreads) p.rows[t * p.k + i] = pos[i];
        if (ROWS == kBulk) {
            // read = tokens of this warp so far, the next of them `my_row`
            for (; worker < p.warps && my_row < t - t0 + tokens && read < fetched; my_row += p.warps, ++read) {
                const int b = worker * p.depth + read % p.depth;
                if (!__all_sync(0xffffffffu, mbar_wait(&full[b], (read / p.depth) & 1))) {
                    if (lane == 0) atomicOr(p.err, kWatchdogTimeout);
                    late = true;
                }
                if (late) continue;  // what was fetched is waited for
                for (int j = lane; j < p.k; j += 32) {
                    const int r = pos[(my_row - (t - t0)) * p.k + j];
                    if (r >= 0 && debug_in_bounds(static_cast<size_t>(r * p.xs_bytes + p.row_bytes) <= p.xs_extent, p.err))
                        bulk_store(p.Xs + r * p.xs_bytes, rows_at + b * p.pitch, p.row_bytes);
                }
                bulk_commit();
                // the buffer of the token before is refilled, with one alone this token's
                if (next_row < t1 - t0 && (read > 0 || p.depth == 1)) {
                    if (p.depth > 1)
                        bulk_wait_read_all_but_one();
                    else
                        bulk_wait_read_all();
                    __syncwarp();
                    fetch();
                }
            }
        } else if (VEC) {
            // the next unit is read before this one is written
            for (int u = warp; u < units; u += kSortThreads / 32) {
                const int ahead_u = u + kSortThreads / 32;
                Segment<kSegment> then;
                if (ahead_u < units) then.load(p, source(ahead_u), ahead_u % segments * kSegmentPieces, lane);
                now.store(p, pos + u / segments * p.k, u % segments * kSegmentPieces, lane);
                now = then;
            }
            if (whole < elements) {
                for (int i = warp; i < tokens; i += kSortThreads / 32) {
                    const uint8_t *from = p.X + static_cast<long long>(t + i) * p.x_bytes;
                    if (p.esize == 2)
                        copy_elements<uint16_t>(p, from, pos + i * p.k, whole, elements, lane);
                    else
                        copy_elements<uint32_t>(p, from, pos + i * p.k, whole, elements, lane);
                }
            }
        } else {
            for (int u = warp; u < units; u += kSortThreads / 32) {
                const int begin = u % segments * kSegmentElements, end = min(begin + kSegmentElements, elements);
                if (p.esize == 2)
                    copy_elements<uint16_t>(p, source(u), pos + u / segments * p.k, begin, end, lane);
                else
                    copy_elements<uint32_t>(p, source(u), pos + u / segments * p.k, begin, end, lane);
            }
        }
    }
    if (ROWS == kBulk) bulk_wait_all();
}

// ------------------------------------------------------------------ back to the tokens
struct CombineArgs {
    int T, k, H, R;
    const void *Ys;
    long long ldys;
    const int *rows;
    const float *weights;
    void *Y;
    long long ldy;
    void *dYs;
    long long lddys;
    float *dweights;
    int lanes;   // threads of a token (gradient: of a slot), a power of two, kCombineThreads at most
    int tokens;  // or slots, of a CTA: kCombineThreads / lanes
    unsigned *err;
    size_t y_extent;  // elements of what is written, checked by GEMM11_DEBUG builds
};
// 8192 tokens, 6 slots, 2048 columns: 40.6 us with 128 threads a CTA, 49.2 with 256,
// 39.5 with 64; 2 slots of 4096 columns (4095 tokens) 17.9, 19.3 and 17.9.
constexpr int kCombineThreads = 128;

// Row of slot i, -1 where it has none.
__device__ __forceinline__ int slot_row(const CombineArgs &p, long long i) {
    const int r = __ldg(p.rows + i);
    return static_cast<unsigned>(r) < static_cast<unsigned>(p.R) ? r : -1;
}

// A thread has U times eight columns of a token and reads the KU rows of a step
// before it adds them, in the order of the slots.
template <int XT, bool VEC, int KU, int U>
__global__ void __launch_bounds__(kCombineThreads) combine_kernel(const CombineArgs p) {
    pdl_wait();
    pdl_launch_dependents();
    const long long t = static_cast<long long>(blockIdx.x) * p.tokens + threadIdx.x / p.lanes;
    if (t >= p.T) return;
    const int step = p.lanes * 8;
    for (int c = static_cast<int>(threadIdx.x % p.lanes) * 8; c < p.H; c += U * step) {
        float sum[U][8];
#pragma unroll
        for (int v = 0; v < U; ++v)
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[v][i] = 0.f;
        for (int j0 = 0; j0 < p.k; j0 += KU) {
            Row8<XT> y[KU][U];
            float w[KU];
            int r[KU];
#pragma unroll
            for (int u = 0; u < KU; ++u) {
                r[u] = j0 + u < p.k ? slot_row(p, t * p.k + j0 + u) : -1;
                w[u] = p.weights && j0 + u < p.k ? __ldg(p.weights + t * p.k + j0 + u) : 1.f;
            }
#pragma unroll
            for (int u = 0; u < KU; ++u)
#pragma unroll
                for (int v = 0; v < U; ++v)
                    if (r[u] >= 0 && c + v * step < p.H) y[u][v].template load<VEC>(p.Ys, r[u] * p.ldys + c + v * step, p.H - c - v * step);
#pragma unroll
            for (int u = 0; u < KU; ++u) {
                if (r[u] < 0) continue;
#pragma unroll
                for (int v = 0; v < U; ++v) {
                    float f[8];
                    y[u][v].widen(f);
#pragma unroll
                    for (int i = 0; i < 8; ++i) sum[v][i] = fmaf(w[u], f[i], sum[v][i]);
                }
            }
        }
#pragma unroll
        for (int v = 0; v < U; ++v) {
            const int cv = c + v * step;
            if (cv >= p.H) break;
            Row8<XT> out;
            out.round(sum[v]);
            if (debug_in_bounds(static_cast<size_t>(t * p.ldy + min(cv + 8, p.H)) <= p.y_extent, p.err)) out.template store<VEC>(p.Y, t * p.ldy + cv, p.H - cv);
        }
    }
}

// The gradient (a CTA a token with the rows of eight slots in registers held two CTAs
// an SM and took 128 us for the 68.6 above): `lanes` threads a slot, which read the token's row (again for each
// of its slots, from the caches) and the slot's, U times eight columns at a time.
// A slot's sum stays within its threads: most often one warp.
template <int XT, bool VEC, int U>
__global__ void __launch_bounds__(kCombineThreads) combine_grad_kernel(const CombineArgs p) {
    __shared__ float part[kCombineThreads / 32];
    pdl_wait();
    pdl_launch_dependents();
    const int at = threadIdx.x % p.lanes, step = p.lanes * 8;
    const long long slot = static_cast<long long>(blockIdx.x) * p.tokens + threadIdx.x / p.lanes;
    const bool live = slot < static_cast<long long>(p.T) * p.k;
    float dot = 0.f;
    if (live) {
        const long long t = slot / p.k;
        const int r = slot_row(p, slot);
        const float w = __ldg(p.weights + slot);
        for (int c = at * 8; r >= 0 && c < p.H; c += U * step) {
            Row8<XT> dy[U], y[U];
#pragma unroll
            for (int v = 0; v < U; ++v) {
                const int cv = c + v * step;
                if (cv < p.H) {
                    dy[v].template load<VEC>(p.Y, t * p.ldy + cv, p.H - cv);
                    y[v].template load<VEC>(p.Ys, r * p.ldys + cv, p.H - cv);
                }
            }
#pragma unroll
            for (int v = 0; v < U; ++v) {
                const int cv = c + v * step;
                if (cv < p.H) {
                    float d[8], f[8];
                    dy[v].widen(d);
                    y[v].widen(f);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        dot = fmaf(d[i], f[i], dot);
                        d[i] *= w;
                    }
                    Row8<XT> out;
                    out.round(d);
                    if (debug_in_bounds(static_cast<size_t>(r * p.lddys + min(cv + 8, p.H)) <= p.y_extent, p.err))
                        out.template store<VEC>(p.dYs, r * p.lddys + cv, p.H - cv);
                }
            }
        }
    }
    for (int d = min(p.lanes, 32) >> 1; d >= 1; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
    if (p.lanes > 32) {
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = dot;
        __syncthreads();
        dot = 0.f;
        if (at == 0)
            for (int i = 0; i < p.lanes / 32; ++i) dot += part[threadIdx.x / 32 + i];
    }
    if (at == 0 && live) p.dweights[slot] = dot;
}

template <typename Args>
cudaError_t launch_pdl(void (*kern)(const Args), unsigned grid, unsigned threads, size_t smem, cudaStream_t stream, const Args &args) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args);
    return e != cudaSuccess ? e : cudaPeekAtLastError();
}

int type_bytes(int type) { return type == kOutF32 ? 4 : 2; }

template <int XT, bool VEC>
cudaError_t launch_combine(CombineArgs a, bool grad, cudaStream_t stream) {
    // Columns of a thread: as many as keep four to eight loads of 16 bytes in flight.
    const int u = grad ? 4 : a.k <= 2 ? 2 : 1;
    const long long units = grad ? static_cast<long long>(a.T) * a.k : a.T;
    a.lanes = 1;
    while (a.lanes < kCombineThreads && a.lanes * 8 * u < a.H) a.lanes *= 2;
    // Many slots: a warp each, whose sum needs no exchange between warps.
    if (grad && units >= 16LL * device_sm_count()) a.lanes = std::min(a.lanes, 32);
    a.tokens = kCombineThreads / a.lanes;
    const unsigned grid = static_cast<unsigned>((units + a.tokens - 1) / a.tokens);
    if (grad) return launch_pdl(combine_grad_kernel<XT, VEC, 4>, grid, kCombineThreads, 0, stream, a);
    if (a.k <= 2) return launch_pdl(combine_kernel<XT, VEC, 2, 2>, grid, kCombineThreads, 0, stream, a);
    if (a.k <= 4) return launch_pdl(combine_kernel<XT, VEC, 4, 1>, grid, kCombineThreads, 0, stream, a);
    return launch_pdl(combine_kernel<XT, VEC, 8, 1>, grid, kCombineThreads, 0, stream, a);
}

cudaError_t combine(const MoeCombine &c, bool grad, cudaStream_t stream) {
    CombineArgs a = {};
    a.T = c.T;
    a.k = c.top_k;
    a.H = c.H;
    a.R = c.R;
    a.Ys = c.Ys;
    a.ldys = c.ldys;
    a.rows = c.rows;
    a.weights = c.weights;
    a.Y = c.Y;
    a.ldy = c.ldy;
    a.dYs = c.dYs;
    a.lddys = c.lddys;
    a.dweights = c.dweights;
    a.err = watchdog_word();
    if (kDebugBuild) {
        a.y_extent = grad ? static_cast<size_t>((c.R - 1LL) * c.lddys + c.H) : static_cast<size_t>((c.T - 1LL) * c.ldy + c.H);
        a.y_extent -= std::min(a.y_extent, debug_shrink_c());
    }
    const int b = type_bytes(c.type);
    const bool vec = rows_aligned(c.Ys, c.ldys, b, c.R) && rows_aligned(c.Y, c.ldy, b, c.T) && (!grad || rows_aligned(c.dYs, c.lddys, b, c.R));
    switch (c.type * 2 + (vec ? 1 : 0)) {
        case 0: return launch_combine<kOutF32, false>(a, grad, stream);
        case 1: return launch_combine<kOutF32, true>(a, grad, stream);
        case 2: return launch_combine<kOutF16, false>(a, grad, stream);
        case 3: return launch_combine<kOutF16, true>(a, grad, stream);
        case 4: return launch_combine<kOutBF16, false>(a, grad, stream);
        default: return launch_combine<kOutBF16, true>(a, grad, stream);
    }
}

}  // namespace

cudaError_t run_moe_dispatch(const MoeDispatch &d, cudaStream_t stream, CallInfo *info) {
    DispatchArgs a = {};
    const int b = type_bytes(d.x_type);
    a.T = d.T;
    a.E = d.E;
    a.k = d.top_k;
    a.n = d.T * d.top_k;
    a.ids = d.ids;
    a.X = static_cast<const uint8_t *>(d.X);
    a.x_bytes = d.ldx * b;
    a.Xs = static_cast<uint8_t *>(d.Xs);
    a.xs_bytes = d.ldxs * b;
    a.row_bytes = d.H * b;
    a.esize = b;
    a.offsets = d.offsets;
    a.rows = d.rows;
    a.err = watchdog_word();
    if (kDebugBuild && d.H > 0) {
        a.xs_extent = static_cast<size_t>((a.n - 1LL) * a.xs_bytes + a.row_bytes);
        a.xs_extent -= std::min(a.xs_extent, debug_shrink_c() * b);
    }
    const bool vec = rows_aligned(d.X, d.ldx, b, d.T) && rows_aligned(d.Xs, d.ldxs, b, a.n);
    const int grid = std::max(1, std::min(d.T, device_sm_count()));
    a.per_cta = std::max(1, (d.T + grid - 1) / grid);
    const unsigned ctas = static_cast<unsigned>(std::max(1LL, (static_cast<long long>(d.T) + a.per_cta - 1) / a.per_cta));
    a.copies = a.n >= 4096 ? 8 : 1;
    while (a.copies > 1 && 2u * sizeof(int) * d.E * a.copies > 32768u) a.copies /= 2;
    const size_t smem = 2u * sizeof(int) * d.E * a.copies;
    info->plan = vec ? "moe_dispatch" : "moe_dispatch_unaligned";
    info->launches = 1;
    if (vec && a.row_bytes % 16 == 0 && a.row_bytes >= kBulkBytes && a.row_bytes <= kBulkSmem) {
        a.pitch = (a.row_bytes + 127) & ~127;
        const size_t first = (smem + 127) & ~size_t(127);
        const int buffers = static_cast<int>(std::min<size_t>({(kBulkSmem - first) / a.pitch, static_cast<size_t>(a.per_cta), static_cast<size_t>(kMaxBuffers)}));
        if (buffers >= std::min(a.per_cta, kMinBuffers)) {
            a.depth = (buffers + kSortThreads / 32 - 1) / (kSortThreads / 32);
            a.warps = buffers / a.depth;
            static unsigned long long smem_set = 0;
            const cudaError_t e = ensure_dynamic_smem(dispatch_kernel<kBulk>, kBulkSmem, smem_set);
            if (e != cudaSuccess) return e;
            return launch_pdl(dispatch_kernel<kBulk>, ctas, kSortThreads, first + static_cast<size_t>(a.warps) * a.depth * a.pitch, stream, a);
        }
    }
    return vec ? launch_pdl(dispatch_kernel<kVectors>, ctas, kSortThreads, smem, stream, a) : launch_pdl(dispatch_kernel<kElements>, ctas, kSortThreads, smem, stream, a);
}

cudaError_t run_moe_combine(const MoeCombine &c, cudaStream_t stream, CallInfo *info) {
    info->plan = "moe_combine";
    info->launches = 1;
    return combine(c, false, stream);
}

cudaError_t run_moe_combine_grad(const MoeCombine &c, cudaStream_t stream, CallInfo *info) {
    info->plan = "moe_combine_grad";
    info->launches = 1;
    return combine(c, true, stream);
}

}  // namespace gemm11

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
// are summed, so no inverse of the order is stored.  Nothing is added with
// atomics, so the results do not depend on the order in which CTAs run.
#include <algorithm>
#include <cstdint>

#include "experts.h"
#include "rows8.cuh"

namespace gemm11 {
namespace {

constexpr int kSortThreads = 1024;
constexpr int kSortBatch = 1024;  // slots that are ranked and then copied together

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
    unsigned *err;
    size_t xs_extent;  // bytes, checked by GEMM11_DEBUG builds
};

// One segment of a row to its k copies: U times 16 bytes a lane.
template <int U>
__device__ __forceinline__ void copy_vec(const DispatchArgs &p, const uint8_t *from, const int *pos, int c0, int lane) {
    const int full = p.row_bytes >> 4;
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int c = c0 + u * 32 + lane;
        if (c < full) v[u] = __ldg(reinterpret_cast<const uint4 *>(from) + c);
    }
    for (int j = 0; j < p.k; ++j) {
        const int r = pos[j];
        if (r < 0) continue;
        uint8_t *to = p.Xs + r * p.xs_bytes;
        if (!debug_in_bounds(static_cast<size_t>(r * p.xs_bytes + p.row_bytes) <= p.xs_extent, p.err)) continue;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + u * 32 + lane;
            if (c < full) reinterpret_cast<uint4 *>(to)[c] = v[u];
        }
    }
}

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
// that it knows where its slots go without waiting for another CTA.
template <bool VEC>
__global__ void __launch_bounds__(kSortThreads) dispatch_kernel(const DispatchArgs p) {
    extern __shared__ int counts[];  // of each expert: slots before this CTA's, then the others
    __shared__ int warp_sum[32];
    __shared__ int pos[kSortBatch];
    int *before = counts, *rest = counts + p.E;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t0 = blockIdx.x * p.per_cta, t1 = min(p.T, t0 + p.per_cta);
    pdl_wait();
    pdl_launch_dependents();
    for (int e = threadIdx.x; e < 2 * p.E; e += kSortThreads) counts[e] = 0;
    __syncthreads();
    const int mine = t0 * p.k;
    for (int i = threadIdx.x; i < p.n; i += kSortThreads) {
        const int e = __ldg(p.ids + i);
        if (static_cast<unsigned>(e) < static_cast<unsigned>(p.E)) atomicAdd((i < mine ? before : rest) + e, 1);
    }
    __syncthreads();

    // before[e] becomes the row of this CTA's first slot of expert e.
    constexpr int kPer = kDispatchMaxExperts / kSortThreads;
    int total[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = threadIdx.x * kPer + i;
        total[i] = e < p.E ? before[e] + rest[e] : 0;
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
        const int e = threadIdx.x * kPer + i;
        if (e < p.E) {
            before[e] += start;
            if (blockIdx.x == 0) p.offsets[e] = start;
        }
        start += total[i];
    }
    if (blockIdx.x == 0 && threadIdx.x == kSortThreads - 1) p.offsets[p.E] = start;
    __syncthreads();

    const int batch = kSortBatch / p.k;  // tokens
    const int segments = VEC ? (p.row_bytes + 2047) / 2048 : (p.row_bytes / p.esize + 127) / 128;
    for (int t = t0; t < t1; t += batch) {
        const int tokens = min(batch, t1 - t), slots = tokens * p.k;
        if (warp == 0) {
            for (int i0 = 0; i0 < slots; i0 += 32) {
                const int i = i0 + lane;
                int e = i < slots ? __ldg(p.ids + t * p.k + i) : -1;
                if (static_cast<unsigned>(e) >= static_cast<unsigned>(p.E)) e = -1;
                const unsigned same = __match_any_sync(0xffffffffu, e);
                const int r = e >= 0 ? before[e] + __popc(same & ((1u << lane) - 1u)) : -1;
                __syncwarp();
                if (e >= 0 && lane == __ffs(same) - 1) before[e] += __popc(same);
                __syncwarp();
                if (i < slots) {
                    pos[i] = r;
                    p.rows[t * p.k + i] = r;
                }
            }
        }
        __syncthreads();
        if (p.row_bytes > 0) {
            for (int u = warp; u < tokens * segments; u += kSortThreads / 32) {
                const int i = u / segments, s = u % segments;
                const uint8_t *from = p.X + static_cast<long long>(t + i) * p.x_bytes;
                const int *to = pos + i * p.k;
                if (VEC) {
                    copy_vec<4>(p, from, to, s * 128, lane);
                    const int elements = p.row_bytes / p.esize, whole = (p.row_bytes >> 4) * (16 / p.esize);
                    if (s == segments - 1 && whole < elements) {
                        if (p.esize == 2)
                            copy_elements<uint16_t>(p, from, to, whole, elements, lane);
                        else
                            copy_elements<uint32_t>(p, from, to, whole, elements, lane);
                    }
                } else {
                    const int first = s * 128, last = min(first + 128, p.row_bytes / p.esize);
                    if (p.esize == 2)
                        copy_elements<uint16_t>(p, from, to, first, last, lane);
                    else
                        copy_elements<uint32_t>(p, from, to, first, last, lane);
                }
            }
        }
        __syncthreads();
    }
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
    int lanes;  // threads of a token, 8 columns each (a power of two, 256 at most)
    int tokens; // of a CTA: kCombineThreads / lanes
    unsigned *err;
    size_t y_extent;  // elements of what is written, checked by GEMM11_DEBUG builds
};
constexpr int kCombineThreads = 256;

// Row of slot i, -1 where it has none.
__device__ __forceinline__ int slot_row(const CombineArgs &p, long long i) {
    const int r = __ldg(p.rows + i);
    return static_cast<unsigned>(r) < static_cast<unsigned>(p.R) ? r : -1;
}

// A thread has eight columns of a token and reads the KU rows of a step before
// it adds them, in the order of the slots.
template <int XT, bool VEC, int KU>
__global__ void __launch_bounds__(kCombineThreads) combine_kernel(const CombineArgs p) {
    pdl_wait();
    pdl_launch_dependents();
    const long long t = static_cast<long long>(blockIdx.x) * p.tokens + threadIdx.x / p.lanes;
    if (t >= p.T) return;
    for (int c = static_cast<int>(threadIdx.x % p.lanes) * 8; c < p.H; c += p.lanes * 8) {
        float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int j0 = 0; j0 < p.k; j0 += KU) {
            Row8<XT> y[KU];
            float w[KU];
            int r[KU];
#pragma unroll
            for (int u = 0; u < KU; ++u) {
                r[u] = j0 + u < p.k ? slot_row(p, t * p.k + j0 + u) : -1;
                w[u] = p.weights && r[u] >= 0 ? __ldg(p.weights + t * p.k + j0 + u) : 1.f;
                if (r[u] >= 0) y[u].template load<VEC>(p.Ys, r[u] * p.ldys + c, p.H - c);
            }
#pragma unroll
            for (int u = 0; u < KU; ++u) {
                if (r[u] < 0) continue;
                float v[8];
                y[u].widen(v);
#pragma unroll
                for (int i = 0; i < 8; ++i) sum[i] = fmaf(w[u], v[i], sum[i]);
            }
        }
        Row8<XT> out;
        out.round(sum);
        if (debug_in_bounds(static_cast<size_t>(t * p.ldy + min(c + 8, p.H)) <= p.y_extent, p.err)) out.template store<VEC>(p.Y, t * p.ldy + c, p.H - c);
    }
}

// The gradient: KU slots at a time, whose dot products stay in registers while
// the columns pass and are then added over the token's threads.
template <int XT, bool VEC, int KU>
__global__ void __launch_bounds__(kCombineThreads) combine_grad_kernel(const CombineArgs p) {
    __shared__ float part[kCombineThreads / 32][KU];
    pdl_wait();
    pdl_launch_dependents();
    const int mine = threadIdx.x / p.lanes, at = threadIdx.x % p.lanes;
    const long long t = static_cast<long long>(blockIdx.x) * p.tokens + mine;
    const bool live = t < p.T;
    for (int j0 = 0; j0 < p.k; j0 += KU) {
        float w[KU], dot[KU];
        int r[KU];
#pragma unroll
        for (int u = 0; u < KU; ++u) {
            r[u] = live && j0 + u < p.k ? slot_row(p, t * p.k + j0 + u) : -1;
            w[u] = r[u] >= 0 ? __ldg(p.weights + t * p.k + j0 + u) : 0.f;
            dot[u] = 0.f;
        }
        if (live) {
            for (int c = at * 8; c < p.H; c += p.lanes * 8) {
                Row8<XT> dy, y[KU];
                dy.template load<VEC>(p.Y, t * p.ldy + c, p.H - c);
#pragma unroll
                for (int u = 0; u < KU; ++u)
                    if (r[u] >= 0) y[u].template load<VEC>(p.Ys, r[u] * p.ldys + c, p.H - c);
                float d[8];
                dy.widen(d);
#pragma unroll
                for (int u = 0; u < KU; ++u) {
                    if (r[u] < 0) continue;
                    float v[8];
                    y[u].widen(v);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        dot[u] = fmaf(d[i], v[i], dot[u]);
                        v[i] = w[u] * d[i];
                    }
                    Row8<XT> out;
                    out.round(v);
                    if (debug_in_bounds(static_cast<size_t>(r[u] * p.lddys + min(c + 8, p.H)) <= p.y_extent, p.err))
                        out.template store<VEC>(p.dYs, r[u] * p.lddys + c, p.H - c);
                }
            }
        }
        const int within = min(p.lanes, 32);
#pragma unroll
        for (int u = 0; u < KU; ++u)
            for (int d = within >> 1; d >= 1; d >>= 1) dot[u] += __shfl_xor_sync(0xffffffffu, dot[u], d);
        if (p.lanes <= 32) {
            if (at == 0 && live) {
#pragma unroll
                for (int u = 0; u < KU; ++u)
                    if (j0 + u < p.k) p.dweights[t * p.k + j0 + u] = dot[u];
            }
        } else {
            __syncthreads();  // the last step's sums are read
            if ((threadIdx.x & 31) == 0) {
#pragma unroll
                for (int u = 0; u < KU; ++u) part[threadIdx.x >> 5][u] = dot[u];
            }
            __syncthreads();
            if (live && at < KU && j0 + at < p.k) {
                float s = 0.f;
                for (int i = 0; i < p.lanes / 32; ++i) s += part[mine * (p.lanes / 32) + i][at];
                p.dweights[t * p.k + j0 + at] = s;
            }
        }
    }
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
cudaError_t launch_combine(const CombineArgs &a, bool grad, cudaStream_t stream) {
    const unsigned grid = static_cast<unsigned>((a.T + a.tokens - 1) / a.tokens);
    if (grad) {
        if (a.k <= 2) return launch_pdl(combine_grad_kernel<XT, VEC, 2>, grid, kCombineThreads, 0, stream, a);
        if (a.k <= 4) return launch_pdl(combine_grad_kernel<XT, VEC, 4>, grid, kCombineThreads, 0, stream, a);
        return launch_pdl(combine_grad_kernel<XT, VEC, 8>, grid, kCombineThreads, 0, stream, a);
    }
    if (a.k <= 2) return launch_pdl(combine_kernel<XT, VEC, 2>, grid, kCombineThreads, 0, stream, a);
    if (a.k <= 4) return launch_pdl(combine_kernel<XT, VEC, 4>, grid, kCombineThreads, 0, stream, a);
    return launch_pdl(combine_kernel<XT, VEC, 8>, grid, kCombineThreads, 0, stream, a);
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
    a.lanes = 1;
    while (a.lanes < 256 && a.lanes * 8 < c.H) a.lanes *= 2;
    a.tokens = kCombineThreads / a.lanes;
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
    const int grid = std::max(1, std::min(d.T, device_sm_count()));
    a.per_cta = (d.T + grid - 1) / grid;
    const unsigned ctas = static_cast<unsigned>(std::max(1, a.per_cta ? (d.T + a.per_cta - 1) / a.per_cta : 1));
    const bool vec = rows_aligned(d.X, d.ldx, b, d.T) && rows_aligned(d.Xs, d.ldxs, b, a.n);
    const size_t smem = 2u * sizeof(int) * d.E;
    info->plan = vec ? "moe_dispatch" : "moe_dispatch_unaligned";
    info->launches = 1;
    return vec ? launch_pdl(dispatch_kernel<true>, ctas, kSortThreads, smem, stream, a) : launch_pdl(dispatch_kernel<false>, ctas, kSortThreads, smem, stream, a);
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

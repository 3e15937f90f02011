// api.cu -- the C ABI of libgemm11.so: argument checks, degenerate shapes,
// dispatch to the FP32 / FP16 paths, status codes, the per-(device, stream)
// split-K scratch and the device watchdog word.
#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <map>
#include <memory>
#include <mutex>
#include <utility>
#include <vector>

#include "../../include/gemm11.h"
#include "fp8.h"
#include "internal.h"
#include "ptx.cuh"

namespace gemm11 {

// One watchdog word per device (every device that loads the library holds a
// copy); kernels receive its address and OR kWatchdogTimeout into it.
__device__ unsigned g_watchdog_word;

namespace {

// One thread waits on an mbarrier that nothing ever arrives on, with the
// same bounded wait the GEMM pipelines use; when it gives up it records the
// timeout in the watchdog word exactly as they do.
__global__ void watchdog_probe_kernel(unsigned *err, unsigned long long limit_ns) {
    __shared__ uint64_t bar;
    if (threadIdx.x != 0) return;
    mbar_init(&bar, 1);
    fence_mbarrier_init();
    if (!mbar_wait(&bar, 0, limit_ns)) atomicOr(err, kWatchdogTimeout);
}

// GEMM11_DEBUG builds: guard bands of kCanaryBytes before and after every
// library-owned scratch buffer, filled with kCanaryByte; every call checks
// them after its own work (canary_check_kernel) and reports a corrupted band.
constexpr size_t kCanaryBytes = 4096;
constexpr unsigned char kCanaryByte = 0xA5;
constexpr unsigned kCanaryWord = 0xA5A5A5A5u;

__global__ void canary_check_kernel(const unsigned *lo, const unsigned *hi, int words, unsigned *err) {
    for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < words; i += gridDim.x * blockDim.x)
        if (lo[i] != kCanaryWord || hi[i] != kCanaryWord) atomicOr(err, kDebugCanaryFault);
}

// Test hook of debug builds: overwrite the first word of a guard band (memory
// that the library allocated, so the write is in bounds) to show the check
// catches it.
__global__ void canary_poke_kernel(unsigned *word) { *word = 0u; }

thread_local int t_last_cuda_error = 0;
thread_local const char *t_last_plan = "none";
thread_local int t_last_launches = 0;
thread_local char t_plan_buf[96];

// Record a finished call's plan for gemm_last_plan / gemm_last_launch_count.
void record_plan(const gemm11::CallInfo &info) {
    if (info.tuned) {
        std::snprintf(t_plan_buf, sizeof(t_plan_buf), "%s+tuned", info.plan);
        t_last_plan = t_plan_buf;
    } else {
        t_last_plan = info.plan;
    }
    t_last_launches = info.launches;
}

constexpr int kMaxDevices = 64;

struct DeviceState {
    std::once_flag once;
    int sm_count = 0;
    unsigned *watchdog = nullptr;
    cudaError_t init_error = cudaSuccess;
};
DeviceState g_dev[kMaxDevices];

// The buffers of one stream.
struct ScratchBuffer {
    void *at = nullptr;
    size_t bytes = 0;
};
struct ScratchEntry {
    ScratchBuffer partials, counters, operands;
};
// The buffers of one stream capture.  The graph that it makes holds their
// addresses, so they belong to that graph: no call outside the capture and no
// other graph gets them, and they live until the graph and its instances are
// destroyed, which `gone` says (set by the graph's user object; the memory is
// freed at a later call, since a destructor of one may not call CUDA).
struct CaptureScratch {
    int dev = 0;
    std::map<uintptr_t, ScratchEntry> streams;             // of each stream that takes part: its branches may overlap
    std::vector<std::pair<ScratchBuffer, bool>> buffers;   // all, outgrown ones too; whether counters
    std::atomic<bool> gone{false};
};
std::mutex g_scratch_mu;
std::map<std::pair<int, uintptr_t>, ScratchEntry> g_scratch;
// By capture id.  Never destroyed: a graph may outlive the library's statics.
std::map<unsigned long long, std::unique_ptr<CaptureScratch>> &g_captures = *new std::map<unsigned long long, std::unique_ptr<CaptureScratch>>;
std::atomic<int> g_captures_gone{0};

// Library scratch allocation: plain cudaMalloc in release builds; debug
// builds put a filled guard band of kCanaryBytes on both sides and hand out
// the address past the first band.
cudaError_t scratch_alloc(void **user, size_t bytes) {
    if (!kDebugBuild) return cudaMalloc(user, bytes);
    unsigned char *raw = nullptr;
    cudaError_t e = cudaMalloc(reinterpret_cast<void **>(&raw), bytes + 2 * kCanaryBytes);
    if (e != cudaSuccess) return e;
    e = cudaMemset(raw, kCanaryByte, kCanaryBytes);
    if (e == cudaSuccess) e = cudaMemset(raw + kCanaryBytes + bytes, kCanaryByte, kCanaryBytes);
    if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);  // the check runs on the call's stream
    if (e != cudaSuccess) {
        cudaFree(raw);
        return e;
    }
    *user = raw + kCanaryBytes;
    return cudaSuccess;
}
void scratch_free(void *user) {
    if (!user) return;
    cudaFree(kDebugBuild ? static_cast<unsigned char *>(user) - kCanaryBytes : user);
}
// Enqueue the guard-band check of one buffer (debug builds).
cudaError_t check_bands(const void *user, size_t bytes, unsigned *err, cudaStream_t stream) {
    if (!user) return cudaSuccess;
    const unsigned char *u = static_cast<const unsigned char *>(user);
    canary_check_kernel<<<4, 256, 0, stream>>>(reinterpret_cast<const unsigned *>(u - kCanaryBytes),
                                               reinterpret_cast<const unsigned *>(u + bytes),
                                               static_cast<int>(kCanaryBytes / 4), err);
    return cudaPeekAtLastError();
}

int current_device() {
    int d = 0;
    if (cudaGetDevice(&d) != cudaSuccess) return -1;
    return d;
}

DeviceState *device_state() {
    const int d = current_device();
    if (d < 0 || d >= kMaxDevices) return nullptr;
    DeviceState &s = g_dev[d];
    std::call_once(s.once, [&s, d] {
        cudaError_t e = cudaDeviceGetAttribute(&s.sm_count, cudaDevAttrMultiProcessorCount, d);
        if (e == cudaSuccess) e = cudaGetSymbolAddress(reinterpret_cast<void **>(&s.watchdog), g_watchdog_word);
        s.init_error = e;
    });
    return &s;
}

int fail_cuda(cudaError_t e) {
    t_last_cuda_error = static_cast<int>(e);
    return GEMM_ERR_CUDA;
}

}  // namespace

int current_device_id() { return current_device(); }

int device_sm_count() {
    DeviceState *s = device_state();
    return (s && s->sm_count > 0) ? s->sm_count : 1;
}

unsigned *watchdog_word() {
    DeviceState *s = device_state();
    return s ? s->watchdog : nullptr;
}

namespace {

// While a stream is being captured allocations need the relaxed capture mode.
class RelaxedCapture {
  public:
    RelaxedCapture() { error_ = cudaThreadExchangeStreamCaptureMode(&mode_); }
    ~RelaxedCapture() {
        if (error_ == cudaSuccess) (void)cudaThreadExchangeStreamCaptureMode(&mode_);
    }
    cudaError_t error() const { return error_; }

  private:
    cudaStreamCaptureMode mode_ = cudaStreamCaptureModeRelaxed;
    cudaError_t error_;
};

struct Capture {
    bool active = false;
    unsigned long long id = 0;
    cudaGraph_t graph = nullptr;
};
Capture capture_of(cudaStream_t stream) {
    Capture c;
    cudaStreamCaptureStatus st = cudaStreamCaptureStatusNone;
    if (cudaStreamGetCaptureInfo(stream, &st, &c.id, &c.graph) != cudaSuccess)
        (void)cudaGetLastError();  // the legacy stream while another one is captured
    else
        c.active = st == cudaStreamCaptureStatusActive;
    return c;
}

void CUDART_CB graph_gone(void *scratch) {
    static_cast<CaptureScratch *>(scratch)->gone.store(true);
    g_captures_gone.fetch_add(1);
}

// Free what belonged to graphs that are gone.
void collect_gone() {
    if (g_captures_gone.load() == 0) return;
    RelaxedCapture relaxed;
    if (relaxed.error() != cudaSuccess) return;
    for (auto it = g_captures.begin(); it != g_captures.end();) {
        if (!it->second->gone.load()) {
            ++it;
            continue;
        }
        for (auto &b : it->second->buffers) scratch_free(b.first.at);
        it = g_captures.erase(it);
        g_captures_gone.fetch_sub(1);
    }
}

// The buffers of the capture, which its graph keeps from the first call on.
cudaError_t capture_scratch(const Capture &c, int dev, CaptureScratch **out) {
    auto it = g_captures.find(c.id);
    if (it == g_captures.end()) {
        it = g_captures.emplace(c.id, std::make_unique<CaptureScratch>()).first;
        it->second->dev = dev;
        cudaUserObject_t object = nullptr;
        cudaError_t e = cudaUserObjectCreate(&object, it->second.get(), graph_gone, 1, cudaUserObjectNoDestructorSync);
        if (e != cudaSuccess) {
            g_captures.erase(it);
            return e;
        }
        e = cudaGraphRetainUserObject(c.graph, object, 1, cudaGraphUserObjectMove);
        if (e != cudaSuccess) {
            (void)cudaUserObjectRelease(object, 1);  // says that it is gone
            return e;
        }
    }
    *out = it->second.get();
    return cudaSuccess;
}

enum class ScratchKind { partials, counters, operands };

// At least `bytes` bytes of one kind for work on `stream`; new counters are zero.
cudaError_t acquire_buffer(cudaStream_t stream, int dev, const Capture &c, ScratchKind kind, size_t bytes, size_t preferred, void **out) {
    CaptureScratch *cs = nullptr;
    if (c.active) {
        const cudaError_t e = capture_scratch(c, dev, &cs);
        if (e != cudaSuccess) return e;
    }
    const uintptr_t key = reinterpret_cast<uintptr_t>(stream);
    ScratchEntry &entry = cs ? cs->streams[key] : g_scratch[{dev, key}];
    ScratchBuffer &b = kind == ScratchKind::partials ? entry.partials : kind == ScratchKind::counters ? entry.counters : entry.operands;
    const bool zero = kind == ScratchKind::counters;
    if (b.bytes < bytes && cs) {
        // Nothing may wait for a stream that is captured; new counters are
        // cleared on a stream of their own, outside the graph.  An outgrown
        // buffer stays with the graph, whose earlier work uses it.
        RelaxedCapture relaxed;
        cudaError_t e = relaxed.error();
        if (e != cudaSuccess) return e;
        cs->buffers.reserve(cs->buffers.size() + 1);
        ScratchBuffer fresh;
        e = scratch_alloc(&fresh.at, bytes);
        if (e != cudaSuccess) return e;
        fresh.bytes = bytes;
        cs->buffers.emplace_back(fresh, zero);
        if (zero) {
            cudaStream_t side = nullptr;
            e = cudaStreamCreateWithFlags(&side, cudaStreamNonBlocking);
            if (e == cudaSuccess) e = cudaMemsetAsync(fresh.at, 0, bytes, side);
            if (e == cudaSuccess) e = cudaStreamSynchronize(side);
            if (side) cudaStreamDestroy(side);
            if (e != cudaSuccess) return e;
        }
        b = fresh;
    } else if (b.bytes < bytes) {
        cudaError_t e = cudaStreamSynchronize(stream);  // work already queued may still use the old buffer
        if (e != cudaSuccess) return e;
        scratch_free(b.at);
        b = ScratchBuffer();
        const size_t want = std::max(bytes, preferred);
        e = scratch_alloc(&b.at, want);
        // On the call's stream: the default stream's work is not ordered with
        // that of a non-blocking stream.
        if (e == cudaSuccess && zero) e = cudaMemsetAsync(b.at, 0, want, stream);
        if (e != cudaSuccess) return e;
        b.bytes = want;
    }
    *out = b.at;
    return cudaSuccess;
}

}  // namespace

cudaError_t acquire_scratch(cudaStream_t stream, size_t partial_floats, size_t ncounters, Scratch *out) try {
    const int dev = current_device();
    if (dev < 0) return cudaErrorInvalidDevice;
    const Capture c = capture_of(stream);
    std::lock_guard<std::mutex> lock(g_scratch_mu);
    collect_gone();
    void *partials = nullptr, *counters = nullptr;
    cudaError_t e = acquire_buffer(stream, dev, c, ScratchKind::partials, partial_floats * sizeof(float),
                                   (partial_floats + partial_floats / 4) * sizeof(float), &partials);
    if (e == cudaSuccess)
        e = acquire_buffer(stream, dev, c, ScratchKind::counters, ncounters * sizeof(unsigned),
                           (ncounters < 1024 ? 1024 : ncounters + ncounters / 4) * sizeof(unsigned), &counters);
    out->partials = static_cast<float *>(partials);
    out->counters = static_cast<unsigned *>(counters);
    return e;
} catch (...) {
    return cudaErrorMemoryAllocation;  // of the tables
}

cudaError_t acquire_operand_scratch(cudaStream_t stream, size_t floats, float **out) try {
    const int dev = current_device();
    if (dev < 0) return cudaErrorInvalidDevice;
    const Capture c = capture_of(stream);
    std::lock_guard<std::mutex> lock(g_scratch_mu);
    collect_gone();
    void *at = nullptr;
    const cudaError_t e = acquire_buffer(stream, dev, c, ScratchKind::operands, floats * sizeof(float), 0, &at);
    *out = static_cast<float *>(at);
    return e;
} catch (...) {
    return cudaErrorMemoryAllocation;
}

size_t debug_shrink_c() {
    if (!kDebugBuild) return 0;
    const char *v = std::getenv("GEMM11_DEBUG_SHRINK_C");
    return v ? static_cast<size_t>(std::strtoull(v, nullptr, 10)) : 0;
}

namespace {

// Read and clear the current device's status word after synchronising
// `stream`; maps its bits to a status.  A non-zero word also resets the
// split-K arrival counters (a CTA that gave up may have left them non-zero).
int read_status_word(DeviceState *ds, cudaStream_t stream) {
    cudaError_t e = cudaStreamSynchronize(stream);
    if (e != cudaSuccess) return fail_cuda(e);
    unsigned word = 0;
    e = cudaMemcpy(&word, ds->watchdog, sizeof(word), cudaMemcpyDeviceToHost);
    if (e != cudaSuccess) return fail_cuda(e);
    if (word == 0) return GEMM_OK;
    const int dev = current_device();
    {
        std::lock_guard<std::mutex> lock(g_scratch_mu);
        for (auto &kv : g_scratch)
            if (kv.first.first == dev && kv.second.counters.at) {
                e = cudaMemset(kv.second.counters.at, 0, kv.second.counters.bytes);
                if (e != cudaSuccess) return fail_cuda(e);
            }
        for (auto &kv : g_captures)
            for (auto &b : kv.second->buffers)
                if (kv.second->dev == dev && b.second) {
                    e = cudaMemset(b.first.at, 0, b.first.bytes);
                    if (e != cudaSuccess) return fail_cuda(e);
                }
    }
    const unsigned zero = 0;
    e = cudaMemcpy(ds->watchdog, &zero, sizeof(zero), cudaMemcpyHostToDevice);
    if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);  // the next call may be on any stream
    if (e != cudaSuccess) return fail_cuda(e);
    return (word & (kDebugBoundsFault | kDebugCanaryFault)) ? GEMM_ERR_DEBUG_CHECK : GEMM_ERR_TIMEOUT;
}

// The end of every call that enqueued work: record its plan; GEMM11_DEBUG
// builds also check the guard bands of this stream's scratch, wait for the
// call's work and report what the device-side checks found ("start fully
// synchronous").
int finish_call(const CallInfo &info, cudaStream_t stream) {
    record_plan(info);
    if (!kDebugBuild) return GEMM_OK;
    DeviceState *ds = device_state();
    if (!ds) return fail_cuda(cudaErrorInvalidDevice);
    const int dev = current_device();
    {
        std::lock_guard<std::mutex> lock(g_scratch_mu);
        auto it = g_scratch.find({dev, reinterpret_cast<uintptr_t>(stream)});
        if (it != g_scratch.end()) {
            ScratchEntry &se = it->second;
            const char *poke = std::getenv("GEMM11_DEBUG_POKE_CANARY");
            if (poke && poke[0] == '1' && se.partials.at) {
                canary_poke_kernel<<<1, 1, 0, stream>>>(
                    reinterpret_cast<unsigned *>(static_cast<unsigned char *>(se.partials.at) + se.partials.bytes));
            }
            cudaError_t e = cudaSuccess;
            for (const ScratchBuffer *b : {&se.partials, &se.counters, &se.operands})
                if (e == cudaSuccess) e = check_bands(b->at, b->bytes, ds->watchdog, stream);
            if (e != cudaSuccess) return fail_cuda(e);
        }
    }
    return read_status_word(ds, stream);
}

}  // namespace
}  // namespace gemm11

using namespace gemm11;

// ------------------------------------------------------------------ tuning table
namespace {

struct TuneKey {
    int path, M, N, K;
    bool operator<(const TuneKey &o) const {
        if (path != o.path) return path < o.path;
        if (M != o.M) return M < o.M;
        if (N != o.N) return N < o.N;
        return K < o.K;
    }
};
std::mutex g_tune_mutex;
std::map<TuneKey, TunePlan> g_tune_table;
std::atomic<bool> g_tune_any{false};  // lets every call skip the lock while the table is empty

bool valid_tune_entry(const gemm_tune_entry &e) {
    if (e.M < 0 || e.N < 0 || e.K < 0 || e.splits < 0 || e.splits > 32) return false;
    if (e.path == GEMM_PATH_F32) return (e.variant == 1 && e.bn == 0) || (e.variant == 2 && e.bn == 0);
    if (e.path != GEMM_PATH_TC) return false;
    switch (e.variant) {
        case 1: return e.bn == 0 || e.bn == 256 || e.bn == 224 || e.bn == 192;
        case 2: return e.bn == 0 || e.bn == 256 || e.bn == 128;
        case 3: return e.bn == 0 || e.bn == 32 || e.bn == 64;
        case 4: return (e.bn == 0 || e.bn == 256 || e.bn == 192 || e.bn == 128) && (e.splits == 0 || (e.splits >= 2 && e.splits <= 8));
        default: return false;
    }
}

}  // namespace

namespace gemm11 {
bool tune_lookup(int path, int M, int N, int K, TunePlan *out) {
    if (!g_tune_any.load(std::memory_order_acquire)) return false;
    std::lock_guard<std::mutex> lock(g_tune_mutex);
    auto it = g_tune_table.find(TuneKey{path, M, N, K});
    if (it == g_tune_table.end()) return false;
    *out = it->second;
    return true;
}
}  // namespace gemm11

extern "C" {

int gemm_tune_set(const gemm_tune_entry *entries, int n) {
    if (n < 0 || (n > 0 && !entries)) return GEMM_ERR_INVALID_ARG;
    for (int i = 0; i < n; ++i)
        if (!valid_tune_entry(entries[i])) return GEMM_ERR_INVALID_ARG;
    std::map<TuneKey, TunePlan> table;
    for (int i = 0; i < n; ++i) {
        const gemm_tune_entry &e = entries[i];
        TunePlan tp;
        tp.variant = e.variant;
        tp.bn = e.bn;
        tp.splits = e.splits;
        table[TuneKey{e.path, e.M, e.N, e.K}] = tp;
    }
    std::lock_guard<std::mutex> lock(g_tune_mutex);
    g_tune_table.swap(table);
    g_tune_any.store(!g_tune_table.empty(), std::memory_order_release);
    return GEMM_OK;
}

int gemm_tune_get(gemm_tune_entry *out, int capacity) {
    std::lock_guard<std::mutex> lock(g_tune_mutex);
    int i = 0;
    for (const auto &kv : g_tune_table) {
        if (out && i < capacity) {
            gemm_tune_entry &e = out[i];
            e.path = kv.first.path;
            e.M = kv.first.M;
            e.N = kv.first.N;
            e.K = kv.first.K;
            e.variant = kv.second.variant;
            e.bn = kv.second.bn;
            e.splits = kv.second.splits;
        }
        ++i;
    }
    return i;
}


int gemm_f32(int M, int N, int K, float alpha, const float *A, int lda, const float *B, int ldb, float beta,
             float *C, int ldc, void *stream) {
    if (M < 0 || N < 0 || K < 0) return GEMM_ERR_INVALID_ARG;
    if (lda < (K > 1 ? K : 1) || ldb < (N > 1 ? N : 1) || ldc < (N > 1 ? N : 1)) return GEMM_ERR_INVALID_ARG;
    if (M == 0 || N == 0) {
        t_last_plan = "noop_empty";
        t_last_launches = 0;
        return GEMM_OK;
    }
    if (!C) return GEMM_ERR_INVALID_ARG;
    const bool product = (K > 0) && (alpha != 0.f);
    if (product && (!A || !B)) return GEMM_ERR_INVALID_ARG;
    DeviceState *ds = device_state();
    if (!ds) return fail_cuda(cudaErrorInvalidDevice);
    if (ds->init_error != cudaSuccess) return fail_cuda(ds->init_error);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    CallInfo info;
    cudaError_t e = product ? run_gemm_f32(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, s, &info)
                            : run_scale_c(M, N, beta, C, ldc, nullptr, 0, s, &info);
    if (e != cudaSuccess) return fail_cuda(e);
    return finish_call(info, s);
}

int gemm_f32_3xtf32(int M, int N, int K, float alpha, const float *A, int lda, const float *B, int ldb, float beta,
                    float *C, int ldc, void *stream) {
    if (M < 0 || N < 0 || K < 0) return GEMM_ERR_INVALID_ARG;
    if (lda < (K > 1 ? K : 1) || ldb < (N > 1 ? N : 1) || ldc < (N > 1 ? N : 1)) return GEMM_ERR_INVALID_ARG;
    if (M == 0 || N == 0) {
        t_last_plan = "noop_empty";
        t_last_launches = 0;
        return GEMM_OK;
    }
    if (!C) return GEMM_ERR_INVALID_ARG;
    const bool product = (K > 0) && (alpha != 0.f);
    if (product && (!A || !B)) return GEMM_ERR_INVALID_ARG;
    // C is written by TMA stores: 16-byte aligned base and rows (a single row
    // has no row stride to align).
    if (product && (((reinterpret_cast<uintptr_t>(C) & 15u) != 0) || (M > 1 && (ldc % 4) != 0)))
        return GEMM_ERR_UNSUPPORTED;
    DeviceState *ds = device_state();
    if (!ds) return fail_cuda(cudaErrorInvalidDevice);
    if (ds->init_error != cudaSuccess) return fail_cuda(ds->init_error);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    CallInfo info;
    cudaError_t e = product ? run_gemm_f32_3xtf32(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, s, &info)
                            : run_scale_c(M, N, beta, C, ldc, nullptr, 0, s, &info);
    if (e == cudaErrorNotSupported) return GEMM_ERR_UNSUPPORTED;
    if (e != cudaSuccess) return fail_cuda(e);
    return finish_call(info, s);
}

}  // extern "C"

namespace {

bool valid_act(int act) { return act >= GEMM_ACT_NONE && act <= GEMM_ACT_GELU_TANH; }
bool valid_fp8(int type) { return type == GEMM_DTYPE_E4M3 || type == GEMM_DTYPE_E5M2; }

// The largest extent of a matrix held in 8 bits: the kernels' indices run over
// the end of one by less than two tiles.
constexpr int kMaxExtent = 0x7FFFFFFF - 511;

// A call with an empty result.
int noop() {
    t_last_plan = "noop_empty";
    t_last_launches = 0;
    return GEMM_OK;
}

// The tensor-core entry points (FP16 or BF16 operands, FP32 accumulate,
// FP32/FP16/BF16 output, fused epilogue, optional strided batch and
// transposed B) share validation and planning.
int gemm_tc_checked(const TcGemm &g, int ab_type, void *stream) {
    if (g.batch < 0 || g.M < 0 || g.N < 0 || g.K < 0) return GEMM_ERR_INVALID_ARG;
    if (!valid_act(g.act)) return GEMM_ERR_INVALID_ARG;
    if (ab_type != GEMM_DTYPE_F16 && ab_type != GEMM_DTYPE_BF16) return GEMM_ERR_INVALID_ARG;
    if (g.c_type != GEMM_DTYPE_F32 && g.c_type != GEMM_DTYPE_F16 && g.c_type != GEMM_DTYPE_BF16)
        return GEMM_ERR_INVALID_ARG;
    if (g.b_trans != 0 && g.b_trans != 1) return GEMM_ERR_INVALID_ARG;
    if (g.batch == 0 || g.M == 0 || g.N == 0) {
        t_last_plan = "noop_empty";
        t_last_launches = 0;
        return GEMM_OK;
    }
    if (!g.C) return GEMM_ERR_INVALID_ARG;
    const long long mn = static_cast<long long>(g.M) * g.N;
    if (g.batch > 1 && (g.stride_a < 0 || g.stride_b < 0 || g.stride_c < mn)) return GEMM_ERR_INVALID_ARG;
    const bool product = (g.K > 0) && (g.alpha != 0.f);
    if (product && (!g.A || !g.B)) return GEMM_ERR_INVALID_ARG;
    // Tensor-map constraints: 16-byte aligned bases, row and matrix strides
    // (the epilogue-only path, alpha == 0 or K == 0, has none).
    auto al16 = [](const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
    if (product) {
        const bool ok = (g.K % 8 == 0) && (g.N % 8 == 0) && al16(g.A) && al16(g.B) && al16(g.C) &&
                        (g.batch == 1 || (g.stride_a % 8 == 0 && g.stride_b % 8 == 0 && g.stride_c % 8 == 0));
        if (!ok) return GEMM_ERR_UNSUPPORTED;
    }
    DeviceState *ds = device_state();
    if (!ds) return fail_cuda(cudaErrorInvalidDevice);
    if (ds->init_error != cudaSuccess) return fail_cuda(ds->init_error);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    CallInfo info;
    cudaError_t e;
    if (!product) {
        e = run_scale_c_batched(g.batch, g.M, g.N, g.beta, g.C, g.batch > 1 ? g.stride_c : mn, g.c_type, g.bias,
                                g.act, s, &info);
    } else {
        TcGemm gg = g;
        gg.bf16 = ab_type == GEMM_DTYPE_BF16;
        if (gg.batch == 1) gg.stride_a = gg.stride_b = 0, gg.stride_c = mn;
        e = run_gemm_f16(gg, s, &info);
        if (e == cudaErrorNotSupported) return GEMM_ERR_UNSUPPORTED;
    }
    if (e != cudaSuccess) return fail_cuda(e);
    return finish_call(info, s);
}

TcGemm tc_single(int M, int N, int K, float alpha, const void *A, const void *B, float beta, void *C, int c_type,
                 const float *bias, int act) {
    TcGemm g;
    g.M = M;
    g.N = N;
    g.K = K;
    g.alpha = alpha;
    g.A = A;
    g.B = B;
    g.beta = beta;
    g.C = C;
    g.c_type = c_type;
    g.bias = bias;
    g.act = act;
    return g;
}

}  // namespace

extern "C" {

int gemm_f16_f32acc_epilogue(int M, int N, int K, float alpha, const void *A, const void *B, float beta, float *C,
                             const float *bias, int act, void *stream) {
    return gemm_tc_checked(tc_single(M, N, K, alpha, A, B, beta, C, GEMM_DTYPE_F32, bias, act), GEMM_DTYPE_F16,
                           stream);
}

int gemm_bf16_f32acc_epilogue(int M, int N, int K, float alpha, const void *A, const void *B, float beta,
                              float *C, const float *bias, int act, void *stream) {
    return gemm_tc_checked(tc_single(M, N, K, alpha, A, B, beta, C, GEMM_DTYPE_F32, bias, act), GEMM_DTYPE_BF16,
                           stream);
}

int gemm_tc_f32acc_epilogue(int M, int N, int K, float alpha, const void *A, const void *B, int ab_type, float beta,
                            void *C, int c_type, const float *bias, int act, void *stream) {
    return gemm_tc_checked(tc_single(M, N, K, alpha, A, B, beta, C, c_type, bias, act), ab_type, stream);
}

int gemm_tc_strided_batched(int batch, int M, int N, int K, float alpha, const void *A, long long stride_a,
                            const void *B, long long stride_b, int ab_type, int b_trans, float beta, void *C,
                            long long stride_c, int c_type, const float *bias, int act, void *stream) {
    TcGemm g = tc_single(M, N, K, alpha, A, B, beta, C, c_type, bias, act);
    g.batch = batch;
    g.stride_a = stride_a;
    g.stride_b = stride_b;
    g.stride_c = stride_c;
    g.b_trans = b_trans;
    return gemm_tc_checked(g, ab_type, stream);
}

int gemm_f16_f32acc_epilogue_noalloc(int M, int N, int K, float alpha, const void *A, const void *B, float beta,
                                     float *C, const float *bias, int act, void *stream) {
    if (M < 0 || N < 0 || K < 0) return GEMM_ERR_INVALID_ARG;
    if (!valid_act(act)) return GEMM_ERR_INVALID_ARG;
    if (M > 64) return GEMM_ERR_UNSUPPORTED;  // whatever alpha, K or N: this entry point is for M <= 64
    if (M == 0 || N == 0) {
        t_last_plan = "noop_empty";
        t_last_launches = 0;
        return GEMM_OK;
    }
    if (!C) return GEMM_ERR_INVALID_ARG;
    const bool product = (K > 0) && (alpha != 0.f);
    if (product && (!A || !B)) return GEMM_ERR_INVALID_ARG;
    if (product) {
        const bool ok = (K % 8 == 0) && (N % 8 == 0) && ((reinterpret_cast<uintptr_t>(A) & 15u) == 0) &&
                        ((reinterpret_cast<uintptr_t>(B) & 15u) == 0) &&
                        ((reinterpret_cast<uintptr_t>(C) & 15u) == 0);
        if (!ok) return GEMM_ERR_UNSUPPORTED;
    }
    DeviceState *ds = device_state();
    if (!ds) return fail_cuda(cudaErrorInvalidDevice);
    if (ds->init_error != cudaSuccess) return fail_cuda(ds->init_error);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    CallInfo info;
    cudaError_t e;
    if (!product) {
        e = run_scale_c(M, N, beta, C, N, bias, act, s, &info);
    } else {
        int reject = 0;
        e = run_gemm_f16_small_m_noalloc(M, N, K, alpha, A, B, beta, C, bias, act, s, &info, &reject);
        if (e == cudaErrorNotSupported) return GEMM_ERR_UNSUPPORTED;
        if (e == cudaSuccess && reject == 1) return GEMM_ERR_UNSUPPORTED;
        if (e == cudaSuccess && reject == 2) return GEMM_ERR_SCRATCH_LIMIT;
    }
    if (e != cudaSuccess) return fail_cuda(e);
    return finish_call(info, s);
}

int gemm_fp8_quantize_block128(int rows, int cols, const void *X, int x_type, long long ldx, void *Q, int q_type,
                               long long ldq, float *S, long long lds, int layout, void *stream) {
    if (rows < 0 || cols < 0 || layout < GEMM_FP8_ROWS || layout > GEMM_FP8_BLOCKS) return GEMM_ERR_INVALID_ARG;
    if (x_type != GEMM_DTYPE_F32 && x_type != GEMM_DTYPE_F16 && x_type != GEMM_DTYPE_BF16) return GEMM_ERR_INVALID_ARG;
    if (!valid_fp8(q_type)) return GEMM_ERR_INVALID_ARG;
    const long long q_cols = layout == GEMM_FP8_COLS ? rows : cols;
    const long long s_cols = layout == GEMM_FP8_ROWS ? rows : layout == GEMM_FP8_COLS ? cols : (cols + 127LL) / 128;
    if (ldx < std::max(1, cols) || ldq < std::max(1LL, q_cols) || lds < std::max(1LL, s_cols)) return GEMM_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return noop();
    if (!X || !Q || !S) return GEMM_ERR_INVALID_ARG;
    if (rows > kMaxExtent || cols > kMaxExtent) return GEMM_ERR_UNSUPPORTED;
    DeviceState *ds = device_state();
    if (!ds) return fail_cuda(cudaErrorInvalidDevice);
    if (ds->init_error != cudaSuccess) return fail_cuda(ds->init_error);
    Fp8Quant q;
    q.rows = rows;
    q.cols = cols;
    q.X = X;
    q.x_type = x_type;
    q.ldx = ldx;
    q.Q = Q;
    q.q_type = q_type;
    q.ldq = ldq;
    q.S = S;
    q.lds = lds;
    q.layout = layout;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    CallInfo info;
    const cudaError_t e = run_fp8_quantize(q, s, &info);
    if (e != cudaSuccess) return fail_cuda(e);
    return finish_call(info, s);
}

int gemm_fp8_block128(int M, int N, int K, float alpha, const void *A, int a_type, long long lda, const float *SA,
                      long long ldsa, const void *B, int b_type, long long ldb, const float *SB, long long ldsb,
                      int b_trans, int b_layout, float beta, void *C, int c_type, long long ldc, const float *bias,
                      int act, void *stream) {
    if (M < 0 || N < 0 || K < 0 || !valid_act(act) || !valid_fp8(a_type) || !valid_fp8(b_type)) return GEMM_ERR_INVALID_ARG;
    if (c_type != GEMM_DTYPE_F32 && c_type != GEMM_DTYPE_F16 && c_type != GEMM_DTYPE_BF16) return GEMM_ERR_INVALID_ARG;
    if (b_trans != 0 && b_trans != 1) return GEMM_ERR_INVALID_ARG;
    if (b_layout != GEMM_FP8_BLOCKS && !(b_layout == GEMM_FP8_ROWS && b_trans)) return GEMM_ERR_INVALID_ARG;
    const long long kb = (K + 127LL) / 128, nb = (N + 127LL) / 128;
    const bool b_rows = b_layout == GEMM_FP8_ROWS;
    if (lda < std::max(1, K) || ldb < std::max(1, b_trans ? K : N) || ldc < std::max(1, N) || ldsa < std::max(1, M) ||
        ldsb < std::max<long long>(1, b_rows ? N : b_trans ? kb : nb))
        return GEMM_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return noop();
    if (!C) return GEMM_ERR_INVALID_ARG;
    if (M > kMaxExtent || N > kMaxExtent || K > kMaxExtent) return GEMM_ERR_UNSUPPORTED;
    const bool product = K > 0 && alpha != 0.f;
    if (product) {
        if (!A || !SA || !B || !SB) return GEMM_ERR_INVALID_ARG;
        auto al16 = [](const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
        const bool ok = al16(A) && al16(B) && al16(SA) && (M == 1 || lda % 16 == 0) &&
                        ((b_trans ? N : K) == 1 || ldb % 16 == 0) && (kb == 1 || ldsa % 4 == 0) &&
                        (!b_rows || (al16(SB) && (kb == 1 || ldsb % 4 == 0)));
        if (!ok) return GEMM_ERR_UNSUPPORTED;
    }
    DeviceState *ds = device_state();
    if (!ds) return fail_cuda(cudaErrorInvalidDevice);
    if (ds->init_error != cudaSuccess) return fail_cuda(ds->init_error);
    Fp8Gemm g;
    g.M = M;
    g.N = N;
    g.K = K;
    g.alpha = alpha;
    g.A = A;
    g.a_type = a_type;
    g.lda = lda;
    g.SA = SA;
    g.ldsa = ldsa;
    g.B = B;
    g.b_type = b_type;
    g.ldb = ldb;
    g.SB = SB;
    g.ldsb = ldsb;
    g.b_trans = b_trans;
    g.b_rows = b_rows;
    g.beta = beta;
    g.C = C;
    g.c_type = c_type;
    g.ldc = ldc;
    g.bias = bias;
    g.act = act;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    CallInfo info;
    const cudaError_t e = product ? run_fp8_gemm(g, s, &info) : run_fp8_scale_c(g, s, &info);
    if (e == cudaErrorNotSupported) return GEMM_ERR_UNSUPPORTED;
    if (e != cudaSuccess) return fail_cuda(e);
    return finish_call(info, s);
}

int gemm_moe_few_tokens(int T, int E, int top_k, int H, int I, const void *X, int x_type, long long ldx,
                        const void *router, int router_type, const void *gate, const void *up, const void *down,
                        int w_type, const float *s_gate, const float *s_up, const float *s_down, int act,
                        int renormalize, void *Y, int y_type, long long ldy, int *ids, float *weights, void *stream) {
    static_assert(kActSilu == GEMM_ACT_SILU, "activation codes");
    if (T < 0 || E < 0 || H < 0 || I < 0 || (renormalize != 0 && renormalize != 1)) return GEMM_ERR_INVALID_ARG;
    if (!valid_act(act) && act != GEMM_ACT_SILU) return GEMM_ERR_INVALID_ARG;
    if (x_type != GEMM_DTYPE_F16 && x_type != GEMM_DTYPE_BF16) return GEMM_ERR_INVALID_ARG;
    if (router_type != GEMM_DTYPE_F32 && router_type != x_type) return GEMM_ERR_INVALID_ARG;
    if (w_type != x_type && w_type != GEMM_DTYPE_E4M3) return GEMM_ERR_INVALID_ARG;
    if (y_type != GEMM_DTYPE_F32 && y_type != GEMM_DTYPE_F16 && y_type != GEMM_DTYPE_BF16) return GEMM_ERR_INVALID_ARG;
    if (ldx < std::max(1, H) || ldy < std::max(1, H)) return GEMM_ERR_INVALID_ARG;
    if (T == 0 || H == 0) return noop();
    if (E < 1 || I < 1 || top_k < 1 || top_k > E) return GEMM_ERR_INVALID_ARG;
    if (!X || !router || !gate || !down || !Y) return GEMM_ERR_INVALID_ARG;
    const bool fp8 = w_type == GEMM_DTYPE_E4M3;
    if (fp8 && (!s_gate || !s_down || (up && !s_up))) return GEMM_ERR_INVALID_ARG;
    auto al16 = [](const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
    const bool ok = top_k <= kMoeMaxTopK && E <= kMoeMaxExperts && T <= kMoeMaxTokens && T * top_k <= kMoeMaxSlots &&
                    H <= kMoeMaxWidth && H % 16 == 0 && I % 16 == 0 && al16(X) && al16(router) && al16(gate) && al16(up) && al16(down) &&
                    (T == 1 || ldx % 8 == 0) && static_cast<long long>(E) * std::max(H, I) < (1LL << 31) &&
                    static_cast<long long>(T) * top_k * I < (1LL << 31);
    if (!ok) return GEMM_ERR_UNSUPPORTED;
    DeviceState *ds = device_state();
    if (!ds) return fail_cuda(cudaErrorInvalidDevice);
    if (ds->init_error != cudaSuccess) return fail_cuda(ds->init_error);
    Moe m;
    m.T = T;
    m.E = E;
    m.top_k = top_k;
    m.H = H;
    m.I = I;
    m.X = X;
    m.x_type = x_type;
    m.ldx = ldx;
    m.router = router;
    m.router_type = router_type;
    m.gate = gate;
    m.up = up;
    m.down = down;
    m.w_type = w_type;
    m.s_gate = s_gate;
    m.s_up = s_up;
    m.s_down = s_down;
    m.Y = Y;
    m.y_type = y_type;
    m.ldy = ldy;
    m.act = act;
    m.renorm = renormalize;
    m.ids = ids;
    m.weights = weights;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    CallInfo info;
    const cudaError_t e = run_moe(m, s, &info);
    if (e == cudaErrorNotSupported) return GEMM_ERR_UNSUPPORTED;
    if (e != cudaSuccess) return fail_cuda(e);
    return finish_call(info, s);
}

const char *gemm_status_string(int status) {
    switch (status) {
        case GEMM_OK: return "GEMM_OK";
        case GEMM_ERR_INVALID_ARG: return "GEMM_ERR_INVALID_ARG: invalid argument";
        case GEMM_ERR_UNSUPPORTED: return "GEMM_ERR_UNSUPPORTED: arguments outside this path's constraints";
        case GEMM_ERR_CUDA: return "GEMM_ERR_CUDA: a CUDA runtime call failed";
        case GEMM_ERR_DEBUG_CHECK:
            return "GEMM_ERR_DEBUG_CHECK: a device-side check of a GEMM11_DEBUG build failed (index out of range or "
                   "a scratch guard band overwritten)";
        case GEMM_ERR_TIMEOUT: return "GEMM_ERR_TIMEOUT: a bounded in-kernel wait ran out";
        case GEMM_ERR_SCRATCH_LIMIT:
            return "GEMM_ERR_SCRATCH_LIMIT: the shape needs more split-K scratch than the fixed no-allocation "
                   "buffer holds (4 MiB of partial tiles, 4096 counters)";
        default: return "unknown gemm status";
    }
}

int gemm_last_cuda_error(void) { return t_last_cuda_error; }

int gemm_debug_build(void) { return kDebugBuild ? 1 : 0; }

int gemm_check(void *stream) {
    DeviceState *ds = device_state();
    if (!ds) return fail_cuda(cudaErrorInvalidDevice);
    if (ds->init_error != cudaSuccess) return fail_cuda(ds->init_error);
    return read_status_word(ds, static_cast<cudaStream_t>(stream));
}

int gemm_watchdog_selftest(int wait_ms, void *stream) {
    if (wait_ms < 1 || wait_ms > 2000) return GEMM_ERR_INVALID_ARG;
    DeviceState *ds = device_state();
    if (!ds) return fail_cuda(cudaErrorInvalidDevice);
    if (ds->init_error != cudaSuccess) return fail_cuda(ds->init_error);
    watchdog_probe_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>(
        ds->watchdog, static_cast<unsigned long long>(wait_ms) * 1000000ull);
    const cudaError_t e = cudaPeekAtLastError();
    if (e != cudaSuccess) return fail_cuda(e);
    t_last_plan = "watchdog_probe";
    t_last_launches = 1;
    return GEMM_OK;
}

int gemm_pipeline_stall_selftest(int M, int N, int K, const void *A, const void *B, float *C, int wait_ms,
                                 void *stream) {
    if (wait_ms < 1 || wait_ms > 2000) return GEMM_ERR_INVALID_ARG;
    if (M < 1 || N < 1 || K < 1 || !A || !B || !C) return GEMM_ERR_INVALID_ARG;
    const bool ok = (K % 8 == 0) && (N % 8 == 0) && ((reinterpret_cast<uintptr_t>(A) & 15u) == 0) &&
                    ((reinterpret_cast<uintptr_t>(B) & 15u) == 0) && ((reinterpret_cast<uintptr_t>(C) & 15u) == 0);
    if (!ok) return GEMM_ERR_UNSUPPORTED;
    DeviceState *ds = device_state();
    if (!ds) return fail_cuda(cudaErrorInvalidDevice);
    if (ds->init_error != cudaSuccess) return fail_cuda(ds->init_error);
    const cudaError_t e = run_hgemm_stall_selftest(M, N, K, A, B, C, static_cast<unsigned long long>(wait_ms) * 1000000ull,
                                                   static_cast<cudaStream_t>(stream));
    if (e == cudaErrorNotSupported) return GEMM_ERR_UNSUPPORTED;
    if (e != cudaSuccess) return fail_cuda(e);
    t_last_plan = "tc_128x128_stalled_producer";
    t_last_launches = 1;
    return GEMM_OK;
}

int gemm_fma_rate_probe(int packed, int iters, double *fma_per_clock_per_sm, void *stream) {
    if ((packed != 0 && packed != 1) || iters < 1 || iters > (1 << 20) || !fma_per_clock_per_sm)
        return GEMM_ERR_INVALID_ARG;
    DeviceState *ds = device_state();
    if (!ds) return fail_cuda(cudaErrorInvalidDevice);
    if (ds->init_error != cudaSuccess) return fail_cuda(ds->init_error);
    const cudaError_t e = run_fma_rate_probe(packed != 0, iters, fma_per_clock_per_sm, static_cast<cudaStream_t>(stream));
    t_last_plan = packed ? "fma2_rate_probe" : "fma_rate_probe";
    t_last_launches = 1;
    if (e == cudaErrorLaunchTimeout) return GEMM_ERR_TIMEOUT;
    if (e != cudaSuccess) return fail_cuda(e);
    return GEMM_OK;
}

int gemm_tc_rate_probe(int iters, double *flop_per_clock_per_sm, void *stream) {
    if (iters < 1 || iters > (1 << 20) || !flop_per_clock_per_sm) return GEMM_ERR_INVALID_ARG;
    DeviceState *ds = device_state();
    if (!ds) return fail_cuda(cudaErrorInvalidDevice);
    if (ds->init_error != cudaSuccess) return fail_cuda(ds->init_error);
    const cudaError_t e = run_tc_rate_probe(iters, flop_per_clock_per_sm, static_cast<cudaStream_t>(stream));
    t_last_plan = "tc_rate_probe";
    t_last_launches = 1;
    if (e == cudaErrorLaunchTimeout) return GEMM_ERR_TIMEOUT;
    if (e != cudaSuccess) return fail_cuda(e);
    return GEMM_OK;
}

int gemm_tma_read_probe(int clusters, int multicast, int stages, int kblocks, int region_mb,
                        double *bytes_per_clock_per_sm, double *total_gbs, void *stream) {
    if (clusters < 1 || (multicast != 0 && multicast != 1) || stages < 1 || stages > 6 || kblocks < 1 ||
        kblocks > (1 << 16) || region_mb < 2 || region_mb > 4096 || !bytes_per_clock_per_sm || !total_gbs)
        return GEMM_ERR_INVALID_ARG;
    DeviceState *ds = device_state();
    if (!ds) return fail_cuda(cudaErrorInvalidDevice);
    if (ds->init_error != cudaSuccess) return fail_cuda(ds->init_error);
    if (2 * clusters > device_sm_count()) return GEMM_ERR_INVALID_ARG;
    const cudaError_t e = run_tma_read_probe(clusters, multicast != 0, stages, kblocks, region_mb,
                                             bytes_per_clock_per_sm, total_gbs, static_cast<cudaStream_t>(stream));
    t_last_plan = multicast ? "tma_read_probe_multicast" : "tma_read_probe";
    t_last_launches = 2;
    if (e == cudaErrorLaunchTimeout) return GEMM_ERR_TIMEOUT;
    if (e != cudaSuccess) return fail_cuda(e);
    return GEMM_OK;
}

const char *gemm_last_plan(void) { return t_last_plan; }

int gemm_last_launch_count(void) { return t_last_launches; }

}  // extern "C"

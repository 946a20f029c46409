// api.cu -- the C ABI declared in include/repro.h: argument validation,
// architecture check, workspace sizing and dispatch to the kernels.  No call
// allocates device memory; every call enqueues on the caller's stream.
#include <stdint.h>
#include <string.h>

#include <atomic>
#include <initializer_list>

#include "internal.h"
#include "repro.h"

namespace repro {

namespace {

constexpr int kDefaultBwdKernel = 8;   // operand prep + tensor-copy-fed kernel
LaunchCfg g_cfg = {-1, -1, -1, 0, kDefaultBwdKernel, -1};

constexpr int kMaxDevices = 64;
int g_arch_ok[kMaxDevices];   // 0 unknown, 1 GB300, -1 other
int g_sms[kMaxDevices];

__device__ int g_device_error;   // set by bounded device-side waits

// exactness of the tensor-core forward on each device: 0 not checked yet,
// 1 the self-test passed, -1 it failed (every forward then takes the exact
// CUDA-core path); and a failure that repro_device_check has not reported yet
std::atomic<int> g_tc_state[kMaxDevices];
std::atomic<int> g_tc_notice[kMaxDevices];

unsigned long long g_launches;    // kernels enqueued by this library

std::atomic<int> g_debug{0};      // repro_set_debug flags

int current_device()
{
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return -1;
    return dev;
}

} // namespace

const LaunchCfg& launch_cfg() { return g_cfg; }

int num_sms()
{
    const int dev = current_device();
    if (dev < 0 || dev >= kMaxDevices)
        return 152;
    if (g_sms[dev] == 0) {
        int v = 0;
        if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || v <= 0)
            v = 152;
        g_sms[dev] = v;
    }
    return g_sms[dev];
}

void count_launches(int k) { __atomic_fetch_add(&g_launches, (unsigned long long)k, __ATOMIC_RELAXED); }

int scan_inputs(void* stream, std::initializer_list<FloatSpan> spans)
{
    if ((g_debug.load(std::memory_order_relaxed) & REPRO_DEBUG_CHECK_FINITE) == 0)
        return REPRO_OK;
    int* err = device_error_word();
    if (!err)
        return REPRO_ERR_LAUNCH;
    for (const FloatSpan& f : spans)
        if (f.p && f.n > 0) {
            // the fast scan loads 16 bytes at a time; row statistics and gains may start on 4
            const cudaStream_t st = static_cast<cudaStream_t>(stream);
            const cudaError_t e = ((uintptr_t)f.p & 15u) == 0
                                      ? launch_check_finite(f.p, f.n, err, st)
                                      : launch_check_finite_rows(f.p, REPRO_F32, 1, f.n, f.n, err, st);
            if (e != cudaSuccess)
                return REPRO_ERR_LAUNCH;
        }
    return REPRO_OK;
}

int* device_error_word()
{
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_device_error) != cudaSuccess)
        return nullptr;
    return static_cast<int*>(p);
}

} // namespace repro

using namespace repro;

namespace {

int check_arch()
{
    const int dev = current_device();
    if (dev < 0)
        return REPRO_ERR_LAUNCH;
    if (dev >= kMaxDevices)
        return REPRO_ERR_ARCH;
    if (g_arch_ok[dev] == 0) {
        int major = 0, minor = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
            return REPRO_ERR_LAUNCH;
        g_arch_ok[dev] = (major == 10 && minor == 3) ? 1 : -1;
    }
    return g_arch_ok[dev] == 1 ? REPRO_OK : REPRO_ERR_ARCH;
}

// output rows are tiled 64 per CTA along grid.y (at most 65535 tiles)
constexpr int64_t kMaxRows = 65535LL * 64;

inline bool al16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
inline bool al4(const void* p) { return ((uintptr_t)p & 3u) == 0; }

inline bool overlap(const void* a, size_t na, const void* b, size_t nb)
{
    if (!a || !b || na == 0 || nb == 0)
        return false;
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return x < y + nb && y < x + na;
}

inline cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }

// grid of a streaming kernel: one 256-thread CTA per 256 work items, at most
// ctas_per_sm per SM (the launch-configuration hook overrides it)
int stream_grid(int64_t work_items, int ctas_per_sm = 8)
{
    const int cfg = g_cfg.elementwise_blocks;
    if (cfg > 0)
        return cfg;
    const int64_t cap = (int64_t)num_sms() * ctas_per_sm;
    const int64_t want = (work_items + 255) / 256;
    return (int)(want < 1 ? 1 : (want > cap ? cap : want));
}

// -1: chosen per shape by the backward launcher
int seg_log2() { return g_cfg.bwd_segment_log2; }

// tensor-core forward for every supported shape unless the launch
// configuration asks for the CUDA-core path
bool use_tc(int64_t M, int64_t N, int64_t K)
{
    return g_cfg.fwd_path != 0 && fwd_tc_supported(M, N, K);
}

// 1 when the current device's exactness check has passed (the test hook's
// forced failure aside), else 0; never runs the check
int tc_state_passed()
{
    const int dev = current_device();
    if (dev < 0 || dev >= kMaxDevices || g_cfg.fwd_selftest == 1)
        return 0;
    return g_tc_state[dev].load() > 0 ? 1 : 0;
}

// Whether a default-path forward may use the tensor cores on the current
// device: 1 yes, 0 take the CUDA-core path, negative a CUDA error.  The first
// call on a device runs the exactness self-test in `ws` (at least
// selftest_ws_bytes()) and synchronises `stream`; a call made while `stream`
// is being captured cannot, so before the check has run it takes the exact
// CUDA-core path.
int tc_gate(void* ws, cudaStream_t stream)
{
    const int dev = current_device();
    if (dev < 0 || dev >= kMaxDevices)
        return -1;
    if (g_cfg.fwd_selftest == 1) {   // test hook: act as if the check had failed
        g_tc_notice[dev].store(1);
        return 0;
    }
    const int state = g_tc_state[dev].load();
    if (state != 0)
        return state > 0 ? 1 : 0;
    cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(stream, &cs) != cudaSuccess)
        return -1;
    if (cs != cudaStreamCaptureStatusNone)
        return 0;
    const int r = run_selftest(ws, stream);
    if (r < 0)
        return -1;
    g_tc_state[dev].store(r == 0 ? 1 : -1);
    if (r != 0)
        g_tc_notice[dev].store(1);
    return r == 0 ? 1 : 0;
}

} // namespace

namespace repro {
int arch_status() { return check_arch(); }
} // namespace repro

extern "C" {

const char* repro_status_str(int s)
{
    switch (s) {
    case REPRO_OK: return "ok";
    case REPRO_ERR_ARG: return "invalid argument (null pointer, mode, flag, q_max or R)";
    case REPRO_ERR_SHAPE: return "invalid shape";
    case REPRO_ERR_ALIGN: return "device pointer not aligned (16 bytes for tensors, 4 for scales)";
    case REPRO_ERR_ARCH: return "current device is not a GB300 (compute capability 10.3)";
    case REPRO_ERR_LAUNCH: return "CUDA runtime error while enqueueing";
    case REPRO_ERR_TIMEOUT: return "a bounded device-side wait gave up";
    case REPRO_ERR_WORKSPACE: return "workspace missing or too small";
    case REPRO_ERR_ALIAS: return "buffers that must not overlap do";
    case REPRO_ERR_SELFTEST: return "the tensor-core forward differs from the exact CUDA-core forward";
    case REPRO_ERR_INDEX: return "a token, position, teacher index or label was out of range";
    case REPRO_ERR_NONFINITE: return "debug mode: a float input held a NaN or an infinity";
    default: return "unknown status";
    }
}

int repro_version(void) { return REPRO_VERSION; }

uint64_t repro_launch_count(void) { return (uint64_t)__atomic_load_n(&g_launches, __ATOMIC_RELAXED); }

int repro_set_debug(int flags)
{
    if (flags & ~REPRO_DEBUG_CHECK_FINITE)
        return REPRO_ERR_ARG;
    g_debug.store(flags, std::memory_order_relaxed);
    return REPRO_OK;
}

int repro_set_launch_cfg(const repro_launch_cfg* cfg)
{
    if (!cfg) {
        g_cfg = LaunchCfg{-1, -1, -1, 0, kDefaultBwdKernel, -1};
        return REPRO_OK;
    }
    if (cfg->bwd_segment_log2 < -1 || cfg->bwd_segment_log2 > 8)
        return REPRO_ERR_ARG;
    if (cfg->reduce_block_log2 < -1 || cfg->reduce_block_log2 > 10)
        return REPRO_ERR_ARG;
    if (cfg->fwd_path < -1 || cfg->fwd_path > 2)
        return REPRO_ERR_ARG;
    if (cfg->elementwise_blocks < -1 || cfg->elementwise_blocks > (1 << 20))
        return REPRO_ERR_ARG;
    if (cfg->bwd_kernel != -1 && cfg->bwd_kernel != 1 && cfg->bwd_kernel != 8)
        return REPRO_ERR_ARG;
    if (cfg->fwd_selftest != -1 && cfg->fwd_selftest != 1)
        return REPRO_ERR_ARG;
    g_cfg.bwd_segment_log2 = cfg->bwd_segment_log2;
    g_cfg.reduce_block_log2 = cfg->reduce_block_log2;
    g_cfg.fwd_path = cfg->fwd_path;
    g_cfg.elementwise_blocks = cfg->elementwise_blocks < 0 ? 0 : cfg->elementwise_blocks;
    g_cfg.bwd_kernel = cfg->bwd_kernel < 0 ? kDefaultBwdKernel : cfg->bwd_kernel;
    g_cfg.fwd_selftest = cfg->fwd_selftest;
    return REPRO_OK;
}

size_t repro_selftest_ws_bytes(void)
{
    return selftest_ws_bytes();
}

int repro_selftest(void* ws, size_t ws_bytes, void* stream)
{
    if (!ws || ws_bytes < selftest_ws_bytes())
        return REPRO_ERR_WORKSPACE;
    if (!al16(ws))
        return REPRO_ERR_ALIGN;
    int st = check_arch();
    if (st != REPRO_OK)
        return st;
    const int r = run_selftest(ws, as_stream(stream));
    if (r < 0)
        return REPRO_ERR_LAUNCH;
    const int dev = current_device();
    if (dev >= 0 && dev < kMaxDevices)
        g_tc_state[dev].store(r == 0 ? 1 : -1);   // the forward's gate uses this result
    return r == 0 ? REPRO_OK : REPRO_ERR_SELFTEST;
}

int repro_wait_probe(int arrive, void* stream)
{
    if (arrive != 0 && arrive != 1)
        return REPRO_ERR_ARG;
    int st = check_arch();
    if (st != REPRO_OK)
        return st;
    return launch_wait_probe(arrive, as_stream(stream)) == cudaSuccess ? REPRO_OK
                                                                       : REPRO_ERR_LAUNCH;
}

int repro_device_check(void* stream)
{
    if (cudaStreamSynchronize(as_stream(stream)) != cudaSuccess)
        return REPRO_ERR_LAUNCH;
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_device_error, sizeof(int)) != cudaSuccess)
        return REPRO_ERR_LAUNCH;
    if (v != 0) {
        // an index report leaves what the debug scan found to the next call
        const bool index = !(v & kErrTimeoutBit) && (v & kErrIndexBit);
        const int left = index ? v & ~kErrIndexBit : 0;
        if (cudaMemcpyToSymbol(g_device_error, &left, sizeof(int)) != cudaSuccess)
            return REPRO_ERR_LAUNCH;
        if (index)
            return REPRO_ERR_INDEX;
        return (v & kErrTimeoutBit) || !(v & kErrNonfiniteBit) ? REPRO_ERR_TIMEOUT : REPRO_ERR_NONFINITE;
    }
    const int dev = current_device();
    if (dev >= 0 && dev < kMaxDevices && g_tc_notice[dev].exchange(0) != 0)
        return REPRO_ERR_SELFTEST;
    return REPRO_OK;
}

size_t repro_wscale_ws_bytes(int64_t n)
{
    if (n <= 0)
        return 0;
    return wscale_ws_bytes(n, 0);   // the largest over every launch configuration
}

int repro_wscale(const float* x, int64_t n, int mode, int qmax, float* scale_out, void* ws,
                 size_t ws_bytes, void* stream)
{
    if (!x || !scale_out)
        return REPRO_ERR_ARG;
    if (mode != REPRO_SCALE_WEIGHT_MEANABS && mode != REPRO_SCALE_ACT_AMAX)
        return REPRO_ERR_ARG;
    if (qmax != REPRO_QMAX)
        return REPRO_ERR_ARG;
    if (n <= 0)
        return REPRO_ERR_SHAPE;
    if (!al16(x) || !al4(scale_out))
        return REPRO_ERR_ALIGN;
    if (!ws || ws_bytes < repro_wscale_ws_bytes(n))
        return REPRO_ERR_WORKSPACE;
    if (!al16(ws))
        return REPRO_ERR_ALIGN;
    if (overlap(ws, ws_bytes, x, (size_t)n * 4) || overlap(ws, ws_bytes, scale_out, 4))
        return REPRO_ERR_ALIAS;
    int st = check_arch();
    if (st != REPRO_OK)
        return st;
    if ((st = scan_inputs(stream, {{x, n}})) != REPRO_OK)
        return st;
    if (mode == REPRO_SCALE_WEIGHT_MEANABS)
        return status_of(launch_wscale_meanabs(x, n, qmax, scale_out, ws, g_cfg.reduce_block_log2,
                                               as_stream(stream)));
    // the launch-configuration hook may set the grid; the workspace holds at
    // least ceil(n / 64) + 64 per-CTA partials, so the grid is capped there
    int grid = amax_grid(n);
    if (g_cfg.elementwise_blocks > 0) {
        const int64_t cap = (n + 63) / 64 + 64;
        grid = (int)(g_cfg.elementwise_blocks < cap ? g_cfg.elementwise_blocks : cap);
    }
    return status_of(launch_wscale_amax(x, n, qmax, scale_out, ws, grid, as_stream(stream)));
}

int repro_quant_i8(const float* x, int64_t n, const float* scale, int qmax, int8_t* q_out,
                   void* stream)
{
    if (qmax != REPRO_QMAX)
        return REPRO_ERR_ARG;
    if (n < 0)
        return REPRO_ERR_SHAPE;
    if (n == 0)
        return REPRO_OK;
    if (!x || !scale || !q_out)
        return REPRO_ERR_ARG;
    if (!al16(x) || !al16(q_out) || !al4(scale))
        return REPRO_ERR_ALIGN;
    if (overlap(q_out, (size_t)n, x, (size_t)n * 4) || overlap(q_out, (size_t)n, scale, 4))
        return REPRO_ERR_ALIAS;
    int st = check_arch();
    if (st != REPRO_OK)
        return st;
    if ((st = scan_inputs(stream, {{x, n}, {scale, 1}})) != REPRO_OK)
        return st;
    // up to 32 CTAs per SM: on GB300 the quantiser streams 92M elements in 78.5 us
    // this way against 90.8 us with the grid capped at one resident wave
    return status_of(launch_quant(x, n, scale, qmax, q_out, stream_grid(n / 16, 32),
                                  as_stream(stream)));
}

size_t repro_wscale_multi_ws_bytes(const int64_t* ns, int count)
{
    if (!ns || count < 1 || count > REPRO_MAX_TENSORS)
        return 0;
    for (int t = 0; t < count; ++t)
        if (ns[t] <= 0)
            return 0;
    return wscale_multi_ws_bytes(ns, count);
}

int repro_wscale_multi(const float* const* xs, const int64_t* ns, int count, int mode, int qmax,
                       float* scales_out, void* ws, size_t ws_bytes, void* stream)
{
    if (!xs || !ns || !scales_out || count < 1 || count > REPRO_MAX_TENSORS)
        return REPRO_ERR_ARG;
    if (mode != REPRO_SCALE_WEIGHT_MEANABS && mode != REPRO_SCALE_ACT_AMAX)
        return REPRO_ERR_ARG;
    if (qmax != REPRO_QMAX)
        return REPRO_ERR_ARG;
    for (int t = 0; t < count; ++t) {
        if (!xs[t])
            return REPRO_ERR_ARG;
        if (ns[t] <= 0)
            return REPRO_ERR_SHAPE;
        if (!al16(xs[t]))
            return REPRO_ERR_ALIGN;
    }
    if (!al4(scales_out))
        return REPRO_ERR_ALIGN;
    const size_t need = wscale_multi_ws_bytes(ns, count);
    if (!ws || ws_bytes < need)
        return REPRO_ERR_WORKSPACE;
    if (!al16(ws))
        return REPRO_ERR_ALIGN;
    const size_t sb = (size_t)count * 4;
    if (overlap(ws, ws_bytes, scales_out, sb))
        return REPRO_ERR_ALIAS;
    for (int t = 0; t < count; ++t)
        if (overlap(ws, ws_bytes, xs[t], (size_t)ns[t] * 4) ||
            overlap(scales_out, sb, xs[t], (size_t)ns[t] * 4))
            return REPRO_ERR_ALIAS;
    int st = check_arch();
    if (st != REPRO_OK)
        return st;
    for (int t = 0; t < count; ++t)
        if ((st = scan_inputs(stream, {{xs[t], ns[t]}})) != REPRO_OK)
            return st;
    return status_of(launch_wscale_multi(xs, ns, count, mode, qmax, scales_out, ws,
                                         g_cfg.reduce_block_log2, as_stream(stream)));
}

int repro_quant_i8_multi(const float* const* xs, const int64_t* ns, int count,
                         const float* scales, int qmax, int8_t* const* q_outs, void* stream)
{
    if (!xs || !ns || !q_outs || !scales || count < 1 || count > REPRO_MAX_TENSORS)
        return REPRO_ERR_ARG;
    if (qmax != REPRO_QMAX)
        return REPRO_ERR_ARG;
    int64_t total = 0;
    for (int t = 0; t < count; ++t) {
        if (ns[t] < 0)
            return REPRO_ERR_SHAPE;
        if (ns[t] == 0)
            continue;
        if (!xs[t] || !q_outs[t])
            return REPRO_ERR_ARG;
        if (!al16(xs[t]) || !al16(q_outs[t]))
            return REPRO_ERR_ALIGN;
        total += ns[t];
    }
    if (!al4(scales))
        return REPRO_ERR_ALIGN;
    const size_t sb = (size_t)count * 4;
    for (int t = 0; t < count; ++t) {
        if (ns[t] == 0)
            continue;
        if (overlap(q_outs[t], (size_t)ns[t], scales, sb))
            return REPRO_ERR_ALIAS;
        for (int u = 0; u < count; ++u) {
            if (ns[u] == 0)
                continue;
            if (overlap(q_outs[t], (size_t)ns[t], xs[u], (size_t)ns[u] * 4) ||
                (u != t && overlap(q_outs[t], (size_t)ns[t], q_outs[u], (size_t)ns[u])))
                return REPRO_ERR_ALIAS;
        }
    }
    if (total == 0)
        return REPRO_OK;
    int st = check_arch();
    if (st != REPRO_OK)
        return st;
    for (int t = 0; t < count; ++t)
        if ((st = scan_inputs(stream, {{xs[t], ns[t]}})) != REPRO_OK)
            return st;
    if ((st = scan_inputs(stream, {{scales, count}})) != REPRO_OK)
        return st;
    return status_of(launch_quant_multi(xs, ns, count, scales, qmax, q_outs,
                                        stream_grid(total / 16, 32), as_stream(stream)));
}

// tensor-core shapes: the bf16 copies, and room for the once-per-device
// exactness check that may run first
static size_t fwd_ws_need(int64_t M, int64_t N, int64_t K)
{
    const size_t a = fwd_tc_ws_bytes(M, N, K), b = selftest_ws_bytes();
    return a > b ? a : b;
}

size_t repro_linear_fwd_ws_bytes(int64_t M, int64_t N, int64_t K)
{
    if (!use_tc(M, N, K))
        return 0;
    return fwd_ws_need(M, N, K);
}

int repro_linear_fwd(const int8_t* xq, const int8_t* wq, const float* s_x, const float* s_w,
                     float* y, int64_t M, int64_t N, int64_t K, void* ws, size_t ws_bytes,
                     void* stream)
{
    if (M < 0 || N < 0 || K < 0 || K > 133144 || M > kMaxRows || N > kMaxRows)
        return REPRO_ERR_SHAPE;
    if (M == 0 || N == 0)
        return REPRO_OK;
    if (!y || !s_x || !s_w || (K > 0 && (!xq || !wq)))
        return REPRO_ERR_ARG;
    if (!al16(y) || (xq && !al16(xq)) || (wq && !al16(wq)) || !al4(s_x) || !al4(s_w))
        return REPRO_ERR_ALIGN;
    const size_t ybytes = (size_t)(M * N) * 4;
    if (overlap(y, ybytes, xq, (size_t)(M * K)) || overlap(y, ybytes, wq, (size_t)(N * K)) ||
        overlap(y, ybytes, s_x, 4) || overlap(y, ybytes, s_w, 4))
        return REPRO_ERR_ALIAS;
    bool tc = use_tc(M, N, K);
    if (tc) {
        const size_t need = fwd_ws_need(M, N, K);
        if (!ws || ws_bytes < need)
            return REPRO_ERR_WORKSPACE;
        if (!al16(ws))
            return REPRO_ERR_ALIGN;
        if (overlap(ws, ws_bytes, y, ybytes) || overlap(ws, ws_bytes, xq, (size_t)(M * K)) ||
            overlap(ws, ws_bytes, wq, (size_t)(N * K)) || overlap(ws, ws_bytes, s_x, 4) ||
            overlap(ws, ws_bytes, s_w, 4))
            return REPRO_ERR_ALIAS;
    }
    int st = check_arch();
    if (st != REPRO_OK)
        return st;
    if ((st = scan_inputs(stream, {{s_x, 1}, {s_w, 1}})) != REPRO_OK)
        return st;
    if (tc && g_cfg.fwd_path < 1) {   // the default path is gated; explicit tile paths are not
        const int gate = tc_gate(ws, as_stream(stream));
        if (gate < 0)
            return REPRO_ERR_LAUNCH;
        tc = gate == 1;
    }
    if (tc)
        return status_of(launch_fwd_tc(xq, wq, s_x, s_w, y, M, N, K, ws, g_cfg.fwd_path != 2,
                                       as_stream(stream)));
    return status_of(launch_fwd_cuda_core(xq, wq, s_x, s_w, y, M, N, K, as_stream(stream)));
}

size_t repro_linear_bwd_ws_bytes(int64_t M, int64_t N, int64_t K)
{
    if (M <= 0 || N <= 0 || K <= 0)
        return 0;
    return bwd_ws_bytes(M, N, K, seg_log2());
}

int repro_linear_bwd(const float* dy, const int8_t* xq, const int8_t* wq, const float* s_x,
                     const float* s_w, float* dx, float* dw, int64_t M, int64_t N, int64_t K,
                     int flags, void* ws, size_t ws_bytes, void* stream)
{
    if (flags & ~REPRO_BWD_DW_ACCUMULATE)
        return REPRO_ERR_ARG;
    if (M < 0 || N < 0 || K < 0 || M > kMaxRows || N > kMaxRows || K > kMaxRows * 64)
        return REPRO_ERR_SHAPE;
    if (!dx && !dw)
        return REPRO_ERR_ARG;
    const bool want_dx = dx && M > 0 && K > 0;
    const bool want_dw = dw && N > 0 && K > 0;
    if (!want_dx && !want_dw)
        return REPRO_OK;
    if ((want_dx && N > 0 && (!dy || !wq || !s_w)) || (want_dw && M > 0 && (!dy || !xq || !s_x)))
        return REPRO_ERR_ARG;
    if ((dy && !al16(dy)) || (xq && !al16(xq)) || (wq && !al16(wq)) || (dx && !al16(dx)) ||
        (dw && !al16(dw)) || (s_x && !al4(s_x)) || (s_w && !al4(s_w)))
        return REPRO_ERR_ALIGN;
    const size_t dyb = (size_t)(M * N) * 4, xqb = (size_t)(M * K), wqb = (size_t)(N * K);
    const size_t dxb = want_dx ? (size_t)(M * K) * 4 : 0, dwb = want_dw ? (size_t)(N * K) * 4 : 0;
    if (overlap(dx, dxb, dy, dyb) || overlap(dx, dxb, xq, xqb) || overlap(dx, dxb, wq, wqb) ||
        overlap(dw, dwb, dy, dyb) || overlap(dw, dwb, xq, xqb) || overlap(dw, dwb, wq, wqb) ||
        overlap(dx, dxb, dw, dwb) || overlap(dx, dxb, s_x, 4) || overlap(dx, dxb, s_w, 4) ||
        overlap(dw, dwb, s_x, 4) || overlap(dw, dwb, s_w, 4))
        return REPRO_ERR_ALIAS;
    const int sl = seg_log2();
    const size_t need = bwd_ws_bytes(M, N, K, sl);
    if (need > 0) {
        if (!ws || ws_bytes < need)
            return REPRO_ERR_WORKSPACE;
        if (!al16(ws))
            return REPRO_ERR_ALIGN;
        if (overlap(ws, ws_bytes, dx, dxb) || overlap(ws, ws_bytes, dw, dwb) ||
            overlap(ws, ws_bytes, dy, dyb) || overlap(ws, ws_bytes, xq, xqb) ||
            overlap(ws, ws_bytes, wq, wqb) || overlap(ws, ws_bytes, s_x, 4) ||
            overlap(ws, ws_bytes, s_w, 4))
            return REPRO_ERR_ALIAS;
    }
    int st = check_arch();
    if (st != REPRO_OK)
        return st;
    if ((st = scan_inputs(stream, {{dy, M * N}, {want_dw ? s_x : nullptr, 1}, {want_dx ? s_w : nullptr, 1}})) != REPRO_OK)
        return st;
    cudaStream_t s = as_stream(stream);
    if (want_dx) {
        cudaError_t e = launch_bwd_dx(dy, wq, s_w, dx, M, N, K, sl, static_cast<float*>(ws), s);
        if (e != cudaSuccess)
            return REPRO_ERR_LAUNCH;
    }
    if (want_dw) {
        cudaError_t e = launch_bwd_dw(dy, xq, s_x, dw, M, N, K, sl,
                                      (flags & REPRO_BWD_DW_ACCUMULATE) != 0,
                                      static_cast<float*>(ws), s);
        if (e != cudaSuccess)
            return REPRO_ERR_LAUNCH;
    }
    return REPRO_OK;
}

int repro_grad_accum(float* acc, const float* g, int64_t n, void* stream)
{
    if (n < 0)
        return REPRO_ERR_SHAPE;
    if (n == 0)
        return REPRO_OK;
    if (!acc || !g)
        return REPRO_ERR_ARG;
    if (!al16(acc) || !al16(g))
        return REPRO_ERR_ALIGN;
    if (overlap(acc, (size_t)n * 4, g, (size_t)n * 4))
        return REPRO_ERR_ALIAS;
    int st = check_arch();
    if (st != REPRO_OK)
        return st;
    if ((st = scan_inputs(stream, {{acc, n}, {g, n}})) != REPRO_OK)
        return st;
    return status_of(launch_grad_accum(acc, g, n, stream_grid(n / 4), as_stream(stream)));
}

size_t repro_sumsq_ws_bytes(int64_t n)
{
    if (n <= 0)
        return 0;
    return wscale_ws_bytes(n, 0);
}

int repro_sumsq(const float* g, int64_t n, float* out, void* ws, size_t ws_bytes, void* stream)
{
    if (!g || !out)
        return REPRO_ERR_ARG;
    if (n <= 0)
        return REPRO_ERR_SHAPE;
    if (!al16(g) || !al4(out))
        return REPRO_ERR_ALIGN;
    if (!ws || ws_bytes < repro_sumsq_ws_bytes(n))
        return REPRO_ERR_WORKSPACE;
    if (!al16(ws))
        return REPRO_ERR_ALIGN;
    if (overlap(ws, ws_bytes, g, (size_t)n * 4) || overlap(ws, ws_bytes, out, 4))
        return REPRO_ERR_ALIAS;
    int st = check_arch();
    if (st != REPRO_OK)
        return st;
    if ((st = scan_inputs(stream, {{g, n}})) != REPRO_OK)
        return st;
    return status_of(launch_sumsq(g, n, out, ws, g_cfg.reduce_block_log2, as_stream(stream)));
}

int repro_adamw_step(float* p, float* m, float* v, const float* g, int64_t n, const float* sumsq,
                     const repro_adamw_hparams* hp, int64_t t, void* stream)
{
    if (!hp || t < 1)
        return REPRO_ERR_ARG;
    if (n < 0)
        return REPRO_ERR_SHAPE;
    if (n == 0)
        return REPRO_OK;
    if (!p || !m || !v || !g || !sumsq)
        return REPRO_ERR_ARG;
    if (!al16(p) || !al16(m) || !al16(v) || !al16(g) || !al4(sumsq))
        return REPRO_ERR_ALIGN;
    const size_t nb = (size_t)n * 4;
    if (overlap(p, nb, m, nb) || overlap(p, nb, v, nb) || overlap(m, nb, v, nb) ||
        overlap(g, nb, p, nb) || overlap(g, nb, m, nb) || overlap(g, nb, v, nb) ||
        overlap(sumsq, 4, p, nb) || overlap(sumsq, 4, m, nb) || overlap(sumsq, 4, v, nb))
        return REPRO_ERR_ALIAS;
    int st = check_arch();
    if (st != REPRO_OK)
        return st;
    if ((st = scan_inputs(stream, {{p, n}, {m, n}, {v, n}, {g, n}, {sumsq, 1}})) != REPRO_OK)
        return st;
    AdamWArgs h{hp->lr, hp->beta1, hp->beta2, hp->eps, hp->weight_decay, hp->max_norm};
    return status_of(launch_adamw(p, m, v, g, n, sumsq, h, t, stream_grid(n / 4), as_stream(stream)));
}

// shared checks of the multi-input folds (running sum, TreeFold)
static int check_parts(const float* const* parts, int count, int64_t n, const float* out)
{
    if (!parts || count < 1 || count > REPRO_MAX_REPLICAS)
        return REPRO_ERR_ARG;
    if (n < 0)
        return REPRO_ERR_SHAPE;
    if (!out)
        return REPRO_ERR_ARG;
    for (int r = 0; r < count; ++r) {
        if (!parts[r])
            return REPRO_ERR_ARG;
        if (!al16(parts[r]))
            return REPRO_ERR_ALIGN;
    }
    if (!al16(out))
        return REPRO_ERR_ALIGN;
    const size_t nb = (size_t)n * 4;
    for (int r = 0; r < count; ++r) {
        if (r == 0 && parts[0] == out)
            continue;
        if (overlap(out, nb, parts[r], nb))
            return REPRO_ERR_ALIAS;
    }
    return REPRO_OK;
}

int repro_running_sum(const float* const* parts, int S, int64_t n, float* out, void* stream)
{
    int st = check_parts(parts, S, n, out);
    if (st != REPRO_OK || n == 0)
        return st;
    st = check_arch();
    if (st != REPRO_OK)
        return st;
    for (int r = 0; r < S; ++r)
        if ((st = scan_inputs(stream, {{parts[r], n}})) != REPRO_OK)
            return st;
    return status_of(launch_running_sum(parts, S, n, out, stream_grid(n / 4), as_stream(stream)));
}

int repro_treefold(const float* const* parts, int R, int64_t n, float* out, void* stream)
{
    if (!parts || R < 1 || R > REPRO_MAX_REPLICAS)
        return REPRO_ERR_ARG;
    if (n < 0)
        return REPRO_ERR_SHAPE;
    if (!out)
        return REPRO_ERR_ARG;
    for (int r = 0; r < R; ++r) {
        if (!parts[r])
            return REPRO_ERR_ARG;
        if (!al16(parts[r]))
            return REPRO_ERR_ALIGN;
    }
    if (!al16(out))
        return REPRO_ERR_ALIGN;
    if (n == 0)
        return REPRO_OK;
    const size_t nb = (size_t)n * 4;
    for (int r = 0; r < R; ++r) {
        if (r == 0 && parts[0] == out)
            continue;
        if (overlap(out, nb, parts[r], nb))
            return REPRO_ERR_ALIAS;
    }
    int st = check_arch();
    if (st != REPRO_OK)
        return st;
    for (int r = 0; r < R; ++r)
        if ((st = scan_inputs(stream, {{parts[r], n}})) != REPRO_OK)
            return st;
    return status_of(launch_treefold(parts, R, n, out, stream_grid(n / 4), as_stream(stream)));
}

size_t repro_attn_fwd_ws_bytes(int64_t B, int64_t T, int64_t Hq, int64_t W)
{
    if (B <= 0 || T <= 0 || Hq <= 0 || W < 0 || T > REPRO_ATTN_MAX_T)
        return 0;
    return attn_fwd_ws_bytes(B, T, Hq, W);
}

int repro_attn_fwd(const float* q, const float* k, const int8_t* vq, const float* s_v, float* o,
                   float* m, float* l, int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                   int64_t W, void* ws, size_t ws_bytes, void* stream)
{
    if (B < 0 || T < 0 || Hq < 1 || Hkv < 1 || W < 0)
        return REPRO_ERR_SHAPE;
    if (D != REPRO_ATTN_HEAD_DIM || Hq % Hkv != 0 || T > REPRO_ATTN_MAX_T || Hq > 65535 ||
        B > 65535)
        return REPRO_ERR_SHAPE;
    if (!q || !k || !vq || !s_v || !o || !m || !l)
        return REPRO_ERR_ARG;
    if (!al16(q) || !al16(k) || !al16(vq) || !al16(o) || !al4(s_v) || !al4(m) || !al4(l))
        return REPRO_ERR_ALIGN;
    if (B == 0 || T == 0)
        return REPRO_OK;
    const size_t nq = (size_t)(B * T * Hq * D) * 4, nk = (size_t)(B * T * Hkv * D);
    const size_t nr = (size_t)(B * T * Hq) * 4;
    if (overlap(o, nq, q, nq) || overlap(o, nq, k, nk * 4) || overlap(o, nq, vq, nk) ||
        overlap(m, nr, o, nq) || overlap(l, nr, o, nq) || overlap(m, nr, l, nr) ||
        overlap(m, nr, q, nq) || overlap(l, nr, q, nq) || overlap(m, nr, k, nk * 4) ||
        overlap(l, nr, k, nk * 4) || overlap(m, nr, vq, nk) || overlap(l, nr, vq, nk) ||
        overlap(o, nq, s_v, 4) || overlap(m, nr, s_v, 4) || overlap(l, nr, s_v, 4))
        return REPRO_ERR_ALIAS;
    if (ws) {
        const size_t need = attn_fwd_ws_bytes(B, T, Hq, W);
        if (ws_bytes < need)
            return REPRO_ERR_WORKSPACE;
        if (!al16(ws))
            return REPRO_ERR_ALIGN;
        const void* bufs[7] = {q, k, vq, s_v, o, m, l};
        const size_t sz[7] = {nq, nk * 4, nk, 4, nq, nr, nr};
        for (int x = 0; x < 7; ++x)
            if (overlap(ws, need, bufs[x], sz[x]))
                return REPRO_ERR_ALIAS;
    }
    int st = check_arch();
    if (st != REPRO_OK)
        return st;
    if ((st = scan_inputs(stream, {{q, B * T * Hq * D}, {k, B * T * Hkv * D}, {s_v, 1}})) != REPRO_OK)
        return st;
    // P.V on the tensor cores needs the logit cache and a device whose exactness
    // check has passed (run here, in the cache's space, if it has not run yet)
    bool tc = false;
    if (ws && g_cfg.fwd_path != 0) {
        const int gate = ws_bytes >= selftest_ws_bytes() ? tc_gate(ws, as_stream(stream))
                                                         : tc_state_passed();
        if (gate < 0)
            return REPRO_ERR_LAUNCH;
        tc = gate == 1;
    }
    return status_of(
        launch_attn_fwd(q, k, vq, s_v, o, m, l, B, T, Hq, Hkv, W, ws, tc, as_stream(stream)));
}

size_t repro_attn_bwd_ws_bytes(int64_t B, int64_t T, int64_t Hq, int64_t W)
{
    if (B <= 0 || T <= 0 || Hq <= 0 || W < -1 || T > REPRO_ATTN_MAX_T)
        return 0;
    return attn_bwd_ws_bytes(B, T, Hq, W);
}

int repro_attn_bwd(const float* q, const float* k, const int8_t* vq, const float* s_v,
                   const float* o, const float* dout, const float* m, const float* l, float* dq,
                   float* dk, float* dv, int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                   int64_t W, void* ws, size_t ws_bytes, const void* fwd_ws, size_t fwd_ws_bytes,
                   void* stream)
{
    if (B < 0 || T < 0 || Hq < 1 || Hkv < 1 || W < 0)
        return REPRO_ERR_SHAPE;
    if (D != REPRO_ATTN_HEAD_DIM || Hq % Hkv != 0 || T > REPRO_ATTN_MAX_T || Hkv > 65535 ||
        B > 65535)
        return REPRO_ERR_SHAPE;
    if (!q || !k || !vq || !s_v || !o || !dout || !m || !l || !dq || !dk || !dv)
        return REPRO_ERR_ARG;
    if (!al16(q) || !al16(k) || !al16(vq) || !al16(o) || !al16(dout) || !al16(dq) || !al16(dk) ||
        !al16(dv) || !al4(s_v) || !al4(m) || !al4(l))
        return REPRO_ERR_ALIGN;
    if (B == 0 || T == 0)
        return REPRO_OK;
    const size_t nq = (size_t)(B * T * Hq * D) * 4, nk = (size_t)(B * T * Hkv * D);
    const size_t nr = (size_t)(B * T * Hq) * 4;
    const void* ins[8] = {q, k, vq, s_v, o, dout, m, l};
    const size_t insz[8] = {nq, nk * 4, nk, 4, nq, nq, nr, nr};
    void* outs[3] = {dq, dk, dv};
    const size_t outsz[3] = {nq, nk * 4, nk * 4};
    for (int x = 0; x < 3; ++x) {
        for (int y = 0; y < 8; ++y)
            if (overlap(outs[x], outsz[x], ins[y], insz[y]))
                return REPRO_ERR_ALIAS;
        for (int y = x + 1; y < 3; ++y)
            if (overlap(outs[x], outsz[x], outs[y], outsz[y]))
                return REPRO_ERR_ALIAS;
    }
    // the cached route keeps its tiles and copies in ws too
    const size_t need = attn_bwd_ws_bytes(B, T, Hq, fwd_ws ? W : -1);
    if (!ws || ws_bytes < need)
        return REPRO_ERR_WORKSPACE;
    if (!al16(ws))
        return REPRO_ERR_ALIGN;
    for (int y = 0; y < 8; ++y)
        if (overlap(ws, need, ins[y], insz[y]))
            return REPRO_ERR_ALIAS;
    for (int x = 0; x < 3; ++x)
        if (overlap(ws, need, outs[x], outsz[x]))
            return REPRO_ERR_ALIAS;
    if (fwd_ws) {
        const size_t fneed = attn_fwd_ws_bytes(B, T, Hq, W);
        if (fwd_ws_bytes < fneed)
            return REPRO_ERR_WORKSPACE;
        if (!al16(fwd_ws))
            return REPRO_ERR_ALIGN;
        if (overlap(fwd_ws, fneed, ws, need))
            return REPRO_ERR_ALIAS;
        for (int x = 0; x < 3; ++x)
            if (overlap(fwd_ws, fneed, outs[x], outsz[x]))
                return REPRO_ERR_ALIAS;
    }
    int st = check_arch();
    if (st != REPRO_OK)
        return st;
    if ((st = scan_inputs(stream, {{q, B * T * Hq * D}, {k, B * T * Hkv * D}, {s_v, 1}, {o, B * T * Hq * D},
                                   {dout, B * T * Hq * D}, {m, B * T * Hq}, {l, B * T * Hq}})) != REPRO_OK)
        return st;
    return status_of(launch_attn_bwd(q, k, vq, s_v, o, dout, m, l, dq, dk, dv, B, T, Hq, Hkv, W,
                                     ws, fwd_ws, as_stream(stream)));
}

// ---------------------------------------------------------------- around the blocks

namespace {

// what a call touches, checked together: no output overlaps anything else
struct Span {
    const void* p;
    size_t bytes;
};

size_t type_bytes(int type) { return type == REPRO_F32 ? 4 : type == REPRO_BF16 ? 2 : 1; }
bool float_type(int type) { return type == REPRO_F32 || type == REPRO_BF16; }
bool aligned_to(const void* p, size_t b) { return (uintptr_t)p % b == 0; }
float flushed(float v) { return v != 0.0f && v > -1.17549435e-38f && v < 1.17549435e-38f ? 0.0f : v; }
bool finite_f(float v) { return v - v == 0.0f; }

// elements from the first to one past the last of `rows` rows of D, ld apart
size_t row_span(int64_t rows, int64_t ld, int64_t D) { return (size_t)((rows - 1) * ld + D); }
// whether that count fits comfortably in 63 bits of bytes (one row has no next)
bool rows_fit(int64_t rows, int64_t ld, int64_t D)
{
    return rows <= (int64_t)1 << 31 && (rows <= 1 || ld <= (int64_t)1 << 28) && D <= (int64_t)1 << 28;
}

bool any_overlap(std::initializer_list<Span> outs, std::initializer_list<Span> ins)
{
    for (const Span* o = outs.begin(); o != outs.end(); ++o) {
        for (const Span& i : ins)
            if (overlap(o->p, o->bytes, i.p, i.bytes))
                return true;
        for (const Span* q = o + 1; q != outs.end(); ++q)
            if (overlap(o->p, o->bytes, q->p, q->bytes))
                return true;
    }
    return false;
}

// debug mode: the scan of a strided tensor
int scan_rows(void* stream, const void* p, int type, int64_t rows, int64_t D, int64_t ld)
{
    if ((g_debug.load(std::memory_order_relaxed) & REPRO_DEBUG_CHECK_FINITE) == 0 || !p || rows <= 0)
        return REPRO_OK;
    int* err = device_error_word();
    if (!err)
        return REPRO_ERR_LAUNCH;
    return status_of(launch_check_finite_rows(p, type, rows, D, ld, err, as_stream(stream)));
}

} // namespace

int repro_embed_fwd(const void* table, int table_type, int64_t table_ld, const float* s_w,
                    const void* tokens, int index_bytes, int64_t n, int64_t V, int64_t D, float scale,
                    int64_t pad, void* out, int out_type, int64_t out_ld, void* stream)
{
    if ((!float_type(table_type) && table_type != REPRO_I8) || !float_type(out_type) ||
        (index_bytes != 4 && index_bytes != 8) || !finite_f(scale) ||
        (table_type == REPRO_I8) != (s_w != nullptr))
        return REPRO_ERR_ARG;
    if (n < 0 || V < 1 || D < 1 || table_ld < D || out_ld < D || !rows_fit(V, table_ld, D) ||
        !rows_fit(n, out_ld, D) || n > INT32_MAX || n * ((D + 511) / 512) > 8 * (int64_t)INT32_MAX)
        return REPRO_ERR_SHAPE;
    if (n == 0)
        return REPRO_OK;
    if (!table || !tokens || !out)
        return REPRO_ERR_ARG;
    const size_t tb = type_bytes(table_type), ob = type_bytes(out_type);
    if (!aligned_to(table, tb) || !aligned_to(out, ob) || !aligned_to(tokens, index_bytes) || !al4(s_w))
        return REPRO_ERR_ALIGN;
    if (any_overlap({{out, row_span(n, out_ld, D) * ob}},
                    {{table, row_span(V, table_ld, D) * tb}, {tokens, (size_t)n * index_bytes}, {s_w, 4}}))
        return REPRO_ERR_ALIAS;
    int st = check_arch();
    if (st != REPRO_OK)
        return st;
    if ((table_type != REPRO_I8 && (st = scan_rows(stream, table, table_type, V, D, table_ld)) != REPRO_OK) ||
        (st = scan_inputs(stream, {{s_w, s_w ? 1 : 0}})) != REPRO_OK)
        return st;
    int* err = device_error_word();
    if (!err)
        return REPRO_ERR_LAUNCH;
    return status_of(launch_embed_fwd({table, table_type, table_ld, s_w, tokens, index_bytes, n, V, D, scale,
                                       pad, out, out_type, out_ld, err}, as_stream(stream)));
}

size_t repro_embed_bwd_ws_bytes(int64_t n, int64_t V, int64_t D)
{
    if (n < 0 || n > REPRO_EMBED_MAX_N || V < 1 || V > REPRO_EMBED_MAX_V || D < 1 || D > (int64_t)1 << 28)
        return 0;
    return embed_bwd_ws_bytes(n, V, D);
}

int repro_embed_bwd(const void* dout, int dout_type, int64_t dout_ld, const void* tokens, int index_bytes,
                    int64_t n, int64_t V, int64_t D, float scale, int64_t pad, float* dtable,
                    int64_t dtable_ld, int flags, void* ws, size_t ws_bytes, void* stream)
{
    if (!float_type(dout_type) || (index_bytes != 4 && index_bytes != 8) || !finite_f(scale) ||
        (flags & ~REPRO_BWD_DW_ACCUMULATE) || !dtable)
        return REPRO_ERR_ARG;
    if (n < 0 || n > REPRO_EMBED_MAX_N || V < 1 || V > REPRO_EMBED_MAX_V || D < 1 || dout_ld < D || dtable_ld < D ||
        !rows_fit(n, dout_ld, D) || !rows_fit(V, dtable_ld, D) || n * ((D + 255) / 256) > 256 * (int64_t)INT32_MAX)
        return REPRO_ERR_SHAPE;
    const bool accumulate = (flags & REPRO_BWD_DW_ACCUMULATE) != 0;
    if (n == 0 && accumulate)
        return REPRO_OK;
    if (n > 0 && (!dout || !tokens))
        return REPRO_ERR_ARG;
    const size_t db = type_bytes(dout_type), need = embed_bwd_ws_bytes(n, V, D);
    if (!aligned_to(dout, db) || !al4(dtable) || !aligned_to(tokens, index_bytes))
        return REPRO_ERR_ALIGN;
    if (!ws || ws_bytes < need)
        return REPRO_ERR_WORKSPACE;
    if (!al16(ws))
        return REPRO_ERR_ALIGN;
    if (any_overlap({{dtable, row_span(V, dtable_ld, D) * 4}, {ws, need}},
                    {{dout, n > 0 ? row_span(n, dout_ld, D) * db : 0}, {tokens, (size_t)n * index_bytes}}))
        return REPRO_ERR_ALIAS;
    int st = check_arch();
    if (st != REPRO_OK)
        return st;
    if ((st = scan_rows(stream, dout, dout_type, n, D, dout_ld)) != REPRO_OK ||
        (accumulate && (st = scan_rows(stream, dtable, REPRO_F32, V, D, dtable_ld)) != REPRO_OK))
        return st;
    int* err = device_error_word();
    if (!err)
        return REPRO_ERR_LAUNCH;
    return status_of(launch_embed_bwd({dout, dout_type, dout_ld, tokens, index_bytes, n, V, D, scale, pad,
                                       dtable, dtable_ld, accumulate, err}, ws, as_stream(stream)));
}

// arguments that the norm's forward and backward share; OK, or what is wrong
static int check_qk(const void* q, int64_t q_ld, int64_t q_hs, const void* k, int64_t k_ld, int64_t k_hs,
                    int type, const float* gain_q, const float* gain_k, const float* rope, int64_t P,
                    const int32_t* positions, int64_t T, float eps, int64_t n, int64_t Hq, int64_t Hkv,
                    int64_t D, int64_t R, int flags, int allowed)
{
    if (!float_type(type) || (flags & ~allowed) || !(eps >= 0.0f) || !finite_f(eps))
        return REPRO_ERR_ARG;
    if (n < 0 || Hq < 1 || Hkv < 0 || D < 1 || D > REPRO_QK_MAX_D || R < 0 || R > D || R % 2 != 0)
        return REPRO_ERR_SHAPE;
    if (q_hs < D || q_ld < 1 || !rows_fit(n, q_ld, q_hs) || (Hkv > 0 && (k_hs < D || k_ld < 1 || !rows_fit(n, k_ld, k_hs))))
        return REPRO_ERR_SHAPE;
    if (Hq > 65535 || Hkv > 65535 || n * (Hq + Hkv) > INT32_MAX)
        return REPRO_ERR_SHAPE;
    if (R > 0 && (P < 1 || P > INT32_MAX || (!positions && T < 1) || T > INT32_MAX))
        return REPRO_ERR_SHAPE;
    if (n == 0)
        return REPRO_OK;
    if (!q || (R > 0 && !rope) || (Hkv > 0 && !k) || (Hkv == 0 && gain_k))
        return REPRO_ERR_ARG;
    const size_t b = type_bytes(type);
    if (!aligned_to(q, b) || !aligned_to(k, b) || !al4(gain_q) || !al4(gain_k) || !al16(rope) || !al4(positions))
        return REPRO_ERR_ALIGN;
    return REPRO_OK;
}

// bytes from the first to past the last element of n tokens of H strided heads
static size_t head_span(int64_t n, int64_t ld, int64_t hs, int64_t H, int64_t D, int type)
{
    return n > 0 && H > 0 ? (size_t)((n - 1) * ld + (H - 1) * hs + D) * type_bytes(type) : 0;
}

// whether n tokens of H strided heads lie apart: token after token, or head after head
static bool heads_apart(int64_t n, int64_t ld, int64_t hs, int64_t H, int64_t D)
{
    return n <= 1 || H < 1 || ld >= (H - 1) * hs + D || (ld >= D && hs >= (n - 1) * ld + D);
}

// whether two such tensors, the second's first element `off` past the first's, take different
// parts of slots at one stride: every position of either is that of its first element modulo it
static bool heads_side_by_side(int64_t n, int64_t ld, int64_t ld2, int64_t hs, int64_t hs2, int64_t off, int64_t D)
{
    if (hs != hs2 || (n > 1 && ld != ld2))
        return false;
    const int64_t slot = n > 1 && ld < hs ? ld : hs;
    const int64_t at = ((off % slot) + slot) % slot;
    return hs % slot == 0 && (n <= 1 || ld % slot == 0) && at >= D && at + D <= slot;
}

// debug mode: the scan of n tokens of H strided heads, head by head
static int scan_heads(void* stream, const void* p, int type, int64_t n, int64_t ld, int64_t hs, int64_t H, int64_t D)
{
    for (int64_t h = 0; h < H; ++h) {
        const int st = scan_rows(stream, static_cast<const char*>(p) + (size_t)(h * hs) * type_bytes(type), type, n, D, ld);
        if (st != REPRO_OK)
            return st;
    }
    return REPRO_OK;
}

int repro_qk_norm_rope_fwd(const void* q, int64_t q_ld, int64_t q_hs, const void* k, int64_t k_ld,
                           int64_t k_hs, int type, const float* gain_q, const float* gain_k,
                           const float* rope, int64_t P, const int32_t* positions, int64_t T, float eps,
                           int64_t n, int64_t Hq, int64_t Hkv, int64_t D, int64_t R, int flags,
                           float* q_out, float* k_out, void* stream)
{
    int st = check_qk(q, q_ld, q_hs, k, k_ld, k_hs, type, gain_q, gain_k, rope, P, positions, T, eps, n, Hq,
                      Hkv, D, R, flags, REPRO_QK_INTERLEAVED);
    if (st != REPRO_OK || n == 0)
        return st;
    if (!q_out || (Hkv > 0 && !k_out))
        return REPRO_ERR_ARG;
    if (!al16(q_out) || !al16(k_out))
        return REPRO_ERR_ALIGN;
    const Span ropes = {rope, (size_t)(P * R) * 4}, pos = {positions, (size_t)n * 4};
    if (any_overlap({{q_out, (size_t)(n * Hq * D) * 4}, {k_out, (size_t)(n * Hkv * D) * 4}},
                    {{q, head_span(n, q_ld, q_hs, Hq, D, type)}, {k, head_span(n, k_ld, k_hs, Hkv, D, type)},
                     ropes, pos, {gain_q, (size_t)D * 4}, {gain_k, (size_t)D * 4}}))
        return REPRO_ERR_ALIAS;
    st = check_arch();
    if (st != REPRO_OK)
        return st;
    if ((st = scan_heads(stream, q, type, n, q_ld, q_hs, Hq, D)) != REPRO_OK ||
        (st = scan_heads(stream, k, type, n, k_ld, k_hs, Hkv, D)) != REPRO_OK ||
        (st = scan_inputs(stream, {{rope, P * R}, {gain_q, D}, {gain_k, D}})) != REPRO_OK)
        return st;
    QkArgs a = {};
    a.t[0] = {q, q_ld, q_hs, Hq, gain_q, q_out, nullptr, nullptr, 0, 0, nullptr};
    a.t[1] = {k, k_ld, k_hs, Hkv, gain_k, k_out, nullptr, nullptr, 0, 0, nullptr};
    a.type = type;
    a.rope = rope;
    a.P = P;
    a.positions = positions;
    a.T = T;
    a.eps = eps;
    a.n = n;
    a.D = D;
    a.R = R;
    a.interleaved = (flags & REPRO_QK_INTERLEAVED) != 0;
    a.inv = (D & (D - 1)) == 0 ? 1.0f / (float)D : 0.0f;
    a.err = device_error_word();
    if (!a.err)
        return REPRO_ERR_LAUNCH;
    return status_of(launch_qk_fwd(a, as_stream(stream)));
}

size_t repro_qk_norm_rope_bwd_ws_bytes(int64_t n, int64_t Hq, int64_t Hkv, int64_t D)
{
    if (n < 0 || Hq < 1 || Hkv < 0 || Hq > 65535 || Hkv > 65535 || D < 1 || D > REPRO_QK_MAX_D ||
        n > INT32_MAX || n * (Hq + Hkv) > INT32_MAX)
        return 0;
    return qk_bwd_ws_bytes(n, Hq, Hkv, D);
}

int repro_qk_norm_rope_bwd(const float* dq_out, const float* dk_out, const void* q, int64_t q_ld,
                           int64_t q_hs, const void* k, int64_t k_ld, int64_t k_hs, int type,
                           const float* gain_q, const float* gain_k, const float* rope, int64_t P,
                           const int32_t* positions, int64_t T, float eps, int64_t n, int64_t Hq,
                           int64_t Hkv, int64_t D, int64_t R, int flags, void* dq, int64_t dq_ld,
                           int64_t dq_hs, void* dk, int64_t dk_ld, int64_t dk_hs, float* dgain_q,
                           float* dgain_k, void* ws, size_t ws_bytes, void* stream)
{
    int st = check_qk(q, q_ld, q_hs, k, k_ld, k_hs, type, gain_q, gain_k, rope, P, positions, T, eps, n, Hq,
                      Hkv, D, R, flags, REPRO_QK_INTERLEAVED | REPRO_BWD_DW_ACCUMULATE);
    if (st != REPRO_OK)
        return st;
    if ((gain_q != nullptr) != (dgain_q != nullptr) || (gain_k != nullptr) != (dgain_k != nullptr))
        return REPRO_ERR_ARG;
    if (dq_hs < D || dq_ld < 1 || !rows_fit(n, dq_ld, dq_hs) ||
        (Hkv > 0 && (dk_hs < D || dk_ld < 1 || !rows_fit(n, dk_ld, dk_hs))))
        return REPRO_ERR_SHAPE;
    const bool accumulate = (flags & REPRO_BWD_DW_ACCUMULATE) != 0;
    if (!al4(dgain_q) || !al4(dgain_k))
        return REPRO_ERR_ALIGN;
    if (n == 0) {   // the gains' gradients of no rows are +0
        if (accumulate || (!dgain_q && !dgain_k))
            return REPRO_OK;
        if ((st = check_arch()) != REPRO_OK)
            return st;
        for (float* d : {dgain_q, dgain_k})
            if (d && cudaMemsetAsync(d, 0, (size_t)D * 4, as_stream(stream)) != cudaSuccess)
                return REPRO_ERR_LAUNCH;
        return REPRO_OK;
    }
    if (!dq_out || !dq || (Hkv > 0 && (!dk_out || !dk)))
        return REPRO_ERR_ARG;
    const size_t b = type_bytes(type);
    if (!al16(dq_out) || !al16(dk_out) || !aligned_to(dq, b) || !aligned_to(dk, b))
        return REPRO_ERR_ALIGN;
    const size_t need = gain_q || gain_k ? qk_bwd_ws_bytes(n, Hq, Hkv, D) : 0;
    if (need > 0 && (!ws || ws_bytes < need))
        return REPRO_ERR_WORKSPACE;
    if (need > 0 && !al16(ws))
        return REPRO_ERR_ALIGN;
    if (!heads_apart(n, dq_ld, dq_hs, Hq, D) || !heads_apart(n, dk_ld, dk_hs, Hkv, D))
        return REPRO_ERR_ALIAS;
    // dq and dk may lie between one another, as in the gradient of the fused output; each is
    // checked against everything else, and they must not share a row range head by head
    const Span sq = {dq, head_span(n, dq_ld, dq_hs, Hq, D, type)}, sk = {dk, head_span(n, dk_ld, dk_hs, Hkv, D, type)};
    const Span dg[2] = {{dgain_q, (size_t)D * 4}, {dgain_k, (size_t)D * 4}}, wss = {ws, need};
    const Span in[8] = {{dq_out, (size_t)(n * Hq * D) * 4}, {dk_out, (size_t)(n * Hkv * D) * 4},
                        {q, head_span(n, q_ld, q_hs, Hq, D, type)}, {k, head_span(n, k_ld, k_hs, Hkv, D, type)},
                        {rope, (size_t)(P * R) * 4}, {positions, (size_t)n * 4}, {gain_q, (size_t)D * 4},
                        {gain_k, (size_t)D * 4}};
    for (const Span& o : {sq, sk, dg[0], dg[1], wss})
        for (const Span& i : in)
            if (overlap(o.p, o.bytes, i.p, i.bytes))
                return REPRO_ERR_ALIAS;
    if (any_overlap({dg[0], dg[1], wss}, {sq, sk}))
        return REPRO_ERR_ALIAS;
    if (overlap(sq.p, sq.bytes, sk.p, sk.bytes)) {
        // interleaved in one buffer: allowed when the token strides agree and a token's heads of
        // q and k are disjoint, or q and k of each head lie side by side at equal strides
        const int64_t off = ((const char*)dk - (const char*)dq) / (int64_t)b;
        const int64_t wq = (Hq - 1) * dq_hs + D, wk = (Hkv - 1) * dk_hs + D;
        const bool ok = dq_ld == dk_ld && (off >= 0 ? off >= wq && off + wk <= dq_ld : -off >= wk && -off + wq <= dq_ld);
        if (!ok && !heads_side_by_side(n, dq_ld, dk_ld, dq_hs, dk_hs, off, D))
            return REPRO_ERR_ALIAS;
    }
    st = check_arch();
    if (st != REPRO_OK)
        return st;
    if ((st = scan_heads(stream, q, type, n, q_ld, q_hs, Hq, D)) != REPRO_OK ||
        (st = scan_heads(stream, k, type, n, k_ld, k_hs, Hkv, D)) != REPRO_OK ||
        (st = scan_inputs(stream, {{dq_out, n * Hq * D}, {dk_out, n * Hkv * D}, {rope, P * R}, {gain_q, D},
                                   {gain_k, D}})) != REPRO_OK)
        return st;
    QkArgs a = {};
    a.t[0] = {q, q_ld, q_hs, Hq, gain_q, nullptr, dq_out, dq, dq_ld, dq_hs, dgain_q};
    a.t[1] = {k, k_ld, k_hs, Hkv, gain_k, nullptr, dk_out, dk, dk_ld, dk_hs, dgain_k};
    a.type = type;
    a.rope = rope;
    a.P = P;
    a.positions = positions;
    a.T = T;
    a.eps = eps;
    a.n = n;
    a.D = D;
    a.R = R;
    a.interleaved = (flags & REPRO_QK_INTERLEAVED) != 0;
    a.inv = (D & (D - 1)) == 0 ? 1.0f / (float)D : 0.0f;
    a.accumulate = accumulate;
    a.err = device_error_word();
    if (!a.err)
        return REPRO_ERR_LAUNCH;
    return status_of(launch_qk_bwd(a, ws, as_stream(stream)));
}

size_t repro_distill_ws_bytes(int64_t n, int64_t V)
{
    if (n < 0 || V < 1 || n > INT32_MAX || V > (int64_t)1 << 28)
        return 0;
    return distill_ws_bytes(n, V);
}

// arguments that the loss and its gradient share
static int check_distill(const void* z, int z_type, int64_t z_ld, const void* t_idx, const void* labels,
                         int index_bytes, int64_t n, int64_t V, int64_t K, const repro_distill_hparams* hp)
{
    if (!float_type(z_type) || (index_bytes != 4 && index_bytes != 8) || !hp)
        return REPRO_ERR_ARG;
    if (!(hp->tau >= 1e-4f && hp->tau <= 1e4f) || !finite_f(hp->w_kd) || !finite_f(hp->w_ce) || !finite_f(hp->w_z))
        return REPRO_ERR_ARG;
    if (n < 0 || V < 1 || K < 0 || z_ld < V || !rows_fit(n, z_ld, V) || K > 65536 || n > INT32_MAX ||
        n * ((V + 574) / 512) > (int64_t)1 << 30)   // block numbers, with room past the last one
        return REPRO_ERR_SHAPE;
    if (n == 0)
        return REPRO_OK;
    if (!z || (K > 0 && !t_idx) || (flushed(hp->w_ce) != 0.0f && !labels))
        return REPRO_ERR_ARG;
    if (!aligned_to(z, type_bytes(z_type)) || !aligned_to(t_idx, index_bytes) || !aligned_to(labels, index_bytes))
        return REPRO_ERR_ALIGN;
    return REPRO_OK;
}

int repro_distill_fwd(const void* z, int z_type, int64_t z_ld, const void* t_idx, const void* t_val,
                      int t_type, const void* labels, int index_bytes, int64_t n, int64_t V, int64_t K,
                      const repro_distill_hparams* hp, int flags, float* loss, float* stats, void* ws,
                      size_t ws_bytes, void* stream)
{
    int st = check_distill(z, z_type, z_ld, t_idx, labels, index_bytes, n, V, K, hp);
    if (st != REPRO_OK)
        return st;
    if (!float_type(t_type) || (flags & ~REPRO_DISTILL_LOGPROBS))
        return REPRO_ERR_ARG;
    if (n == 0)
        return REPRO_OK;
    if (!loss || !stats || (K > 0 && !t_val))
        return REPRO_ERR_ARG;
    if (!aligned_to(t_val, type_bytes(t_type)) || !al4(loss) || !al4(stats))
        return REPRO_ERR_ALIGN;
    const size_t need = distill_ws_bytes(n, V);
    if (!ws || ws_bytes < need)
        return REPRO_ERR_WORKSPACE;
    if (!al16(ws))
        return REPRO_ERR_ALIGN;
    if (any_overlap({{loss, (size_t)n * 4}, {stats, (size_t)(n * (REPRO_DISTILL_STATS + K)) * 4}, {ws, need}},
                    {{z, row_span(n, z_ld, V) * type_bytes(z_type)}, {t_idx, (size_t)(n * K) * index_bytes},
                     {t_val, (size_t)(n * K) * type_bytes(t_type)}, {labels, (size_t)n * index_bytes}}))
        return REPRO_ERR_ALIAS;
    st = check_arch();
    if (st != REPRO_OK)
        return st;
    if ((st = scan_rows(stream, z, z_type, n, V, z_ld)) != REPRO_OK)
        return st;
    DistillArgs a = {};
    a.z = z;
    a.z_type = z_type;
    a.z_ld = z_ld;
    a.t_idx = t_idx;
    a.t_val = t_val;
    a.t_type = t_type;
    a.labels = labels;
    a.index_bytes = index_bytes;
    a.n = n;
    a.V = V;
    a.K = K;
    a.tau = hp->tau;
    a.w_kd = flushed(hp->w_kd);
    a.w_ce = flushed(hp->w_ce);
    a.w_z = flushed(hp->w_z);
    a.logprobs = (flags & REPRO_DISTILL_LOGPROBS) != 0;
    a.loss = loss;
    a.stats = stats;
    a.err = device_error_word();
    if (!a.err)
        return REPRO_ERR_LAUNCH;
    return status_of(launch_distill_fwd(a, ws, as_stream(stream)));
}

int repro_distill_bwd(const void* z, int z_type, int64_t z_ld, const void* t_idx, const void* labels,
                      int index_bytes, int64_t n, int64_t V, int64_t K, const repro_distill_hparams* hp,
                      const float* stats, const float* g, int64_t g_n, void* dz, int64_t dz_ld, void* stream)
{
    int st = check_distill(z, z_type, z_ld, t_idx, labels, index_bytes, n, V, K, hp);
    if (st != REPRO_OK)
        return st;
    if (dz_ld < V || !rows_fit(n, dz_ld, V))
        return REPRO_ERR_SHAPE;
    if (n == 0)
        return REPRO_OK;
    if (!stats || !g || !dz || (g_n != 1 && g_n != n))
        return REPRO_ERR_ARG;
    const size_t b = type_bytes(z_type);
    if (!al4(stats) || !al4(g) || !aligned_to(dz, b))
        return REPRO_ERR_ALIGN;
    const Span out = {dz, row_span(n, dz_ld, V) * b};
    if (any_overlap({out}, {{t_idx, (size_t)(n * K) * index_bytes}, {labels, (size_t)n * index_bytes},
                            {stats, (size_t)(n * (REPRO_DISTILL_STATS + K)) * 4}, {g, (size_t)g_n * 4}}))
        return REPRO_ERR_ALIAS;
    if (!(dz == z && dz_ld == z_ld) && overlap(dz, out.bytes, z, row_span(n, z_ld, V) * b))
        return REPRO_ERR_ALIAS;
    st = check_arch();
    if (st != REPRO_OK)
        return st;
    if ((st = scan_rows(stream, z, z_type, n, V, z_ld)) != REPRO_OK ||
        (st = scan_inputs(stream, {{g, g_n}})) != REPRO_OK)
        return st;
    DistillArgs a = {};
    a.z = z;
    a.z_type = z_type;
    a.z_ld = z_ld;
    a.t_idx = t_idx;
    a.labels = labels;
    a.index_bytes = index_bytes;
    a.n = n;
    a.V = V;
    a.K = K;
    a.tau = hp->tau;
    a.w_kd = flushed(hp->w_kd);
    a.w_ce = flushed(hp->w_ce);
    a.w_z = flushed(hp->w_z);
    a.stats = const_cast<float*>(stats);
    a.g = g;
    a.g_stride = g_n == 1 ? 0 : 1;
    a.dz = dz;
    a.dz_ld = dz_ld;
    return status_of(launch_distill_bwd(a, as_stream(stream)));
}

// ---------------------------------------------------------------- the feed-forward half

// arguments that the block norm's forward and backward share
static int check_norm(bool has_y, int type, int u_type, const void* gate, int64_t gate_ld, const float* gain_post,
                      float alpha, float beta, int64_t n, int64_t D, int flags, int allowed)
{
    if (!float_type(type) || !float_type(u_type) || (flags & ~allowed) || (has_y && (!finite_f(alpha) || !finite_f(beta))))
        return REPRO_ERR_ARG;
    if ((!has_y && (gate || gain_post || (flags & (REPRO_NORM_POST | REPRO_NORM_GATE_ROWS)))) ||
        (gain_post && !(flags & REPRO_NORM_POST)) || (!gate && (flags & REPRO_NORM_GATE_ROWS)))
        return REPRO_ERR_ARG;
    if (n < 0 || D < 1 || D > REPRO_NORM_MAX_D || ((flags & REPRO_NORM_GATE_ROWS) && (gate_ld < D || !rows_fit(n, gate_ld, D))))
        return REPRO_ERR_SHAPE;
    return REPRO_OK;
}

// bytes of n strided rows, 0 for a missing tensor
static size_t rows_bytes(const void* p, int64_t n, int64_t ld, int64_t D, int type)
{
    return p && n > 0 ? row_span(n, ld, D) * type_bytes(type) : 0;
}

static bool bad_rows(const void* p, int64_t n, int64_t ld, int64_t D) { return p && (ld < D || !rows_fit(n, ld, D)); }

int repro_block_norm_fwd(const void* x, int64_t x_ld, const void* y, int64_t y_ld, int type, const void* gate,
                         int64_t gate_ld, const float* gain_post, const float* gain_pre, float alpha, float beta,
                         float eps, int64_t n, int64_t D, int flags, void* h, int64_t h_ld, void* u, int u_type,
                         int64_t u_ld, float* stats, void* stream)
{
    int st = check_norm(y, type, u_type, gate, gate_ld, gain_post, alpha, beta, n, D, flags,
                        REPRO_NORM_POST | REPRO_NORM_GATE_ROWS);
    if (st != REPRO_OK)
        return st;
    if (!(eps >= 0.0f) || !finite_f(eps) || (y != nullptr) != (h != nullptr) || (!y && !u && n > 0) || (!u && gain_pre))
        return REPRO_ERR_ARG;
    if (x_ld < D || !rows_fit(n, x_ld, D) || bad_rows(y, n, y_ld, D) || bad_rows(h, n, h_ld, D) || bad_rows(u, n, u_ld, D))
        return REPRO_ERR_SHAPE;
    if (n == 0)
        return REPRO_OK;
    if (!x)
        return REPRO_ERR_ARG;
    const bool rows = (flags & REPRO_NORM_GATE_ROWS) != 0;
    const size_t b = type_bytes(type);
    if (!aligned_to(x, b) || !aligned_to(y, b) || !aligned_to(h, b) || !aligned_to(gate, rows ? b : 4) ||
        !aligned_to(u, type_bytes(u_type)) || !al4(gain_post) || !al4(gain_pre) || !al4(stats))
        return REPRO_ERR_ALIGN;
    const bool in_place = h == x && (n == 1 || h_ld == x_ld);
    const Span sx = {x, in_place ? 0 : rows_bytes(x, n, x_ld, D, type)};
    if (any_overlap({{h, rows_bytes(h, n, h_ld, D, type)}, {u, rows_bytes(u, n, u_ld, D, u_type)}, {stats, (size_t)n * 8}},
                    {sx, {y, rows_bytes(y, n, y_ld, D, type)},
                     {gate, rows ? rows_bytes(gate, n, gate_ld, D, type) : (size_t)D * 4}, {gain_post, (size_t)D * 4},
                     {gain_pre, (size_t)D * 4}}))
        return REPRO_ERR_ALIAS;
    if ((st = check_arch()) != REPRO_OK)
        return st;
    if ((st = scan_rows(stream, x, type, n, D, x_ld)) != REPRO_OK || (st = scan_rows(stream, y, type, n, D, y_ld)) != REPRO_OK ||
        (rows && (st = scan_rows(stream, gate, type, n, D, gate_ld)) != REPRO_OK) ||
        (st = scan_inputs(stream, {{rows ? nullptr : static_cast<const float*>(gate), D}, {gain_post, D}, {gain_pre, D}})) != REPRO_OK)
        return st;
    NormArgs a = {};
    a.x = x, a.x_ld = x_ld, a.y = y, a.y_ld = y_ld, a.type = type, a.u_type = u_type;
    a.gate = gate, a.gate_ld = gate_ld, a.gate_rows = rows, a.post = (flags & REPRO_NORM_POST) != 0;
    a.gain_post = gain_post, a.gain_pre = gain_pre;
    a.alpha = alpha, a.beta = beta, a.eps = eps, a.n = n, a.D = D;
    a.h = h, a.h_ld = h_ld, a.u = u, a.u_ld = u_ld, a.stats = stats;
    return status_of(launch_norm_fwd(a, as_stream(stream)));
}

size_t repro_block_norm_bwd_ws_bytes(int64_t n, int64_t D)
{
    if (n <= 0 || n > (int64_t)1 << 31 || D < 1 || D > REPRO_NORM_MAX_D)
        return 0;
    return norm_bwd_ws_bytes(n, D);
}

int repro_block_norm_bwd(const void* dh, int64_t dh_ld, const void* du, int u_type, int64_t du_ld, const void* h,
                         int64_t h_ld, const void* y, int64_t y_ld, int type, const void* gate, int64_t gate_ld,
                         const float* gain_post, const float* gain_pre, const float* stats, float alpha, float beta,
                         int64_t n, int64_t D, int flags, void* dx, int64_t dx_ld, void* dy, int64_t dy_ld, void* dgate,
                         int64_t dgate_ld, float* dgain_post, float* dgain_pre, void* ws, size_t ws_bytes, void* stream)
{
    int st = check_norm(y, type, u_type, gate, gate_ld, gain_post, alpha, beta, n, D, flags,
                        REPRO_NORM_POST | REPRO_NORM_GATE_ROWS | REPRO_BWD_DW_ACCUMULATE);
    if (st != REPRO_OK)
        return st;
    const bool rows = (flags & REPRO_NORM_GATE_ROWS) != 0, accumulate = (flags & REPRO_BWD_DW_ACCUMULATE) != 0;
    if ((gate != nullptr) != (dgate != nullptr) || (gain_post != nullptr) != (dgain_post != nullptr) ||
        (gain_pre != nullptr) != (dgain_pre != nullptr) || (y != nullptr) != (dy != nullptr) ||
        (n > 0 && ((!dh && !du) || !dx || !stats)) || (n > 0 && (du != nullptr) != (h != nullptr)) ||
        (n > 0 && !du && gain_pre))
        return REPRO_ERR_ARG;
    if (bad_rows(dh, n, dh_ld, D) || bad_rows(du, n, du_ld, D) || bad_rows(h, n, h_ld, D) || bad_rows(y, n, y_ld, D) ||
        bad_rows(dx, n, dx_ld, D) || bad_rows(dy, n, dy_ld, D) || (rows && bad_rows(dgate, n, dgate_ld, D)))
        return REPRO_ERR_SHAPE;
    const size_t b = type_bytes(type);
    if (!aligned_to(dh, b) || !aligned_to(h, b) || !aligned_to(y, b) || !aligned_to(dx, b) || !aligned_to(dy, b) ||
        !aligned_to(gate, rows ? b : 4) || !aligned_to(dgate, rows ? b : 4) || !aligned_to(du, type_bytes(u_type)) ||
        !al4(gain_post) || !al4(gain_pre) || !al4(stats) || !al4(dgain_post) || !al4(dgain_pre))
        return REPRO_ERR_ALIGN;
    float* sums[3] = {rows ? nullptr : static_cast<float*>(dgate), dgain_post, dgain_pre};
    if (n == 0) {   // sums over no tokens are +0
        if (accumulate || (!sums[0] && !sums[1] && !sums[2]))
            return REPRO_OK;
        if ((st = check_arch()) != REPRO_OK)
            return st;
        for (float* s : sums)
            if (s && cudaMemsetAsync(s, 0, (size_t)D * 4, as_stream(stream)) != cudaSuccess)
                return REPRO_ERR_LAUNCH;
        return REPRO_OK;
    }
    const size_t need = sums[0] || sums[1] || sums[2] ? norm_bwd_ws_bytes(n, D) : 0, col = (size_t)D * 4;
    if (need > 0 && (!ws || ws_bytes < need))
        return REPRO_ERR_WORKSPACE;
    if (need > 0 && !al16(ws))
        return REPRO_ERR_ALIGN;
    const bool in_place = dx == dh && (n == 1 || dx_ld == dh_ld);
    if (any_overlap({{dx, rows_bytes(dx, n, dx_ld, D, type)}, {dy, rows_bytes(dy, n, dy_ld, D, type)},
                     {dgate, rows ? rows_bytes(dgate, n, dgate_ld, D, type) : col}, {dgain_post, col}, {dgain_pre, col},
                     {ws, need}},
                    {{dh, in_place ? 0 : rows_bytes(dh, n, dh_ld, D, type)}, {du, rows_bytes(du, n, du_ld, D, u_type)},
                     {h, rows_bytes(h, n, h_ld, D, type)}, {y, rows_bytes(y, n, y_ld, D, type)},
                     {gate, rows ? rows_bytes(gate, n, gate_ld, D, type) : col}, {gain_post, col}, {gain_pre, col},
                     {stats, (size_t)n * 8}}))
        return REPRO_ERR_ALIAS;
    if ((st = check_arch()) != REPRO_OK)
        return st;
    if ((st = scan_rows(stream, dh, type, n, D, dh_ld)) != REPRO_OK || (st = scan_rows(stream, du, u_type, n, D, du_ld)) != REPRO_OK ||
        (st = scan_rows(stream, h, type, n, D, h_ld)) != REPRO_OK || (st = scan_rows(stream, y, type, n, D, y_ld)) != REPRO_OK ||
        (rows && (st = scan_rows(stream, gate, type, n, D, gate_ld)) != REPRO_OK) ||
        (st = scan_inputs(stream, {{rows ? nullptr : static_cast<const float*>(gate), D}, {gain_post, D}, {gain_pre, D}, {stats, 2 * n}})) !=
            REPRO_OK)
        return st;
    NormArgs a = {};
    a.y = y, a.y_ld = y_ld, a.type = type, a.u_type = u_type;
    a.gate = gate, a.gate_ld = gate_ld, a.gate_rows = rows, a.post = (flags & REPRO_NORM_POST) != 0;
    a.accumulate = accumulate, a.gain_post = gain_post, a.gain_pre = gain_pre;
    a.alpha = alpha, a.beta = beta, a.n = n, a.D = D, a.stats = const_cast<float*>(stats);
    a.dh = dh, a.dh_ld = dh_ld, a.du = du, a.du_ld = du_ld, a.hs = h, a.hs_ld = h_ld;
    a.dx = dx, a.dx_ld = dx_ld, a.dy = dy, a.dy_ld = dy_ld, a.dgate = dgate, a.dgate_ld = dgate_ld;
    a.dgain_post = dgain_post, a.dgain_pre = dgain_pre;
    return status_of(launch_norm_bwd(a, ws, as_stream(stream)));
}

size_t repro_quant_rows_i8_ws_bytes(int64_t n, int64_t D, int flags)
{
    if (n < 0 || D < 1 || D > (int64_t)1 << 28)
        return 0;
    return quant_rows_ws_bytes(n, D, (flags & REPRO_QUANT_COLUMNS) != 0);
}

int repro_quant_rows_i8(const void* x, int type, int64_t x_ld, const float* mul, int64_t n, int64_t D, int flags,
                        int8_t* q, int64_t q_ld, float* scales, void* ws, size_t ws_bytes, void* stream)
{
    if (!float_type(type) || (flags & ~REPRO_QUANT_COLUMNS))
        return REPRO_ERR_ARG;
    if (n < 0 || D < 1 || x_ld < D || q_ld < D || !rows_fit(n, x_ld, D) || !rows_fit(n, q_ld, D))
        return REPRO_ERR_SHAPE;
    const bool columns = (flags & REPRO_QUANT_COLUMNS) != 0;
    if (n == 0 && !columns)
        return REPRO_OK;
    if (!scales || (n > 0 && (!x || !q)))
        return REPRO_ERR_ARG;
    const size_t need = n > 0 ? quant_rows_ws_bytes(n, D, columns) : 0;
    if (!aligned_to(x, type_bytes(type)) || !al4(mul) || !al4(scales))
        return REPRO_ERR_ALIGN;
    if (need > 0 && (!ws || ws_bytes < need))
        return REPRO_ERR_WORKSPACE;
    if (need > 0 && !al16(ws))
        return REPRO_ERR_ALIGN;
    const size_t sbytes = (size_t)(columns ? D : n) * 4, mbytes = (size_t)(columns ? n : D) * 4;
    if (any_overlap({{q, n > 0 ? row_span(n, q_ld, D) : 0}, {scales, sbytes}, {ws, need}},
                    {{x, rows_bytes(x, n, x_ld, D, type)}, {mul, mbytes}}))
        return REPRO_ERR_ALIAS;
    int st = check_arch();
    if (st != REPRO_OK)
        return st;
    if (n == 0)   // columns of no rows
        return cudaMemsetAsync(scales, 0, sbytes, as_stream(stream)) == cudaSuccess ? REPRO_OK : REPRO_ERR_LAUNCH;
    if ((st = scan_rows(stream, x, type, n, D, x_ld)) != REPRO_OK ||
        (st = scan_inputs(stream, {{mul, columns ? n : D}})) != REPRO_OK)
        return st;
    return status_of(launch_quant_rows({x, type, x_ld, mul, n, D, columns, q, q_ld, scales}, ws, as_stream(stream)));
}

static size_t matmul_ws_need(int64_t M, int64_t N, int64_t K, int flags)
{
    const size_t need = matmul_i8_ws_bytes(M, N, K, flags & REPRO_MM_A_T, flags & REPRO_MM_B_T);
    return need == 0 || need > selftest_ws_bytes() ? need : selftest_ws_bytes();   // the first call's check runs there
}

size_t repro_matmul_i8_ws_bytes(int64_t M, int64_t N, int64_t K, int flags)
{
    if (M <= 0 || N <= 0 || K <= 0 || M > REPRO_MM_MAX_ROWS || N > REPRO_MM_MAX_ROWS || K > 133144)
        return 0;
    return matmul_ws_need(M, N, K, flags);
}

int repro_matmul_i8(const int8_t* a, int64_t a_ld, const int8_t* b, int64_t b_ld, const float* s_a, const float* s_b,
                    int64_t M, int64_t N, int64_t K, int flags, void* y, int y_type, int64_t y_ld, void* ws,
                    size_t ws_bytes, void* stream)
{
    const bool accumulate = (flags & REPRO_BWD_DW_ACCUMULATE) != 0, a_t = (flags & REPRO_MM_A_T) != 0, b_t = (flags & REPRO_MM_B_T) != 0;
    if (!float_type(y_type) || (flags & ~(REPRO_BWD_DW_ACCUMULATE | REPRO_MM_A_T | REPRO_MM_B_T)) || (accumulate && y_type != REPRO_F32))
        return REPRO_ERR_ARG;
    if (M < 0 || N < 0 || K < 0 || M > REPRO_MM_MAX_ROWS || N > REPRO_MM_MAX_ROWS || K > 133144)
        return REPRO_ERR_SHAPE;
    const int64_t ar = a_t ? K : M, ac = a_t ? M : K, br = b_t ? K : N, bc = b_t ? N : K;
    if (a_ld < ac || b_ld < bc || y_ld < N || !rows_fit(ar, a_ld, ac) || !rows_fit(br, b_ld, bc) || !rows_fit(M, y_ld, N))
        return REPRO_ERR_SHAPE;
    if (M == 0 || N == 0 || (K == 0 && accumulate))
        return REPRO_OK;
    if (!y || (K > 0 && (!a || !b)))
        return REPRO_ERR_ARG;
    if (!aligned_to(y, type_bytes(y_type)) || !al4(s_a) || !al4(s_b))
        return REPRO_ERR_ALIGN;
    const size_t need = K > 0 ? matmul_ws_need(M, N, K, flags) : 0;
    if (need > 0 && (!ws || ws_bytes < need))
        return REPRO_ERR_WORKSPACE;
    if (need > 0 && !al16(ws))
        return REPRO_ERR_ALIGN;
    if (any_overlap({{y, row_span(M, y_ld, N) * type_bytes(y_type)}, {ws, need}},
                    {{a, K > 0 ? row_span(ar, a_ld, ac) : 0}, {b, K > 0 ? row_span(br, b_ld, bc) : 0},
                     {s_a, (size_t)M * 4}, {s_b, (size_t)N * 4}}))
        return REPRO_ERR_ALIAS;
    int st = check_arch();
    if (st != REPRO_OK)
        return st;
    if ((st = scan_inputs(stream, {{s_a, M}, {s_b, N}})) != REPRO_OK ||
        (accumulate && (st = scan_rows(stream, y, y_type, M, N, y_ld)) != REPRO_OK))
        return st;
    bool tc = need > 0 && g_cfg.fwd_path != 0;
    if (tc && g_cfg.fwd_path < 1) {
        const int gate = tc_gate(ws, as_stream(stream));
        if (gate < 0)
            return REPRO_ERR_LAUNCH;
        tc = gate == 1;
    }
    return status_of(launch_matmul_i8({a, b, a_ld, b_ld, a_t, b_t, s_a, s_b, M, N, K, y, y_type, y_ld, accumulate}, ws, tc,
                                      as_stream(stream)));
}

// what the activation's forward and backward share
static int check_swiglu(int type, int a_type, int64_t n, int64_t F, const void* gu, int64_t gu_ld, const void* a, int64_t a_ld,
                        const int8_t* codes, const float* scales)
{
    if (!float_type(type) || !float_type(a_type) || (codes != nullptr) != (scales != nullptr))
        return REPRO_ERR_ARG;
    if (n < 0 || F < 1 || F > (int64_t)1 << 27 || bad_rows(gu, n, gu_ld, 2 * F) || bad_rows(a, n, a_ld, F) ||
        n > (int64_t)1 << 31)
        return REPRO_ERR_SHAPE;
    if (!aligned_to(gu, type_bytes(type)) || !aligned_to(a, type_bytes(a_type)) || !al16(codes) || !al4(scales))
        return REPRO_ERR_ALIGN;
    return REPRO_OK;
}

static int64_t swiglu_groups(int64_t F) { return (F + REPRO_SWIGLU_GROUP - 1) / REPRO_SWIGLU_GROUP; }

int repro_swiglu_fwd(const void* gu, int type, int64_t gu_ld, int64_t n, int64_t F, void* a, int a_type, int64_t a_ld,
                     int8_t* codes, float* scales, void* stream)
{
    int st = check_swiglu(type, a_type, n, F, gu, gu_ld, a, a_ld, codes, scales);
    if (st != REPRO_OK || n == 0)
        return st;
    if (!gu || !a)
        return REPRO_ERR_ARG;
    const size_t groups = (size_t)(2 * n * swiglu_groups(F));
    if (any_overlap({{a, rows_bytes(a, n, a_ld, F, a_type)}, {codes, groups * REPRO_SWIGLU_GROUP}, {scales, groups * 4}},
                    {{gu, rows_bytes(gu, n, gu_ld, 2 * F, type)}}))
        return REPRO_ERR_ALIAS;
    if ((st = check_arch()) != REPRO_OK || (st = scan_rows(stream, gu, type, n, 2 * F, gu_ld)) != REPRO_OK)
        return st;
    SwigluArgs s = {};
    s.gu = gu, s.type = type, s.gu_ld = gu_ld, s.a_type = a_type, s.a_ld = a_ld, s.codes = codes, s.scales = scales;
    s.n = n, s.F = F, s.a = a;
    return status_of(launch_swiglu_fwd(s, as_stream(stream)));
}

int repro_swiglu_bwd(const void* da, int a_type, int64_t da_ld, const void* gu, int64_t gu_ld, const int8_t* codes,
                     const float* scales, int64_t n, int64_t F, void* dgu, int type, int64_t dgu_ld, void* stream)
{
    int st = check_swiglu(type, a_type, n, F, gu, gu_ld, da, da_ld, codes, scales);
    if (st != REPRO_OK)
        return st;
    if (bad_rows(dgu, n, dgu_ld, 2 * F))
        return REPRO_ERR_SHAPE;
    if (n == 0)
        return REPRO_OK;
    if (!da || !dgu || (gu != nullptr) == (codes != nullptr))
        return REPRO_ERR_ARG;
    if (!aligned_to(dgu, type_bytes(type)))
        return REPRO_ERR_ALIGN;
    const size_t groups = (size_t)(2 * n * swiglu_groups(F));
    if (any_overlap({{dgu, rows_bytes(dgu, n, dgu_ld, 2 * F, type)}},
                    {{gu, rows_bytes(gu, n, gu_ld, 2 * F, type)}, {da, rows_bytes(da, n, da_ld, F, a_type)},
                     {codes, groups * REPRO_SWIGLU_GROUP}, {scales, groups * 4}}))
        return REPRO_ERR_ALIAS;
    if ((st = check_arch()) != REPRO_OK || (st = scan_rows(stream, da, a_type, n, F, da_ld)) != REPRO_OK ||
        (st = scan_rows(stream, gu, type, n, 2 * F, gu_ld)) != REPRO_OK ||
        (st = scan_inputs(stream, {{scales, (int64_t)groups}})) != REPRO_OK)
        return st;
    SwigluArgs s = {};
    s.gu = gu, s.type = type, s.gu_ld = gu_ld, s.da = da, s.a_type = a_type, s.a_ld = da_ld;
    s.codes = const_cast<int8_t*>(codes), s.scales = const_cast<float*>(scales);
    s.n = n, s.F = F, s.dgu = dgu, s.dgu_ld = dgu_ld;
    return status_of(launch_swiglu_bwd(s, as_stream(stream)));
}

size_t repro_state_hash_ws_bytes(const int64_t* nbytes, int nbuf)
{
    if (nbuf < 0 || nbuf > REPRO_HASH_MAX_BUFFERS || (nbuf > 0 && !nbytes))
        return 0;
    for (int b = 0; b < nbuf; ++b)
        if (nbytes[b] < 0)
            return 0;
    return hash_ws_bytes(hash_leaf_count(nbytes, nbuf, REPRO_HASH_LEAF_BYTES));
}

int repro_state_hash(const void* const* bufs, const int64_t* nbytes, int nbuf, uint8_t* digest,
                     void* ws, size_t ws_bytes, void* stream)
{
    if (nbuf < 0 || nbuf > REPRO_HASH_MAX_BUFFERS || !digest)
        return REPRO_ERR_ARG;
    if (nbuf > 0 && (!bufs || !nbytes))
        return REPRO_ERR_ARG;
    for (int b = 0; b < nbuf; ++b) {
        if (nbytes[b] < 0)
            return REPRO_ERR_SHAPE;
        if (nbytes[b] > 0 && !bufs[b])
            return REPRO_ERR_ARG;
        if (nbytes[b] > 0 && !al16(bufs[b]))
            return REPRO_ERR_ALIGN;
    }
    if (!al16(digest))
        return REPRO_ERR_ALIGN;
    const size_t need = hash_ws_bytes(hash_leaf_count(nbytes, nbuf, REPRO_HASH_LEAF_BYTES));
    if (need > 0) {
        if (!ws || ws_bytes < need)
            return REPRO_ERR_WORKSPACE;
        if (!al16(ws))
            return REPRO_ERR_ALIGN;
        if (overlap(ws, need, digest, 32))
            return REPRO_ERR_ALIAS;
        for (int b = 0; b < nbuf; ++b)
            if (overlap(ws, need, bufs[b], (size_t)nbytes[b]))
                return REPRO_ERR_ALIAS;
    }
    int st = check_arch();
    if (st != REPRO_OK)
        return st;
    return status_of(launch_state_hash(bufs, nbytes, nbuf, REPRO_HASH_LEAF_BYTES, digest, ws,
                                       as_stream(stream)));
}

} // extern "C"

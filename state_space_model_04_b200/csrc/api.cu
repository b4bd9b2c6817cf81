// api.cu -- the extern "C" boundary of libssd_b200.so (declared in include/ssd.h).
//
// Host-side only: argument validation (before anything is enqueued), workspace carving
// and dispatch to the sm_100a kernels.  No device memory is allocated here.
#include "backward.cuh"
#include "common.cuh"

#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <atomic>
#include <cmath>
#include <mutex>
#include <string>
#include <tuple>
#include <vector>

namespace ssd {

// kernels (defined in the other translation units)
size_t prefill_simt_workspace_bytes(int b, int T, int H, int N, int L, int io);
int launch_prefill_simt(int b, int T, int H, int N, int G, int L, int io, const void* x,
                        const float* dt, const DtMap& dtm, const float* A, const void* Bm, const void* Cm,
                        const float* D, const float* h0, void* y, float* hf, void* ws,
                        cudaStream_t s);
bool prefill_tc_supported(int P, int N, int io);
size_t prefill_tc_workspace_bytes(int b, int T, int H);
int launch_prefill_tc(int b, int T, int H, int G, const void* x, const float* dt, const DtMap& dtm, const float* A,
                      const void* Bm,
                      const void* Cm, const float* D, const float* h0, void* y, float* hf, void* ws,
                      cudaStream_t s);
int prefill_tc_status(void* ws, cudaStream_t s);
void prefill_tc_starve_next(unsigned long long wait_ns);
void prefill_tc_force_segments(int nseg);
void prefill_tc_force_split(int n_full, int nseg);
void prefill_tc_decay_mode(int mode);
int prefill_tc_segments(int b, int T, int H);
int prefill_tc_whole_units(int b, int T, int H);
size_t prefill_tc_local_state_workspace_bytes(int b, int T, int H);
int launch_prefill_tc_local_state(int b, int T, int H, int G, const void* x, const float* dt, const float* A,
                                  const void* Bm, float* h_local, float* log_decay, void* ws, cudaStream_t s);
int launch_context_scan(int rank, int b, int H, const float* h0, const float* h_all, const float* ld_all,
                        float* h_in, cudaStream_t s);
size_t decode_workspace_bytes(int layers, int b, int G);
int launch_decode_step(int layers, int b, int H, int N, int G, int act, int io, float* h,
                       float* conv_state, const void* xbc, const float* dt, const float* A,
                       const float* D, const float* conv_w, const float* conv_b, void* y,
                       void* ws, cudaStream_t s);
int create_decode_plan(ssd_decode_plan** out, int layers, int b, int H, int N, int G, int act,
                       int io, float* h, float* conv_state, const void* xbc_ring,
                       const float* dt_ring, int ring, const float* A, const float* D,
                       const float* conv_w, const float* conv_b, void* y_ring, int n_steps,
                       void* ws);
int launch_decode_plan(ssd_decode_plan* plan, cudaStream_t s);
int destroy_decode_plan(ssd_decode_plan* plan);
int decode_noalloc_scratch(void** ptr, size_t* bytes);
size_t backward_simt_workspace_bytes(const BwdArgs& a);
bool backward_simt_fits(const BwdArgs& a);
int launch_backward_simt(const BwdArgs& a, void* ws, cudaStream_t s);
bool backward_tc_supported(int P, int N, int io);
size_t backward_tc_workspace_bytes(const BwdArgs& a);
int launch_backward_tc(const BwdArgs& a, void* ws, size_t offset, cudaStream_t s);
void backward_tc_starve_next(unsigned long long wait_ns);
int backward_tc_lag_next(int role);
size_t norm_workspace_bytes(long long rows, int D, int groups);
int launch_residual_norm(long long rows, int D, int io, int res_dtype, const void* x, long long ld_x,
                         const void* res, long long ld_res, float scale, const float* w, float eps, void* out,
                         long long ld_out, void* r, long long ld_r, cudaStream_t s);
int launch_residual_norm_backward(long long rows, int D, int io, int res_dtype, const void* dout, long long ld_dout,
                                  const void* r, long long ld_r, const float* w, const void* dro, long long ld_dro,
                                  float scale, float eps, void* dx, long long ld_dx, void* dres, long long ld_dres,
                                  float* dw, void* ws, cudaStream_t s);
int launch_gated_norm(long long rows, int D, int groups, int io, int norm_first, const void* y, long long ld_y,
                      const void* z, long long ld_z, const float* w, float eps, void* out, long long ld_out,
                      cudaStream_t s);
int launch_gated_norm_backward(long long rows, int D, int groups, int io, int norm_first, const void* dout,
                               long long ld_dout, const void* y, long long ld_y, const void* z, long long ld_z,
                               const float* w, float eps, void* dy, long long ld_dy, void* dz, long long ld_dz,
                               float* dw, void* ws, cudaStream_t s);

static thread_local char g_detail[512];

int set_error(int status, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_detail, sizeof(g_detail), fmt, ap);
    va_end(ap);
    return status;
}

int cuda_status(cudaError_t e, const char* where) {
    return set_error(SSD_ERR_CUDA, "%s: %s (%s)", where, cudaGetErrorName(e), cudaGetErrorString(e));
}

int device_sms() {
    static const int n = [] {
        int dev = 0, v = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
            v <= 0)
            v = 148;
        return v;
    }();
    return n;
}

// The dynamic shared-memory limit is a per-device attribute of a kernel: set it once per
// (kernel, device, size) instead of on every launch (a host call each time).
int smem_limit_once(const void* func, int bytes) {
    static std::mutex mu;
    static std::vector<std::tuple<const void*, int, int>> done;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_status(e, "cudaGetDevice");
    std::lock_guard<std::mutex> lock(mu);
    for (const auto& d : done)
        if (std::get<0>(d) == func && std::get<1>(d) == dev && std::get<2>(d) >= bytes) return SSD_OK;
    e = cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return cuda_status(e, "cudaFuncSetAttribute(MaxDynamicSharedMemorySize)");
    // the single-GPU prefill kernels all ask for the largest shared-memory carveout, so that
    // the small ones launched between large ones leave the SMs' L1/shared split as it is
    e = cudaFuncSetAttribute(func, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return cuda_status(e, "cudaFuncSetAttribute(PreferredSharedMemoryCarveout)");
    done.emplace_back(func, dev, bytes);
    return SSD_OK;
}

// ---- launch accounting and event timing
namespace {
constexpr int kMaxProf = 65536;
std::atomic<uint64_t> g_launches{0};
bool g_prof = false;
int g_prof_n = 0;
int g_open = -1;
std::vector<cudaEvent_t> g_ev;     // 2 per recorded launch, created on demand and reused
std::vector<int> g_rec_name;       // name index per recorded launch
std::vector<std::string> g_names;  // distinct names in first-launch order
}  // namespace

void count_launches(uint64_t n) { g_launches += n; }

void prof_start(const char* name, cudaStream_t s) {
    if (!g_prof || g_prof_n >= kMaxProf) return;
    int idx = -1;
    for (size_t i = 0; i < g_names.size(); ++i)
        if (g_names[i] == name) { idx = (int)i; break; }
    if (idx < 0) { g_names.emplace_back(name); idx = (int)g_names.size() - 1; }
    while ((int)g_ev.size() < 2 * (g_prof_n + 1)) {
        cudaEvent_t e;
        if (cudaEventCreate(&e) != cudaSuccess) return;
        g_ev.push_back(e);
    }
    if ((int)g_rec_name.size() <= g_prof_n) g_rec_name.resize(g_prof_n + 1);
    g_rec_name[g_prof_n] = idx;
    cudaEventRecord(g_ev[2 * g_prof_n], s);
    g_open = g_prof_n;
}

void prof_stop(cudaStream_t s) {
    if (!g_prof || g_open < 0) return;
    cudaEventRecord(g_ev[2 * g_open + 1], s);
    g_prof_n = g_open + 1;
    g_open = -1;
}

namespace {

constexpr int kMaxGridYZ = 65535;

struct Range {
    const void* p;
    size_t n;
};

bool overlaps(Range a, Range b) {
    if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
    const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
    return a0 < b0 + b.n && b0 < a0 + a.n;
}

int check_ptr(const void* p, const char* name, bool required) {
    if (!p) {
        if (required) return set_error(SSD_ERR_INVALID_ARG, "%s is NULL", name);
        return SSD_OK;
    }
    if (!aligned16(p)) return set_error(SSD_ERR_INVALID_ARG, "%s is not 16-byte aligned", name);
    return SSD_OK;
}

#define SSD_CHECK(expr)                 \
    do {                                \
        int st_ = (expr);               \
        if (st_ != SSD_OK) return st_;  \
    } while (0)

int check_prefill_shape(int b, int T, int H, int P, int N, int G, int chunk, int io) {
    if (io != SSD_F32 && io != SSD_BF16) return set_error(SSD_ERR_INVALID_ARG, "io_dtype %d is not SSD_F32/SSD_BF16", io);
    if (b < 0 || T < 0) return set_error(SSD_ERR_INVALID_ARG, "negative size b=%d T=%d", b, T);
    if (H < 1 || P < 1 || N < 1 || G < 1) return set_error(SSD_ERR_INVALID_ARG, "H, P, N, G must be >= 1 (H=%d P=%d N=%d G=%d)", H, P, N, G);
    if (H % G) return set_error(SSD_ERR_INVALID_ARG, "H=%d is not a multiple of G=%d", H, G);
    if (chunk != 64 && chunk != 128 && chunk != 256) return set_error(SSD_ERR_INVALID_ARG, "chunk=%d not in {64,128,256}", chunk);
    if (P != 64) return set_error(SSD_ERR_UNSUPPORTED, "P=%d (only 64 is implemented)", P);
    if (N != 64 && N != 128) return set_error(SSD_ERR_UNSUPPORTED, "N=%d (only 64 and 128 are implemented)", N);
    if (H > kMaxGridYZ || b > kMaxGridYZ) return set_error(SSD_ERR_UNSUPPORTED, "H=%d or b=%d above 65535", H, b);
    return SSD_OK;
}

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" {

int ssd_version(void) { return 100; }

const char* ssd_status_string(int status) {
    switch (status) {
        case SSD_OK: return "SSD_OK";
        case SSD_ERR_INVALID_ARG: return "SSD_ERR_INVALID_ARG: invalid argument";
        case SSD_ERR_UNSUPPORTED: return "SSD_ERR_UNSUPPORTED: shape not implemented";
        case SSD_ERR_CUDA: return "SSD_ERR_CUDA: CUDA call failed";
        case SSD_ERR_TIMEOUT: return "SSD_ERR_TIMEOUT: bounded device wait expired";
        case SSD_ERR_WORKSPACE: return "SSD_ERR_WORKSPACE: workspace missing or too small";
        case SSD_ERR_INTERNAL: return "SSD_ERR_INTERNAL: device consistency check failed";
        default: return "unknown ssd_status";
    }
}

const char* ssd_last_error(void) { return g_detail; }

uint64_t ssd_launch_count(void) { return g_launches.load(); }

int ssd_profile_begin(void) {
    g_prof = true;
    g_prof_n = 0;
    g_open = -1;
    g_names.clear();
    return SSD_OK;
}

int ssd_profile_end(ssd_kernel_time* out, int max_entries) {
    g_prof = false;
    std::vector<double> tot(g_names.size(), 0.0);
    std::vector<int> cnt(g_names.size(), 0);
    for (int i = 0; i < g_prof_n; ++i) {
        cudaError_t e = cudaEventSynchronize(g_ev[2 * i + 1]);
        float ms = 0.f;
        if (e == cudaSuccess) e = cudaEventElapsedTime(&ms, g_ev[2 * i], g_ev[2 * i + 1]);
        if (e != cudaSuccess) return -cuda_status(e, "ssd_profile_end");
        tot[g_rec_name[i]] += ms;
        cnt[g_rec_name[i]] += 1;
    }
    int n = 0;
    for (size_t k = 0; k < g_names.size() && n < max_entries && out; ++k, ++n) {
        snprintf(out[n].name, sizeof(out[n].name), "%s", g_names[k].c_str());
        out[n].launches = cnt[k];
        out[n].total_ms = tot[k];
    }
    g_prof_n = 0;
    return n;
}

// Prefill workspace: [0, 256) device status word, then the path's scratch.
static constexpr size_t kStatusBytes = 256;

// ssd_debug_force_fma_prefill: every prefill takes the fp32-FMA path
static std::atomic<int> g_force_fma{0};
static bool use_tc(int P, int N, int io) { return prefill_tc_supported(P, N, io) && !g_force_fma.load(); }

static size_t prefill_ws_bytes(int b, int T, int H, int P, int N, int chunk, int io) {
    if (use_tc(P, N, io)) return kStatusBytes + prefill_tc_workspace_bytes(b, T, H);
    return kStatusBytes + prefill_simt_workspace_bytes(b, T, H, N, chunk, io);
}

size_t ssd_prefill_workspace_size(int b, int T, int H, int P, int N, int G, int chunk, int io_dtype) {
    if (check_prefill_shape(b, T, H, P, N, G, chunk, io_dtype) != SSD_OK) return 0;
    if (b == 0 || T == 0) return 0;
    return prefill_ws_bytes(b, T, H, P, N, chunk, io_dtype);
}

int ssd_debug_starve_next_prefill(unsigned long long wait_limit_ns) {
    g_detail[0] = 0;
    if (wait_limit_ns < 1000000ull || wait_limit_ns > 10000000000ull)
        return set_error(SSD_ERR_INVALID_ARG, "wait_limit_ns %llu outside [1e6, 1e10]", wait_limit_ns);
    prefill_tc_starve_next(wait_limit_ns);
    return SSD_OK;
}

int ssd_prefill_segments(int b, int T, int H, int P, int N, int G, int chunk, int io_dtype) {
    if (check_prefill_shape(b, T, H, P, N, G, chunk, io_dtype) != SSD_OK) return 0;
    if (b == 0 || T == 0 || !use_tc(P, N, io_dtype)) return 1;
    return prefill_tc_segments(b, T, H);
}

int ssd_prefill_whole_units(int b, int T, int H, int P, int N, int G, int chunk, int io_dtype) {
    if (check_prefill_shape(b, T, H, P, N, G, chunk, io_dtype) != SSD_OK) return -1;
    if (b == 0 || T == 0 || !use_tc(P, N, io_dtype)) return b * H;
    return prefill_tc_whole_units(b, T, H);
}

size_t ssd_prefill_local_state_workspace_size(int b, int T, int H, int P, int N, int G, int io_dtype) {
    if (check_prefill_shape(b, T, H, P, N, G, 256, io_dtype) != SSD_OK || !prefill_tc_supported(P, N, io_dtype))
        return 0;
    if (b == 0 || T == 0) return 0;
    return prefill_tc_local_state_workspace_bytes(b, T, H);
}

int ssd_prefill_local_state(int b, int T, int H, int P, int N, int G, int io_dtype, const void* x, const float* dt,
                            const float* A, const void* B, float* h_local, float* log_decay, void* workspace,
                            size_t workspace_bytes, void* stream) {
    g_detail[0] = 0;
    SSD_CHECK(check_prefill_shape(b, T, H, P, N, G, 256, io_dtype));
    if (!prefill_tc_supported(P, N, io_dtype))
        return set_error(SSD_ERR_UNSUPPORTED, "local state: tensor-core shapes only (bf16, P = 64, N = 128)");
    SSD_CHECK(check_ptr(h_local, "h_local", true));
    SSD_CHECK(check_ptr(log_decay, "log_decay", true));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const size_t state_bytes = (size_t)b * H * P * N * sizeof(float), ld_bytes = (size_t)b * H * sizeof(float);
    if (overlaps({h_local, state_bytes}, {log_decay, ld_bytes}))
        return set_error(SSD_ERR_INVALID_ARG, "h_local overlaps log_decay");
    if (b == 0) return SSD_OK;
    if (T == 0) {  // no tokens: nothing accumulates and nothing decays
        SSD_CUDA_TRY(cudaMemsetAsync(h_local, 0, state_bytes, s));
        SSD_CUDA_TRY(cudaMemsetAsync(log_decay, 0, ld_bytes, s));
        return SSD_OK;
    }
    SSD_CHECK(check_ptr(x, "x", true));
    SSD_CHECK(check_ptr(dt, "dt", true));
    SSD_CHECK(check_ptr(A, "A", true));
    SSD_CHECK(check_ptr(B, "B", true));
    const Range outs[] = {{h_local, state_bytes}, {log_decay, ld_bytes}};
    const Range rin[] = {{x, (size_t)b * T * H * P * 2}, {B, (size_t)b * T * G * N * 2}, {dt, (size_t)b * T * H * 4},
                         {A, (size_t)H * 4}};
    for (const Range& o : outs)
        for (const Range& i : rin)
            if (overlaps(o, i)) return set_error(SSD_ERR_INVALID_ARG, "an output overlaps an input");
    const size_t need = prefill_tc_local_state_workspace_bytes(b, T, H);
    if (!workspace || workspace_bytes < need)
        return set_error(SSD_ERR_WORKSPACE, "workspace %zu bytes at %p, need %zu", workspace_bytes, workspace, need);
    if (!aligned16(workspace)) return set_error(SSD_ERR_INVALID_ARG, "workspace is not 16-byte aligned");
    for (const Range& o : outs)
        if (overlaps({workspace, need}, o)) return set_error(SSD_ERR_INVALID_ARG, "workspace overlaps an output");
    for (const Range& i : rin)
        if (overlaps({workspace, need}, i)) return set_error(SSD_ERR_INVALID_ARG, "workspace overlaps an input");
    return launch_prefill_tc_local_state(b, T, H, G, x, dt, A, B, h_local, log_decay, workspace, s);
}

int ssd_prefill_context_scan(int world, int rank, int b, int H, int P, int N, const float* h0, const float* h_local_all,
                             const float* log_decay_all, float* h_in, void* stream) {
    g_detail[0] = 0;
    if (world < 1 || rank < 0 || rank >= world)
        return set_error(SSD_ERR_INVALID_ARG, "rank %d outside [0, world=%d)", rank, world);
    if (b < 0 || H < 1) return set_error(SSD_ERR_INVALID_ARG, "b=%d H=%d", b, H);
    if (P != 64 || N != 128) return set_error(SSD_ERR_UNSUPPORTED, "context scan: P = 64, N = 128 only");
    if (H > kMaxGridYZ || b > kMaxGridYZ) return set_error(SSD_ERR_UNSUPPORTED, "H=%d or b=%d above 65535", H, b);
    SSD_CHECK(check_ptr(h0, "h0", false));
    SSD_CHECK(check_ptr(h_in, "h_in", true));
    if (rank > 0) {
        SSD_CHECK(check_ptr(h_local_all, "h_local_all", true));
        SSD_CHECK(check_ptr(log_decay_all, "log_decay_all", true));
    }
    const size_t state_bytes = (size_t)b * H * P * N * sizeof(float);
    if (overlaps({h_in, state_bytes}, {h_local_all, (size_t)world * state_bytes}) ||
        overlaps({h_in, state_bytes}, {log_decay_all, (size_t)world * b * H * 4}) ||
        (h0 && h0 != h_in && overlaps({h_in, state_bytes}, {h0, state_bytes})))
        return set_error(SSD_ERR_INVALID_ARG, "h_in overlaps an input (only exact aliasing of h0 is allowed)");
    if (b == 0) return SSD_OK;
    return launch_context_scan(rank, b, H, h0, h_local_all, log_decay_all, h_in, static_cast<cudaStream_t>(stream));
}

int ssd_debug_decay_precision(int mode) {
    g_detail[0] = 0;
    if (mode < 0 || mode > 2) return set_error(SSD_ERR_INVALID_ARG, "decay precision mode %d is not 0, 1 or 2", mode);
    prefill_tc_decay_mode(mode);
    return SSD_OK;
}

int ssd_debug_force_prefill_split(int n_full, int nseg) {
    g_detail[0] = 0;
    if (n_full < 0 || nseg < 0) return set_error(SSD_ERR_INVALID_ARG, "n_full %d / nseg %d negative", n_full, nseg);
    prefill_tc_force_split(n_full, nseg);
    return SSD_OK;
}

int ssd_debug_force_fma_prefill(int on) {
    g_detail[0] = 0;
    if (on != 0 && on != 1) return set_error(SSD_ERR_INVALID_ARG, "on is %d, not 0 or 1", on);
    g_force_fma.store(on);
    return SSD_OK;
}

int ssd_debug_force_prefill_segments(int nseg) {
    g_detail[0] = 0;
    if (nseg < 0) return set_error(SSD_ERR_INVALID_ARG, "nseg %d is negative", nseg);
    prefill_tc_force_segments(nseg);
    return SSD_OK;
}

int ssd_prefill_check(void* workspace, void* stream) {
    g_detail[0] = 0;
    if (!workspace) return set_error(SSD_ERR_INVALID_ARG, "workspace is NULL");
    return prefill_tc_status(workspace, static_cast<cudaStream_t>(stream));
}

static int prefill_impl(int b, int T, int H, int P, int N, int G, int chunk, int io_dtype, const void* x,
                        const float* dt, const DtMap& dtm, const float* A, const void* B, const void* C,
                        const float* D, const float* h0, void* y, float* h_final, void* workspace,
                        size_t workspace_bytes, void* stream) {
    SSD_CHECK(check_prefill_shape(b, T, H, P, N, G, chunk, io_dtype));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const size_t state_bytes = (size_t)b * H * P * N * sizeof(float);
    SSD_CHECK(check_ptr(h0, "h0", false));
    SSD_CHECK(check_ptr(h_final, "h_final", false));
    if (h0 && h_final && h0 != h_final && overlaps({h0, state_bytes}, {h_final, state_bytes}))
        return set_error(SSD_ERR_INVALID_ARG, "h_final partially overlaps h0 (only exact aliasing is allowed)");
    if (b == 0) return SSD_OK;
    if (T == 0) {  // no tokens: the state passes through unchanged
        if (h_final && h_final != h0) {
            if (h0) SSD_CUDA_TRY(cudaMemcpyAsync(h_final, h0, state_bytes, cudaMemcpyDeviceToDevice, s));
            else SSD_CUDA_TRY(cudaMemsetAsync(h_final, 0, state_bytes, s));
        }
        return SSD_OK;
    }
    SSD_CHECK(check_ptr(x, "x", true));
    SSD_CHECK(check_ptr(dt, "dt", true));
    SSD_CHECK(check_ptr(A, "A", true));
    SSD_CHECK(check_ptr(B, "B", true));
    SSD_CHECK(check_ptr(C, "C", true));
    SSD_CHECK(check_ptr(D, "D", true));
    SSD_CHECK(check_ptr(y, "y", true));
    const size_t io_b = io_dtype == SSD_BF16 ? 2 : 4;
    const Range ry{y, (size_t)b * T * H * P * io_b};
    const Range rin[] = {{x, (size_t)b * T * H * P * io_b}, {B, (size_t)b * T * G * N * io_b},
                         {C, (size_t)b * T * G * N * io_b}, {dt, (size_t)b * T * H * 4},
                         {A, (size_t)H * 4}, {D, (size_t)H * 4}, {h0, h0 ? state_bytes : 0}};
    const char* names[] = {"x", "B", "C", "dt", "A", "D", "h0"};
    for (int i = 0; i < 7; ++i) {
        if (overlaps(ry, rin[i])) return set_error(SSD_ERR_INVALID_ARG, "y overlaps input %s", names[i]);
        if (i < 6 && overlaps({h_final, h_final ? state_bytes : 0}, rin[i]))
            return set_error(SSD_ERR_INVALID_ARG, "h_final overlaps input %s", names[i]);
    }
    if (overlaps(ry, {h_final, h_final ? state_bytes : 0})) return set_error(SSD_ERR_INVALID_ARG, "y overlaps h_final");
    const size_t need = prefill_ws_bytes(b, T, H, P, N, chunk, io_dtype);
    if (!workspace || workspace_bytes < need)
        return set_error(SSD_ERR_WORKSPACE, "workspace %zu bytes at %p, need %zu", workspace_bytes, workspace, need);
    if (!aligned16(workspace)) return set_error(SSD_ERR_INVALID_ARG, "workspace is not 16-byte aligned");
    if (overlaps({workspace, need}, ry)) return set_error(SSD_ERR_INVALID_ARG, "workspace overlaps y");
    if (overlaps({workspace, need}, {h_final, h_final ? state_bytes : 0}))
        return set_error(SSD_ERR_INVALID_ARG, "workspace overlaps h_final");
    for (int i = 0; i < 7; ++i)
        if (overlaps({workspace, need}, rin[i])) return set_error(SSD_ERR_INVALID_ARG, "workspace overlaps %s", names[i]);
    if (use_tc(P, N, io_dtype))
        return launch_prefill_tc(b, T, H, G, x, dt, dtm, A, B, C, D, h0, y, h_final, workspace, s);
    SSD_CUDA_TRY(cudaMemsetAsync(workspace, 0, sizeof(int), s));
    return launch_prefill_simt(b, T, H, N, G, chunk, io_dtype, x, dt, dtm, A, B, C, D, h0, y, h_final,
                               static_cast<char*>(workspace) + kStatusBytes, s);
}

int ssd_prefill(int b, int T, int H, int P, int N, int G, int chunk, int io_dtype,
                const void* x, const float* dt, const float* A, const void* B, const void* C,
                const float* D, const float* h0, void* y, float* h_final, void* workspace,
                size_t workspace_bytes, void* stream) {
    g_detail[0] = 0;
    const DtMap plain{nullptr, 0.f, 0.f, 0};
    return prefill_impl(b, T, H, P, N, G, chunk, io_dtype, x, dt, plain, A, B, C, D, h0, y, h_final, workspace,
                        workspace_bytes, stream);
}

int ssd_prefill_dt_raw(int b, int T, int H, int P, int N, int G, int chunk, int io_dtype,
                       const void* x, const float* dt_raw, const float* dt_bias, float dt_min, float dt_max,
                       const float* A, const void* B, const void* C, const float* D, const float* h0,
                       void* y, float* h_final, void* workspace, size_t workspace_bytes, void* stream) {
    g_detail[0] = 0;
    if (!(dt_min >= 0.f) || !(dt_max > dt_min))  // also rejects NaN limits
        return set_error(SSD_ERR_INVALID_ARG, "dt clamp range [%g, %g] must satisfy 0 <= dt_min < dt_max",
                         (double)dt_min, (double)dt_max);
    SSD_CHECK(check_ptr(dt_bias, "dt_bias", false));
    if (dt_bias && H > 0 && overlaps({dt_bias, (size_t)H * 4}, {y, (size_t)b * T * H * P * (io_dtype == SSD_BF16 ? 2 : 4)}))
        return set_error(SSD_ERR_INVALID_ARG, "y overlaps input dt_bias");
    const DtMap raw{dt_bias, dt_min, dt_max, 1};
    return prefill_impl(b, T, H, P, N, G, chunk, io_dtype, x, dt_raw, raw, A, B, C, D, h0, y, h_final, workspace,
                        workspace_bytes, stream);
}

size_t ssd_decode_workspace_size(int layers, int b, int G) {
    if (layers < 1 || b < 1 || G < 1) return 0;
    return decode_workspace_bytes(layers, b, G);
}

static int check_decode(int layers, int b, int H, int P, int N, int G, int kconv, int act, int io,
                        const float* h, const float* conv_state, const float* A, const float* D,
                        const float* conv_w, const float* conv_b, void* ws, size_t ws_bytes) {
    if (io != SSD_F32 && io != SSD_BF16) return set_error(SSD_ERR_INVALID_ARG, "io_dtype %d is not SSD_F32/SSD_BF16", io);
    if (act != SSD_ACT_NONE && act != SSD_ACT_SILU) return set_error(SSD_ERR_INVALID_ARG, "act %d is not SSD_ACT_NONE/SSD_ACT_SILU", act);
    if (layers < 0 || b < 0) return set_error(SSD_ERR_INVALID_ARG, "negative size layers=%d b=%d", layers, b);
    if (H < 1 || P < 1 || N < 1 || G < 1) return set_error(SSD_ERR_INVALID_ARG, "H, P, N, G must be >= 1");
    if (H % G) return set_error(SSD_ERR_INVALID_ARG, "H=%d is not a multiple of G=%d", H, G);
    if (kconv < 1) return set_error(SSD_ERR_INVALID_ARG, "kconv=%d must be >= 1", kconv);
    if (kconv != 4) return set_error(SSD_ERR_UNSUPPORTED, "kconv=%d (only 4 is implemented)", kconv);
    if (P != 64) return set_error(SSD_ERR_UNSUPPORTED, "P=%d (only 64 is implemented)", P);
    if (N != 64 && N != 128) return set_error(SSD_ERR_UNSUPPORTED, "N=%d (only 64 and 128 are implemented)", N);
    if (layers > kMaxGridYZ || b > kMaxGridYZ) return set_error(SSD_ERR_UNSUPPORTED, "layers or b above 65535");
    if (layers == 0 || b == 0) return SSD_OK;
    SSD_CHECK(check_ptr(h, "h", true));
    SSD_CHECK(check_ptr(conv_state, "conv_state", true));
    SSD_CHECK(check_ptr(A, "A", true));
    SSD_CHECK(check_ptr(D, "D", true));
    SSD_CHECK(check_ptr(conv_w, "conv_w", true));
    SSD_CHECK(check_ptr(conv_b, "conv_b", true));
    const size_t need = decode_workspace_bytes(layers, b, G);
    if (!ws || ws_bytes < need) return set_error(SSD_ERR_WORKSPACE, "workspace %zu bytes at %p, need %zu", ws_bytes, ws, need);
    if (!aligned16(ws)) return set_error(SSD_ERR_INVALID_ARG, "workspace is not 16-byte aligned");
    return SSD_OK;
}

// The buffers a decode step writes (h, conv_state, y and the workspace's arrival counters)
// must not overlap one another or any buffer the step reads (xbc, dt, A, D, conv_w, conv_b);
// for a plan, xbc, dt and y hold `ring` steps.
static int check_decode_overlaps(int layers, int b, int H, int P, int N, int G, int kconv, int io_dtype,
                                 const float* h, const float* conv_state, const void* xbc, const float* dt,
                                 const float* A, const float* D, const float* conv_w, const float* conv_b,
                                 const void* y, int ring, const void* ws) {
    const size_t io_b = io_dtype == SSD_BF16 ? 2 : 4;
    const size_t Dc = (size_t)H * P + 2 * (size_t)G * N, lb = (size_t)layers * b, R = (size_t)ring;
    const Range writes[] = {{h, lb * H * P * N * 4}, {conv_state, lb * Dc * (kconv - 1) * 4},
                            {y, R * lb * H * P * io_b}, {ws, decode_workspace_bytes(layers, b, G)}};
    const Range reads[] = {{xbc, R * lb * Dc * io_b},         {dt, R * lb * H * 4},
                           {A, (size_t)layers * H * 4},       {D, (size_t)layers * H * 4},
                           {conv_w, (size_t)layers * Dc * kconv * 4}, {conv_b, (size_t)layers * Dc * 4}};
    const char* wname[] = {"h", "conv_state", "y", "workspace"};
    const char* rname[] = {"xbc", "dt", "A", "D", "conv_w", "conv_b"};
    for (int i = 0; i < 4; ++i) {
        for (int j = i + 1; j < 4; ++j)
            if (overlaps(writes[i], writes[j]))
                return set_error(SSD_ERR_INVALID_ARG, "%s overlaps %s", wname[i], wname[j]);
        for (int j = 0; j < 6; ++j)
            if (overlaps(writes[i], reads[j]))
                return set_error(SSD_ERR_INVALID_ARG, "%s overlaps %s", wname[i], rname[j]);
    }
    return SSD_OK;
}

int ssd_decode_step(int layers, int b, int H, int P, int N, int G, int kconv, int act, int io_dtype,
                    float* h, float* conv_state, const void* xbc, const float* dt, const float* A,
                    const float* D, const float* conv_w, const float* conv_b, void* y,
                    void* workspace, size_t workspace_bytes, void* stream) {
    g_detail[0] = 0;
    SSD_CHECK(check_decode(layers, b, H, P, N, G, kconv, act, io_dtype, h, conv_state, A, D, conv_w,
                           conv_b, workspace, workspace_bytes));
    if (layers == 0 || b == 0) return SSD_OK;
    SSD_CHECK(check_ptr(xbc, "xbc", true));
    SSD_CHECK(check_ptr(dt, "dt", true));
    SSD_CHECK(check_ptr(y, "y", true));
    SSD_CHECK(check_decode_overlaps(layers, b, H, P, N, G, kconv, io_dtype, h, conv_state, xbc, dt, A, D, conv_w,
                                    conv_b, y, 1, workspace));
    return launch_decode_step(layers, b, H, N, G, act, io_dtype, h, conv_state, xbc, dt, A, D, conv_w,
                              conv_b, y, workspace, static_cast<cudaStream_t>(stream));
}

int ssd_decode_step_noalloc(int layers, int b, int H, int P, int N, int G, int kconv, int act,
                            int io_dtype, float* h, float* conv_state, const void* xbc,
                            const float* dt, const float* A, const float* D, const float* conv_w,
                            const float* conv_b, void* y, void* stream) {
    g_detail[0] = 0;
    if (layers > 0 && b > 0 && G > 0 &&
        (size_t)layers * (size_t)b * (size_t)G > (size_t)SSD_DECODE_NOALLOC_MAX_COUNTERS)
        return set_error(SSD_ERR_INVALID_ARG,
                         "layers*b*G = %zu exceeds the %d arrival counters of the allocation-free decode step",
                         (size_t)layers * b * G, SSD_DECODE_NOALLOC_MAX_COUNTERS);
    void* scratch = nullptr;
    size_t cap = 0;
    if (layers > 0 && b > 0) SSD_CHECK(decode_noalloc_scratch(&scratch, &cap));
    // the library's own scratch stands in for the caller workspace of ssd_decode_step
    return ssd_decode_step(layers, b, H, P, N, G, kconv, act, io_dtype, h, conv_state, xbc, dt, A, D,
                           conv_w, conv_b, y, scratch, cap, stream);
}

int ssd_decode_plan_create(ssd_decode_plan** plan, int layers, int b, int H, int P, int N, int G,
                           int kconv, int act, int io_dtype, float* h, float* conv_state,
                           const void* xbc_ring, const float* dt_ring, int ring, const float* A,
                           const float* D, const float* conv_w, const float* conv_b, void* y_ring,
                           int n_steps, void* workspace, size_t workspace_bytes) {
    g_detail[0] = 0;
    if (!plan) return set_error(SSD_ERR_INVALID_ARG, "plan is NULL");
    *plan = nullptr;
    SSD_CHECK(check_decode(layers, b, H, P, N, G, kconv, act, io_dtype, h, conv_state, A, D, conv_w,
                           conv_b, workspace, workspace_bytes));
    if (layers == 0 || b == 0) return set_error(SSD_ERR_INVALID_ARG, "a decode plan needs layers >= 1 and b >= 1");
    if (ring < 1) return set_error(SSD_ERR_INVALID_ARG, "ring=%d must be >= 1", ring);
    if (n_steps < 0) return set_error(SSD_ERR_INVALID_ARG, "n_steps=%d must be >= 0", n_steps);
    SSD_CHECK(check_ptr(xbc_ring, "xbc_ring", true));
    SSD_CHECK(check_ptr(dt_ring, "dt_ring", true));
    SSD_CHECK(check_ptr(y_ring, "y_ring", true));
    SSD_CHECK(check_decode_overlaps(layers, b, H, P, N, G, kconv, io_dtype, h, conv_state, xbc_ring, dt_ring, A, D,
                                    conv_w, conv_b, y_ring, ring, workspace));
    return create_decode_plan(plan, layers, b, H, N, G, act, io_dtype, h, conv_state, xbc_ring, dt_ring,
                              ring, A, D, conv_w, conv_b, y_ring, n_steps, workspace);
}

int ssd_decode_plan_launch(ssd_decode_plan* plan, void* stream) {
    g_detail[0] = 0;
    if (!plan) return set_error(SSD_ERR_INVALID_ARG, "plan is NULL");
    return launch_decode_plan(plan, static_cast<cudaStream_t>(stream));
}

int ssd_decode_plan_destroy(ssd_decode_plan* plan) {
    g_detail[0] = 0;
    if (!plan) return SSD_OK;
    return destroy_decode_plan(plan);
}

int ssd_decode_loop(int layers, int b, int H, int P, int N, int G, int kconv, int act, int io_dtype, float* h,
                    float* conv_state, const void* xbc_ring, const float* dt_ring, int ring, const float* A,
                    const float* D, const float* conv_w, const float* conv_b, void* y_ring, int n_steps,
                    void* workspace, size_t workspace_bytes, void* stream) {
    ssd_decode_plan* plan = nullptr;
    SSD_CHECK(ssd_decode_plan_create(&plan, layers, b, H, P, N, G, kconv, act, io_dtype, h, conv_state, xbc_ring,
                                     dt_ring, ring, A, D, conv_w, conv_b, y_ring, n_steps, workspace,
                                     workspace_bytes));
    const int st = ssd_decode_plan_launch(plan, stream);
    // an executable graph destroyed while in flight is freed when it completes
    const int st2 = destroy_decode_plan(plan);
    return st != SSD_OK ? st : st2;
}

// ---- gradients of the prefill

static bool backward_use_tc(const BwdArgs& a) { return backward_tc_supported(64, a.N, a.io) && !g_force_fma.load(); }

static size_t backward_ws_bytes(const BwdArgs& a) {
    return kStatusBytes + (backward_use_tc(a) ? backward_tc_workspace_bytes(a) : backward_simt_workspace_bytes(a));
}

int ssd_debug_starve_next_prefill_backward(unsigned long long wait_limit_ns) {
    g_detail[0] = 0;
    if (wait_limit_ns < 1000000ull || wait_limit_ns > 10000000000ull)
        return set_error(SSD_ERR_INVALID_ARG, "wait_limit_ns %llu outside [1e6, 1e10]", wait_limit_ns);
    backward_tc_starve_next(wait_limit_ns);
    return SSD_OK;
}

int ssd_debug_lag_next_prefill_backward(int role) {
    g_detail[0] = 0;
    return backward_tc_lag_next(role);
}

static BwdArgs backward_shape(int b, int T, int H, int N, int G, int io) {
    BwdArgs a = {};
    a.b = b, a.T = T, a.H = H, a.N = N, a.G = G, a.io = io;
    return a;
}

size_t ssd_prefill_backward_workspace_size(int b, int T, int H, int P, int N, int G, int io_dtype) {
    if (check_prefill_shape(b, T, H, P, N, G, 64, io_dtype) != SSD_OK) return 0;
    if (b == 0 || T == 0) return 0;
    const BwdArgs a = backward_shape(b, T, H, N, G, io_dtype);
    return backward_simt_fits(a) ? backward_ws_bytes(a) : 0;
}

static int backward_impl(const BwdArgs& a, int P, void* workspace, size_t workspace_bytes, cudaStream_t s) {
    const int b = a.b, T = a.T, H = a.H, N = a.N, G = a.G;
    SSD_CHECK(check_prefill_shape(b, T, H, P, N, G, 64, a.io));
    const size_t io_b = a.io == SSD_BF16 ? 2 : 4, tok = (size_t)b * T;
    const size_t state = (size_t)b * H * P * N * sizeof(float), xb = tok * H * P * io_b, bb = tok * G * N * io_b,
                 db = tok * H * 4, hb = (size_t)H * 4;
    struct Buf {
        const char* name;
        const void* p;
        size_t n;
        bool required;
    };
    const Buf ins[] = {{"dy", a.dy, xb, true},     {"x", a.x, xb, true},     {"dt", a.dt, db, true},
                       {"A", a.A, hb, true},       {"B", a.B, bb, true},     {"C", a.C, bb, true},
                       {"D", a.D, hb, true},       {"h0", a.h0, state, false},
                       {"dh_final", a.dhf, state, false}, {"dt_bias", a.dtm.bias, hb, false}};
    const Buf outs[] = {{"dx", a.dx, xb, true},    {"ddt", a.ddt, db, true}, {"dA", a.dA, hb, true},
                        {"dB", a.dB, bb, true},    {"dC", a.dC, bb, true},   {"dD", a.dD, hb, true},
                        {"dh0", a.dh0, state, false}, {"ddt_bias", a.dbias, hb, false}};
    const bool empty = b == 0 || T == 0;
    for (const Buf& i : ins) SSD_CHECK(check_ptr(i.p, i.name, i.required && !empty));
    for (const Buf& o : outs) SSD_CHECK(check_ptr(o.p, o.name, o.required && (o.n == hb || !empty)));
    for (size_t i = 0; i < sizeof(outs) / sizeof(outs[0]); ++i) {
        for (const Buf& in : ins)
            if (overlaps({outs[i].p, outs[i].n}, {in.p, in.n}))
                return set_error(SSD_ERR_INVALID_ARG, "%s overlaps input %s", outs[i].name, in.name);
        for (size_t j = 0; j < i; ++j)
            if (overlaps({outs[i].p, outs[i].n}, {outs[j].p, outs[j].n}))
                return set_error(SSD_ERR_INVALID_ARG, "%s overlaps %s", outs[i].name, outs[j].name);
    }
    if (empty) {  // no tokens: empty sums, and the state's adjoint passes through unchanged
        SSD_CUDA_TRY(cudaMemsetAsync(a.dA, 0, hb, s));
        SSD_CUDA_TRY(cudaMemsetAsync(a.dD, 0, hb, s));
        if (a.dbias) SSD_CUDA_TRY(cudaMemsetAsync(a.dbias, 0, hb, s));
        if (a.dh0 && state) {
            if (a.dhf) SSD_CUDA_TRY(cudaMemcpyAsync(a.dh0, a.dhf, state, cudaMemcpyDeviceToDevice, s));
            else SSD_CUDA_TRY(cudaMemsetAsync(a.dh0, 0, state, s));
        }
        return SSD_OK;
    }
    if (!backward_simt_fits(a)) return set_error(SSD_ERR_UNSUPPORTED, "b * T * H too large for one call");
    const size_t need = backward_ws_bytes(a);
    if (!workspace || workspace_bytes < need)
        return set_error(SSD_ERR_WORKSPACE, "workspace %zu bytes at %p, need %zu", workspace_bytes, workspace, need);
    if (!aligned16(workspace)) return set_error(SSD_ERR_INVALID_ARG, "workspace is not 16-byte aligned");
    for (const Buf& i : ins)
        if (overlaps({workspace, need}, {i.p, i.n})) return set_error(SSD_ERR_INVALID_ARG, "workspace overlaps %s", i.name);
    for (const Buf& o : outs)
        if (overlaps({workspace, need}, {o.p, o.n})) return set_error(SSD_ERR_INVALID_ARG, "workspace overlaps %s", o.name);
    if (backward_use_tc(a)) return launch_backward_tc(a, workspace, kStatusBytes, s);
    SSD_CUDA_TRY(cudaMemsetAsync(workspace, 0, sizeof(int), s));
    return launch_backward_simt(a, static_cast<char*>(workspace) + kStatusBytes, s);
}

int ssd_prefill_backward(int b, int T, int H, int P, int N, int G, int io_dtype, const void* dy, const void* x,
                         const float* dt, const float* A, const void* B, const void* C, const float* D,
                         const float* h0, const float* dh_final, void* dx, float* ddt, float* dA, void* dB, void* dC,
                         float* dD, float* dh0, void* workspace, size_t workspace_bytes, void* stream) {
    g_detail[0] = 0;
    const BwdArgs a{b, T, H, N, G, io_dtype, dy, x, dt, DtMap{nullptr, 0.f, 0.f, 0}, A, B, C, D, h0, dh_final,
                    dx, ddt, dA, dB, dC, dD, dh0, nullptr};
    return backward_impl(a, P, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

int ssd_prefill_backward_dt_raw(int b, int T, int H, int P, int N, int G, int io_dtype, const void* dy, const void* x,
                                const float* dt_raw, const float* dt_bias, float dt_min, float dt_max, const float* A,
                                const void* B, const void* C, const float* D, const float* h0, const float* dh_final,
                                void* dx, float* ddt_raw, float* ddt_bias, float* dA, void* dB, void* dC, float* dD,
                                float* dh0, void* workspace, size_t workspace_bytes, void* stream) {
    g_detail[0] = 0;
    if (!(dt_min >= 0.f) || !(dt_max > dt_min))  // also rejects NaN limits
        return set_error(SSD_ERR_INVALID_ARG, "dt clamp range [%g, %g] must satisfy 0 <= dt_min < dt_max",
                         (double)dt_min, (double)dt_max);
    const BwdArgs a{b, T, H, N, G, io_dtype, dy, x, dt_raw, DtMap{dt_bias, dt_min, dt_max, 1}, A, B, C, D, h0, dh_final,
                    dx, ddt_raw, dA, dB, dC, dD, dh0, ddt_bias};
    return backward_impl(a, P, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

// ---- norms around a block

// A matrix operand of a norm call: rows of D elements, ld elements apart.
struct NormMat {
    const char* name;
    const void* p;
    long long ld;
    int elem;       // bytes an element
    bool required, written;
};

static constexpr int kNormMaxLen = 16384;  // elements one reduction spans (registers of a block)

static Range norm_range(const NormMat& m, long long rows, int D) {
    if (!m.p || rows == 0) return {nullptr, 0};
    return {m.p, ((size_t)(rows - 1) * (size_t)m.ld + (size_t)D) * m.elem};
}

// Do two matrices share an element?  Rows of the same stride in bytes may lie side by side, as two
// column slices of one buffer do.
static bool mats_overlap(const NormMat& a, const NormMat& b, long long rows, int D) {
    if (!overlaps(norm_range(a, rows, D), norm_range(b, rows, D))) return false;
    const size_t ld = (size_t)a.ld * a.elem, na = (size_t)D * a.elem, nb = (size_t)D * b.elem;
    if (ld != (size_t)b.ld * b.elem) return true;
    const uintptr_t pa = (uintptr_t)a.p, pb = (uintptr_t)b.p;
    const size_t d = pb >= pa ? (pb - pa) % ld : (ld - (pa - pb) % ld) % ld;  // b's column in a's rows
    return d < na || d + nb > ld;
}

// Shapes, pointers and overlaps of a norm call.  `inplace` names a pair (input, output) that may
// be the same memory with the same stride.
static int check_norm(long long rows, int D, int groups, int io, int res_dtype, float eps, const NormMat* mats, int n,
                      const float* weight, const float* dweight, int inplace_in, int inplace_out) {
    if (io != SSD_F32 && io != SSD_BF16) return set_error(SSD_ERR_INVALID_ARG, "io_dtype %d is not SSD_F32/SSD_BF16", io);
    if (res_dtype != SSD_F32 && res_dtype != SSD_BF16)
        return set_error(SSD_ERR_INVALID_ARG, "res_dtype %d is not SSD_F32/SSD_BF16", res_dtype);
    if (io == SSD_F32 && res_dtype == SSD_BF16)
        return set_error(SSD_ERR_UNSUPPORTED, "a bf16 residual beside fp32 io is not implemented");
    if (rows < 0) return set_error(SSD_ERR_INVALID_ARG, "negative size rows=%lld", rows);
    if (D < 1 || groups < 1 || D % groups)
        return set_error(SSD_ERR_INVALID_ARG, "D=%d groups=%d: D must be a positive multiple of groups", D, groups);
    if (D / groups > kNormMaxLen) return set_error(SSD_ERR_UNSUPPORTED, "a norm over %d elements (at most %d)", D / groups, kNormMaxLen);
    if (groups > kMaxGridYZ) return set_error(SSD_ERR_UNSUPPORTED, "groups=%d above 65535", groups);
    if (!(eps >= 0.f) || std::isinf(eps)) return set_error(SSD_ERR_INVALID_ARG, "eps=%g must be finite and >= 0", (double)eps);
    SSD_CHECK(check_ptr(weight, "weight", true));
    SSD_CHECK(check_ptr(dweight, "dweight", false));
    if (rows == 0) return SSD_OK;
    for (int i = 0; i < n; ++i) {
        const NormMat& m = mats[i];
        if (!m.p) {
            if (m.required) return set_error(SSD_ERR_INVALID_ARG, "%s is NULL", m.name);
            continue;
        }
        if ((uintptr_t)m.p % m.elem) return set_error(SSD_ERR_INVALID_ARG, "%s is not aligned to its elements", m.name);
        if (m.ld < D) return set_error(SSD_ERR_INVALID_ARG, "%s has a row stride of %lld, below D=%d", m.name, m.ld, D);
        if (m.ld > (1LL << 56) / rows)
            return set_error(SSD_ERR_INVALID_ARG, "%s: %lld rows %lld apart pass the address space", m.name, rows, m.ld);
    }
    const Range rw{weight, (size_t)D * 4}, rdw{dweight, dweight ? (size_t)D * 4 : 0};
    if (overlaps(rdw, rw)) return set_error(SSD_ERR_INVALID_ARG, "dweight overlaps weight");
    for (int i = 0; i < n; ++i) {
        const Range ri = norm_range(mats[i], rows, D);
        if (overlaps(rdw, ri)) return set_error(SSD_ERR_INVALID_ARG, "dweight overlaps %s", mats[i].name);
        if (!mats[i].written) continue;
        if (overlaps(ri, rw)) return set_error(SSD_ERR_INVALID_ARG, "%s overlaps weight", mats[i].name);
        for (int j = 0; j < n; ++j) {
            if (j == i || (mats[j].written && j < i)) continue;
            if (i == inplace_out && j == inplace_in && mats[i].p == mats[j].p && mats[i].ld == mats[j].ld) continue;
            if (mats_overlap(mats[i], mats[j], rows, D))
                return set_error(SSD_ERR_INVALID_ARG, "%s overlaps %s", mats[i].name, mats[j].name);
        }
    }
    return SSD_OK;
}

// The backward passes' workspace: needed for dweight only.
static int check_norm_workspace(long long rows, int D, int groups, const NormMat* mats, int n, const float* weight,
                                const float* dweight, void* ws, size_t ws_bytes) {
    if (!dweight) return SSD_OK;
    const size_t need = norm_workspace_bytes(rows, D, groups);
    if (!ws || ws_bytes < need) return set_error(SSD_ERR_WORKSPACE, "workspace %zu bytes at %p, need %zu", ws_bytes, ws, need);
    if (!aligned16(ws)) return set_error(SSD_ERR_INVALID_ARG, "workspace is not 16-byte aligned");
    const Range rws{ws, need};
    if (overlaps(rws, {weight, (size_t)D * 4}) || overlaps(rws, {dweight, (size_t)D * 4}))
        return set_error(SSD_ERR_INVALID_ARG, "workspace overlaps weight or dweight");
    for (int i = 0; i < n; ++i)
        if (overlaps(rws, norm_range(mats[i], rows, D)))
            return set_error(SSD_ERR_INVALID_ARG, "workspace overlaps %s", mats[i].name);
    return SSD_OK;
}

static int elem_bytes(int dtype) { return dtype == SSD_BF16 ? 2 : 4; }

size_t ssd_norm_backward_workspace_size(long long rows, int D, int groups) {
    if (rows < 1 || D < 1 || groups < 1 || D % groups || D / groups > kNormMaxLen || groups > kMaxGridYZ) return 0;
    return norm_workspace_bytes(rows, D, groups);
}

int ssd_residual_norm(long long rows, int D, int io_dtype, int res_dtype, const void* x, long long ld_x,
                      const void* residual, long long ld_residual, float scale, const float* weight, float eps,
                      void* out, long long ld_out, void* residual_out, long long ld_residual_out, void* stream) {
    g_detail[0] = 0;
    const int eb = elem_bytes(io_dtype), rb = elem_bytes(res_dtype);
    const NormMat mats[] = {{"x", x, ld_x, eb, true, false},
                            {"residual", residual, ld_residual, rb, false, false},
                            {"out", out, ld_out, eb, true, true},
                            {"residual_out", residual_out, ld_residual_out, rb, false, true}};
    SSD_CHECK(check_norm(rows, D, 1, io_dtype, res_dtype, eps, mats, 4, weight, nullptr, 1, 3));
    if (!std::isfinite(scale)) return set_error(SSD_ERR_INVALID_ARG, "scale must be finite");
    if (rows == 0) return SSD_OK;
    return launch_residual_norm(rows, D, io_dtype, res_dtype, x, ld_x, residual, ld_residual, scale, weight, eps, out,
                                ld_out, residual_out, ld_residual_out, static_cast<cudaStream_t>(stream));
}

int ssd_residual_norm_backward(long long rows, int D, int io_dtype, int res_dtype, const void* dout, long long ld_dout,
                               const void* r, long long ld_r, const float* weight, const void* dresidual_out,
                               long long ld_dresidual_out, float scale, float eps, void* dx, long long ld_dx,
                               void* dresidual, long long ld_dresidual, float* dweight, void* workspace,
                               size_t workspace_bytes, void* stream) {
    g_detail[0] = 0;
    const int eb = elem_bytes(io_dtype), rb = elem_bytes(res_dtype);
    const NormMat mats[] = {{"dout", dout, ld_dout, eb, true, false},
                            {"r", r, ld_r, rb, true, false},
                            {"dresidual_out", dresidual_out, ld_dresidual_out, rb, false, false},
                            {"dx", dx, ld_dx, eb, false, true},
                            {"dresidual", dresidual, ld_dresidual, rb, false, true}};
    SSD_CHECK(check_norm(rows, D, 1, io_dtype, res_dtype, eps, mats, 5, weight, dweight, 2, 4));
    if (!std::isfinite(scale)) return set_error(SSD_ERR_INVALID_ARG, "scale must be finite");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (rows == 0) {  // no rows: nothing but an empty sum
        if (dweight) SSD_CUDA_TRY(cudaMemsetAsync(dweight, 0, (size_t)D * 4, s));
        return SSD_OK;
    }
    SSD_CHECK(check_norm_workspace(rows, D, 1, mats, 5, weight, dweight, workspace, workspace_bytes));
    return launch_residual_norm_backward(rows, D, io_dtype, res_dtype, dout, ld_dout, r, ld_r, weight, dresidual_out,
                                         ld_dresidual_out, scale, eps, dx, ld_dx, dresidual, ld_dresidual, dweight,
                                         workspace, s);
}

int ssd_gated_norm(long long rows, int D, int groups, int io_dtype, int norm_before_gate, const void* y, long long ld_y,
                   const void* z, long long ld_z, const float* weight, float eps, void* out, long long ld_out,
                   void* stream) {
    g_detail[0] = 0;
    const int eb = elem_bytes(io_dtype);
    const NormMat mats[] = {{"y", y, ld_y, eb, true, false}, {"z", z, ld_z, eb, true, false},
                            {"out", out, ld_out, eb, true, true}};
    if (norm_before_gate != 0 && norm_before_gate != 1)
        return set_error(SSD_ERR_INVALID_ARG, "norm_before_gate is %d, not 0 or 1", norm_before_gate);
    SSD_CHECK(check_norm(rows, D, groups, io_dtype, SSD_F32, eps, mats, 3, weight, nullptr, -1, -1));
    if (rows == 0) return SSD_OK;
    return launch_gated_norm(rows, D, groups, io_dtype, norm_before_gate, y, ld_y, z, ld_z, weight, eps, out, ld_out,
                             static_cast<cudaStream_t>(stream));
}

int ssd_gated_norm_backward(long long rows, int D, int groups, int io_dtype, int norm_before_gate, const void* dout,
                            long long ld_dout, const void* y, long long ld_y, const void* z, long long ld_z,
                            const float* weight, float eps, void* dy, long long ld_dy, void* dz, long long ld_dz,
                            float* dweight, void* workspace, size_t workspace_bytes, void* stream) {
    g_detail[0] = 0;
    const int eb = elem_bytes(io_dtype);
    const NormMat mats[] = {{"dout", dout, ld_dout, eb, true, false}, {"y", y, ld_y, eb, true, false},
                            {"z", z, ld_z, eb, true, false},          {"dy", dy, ld_dy, eb, true, true},
                            {"dz", dz, ld_dz, eb, true, true}};
    if (norm_before_gate != 0 && norm_before_gate != 1)
        return set_error(SSD_ERR_INVALID_ARG, "norm_before_gate is %d, not 0 or 1", norm_before_gate);
    SSD_CHECK(check_norm(rows, D, groups, io_dtype, SSD_F32, eps, mats, 5, weight, dweight, -1, -1));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (rows == 0) {
        if (dweight) SSD_CUDA_TRY(cudaMemsetAsync(dweight, 0, (size_t)D * 4, s));
        return SSD_OK;
    }
    SSD_CHECK(check_norm_workspace(rows, D, groups, mats, 5, weight, dweight, workspace, workspace_bytes));
    return launch_gated_norm_backward(rows, D, groups, io_dtype, norm_before_gate, dout, ld_dout, y, ld_y, z, ld_z,
                                      weight, eps, dy, ld_dy, dz, ld_dz, dweight, workspace, s);
}

}  // extern "C"

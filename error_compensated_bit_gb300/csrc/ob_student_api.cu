// C ABI of the student-training operators: argument checks and launches. The contract is
// in include/ob.h.
#include <atomic>
#include <cmath>

#include "ob_student.h"

using namespace ob;

namespace {

bool dtype_ok(int d) { return d == OB_F32 || d == OB_F16 || d == OB_BF16; }
size_t dtype_bytes(int d) { return d == OB_F32 ? 4 : 2; }

int want(const void* p, size_t align)
{
    if (!p) return OB_EINVAL;
    return reinterpret_cast<uintptr_t>(p) % align ? OB_EALIGN : OB_OK;
}

int may(const void* p, size_t align) { return p ? want(p, align) : OB_OK; }

// Sizes the kernels index: tokens of a row and channels in 31 bits, rows x tokens x channels
// in 62, and the tiles (at least 32 channels by 64 steps, see ob_scan.cu) in 31.
int check_scan_sizes(int64_t B, int64_t T, int64_t D, int dtype)
{
    if (!dtype_ok(dtype) || B < 0 || T < 0 || D < 0) return OB_EINVAL;
    if (T >= (int64_t{1} << 31) - 1024 || D >= (int64_t{1} << 31) - 1024 || B >= (int64_t{1} << 31)) return OB_EINVAL;
    if (B == 0 || D == 0) return OB_OK;
    const double cols = (double)B * ((D + 31) / 32), tiles = cols * ((T + 63) / 64 + 1);
    return tiles < 2147483648.0 ? OB_OK : OB_EINVAL;
}

int check_view(const ob_view* v, size_t align) { return v ? want(v->ptr, align) : OB_EINVAL; }

#define OB_TRY(expr)                     \
    do {                                 \
        const int rc_ = (expr);          \
        if (rc_ != OB_OK) return rc_;    \
    } while (0)

int done(cudaError_t e) { return e == cudaSuccess ? OB_OK : report_cuda(e); }

}  // namespace

cudaError_t ob::current_device(DeviceFacts* facts)
{
    constexpr int kDevices = 64;
    static std::atomic<int> sms[kDevices];     // 0: not asked yet
    int d = 0;
    cudaError_t e = cudaGetDevice(&d);
    if (e != cudaSuccess) return e;
    int n = d < kDevices ? sms[d].load(std::memory_order_relaxed) : 0;
    if (n == 0) {
        e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, d);
        if (e != cudaSuccess) return e;
        if (d < kDevices) sms[d].store(n, std::memory_order_relaxed);
    }
    facts->device = d;
    facts->sms = n;
    return cudaSuccess;
}

extern "C" {

size_t ob_gated_scan_workspace_bytes(int64_t B, int64_t T, int64_t D, int dtype, int backward)
{
    if (check_scan_sizes(B, T, D, dtype) != OB_OK) return 0;
    return scan_workspace_bytes(B, T, D, dtype, backward);
}

int ob_gated_scan_fwd(int64_t B, int64_t T, int64_t D, int dtype, const ob_view* x, const ob_view* r,
                      const ob_view* i, const float* decay, const float* h0, const uint8_t* reset, void* y,
                      float* h_last, float* states, void* ws, void* stream)
{
    OB_TRY(check_scan_sizes(B, T, D, dtype));
    if (B == 0 || D == 0) return OB_OK;
    const size_t al = dtype_bytes(dtype);
    OB_TRY(may(h0, 4));
    OB_TRY(may(h_last, 4));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (T == 0) {
        if (!h_last) return OB_OK;
        const size_t bytes = (size_t)B * D * 4;
        return done(h0 ? cudaMemcpyAsync(h_last, h0, bytes, cudaMemcpyDeviceToDevice, s)
                       : cudaMemsetAsync(h_last, 0, bytes, s));
    }
    OB_TRY(check_view(x, al));
    OB_TRY(check_view(r, al));
    OB_TRY(check_view(i, al));
    OB_TRY(want(decay, 4));
    OB_TRY(want(y, al));
    OB_TRY(may(states, 4));
    OB_TRY(want(ws, 256));
    ScanArgs a{};
    a.B = B, a.T = T, a.D = D, a.dtype = dtype;
    a.x = *x, a.r = *r, a.i = *i;
    a.decay = decay, a.h0 = h0, a.reset = reset;
    a.y = y, a.h_last = h_last, a.states = states, a.ws = ws;
    return done(launch_scan_fwd(a, s));
}

int ob_gated_scan_bwd(int64_t B, int64_t T, int64_t D, int dtype, const ob_view* x, const ob_view* r,
                      const ob_view* i, const float* decay, const uint8_t* reset, const float* states,
                      const ob_view* dy, const float* dh_last, void* dx, void* dr, void* di, float* ddecay,
                      float* dh0, void* ws, void* stream)
{
    OB_TRY(check_scan_sizes(B, T, D, dtype));
    if (D == 0) return OB_OK;
    const size_t al = dtype_bytes(dtype);
    OB_TRY(want(ddecay, 4));
    OB_TRY(may(dh_last, 4));
    OB_TRY(may(dh0, 4));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (B == 0 || T == 0) {
        if (B > 0 && dh0) {
            const size_t bytes = (size_t)B * D * 4;
            const cudaError_t e = dh_last ? cudaMemcpyAsync(dh0, dh_last, bytes, cudaMemcpyDeviceToDevice, s)
                                          : cudaMemsetAsync(dh0, 0, bytes, s);
            if (e != cudaSuccess) return report_cuda(e);
        }
        return done(cudaMemsetAsync(ddecay, 0, (size_t)D * 4, s));
    }
    OB_TRY(check_view(x, al));
    OB_TRY(check_view(r, al));
    OB_TRY(check_view(i, al));
    OB_TRY(want(decay, 4));
    OB_TRY(want(states, 4));
    if (dy) OB_TRY(may(dy->ptr, al));
    OB_TRY(want(dx, al));
    OB_TRY(want(dr, al));
    OB_TRY(want(di, al));
    OB_TRY(want(ws, 256));
    ScanArgs a{};
    a.B = B, a.T = T, a.D = D, a.dtype = dtype;
    a.x = *x, a.r = *r, a.i = *i;
    if (dy) a.dy = *dy;
    a.decay = decay, a.reset = reset, a.states = const_cast<float*>(states);
    a.dh_last = dh_last, a.dx = dx, a.dr = dr, a.di = di, a.ddecay = ddecay, a.dh0 = dh0, a.ws = ws;
    return done(launch_scan_bwd(a, s));
}

int ob_gated_scan_step(int64_t B, int64_t D, int dtype, const void* x, int64_t xs, const void* r, int64_t rs,
                       const void* i, int64_t is, const float* decay, const uint8_t* reset, float* h, void* y,
                       void* stream)
{
    OB_TRY(check_scan_sizes(B, 1, D, dtype));
    if (B == 0 || D == 0) return OB_OK;
    const size_t al = dtype_bytes(dtype);
    OB_TRY(want(x, al));
    OB_TRY(want(r, al));
    OB_TRY(want(i, al));
    OB_TRY(want(decay, 4));
    OB_TRY(want(h, 4));
    OB_TRY(want(y, al));
    ScanStepArgs a{B, D, dtype, x, r, i, xs, rs, is, decay, reset, h, y};
    return done(launch_scan_step(a, static_cast<cudaStream_t>(stream)));
}

int ob_gated_scan_read_status(const void* ws, unsigned* status, void* stream)
{
    if (!status) return OB_EINVAL;
    OB_TRY(want(ws, 256));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaMemcpyAsync(status, ws, sizeof(unsigned), cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    return done(e);
}

int ob_operators_read_status(unsigned* status, void* stream)
{
    if (!status) return OB_EINVAL;
    unsigned scan = 0u, distill = 0u;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = scan_status(&scan, s);
    if (e == cudaSuccess) e = distill_status(&distill, s);
    if (e == cudaSuccess) *status = scan | distill;
    return done(e);
}

int ob_selftest_scan_wait(void* ws, uint64_t limit_ns, void* stream)
{
    OB_TRY(want(ws, 256));
    if (limit_ns < 1 || limit_ns > 2000000000ull) return OB_EINVAL;
    return done(launch_scan_wait(ws, limit_ns, static_cast<cudaStream_t>(stream)));
}

size_t ob_distill_workspace_bytes(int64_t N, int64_t V, int dtype)
{
    if (!dtype_ok(dtype) || N < 0 || V < 1) return 0;
    return distill_workspace_bytes(N, V, dtype);
}

static int check_distill(int64_t N, int64_t V, int64_t K, int dtype, const void* logits, const void* index,
                         int index_bits, const void* top, int top_dtype, const float* top_lse,
                         const float* weight, float temperature)
{
    const size_t al = dtype_bytes(dtype);
    OB_TRY(want(logits, al));
    if (K > 0) {
        OB_TRY(want(index, index_bits / 8));
        OB_TRY(want(top, dtype_bytes(top_dtype)));
    }
    OB_TRY(may(top_lse, 4));
    return may(weight, 4);
}

static int check_distill_sizes(int64_t N, int64_t V, int64_t K, int dtype, int index_bits, int top_dtype,
                               float temperature)
{
    if (!dtype_ok(dtype) || !dtype_ok(top_dtype) || (index_bits != 32 && index_bits != 64)) return OB_EINVAL;
    if (N < 0 || N >= (int64_t{1} << 31) || V < 1 || V >= (int64_t{1} << 31) - 65536) return OB_EINVAL;
    if (K < 0 || K > OB_DISTILL_MAX_K) return OB_EINVAL;
    if (!std::isfinite(temperature) || !(temperature > 0.0f) || !std::isfinite(1.0f / temperature)) return OB_EINVAL;
    return OB_OK;
}

int ob_distill(int64_t N, int64_t V, int64_t K, int dtype, const void* logits, int64_t zs, const void* index,
               int index_bits, const void* top, int top_dtype, const float* top_lse, const float* weight,
               float temperature, float* loss, void* dlogits, int64_t ds, float* stats, void* ws, void* stream)
{
    OB_TRY(check_distill_sizes(N, V, K, dtype, index_bits, top_dtype, temperature));
    if (N == 0) return OB_OK;
    OB_TRY(check_distill(N, V, K, dtype, logits, index, index_bits, top, top_dtype, top_lse, weight, temperature));
    OB_TRY(want(loss, 4));
    OB_TRY(may(dlogits, dtype_bytes(dtype)));
    if (dlogits == logits && N > 1 && ds != zs) return OB_EINVAL;
    if (dlogits && N > 1 && (ds < 0 ? -ds : ds) < V) return OB_EINVAL;
    OB_TRY(may(stats, 16));
    if (dlogits && distill_workspace_bytes(N, V, dtype)) OB_TRY(want(ws, 256));
    DistillArgs a{N, V, (int)K, dtype, index_bits, top_dtype, logits, zs, index, top, top_lse, weight, nullptr,
                  1.0f / temperature, loss, dlogits, ds, stats};
    return done(launch_distill(a, ws, static_cast<cudaStream_t>(stream)));
}

int ob_distill_bwd(int64_t N, int64_t V, int64_t K, int dtype, const void* logits, int64_t zs, const void* index,
                   int index_bits, const void* top, int top_dtype, const float* top_lse, const float* weight,
                   float temperature, const float* stats, const float* dloss, void* dlogits, int64_t ds,
                   void* stream)
{
    OB_TRY(check_distill_sizes(N, V, K, dtype, index_bits, top_dtype, temperature));
    if (N == 0) return OB_OK;
    OB_TRY(check_distill(N, V, K, dtype, logits, index, index_bits, top, top_dtype, top_lse, weight, temperature));
    OB_TRY(want(stats, 16));
    OB_TRY(want(dloss, 4));
    OB_TRY(want(dlogits, dtype_bytes(dtype)));
    if (dlogits == logits && N > 1 && ds != zs) return OB_EINVAL;
    if (N > 1 && (ds < 0 ? -ds : ds) < V) return OB_EINVAL;
    DistillArgs a{N, V, (int)K, dtype, index_bits, top_dtype, logits, zs, index, top, top_lse, weight, dloss,
                  1.0f / temperature, nullptr, dlogits, ds, const_cast<float*>(stats)};
    return done(launch_distill_bwd(a, static_cast<cudaStream_t>(stream)));
}

int ob_selftest_distill_wait(int64_t N, int64_t V, int64_t K, const float* logits, const int64_t* index,
                             const float* top, float* loss, float* dlogits, void* stream)
{
    OB_TRY(check_distill_sizes(N, V, K, OB_F32, 64, OB_F32, 1.0f));
    if (N == 0 || V < 32768 || V > 131072) return OB_EINVAL;
    OB_TRY(check_distill(N, V, K, OB_F32, logits, index, 64, top, OB_F32, nullptr, nullptr, 1.0f));
    OB_TRY(want(loss, 4));
    OB_TRY(want(dlogits, 4));
    DistillArgs a{N, V, (int)K, OB_F32, 64, OB_F32, logits, V, index, top, nullptr, nullptr, nullptr,
                  1.0f, loss, dlogits, V, nullptr};
    return done(launch_distill_late(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

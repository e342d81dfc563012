// Internal launch interface of the student-training operators: between their C ABI
// (ob_student_api.cu) and their kernels (ob_scan.cu, ob_distill.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/ob.h"

namespace ob {

// Records a CUDA error for ob_last_cuda_error; returns OB_ECUDA (ob_api.cu).
int report_cuda(cudaError_t e);

// Facts of the current device that cost a driver call each, remembered per device.
struct DeviceFacts {
    int device = -1, sms = 0;
};
cudaError_t current_device(DeviceFacts* facts);

// Launches by launch() a kernel whose dynamic shared memory needs an opt-in. The opt-in belongs to the
// kernel in one device's context; it is made for the largest size the kernel is launched with
// (`most`) at its first launch on a device, and once more should a launch say that it is missing (the
// context was reset).
template <auto kKernel, typename F>
cudaError_t with_opt_in(int device, size_t most, F&& launch)
{
    static std::atomic<uint64_t> done{0};
    const uint64_t bit = uint64_t{1} << (device & 63);
    if (!(done.load(std::memory_order_relaxed) & bit) || device > 63) {
        const cudaError_t e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
        if (e != cudaSuccess) return e;
        done.fetch_or(bit, std::memory_order_relaxed);
    }
    cudaError_t e = launch();
    if (e == cudaErrorInvalidValue) {
        cudaGetLastError();
        e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
        if (e == cudaSuccess) e = launch();
    }
    return e;
}

// Synchronizes the stream; the value of a status word of the current device, which is cleared.
template <typename Word>
cudaError_t take_status(const Word& word, unsigned* status, cudaStream_t s)
{
    static const unsigned zero = 0u;
    cudaError_t e = cudaMemcpyFromSymbolAsync(status, word, sizeof(unsigned), 0, cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess || *status == 0u) return e;
    e = cudaMemcpyToSymbolAsync(word, &zero, sizeof(unsigned), 0, cudaMemcpyHostToDevice, s);
    return e != cudaSuccess ? e : cudaStreamSynchronize(s);
}

struct ScanArgs {
    int64_t B, T, D;
    int dtype;
    ob_view x, r, i, dy;          // dy.ptr null: zero (backward)
    const float* decay;           // [D]
    const float* h0;              // [B][D] or null (forward)
    const uint8_t* reset;         // [B][T] or null
    void* y;                      // [B][T][D] (forward)
    float* h_last;                // [B][D] or null (forward)
    float* states;                // [B][ceil(T/64)][D]; forward writes (or null), backward reads
    const float* dh_last;         // [B][D] or null (backward)
    void *dx, *dr, *di;           // [B][T][D] (backward)
    float* ddecay;                // [D] (backward)
    float* dh0;                   // [B][D] or null (backward)
    void* ws;
};

struct ScanStepArgs {
    int64_t B, D;
    int dtype;
    const void *x, *r, *i;
    int64_t xs, rs, is;           // row strides
    const float* decay;
    const uint8_t* reset;         // [B] or null
    float* h;
    void* y;
};

struct DistillArgs {
    int64_t N, V;
    int K, dtype, index_bits, top_dtype;
    const void* logits;
    int64_t zs;                   // row stride of logits
    const void* index;
    const void* top;
    const float* top_lse;         // [N] or null
    const float* weight;          // [N] or null
    const float* dloss;           // [N] or null (1): the backward pass's upstream gradient
    float inv_tau;
    float* loss;                  // [N]
    void* dlogits;                // [N][V] or null
    int64_t ds;                   // row stride of dlogits
    float* stats;                 // [N][4] or null: RowGrad in ob_distill.cu (inv 0: no loss)
};

size_t scan_workspace_bytes(int64_t B, int64_t T, int64_t D, int dtype, int backward);
cudaError_t launch_scan_fwd(const ScanArgs& a, cudaStream_t s);
cudaError_t launch_scan_bwd(const ScanArgs& a, cudaStream_t s);
cudaError_t launch_scan_step(const ScanStepArgs& a, cudaStream_t s);
cudaError_t launch_scan_wait(void* ws, uint64_t limit_ns, cudaStream_t s);     // a wait that runs out, for tests
cudaError_t scan_status(unsigned* status, cudaStream_t s);

size_t distill_workspace_bytes(int64_t N, int64_t V, int dtype);
cudaError_t launch_distill(const DistillArgs& a, void* ws, cudaStream_t s);
cudaError_t launch_distill_bwd(const DistillArgs& a, cudaStream_t s);
// Loss and gradient (float32) with one block of each cluster late, for tests.
cudaError_t launch_distill_late(const DistillArgs& a, cudaStream_t s);
cudaError_t distill_status(unsigned* status, cudaStream_t s);

}  // namespace ob

// What a plan keeps in device memory, from the host.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>

namespace psm {

// Copy to device memory of the current device, there when the call returns.  By a stream of its
// own: cudaMemset and cudaMemcpy go by the legacy default stream, behind what a
// program has queued there, they return before the device has the bytes, and a run on
// a non-blocking stream would not wait for them.
inline bool upload(void* to, const void* from, size_t bytes) {
    cudaStream_t s = nullptr;
    bool ok = cudaStreamCreateWithFlags(&s, cudaStreamNonBlocking) == cudaSuccess;
    if (ok) {
        ok = cudaMemcpyAsync(to, from, bytes, cudaMemcpyHostToDevice, s) == cudaSuccess;
        ok = cudaStreamSynchronize(s) == cudaSuccess && ok;
        cudaStreamDestroy(s);
    }
    if (!ok) cudaGetLastError();
    return ok;
}

}  // namespace psm

// What the C entry points share: error recording, alignment and device checks.
#pragma once

#include <cstdint>
#include <new>

#include "../../include/tide.h"
#include "tide_internal.h"

#define TIDE_CUDA(call)                                          \
    do {                                                         \
        cudaError_t e_ = (call);                                 \
        if (e_ != cudaSuccess) return tide::record_cuda_error(e_); \
    } while (0)

namespace tide {

// bytes: a power of two
inline bool aligned(const void* p, size_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

inline int check_device(int want) {
    int dev = -1;
    TIDE_CUDA(cudaGetDevice(&dev));
    return dev == want ? TIDE_OK : TIDE_EINVAL;
}

// What a synchronous call uploaded has arrived.  A memset, or a copy from pageable memory that has been staged, may
// return before, and streams made with cudaStreamNonBlocking are not ordered behind the stream that it is on.
inline cudaError_t wait_for_uploads() { return cudaStreamSynchronize(cudaStreamLegacy); }

// Pointer tables of a ring are shared with later calls, so work that reads one is not put into a graph.
inline int check_not_captured(cudaStream_t stream) {
    cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
    TIDE_CUDA(cudaStreamIsCapturing(stream, &status));
    return status == cudaStreamCaptureStatusNone ? TIDE_OK : TIDE_EINVAL;
}

// Entry points return a status, never an exception: an allocation that fails (host vectors of the
// pointer tables and plans) becomes TIDE_ENOMEM, anything else thrown (a mutex error) TIDE_EINVAL.
template <class F>
int no_throw(F&& f) {
    try {
        return f();
    } catch (const std::bad_alloc&) {
        return TIDE_ENOMEM;
    } catch (...) {
        return TIDE_EINVAL;
    }
}

}  // namespace tide

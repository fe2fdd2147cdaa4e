// Identity of the current CUDA context, for caches of device addresses that
// belong to one context (the device image of this library is loaded once per
// context: destroying a device's primary context with cudaDeviceReset unloads
// it, and the next context may place its variables elsewhere).
#pragma once

#include <cuda_runtime.h>

namespace mate {

// While it lives, runtime calls of this thread that a global-mode stream capture
// forbids (a memory call, a first symbol lookup) neither fail nor end the capture.
// They enqueue nothing here, so leaving them out of the graph is right.
struct CaptureRelaxed {
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    CaptureRelaxed() { cudaThreadExchangeStreamCaptureMode(&mode); }
    ~CaptureRelaxed() { cudaThreadExchangeStreamCaptureMode(&mode); }
    CaptureRelaxed(const CaptureRelaxed &) = delete;
    CaptureRelaxed &operator=(const CaptureRelaxed &) = delete;
};

// Unique id of the calling thread's current context (cuCtxGetId, reached
// through the runtime's driver entry points). Returns 0 if it cannot be read;
// callers then fall back to keying their cache by device only.
unsigned long long current_context_id();

}  // namespace mate

// gdn_host.cuh -- host-side services shared by the C entry points: the per-device
// status word, the per-launch event timing and small helpers.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace gdn {

// The current device's status word (nullptr on failure).
unsigned *status_ptr();

// While timing is enabled, brackets the launches made during its lifetime by two
// events on the launch stream.
struct TimedLaunch {
    const char *name;
    cudaStream_t st;
    cudaEvent_t a = nullptr;
    TimedLaunch(const char *n, cudaStream_t s);
    ~TimedLaunch();
};

inline size_t align_up(size_t x, size_t a = 256) { return (x + a - 1) / a * a; }

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

// Streaming multiprocessors of the current device.
inline int sm_count() {
    int sms = 148, dev = 0, v = 0;
    if (cudaGetDevice(&dev) == cudaSuccess &&
        cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess && v > 0)
        sms = v;
    return sms;
}

}  // namespace gdn

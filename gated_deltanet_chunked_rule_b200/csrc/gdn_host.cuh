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

// Launches a kernel; `follows`: the launch before it on the stream is a kernel of the same call, and
// this one calls wait_for_previous before it reads what that one wrote, or writes what it reads. It
// may then come up while that one ends.
template <typename... Want, typename... Have>
cudaError_t launch(bool follows, void (*kernel)(Want...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, Have &&...args) {
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = grid, c.blockDim = block, c.dynamicSmemBytes = smem, c.stream = stream;
    c.attrs = &early, c.numAttrs = follows ? 1 : 0;
    return cudaLaunchKernelEx(&c, kernel, static_cast<Want>(args)...);
}

}  // namespace gdn

// Host-side helpers shared by the C ABI's translation units (defined in kda_api.cu).
#pragma once
#include <cstddef>
#include <cstdint>

#include "kda_internal.cuh"
#include "kda_per_device.h"

namespace kda {

// Record a CUDA failure for kda_last_cuda_error, clear the runtime's (non-sticky) last
// error, pass `status` on.
int cuda_fail(int status, cudaError_t e);

// The current device, its error word and its SM count; KDA_ERR_ARCH if it is not a
// compute capability 10.3 GPU.  Set up once per device.
int device_setup(int* dev_out, int** err_out, int* sms_out = nullptr);

// Tensor map of `rows` rows of `inner` 16-bit elements, `pitch` elements apart, for boxes of 64
// elements x `box_rows` rows in the 128-byte swizzle.
cudaError_t encode_rows_map(CUtensorMap* map, const void* base, long long inner, long long rows,
                            long long pitch, int box_rows);

// Records the launches between its construction and its destruction, with their device
// time, under a kernel id (kda_profile_*); nothing while recording is off.
class LaunchTimer {
public:
    LaunchTimer(int kernel, cudaStream_t s);
    ~LaunchTimer();
    LaunchTimer(const LaunchTimer&) = delete;
    LaunchTimer& operator=(const LaunchTimer&) = delete;

private:
    int kernel_;
    cudaStream_t stream_;
    cudaEvent_t start_ = nullptr, stop_ = nullptr;
};

template <class F>
cudaError_t timed_launch(int kernel, cudaStream_t s, F&& launch) {
    LaunchTimer timer(kernel, s);
    return launch();
}

constexpr size_t kAlign = 256;
inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

inline bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
    if (!a || !b || na == 0 || nb == 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

// Sets an attribute of a kernel on the current device, the first time that it is used there.
template <auto Kernel, cudaFuncAttribute Attribute>
cudaError_t set_once(int value) {
    static OncePerDevice once;
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDeviceIndex) return cudaErrorInvalidDevice;
    return once(dev, [&] { return cudaFuncSetAttribute(Kernel, Attribute, value); });
}
// Lets a kernel use more than 48 KB of dynamic shared memory
template <auto Kernel>
cudaError_t allow_smem(size_t bytes) {
    return set_once<Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize>((int)bytes);
}
// Lets a kernel run in clusters of more than 8 CTAs
template <auto Kernel>
cudaError_t allow_large_clusters() {
    return set_once<Kernel, cudaFuncAttributeNonPortableClusterSizeAllowed>(1);
}

inline bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

}  // namespace kda

// lp_host.h -- small host helpers shared by the C-ABI translation units.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace lp {

constexpr size_t kAlign = 256;
constexpr int64_t kDefaultTimeoutNs = 1000000000LL;  // 1 s

inline size_t align_up(size_t v) { return (v + kAlign - 1) & ~(kAlign - 1); }
inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

// Records e for lp_last_cuda_error and returns LP_ECUDA.
int cuda_fail(cudaError_t e);

// Makes the plan's device current for the scope; restores the caller's.
struct DeviceGuard {
    int prev = -1;
    bool ok = true;
    explicit DeviceGuard(int dev) {
        if (cudaGetDevice(&prev) != cudaSuccess) {
            ok = false;
            return;
        }
        if (prev != dev && cudaSetDevice(dev) != cudaSuccess) ok = false;
    }
    ~DeviceGuard() {
        int cur = -1;
        if (prev >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev) cudaSetDevice(prev);
    }
};

}  // namespace lp

// Host code that the entry points of several operators share: device checks,
// validation of sizes, strides and addresses, launches.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>
#include <cstring>
#include <initializer_list>

#include "gemm_f16_nt.h"

namespace g16 {
namespace host {

constexpr int kMaxDevices = 64;
inline std::atomic<int> g_cus[kMaxDevices];   // compute units; 0 unknown, -1 not gfx950

inline int device_cus(int* cus)
{
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return GEMM_F16_NT_DEVICE;
    int n = g_cus[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        hipDeviceProp_t prop;
        n = -1;
        if (hipGetDeviceProperties(&prop, dev) == hipSuccess && std::strncmp(prop.gcnArchName, "gfx950", 6) == 0 &&
            prop.multiProcessorCount > 0)
            n = prop.multiProcessorCount;
        g_cus[dev].store(n, std::memory_order_relaxed);   // threads that ask at once store the same
    }
    if (n < 0) return GEMM_F16_NT_DEVICE;
    *cus = n;
    return GEMM_F16_NT_OK;
}

constexpr int64_t kMaxStride = int64_t(1) << 40;      // elements; keeps every offset inside 63 bits

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline bool overlaps(const void* a, int64_t abytes, const void* b, int64_t bbytes)
{
    if (abytes <= 0 || bbytes <= 0) return false;
    const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
    return a0 < b0 + (uintptr_t)bbytes && b0 < a0 + (uintptr_t)abytes;
}

struct Axis {
    int64_t n, stride;
};

// Bytes from a tensor's first to its last element; 0 if it has none, -1 for
// a bad stride.
inline int64_t extent(int64_t d, std::initializer_list<Axis> axes)
{
    __int128 last = d - 1;
    for (const Axis& a : axes) {
        if (a.n == 0) return 0;
        if (a.stride < 0 || a.stride > kMaxStride) return -1;
        last += (__int128)(a.n - 1) * a.stride;
    }
    const __int128 bytes = 2 * (last + 1);
    return bytes < ((__int128)1 << 60) ? (int64_t)bytes : -1;
}

inline bool aligned16(const void* p, std::initializer_list<int64_t> strides)
{
    uint64_t all = (uintptr_t)p >> 1 | ((uintptr_t)p & 1);
    for (int64_t s : strides) all |= (uint64_t)s;
    return (all & 7) == 0;
}

inline int launch(const void* f, int64_t wgs, int threads, const void* args, hipStream_t s)
{
    void* a[] = {const_cast<void*>(args)};
    return hipLaunchKernel(f, dim3((unsigned)wgs), dim3(threads), a, 0, s) == hipSuccess ? GEMM_F16_NT_OK : GEMM_F16_NT_LAUNCH;
}

inline int check_workspace(const void* ws, int64_t have, int64_t need)
{
    if (need == 0) return GEMM_F16_NT_OK;
    if (ws == nullptr || have < need) return GEMM_F16_NT_INVALID_ARG;
    return ((uintptr_t)ws & 15) != 0 ? GEMM_F16_NT_UNSUPPORTED : GEMM_F16_NT_OK;
}

}  // namespace host
}  // namespace g16

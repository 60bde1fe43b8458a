// host.hpp -- host-side helpers of the layer operators' C entry points: error
// codes, the device check, argument checks and launches.
#pragma once

#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <atomic>

#include "gemm_rs_layer.h"

namespace gemm_rs_layer {

inline thread_local char g_hip_msg[256] = "";

inline int hip_fail(hipError_t e, const char* what)
{
    snprintf(g_hip_msg, sizeof g_hip_msg, "%s: %s", what, hipGetErrorString(e));
    return GEMM_RS_ERR_HIP;
}

constexpr int kMaxDevices = 64;

// The current device is a gfx950: looked up once per device.
inline int check_device(int* device = nullptr)
{
    static std::atomic<int> known[kMaxDevices];  // 0: not looked up, 1: gfx950, 2: another
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e == hipErrorNoDevice || e == hipErrorInvalidDevice) return GEMM_RS_ERR_NO_DEVICE;
    if (e != hipSuccess) return hip_fail(e, "hipGetDevice");
    if (dev < 0 || dev >= kMaxDevices) return GEMM_RS_ERR_NO_DEVICE;
    if (device) *device = dev;
    int k = known[dev].load(std::memory_order_relaxed);
    if (k == 0) {
        hipDeviceProp_t p;
        e = hipGetDeviceProperties(&p, dev);
        if (e != hipSuccess) return hip_fail(e, "hipGetDeviceProperties");
        k = strncmp(p.gcnArchName, "gfx950", 6) == 0 ? 1 : 2;
        known[dev].store(k, std::memory_order_relaxed);
    }
    return k == 1 ? GEMM_RS_OK : GEMM_RS_ERR_NO_DEVICE;
}

template <class A>
int launch(void (*kernel)(A), dim3 grid, int threads, const A& args, void* stream, const char* what)
{
    void* p[] = {const_cast<A*>(&args)};
    const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, dim3(threads), p, 0,
                                         static_cast<hipStream_t>(stream));
    return e == hipSuccess ? GEMM_RS_OK : hip_fail(e, what);
}

inline int elem_bytes(int dtype) { return dtype == GEMM_RS_DTYPE_F32 ? 4 : 2; }
inline bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Every buffer of a call: present and aligned to its element.
struct Checker {
    int code = GEMM_RS_OK;
    void need(const void* p, size_t align)
    {
        if (!p) fail(GEMM_RS_ERR_INVALID_ARG);
        else if (!aligned(p, align)) fail(GEMM_RS_ERR_MISALIGNED);
    }
    void maybe(const void* p, size_t align)
    {
        if (p) need(p, align);
    }
    void stride(int64_t s, int64_t width)
    {
        if (s < width || s > (int64_t(1) << 40)) fail(GEMM_RS_ERR_INVALID_ARG);
    }
    void fail(int c)
    {
        if (code == GEMM_RS_OK) code = c;
    }
};

constexpr int64_t kMaxRows = int64_t(1) << 31;
// A launch has fewer than 2^32 threads in its first dimension.
constexpr int64_t kMaxThreads = (int64_t(1) << 32) - 1;
constexpr int kCus = 256;  // compute units of an MI355X

}  // namespace gemm_rs_layer

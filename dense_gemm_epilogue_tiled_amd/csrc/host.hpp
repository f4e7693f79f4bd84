// Host-side helpers shared by the library's translation units: limits, pitch
// and overlap checks, the device check and the kernel launch.
#pragma once

#include <hip/hip_runtime.h>

#include <atomic>
#include <cstdint>
#include <cstring>

#include "../../include/gemm_relu.h"

namespace {

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxSpanBytes = int64_t(1) << 62;
constexpr int64_t kWorkspaceAlign = 256;  // required alignment of a workspace (bytes)

// Number of bytes spanned by a rows x cols matrix with pitch ld (0 if empty);
// -1 when it does not fit the library's limits.
int64_t span_bytes(int64_t rows, int64_t cols, int64_t ld) {
    if (rows == 0 || cols == 0) return 0;
    // (rows - 1) * ld + cols elements, checked against 2^62 bytes.
    const int64_t limit = kMaxSpanBytes / 2;
    if (rows - 1 > 0 && ld > (limit - cols) / (rows - 1)) return -1;
    return ((rows - 1) * ld + cols) * 2;
}

// Bytes spanned by a rows x cols matrix of 1-byte elements with pitch ld.
int64_t span_bytes8(int64_t rows, int64_t cols, int64_t ld) {
    if (rows == 0 || cols == 0) return 0;
    const int64_t limit = kMaxSpanBytes;
    if (rows - 1 > 0 && ld > (limit - cols) / (rows - 1)) return -1;
    return (rows - 1) * ld + cols;
}

bool overlaps(uintptr_t a, int64_t alen, uintptr_t b, int64_t blen) {
    if (alen <= 0 || blen <= 0) return false;
    return a < b + (uintptr_t)blen && b < a + (uintptr_t)alen;
}

// ---- device check (once per device) ------------------------------------------

constexpr int kMaxDevices = 64;
std::atomic<int> g_device_state[kMaxDevices];  // 0 unknown, 1 gfx950, 2 other

int check_device() {
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0) return GR_ERR_NO_DEVICE;
    if (dev >= kMaxDevices) return GR_ERR_UNSUPPORTED_DEVICE;
    int state = g_device_state[dev].load(std::memory_order_acquire);
    if (state == 0) {
        hipDeviceProp_t prop;
        if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return GR_ERR_NO_DEVICE;
        state = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : 2;
        g_device_state[dev].store(state, std::memory_order_release);
    }
    return state == 1 ? GR_OK : GR_ERR_UNSUPPORTED_DEVICE;
}

template <typename... Args>
int launch_lds(void (*kernel)(Args...), dim3 grid, int threads, int dynamic_lds, hipStream_t stream, Args... args) {
    void* argv[] = {static_cast<void*>(&args)...};
    hipError_t e =
        hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, dim3(threads), argv, dynamic_lds, stream);
    return e == hipSuccess ? GR_OK : GR_ERR_LAUNCH;
}

template <typename... Args>
int launch_grid(void (*kernel)(Args...), dim3 grid, int threads, hipStream_t stream, Args... args) {
    return launch_lds(kernel, grid, threads, 0, stream, args...);
}

template <typename... Args>
int launch(void (*kernel)(Args...), int64_t grid, int threads, hipStream_t stream, Args... args) {
    return launch_grid(kernel, dim3((uint32_t)grid), threads, stream, args...);
}

}  // namespace

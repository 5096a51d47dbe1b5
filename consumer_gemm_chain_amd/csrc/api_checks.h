// api_checks.h -- what the C entry points of the operators around the chain
// share: error reports, device selection, limits and argument checks.
#pragma once

#include <hip/hip_runtime.h>

#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include "../../include/mlp_chain.h"
#include "chain_launch.h"

namespace {

int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int fail(int code, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    // an error of the runtime is reported here, not once more by the caller's
    // next look at the thread's last error
    if (code == MLP_EHIP || code == MLP_ENOMEM) (void)hipGetLastError();
    return mlpc_set_error(code, buf);
}

struct DeviceGuard {
    int prev = -1;
    bool ok = true;
    explicit DeviceGuard(int dev) {
        if (hipGetDevice(&prev) != hipSuccess) { ok = false; return; }
        if (prev != dev && hipSetDevice(dev) != hipSuccess) ok = false;
    }
    ~DeviceGuard() {
        int cur = -1;
        if (prev >= 0 && hipGetDevice(&cur) == hipSuccess && cur != prev) (void)hipSetDevice(prev);
    }
};

constexpr int64_t MAX_WIDTH = (int64_t)1 << 22;
constexpr int64_t MAX_ROWS = (int64_t)1 << 24;
// Row strides: offsets are 64-bit (2^24 rows of MAX_LD stay in range), but for
// the products' operands, whose DMA has 32-bit byte offsets within a tile: of up
// to 256 rows, or of 64 rows and all columns (at most 2^23) where the reduction
// runs across rows.
constexpr int64_t MAX_LD = (int64_t)1 << 36;
constexpr int64_t MAX_DMA_LD = (int64_t)1 << 23;

// The largest stride of a product's operand of `rows` rows.
int64_t dma_ld(int64_t rows) {
    const int64_t few = (((int64_t)1 << 31) - ((int64_t)1 << 24)) / (rows < 256 ? rows : 256);
    return few > MAX_DMA_LD ? few : MAX_DMA_LD;
}

size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

bool misaligned(const void* p, unsigned a) { return ((uintptr_t)p & (a - 1)) != 0; }

// A 2-d operand of the linear layer: 16-byte rows of `width` elements, at most `most` apart.
int check_matrix(const char* name, const void* p, int64_t ld, int64_t width, int64_t most) {
    if (!p || misaligned(p, 16)) return fail(MLP_EINVAL, "%s must be a non-NULL 16-byte aligned device pointer", name);
    if (ld < width || ld % 8 || ld > most)
        return fail(MLP_EINVAL, "the row stride of %s must be a multiple of 8 in %lld..%lld elements, got %lld", name,
                    (long long)width, (long long)most, (long long)ld);
    return MLP_OK;
}

int check_rows_count(int64_t rows, int64_t most) {
    if (rows < 0 || rows > most)
        return fail(MLP_EINVAL, "rows must be in 0..%lld, got %lld", (long long)most, (long long)rows);
    return MLP_OK;
}

int check_dtype(int dtype) {
    if (dtype != MLP_DTYPE_F16 && dtype != MLP_DTYPE_BF16) return fail(MLP_EINVAL, "unknown dtype %d", dtype);
    return MLP_OK;
}

int current_device(int* dev) {
    const hipError_t e = hipGetDevice(dev);
    return e == hipSuccess ? MLP_OK : fail(MLP_EHIP, "no HIP device: %s", hipGetErrorString(e));
}

int launched(hipError_t e) {
    return e == hipSuccess ? MLP_OK : fail(MLP_EHIP, "kernel launch failed: %s", hipGetErrorString(e));
}

// Wait for the last call that used the workspace, if there is one, and release it.
int release(int device, hipStream_t last, void* ws) {
    if (!ws) return MLP_OK;
    DeviceGuard g(device);
    const hipError_t e1 = hipStreamSynchronize(last);
    const hipError_t e2 = hipFree(ws);
    if (e1 != hipSuccess || e2 != hipSuccess)
        return fail(MLP_EHIP, "destroy: %s", hipGetErrorString(e1 != hipSuccess ? e1 : e2));
    return MLP_OK;
}

}  // namespace

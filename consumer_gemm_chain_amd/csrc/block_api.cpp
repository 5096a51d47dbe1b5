// block_api.cpp -- the C ABI declared in include/mlp_block.h: argument
// checks, workspace ownership and launches.
#include <hip/hip_runtime.h>

#include <math.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include <new>

#include "../../include/mlp_block.h"
#include "block_launch.h"
#include "chain_launch.h"

struct mlp_norm {
    int H;
    int dtype;
    int device;
    float eps;
    float* part;                // [max parts][2][H]
    hipStream_t last_stream;
};

struct mlp_linear {
    int64_t max_rows;
    int K, N, gN;
    int act, dtype, device;
    void* ws;                   // dz [max_rows, gN] (activations only) | column-sum partials
    uint16_t* dz;
    float* part;                // [max parts][gN]
    hipStream_t last_stream;
};

namespace {

int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int fail(int code, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
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

size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

bool misaligned(const void* p, unsigned a) { return ((uintptr_t)p & (a - 1)) != 0; }

// A 2-d operand of the norm: rows of H elements `ld` apart.
int check_rows(const char* name, const void* p, int64_t ld, int64_t H) {
    if (!p || misaligned(p, 2)) return fail(MLP_EINVAL, "%s must be a non-NULL 2-byte aligned device pointer", name);
    if (ld < H || ld > MAX_WIDTH * 4)
        return fail(MLP_EINVAL, "the row stride of %s must be in %lld..%lld elements, got %lld", name, (long long)H,
                    (long long)(MAX_WIDTH * 4), (long long)ld);
    return MLP_OK;
}

// A 2-d operand of the linear layer: 16-byte rows of `width` elements.
int check_matrix(const char* name, const void* p, int64_t ld, int64_t width) {
    if (!p || misaligned(p, 16)) return fail(MLP_EINVAL, "%s must be a non-NULL 16-byte aligned device pointer", name);
    if (ld < width || ld % 8 || ld > MAX_WIDTH * 2)
        return fail(MLP_EINVAL, "the row stride of %s must be a multiple of 8 in %lld..%lld elements, got %lld", name,
                    (long long)width, (long long)(MAX_WIDTH * 2), (long long)ld);
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

// Wait for the handle's last call and release its workspace.
int release(int device, hipStream_t last, void* ws) {
    DeviceGuard g(device);
    const hipError_t e1 = hipStreamSynchronize(last);
    const hipError_t e2 = ws ? hipFree(ws) : hipSuccess;
    if (e1 != hipSuccess || e2 != hipSuccess)
        return fail(MLP_EHIP, "destroy: %s", hipGetErrorString(e1 != hipSuccess ? e1 : e2));
    return MLP_OK;
}

}  // namespace

extern "C" {

mlp_norm_t mlp_norm_create(int64_t H, int dtype, float eps) {
    if (H < 1 || H > MAX_WIDTH) {
        fail(MLP_EINVAL, "H must be in 1..%lld, got %lld", (long long)MAX_WIDTH, (long long)H);
        return nullptr;
    }
    if (check_dtype(dtype) != MLP_OK) return nullptr;
    if (!(eps >= 0.f) || isinf(eps)) {
        fail(MLP_EINVAL, "eps must be finite and not negative, got %g", (double)eps);
        return nullptr;
    }
    int dev = 0;
    if (current_device(&dev) != MLP_OK) return nullptr;
    mlp_norm* h = new (std::nothrow) mlp_norm();
    if (!h) {
        fail(MLP_ENOMEM, "out of host memory");
        return nullptr;
    }
    h->H = (int)H;
    h->dtype = dtype;
    h->device = dev;
    h->eps = eps;
    const size_t bytes = (size_t)mlpc_norm_max_parts() * 2 * H * sizeof(float);
    const hipError_t e = hipMalloc(reinterpret_cast<void**>(&h->part), bytes);
    if (e != hipSuccess) {
        fail(MLP_ENOMEM, "hipMalloc of %zu workspace bytes failed: %s", bytes, hipGetErrorString(e));
        delete h;
        return nullptr;
    }
    return h;
}

int mlp_norm_forward(mlp_norm_t h, int64_t rows, const void* x, int64_t ldx, const void* weight, const void* bias,
                     void* y, int64_t ldy, float* mean, float* rstd, void* hip_stream) {
    if (!h) return fail(MLP_EINVAL, "NULL handle");
    int rc = check_rows_count(rows, MAX_ROWS);
    if (rc != MLP_OK || rows == 0) return rc;
    rc = check_rows("x", x, ldx, h->H);
    if (rc == MLP_OK) rc = check_rows("y", y, ldy, h->H);
    if (rc != MLP_OK) return rc;
    if (misaligned(weight, 2) || misaligned(bias, 2) || misaligned(mean, 4) || misaligned(rstd, 4))
        return fail(MLP_EINVAL, "weight and bias must be 2-byte aligned, mean and rstd 4-byte aligned");
    DeviceGuard g(h->device);
    if (!g.ok) return fail(MLP_EHIP, "cannot select the handle's device %d", h->device);
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    h->last_stream = s;
    mlpc::NormArgs a{};
    a.x = static_cast<const uint16_t*>(x);
    a.weight = static_cast<const uint16_t*>(weight);
    a.bias = static_cast<const uint16_t*>(bias);
    a.y = static_cast<uint16_t*>(y);
    a.mean = mean;
    a.rstd = rstd;
    a.rows = rows;
    a.ldx = ldx;
    a.ldy = ldy;
    a.H = h->H;
    a.eps = h->eps;
    return launched(mlpc_norm_forward(a, h->dtype, s));
}

int mlp_norm_backward(mlp_norm_t h, int64_t rows, const void* dy, int64_t lddy, const void* x, int64_t ldx,
                      const void* weight, const float* mean, const float* rstd, const void* dres, int64_t lddres,
                      void* dx, int64_t lddx, void* dweight, void* dbias, void* hip_stream) {
    if (!h) return fail(MLP_EINVAL, "NULL handle");
    int rc = check_rows_count(rows, MAX_ROWS);
    const bool any = rc == MLP_OK && rows > 0;
    if (any) rc = check_rows("dy", dy, lddy, h->H);
    if (any && rc == MLP_OK) rc = check_rows("x", x, ldx, h->H);
    if (any && rc == MLP_OK) rc = check_rows("dx", dx, lddx, h->H);
    if (any && rc == MLP_OK && dres) rc = check_rows("dres", dres, lddres, h->H);
    if (rc != MLP_OK) return rc;
    if (any && (!mean || !rstd || misaligned(mean, 4) || misaligned(rstd, 4)))
        return fail(MLP_EINVAL, "mean and rstd must be non-NULL 4-byte aligned device pointers");
    if (misaligned(weight, 2) || misaligned(dweight, 2) || misaligned(dbias, 2))
        return fail(MLP_EINVAL, "weight, dweight and dbias must be 2-byte aligned");
    if (any && dres == dx && lddres != lddx) return fail(MLP_EINVAL, "dx in dres's buffer needs dres's row stride");
    DeviceGuard g(h->device);
    if (!g.ok) return fail(MLP_EHIP, "cannot select the handle's device %d", h->device);
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    h->last_stream = s;
    if (rows == 0 && !dweight && !dbias) return MLP_OK;
    mlpc::NormArgs a{};
    a.x = static_cast<const uint16_t*>(x);
    a.weight = static_cast<const uint16_t*>(weight);
    a.dy = static_cast<const uint16_t*>(dy);
    a.dres = static_cast<const uint16_t*>(dres);
    a.dx = static_cast<uint16_t*>(dx);
    a.mean = const_cast<float*>(mean);
    a.rstd = const_cast<float*>(rstd);
    a.dweight = static_cast<uint16_t*>(dweight);
    a.dbias = static_cast<uint16_t*>(dbias);
    a.part = h->part;
    a.rows = rows;
    a.ldx = ldx;
    a.lddy = lddy;
    a.lddres = lddres;
    a.lddx = lddx;
    a.H = h->H;
    a.parts = mlpc_norm_parts(rows);
    return launched(mlpc_norm_backward(a, h->dtype, s));
}

int mlp_norm_destroy(mlp_norm_t h) {
    if (!h) return MLP_OK;
    const int rc = release(h->device, h->last_stream, h->part);
    delete h;
    return rc;
}

mlp_linear_t mlp_linear_create(int64_t max_rows, int64_t K, int64_t N, int act, int dtype) {
    if (max_rows < 1 || max_rows > MAX_ROWS || K < 8 || N < 8 || K >= MAX_WIDTH || N >= MAX_WIDTH) {
        fail(MLP_EINVAL, "sizes must be max_rows in 1..%lld, K and N in 8..%lld (got max_rows=%lld K=%lld N=%lld)",
             (long long)MAX_ROWS, (long long)(MAX_WIDTH - 8), (long long)max_rows, (long long)K, (long long)N);
        return nullptr;
    }
    if (K % 8 != 0 || N % 8 != 0) {
        fail(MLP_EINVAL, "K and N must be multiples of 8 (16-byte rows), got K=%lld N=%lld", (long long)K, (long long)N);
        return nullptr;
    }
    if (act < MLP_ACT_NONE || act > MLP_ACT_SWIGLU) {
        fail(MLP_EINVAL, "unknown activation %d", act);
        return nullptr;
    }
    if (check_dtype(dtype) != MLP_OK) return nullptr;
    int dev = 0;
    if (current_device(&dev) != MLP_OK) return nullptr;
    mlp_linear* h = new (std::nothrow) mlp_linear();
    if (!h) {
        fail(MLP_ENOMEM, "out of host memory");
        return nullptr;
    }
    h->max_rows = max_rows;
    h->K = (int)K;
    h->N = (int)N;
    h->gN = (int)(act == MLP_ACT_SWIGLU ? 2 * N : N);
    h->act = act;
    h->dtype = dtype;
    h->device = dev;
    const size_t dz_b = act == MLP_ACT_NONE ? 0 : align_up((size_t)max_rows * h->gN * 2, 256);
    const size_t part_b = align_up((size_t)mlpc_dz_max_parts() * h->gN * sizeof(float), 256);
    const hipError_t e = hipMalloc(&h->ws, dz_b + part_b);
    if (e != hipSuccess) {
        fail(MLP_ENOMEM, "hipMalloc of %zu workspace bytes failed: %s", dz_b + part_b, hipGetErrorString(e));
        delete h;
        return nullptr;
    }
    char* p = static_cast<char*>(h->ws);
    h->dz = dz_b ? reinterpret_cast<uint16_t*>(p) : nullptr;
    h->part = reinterpret_cast<float*>(p + dz_b);
    return h;
}

int mlp_linear_forward(mlp_linear_t h, int64_t rows, const void* x, int64_t ldx, const void* w, int64_t ldw,
                       const void* bias, const void* residual, int64_t ldres, void* y, int64_t ldy, void* z,
                       int64_t ldz, void* hip_stream) {
    if (!h) return fail(MLP_EINVAL, "NULL handle");
    int rc = check_rows_count(rows, h->max_rows);
    if (rc != MLP_OK || rows == 0) return rc;
    rc = check_matrix("x", x, ldx, h->K);
    if (rc == MLP_OK) rc = check_matrix("w", w, ldw, h->gN);
    if (rc == MLP_OK) rc = check_matrix("y", y, ldy, h->N);
    if (rc == MLP_OK && residual) rc = check_matrix("residual", residual, ldres, h->N);
    if (rc == MLP_OK && z) rc = check_matrix("z", z, ldz, h->gN);
    if (rc != MLP_OK) return rc;
    if (misaligned(bias, 16)) return fail(MLP_EINVAL, "bias must be 16-byte aligned");
    if (residual == y && ldres != ldy) return fail(MLP_EINVAL, "y in the residual's buffer needs its row stride");
    DeviceGuard g(h->device);
    if (!g.ok) return fail(MLP_EHIP, "cannot select the handle's device %d", h->device);
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    h->last_stream = s;
    mlpc::GemmArgs a{};
    a.a = static_cast<const uint16_t*>(x);
    a.b = static_cast<const uint16_t*>(w);
    a.d = static_cast<uint16_t*>(y);
    a.lda = ldx;
    a.ldb = ldw;
    a.ldd = ldy;
    a.M = (int)rows;
    a.N = h->N;
    a.K = h->K;
    a.up = h->gN - h->N;
    a.act = h->act;
    a.bias = static_cast<const uint16_t*>(bias);
    a.res = static_cast<const uint16_t*>(residual);
    a.z = static_cast<uint16_t*>(z);
    a.ldr = ldres;
    a.ldz = ldz;
    return launched(mlpc_gemm(a, mlpc::PASS_FWD, h->dtype, s));
}

int mlp_linear_backward(mlp_linear_t h, int64_t rows, const void* dy, int64_t lddy, const void* x, int64_t ldx,
                        const void* w, int64_t ldw, const void* z, int64_t ldz, void* dx, int64_t lddx, void* dw,
                        int64_t lddw, void* db, void* hip_stream) {
    if (!h) return fail(MLP_EINVAL, "NULL handle");
    const bool act = h->act != MLP_ACT_NONE;
    int rc = check_rows_count(rows, h->max_rows);
    const bool any = rc == MLP_OK && rows > 0;
    if (any) rc = check_matrix("dy", dy, lddy, h->N);
    if (any && rc == MLP_OK && act) rc = check_matrix("z", z, ldz, h->gN);
    if (any && rc == MLP_OK && dx) rc = check_matrix("dx", dx, lddx, h->K);
    if (any && rc == MLP_OK && dx) rc = check_matrix("w", w, ldw, h->gN);
    if (any && rc == MLP_OK && dw) rc = check_matrix("x", x, ldx, h->K);
    if (rc == MLP_OK && dw) rc = check_matrix("dw", dw, lddw, h->gN);
    if (rc != MLP_OK) return rc;
    if (misaligned(db, 16)) return fail(MLP_EINVAL, "db must be 16-byte aligned");
    DeviceGuard g(h->device);
    if (!g.ok) return fail(MLP_EHIP, "cannot select the handle's device %d", h->device);
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    h->last_stream = s;
    const uint16_t* dz = static_cast<const uint16_t*>(dy);
    int64_t lddz = lddy;
    if (db || (act && (dx || dw) && rows > 0)) {
        mlpc::DzArgs d{};
        d.dy = dz;
        d.z = static_cast<const uint16_t*>(z);
        d.dz = h->dz;
        d.db = static_cast<uint16_t*>(db);
        d.part = h->part;
        d.lddy = lddy;
        d.ldz = ldz;
        d.lddz = h->gN;
        d.rows = rows;
        d.N = h->N;
        d.act = h->act;
        d.parts = mlpc_dz_parts(rows);
        rc = launched(mlpc_dz(d, h->dtype, s));
        if (rc != MLP_OK) return rc;
    }
    if (act) {
        dz = h->dz;
        lddz = h->gN;
    }
    if (dx && rows > 0) {
        mlpc::GemmArgs a{};
        a.a = dz;
        a.b = static_cast<const uint16_t*>(w);
        a.d = static_cast<uint16_t*>(dx);
        a.lda = lddz;
        a.ldb = ldw;
        a.ldd = lddx;
        a.M = (int)rows;
        a.N = h->K;
        a.K = h->gN;
        rc = launched(mlpc_gemm(a, mlpc::PASS_DX, h->dtype, s));
        if (rc != MLP_OK) return rc;
    }
    if (dw) {
        mlpc::GemmArgs a{};
        a.a = static_cast<const uint16_t*>(x);
        a.b = dz;
        a.d = static_cast<uint16_t*>(dw);
        a.lda = ldx;
        a.ldb = lddz;
        a.ldd = lddw;
        a.M = h->K;
        a.N = h->gN;
        a.K = (int)rows;
        return launched(mlpc_gemm(a, mlpc::PASS_DW, h->dtype, s));
    }
    return MLP_OK;
}

int mlp_linear_destroy(mlp_linear_t h) {
    if (!h) return MLP_OK;
    const int rc = release(h->device, h->last_stream, h->ws);
    delete h;
    return rc;
}

}  // extern "C"

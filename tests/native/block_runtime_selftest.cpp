// Drives the block operators' handles (block_api.cpp) on a stand-in for the
// HIP runtime and the launchers, defined here: no GPU and no HIP library are
// needed, and every runtime call of an entry point can be seen and made to
// fail.  Prints "<n> failures" and exits 0 on success.
#include <stdio.h>
#include <string.h>

#include <vector>

#include "../../include/mlp_block.h"
#include "../../consumer_gemm_chain_amd/csrc/block_launch.h"
#include "../../consumer_gemm_chain_amd/csrc/linear_configs.h"

static int failures = 0;
static char last[512];
#define CHECK(c) do { if (!(c)) { ++failures; printf("line %d: %s (%s)\n", __LINE__, #c, last); } } while (0)

int mlpc_set_error(int code, const char* msg) {
    snprintf(last, sizeof last, "%s", msg);
    return code;
}

// ---------------------------------------------------------------- the runtime

static hipError_t pending = hipSuccess;             // the thread's last error
static hipError_t malloc_fails = hipSuccess, memset_fails = hipSuccess, sync_fails = hipSuccess, launch_fails = hipSuccess;
static std::vector<hipStream_t> waited;             // streams waited for
static int blocks = 0;                              // allocations alive

static hipError_t done(hipError_t e) {
    if (e != hipSuccess) pending = e;
    return e;
}

extern "C" {
hipError_t hipGetDevice(int* d) { *d = 0; return hipSuccess; }
hipError_t hipSetDevice(int) { return hipSuccess; }
hipError_t hipDeviceGetAttribute(int* v, hipDeviceAttribute_t, int) { *v = 256; return hipSuccess; }
hipError_t hipMalloc(void** p, size_t) {
    if (malloc_fails != hipSuccess) return done(malloc_fails);
    *p = ::operator new(4096);
    ++blocks;
    return hipSuccess;
}
hipError_t hipFree(void* p) {
    ::operator delete(p);
    --blocks;
    return hipSuccess;
}
hipError_t hipMemset(void*, int, size_t) { return done(memset_fails); }
hipError_t hipStreamSynchronize(hipStream_t s) {
    waited.push_back(s);
    return done(sync_fails);
}
hipError_t hipGetLastError(void) {
    const hipError_t e = pending;
    pending = hipSuccess;
    return e;
}
const char* hipGetErrorString(hipError_t) { return "an error"; }
}

// -------------------------------------------------------------- the launchers

using namespace mlpc;
int mlpc_linear_num_configs() { return MLPC_NUM_LINEAR_CONFIGS; }
LinearCfgInfo mlpc_linear_config(int cfg) {
#define ROW(id, bm, bn, wm, wn, ns, ks, occ) \
    if (cfg == id) return LinearCfgInfo{bm, bn, 64 * wm * wn, ns * (bm + bn) * ks * 2};
    MLPC_LINEAR_CONFIGS(ROW)
    return LinearCfgInfo{};
}
bool mlpc_linear_has(int cfg, int pass) {
    if (pass > PASS_DW) return cfg != 0 && cfg != 7;
    return pass == PASS_DW ? mlpc_linear_config(cfg).BM >= 128 : cfg != 7;
}
hipError_t mlpc_gemm(const GemmArgs&, int, int, int, hipStream_t) { return done(launch_fails); }
hipError_t mlpc_gemm_both(const GemmArgs&, const GemmArgs&, const DzArgs&, int, int, hipStream_t) { return done(launch_fails); }
hipError_t mlpc_gemm_reduce(const GemmArgs&, int, hipStream_t) { return done(launch_fails); }
hipError_t mlpc_dz(const DzArgs&, int, bool, hipStream_t) { return done(launch_fails); }
int mlpc_dz_parts(int64_t) { return 1; }
int mlpc_dz_max_parts() { return 64; }
hipError_t mlpc_norm_forward(const NormArgs&, int, int, hipStream_t) { return done(launch_fails); }
hipError_t mlpc_norm_backward(const NormArgs&, int, hipStream_t) { return done(launch_fails); }
int mlpc_norm_parts(int64_t, int, int) { return 1; }
int mlpc_norm_max_parts(int, int) { return 256; }

// ------------------------------------------------------------------ the checks

alignas(16) static uint16_t buf[4096];
static float stat[64];

static int norm_forward(mlp_norm_t h, hipStream_t s) { return mlp_norm_forward(h, 4, buf, 64, buf, buf, buf, 64, stat, stat, s); }
static int norm_backward(mlp_norm_t h, hipStream_t s) {
    return mlp_norm_backward(h, 4, buf, 64, buf, 64, buf, stat, stat, nullptr, 0, buf, 64, buf, buf, s);
}
static int linear_forward(mlp_linear_t h, hipStream_t s) {
    return mlp_linear_forward(h, 4, buf, 64, buf, 64, nullptr, nullptr, 0, buf, 64, nullptr, 0, s);
}

// An error that an entry point returns is not left behind as the thread's last
// error too, where the caller's next call would find it.
static void errors_are_reported_once() {
    malloc_fails = hipErrorOutOfMemory;
    CHECK(!mlp_linear_create(4, 64, 64, 0, 0, 1) && strstr(last, "hipMalloc") && pending == hipSuccess);
    CHECK(!mlp_norm_create(64, 0, 1e-5f, 1) && strstr(last, "hipMalloc") && pending == hipSuccess);
    malloc_fails = hipSuccess;
    memset_fails = hipErrorUnknown;
    CHECK(!mlp_linear_create(4, 64, 64, 0, 0, 1) && strstr(last, "clearing") && pending == hipSuccess);
    memset_fails = hipSuccess;
    mlp_norm_t n = mlp_norm_create(64, 0, 1e-5f, 1);
    mlp_linear_t l = mlp_linear_create(4, 64, 64, 0, 0, 1);
    CHECK(n && l);
    launch_fails = hipErrorInvalidConfiguration;
    CHECK(norm_forward(n, nullptr) == MLP_EHIP && pending == hipSuccess);
    CHECK(norm_backward(n, nullptr) == MLP_EHIP && pending == hipSuccess);
    CHECK(linear_forward(l, nullptr) == MLP_EHIP && pending == hipSuccess);
    launch_fails = hipSuccess;
    // (an error of the caller's own stays the caller's through calls that succeed)
    pending = hipErrorInvalidValue;
    CHECK(norm_forward(n, nullptr) == MLP_OK && norm_backward(n, nullptr) == MLP_OK && linear_forward(l, nullptr) == MLP_OK);
    CHECK(pending == hipErrorInvalidValue);
    pending = hipSuccess;
    sync_fails = hipErrorUnknown;
    CHECK(mlp_norm_destroy(n) == MLP_EHIP && pending == hipSuccess);
    CHECK(mlp_linear_destroy(l) == MLP_EHIP && pending == hipSuccess);
    sync_fails = hipSuccess;
}

// destroy waits for the work that may still use the workspace it frees: the
// last gradient, on whatever stream a forward pass (which uses none) came after.
static void destroy_waits_for_the_workspace() {
    hipStream_t one = reinterpret_cast<hipStream_t>(stat), other = reinterpret_cast<hipStream_t>(buf);
    mlp_norm_t n = mlp_norm_create(64, 0, 1e-5f, 1);
    CHECK(norm_backward(n, one) == MLP_OK && norm_forward(n, other) == MLP_OK);
    waited.clear();
    CHECK(mlp_norm_destroy(n) == MLP_OK);
    CHECK(waited.size() == 1 && waited[0] == one);
    // a handle without a workspace has nothing to wait for
    n = mlp_norm_create(64, 0, 1e-5f, 0);
    CHECK(norm_forward(n, one) == MLP_OK);
    waited.clear();
    CHECK(mlp_norm_destroy(n) == MLP_OK && waited.empty());
    mlp_linear_t l = mlp_linear_create(4, 64, 64, 0, 0, 1);
    CHECK(linear_forward(l, one) == MLP_OK && linear_forward(l, other) == MLP_OK);
    waited.clear();
    CHECK(mlp_linear_destroy(l) == MLP_OK);
    CHECK(waited.size() == 1 && waited[0] == other);
}

// The strides a linear layer takes: an operand's DMA offsets, which are 32-bit
// (rows of a tile for x W and dz W^T; 64 rows and the columns for x^T dz), hold
// for every stride that is not refused.
static void strides() {
    const int64_t rows[] = {1, 2, 7, 40, 63, 64, 65, 200, 255, 256, 257, 5000};
    for (int64_t r : rows) {
        mlp_linear_t l = mlp_linear_create(r, 64, 64, 0, 0, 1);
        auto x = [&](int64_t ld) { return mlp_linear_forward(l, r, buf, ld, buf, 64, nullptr, nullptr, 0, buf, 64, nullptr, 0, nullptr); };
        auto dy = [&](int64_t ld) { return mlp_linear_backward(l, r, buf, ld, buf, 64, buf, 64, nullptr, 0, buf, 64, buf, 64, nullptr, nullptr); };
        auto dwx = [&](int64_t ld) { return mlp_linear_backward(l, r, buf, 64, buf, ld, buf, 64, nullptr, 0, nullptr, 0, buf, 64, nullptr, nullptr); };
        CHECK(x((int64_t)1 << 23) == MLP_OK && dy((int64_t)1 << 23) == MLP_OK && dwx((int64_t)1 << 23) == MLP_OK);
        int64_t most = 8;       // by bisection
        for (int64_t step = (int64_t)1 << 40; step >= 8; step /= 2)
            if (x(most + step) == MLP_OK) most += step;
        CHECK(dy(most) == MLP_OK && dwx(most) == MLP_OK && dy(most + 8) == MLP_EINVAL && dwx(most + 8) == MLP_EINVAL);
        const int64_t tile = r < 256 ? r : 256, deep = r < 64 ? r : 64, columns = (int64_t)1 << 23;
        CHECK(((tile - 1) * most + 64) * 2 < (int64_t)1 << 32 && ((deep - 1) * most + columns) * 2 <= (int64_t)1 << 32);
        // the other operands' offsets are 64-bit, W's stride is limited alone
        const int64_t far = (int64_t)1 << 36;
        CHECK(mlp_linear_forward(l, r, buf, 64, buf, 64, nullptr, buf, far, buf + 8, far, buf, far, nullptr) == MLP_OK);
        CHECK(mlp_linear_forward(l, r, buf, 64, buf, (1 << 23) + 8, nullptr, nullptr, 0, buf, 64, nullptr, 0, nullptr) == MLP_EINVAL);
        CHECK(mlp_linear_forward(l, r, buf, 64, buf, 64, nullptr, nullptr, 0, buf, far + 8, nullptr, 0, nullptr) == MLP_EINVAL);
        CHECK(mlp_linear_destroy(l) == MLP_OK);
    }
}

int main() {
    strides();
    errors_are_reported_once();
    destroy_waits_for_the_workspace();
    CHECK(blocks == 0);
    printf("%d failures\n", failures);
    return failures != 0;
}

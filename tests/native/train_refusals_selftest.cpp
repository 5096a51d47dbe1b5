// Arguments that fp32 cannot hold, on a stand-in for the HIP runtime and the
// launchers, defined here (no GPU, no HIP library).  Prints "<n> failures" and
// exits 0 on success.
#include <math.h>
#include <stdio.h>
#include <string.h>

#include "../../consumer_gemm_chain_amd/csrc/train_launch.h"
#include "../../include/mlp_train.h"

static int failures = 0;
static char last[512];
#define CHECK(c) do { if (!(c)) { ++failures; printf("line %d: %s (%s)\n", __LINE__, #c, last); } } while (0)

int mlpc_set_error(int code, const char* msg) {
    snprintf(last, sizeof last, "%s", msg);
    return code;
}

extern "C" {
hipError_t hipGetDevice(int* d) { *d = 0; return hipSuccess; }
hipError_t hipSetDevice(int) { return hipSuccess; }
hipError_t hipDeviceGetAttribute(int* v, hipDeviceAttribute_t, int) { *v = 256; return hipSuccess; }
hipError_t hipMalloc(void** p, size_t) { *p = last; return hipSuccess; }
hipError_t hipFree(void*) { return hipSuccess; }
hipError_t hipMemset(void*, int, size_t) { return hipSuccess; }
hipError_t hipStreamSynchronize(hipStream_t) { return hipSuccess; }
hipError_t hipGetLastError(void) { return hipSuccess; }
const char* hipGetErrorString(hipError_t) { return "an error"; }
}

using namespace mlpc;
int mlpc_linear_num_configs() { return 1; }
LinearCfgInfo mlpc_linear_config(int) { return LinearCfgInfo{64, 128, 256, 0}; }
bool mlpc_linear_has(int, int) { return true; }
hipError_t mlpc_loss_rows(const LossArgs&, bool, int, hipStream_t) { return hipSuccess; }
hipError_t mlpc_loss_logits(const LossArgs&, int, bool, int, hipStream_t) { return hipSuccess; }
hipError_t mlpc_loss_products(const LossArgs&, int, int, hipStream_t) { return hipSuccess; }
hipError_t mlpc_loss_join(const LossArgs&, hipStream_t) { return hipSuccess; }
hipError_t mlpc_loss_dx(const LossArgs&, int, hipStream_t) { return hipSuccess; }
hipError_t mlpc_norm_sum(const NormTable&, int, int, hipStream_t) { return hipSuccess; }
hipError_t mlpc_norm_join(const NormJoin&, hipStream_t) { return hipSuccess; }
hipError_t mlpc_adamw_begin(const AdamBegin&, hipStream_t) { return hipSuccess; }
hipError_t mlpc_adamw(const AdamTable&, int, int, hipStream_t) { return hipSuccess; }

int main() {
    static float norm, scale;
    mlp_grad_norm_t n = mlp_grad_norm_create(0);
    CHECK(n);
    auto call = [&](double unscale) {
        last[0] = 0;
        return mlp_grad_norm_forward(n, 0, nullptr, nullptr, unscale, 1.0, &norm, &scale, nullptr);
    };
    for (double sign : {1.0, -1.0}) {
        for (double u : {1.0, 0x1p-126, 0x1p-30, 1e30, (double)3.4028234663852886e38f}) CHECK(call(sign * u) == MLP_OK);
        for (double u : {0.0, 5e-324, 1e-46, 1e-40, 0x1p-126 * (1 - 0x1p-30), 3.5e38, 1e39, 1e300, (double)INFINITY, (double)NAN})
            CHECK(call(sign * u) == MLP_EINVAL && strstr(last, "unscale"));
    }
    CHECK(mlp_grad_norm_destroy(n) == MLP_OK);
    printf("%d failures\n", failures);
    return failures != 0;
}

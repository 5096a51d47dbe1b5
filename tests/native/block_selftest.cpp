// Drives the block operators' host-only entry points (planner, argument
// checks) for a sanitizer build: no kernel is linked, the launchers are stubs
// that must not be reached.  Prints "<n> failures" and exits 0 on success.
#include <stdio.h>
#include <string.h>

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

using namespace mlpc;
int mlpc_linear_num_configs() { return MLPC_NUM_LINEAR_CONFIGS; }
LinearCfgInfo mlpc_linear_config(int cfg) {
#define ROW(id, bm, bn, wm, wn, ns, ks, occ) \
    if (cfg == id) return LinearCfgInfo{bm, bn, 64 * wm * wn, ns * (bm + bn) * ks * 2};
    MLPC_LINEAR_CONFIGS(ROW)
    return LinearCfgInfo{};
}
bool mlpc_linear_has(int cfg, int pass) { return pass > PASS_DW ? cfg != 0 && cfg != 7 : pass == PASS_DW ? mlpc_linear_config(cfg).BM >= 128 : cfg != 7; }
static hipError_t unreached() { ++failures; return hipErrorUnknown; }
hipError_t mlpc_gemm(const GemmArgs&, int, int, int, hipStream_t) { return unreached(); }
hipError_t mlpc_gemm_both(const GemmArgs&, const GemmArgs&, const DzArgs&, int, int, hipStream_t) { return unreached(); }
hipError_t mlpc_gemm_reduce(const GemmArgs&, int, hipStream_t) { return unreached(); }
hipError_t mlpc_dz(const DzArgs&, int, bool, hipStream_t) { return unreached(); }
int mlpc_dz_parts(int64_t) { return 1; }
int mlpc_dz_max_parts() { return 64; }
hipError_t mlpc_norm_forward(const NormArgs&, int, int, hipStream_t) { return unreached(); }
hipError_t mlpc_norm_backward(const NormArgs&, int, hipStream_t) { return unreached(); }
int mlpc_norm_parts(int64_t, int, int) { return 1; }
int mlpc_norm_max_parts(int, int) { return 256; }

int main() {
    int64_t plan[9];
    const int64_t rows[] = {1, 3, 16, 17, 64, 127, 300, 1000, 2048, 8191, 1 << 24};
    const int64_t widths[] = {8, 64, 72, 512, 2752, 12288, (1 << 22) - 8};
    for (int64_t r : rows)
        for (int64_t k : widths)
            for (int64_t n : widths)
                for (int act = 0; act < 3; ++act)
                    for (int pass = 0; pass < PASSES; ++pass) {
                        memset(plan, 0xff, sizeof plan);
                        CHECK(mlp_linear_plan(r, k, n, act, pass, 256, plan, 9) == MLP_OK);
                        CHECK(plan[0] >= 0 && plan[0] < MLPC_NUM_LINEAR_CONFIGS && plan[1] >= 1 && plan[1] <= 32);
                    }
    int64_t guard[4] = {7, 7, 7, 7};
    CHECK(mlp_linear_plan(64, 512, 512, 0, 0, 256, guard, 3) == MLP_OK && guard[3] == 7);
    CHECK(mlp_linear_plan(64, 512, 512, 0, 0, 256, guard, 2) == MLP_EINVAL);
    CHECK(mlp_linear_plan(64, 512, 512, 0, 0, 256, nullptr, 9) == MLP_EINVAL);
    CHECK(mlp_linear_plan(0, 512, 512, 0, 0, 256, plan, 9) == MLP_EINVAL && strstr(last, "rows"));
    CHECK(mlp_linear_plan(64, 511, 512, 0, 0, 256, plan, 9) == MLP_EINVAL);
    CHECK(mlp_linear_plan(64, 512, (int64_t)1 << 40, 0, 0, 256, plan, 9) == MLP_EINVAL);
    CHECK(!mlp_linear_create(-1, 8, 8, 0, 0, 1) && !mlp_linear_create(1, 8, 8, 0, 7, 1) && !mlp_linear_create(1, 8, 8, 9, 0, 1));
    CHECK(!mlp_norm_create(0, 0, 1e-5f, 1) && !mlp_norm_create(8, 3, 1e-5f, 1) && !mlp_norm_create(8, 0, -1.f, 0));
    CHECK(mlp_norm_forward(nullptr, 1, plan, 8, nullptr, nullptr, plan, 8, nullptr, nullptr, nullptr) == MLP_EINVAL);
    CHECK(mlp_linear_debug_set_plan(nullptr, 0, 0, 1) == MLP_EINVAL);
    CHECK(mlp_norm_destroy(nullptr) == MLP_OK && mlp_linear_destroy(nullptr) == MLP_OK);
    printf("%d failures\n", failures);
    return failures != 0;
}

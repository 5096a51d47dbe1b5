// linear_dispatch.cpp -- table of the linear layer's tile configurations (each
// one's kernels live in their own object, built from linear_kernels.hip).
#include "block_launch.h"
#include "linear_configs.h"

using namespace mlpc;

#define MLPC_DECL(id, ...)                                                            \
    hipError_t mlpc_linear_launch##id(const GemmArgs&, int, int, hipStream_t);        \
    hipError_t mlpc_linear_both##id(const GemmArgs&, const GemmArgs&, const DzArgs&, int, hipStream_t); \
    LinearCfgInfo mlpc_linear_info##id();                                             \
    bool mlpc_linear_has##id(int);
MLPC_LINEAR_CONFIGS(MLPC_DECL)
#undef MLPC_DECL

int mlpc_linear_num_configs() { return MLPC_NUM_LINEAR_CONFIGS; }

LinearCfgInfo mlpc_linear_config(int cfg) {
#define MLPC_CASE(n, ...) \
    case n: return mlpc_linear_info##n();
    switch (cfg) { MLPC_LINEAR_CONFIGS(MLPC_CASE) default: return LinearCfgInfo{}; }
#undef MLPC_CASE
}

bool mlpc_linear_has(int cfg, int pass) {
#define MLPC_CASE(n, ...) \
    case n: return mlpc_linear_has##n(pass);
    switch (cfg) { MLPC_LINEAR_CONFIGS(MLPC_CASE) default: return false; }
#undef MLPC_CASE
}

hipError_t mlpc_gemm(const GemmArgs& a, int cfg, int pass, int dtype, hipStream_t s) {
#define MLPC_CASE(n, ...) \
    case n: return mlpc_linear_launch##n(a, pass, dtype, s);
    switch (cfg) { MLPC_LINEAR_CONFIGS(MLPC_CASE) default: return hipErrorInvalidValue; }
#undef MLPC_CASE
}

hipError_t mlpc_gemm_both(const GemmArgs& dx, const GemmArgs& dw, const DzArgs& dz, int cfg, int dtype, hipStream_t s) {
#define MLPC_CASE(n, ...) \
    case n: return mlpc_linear_both##n(dx, dw, dz, dtype, s);
    switch (cfg) { MLPC_LINEAR_CONFIGS(MLPC_CASE) default: return hipErrorInvalidValue; }
#undef MLPC_CASE
}

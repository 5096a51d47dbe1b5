// loss_dispatch.cpp -- table of the cross entropy's tile configurations (each
// one's kernels live in their own object, built from loss_kernels.hip).
#include "loss_configs.h"
#include "train_launch.h"

using namespace mlpc;

#define MLPC_DECL(id, ...)                                                        \
    hipError_t mlpc_loss_logits##id(const LossArgs&, bool, int, hipStream_t);     \
    hipError_t mlpc_loss_products##id(const LossArgs&, int, hipStream_t);
MLPC_LOSS_CONFIGS(MLPC_DECL)
#undef MLPC_DECL

hipError_t mlpc_loss_logits(const LossArgs& a, int cfg, bool backward, int dtype, hipStream_t s) {
#define MLPC_CASE(n, ...) \
    case n: return mlpc_loss_logits##n(a, backward, dtype, s);
    switch (cfg) { MLPC_LOSS_CONFIGS(MLPC_CASE) default: return hipErrorInvalidValue; }
#undef MLPC_CASE
}

hipError_t mlpc_loss_products(const LossArgs& a, int cfg, int dtype, hipStream_t s) {
#define MLPC_CASE(n, ...) \
    case n: return mlpc_loss_products##n(a, dtype, s);
    switch (cfg) { MLPC_LOSS_CONFIGS(MLPC_CASE) default: return hipErrorInvalidValue; }
#undef MLPC_CASE
}

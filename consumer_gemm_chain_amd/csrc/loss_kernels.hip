// loss_kernels.hip -- the products of the cross entropy, one object per tile
// configuration (-DMLPC_LOSS=<id>, loss_configs.h).
#include <hip/hip_runtime.h>

#include "loss_configs.h"
#include "loss_device.hpp"

namespace mlpc {

#define MLPC_PICK(id, bm, bn, wm, wn, ns, ks, occ, early) \
    if constexpr (id == MLPC_LOSS) return LinCfg<bm, bn, wm, wn, ns, ks, occ, early>{};
static constexpr auto this_cfg() { MLPC_LOSS_CONFIGS(MLPC_PICK) }
#undef MLPC_PICK
using Cfg = decltype(this_cfg());

// The configurations that the linear layer has for both products in one launch.
static constexpr bool HAS_PRODUCTS = MLPC_LOSS != 0;

// Rows of tiles for any number of rows up to `rows`: tall tiles may be of 160 to
// 256 rows.
static uint32_t row_tiles(int64_t rows) {
    constexpr int least = Cfg::FM == 8 ? 160 : Cfg::BM;
    return (uint32_t)((rows + least - 1) / least);
}

template <int DT>
static hipError_t logits(const LossArgs& a, bool backward, hipStream_t s) {
    const dim3 grid((a.packing ? row_tiles(a.rows) : a.Mt) * a.Nt);
    return backward ? launch(loss_logits_kernel<Cfg, DT, true>, grid, Cfg::NT, s, a)
                    : launch(loss_logits_kernel<Cfg, DT, false>, grid, Cfg::NT, s, a);
}

template <int DT>
static hipError_t products(const LossArgs& a, hipStream_t s) {
    if constexpr (HAS_PRODUCTS) {
        const uint32_t dx = a.dx ? (row_tiles(a.rows) * a.dxNt * a.S + 7) / 8 * 8 : 0, dw = a.dw ? a.dwMt * a.dwNt : 0;
        return launch(loss_products_kernel<Cfg, DT>, dim3(dx + dw), Cfg::NT, s, a, dx);
    }
    return hipErrorInvalidValue;
}

}  // namespace mlpc

using namespace mlpc;

#define MLPC_CAT2(a, b) a##b
#define MLPC_CAT(a, b) MLPC_CAT2(a, b)

hipError_t MLPC_CAT(mlpc_loss_logits, MLPC_LOSS)(const LossArgs& a, bool backward, int dtype, hipStream_t s) {
    return dtype == DT_F16 ? logits<DT_F16>(a, backward, s) : logits<DT_BF16>(a, backward, s);
}

hipError_t MLPC_CAT(mlpc_loss_products, MLPC_LOSS)(const LossArgs& a, int dtype, hipStream_t s) {
    return dtype == DT_F16 ? products<DT_F16>(a, s) : products<DT_BF16>(a, s);
}

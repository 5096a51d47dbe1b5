// linear_kernels.hip -- the products of the linear layer, one object per tile
// configuration (-DMLPC_LIN=<id>, linear_configs.h).
#include <hip/hip_runtime.h>

#include "linear_configs.h"
#include "linear_device.hpp"

namespace mlpc {

#define MLPC_PICK(id, bm, bn, wm, wn, ns, ks, occ) \
    if constexpr (id == MLPC_LIN) return LinCfg<bm, bn, wm, wn, ns, ks, occ>{};
static constexpr auto this_cfg() { MLPC_LINEAR_CONFIGS(MLPC_PICK) }
#undef MLPC_PICK
using Cfg = decltype(this_cfg());

// x^T dz has K rows of output, never few: it goes without the short tiles.  It
// writes as much as it reads, so it alone has the two-per-CU 256 x 128 tiles
// (8192 x 7168 over 1000 rows: 115 us against 127 with 256 x 256; x W and
// dz W^T run 2-15% slower on them than on configurations 3 to 5).
// Both products in one launch go without the 16-row tiles and configuration 7.
static constexpr bool HAS_BOTH = MLPC_LIN != 0 && MLPC_LIN != 7;

static constexpr bool has(int pass) {
    if (pass == PASS_BOTH_DX || pass == PASS_BOTH_DW) return HAS_BOTH;
    return pass == PASS_DW ? Cfg::BM >= 128 : MLPC_LIN != 7;
}

// Workgroups of a product.
static uint32_t blocks(const GemmArgs& a) { return a.direct + (a.Mt * a.Nt - a.direct) * a.S; }

template <int DT>
static hipError_t both(const GemmArgs& dx, const GemmArgs& dw, const DzArgs& dz, hipStream_t s) {
    if constexpr (HAS_BOTH) {
        const uint32_t n = blocks(dx), db = dz.db ? (dw.N + Cfg::NT - 1) / Cfg::NT : 0;
        return launch(linear_both_kernel<Cfg, DT>, dim3(db + n + blocks(dw)), Cfg::NT, s, dx, dw, dz, db, n);
    }
    return hipErrorInvalidValue;
}

template <int DT>
static hipError_t one(const GemmArgs& a, int pass, hipStream_t s) {
    const dim3 grid(blocks(a));
    if constexpr (has(PASS_FWD)) {
        if (pass == PASS_FWD) return launch(linear_kernel<Cfg, DT, PASS_FWD>, grid, Cfg::NT, s, a);
        if (pass == PASS_DX) return launch(linear_kernel<Cfg, DT, PASS_DX>, grid, Cfg::NT, s, a);
    }
    if constexpr (has(PASS_DW)) {
        if (pass == PASS_DW) return launch(linear_kernel<Cfg, DT, PASS_DW>, grid, Cfg::NT, s, a);
    }
    return hipErrorInvalidValue;
}

}  // namespace mlpc

using namespace mlpc;

#define MLPC_CAT2(a, b) a##b
#define MLPC_CAT(a, b) MLPC_CAT2(a, b)

hipError_t MLPC_CAT(mlpc_linear_launch, MLPC_LIN)(const GemmArgs& a, int pass, int dtype, hipStream_t s) {
    return dtype == DT_F16 ? one<DT_F16>(a, pass, s) : one<DT_BF16>(a, pass, s);
}

hipError_t MLPC_CAT(mlpc_linear_both, MLPC_LIN)(const GemmArgs& dx, const GemmArgs& dw, const DzArgs& dz, int dtype,
                                              hipStream_t s) {
    return dtype == DT_F16 ? both<DT_F16>(dx, dw, dz, s) : both<DT_BF16>(dx, dw, dz, s);
}

LinearCfgInfo MLPC_CAT(mlpc_linear_info, MLPC_LIN)() { return LinearCfgInfo{Cfg::BM, Cfg::BN, Cfg::NT, Cfg::RING}; }

bool MLPC_CAT(mlpc_linear_has, MLPC_LIN)(int pass) { return has(pass); }

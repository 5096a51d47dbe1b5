// loss_configs.h -- the tile configurations of the cross entropy's products.
// X(id, BM, BN, WM, WN, NS, KS, OCC) as in linear_configs.h.
#pragma once

#define MLPC_LOSS_CONFIGS(X)                                                                       \
    X(0, 16, 128, 1, 2, 4, 64, 1)                                                                  \
    X(1, 64, 128, 2, 2, 3, 64, 2)                                                                  \
    X(2, 128, 128, 4, 2, 4, 64, 2)                                                                 \
    X(3, 256, 256, 2, 4, 4, 32, 2)                                                                 \
    X(4, 256, 256, 2, 2, 4, 32, 1)                                                                 \
    X(5, 256, 256, 2, 2, 2, 64, 1)                                                                 \
    X(6, 128, 256, 2, 4, 3, 64, 2)                                                                 \
    X(7, 256, 128, 2, 2, 3, 32, 2)                                                                 \
    X(8, 128, 128, 2, 2, 3, 32, 2)

#define MLPC_LOSS_COUNT(id, ...) +1
constexpr int MLPC_NUM_LOSS_CONFIGS = 0 MLPC_LOSS_CONFIGS(MLPC_LOSS_COUNT);

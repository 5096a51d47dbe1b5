// loss_configs.h -- the tile configurations of the cross entropy's products.
// X(id, BM, BN, WM, WN, NS, KS, OCC, EARLY) as in linear_configs.h, whose tiles
// with the same id they are: its estimates choose among them.
#pragma once

// EARLY: 256 x 256 as two stages of 64 wait for each other half as often as four
// of 32, and with two rows read early no LDS latency is left before a wait: 4096 x
// 8192 x 32000, z with its softmax 1705 us with four stages of 32, 1604 with two
// of 64, 1567 (1.37 PFLOP/s) with two rows early as well; backward 5070, 4922,
// 4830.  On configurations 3 and 5 the early rows gain 1%, on 6 nothing.
#define MLPC_LOSS_CONFIGS(X)                                                                         \
    X(0, 16, 128, 1, 2, 4, 64, 1, 0)                                                                 \
    X(1, 64, 128, 2, 2, 3, 64, 2, 0)                                                                 \
    X(2, 128, 128, 4, 2, 4, 64, 2, 0)                                                                \
    X(3, 256, 128, 4, 2, 3, 64, 2, 2)                                                                \
    X(4, 256, 256, 2, 4, 2, 64, 2, 2)                                                                \
    X(5, 128, 256, 2, 4, 3, 64, 2, 2)                                                                \
    X(6, 128, 128, 2, 2, 3, 32, 2, 0)

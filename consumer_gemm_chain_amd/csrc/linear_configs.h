// linear_configs.h -- the tile configurations of the linear layer's products.
// X(id, BM, BN, WM, WN, NS, KS, OCC): BM x BN tile of WM x WN waves, NS LDS
// stages of KS reduction elements each, register target OCC waves per SIMD.
#pragma once

#define MLPC_LINEAR_CONFIGS(X)                                                                     \
    X(0, 16, 128, 1, 2, 4, 64, 1)    /* up to 16 rows: weight streaming, two workgroups per CU */  \
    X(1, 64, 128, 2, 2, 3, 64, 2)    /* up to 64 rows: two workgroups per CU */                    \
    X(2, 128, 128, 4, 2, 4, 64, 2)   /* few tiles: a deep ring, one workgroup per CU */            \
    X(3, 256, 128, 4, 2, 3, 64, 2)                                                                 \
    X(4, 256, 256, 2, 4, 4, 32, 2)   /* large products: fewest operand bytes per multiply */       \
    X(5, 128, 256, 2, 4, 3, 64, 2)   /* rows just past a multiple of 256 */                        \
    X(6, 128, 128, 2, 2, 3, 32, 2)   /* short reductions: three workgroups per CU */               \
    X(7, 256, 128, 2, 2, 3, 32, 2)   /* x^T dz: two workgroups per CU, one's stores under the other's MFMAs */

#define MLPC_LINEAR_COUNT(id, ...) +1
constexpr int MLPC_NUM_LINEAR_CONFIGS = 0 MLPC_LINEAR_CONFIGS(MLPC_LINEAR_COUNT);

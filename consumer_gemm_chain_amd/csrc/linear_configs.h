// linear_configs.h -- the tile configurations of the linear layer's products.
// X(id, BM, BN, WM, WN, NS, KS, OCC): BM x BN tile of WM x WN waves, NS LDS
// stages of KS reduction elements each, register target OCC waves per SIMD.
// Each is the fastest somewhere (x W in us, best split each; 12288 x 6144
// unless other sizes are given): 1 row 0: 31.0, 1: 29.8; 8192 x 2752 swiglu,
// 16 rows 0: 20.9, 1: 21.1; 128 rows 2: 42, 5: 44, 3: 50; 256 rows 3: 56,
// 5: 59; 300 rows 5: 72, 4: 80, 3: 90; 2048 rows 4: 280, 3: 287; 6144 x 12288,
// 2048 rows 3: 277, 4: 283; x^T dz of 64 rows 6: 41, 4: 52, of 1000 rows
// 8192 x 7168 7: 115, 4: 127.
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

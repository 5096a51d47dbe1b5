// train_launch.h -- internal interface between the C ABI of the training
// step's operators (train_api.cpp) and their kernels (loss_kernels.hip,
// loss_rows.hip, optim_kernels.hip).  Not part of the public ABI.
#pragma once

#include "../../include/mlp_train.h"
#include "block_launch.h"

namespace mlpc {

// What the loss's kernels know of a call's rows, made on the device.  The rows
// that count are packed (row r is packed row place[r]), and the products run
// over the n packed rows only.  Calls whose rows fit one tile would gain nothing
// by that: theirs stay where they are, and dz is 0 in rows that are left out.
struct LossInfo {
    int n;
    float unit;             // dz is held in units of this
    int copied;             // the products' x is the workspace's: packed, or with zeros in the rows left out
};

// How tall tiles, of 5 to 8 fragments of 32 rows, take n rows in least time, if
// each row of tiles has `columns` tiles, dealt to `cus` CUs in rounds (0: among
// other work): 670 rows are three tiles of seven fragments, 700 one of eight and
// two of seven.  A tile costs as much as 1.2 fragments more than its products; half
// of what a last, partial round wastes comes back as the others' higher clocks
// (1000 x 12288 x 50001 with a third of the rows left out, z alone: 256 rows per
// tile 1030 us, 160 rows, which fill the rounds best, 1225, 224 rows 955).  With
// one height for all of a call's tiles 8192 -> 32000 bf16 took, z and gradient, 2300
// rows 1090 and 3065 us, with these 985 and 2975; 3686 rows 1562 and 4584, 1495 and
// 4488; 330 rows 224 and 693, 220 and 690.
struct Fragments {
    int tiles, base, extra;     // the first `extra` tiles have base + 1 fragments
    float cost, whole;          // in units of a fragment, and that of tiles of 8
};

__host__ __device__ inline Fragments fragments_for(int n, uint32_t columns, uint32_t cus) {
    const int all = (n + 31) / 32, least = (all + 7) / 8, most = (all + 4) / 5;
    Fragments best{};
    if (all == 0) return best;      // every row is left out: no tile, and no number of them to divide by
    for (int k = least; k <= most && k < least + 4; ++k) {
        const uint32_t tiles = (uint32_t)k * columns;
        const float rounds = cus ? 0.5f * ((float)((tiles + cus - 1) / cus) + (float)tiles / (float)cus) : (float)tiles;
        const float height = (float)all / (float)k, c = rounds * ((height < 5.f ? 5.f : height) + 1.2f);
        if (k == least) best.whole = rounds * 9.2f;
        if (k > least && c >= best.cost) continue;
        best.cost = c;
        best.tiles = k;
        best.base = all / k < 5 ? 5 : all / k;
        best.extra = all - k * best.base < 0 ? 0 : all - k * best.base;
    }
    return best;
}

struct LossRow {            // of a packed row, for dz
    float lse, a, b;        // dz = a exp(z - lse) - b [v = target], in units
    int target;             // -1: left out
};

struct LossArgs {
    int64_t rows;
    int H, V;
    const uint16_t* x;
    int64_t ldx;
    const uint16_t* w;
    int64_t ldw;
    const int64_t* target;
    const float *lse_in, *dloss, *dlse;     // backward; dloss, dlse: nullptr
    float *loss, *lse;                      // forward; loss: nullptr
    uint16_t *dx, *dw;                      // nullptr: not computed
    int64_t lddx, lddw;
    // workspace
    LossInfo* info;
    int* place;             // [rows]; -1: left out
    LossRow* row;           // [rows] packed (info); the forward pass uses its target alone
    uint16_t* packed;       // [rows, H] of x
    float2* part;           // [rows][Nt] maximum and sum of exp(z - maximum) of each tile's columns
    float* picked;          // [rows] z at the target
    uint16_t* dz;           // [rows, lddz] of a piece
    int64_t lddz;
    float* sums;            // [S][rows, H] dx in units, of the pieces so far
    const void* zero;
    // a piece of the vocabulary
    int v0, vn;
    bool first;             // sums start here
    bool packing;           // the rows have been packed
    bool direct;            // dx is written by the products, not its sums
    // plan: tiles of the launch's products; dx's reduction in S parts of ksp slabs
    uint32_t Mt, Nt;        // x W^T
    uint32_t dxNt, S, ksp;
    uint32_t dwMt, dwNt;
    int tiles;              // of the forward pass: Nt
    uint32_t cus;
};

// Tables of tensors travel as kernel arguments (at most 4 KB with the implicit
// ones), so a call needs
// no copy and no memory of its own; entry i's chunks begin at first[i].
constexpr int NORM_CHUNK = 8192;        // elements
constexpr int NORM_PARTS = 2048;        // workgroups, and partial sums

struct NormTable {
    static constexpr int MAX = 184;
    const uint16_t* grad[MAX];
    int64_t n[MAX];
    uint32_t first[MAX];
    int count;
    uint32_t chunks;
    bool add;               // to the partial sums of earlier tables
    double* part;           // [NORM_PARTS]
};

struct NormJoin {
    const double* part;
    int parts;
    double unscale, max_norm;
    float *norm, *scale;    // scale: nullptr
};

constexpr int ADAM_CHUNK = 2048;        // elements of a workgroup

// Of a step, made on the device.
struct AdamStep {
    double lr;
    float scale, size, root;    // gradients' factor; lr / (1 - beta1^t); 1 / sqrt(1 - beta2^t)
    uint32_t key;               // of the random bits
    bool run;
};

struct AdamBegin {
    AdamStep* step;
    int64_t* t;
    const float *scale, *lr_scale;      // nullptr: 1
    double lr, beta1, beta2;
    uint32_t seed;
};

struct AdamTable {
    static constexpr int MAX = 48;
    const uint16_t* grad[MAX];
    uint16_t* w[MAX];
    float* master[MAX];
    void *m[MAX], *v[MAX];
    float *m_scale[MAX], *v_scale[MAX];
    double decay[MAX];
    int64_t n[MAX];
    uint32_t first[MAX];
    int count, number;      // number: of the first entry in the call
    uint32_t chunks;
    float beta1, rest1, beta2, rest2, eps;
    bool chance;            // m in 8 bits is rounded by chance, as v is
    const AdamStep* step;
};

static_assert(sizeof(NormTable) <= 3840 && sizeof(AdamTable) <= 3840, "kernel arguments");

}  // namespace mlpc

// Pack the rows that count, find dz's unit (backward) and gather x.
hipError_t mlpc_loss_rows(const mlpc::LossArgs& a, bool backward, int dtype, hipStream_t s);
// z's tiles of a piece: their maxima, sums and picked elements, or dz.
hipError_t mlpc_loss_logits(const mlpc::LossArgs& a, int cfg, bool backward, int dtype, hipStream_t s);
// dx's sums and dw of a piece, each unless its pointer is nullptr.
hipError_t mlpc_loss_products(const mlpc::LossArgs& a, int cfg, int dtype, hipStream_t s);
// loss and lse from the tiles'.
hipError_t mlpc_loss_join(const mlpc::LossArgs& a, hipStream_t s);
// dx from its sums.
hipError_t mlpc_loss_dx(const mlpc::LossArgs& a, int dtype, hipStream_t s);

// The partial sums of a table's squares, by `parts` workgroups, and their join.
hipError_t mlpc_norm_sum(const mlpc::NormTable& a, int dtype, int parts, hipStream_t s);
hipError_t mlpc_norm_join(const mlpc::NormJoin& a, hipStream_t s);
// The step's number and factors, and a table's tensors.
hipError_t mlpc_adamw_begin(const mlpc::AdamBegin& a, hipStream_t s);
hipError_t mlpc_adamw(const mlpc::AdamTable& a, int dtype, int bits, hipStream_t s);

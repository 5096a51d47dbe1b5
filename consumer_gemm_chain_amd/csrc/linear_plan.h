// linear_plan.h -- how a product on the linear layer's tiles runs, and what it
// is estimated to take.
#pragma once

#include <math.h>
#include <stdint.h>

#include "block_launch.h"
#include "chain_launch.h"

// How a product runs: tile configuration, tiles, the tiles computed whole, the
// parts of the others' reduction and slabs per part.
struct Plan {
    int cfg;
    uint32_t Mt, Nt, direct, S, ksp;
    size_t part_bytes;
};

namespace {

// Parts a reduction may have.
constexpr uint32_t MAX_SPLIT = 32;

// The plan of a product of M x N columns (both halves of swiglu's B) over K
// with configuration cfg and at most `split` parts (no part is empty).  As
// many tiles as fill whole rounds of the chip are never split, only those of
// the last, partial round.
Plan make_plan(int cfg, int64_t M, int64_t N, int64_t K, uint32_t split, int cus) {
    const mlpc::LinearCfgInfo c = mlpc_linear_config(cfg);
    const uint32_t slabs = (uint32_t)(K / mlpc::BK);
    Plan p;
    p.cfg = cfg;
    p.Mt = (uint32_t)((M + c.BM - 1) / c.BM);
    p.Nt = (uint32_t)((N + c.BN - 1) / c.BN);
    const uint32_t tiles = p.Mt * p.Nt;
    if (split > slabs) split = slabs;
    if (split < 1) split = 1;
    p.ksp = slabs ? (slabs + split - 1) / split : 0;
    p.S = slabs ? (slabs + p.ksp - 1) / p.ksp : 1;
    p.direct = p.S > 1 ? tiles - tiles % (uint32_t)cus : 0;
    if (p.direct == tiles) p.S = 1;
    p.part_bytes = p.S > 1 ? (size_t)(tiles - p.direct) * p.S * c.BM * c.BN * 4 : 0;
    return p;
}

// What the planner considers: tiles of at most twice the rows (64-row tiles
// always), and splits into at most one part per CU.  More never were fastest,
// and the limits bound the workspace of the partials.
bool config_fits(const mlpc::LinearCfgInfo& c, int64_t M) { return c.BM <= 64 || c.BM <= 2 * M; }

bool split_fits(const Plan& p, int cus) { return p.S == 1 || (p.Mt * p.Nt - p.direct) * p.S <= (uint32_t)cus; }

// When the last of `slots` places for workgroups falls free, if groups of
// equal workgroups (their number and duration) are dealt in turn to the place
// that is free first.
double dealt(const double (*group)[2], int groups, double slots) {
    double at[8] = {0.0}, n[8] = {slots};       // places by the time they fall free, ascending
    int levels = 1;
    for (int g = 0; g < groups; ++g) {
        double left = group[g][0];
        const double d = group[g][1];
        while (left > 0.0) {
            const double cycles = floor(left / slots);
            if (at[levels - 1] - at[0] <= d && cycles >= 1.0) {
                // every place takes as many
                for (int i = 0; i < levels; ++i) at[i] += cycles * d;
                left -= cycles * slots;
                continue;
            }
            const double k = left < n[0] ? left : n[0], t = at[0] + d;
            left -= k;
            n[0] -= k;
            int i = 0;
            if (n[0] <= 0.0) {
                for (--levels; i < levels; ++i) {
                    at[i] = at[i + 1];
                    n[i] = n[i + 1];
                }
            }
            for (i = levels; i > 0 && at[i - 1] > t; --i) {
                at[i] = at[i - 1];
                n[i] = n[i - 1];
            }
            at[i] = t;
            n[i] = k;
            ++levels;
        }
    }
    return at[levels - 1];
}

// A plan with the sizes it is for.
struct Work {
    Plan p;
    int64_t M, N, K;
};

// What a launch's time is estimated from, per tile configuration: a workgroup
// takes `slab` microseconds per 64-deep slab among several rounds of workgroups,
// `alone` times that with a single one, and `fixed` for its prologue and
// epilogue; the chip's power caps the multiplication rate whatever the
// schedule at `cap` MFLOP per microsecond.  Workgroups of a CU share it: beyond
// the first, one adds `share` places and each takes that much longer.  Partials
// travel at `join` MB per microsecond after a launch of `launch`; a ragged slab
// costs `ragged` of a whole one.  Operands are read at `read` and outputs
// written at `write` MB per microsecond at best; operands that no other running
// workgroup reads too arrive at `all` MB per microsecond in all and `cu` KB per
// CU (caches included).
struct Rates {
    double slab[8], alone[8], fixed[8], cap[8];
    double share, launch, join, ragged, read, write, all, cu;
};

// One product: fitted to every configuration and split of 529 sizes of x W and
// 244 of x^T dz drawn over 1 to 8192 rows.  On sizes drawn afterwards the chosen
// plan took 0.8% and 1.7% longer than the fastest on average, at worst 28% (a
// split where none was needed, 8.6 us).
const Rates SINGLE = {{0.416, 0.618, 0.72, 0.884, 1.54, 0.892, 0.707, 0.718},
                      {0.985, 0.816, 0.959, 1.17, 0.898, 0.977, 1.46, 1.33},
                      {1.55, 2.42, 3.78, 7.78, 17.5, 8.67, 1.37, 5.78},
                      {1150, 1150, 900, 1120, 1230, 1080, 1150, 1150},
                      0.328, 5.48, 4.52, 1, 7.2, 2.49, 7.77, 34};
// Both products of the gradient in one launch: the same of 541 sizes; 1.5%, at
// worst 22%.  Configurations 0 and 7 do not have it.
const Rates BOTH = {{0, 0.44, 0.647, 0.799, 1.65, 1.53, 0.547, 0},
                    {0, 0.93, 0.862, 1.04, 0.848, 0.502, 1.74, 0},
                    {0, 1.37, 3.12, 4.64, 9.04, 4.23, 1.55, 0},
                    {1, 1080, 770, 960, 1210, 1500, 1150, 1},
                    0.418, 6.65, 6.15, 0.324, 4.76, 3.2, 6.86, 107};

// Estimated microseconds of the products `w` of one configuration in one
// launch, and their partials' way out and back.  Small ones take no less than
// the host's time for their launches.  A product's multiplications take `part`
// of what its whole tiles would (the first one's, if its tiles are shorter).
double plan_cost(const Work* w, int products, const Rates& t, int cus, double part = 1.0) {
    static const int per_cu[] = {2, 2, 1, 1, 1, 1, 3, 2};
    const int cfg = w[0].p.cfg;
    const mlpc::LinearCfgInfo c = mlpc_linear_config(cfg);
    double total = 0.0;
    for (int i = 0; i < products; ++i) total += w[i].p.direct + ((double)w[i].p.Mt * w[i].p.Nt - w[i].p.direct) * w[i].p.S;
    const double active = fmin(total, cus);
    const double room = 1.0 + t.share * (fmin(per_cu[cfg], ceil(total / cus)) - 1.0);
    // (sharing does not make a workgroup faster than it is alone)
    const double slab = t.slab[cfg] * (total <= cus ? t.alone[cfg] : fmax(1.0, t.alone[cfg] / room));
    double group[4][2], power = 0.0, memory = 0.0, join = 0.0, launches = 6.0;
    int groups = 0;
    for (int i = 0; i < products; ++i) {
        const Plan& p = w[i].p;
        const double M = (double)w[i].M, N = (double)w[i].N, K = (double)w[i].K, tiles = (double)p.Mt * p.Nt, split = tiles - p.direct;
        const double bytes = 128.0 * ((double)c.BN / p.Mt + (double)c.BM / p.Nt);
        const double whole = i == 0 ? part : 1.0;
        const double per = fmax(slab * whole, fmax(bytes * active / (t.all * 1e6), bytes / (t.cu * 1e3)));
        power += whole * tiles * c.BM * c.BN * K * 2e-6 / t.cap[cfg];
        memory += 2.0 * (M * K + K * N) / (t.read * 1e6) + 2.0 * M * N / (t.write * 1e6);
        if (p.S == 1 || p.direct) {
            group[groups][0] = p.S == 1 ? tiles : p.direct;
            group[groups++][1] = room * (t.fixed[cfg] + (floor(K / mlpc::BK) + (w[i].K % mlpc::BK ? t.ragged : 0.0)) * per);
        }
        if (p.S == 1) continue;
        group[groups][0] = split * p.S;
        group[groups++][1] = room * (t.fixed[cfg] + p.ksp * per);
        const double values = split * c.BM * c.BN * fmin(1.0, M / ((double)p.Mt * c.BM)) * fmin(1.0, N / ((double)p.Nt * c.BN));
        join += t.launch + values * 4 * p.S * 2 / (t.join * 1e6);
        launches += 2.8;
    }
    const double run = dealt(group, groups, floor(cus * room));
    // (below the launches' floor the estimate itself tells plans apart)
    return fmax(fmax(run, fmax(power, memory)) + join, launches) + 0.01 * (run + join);
}

}  // namespace

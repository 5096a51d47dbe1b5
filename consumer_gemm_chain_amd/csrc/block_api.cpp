// block_api.cpp -- the C ABI declared in include/mlp_block.h: argument
// checks, workspace ownership and launches.
#include <hip/hip_runtime.h>

#include <math.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include <new>

#include "../../include/mlp_block.h"
#include "block_launch.h"
#include "chain_launch.h"

struct mlp_norm {
    int H;
    int dtype;
    int device, cus;
    float eps;
    float* part;                // [max parts][2][H]; nullptr: no gradient
    hipStream_t last_stream;
};

// How a product runs: tile configuration, tiles, the tiles computed whole, the
// parts of the others' reduction and slabs per part.
struct Plan {
    int cfg;
    uint32_t Mt, Nt, direct, S, ksp;
    size_t part_bytes;
};

struct mlp_linear {
    int64_t max_rows;
    int K, N, gN;
    int act, dtype, device, cus;
    int forced_cfg[mlpc::PASSES], forced_split[mlpc::PASSES];       // per pass; -1 / 0: the planner's
    int64_t plan_rows[mlpc::PASSES];        // the row count plan[pass] is for (-1: none)
    Plan plan[mlpc::PASS_DW + 1];
    Plan both[2];                           // the gradient's two products in one launch
    // workspace (one allocation): zero page | dz [max_rows, gN] (activations
    // only) | column-sum partials [max parts][gN] | split partials; dz and the
    // column sums only with the gradient
    void* ws;
    void* zero;
    uint16_t* dz;
    float* colsum;
    float* part;
    size_t part_bytes;
    hipStream_t last_stream;
};

namespace {

int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int fail(int code, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return mlpc_set_error(code, buf);
}

struct DeviceGuard {
    int prev = -1;
    bool ok = true;
    explicit DeviceGuard(int dev) {
        if (hipGetDevice(&prev) != hipSuccess) { ok = false; return; }
        if (prev != dev && hipSetDevice(dev) != hipSuccess) ok = false;
    }
    ~DeviceGuard() {
        int cur = -1;
        if (prev >= 0 && hipGetDevice(&cur) == hipSuccess && cur != prev) (void)hipSetDevice(prev);
    }
};

constexpr int64_t MAX_WIDTH = (int64_t)1 << 22;
constexpr int64_t MAX_ROWS = (int64_t)1 << 24;

size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

bool misaligned(const void* p, unsigned a) { return ((uintptr_t)p & (a - 1)) != 0; }

// A 2-d operand of the norm: rows of H elements `ld` apart.
int check_rows(const char* name, const void* p, int64_t ld, int64_t H) {
    if (!p || misaligned(p, 2)) return fail(MLP_EINVAL, "%s must be a non-NULL 2-byte aligned device pointer", name);
    if (ld < H || ld > MAX_WIDTH * 4)
        return fail(MLP_EINVAL, "the row stride of %s must be in %lld..%lld elements, got %lld", name, (long long)H,
                    (long long)(MAX_WIDTH * 4), (long long)ld);
    return MLP_OK;
}

// A 2-d operand of the linear layer: 16-byte rows of `width` elements.
int check_matrix(const char* name, const void* p, int64_t ld, int64_t width) {
    if (!p || misaligned(p, 16)) return fail(MLP_EINVAL, "%s must be a non-NULL 16-byte aligned device pointer", name);
    if (ld < width || ld % 8 || ld > MAX_WIDTH * 2)
        return fail(MLP_EINVAL, "the row stride of %s must be a multiple of 8 in %lld..%lld elements, got %lld", name,
                    (long long)width, (long long)(MAX_WIDTH * 2), (long long)ld);
    return MLP_OK;
}

int check_rows_count(int64_t rows, int64_t most) {
    if (rows < 0 || rows > most)
        return fail(MLP_EINVAL, "rows must be in 0..%lld, got %lld", (long long)most, (long long)rows);
    return MLP_OK;
}

int check_dtype(int dtype) {
    if (dtype != MLP_DTYPE_F16 && dtype != MLP_DTYPE_BF16) return fail(MLP_EINVAL, "unknown dtype %d", dtype);
    return MLP_OK;
}

// Argument checks shared by create and plan.
int check_linear(int64_t rows, int64_t K, int64_t N, int act) {
    if (rows < 1 || rows > MAX_ROWS || K < 8 || N < 8 || K >= MAX_WIDTH || N >= MAX_WIDTH)
        return fail(MLP_EINVAL, "sizes must be rows in 1..%lld, K and N in 8..%lld (got rows=%lld K=%lld N=%lld)",
                    (long long)MAX_ROWS, (long long)(MAX_WIDTH - 8), (long long)rows, (long long)K, (long long)N);
    if (K % 8 != 0 || N % 8 != 0)
        return fail(MLP_EINVAL, "K and N must be multiples of 8 (16-byte rows), got K=%lld N=%lld", (long long)K,
                    (long long)N);
    if (act < MLP_ACT_NONE || act > MLP_ACT_SWIGLU) return fail(MLP_EINVAL, "unknown activation %d", act);
    return MLP_OK;
}

int current_device(int* dev) {
    const hipError_t e = hipGetDevice(dev);
    return e == hipSuccess ? MLP_OK : fail(MLP_EHIP, "no HIP device: %s", hipGetErrorString(e));
}

int launched(hipError_t e) {
    return e == hipSuccess ? MLP_OK : fail(MLP_EHIP, "kernel launch failed: %s", hipGetErrorString(e));
}

// ------------------------------------------------------------------ planner

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

// Estimated microseconds of a plan, fitted to sweeps of every configuration
// and split over the package's sizes and rows from 1 to 8192 (the cheapest
// plan by this estimate is within 6% of the fastest measured on all but one of
// them).  A workgroup takes `slab` microseconds per 64-deep slab with several
// rounds of workgroups, `alone` times that with a single one, and `fixed` for
// its prologue and epilogue.  Operands that no other running workgroup reads
// too arrive at 6.8 MB per microsecond in all and 35 KB per CU (caches
// included).  The chip's power caps the multiplication rate whatever the
// schedule: `cap` MFLOP per microsecond.  A split adds a launch and the
// partials' way out and back.  Small products take no less than the host's
// time for their launches.
double plan_cost(const Plan& p, int64_t M, int64_t N, int64_t K, int cus) {
    static const double slab[] = {0.36, 0.38, 0.54, 0.84, 1.42, 0.98, 0.61, 0.86};
    static const double alone[] = {1.07, 1.31, 0.96, 0.92, 0.91, 0.80, 1.12, 1.0};
    static const double fixed[] = {1.7, 1.1, 3.2, 6.3, 10.7, 6.0, 1.6, 2.8};
    static const double cap[] = {1150, 1150, 876, 1100, 1227, 1070, 1150, 1150};
    const mlpc::LinearCfgInfo c = mlpc_linear_config(p.cfg);
    const uint32_t slabs = (uint32_t)(K / mlpc::BK), tiles = p.Mt * p.Nt;
    const double bytes = 128.0 * ((double)c.BN / p.Mt + (double)c.BM / p.Nt);
    // rounds of `count` workgroups of `n` slabs each
    auto rounds = [&](double count, uint32_t n) {
        const double r = ceil(count / cus), active = count < cus ? count : cus;
        const double compute = slab[p.cfg] * (tiles * p.S <= (uint32_t)cus ? alone[p.cfg] : 1.0);
        return r * (fixed[p.cfg] + n * fmax(compute, fmax(bytes * active / 6.8e6, bytes / 35.4e3)));
    };
    const double power = (double)tiles * c.BM * c.BN * K * 2e-6 / cap[p.cfg];
    if (p.S == 1) {
        // (the host's floor, with the estimate itself to tell such plans apart)
        const double cost = fmax(rounds(tiles, slabs), power);
        return fmax(cost, 6.0) + 0.01 * cost;
    }
    const double split = tiles - p.direct;
    const double values = split * c.BM * c.BN * fmin(1.0, (double)M / ((double)p.Mt * c.BM)) * fmin(1.0, (double)N / ((double)p.Nt * c.BN));
    const double cost = fmax(rounds(p.direct, slabs) + rounds(split * p.S, p.ksp), power) + 3.2 + values * 4 * p.S * 2 / 4.2e6;
    return fmax(cost, 9.0) + 0.01 * cost;
}

Plan choose_plan(int64_t M, int64_t N, int64_t K, int pass, int cus) {
    Plan best{};
    double cost = 0.0;
    bool found = false;
    for (int cfg = 0; cfg < mlpc_linear_num_configs(); ++cfg) {
        if (!mlpc_linear_has(cfg, pass)) continue;
        // (x^T dz has no short tiles)
        if (pass != mlpc::PASS_DW && !config_fits(mlpc_linear_config(cfg), M)) continue;
        uint32_t last = 0;
        for (uint32_t split = 1; split <= MAX_SPLIT; ++split) {
            const Plan p = make_plan(cfg, M, N, K, split, cus);
            if (p.S == last) continue;
            last = p.S;
            if (!split_fits(p, cus)) break;
            const double c = plan_cost(p, M, N, K, cus);
            if (!found || c < cost) {
                best = p;
                cost = c;
                found = true;
            }
        }
    }
    return best;
}

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

// Estimated microseconds of both products of the gradient in one launch, dz
// W^T's workgroups first.  As plan_cost, with constants of its own fitted to
// 190 sizes of 1 to 8192 rows (over 118 others the chosen plan is 1.4% slower
// than the fastest on average, at worst 25%: small ones the launches bound); workgroups of different lengths share a CU, so the chip is `room`
// places per CU on which each takes that much longer.
double both_cost(const Plan (&p)[2], int64_t rows, int64_t K, int64_t N, int cus) {
    static const double slab[] = {0, 0.42, 0.57, 0.81, 1.59, 0.95, 0.74, 0};
    static const double alone[] = {0, 1.0, 0.79, 0.98, 0.98, 0.57, 1.92, 0};
    static const double fixed[] = {0, 1.3, 3.0, 4.2, 7.8, 7.0, 1.2, 0};
    static const double cap[] = {1, 1080, 770, 960, 1210, 1500, 1150, 1};
    static const int per_cu[] = {0, 2, 1, 1, 1, 1, 3, 0};
    const int cfg = p[0].cfg;
    const mlpc::LinearCfgInfo c = mlpc_linear_config(cfg);
    double total = 0.0;
    for (const Plan& q : p) total += q.direct + (double)(q.Mt * q.Nt - q.direct) * q.S;
    const double active = total < cus ? total : cus;
    const double room = 1.0 + 0.42 * (fmin(per_cu[cfg], ceil(total / cus)) - 1.0);
    double group[4][2], power = 0.0, join = 0.0, launches = 6.0;
    int groups = 0;
    for (int i = 0; i < 2; ++i) {
        const Plan& q = p[i];
        const int64_t m = i ? K : rows, n = i ? N : K, k = i ? rows : N;
        const double bytes = 128.0 * ((double)c.BN / q.Mt + (double)c.BM / q.Nt), split = (double)(q.Mt * q.Nt) - q.direct;
        const double per = fmax(slab[cfg] * (total <= cus ? alone[cfg] : 1.0), fmax(bytes * active / 6.8e6, bytes / 35.4e3));
        const double whole = room * (fixed[cfg] + ((double)(k / mlpc::BK) + (k % mlpc::BK ? 0.4 : 0.0)) * per);
        power += (double)q.Mt * q.Nt * c.BM * c.BN * k * 2e-6 / cap[cfg];
        if (q.S == 1 || q.direct) {
            group[groups][0] = q.S == 1 ? q.direct + split : q.direct;
            group[groups++][1] = whole;
        }
        if (q.S == 1) continue;
        group[groups][0] = split * q.S;
        group[groups++][1] = room * (fixed[cfg] + q.ksp * per);
        const double values = split * c.BM * c.BN * fmin(1.0, (double)m / ((double)q.Mt * c.BM)) * fmin(1.0, (double)n / ((double)q.Nt * c.BN));
        join += 6.9 + values * 4 * q.S * 2 / 6.2e6;
        launches += 2.6;
    }
    const double run = dealt(group, groups, floor(cus * room));
    const double memory = 2.0 * (2.0 * rows * K + 2.0 * K * N + (double)rows * N) / 4.2e6;
    return fmax(fmax(run, fmax(power, memory)) + join, launches) + 0.01 * (run + join);
}

// Both products of the gradient in one launch, always: against launches of
// their own, over 118 sizes of 1 to 8192 rows drawn after the fit, 24% less time
// on average, at worst 6% more.  At most one of the two is split.
void choose_both(int64_t rows, int64_t K, int64_t N, int cus, Plan (&best)[2]) {
    double cost = 0.0;
    bool found = false;
    for (int cfg = 0; cfg < mlpc_linear_num_configs(); ++cfg) {
        if (!mlpc_linear_has(cfg, mlpc::PASS_BOTH_DX) || !config_fits(mlpc_linear_config(cfg), rows)) continue;
        for (int which = 0; which < 2; ++which) {
            uint32_t last = which;      // (unsplit plans once)
            for (uint32_t split = 1; split <= MAX_SPLIT; ++split) {
                const Plan p[2] = {make_plan(cfg, rows, K, N, which ? 1 : split, cus),
                                   make_plan(cfg, K, N, rows, which ? split : 1, cus)};
                if (p[which].S == last) continue;
                last = p[which].S;
                if (!split_fits(p[which], cus)) break;
                const double c = both_cost(p, rows, K, N, cus);
                if (!found || c < cost) {
                    best[0] = p[0];
                    best[1] = p[1];
                    cost = c;
                    found = true;
                }
            }
        }
    }
}

// Rows, columns and reduction of a pass.
void pass_sizes(int pass, int64_t rows, int64_t K, int64_t gN, int64_t* m, int64_t* n, int64_t* k) {
    *m = pass == mlpc::PASS_DW ? K : rows;
    *n = pass == mlpc::PASS_DX ? K : gN;
    *k = pass == mlpc::PASS_FWD ? K : pass == mlpc::PASS_DX ? gN : rows;
}

// Largest split workspace of any plan for up to max_rows rows.
size_t max_part_bytes(int64_t max_rows, int64_t K, int64_t gN, bool grad, int cus) {
    size_t most = 0;
    for (int pass = 0; pass < (grad ? 3 : 1); ++pass)
        for (int cfg = 0; cfg < mlpc_linear_num_configs(); ++cfg) {
            int64_t m, n, k;
            pass_sizes(pass, max_rows, K, gN, &m, &n, &k);
            const mlpc::LinearCfgInfo c = mlpc_linear_config(cfg);
            if (!mlpc_linear_has(cfg, pass) || (pass != mlpc::PASS_DW && !config_fits(c, m))) continue;
            const size_t slabs = (size_t)(k / mlpc::BK);
            if (slabs < 2) continue;
            size_t parts = (size_t)((m + c.BM - 1) / c.BM) * (size_t)((n + c.BN - 1) / c.BN) * (slabs < MAX_SPLIT ? slabs : MAX_SPLIT);
            if (parts > (size_t)cus) parts = (size_t)cus;
            const size_t b = parts * c.BM * c.BN * 4;
            if (b > most) most = b;
        }
    return most;
}

// A product's tiles, parts and its share of the workspace.
void set_plan(mlp_linear* h, const Plan& p, size_t part_offset, mlpc::GemmArgs& a) {
    const mlpc::LinearCfgInfo c = mlpc_linear_config(p.cfg);
    a.Mt = p.Mt;
    a.Nt = p.Nt;
    a.direct = p.direct;
    a.S = p.S;
    a.ksp = p.ksp;
    a.BM = c.BM;
    a.BN = c.BN;
    a.part = h->part + part_offset / sizeof(float);
    a.zero = h->zero;
}

int run_product(mlp_linear* h, int pass, int64_t rows, mlpc::GemmArgs& a, hipStream_t s) {
    const int64_t n = a.up ? (int64_t)a.N + a.up : a.N;
    if (h->plan_rows[pass] != rows) {
        h->plan[pass] = h->forced_cfg[pass] < 0
                            ? choose_plan(a.M, n, a.K, pass, h->cus)
                            : make_plan(h->forced_cfg[pass], a.M, n, a.K, (uint32_t)h->forced_split[pass], h->cus);
        h->plan_rows[pass] = rows;
    }
    const Plan& p = h->plan[pass];
    if (p.part_bytes > h->part_bytes)
        return fail(MLP_EINVAL, "the split needs %zu workspace bytes of %zu", p.part_bytes, h->part_bytes);
    set_plan(h, p, 0, a);
    hipError_t e = mlpc_gemm(a, p.cfg, pass, h->dtype, s);
    if (e == hipSuccess && p.S > 1) e = mlpc_gemm_reduce(a, h->dtype, s);
    return e == hipSuccess ? MLP_OK : fail(MLP_EHIP, "kernel launch failed: %s", hipGetErrorString(e));
}

// Both products of the gradient.
int run_both(mlp_linear* h, int64_t rows, mlpc::GemmArgs& dx, mlpc::GemmArgs& dw, const mlpc::DzArgs& dz, hipStream_t s) {
    Plan (&p)[2] = h->both;
    if (h->plan_rows[mlpc::PASS_BOTH_DX] != rows) {
        const int cfg = h->forced_cfg[mlpc::PASS_BOTH_DX];
        if (cfg < 0) {
            choose_both(rows, h->K, h->gN, h->cus, p);
        } else {
            p[0] = make_plan(cfg, rows, h->K, h->gN, (uint32_t)h->forced_split[mlpc::PASS_BOTH_DX], h->cus);
            p[1] = make_plan(cfg, h->K, h->gN, rows, (uint32_t)h->forced_split[mlpc::PASS_BOTH_DW], h->cus);
        }
        h->plan_rows[mlpc::PASS_BOTH_DX] = rows;
    }
    if (p[0].part_bytes + p[1].part_bytes > h->part_bytes)
        return fail(MLP_EINVAL, "the splits need %zu workspace bytes of %zu", p[0].part_bytes + p[1].part_bytes, h->part_bytes);
    set_plan(h, p[0], 0, dx);
    set_plan(h, p[1], p[0].part_bytes, dw);
    hipError_t e = mlpc_gemm_both(dx, dw, dz, p[0].cfg, h->dtype, s);
    if (e == hipSuccess && p[0].S > 1) e = mlpc_gemm_reduce(dx, h->dtype, s);
    if (e == hipSuccess && p[1].S > 1) e = mlpc_gemm_reduce(dw, h->dtype, s);
    return launched(e);
}

// Wait for the handle's last call and release its workspace.
int release(int device, hipStream_t last, void* ws) {
    DeviceGuard g(device);
    const hipError_t e1 = hipStreamSynchronize(last);
    const hipError_t e2 = ws ? hipFree(ws) : hipSuccess;
    if (e1 != hipSuccess || e2 != hipSuccess)
        return fail(MLP_EHIP, "destroy: %s", hipGetErrorString(e1 != hipSuccess ? e1 : e2));
    return MLP_OK;
}

}  // namespace

extern "C" {

mlp_norm_t mlp_norm_create(int64_t H, int dtype, float eps, int grad) {
    if (H < 1 || H > MAX_WIDTH) {
        fail(MLP_EINVAL, "H must be in 1..%lld, got %lld", (long long)MAX_WIDTH, (long long)H);
        return nullptr;
    }
    if (check_dtype(dtype) != MLP_OK) return nullptr;
    if (!(eps >= 0.f) || isinf(eps)) {
        fail(MLP_EINVAL, "eps must be finite and not negative, got %g", (double)eps);
        return nullptr;
    }
    int dev = 0;
    if (current_device(&dev) != MLP_OK) return nullptr;
    mlp_norm* h = new (std::nothrow) mlp_norm();
    if (!h) {
        fail(MLP_ENOMEM, "out of host memory");
        return nullptr;
    }
    h->H = (int)H;
    h->dtype = dtype;
    h->device = dev;
    h->eps = eps;
    hipError_t e = hipDeviceGetAttribute(&h->cus, hipDeviceAttributeMultiprocessorCount, dev);
    if (e != hipSuccess) {
        fail(MLP_EHIP, "hipDeviceGetAttribute failed: %s", hipGetErrorString(e));
        delete h;
        return nullptr;
    }
    const size_t bytes = grad ? (size_t)mlpc_norm_max_parts(h->H, h->cus) * 2 * H * sizeof(float) : 0;
    if (bytes) e = hipMalloc(reinterpret_cast<void**>(&h->part), bytes);
    if (e != hipSuccess) {
        fail(MLP_ENOMEM, "hipMalloc of %zu workspace bytes failed: %s", bytes, hipGetErrorString(e));
        delete h;
        return nullptr;
    }
    return h;
}

int mlp_norm_forward(mlp_norm_t h, int64_t rows, const void* x, int64_t ldx, const void* weight, const void* bias,
                     void* y, int64_t ldy, float* mean, float* rstd, void* hip_stream) {
    if (!h) return fail(MLP_EINVAL, "NULL handle");
    int rc = check_rows_count(rows, MAX_ROWS);
    if (rc != MLP_OK || rows == 0) return rc;
    rc = check_rows("x", x, ldx, h->H);
    if (rc == MLP_OK) rc = check_rows("y", y, ldy, h->H);
    if (rc != MLP_OK) return rc;
    if (misaligned(weight, 2) || misaligned(bias, 2) || misaligned(mean, 4) || misaligned(rstd, 4))
        return fail(MLP_EINVAL, "weight and bias must be 2-byte aligned, mean and rstd 4-byte aligned");
    DeviceGuard g(h->device);
    if (!g.ok) return fail(MLP_EHIP, "cannot select the handle's device %d", h->device);
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    h->last_stream = s;
    mlpc::NormArgs a{};
    a.x = static_cast<const uint16_t*>(x);
    a.weight = static_cast<const uint16_t*>(weight);
    a.bias = static_cast<const uint16_t*>(bias);
    a.y = static_cast<uint16_t*>(y);
    a.mean = mean;
    a.rstd = rstd;
    a.rows = rows;
    a.ldx = ldx;
    a.ldy = ldy;
    a.H = h->H;
    a.eps = h->eps;
    return launched(mlpc_norm_forward(a, h->dtype, h->cus, s));
}

int mlp_norm_backward(mlp_norm_t h, int64_t rows, const void* dy, int64_t lddy, const void* x, int64_t ldx,
                      const void* weight, const float* mean, const float* rstd, const void* dres, int64_t lddres,
                      void* dx, int64_t lddx, void* dweight, void* dbias, void* hip_stream) {
    if (!h) return fail(MLP_EINVAL, "NULL handle");
    if (!h->part) return fail(MLP_EINVAL, "the handle was created without its gradient");
    int rc = check_rows_count(rows, MAX_ROWS);
    const bool any = rc == MLP_OK && rows > 0;
    if (any) rc = check_rows("dy", dy, lddy, h->H);
    if (any && rc == MLP_OK) rc = check_rows("x", x, ldx, h->H);
    if (any && rc == MLP_OK) rc = check_rows("dx", dx, lddx, h->H);
    if (any && rc == MLP_OK && dres) rc = check_rows("dres", dres, lddres, h->H);
    if (rc != MLP_OK) return rc;
    if (any && (!mean || !rstd || misaligned(mean, 4) || misaligned(rstd, 4)))
        return fail(MLP_EINVAL, "mean and rstd must be non-NULL 4-byte aligned device pointers");
    if (misaligned(weight, 2) || misaligned(dweight, 2) || misaligned(dbias, 2))
        return fail(MLP_EINVAL, "weight, dweight and dbias must be 2-byte aligned");
    if (any && dres == dx && lddres != lddx) return fail(MLP_EINVAL, "dx in dres's buffer needs dres's row stride");
    DeviceGuard g(h->device);
    if (!g.ok) return fail(MLP_EHIP, "cannot select the handle's device %d", h->device);
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    h->last_stream = s;
    if (rows == 0 && !dweight && !dbias) return MLP_OK;
    mlpc::NormArgs a{};
    a.x = static_cast<const uint16_t*>(x);
    a.weight = static_cast<const uint16_t*>(weight);
    a.dy = static_cast<const uint16_t*>(dy);
    a.dres = static_cast<const uint16_t*>(dres);
    a.dx = static_cast<uint16_t*>(dx);
    a.mean = const_cast<float*>(mean);
    a.rstd = const_cast<float*>(rstd);
    a.dweight = static_cast<uint16_t*>(dweight);
    a.dbias = static_cast<uint16_t*>(dbias);
    a.part = h->part;
    a.rows = rows;
    a.ldx = ldx;
    a.lddy = lddy;
    a.lddres = lddres;
    a.lddx = lddx;
    a.H = h->H;
    a.parts = mlpc_norm_parts(rows, h->H, h->cus);
    return launched(mlpc_norm_backward(a, h->dtype, s));
}

int mlp_norm_destroy(mlp_norm_t h) {
    if (!h) return MLP_OK;
    const int rc = release(h->device, h->last_stream, h->part);
    delete h;
    return rc;
}

mlp_linear_t mlp_linear_create(int64_t max_rows, int64_t K, int64_t N, int act, int dtype, int grad) {
    if (check_linear(max_rows, K, N, act) != MLP_OK) return nullptr;
    if (check_dtype(dtype) != MLP_OK) return nullptr;
    int dev = 0;
    if (current_device(&dev) != MLP_OK) return nullptr;
    mlp_linear* h = new (std::nothrow) mlp_linear();
    if (!h) {
        fail(MLP_ENOMEM, "out of host memory");
        return nullptr;
    }
    h->max_rows = max_rows;
    h->K = (int)K;
    h->N = (int)N;
    h->gN = (int)(act == MLP_ACT_SWIGLU ? 2 * N : N);
    h->act = act;
    h->dtype = dtype;
    h->device = dev;
    for (int i = 0; i < mlpc::PASSES; ++i) {
        h->forced_cfg[i] = -1;
        h->forced_split[i] = 0;
        h->plan_rows[i] = -1;
    }
    hipError_t e = hipDeviceGetAttribute(&h->cus, hipDeviceAttributeMultiprocessorCount, dev);
    if (e != hipSuccess) {
        fail(MLP_EHIP, "hipDeviceGetAttribute failed: %s", hipGetErrorString(e));
        delete h;
        return nullptr;
    }
    const size_t zero_b = 256;
    const size_t dz_b = !grad || act == MLP_ACT_NONE ? 0 : align_up((size_t)max_rows * h->gN * 2, 256);
    const size_t col_b = !grad ? 0 : align_up((size_t)mlpc_dz_max_parts() * h->gN * sizeof(float), 256);
    h->part_bytes = max_part_bytes(max_rows, K, h->gN, grad != 0, h->cus);
    const size_t bytes = zero_b + dz_b + col_b + h->part_bytes;
    e = hipMalloc(&h->ws, bytes);
    if (e != hipSuccess) {
        fail(MLP_ENOMEM, "hipMalloc of %zu workspace bytes failed: %s", bytes, hipGetErrorString(e));
        delete h;
        return nullptr;
    }
    char* p = static_cast<char*>(h->ws);
    h->zero = p;
    p += zero_b;
    h->dz = dz_b ? reinterpret_cast<uint16_t*>(p) : nullptr;
    p += dz_b;
    h->colsum = col_b ? reinterpret_cast<float*>(p) : nullptr;
    p += col_b;
    h->part = h->part_bytes ? reinterpret_cast<float*>(p) : nullptr;
    e = hipMemset(h->ws, 0, zero_b);
    if (e == hipSuccess) e = hipStreamSynchronize(nullptr);
    if (e != hipSuccess) {
        fail(MLP_EHIP, "clearing the workspace failed: %s", hipGetErrorString(e));
        (void)hipFree(h->ws);
        delete h;
        return nullptr;
    }
    return h;
}

int mlp_linear_forward(mlp_linear_t h, int64_t rows, const void* x, int64_t ldx, const void* w, int64_t ldw,
                       const void* bias, const void* residual, int64_t ldres, void* y, int64_t ldy, void* z,
                       int64_t ldz, void* hip_stream) {
    if (!h) return fail(MLP_EINVAL, "NULL handle");
    int rc = check_rows_count(rows, h->max_rows);
    if (rc != MLP_OK || rows == 0) return rc;
    rc = check_matrix("x", x, ldx, h->K);
    if (rc == MLP_OK) rc = check_matrix("w", w, ldw, h->gN);
    if (rc == MLP_OK) rc = check_matrix("y", y, ldy, h->N);
    if (rc == MLP_OK && residual) rc = check_matrix("residual", residual, ldres, h->N);
    if (rc == MLP_OK && z) rc = check_matrix("z", z, ldz, h->gN);
    if (rc != MLP_OK) return rc;
    if (misaligned(bias, 16)) return fail(MLP_EINVAL, "bias must be 16-byte aligned");
    if (residual == y && ldres != ldy) return fail(MLP_EINVAL, "y in the residual's buffer needs its row stride");
    DeviceGuard g(h->device);
    if (!g.ok) return fail(MLP_EHIP, "cannot select the handle's device %d", h->device);
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    h->last_stream = s;
    mlpc::GemmArgs a{};
    a.a = static_cast<const uint16_t*>(x);
    a.b = static_cast<const uint16_t*>(w);
    a.d = static_cast<uint16_t*>(y);
    a.lda = ldx;
    a.ldb = ldw;
    a.ldd = ldy;
    a.M = (int)rows;
    a.N = h->N;
    a.K = h->K;
    a.up = h->gN - h->N;
    a.act = h->act;
    a.bias = static_cast<const uint16_t*>(bias);
    a.res = static_cast<const uint16_t*>(residual);
    a.z = static_cast<uint16_t*>(z);
    a.ldr = ldres;
    a.ldz = ldz;
    return run_product(h, mlpc::PASS_FWD, rows, a, s);
}

int mlp_linear_backward(mlp_linear_t h, int64_t rows, const void* dy, int64_t lddy, const void* x, int64_t ldx,
                        const void* w, int64_t ldw, const void* z, int64_t ldz, void* dx, int64_t lddx, void* dw,
                        int64_t lddw, void* db, void* hip_stream) {
    if (!h) return fail(MLP_EINVAL, "NULL handle");
    if (!h->colsum) return fail(MLP_EINVAL, "the handle was created without its gradient");
    const bool act = h->act != MLP_ACT_NONE;
    int rc = check_rows_count(rows, h->max_rows);
    const bool any = rc == MLP_OK && rows > 0;
    if (any) rc = check_matrix("dy", dy, lddy, h->N);
    if (any && rc == MLP_OK && act) rc = check_matrix("z", z, ldz, h->gN);
    if (any && rc == MLP_OK && dx) rc = check_matrix("dx", dx, lddx, h->K);
    if (any && rc == MLP_OK && dx) rc = check_matrix("w", w, ldw, h->gN);
    if (any && rc == MLP_OK && dw) rc = check_matrix("x", x, ldx, h->K);
    if (rc == MLP_OK && dw) rc = check_matrix("dw", dw, lddw, h->gN);
    if (rc != MLP_OK) return rc;
    if (misaligned(db, 16)) return fail(MLP_EINVAL, "db must be 16-byte aligned");
    DeviceGuard g(h->device);
    if (!g.ok) return fail(MLP_EHIP, "cannot select the handle's device %d", h->device);
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    h->last_stream = s;
    const uint16_t* dz = static_cast<const uint16_t*>(dy);
    int64_t lddz = lddy;
    const bool both = dx && dw && rows > 0 && h->forced_cfg[mlpc::PASS_DX] < 0 && h->forced_cfg[mlpc::PASS_DW] < 0;
    mlpc::DzArgs d{};
    if (db || (act && (dx || dw) && rows > 0)) {
        d.dy = dz;
        d.z = static_cast<const uint16_t*>(z);
        d.dz = h->dz;
        d.db = static_cast<uint16_t*>(db);
        d.part = h->colsum;
        d.lddy = lddy;
        d.ldz = ldz;
        d.lddz = h->gN;
        d.rows = rows;
        d.N = h->N;
        d.act = h->act;
        d.parts = mlpc_dz_parts(rows);
        rc = launched(mlpc_dz(d, h->dtype, !both, s));
        if (rc != MLP_OK) return rc;
        if (d.parts == 1) d.db = nullptr;
    }
    if (act) {
        dz = h->dz;
        lddz = h->gN;
    }
    mlpc::GemmArgs a{}, b{};
    if (dx && rows > 0) {
        a.a = dz;
        a.b = static_cast<const uint16_t*>(w);
        a.d = static_cast<uint16_t*>(dx);
        a.lda = lddz;
        a.ldb = ldw;
        a.ldd = lddx;
        a.M = (int)rows;
        a.N = h->K;
        a.K = h->gN;
    }
    if (dw) {
        b.a = static_cast<const uint16_t*>(x);
        b.b = dz;
        b.d = static_cast<uint16_t*>(dw);
        b.lda = ldx;
        b.ldb = lddz;
        b.ldd = lddw;
        b.M = h->K;
        b.N = h->gN;
        b.K = (int)rows;
    }
    if (both)
        return run_both(h, rows, a, b, d, s);
    if (dx && rows > 0) rc = run_product(h, mlpc::PASS_DX, rows, a, s);
    if (rc == MLP_OK && dw) rc = run_product(h, mlpc::PASS_DW, rows, b, s);
    return rc;
}

int mlp_linear_plan(int64_t rows, int64_t K, int64_t N, int act, int pass, int cus, int64_t* plan, int n) {
    if (!plan || n < 3) return fail(MLP_EINVAL, "mlp_linear_plan needs an array of at least 3 slots");
    if (check_linear(rows, K, N, act) != MLP_OK) return MLP_EINVAL;
    if (pass < 0 || pass >= mlpc::PASSES) return fail(MLP_EINVAL, "unknown pass %d", pass);
    if (cus < 8) return fail(MLP_EINVAL, "cus must be >= 8, got %d", cus);
    const int64_t gN = act == MLP_ACT_SWIGLU ? 2 * N : N;
    Plan p;
    if (pass == mlpc::PASS_BOTH_DX || pass == mlpc::PASS_BOTH_DW) {
        Plan both[2];
        choose_both(rows, K, gN, cus, both);
        p = both[pass - mlpc::PASS_BOTH_DX];
    } else {
        int64_t m, nn, k;
        pass_sizes(pass, rows, K, gN, &m, &nn, &k);
        p = choose_plan(m, nn, k, pass, cus);
    }
    const mlpc::LinearCfgInfo c = mlpc_linear_config(p.cfg);
    const int64_t v[9] = {p.cfg, p.S, c.BM, c.BN, p.Mt, p.Nt, p.ksp, (int64_t)p.part_bytes, p.direct};
    for (int i = 0; i < n && i < 9; ++i) plan[i] = v[i];
    return MLP_OK;
}

int mlp_linear_debug_set_plan(mlp_linear_t h, int pass, int config_id, int split) {
    if (!h) return fail(MLP_EINVAL, "NULL handle");
    if (pass < 0 || pass >= mlpc::PASSES) return fail(MLP_EINVAL, "unknown pass %d", pass);
    if (config_id < -1 || config_id >= mlpc_linear_num_configs() || (config_id >= 0 && !mlpc_linear_has(config_id, pass)))
        return fail(MLP_EINVAL, "pass %d has no tile configuration %d", pass, config_id);
    if (split < 0 || split > (int)MAX_SPLIT || (config_id < 0 && split != 0))
        return fail(MLP_EINVAL, "a configuration's split must be in 0..%u, got %d", MAX_SPLIT, split);
    const bool both = pass == mlpc::PASS_BOTH_DX || pass == mlpc::PASS_BOTH_DW;
    const int other = both ? mlpc::PASS_BOTH_DX + mlpc::PASS_BOTH_DW - pass : pass;
    if (config_id < 0) h->forced_split[other] = 0;
    h->forced_cfg[pass] = h->forced_cfg[other] = config_id;
    h->forced_split[pass] = split;
    h->plan_rows[pass] = h->plan_rows[other] = -1;
    return MLP_OK;
}

int mlp_linear_destroy(mlp_linear_t h) {
    if (!h) return MLP_OK;
    const int rc = release(h->device, h->last_stream, h->ws);
    delete h;
    return rc;
}

}  // extern "C"

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
    hipStream_t last_stream;    // of the last gradient: the forward pass leaves the handle alone
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
    // an error of the runtime is reported here, not once more by the caller's
    // next look at the thread's last error
    if (code == MLP_EHIP || code == MLP_ENOMEM) (void)hipGetLastError();
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
// Row strides: offsets are 64-bit (2^24 rows of MAX_LD stay in range), but for
// the products' operands, whose DMA has 32-bit byte offsets within a tile: of up
// to 256 rows, or of 64 rows and all columns (at most 2^23) where the reduction
// runs across rows.
constexpr int64_t MAX_LD = (int64_t)1 << 36;
constexpr int64_t MAX_DMA_LD = (int64_t)1 << 23;

// The largest stride of a product's operand of `rows` rows.
int64_t dma_ld(int64_t rows) {
    const int64_t few = (((int64_t)1 << 31) - ((int64_t)1 << 24)) / (rows < 256 ? rows : 256);
    return few > MAX_DMA_LD ? few : MAX_DMA_LD;
}

size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

bool misaligned(const void* p, unsigned a) { return ((uintptr_t)p & (a - 1)) != 0; }

// A 2-d operand of the norm: rows of H elements `ld` apart.
int check_rows(const char* name, const void* p, int64_t ld, int64_t H) {
    if (!p || misaligned(p, 2)) return fail(MLP_EINVAL, "%s must be a non-NULL 2-byte aligned device pointer", name);
    if (ld < H || ld > MAX_LD)
        return fail(MLP_EINVAL, "the row stride of %s must be in %lld..%lld elements, got %lld", name, (long long)H,
                    (long long)MAX_LD, (long long)ld);
    return MLP_OK;
}

// A 2-d operand of the linear layer: 16-byte rows of `width` elements, at most `most` apart.
int check_matrix(const char* name, const void* p, int64_t ld, int64_t width, int64_t most) {
    if (!p || misaligned(p, 16)) return fail(MLP_EINVAL, "%s must be a non-NULL 16-byte aligned device pointer", name);
    if (ld < width || ld % 8 || ld > most)
        return fail(MLP_EINVAL, "the row stride of %s must be a multiple of 8 in %lld..%lld elements, got %lld", name,
                    (long long)width, (long long)most, (long long)ld);
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
// the host's time for their launches.
double plan_cost(const Work* w, int products, const Rates& t, int cus) {
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
        const double per = fmax(slab, fmax(bytes * active / (t.all * 1e6), bytes / (t.cu * 1e3)));
        power += tiles * c.BM * c.BN * K * 2e-6 / t.cap[cfg];
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
            const Work w = {make_plan(cfg, M, N, K, split, cus), M, N, K};
            if (w.p.S == last) continue;
            last = w.p.S;
            if (!split_fits(w.p, cus)) break;
            const double c = plan_cost(&w, 1, SINGLE, cus);
            if (!found || c < cost) {
                best = w.p;
                cost = c;
                found = true;
            }
        }
    }
    return best;
}

// Both products of the gradient in one launch, always: against launches of
// their own, over 80 sizes of 1 to 8192 rows drawn after the fit, 24% less time
// on average, at worst 17% more (6 x 4600 x 4856: 27 -> 32 us).  At most one of
// the two is split.
void choose_both(int64_t rows, int64_t K, int64_t N, int cus, Plan (&best)[2]) {
    double cost = 0.0;
    bool found = false;
    for (int cfg = 0; cfg < mlpc_linear_num_configs(); ++cfg) {
        if (!mlpc_linear_has(cfg, mlpc::PASS_BOTH_DX) || !config_fits(mlpc_linear_config(cfg), rows)) continue;
        for (int which = 0; which < 2; ++which) {
            uint32_t last = which;      // (unsplit plans once)
            for (uint32_t split = 1; split <= MAX_SPLIT; ++split) {
                const Work w[2] = {{make_plan(cfg, rows, K, N, which ? 1 : split, cus), rows, K, N},
                                   {make_plan(cfg, K, N, rows, which ? split : 1, cus), K, N, rows}};
                if (w[which].p.S == last) continue;
                last = w[which].p.S;
                if (!split_fits(w[which].p, cus)) break;
                const double c = plan_cost(w, 2, BOTH, cus);
                if (!found || c < cost) {
                    best[0] = w[0].p;
                    best[1] = w[1].p;
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

// Wait for the last call that used the workspace, if there is one, and release it.
int release(int device, hipStream_t last, void* ws) {
    if (!ws) return MLP_OK;
    DeviceGuard g(device);
    const hipError_t e1 = hipStreamSynchronize(last);
    const hipError_t e2 = hipFree(ws);
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
    rc = check_matrix("x", x, ldx, h->K, dma_ld(rows));
    if (rc == MLP_OK) rc = check_matrix("w", w, ldw, h->gN, MAX_DMA_LD);
    if (rc == MLP_OK) rc = check_matrix("y", y, ldy, h->N, MAX_LD);
    if (rc == MLP_OK && residual) rc = check_matrix("residual", residual, ldres, h->N, MAX_LD);
    if (rc == MLP_OK && z) rc = check_matrix("z", z, ldz, h->gN, MAX_LD);
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
    // (without an activation dy is dz, an operand of the products)
    if (any) rc = check_matrix("dy", dy, lddy, h->N, act ? MAX_LD : dma_ld(rows));
    if (any && rc == MLP_OK && act) rc = check_matrix("z", z, ldz, h->gN, MAX_LD);
    if (any && rc == MLP_OK && dx) rc = check_matrix("dx", dx, lddx, h->K, MAX_LD);
    if (any && rc == MLP_OK && dx) rc = check_matrix("w", w, ldw, h->gN, MAX_DMA_LD);
    if (any && rc == MLP_OK && dw) rc = check_matrix("x", x, ldx, h->K, dma_ld(rows));
    if (rc == MLP_OK && dw) rc = check_matrix("dw", dw, lddw, h->gN, MAX_LD);
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

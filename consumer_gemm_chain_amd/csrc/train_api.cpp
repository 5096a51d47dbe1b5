// train_api.cpp -- the C ABI declared in include/mlp_train.h: argument checks,
// workspace ownership and launches.
#include <hip/hip_runtime.h>

#include <float.h>
#include <math.h>
#include <stdint.h>

#include <new>

#include "../../include/mlp_train.h"
#include "api_checks.h"
#include "linear_plan.h"
#include "train_launch.h"

struct mlp_loss {
    int64_t max_rows;
    int H, V;
    int dtype, device, cus;
    bool grad;
    int forced_cfg[2], forced_split;    // logits, products; -1 / 0: the planner's
    struct {
        int64_t rows;                   // that the plan is for (-1: none)
        int outputs;                    // 1: dx, 2: dw
        int cfg_z, cfg;
        uint32_t parts;
    } forward_plan, plan;
    // workspace (one allocation)
    void* ws;
    void* zero;
    mlpc::LossInfo* info;
    int* place;
    mlpc::LossRow* row;
    uint16_t* packed;
    float2* part;
    float* picked;
    uint16_t* dz;
    float* sums;
    size_t dz_elems, sum_elems, part_elems;
    hipStream_t last_stream;
};

struct mlp_grad_norm {
    int dtype, device;
    double* part;               // [NORM_PARTS]
    hipStream_t last_stream;
};

struct mlp_adamw {
    int dtype, bits, device;
    double beta1, beta2, eps;
    uint32_t seed;
    mlpc::AdamStep* step;
    hipStream_t last_stream;
};

namespace {

constexpr size_t DZ_BYTES = (size_t)256 << 20;          // of a piece of dz
constexpr size_t SPLIT_BYTES = (size_t)64 << 20;        // of dx's sums in parts
constexpr int64_t MAX_PRODUCT = (int64_t)1 << 38;
constexpr int PIECE = 256;                              // columns of a piece: a multiple of this
constexpr int MIN_TILE = 128;                           // columns of the narrowest tile

uint32_t up_div(int64_t a, int64_t b) { return (uint32_t)((a + b - 1) / b); }

}  // namespace

extern "C" {

mlp_loss_t mlp_loss_create(int64_t max_rows, int64_t H, int64_t V, int dtype, int grad) {
    if (max_rows < 1 || max_rows > MAX_ROWS || H < 8 || H >= MAX_WIDTH || H % 8 || V < 1 || V >= MAX_WIDTH) {
        fail(MLP_EINVAL, "sizes must be max_rows in 1..%lld, H a multiple of 8 in 8..%lld, V in 1..%lld (got max_rows=%lld H=%lld V=%lld)",
             (long long)MAX_ROWS, (long long)(MAX_WIDTH - 8), (long long)(MAX_WIDTH - 1), (long long)max_rows, (long long)H,
             (long long)V);
        return nullptr;
    }
    // (with the largest tiles, 256 x 256 by 512 threads, a launch has at most 2^31 threads)
    if (max_rows > MAX_PRODUCT / V || max_rows > MAX_PRODUCT / H || H > MAX_PRODUCT / V) {
        fail(MLP_EINVAL, "max_rows V, max_rows H and H V must be at most 2^38 (got max_rows=%lld H=%lld V=%lld)", (long long)max_rows,
             (long long)H, (long long)V);
        return nullptr;
    }
    if (check_dtype(dtype) != MLP_OK) return nullptr;
    int dev = 0;
    if (current_device(&dev) != MLP_OK) return nullptr;
    mlp_loss* h = new (std::nothrow) mlp_loss();
    if (!h) {
        fail(MLP_ENOMEM, "out of host memory");
        return nullptr;
    }
    h->max_rows = max_rows;
    h->H = (int)H;
    h->V = (int)V;
    h->dtype = dtype;
    h->device = dev;
    h->grad = grad != 0;
    h->forced_cfg[0] = h->forced_cfg[1] = -1;
    h->forward_plan.rows = h->plan.rows = -1;
    hipError_t e = hipDeviceGetAttribute(&h->cus, hipDeviceAttributeMultiprocessorCount, dev);
    if (e != hipSuccess) {
        fail(MLP_EHIP, "hipDeviceGetAttribute failed: %s", hipGetErrorString(e));
        delete h;
        return nullptr;
    }
    const size_t R = (size_t)max_rows;
    h->part_elems = R * up_div(V, MIN_TILE);
    const size_t columns = ((size_t)V + PIECE - 1) / PIECE * PIECE;
    const size_t piece = DZ_BYTES / 2 / R / PIECE * PIECE;
    h->dz_elems = grad ? R * (piece < PIECE ? PIECE : piece > columns ? columns : piece) : 0;
    const size_t one = R * H * sizeof(float), split = one * 32 < SPLIT_BYTES ? one * 32 : SPLIT_BYTES;
    h->sum_elems = grad ? (one > split ? one : split) / sizeof(float) : 0;
    const size_t sizes[8] = {256, sizeof(mlpc::LossInfo), R * sizeof(int), R * sizeof(mlpc::LossRow), R * H * 2,
                             h->part_elems * sizeof(float2) + R * sizeof(float), h->dz_elems * 2, h->sum_elems * sizeof(float)};
    size_t at[9] = {0};
    for (int i = 0; i < 8; ++i) at[i + 1] = at[i] + align_up(sizes[i], 256);
    e = hipMalloc(&h->ws, at[8]);
    if (e != hipSuccess) {
        fail(MLP_ENOMEM, "hipMalloc of %zu workspace bytes failed: %s", at[8], hipGetErrorString(e));
        delete h;
        return nullptr;
    }
    char* p = static_cast<char*>(h->ws);
    h->zero = p;
    h->info = reinterpret_cast<mlpc::LossInfo*>(p + at[1]);
    h->place = reinterpret_cast<int*>(p + at[2]);
    h->row = reinterpret_cast<mlpc::LossRow*>(p + at[3]);
    h->packed = reinterpret_cast<uint16_t*>(p + at[4]);
    h->part = reinterpret_cast<float2*>(p + at[5]);
    h->picked = reinterpret_cast<float*>(h->part + h->part_elems);
    h->dz = reinterpret_cast<uint16_t*>(p + at[6]);
    h->sums = reinterpret_cast<float*>(p + at[7]);
    e = hipMemset(h->ws, 0, 256);
    if (e == hipSuccess) e = hipStreamSynchronize(nullptr);
    if (e != hipSuccess) {
        fail(MLP_EHIP, "clearing the workspace failed: %s", hipGetErrorString(e));
        (void)hipFree(h->ws);
        delete h;
        return nullptr;
    }
    return h;
}

}  // extern "C"

namespace {

int check_vector(const char* name, const void* p, unsigned align) {
    if (!p || misaligned(p, align))
        return fail(MLP_EINVAL, "%s must be a non-NULL %u-byte aligned device pointer", name, align);
    return MLP_OK;
}

int check_loss(const mlp_loss* h, int64_t rows, const void* x, int64_t ldx, const void* w, int64_t ldw,
               const int64_t* target) {
    int rc = check_matrix("x", x, ldx, h->H, dma_ld(rows));
    if (rc == MLP_OK) rc = check_matrix("w", w, ldw, h->H, MAX_DMA_LD);
    if (rc == MLP_OK) rc = check_vector("target", target, 8);
    return rc;
}

mlpc::LossArgs loss_args(const mlp_loss* h, int64_t rows, const void* x, int64_t ldx, const void* w, int64_t ldw,
                         const int64_t* target) {
    mlpc::LossArgs a{};
    a.rows = rows;
    a.H = h->H;
    a.V = h->V;
    a.x = static_cast<const uint16_t*>(x);
    a.ldx = ldx;
    a.w = static_cast<const uint16_t*>(w);
    a.ldw = ldw;
    a.target = target;
    a.info = h->info;
    a.place = h->place;
    a.row = h->row;
    a.packed = h->packed;
    a.part = h->part;
    a.picked = h->picked;
    a.dz = h->dz;
    a.sums = h->sums;
    a.zero = h->zero;
    a.cus = (uint32_t)h->cus;
    return a;
}

void set_logits(mlpc::LossArgs& a, int cfg, int v0, int vn) {
    const mlpc::LinearCfgInfo c = mlpc_linear_config(cfg);
    a.v0 = v0;
    a.vn = vn;
    a.Mt = up_div(a.rows, c.BM);
    a.Nt = up_div(vn, c.BN);
}

// The products run on tiles that the linear layer has for them, unsplit but for
// dx, and its estimates choose among these, with rates fitted to every
// configuration (and split) of 348 sizes (470 for dW alone) of 1 to 4096 rows.  On
// 120 sizes drawn afterwards (dW, dx alone: 580) the chosen tiles took 1.2% (z),
// 5.5% (both products), 4.1% (dx alone) and 1.7% (dW alone; 4.5% with both
// products' rates, 48 x 8192 x 32000 330 -> 245 us) longer than the fastest on
// average; with the linear layer's own rates z 2.7% and both products 7.0%.
const Rates LOGITS = {{0.586, 0.787, 0.732, 1.09, 2.2, 0.966, 0.658, 0},
                      {0.921, 0.845, 1.25, 1.16, 0.904, 1.47, 2.69, 0},
                      {1.66, 3.06, 5.84, 14.9, 23.8, 12.1, 3.19, 0},
                      {1140, 1150, 904, 1120, 1230, 1070, 1150, 1},
                      0.27, 5.49, 4.55, 3.02, 7.23, 2.43, 6.8, 35.8};
const Rates PRODUCTS = {{0, 0.408, 0.745, 0.799, 1.9, 1.24, 0.605, 0},
                        {0, 0.902, 0.951, 1.21, 0.799, 0.5, 1.82, 0},
                        {0, 1.39, 2.78, 7.66, 6.31, 12, 1.6, 0},
                        {1, 1080, 769, 595, 1210, 1500, 648, 1},
                        0.383, 2.32, 2.32, 0.428, 8.65, 3.3, 6.45, 107};
const Rates DW_ALONE = {{0, 0.624, 0.71, 0.596, 1.74, 1.08, 0.627, 0},
                        {0, 0.588, 0.608, 1.93, 1.14, 1, 1.85, 0},
                        {0, 1.04, 10.3, 11.8, 10.8, 11.1, 1.33, 0},
                        {1, 1080, 769, 687, 1210, 1500, 527, 1},
                        0.293, 4.33, 3.2, 1.45, 3.37, 4.52, 5.35, 106};
constexpr double PACK_US = 15.5;        // more than one row of tiles: rows are packed first

// A launch has fewer than 2^32 threads.
bool launchable(int cfg, int64_t blocks) { return blocks * mlpc_linear_config(cfg).NT < ((int64_t)1 << 32); }

// What the products of `rows` rows take of whole tiles' time.
double tall_part(int cfg, int64_t rows, uint32_t columns, int cus) {
    if (mlpc_linear_config(cfg).BM < 256 || mlpc_linear_config(cfg).BN < 256 || rows <= 256) return 1.0;
    const mlpc::Fragments f = mlpc::fragments_for((int)rows, columns, (uint32_t)cus);
    return f.cost / f.whole;
}

int logits_cfg(const mlp_loss* h, int64_t rows, int64_t vn) {
    if (h->forced_cfg[0] >= 0) return h->forced_cfg[0];
    int best = 4;
    double cost = 0.0;
    bool found = false;
    for (int cfg = 0; cfg < mlpc_linear_num_configs(); ++cfg) {
        if (!mlpc_linear_has(cfg, mlpc::PASS_DX) || !config_fits(mlpc_linear_config(cfg), rows)) continue;
        const Work w = {make_plan(cfg, rows, vn, h->H, 1, h->cus), rows, vn, h->H};
        if (!launchable(cfg, (int64_t)w.p.Mt * w.p.Nt * 2)) continue;
        const double c = plan_cost(&w, 1, LOGITS, h->cus, tall_part(cfg, rows, w.p.Nt, h->cus)) + (w.p.Mt > 1 ? PACK_US : 0.0);
        if (!found || c < cost) best = cfg, cost = c, found = true;
    }
    return best;
}

// Tile configuration of both products of a piece, and the parts of dx's
// reduction, at most `room`: dx's tiles have long reductions and may be few.
int products_cfg(const mlp_loss* h, int64_t rows, int64_t vn, bool dx, bool dw, int64_t room, uint32_t* parts) {
    int best = 4;
    double cost = 0.0;
    bool found = false;
    *parts = 1;
    for (int cfg = 0; cfg < mlpc_linear_num_configs(); ++cfg) {
        if (h->forced_cfg[1] >= 0 ? cfg != h->forced_cfg[1] : !mlpc_linear_has(cfg, mlpc::PASS_BOTH_DX)) continue;
        uint32_t last = 0;
        for (int64_t S = 1; S <= 32 && S <= room; ++S) {
            if (h->forced_split > 0 && S != h->forced_split && S < room) continue;
            Work w[2] = {{make_plan(cfg, rows, h->H, vn, (uint32_t)S, h->cus), rows, h->H, vn},
                         {make_plan(cfg, vn, h->H, rows, 1, h->cus), vn, h->H, rows}};
            if (w[0].p.S == last) continue;
            last = w[0].p.S;
            if (!launchable(cfg, ((int64_t)w[0].p.Mt * w[0].p.Nt * w[0].p.S + (int64_t)w[1].p.Mt * w[1].p.Nt) * 2)) continue;
            w[0].p.direct = 0;
            const double c = !dx ? plan_cost(w + 1, 1, DW_ALONE, h->cus)
                                 : plan_cost(w, dw ? 2 : 1, PRODUCTS, h->cus, tall_part(cfg, rows, 1, 0));
            if (!found || c < cost) best = cfg, cost = c, *parts = (uint32_t)S, found = true;
            if (!dx) break;
        }
    }
    return best;
}

}  // namespace

extern "C" {

int mlp_loss_forward(mlp_loss_t h, int64_t rows, const void* x, int64_t ldx, const void* w, int64_t ldw,
                     const int64_t* target, float* loss, float* lse, void* hip_stream) {
    if (!h) return fail(MLP_EINVAL, "NULL handle");
    int rc = check_rows_count(rows, h->max_rows);
    if (rc != MLP_OK || rows == 0) return rc;
    rc = check_loss(h, rows, x, ldx, w, ldw, target);
    if (rc == MLP_OK) rc = check_vector("lse", lse, 4);
    if (rc != MLP_OK) return rc;
    if (misaligned(loss, 4)) return fail(MLP_EINVAL, "loss must be 4-byte aligned");
    DeviceGuard g(h->device);
    if (!g.ok) return fail(MLP_EHIP, "cannot select the handle's device %d", h->device);
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    h->last_stream = s;
    mlpc::LossArgs a = loss_args(h, rows, x, ldx, w, ldw, target);
    a.loss = loss;
    a.lse = lse;
    if (h->forward_plan.rows != rows) {
        h->forward_plan.cfg_z = logits_cfg(h, rows, h->V);
        h->forward_plan.rows = rows;
    }
    const int cfg = h->forward_plan.cfg_z;
    set_logits(a, cfg, 0, h->V);
    a.tiles = (int)a.Nt;
    a.packing = a.Mt > 1;
    hipError_t e = a.packing ? mlpc_loss_rows(a, false, h->dtype, s) : hipSuccess;
    if (e == hipSuccess) e = mlpc_loss_logits(a, cfg, false, h->dtype, s);
    if (e == hipSuccess) e = mlpc_loss_join(a, s);
    return launched(e);
}

int mlp_loss_backward(mlp_loss_t h, int64_t rows, const void* x, int64_t ldx, const void* w, int64_t ldw,
                      const int64_t* target, const float* lse, const float* dloss, const float* dlse, void* dx,
                      int64_t lddx, void* dw, int64_t lddw, void* hip_stream) {
    if (!h) return fail(MLP_EINVAL, "NULL handle");
    if (!h->grad) return fail(MLP_EINVAL, "the handle was created without its gradient");
    int rc = check_rows_count(rows, h->max_rows);
    const bool any = rc == MLP_OK && rows > 0;
    if (any) rc = check_loss(h, rows, x, ldx, w, ldw, target);
    if (any && rc == MLP_OK) rc = check_vector("lse", lse, 4);
    if (any && rc == MLP_OK && dx) rc = check_matrix("dx", dx, lddx, h->H, MAX_LD);
    if (rc == MLP_OK && dw) rc = check_matrix("dw", dw, lddw, h->H, MAX_LD);
    if (rc != MLP_OK) return rc;
    if (misaligned(dloss, 4) || misaligned(dlse, 4)) return fail(MLP_EINVAL, "dloss and dlse must be 4-byte aligned");
    DeviceGuard g(h->device);
    if (!g.ok) return fail(MLP_EHIP, "cannot select the handle's device %d", h->device);
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    h->last_stream = s;
    mlpc::LossArgs a = loss_args(h, rows, x, ldx, w, ldw, target);
    a.lse_in = lse;
    a.dloss = dloss;
    a.dlse = dlse;
    a.dx = rows > 0 ? static_cast<uint16_t*>(dx) : nullptr;
    a.dw = static_cast<uint16_t*>(dw);
    a.lddx = lddx;
    a.lddw = lddw;
    if (!a.dx && !a.dw) return MLP_OK;
    // pieces of equal width, as few as the workspace of dz allows
    const int64_t most = rows > 0 ? (int64_t)(h->dz_elems / (size_t)rows) / PIECE * PIECE : h->V;
    const uint32_t pieces = up_div(h->V, most);
    const int width = (int)(up_div(up_div(h->V, pieces), PIECE) * PIECE);
    a.lddz = width;
    const int outputs = (a.dx ? 1 : 0) | (a.dw ? 2 : 0);
    if (h->plan.rows != rows || h->plan.outputs != outputs) {
        const int64_t some = rows > 0 ? rows : 1, room = (int64_t)(h->sum_elems / ((size_t)some * h->H));
        h->plan.cfg_z = logits_cfg(h, some, width);
        h->plan.cfg = products_cfg(h, some, width, a.dx != nullptr, a.dw != nullptr, room, &h->plan.parts);
        h->plan.rows = rows;
        h->plan.outputs = outputs;
    }
    const int cfg_z = h->plan.cfg_z, cfg = h->plan.cfg;
    a.S = h->plan.parts;
    const mlpc::LinearCfgInfo c = mlpc_linear_config(cfg);
    a.dxNt = a.dwNt = up_div(h->H, c.BN);
    set_logits(a, cfg_z, 0, width);
    a.packing = a.Mt != 1;
    a.direct = !a.packing && pieces == 1 && a.S == 1;
    hipError_t e = a.packing ? mlpc_loss_rows(a, true, h->dtype, s) : hipSuccess;
    for (int64_t v0 = 0; v0 < h->V && e == hipSuccess; v0 += width) {
        const int vn = (int)(h->V - v0 < width ? h->V - v0 : width);
        set_logits(a, cfg_z, (int)v0, vn);
        a.first = v0 == 0;
        a.ksp = up_div(vn / 64, a.S);
        a.dwMt = up_div(vn, c.BM);
        if (rows > 0) e = mlpc_loss_logits(a, cfg_z, true, h->dtype, s);
        if (e == hipSuccess) e = mlpc_loss_products(a, cfg, h->dtype, s);
    }
    if (e == hipSuccess && a.dx && !a.direct) e = mlpc_loss_dx(a, h->dtype, s);
    return launched(e);
}

int mlp_loss_destroy(mlp_loss_t h) {
    if (!h) return MLP_OK;
    const int rc = release(h->device, h->last_stream, h->ws);
    delete h;
    return rc;
}

int mlp_loss_debug_set_plan(mlp_loss_t h, int product, int config_id, int split) {
    if (!h) return fail(MLP_EINVAL, "NULL handle");
    if (product < 0 || product > 1) return fail(MLP_EINVAL, "unknown product %d", product);
    if (config_id < -1 || config_id >= mlpc_linear_num_configs() ||
        (config_id >= 0 && !mlpc_linear_has(config_id, product ? mlpc::PASS_BOTH_DX : mlpc::PASS_DX)))
        return fail(MLP_EINVAL, "product %d has no tile configuration %d", product, config_id);
    if (split < 0 || split > 32) return fail(MLP_EINVAL, "the split must be in 0..32, got %d", split);
    h->forced_cfg[product] = config_id;
    h->forward_plan.rows = h->plan.rows = -1;
    if (product == 1) h->forced_split = split;
    return MLP_OK;
}

}  // extern "C"

namespace {

constexpr int64_t MAX_TENSORS = (int64_t)1 << 20;
// Of a tensor: one workgroup per chunk, and a launch has fewer than 2^32 threads.
constexpr int64_t MAX_ELEMENTS = (int64_t)1 << 34;
constexpr uint32_t MAX_CHUNKS = ((uint32_t)1 << 24) - 1;
// The largest beta1 with which an m of 8 bits is rounded to nearest.  A step
// without a gradient takes (1 - beta1) m away, and e4m3's half step is up to m / 18:
// from 17/18 on such an m would stay for good while v falls (0.95: 0.84 of m's norm
// is left after 400 steps, of which 1e-9 should be; 0.94: 1e-15).
constexpr double M_NEAREST = 15.0 / 16.0;

int check_count(int64_t count, const void* array) {
    if (count < 0 || count > MAX_TENSORS || (count > 0 && !array))
        return fail(MLP_EINVAL, "count must be in 0..%lld with arrays of as many, got %lld", (long long)MAX_TENSORS, (long long)count);
    return MLP_OK;
}

int check_elements(int64_t i, int64_t n) {
    if (n < 0 || n >= MAX_ELEMENTS)
        return fail(MLP_EINVAL, "tensor %lld has %lld elements, expected 0..2^34 - 1", (long long)i, (long long)n);
    return MLP_OK;
}

int check_element_pointer(const char* name, int64_t i, const void* p, unsigned align) {
    if (!p || misaligned(p, align))
        return fail(MLP_EINVAL, "%s of tensor %lld must be a non-NULL %u-byte aligned device pointer", name, (long long)i, align);
    return MLP_OK;
}

// A handle on the current device with `bytes` of workspace.
template <class T>
T* optimizer(int dtype, void** ws, size_t bytes, T* h) {
    if (!h) {
        fail(MLP_ENOMEM, "out of host memory");
        return nullptr;
    }
    h->dtype = dtype;
    int rc = current_device(&h->device);
    if (rc == MLP_OK) {
        const hipError_t e = hipMalloc(ws, bytes);
        if (e != hipSuccess) rc = fail(MLP_ENOMEM, "hipMalloc of %zu workspace bytes failed: %s", bytes, hipGetErrorString(e));
    }
    if (rc == MLP_OK) return h;
    delete h;
    return nullptr;
}

}  // namespace

extern "C" {

mlp_grad_norm_t mlp_grad_norm_create(int dtype) {
    if (check_dtype(dtype) != MLP_OK) return nullptr;
    mlp_grad_norm* h = new (std::nothrow) mlp_grad_norm();
    return optimizer(dtype, h ? reinterpret_cast<void**>(&h->part) : nullptr, mlpc::NORM_PARTS * sizeof(double), h);
}

int mlp_grad_norm_forward(mlp_grad_norm_t h, int64_t count, const int64_t* sizes, const void* const* grads,
                          double unscale, double max_norm, float* norm, float* scale, void* hip_stream) {
    if (!h) return fail(MLP_EINVAL, "NULL handle");
    int rc = check_count(count, sizes);
    if (rc == MLP_OK) rc = check_count(count, grads);
    int64_t chunks = 0;
    for (int64_t i = 0; i < count && rc == MLP_OK; ++i) {
        rc = check_elements(i, sizes[i]);
        if (rc == MLP_OK && sizes[i] > 0) rc = check_element_pointer("the gradient", i, grads[i], 2);
        if (rc == MLP_OK) chunks += (sizes[i] + mlpc::NORM_CHUNK - 1) / mlpc::NORM_CHUNK;
    }
    if (rc == MLP_OK) rc = check_vector("norm", norm, 4);
    if (rc != MLP_OK) return rc;
    if (misaligned(scale, 4)) return fail(MLP_EINVAL, "scale must be 4-byte aligned");
    // (beyond fp32's normal numbers the scale would be infinite or 0 beside a finite norm)
    if (!(fabs(unscale) >= FLT_MIN && fabs(unscale) <= FLT_MAX))
        return fail(MLP_EINVAL, "the magnitude of unscale must be a normal fp32 number, got %g", unscale);
    if (!(max_norm > 0.0)) return fail(MLP_EINVAL, "max_norm must be positive, got %g", max_norm);
    if (chunks > INT32_MAX) return fail(MLP_EINVAL, "the tensors have more than 2^44 elements");
    DeviceGuard g(h->device);
    if (!g.ok) return fail(MLP_EHIP, "cannot select the handle's device %d", h->device);
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    h->last_stream = s;
    const int parts = (int)(chunks < mlpc::NORM_PARTS ? chunks : mlpc::NORM_PARTS);
    mlpc::NormTable a{};
    a.part = h->part;
    hipError_t e = hipSuccess;
    for (int64_t i = 0; i < count && e == hipSuccess; ++i) {
        if (sizes[i] > 0) {
            a.grad[a.count] = static_cast<const uint16_t*>(grads[i]);
            a.n[a.count] = sizes[i];
            a.first[a.count++] = a.chunks;
            a.chunks += (uint32_t)((sizes[i] + mlpc::NORM_CHUNK - 1) / mlpc::NORM_CHUNK);
        }
        if (a.count == 0 || (a.count < mlpc::NormTable::MAX && i + 1 < count)) continue;
        e = mlpc_norm_sum(a, h->dtype, parts, s);
        a.add = true;
        a.count = 0;
        a.chunks = 0;
    }
    mlpc::NormJoin j{h->part, parts, unscale, max_norm, norm, scale};
    if (e == hipSuccess) e = mlpc_norm_join(j, s);
    return launched(e);
}

int mlp_grad_norm_destroy(mlp_grad_norm_t h) {
    if (!h) return MLP_OK;
    const int rc = release(h->device, h->last_stream, h->part);
    delete h;
    return rc;
}

mlp_adamw_t mlp_adamw_create(int dtype, int bits, double beta1, double beta2, double eps, uint32_t seed) {
    if (check_dtype(dtype) != MLP_OK) return nullptr;
    if (bits != 32 && bits != 8) {
        fail(MLP_EINVAL, "states have 32 or 8 bits, got %d", bits);
        return nullptr;
    }
    if (!(beta1 >= 0.0 && beta1 < 1.0 && beta2 >= 0.0 && beta2 < 1.0)) {
        fail(MLP_EINVAL, "beta1 and beta2 must be in [0, 1), got %g and %g", beta1, beta2);
        return nullptr;
    }
    // (a smaller one has no reciprocal in fp32: elements whose v is 0 would become NaN)
    if (!(eps == 0.0 || (eps >= 0x1p-126 && eps < INFINITY))) {
        fail(MLP_EINVAL, "eps must be finite and either 0 or at least 2^-126, got %g", eps);
        return nullptr;
    }
    mlp_adamw* h = new (std::nothrow) mlp_adamw();
    if (!optimizer(dtype, h ? reinterpret_cast<void**>(&h->step) : nullptr, sizeof(mlpc::AdamStep), h)) return nullptr;
    h->bits = bits;
    h->beta1 = beta1;
    h->beta2 = beta2;
    h->eps = eps;
    h->seed = seed;
    return h;
}

int mlp_adamw_step(mlp_adamw_t h, int64_t count, const mlp_adamw_tensor* tensors, const void* const* grads, double lr,
                   const float* lr_scale, const float* scale, int64_t* t, void* hip_stream) {
    if (!h) return fail(MLP_EINVAL, "NULL handle");
    int rc = check_count(count, tensors);
    if (rc == MLP_OK) rc = check_count(count, grads);
    if (rc == MLP_OK) rc = check_vector("t", t, 8);
    if (rc != MLP_OK) return rc;
    if (misaligned(lr_scale, 4) || misaligned(scale, 4)) return fail(MLP_EINVAL, "lr_scale and scale must be 4-byte aligned");
    if (!(fabs(lr) < INFINITY)) return fail(MLP_EINVAL, "lr must be finite, got %g", lr);
    for (int64_t i = 0; i < count && rc == MLP_OK; ++i) {
        const mlp_adamw_tensor& q = tensors[i];
        rc = check_elements(i, q.n);
        if (rc == MLP_OK && !(fabs(q.decay) < INFINITY)) rc = fail(MLP_EINVAL, "the decay of tensor %lld must be finite", (long long)i);
        if (rc != MLP_OK || q.n == 0) continue;
        const unsigned align = h->bits == 32 ? 4 : 1;
        rc = check_element_pointer("the gradient", i, grads[i], 2);
        if (rc == MLP_OK) rc = check_element_pointer("w", i, q.w, 2);
        if (rc == MLP_OK && q.master) rc = check_element_pointer("master", i, q.master, 4);
        if (rc == MLP_OK) rc = check_element_pointer("m", i, q.m, align);
        if (rc == MLP_OK) rc = check_element_pointer("v", i, q.v, align);
        if (rc == MLP_OK && h->bits == 8) rc = check_element_pointer("m_scale", i, q.m_scale, 4);
        if (rc == MLP_OK && h->bits == 8) rc = check_element_pointer("v_scale", i, q.v_scale, 4);
    }
    if (rc != MLP_OK) return rc;
    DeviceGuard g(h->device);
    if (!g.ok) return fail(MLP_EHIP, "cannot select the handle's device %d", h->device);
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    h->last_stream = s;
    const mlpc::AdamBegin b{h->step, t, scale, lr_scale, lr, h->beta1, h->beta2, h->seed};
    hipError_t e = mlpc_adamw_begin(b, s);
    mlpc::AdamTable a{};
    a.beta1 = (float)h->beta1;
    a.rest1 = (float)(1.0 - h->beta1);
    a.beta2 = (float)h->beta2;
    a.rest2 = (float)(1.0 - h->beta2);
    a.eps = (float)h->eps;
    a.chance = h->beta1 > M_NEAREST;
    a.step = h->step;
    for (int64_t i = 0; i < count && e == hipSuccess; ++i) {
        const mlp_adamw_tensor& q = tensors[i];
        const int k = a.count;
        if (k == 0) a.number = (int)i;
        // (an empty tensor keeps its place: random bits go by the tensor's number)
        a.grad[k] = static_cast<const uint16_t*>(grads[i]);
        a.w[k] = static_cast<uint16_t*>(q.w);
        a.master[k] = q.master;
        a.m[k] = q.m;
        a.v[k] = q.v;
        a.m_scale[k] = q.m_scale;
        a.v_scale[k] = q.v_scale;
        a.decay[k] = q.decay;
        a.n[k] = q.n;
        a.first[k] = a.chunks;
        a.chunks += (uint32_t)((q.n + mlpc::ADAM_CHUNK - 1) / mlpc::ADAM_CHUNK);
        a.count = k + 1;
        const int64_t next = i + 1 < count ? (tensors[i + 1].n + mlpc::ADAM_CHUNK - 1) / mlpc::ADAM_CHUNK : 0;
        if (a.count < mlpc::AdamTable::MAX && i + 1 < count && a.chunks + next <= MAX_CHUNKS) continue;
        if (a.chunks > 0) e = mlpc_adamw(a, h->dtype, h->bits, s);
        a.count = 0;
        a.chunks = 0;
    }
    return launched(e);
}

int mlp_adamw_destroy(mlp_adamw_t h) {
    if (!h) return MLP_OK;
    const int rc = release(h->device, h->last_stream, h->step);
    delete h;
    return rc;
}

}  // extern "C"

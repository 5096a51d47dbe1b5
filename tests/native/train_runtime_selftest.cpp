// Drives the training step's handles (train_api.cpp) on a stand-in for the HIP
// runtime and the launchers, defined here: no GPU and no HIP library are needed,
// every runtime call of an entry point can be seen and made to fail, and every
// launch's arguments are checked against the workspace that they use.  Prints
// "<n> failures" and exits 0 on success.
#include <math.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <map>
#include <vector>

#include "../../consumer_gemm_chain_amd/csrc/linear_configs.h"
#include "../../consumer_gemm_chain_amd/csrc/train_launch.h"
#include "../../include/mlp_train.h"

static int failures = 0;
static char last[512];
#define CHECK(c) do { if (!(c)) { ++failures; printf("line %d: %s (%s)\n", __LINE__, #c, last); } } while (0)

int mlpc_set_error(int code, const char* msg) {
    snprintf(last, sizeof last, "%s", msg);
    return code;
}

// ---------------------------------------------------------------- the runtime

static hipError_t pending = hipSuccess;             // the thread's last error
static hipError_t malloc_fails = hipSuccess, memset_fails = hipSuccess, sync_fails = hipSuccess, launch_fails = hipSuccess;
static std::vector<hipStream_t> waited;             // streams waited for
static std::map<char*, size_t> blocks;              // address ranges alive (never touched)
static char* next_block = reinterpret_cast<char*>((uintptr_t)1 << 40);

static hipError_t done(hipError_t e) {
    if (e != hipSuccess) pending = e;
    return e;
}

extern "C" {
hipError_t hipGetDevice(int* d) { *d = 0; return hipSuccess; }
hipError_t hipSetDevice(int) { return hipSuccess; }
hipError_t hipDeviceGetAttribute(int* v, hipDeviceAttribute_t, int) { *v = 256; return hipSuccess; }
hipError_t hipMalloc(void** p, size_t n) {
    if (malloc_fails != hipSuccess) return done(malloc_fails);
    *p = next_block;
    blocks[next_block] = n;
    next_block += (n + 65535) / 4096 * 4096;
    return hipSuccess;
}
hipError_t hipFree(void* p) {
    CHECK(blocks.erase(static_cast<char*>(p)) == 1);
    return hipSuccess;
}
hipError_t hipMemset(void*, int, size_t) { return done(memset_fails); }
hipError_t hipStreamSynchronize(hipStream_t s) {
    waited.push_back(s);
    return done(sync_fails);
}
hipError_t hipGetLastError(void) {
    const hipError_t e = pending;
    pending = hipSuccess;
    return e;
}
const char* hipGetErrorString(hipError_t) { return "an error"; }
}

// Whether [p, p + n) lies in one allocation.
static bool inside(const void* p, size_t n) {
    const char* q = static_cast<const char*>(p);
    for (auto& b : blocks)
        if (q >= b.first && q + n <= b.first + b.second) return true;
    return false;
}

// -------------------------------------------------------------- the launchers

using namespace mlpc;
int mlpc_linear_num_configs() { return MLPC_NUM_LINEAR_CONFIGS; }
LinearCfgInfo mlpc_linear_config(int cfg) {
#define ROW(id, bm, bn, wm, wn, ns, ks, occ) \
    if (cfg == id) return LinearCfgInfo{bm, bn, 64 * wm * wn, ns * (bm + bn) * ks * 2};
    MLPC_LINEAR_CONFIGS(ROW)
    return LinearCfgInfo{};
}
bool mlpc_linear_has(int cfg, int pass) {
    if (pass > PASS_DW) return cfg != 0 && cfg != 7;
    return pass == PASS_DW ? mlpc_linear_config(cfg).BM >= 128 : cfg != 7;
}

static std::vector<LossArgs> logits, products;      // of the call
static int rows_packed, joins, dx_done;

// Everything of the workspace that a launch may touch, and its pieces apart.
static void check_workspace(const LossArgs& a) {
    const size_t R = (size_t)a.rows, H = (size_t)a.H;
    CHECK(inside(a.zero, 16) && inside(a.info, sizeof(LossInfo)) && inside(a.place, R * 4) && inside(a.row, R * sizeof(LossRow)));
    CHECK(inside(a.packed, R * H * 2) && inside(a.picked, R * 4));
}

hipError_t mlpc_loss_rows(const LossArgs& a, bool, int, hipStream_t) {
    check_workspace(a);
    ++rows_packed;
    return done(launch_fails);
}
hipError_t mlpc_loss_logits(const LossArgs& a, int cfg, bool backward, int, hipStream_t) {
    const LinearCfgInfo c = mlpc_linear_config(cfg);
    const size_t R = (size_t)a.rows;
    check_workspace(a);
    CHECK(mlpc_linear_has(cfg, PASS_DX) && a.v0 >= 0 && a.vn > 0 && a.v0 + a.vn <= a.V);
    CHECK((int64_t)a.Mt * c.BM >= a.rows && (int64_t)(a.Mt - 1) * c.BM < a.rows && (int64_t)a.Nt * c.BN >= a.vn);
    CHECK(a.packing == (a.Mt > 1) && ((a.rows + 159) / 160 + 1) * (int64_t)a.Nt * c.NT < (int64_t)1 << 32);
    if (backward) CHECK(a.lddz >= a.vn && a.lddz % 8 == 0 && inside(a.dz, R * (size_t)a.lddz * 2));
    else CHECK(a.tiles == (int)a.Nt && inside(a.part, R * a.Nt * 8));
    logits.push_back(a);
    return done(launch_fails);
}
hipError_t mlpc_loss_products(const LossArgs& a, int cfg, int, hipStream_t) {
    const LinearCfgInfo c = mlpc_linear_config(cfg);
    CHECK(mlpc_linear_has(cfg, PASS_BOTH_DX) && (a.dx || a.dw) && a.S >= 1 && a.S <= 32);
    CHECK((size_t)a.S * a.ksp >= (size_t)(a.vn / 64) && (int64_t)a.dxNt * c.BN >= a.H && (int64_t)a.dwMt * c.BM >= a.vn);
    if (a.dx && !a.direct) CHECK(inside(a.sums, (size_t)a.S * a.rows * a.H * 4));
    CHECK(!a.direct || (!a.packing && a.S == 1));
    products.push_back(a);
    return done(launch_fails);
}
hipError_t mlpc_loss_join(const LossArgs&, hipStream_t) { ++joins; return done(launch_fails); }
hipError_t mlpc_loss_dx(const LossArgs&, int, hipStream_t) { ++dx_done; return done(launch_fails); }

static std::vector<NormTable> sums;
static std::vector<AdamTable> tables;
static int begun;
static NormJoin joined;
hipError_t mlpc_norm_sum(const NormTable& a, int, int parts, hipStream_t) {
    CHECK(parts > 0 && parts <= NORM_PARTS && inside(a.part, parts * sizeof(double)) && a.count > 0 && a.count <= NormTable::MAX);
    sums.push_back(a);
    return done(launch_fails);
}
hipError_t mlpc_norm_join(const NormJoin& a, hipStream_t) { joined = a; return done(launch_fails); }
hipError_t mlpc_adamw_begin(const AdamBegin& a, hipStream_t) {
    CHECK(inside(a.step, sizeof(AdamStep)));
    ++begun;
    return done(launch_fails);
}
hipError_t mlpc_adamw(const AdamTable& a, int, int, hipStream_t) {
    CHECK(a.count > 0 && a.count <= AdamTable::MAX && a.chunks > 0 && (int64_t)a.chunks * 256 < (int64_t)1 << 32);
    tables.push_back(a);
    return done(launch_fails);
}

// ------------------------------------------------------------------ the checks

alignas(16) static uint16_t buf[4096];
static float stat[64];
static int64_t ids[64];

static int forward(mlp_loss_t h, int64_t rows, int64_t H, hipStream_t s = nullptr) {
    logits.clear();
    return mlp_loss_forward(h, rows, buf, H, buf, H, ids, stat, stat + 8, s);
}
static int backward(mlp_loss_t h, int64_t rows, int64_t H, bool dx = true, bool dw = true, hipStream_t s = nullptr) {
    logits.clear();
    products.clear();
    return mlp_loss_backward(h, rows, buf, H, buf, H, ids, stat, stat, nullptr, dx ? buf : nullptr, H, dw ? buf : nullptr, H, s);
}

// Every size's launches stay within the workspace that create took, and the
// gradient's pieces cover the vocabulary once.
static void workspaces() {
    const int64_t sizes[][3] = {{1, 8, 1}, {1, 512, 1000}, {3, 72, 257}, {64, 512, 5000}, {257, 328, 999}, {1000, 12288, 50001},
                                {4096, 8192, 128000}, {70000, 512, 100003}, {1 << 20, 64, 200000}, {1 << 24, 8, 16000}, {5, 8, 4000000}};
    for (auto& q : sizes) {
        mlp_loss_t h = mlp_loss_create(q[0], q[1], q[2], 0, 1);
        CHECK(h);
        if (!h) continue;
        const int64_t rows[] = {q[0], 1, q[0] / 2 + 1, q[0] < 300 ? q[0] : 300, q[0] < 60 ? q[0] : 60};
        for (int64_t r : rows) {
            CHECK(forward(h, r, q[1]) == MLP_OK && logits.size() == 1 && logits[0].vn == q[2]);
            for (int outputs = 1; outputs < 4; ++outputs) {
                CHECK(backward(h, r, q[1], outputs & 1, outputs & 2) == MLP_OK && logits.size() == products.size());
                int64_t v = 0;
                for (size_t i = 0; i < products.size(); ++i) {
                    CHECK(products[i].v0 == v && logits[i].v0 == v && products[i].first == (v == 0) && logits[i].vn == products[i].vn);
                    v += products[i].vn;
                }
                CHECK(v == q[2]);
            }
            // a plan is kept for its rows and outputs alone
            CHECK(backward(h, r, q[1]) == MLP_OK && forward(h, r, q[1]) == MLP_OK);
        }
        CHECK(backward(h, 0, q[1]) == MLP_OK && logits.empty() && !products.empty());
        CHECK(mlp_loss_forward(h, 0, nullptr, 0, nullptr, 0, nullptr, nullptr, nullptr, nullptr) == MLP_OK);
        CHECK(mlp_loss_destroy(h) == MLP_OK);
    }
}

static void refusals() {
    mlp_loss_t h = mlp_loss_create(8, 64, 100, 0, 1), f = mlp_loss_create(8, 64, 100, 0, 0);
    CHECK(h && f);
    auto fwd = [&](int64_t rows, const void* x, int64_t ldx, const void* w, int64_t ldw, const int64_t* t, float* loss, float* lse) {
        return mlp_loss_forward(h, rows, x, ldx, w, ldw, t, loss, lse, nullptr);
    };
    float* odd = reinterpret_cast<float*>(reinterpret_cast<char*>(stat) + 2);
    CHECK(fwd(9, buf, 64, buf, 64, ids, stat, stat) == MLP_EINVAL && strstr(last, "rows"));
    CHECK(fwd(-1, buf, 64, buf, 64, ids, stat, stat) == MLP_EINVAL);
    CHECK(fwd(2, nullptr, 64, buf, 64, ids, stat, stat) == MLP_EINVAL && strstr(last, "x must"));
    CHECK(fwd(2, buf + 1, 64, buf, 64, ids, stat, stat) == MLP_EINVAL);
    CHECK(fwd(2, buf, 56, buf, 64, ids, stat, stat) == MLP_EINVAL && strstr(last, "stride of x"));
    CHECK(fwd(2, buf, 68, buf, 64, ids, stat, stat) == MLP_EINVAL);
    CHECK(fwd(2, buf, 64, nullptr, 64, ids, stat, stat) == MLP_EINVAL && strstr(last, "w must"));
    CHECK(fwd(2, buf, 64, buf, (1 << 23) + 8, ids, stat, stat) == MLP_EINVAL && strstr(last, "stride of w"));
    CHECK(fwd(2, buf, 64, buf, 64, nullptr, stat, stat) == MLP_EINVAL && strstr(last, "target"));
    CHECK(fwd(2, buf, 64, buf, 64, ids, stat, nullptr) == MLP_EINVAL && strstr(last, "lse"));
    CHECK(fwd(2, buf, 64, buf, 64, ids, odd, stat) == MLP_EINVAL);
    CHECK(fwd(2, buf, 64, buf, 64, ids, nullptr, stat) == MLP_OK);
    CHECK(mlp_loss_backward(f, 2, buf, 64, buf, 64, ids, stat, stat, stat, buf, 64, buf, 64, nullptr) == MLP_EINVAL && strstr(last, "gradient"));
    CHECK(mlp_loss_backward(h, 2, buf, 64, buf, 64, ids, nullptr, stat, stat, buf, 64, buf, 64, nullptr) == MLP_EINVAL && strstr(last, "lse"));
    CHECK(mlp_loss_backward(h, 2, buf, 64, buf, 64, ids, stat, odd, stat, buf, 64, buf, 64, nullptr) == MLP_EINVAL);
    CHECK(mlp_loss_backward(h, 2, buf, 64, buf, 64, ids, stat, stat, odd, buf, 64, buf, 64, nullptr) == MLP_EINVAL);
    CHECK(mlp_loss_backward(h, 2, buf, 64, buf, 64, ids, stat, stat, stat, buf + 4, 64, buf, 64, nullptr) == MLP_EINVAL && strstr(last, "dx"));
    CHECK(mlp_loss_backward(h, 2, buf, 64, buf, 64, ids, stat, stat, stat, buf, 64, buf, 60, nullptr) == MLP_EINVAL && strstr(last, "dw"));
    CHECK(mlp_loss_backward(h, 2, buf, 64, buf, 64, ids, stat, nullptr, nullptr, nullptr, 0, nullptr, 0, nullptr) == MLP_OK);
    CHECK(mlp_loss_debug_set_plan(h, 2, 0, 0) == MLP_EINVAL && mlp_loss_debug_set_plan(h, 0, 7, 0) == MLP_EINVAL);
    CHECK(mlp_loss_debug_set_plan(h, 1, 0, 0) == MLP_EINVAL && mlp_loss_debug_set_plan(h, 1, 1, 33) == MLP_EINVAL);
    CHECK(mlp_loss_debug_set_plan(h, 1, -1, 0) == MLP_OK);
    CHECK(mlp_loss_destroy(h) == MLP_OK && mlp_loss_destroy(f) == MLP_OK);

    mlp_grad_norm_t n = mlp_grad_norm_create(0);
    int64_t size[] = {5, -1}, one[] = {5}, wide[] = {(int64_t)1 << 34};
    const void* grads[] = {buf, buf};
    const void* none[] = {nullptr};
    const void* byte[] = {reinterpret_cast<char*>(buf) + 1};
    CHECK(mlp_grad_norm_forward(n, 2, size, grads, 1, 1, stat, stat, nullptr) == MLP_EINVAL && strstr(last, "tensor 1"));
    CHECK(mlp_grad_norm_forward(n, 1, wide, grads, 1, 1, stat, stat, nullptr) == MLP_EINVAL);
    CHECK(mlp_grad_norm_forward(n, 1, one, none, 1, 1, stat, stat, nullptr) == MLP_EINVAL && strstr(last, "tensor 0"));
    CHECK(mlp_grad_norm_forward(n, 1, one, byte, 1, 1, stat, stat, nullptr) == MLP_EINVAL);
    CHECK(mlp_grad_norm_forward(n, 1, nullptr, grads, 1, 1, stat, stat, nullptr) == MLP_EINVAL && strstr(last, "count"));
    CHECK(mlp_grad_norm_forward(n, -1, one, grads, 1, 1, stat, stat, nullptr) == MLP_EINVAL);
    CHECK(mlp_grad_norm_forward(n, 1, one, grads, 0, 1, stat, stat, nullptr) == MLP_EINVAL && strstr(last, "unscale"));
    CHECK(mlp_grad_norm_forward(n, 1, one, grads, NAN, 1, stat, stat, nullptr) == MLP_EINVAL);
    CHECK(mlp_grad_norm_forward(n, 1, one, grads, 1, 0, stat, stat, nullptr) == MLP_EINVAL && strstr(last, "max_norm"));
    CHECK(mlp_grad_norm_forward(n, 1, one, grads, 1, NAN, stat, stat, nullptr) == MLP_EINVAL);
    CHECK(mlp_grad_norm_forward(n, 1, one, grads, 1, 1, nullptr, stat, nullptr) == MLP_EINVAL && strstr(last, "norm"));
    CHECK(mlp_grad_norm_forward(n, 1, one, grads, 1, INFINITY, stat, nullptr, nullptr) == MLP_OK);
    CHECK(mlp_grad_norm_destroy(n) == MLP_OK);

    for (int bits : {32, 8}) {
        mlp_adamw_t a = mlp_adamw_create(0, bits, 0.9, 0.95, 1e-8, 1);
        const mlp_adamw_tensor good = {5, buf, stat, stat, stat, stat, stat, 0.1};
        auto step = [&](mlp_adamw_tensor t, const void* g, double lr = 1e-3) {
            const void* gs[] = {g};
            return mlp_adamw_step(a, 1, &t, gs, lr, nullptr, nullptr, ids, nullptr);
        };
        CHECK(step(good, buf) == MLP_OK);
        mlp_adamw_tensor t = good;
        t.n = -1;
        CHECK(step(t, buf) == MLP_EINVAL);
        t = good, t.w = nullptr;
        CHECK(step(t, buf) == MLP_EINVAL && strstr(last, "w of tensor 0"));
        t = good, t.m = nullptr;
        CHECK(step(t, buf) == MLP_EINVAL);
        t = good, t.v = nullptr;
        CHECK(step(t, buf) == MLP_EINVAL);
        t = good, t.master = odd;
        CHECK(step(t, buf) == MLP_EINVAL && strstr(last, "master"));
        t = good, t.m_scale = nullptr;
        CHECK(step(t, buf) == (bits == 8 ? MLP_EINVAL : MLP_OK));
        t = good, t.v_scale = nullptr;
        CHECK(step(t, buf) == (bits == 8 ? MLP_EINVAL : MLP_OK));
        t = good, t.decay = NAN;
        CHECK(step(t, buf) == MLP_EINVAL && strstr(last, "decay"));
        t = good, t.master = nullptr;
        CHECK(step(t, buf) == MLP_OK && step(good, nullptr) == MLP_EINVAL && step(good, buf, INFINITY) == MLP_EINVAL);
        t = {0, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 0};
        CHECK(step(t, nullptr) == MLP_OK);
        const void* gs[] = {buf};
        CHECK(mlp_adamw_step(a, 1, &good, gs, 1, nullptr, nullptr, nullptr, nullptr) == MLP_EINVAL && strstr(last, "t must"));
        CHECK(mlp_adamw_step(a, 1, &good, gs, 1, odd, nullptr, ids, nullptr) == MLP_EINVAL);
        CHECK(mlp_adamw_step(a, 1, &good, gs, 1, nullptr, odd, ids, nullptr) == MLP_EINVAL);
        CHECK(mlp_adamw_step(a, 1, nullptr, gs, 1, nullptr, nullptr, ids, nullptr) == MLP_EINVAL);
        CHECK(mlp_adamw_step(a, 1, &good, nullptr, 1, nullptr, nullptr, ids, nullptr) == MLP_EINVAL);
        CHECK(mlp_adamw_step(a, 0, nullptr, nullptr, 1, nullptr, nullptr, ids, nullptr) == MLP_OK);
        CHECK(mlp_adamw_destroy(a) == MLP_OK);
    }
}

// The tables of a call hold every tensor once, in order, with all its chunks.
static void tensor_tables() {
    mlp_grad_norm_t n = mlp_grad_norm_create(0);
    mlp_adamw_t a = mlp_adamw_create(0, 8, 0.9, 0.95, 1e-8, 1);
    for (int count : {0, 1, 47, 48, 49, 96, 183, 184, 185, 500}) {
        std::vector<int64_t> size;
        std::vector<const void*> grads;
        std::vector<mlp_adamw_tensor> tensors;
        for (int i = 0; i < count; ++i) {
            size.push_back(i % 7 == 3 ? 0 : (int64_t)1 + (i * 7919) % 50000);
            grads.push_back(size[i] ? buf + i : nullptr);
            tensors.push_back({size[i], buf, stat, buf, buf, stat, stat, 0.0});
        }
        sums.clear();
        tables.clear();
        begun = 0;
        CHECK(mlp_grad_norm_forward(n, count, size.data(), grads.data(), 1, 1, stat, stat, nullptr) == MLP_OK);
        CHECK(mlp_adamw_step(a, count, tensors.data(), grads.data(), 1e-3, nullptr, nullptr, ids, nullptr) == MLP_OK && begun == 1);
        std::vector<const void*> seen;
        bool first = true;
        for (auto& t : sums) {
            uint32_t chunks = 0;
            for (int i = 0; i < t.count; ++i) {
                seen.push_back(t.grad[i]);
                CHECK(t.first[i] == chunks);
                chunks += (uint32_t)((t.n[i] + NORM_CHUNK - 1) / NORM_CHUNK);
            }
            CHECK(chunks == t.chunks && t.add == !first);
            first = false;
        }
        std::vector<const void*> all;
        for (auto g : grads)
            if (g) all.push_back(g);
        CHECK(seen == all);
        seen.clear();
        int number = 0;
        for (auto& t : tables) {
            CHECK(t.number >= number);
            number = t.number;
            uint32_t chunks = 0;
            for (int i = 0; i < t.count; ++i, ++number) {
                CHECK(t.grad[i] == grads[number] && t.n[i] == size[number] && t.first[i] == chunks);
                if (t.n[i]) seen.push_back(t.grad[i]);
                chunks += (uint32_t)((t.n[i] + ADAM_CHUNK - 1) / ADAM_CHUNK);
            }
            CHECK(chunks == t.chunks);
        }
        CHECK(seen == all);
    }
    // tensors whose chunks do not fit one launch take several
    std::vector<mlp_adamw_tensor> big(5, mlp_adamw_tensor{((int64_t)1 << 34) - 1, buf, stat, buf, buf, stat, stat, 0.0});
    std::vector<const void*> grads(5, buf);
    tables.clear();
    CHECK(mlp_adamw_step(a, 5, big.data(), grads.data(), 1e-3, nullptr, nullptr, ids, nullptr) == MLP_OK && tables.size() == 5);
    CHECK(mlp_grad_norm_destroy(n) == MLP_OK && mlp_adamw_destroy(a) == MLP_OK);
}

// An error that an entry point returns is not left behind as the thread's last
// error too, where the caller's next call would find it.
static void errors_are_reported_once() {
    const int64_t size[] = {5};
    const void* grads[] = {buf};
    const mlp_adamw_tensor tensor = {5, buf, stat, stat, stat, stat, stat, 0.1};
    malloc_fails = hipErrorOutOfMemory;
    CHECK(!mlp_loss_create(4, 64, 64, 0, 1) && strstr(last, "hipMalloc") && pending == hipSuccess);
    CHECK(!mlp_grad_norm_create(0) && strstr(last, "hipMalloc") && pending == hipSuccess);
    CHECK(!mlp_adamw_create(0, 32, 0.9, 0.9, 0, 0) && strstr(last, "hipMalloc") && pending == hipSuccess);
    malloc_fails = hipSuccess;
    memset_fails = hipErrorUnknown;
    CHECK(!mlp_loss_create(4, 64, 64, 0, 1) && strstr(last, "clearing") && pending == hipSuccess);
    memset_fails = hipSuccess;
    mlp_loss_t l = mlp_loss_create(4, 64, 64, 0, 1);
    mlp_grad_norm_t n = mlp_grad_norm_create(0);
    mlp_adamw_t a = mlp_adamw_create(0, 32, 0.9, 0.9, 0, 0);
    auto norm = [&] { return mlp_grad_norm_forward(n, 1, size, grads, 1, 1, stat, stat, nullptr); };
    auto step = [&] { return mlp_adamw_step(a, 1, &tensor, grads, 1, nullptr, nullptr, ids, nullptr); };
    launch_fails = hipErrorInvalidConfiguration;
    CHECK(forward(l, 4, 64) == MLP_EHIP && pending == hipSuccess && backward(l, 4, 64) == MLP_EHIP && pending == hipSuccess);
    CHECK(norm() == MLP_EHIP && pending == hipSuccess && step() == MLP_EHIP && pending == hipSuccess);
    launch_fails = hipSuccess;
    // (an error of the caller's own stays the caller's through calls that succeed)
    pending = hipErrorInvalidValue;
    CHECK(forward(l, 4, 64) == MLP_OK && backward(l, 4, 64) == MLP_OK && norm() == MLP_OK && step() == MLP_OK);
    CHECK(pending == hipErrorInvalidValue);
    pending = hipSuccess;
    sync_fails = hipErrorUnknown;
    CHECK(mlp_loss_destroy(l) == MLP_EHIP && mlp_grad_norm_destroy(n) == MLP_EHIP && mlp_adamw_destroy(a) == MLP_EHIP);
    CHECK(pending == hipSuccess);
    sync_fails = hipSuccess;
}

// destroy waits for the stream of the last call, which may still use the workspace.
static void destroy_waits_for_the_workspace() {
    hipStream_t one = reinterpret_cast<hipStream_t>(stat), other = reinterpret_cast<hipStream_t>(buf);
    mlp_loss_t l = mlp_loss_create(4, 64, 64, 0, 1);
    CHECK(backward(l, 4, 64, true, true, one) == MLP_OK && forward(l, 4, 64, other) == MLP_OK);
    waited.clear();
    CHECK(mlp_loss_destroy(l) == MLP_OK && waited.size() == 1 && waited[0] == other);
    mlp_grad_norm_t n = mlp_grad_norm_create(0);
    CHECK(mlp_grad_norm_forward(n, 0, nullptr, nullptr, 1, 1, stat, stat, one) == MLP_OK);
    waited.clear();
    CHECK(mlp_grad_norm_destroy(n) == MLP_OK && waited.size() == 1 && waited[0] == one);
    mlp_adamw_t a = mlp_adamw_create(0, 8, 0.9, 0.9, 0, 0);
    CHECK(mlp_adamw_step(a, 0, nullptr, nullptr, 1, nullptr, nullptr, ids, other) == MLP_OK);
    waited.clear();
    CHECK(mlp_adamw_destroy(a) == MLP_OK && waited.size() == 1 && waited[0] == other);
}

int main() {
    workspaces();
    refusals();
    tensor_tables();
    errors_are_reported_once();
    destroy_waits_for_the_workspace();
    CHECK(blocks.empty());
    printf("%d failures\n", failures);
    return failures != 0;
}

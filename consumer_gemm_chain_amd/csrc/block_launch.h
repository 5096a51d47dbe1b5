// block_launch.h -- internal interface between the C ABI of the MLP block's
// operators (block_api.cpp) and their kernels (norm_kernels.hip,
// linear_kernels.hip).  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mlpc {

struct NormArgs {
    const uint16_t* x;
    const uint16_t* weight;     // nullptr: 1
    const uint16_t* bias;       // nullptr: 0 (forward)
    uint16_t* y;                // forward
    const uint16_t* dy;         // backward
    const uint16_t* dres;       // nullptr: none (backward)
    uint16_t* dx;               // backward
    float* mean;                // forward: outputs or nullptr; backward: inputs
    float* rstd;
    uint16_t* dweight;          // nullptr: not computed
    uint16_t* dbias;
    float* part;                // [parts][2][H] column sums of the row groups
    int64_t rows;
    int64_t ldx, ldy, lddy, lddres, lddx;
    int H;
    int parts;
    float eps;
};

// One product D[M, N] = sum_k A(m, k) B(k, n) of the linear layer.  PASS_FWD:
// A = x [M, K], B = W [K, N]; PASS_DX: A = dz [M, K], B = W^T, stored as
// W [N, K]; PASS_DW: A = x^T, stored as x [K, M], B = dz [K, N].
// PASS_BOTH_DX and PASS_BOTH_DW are the last two as parts of one launch.
enum { PASS_FWD = 0, PASS_DX = 1, PASS_DW = 2, PASS_BOTH_DX = 3, PASS_BOTH_DW = 4, PASSES = 5 };

struct GemmArgs {
    const uint16_t* a;
    const uint16_t* b;
    uint16_t* d;
    int64_t lda, ldb, ldd;
    int M, N, K;                // N: output columns (swiglu: of one half)
    int up;                     // swiglu: distance of the up half's columns in B, bias and z; else 0
    int act;
    const uint16_t* bias;       // nullptr: none
    const uint16_t* res;        // nullptr: none
    uint16_t* z;                // nullptr: not saved
    int64_t ldr, ldz;
    // plan: tiles; the first `direct` of the tile order are computed whole,
    // the others in S parts of ksp slabs
    uint32_t Mt, Nt, direct, S, ksp;
    int BM, BN;                 // the configuration's tile
    float* part;                // [Mt * Nt - direct][S][BM][BN] (S > 1)
    const void* zero;           // 16 zero bytes
};

struct LinearCfgInfo {
    int BM, BN, NT, lds;
};

// dz = dy act'(z), and the column sums of dz.
struct DzArgs {
    const uint16_t* dy;
    const uint16_t* z;          // nullptr: act none
    uint16_t* dz;               // nullptr: not stored (act none)
    uint16_t* db;               // nullptr: no column sums
    float* part;                // [parts][gN] column sums of the row groups
    int64_t lddy, ldz, lddz;
    int64_t rows;
    int N;
    int act;
    int parts;
};

template <class T>
struct Param {
    using type = T;
};

// Launch `kernel` and return the launch's own status: hipGetLastError would
// also report an error that an earlier call of the thread, ours or not, left.
template <class... P>
hipError_t launch(void (*kernel)(P...), dim3 grid, int threads, hipStream_t s, typename Param<P>::type... args) {
    void* p[] = {&args...};
    return hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, dim3(threads), p, 0, s);
}

}  // namespace mlpc

hipError_t mlpc_norm_forward(const mlpc::NormArgs& a, int dtype, int cus, hipStream_t s);
hipError_t mlpc_norm_backward(const mlpc::NormArgs& a, int dtype, hipStream_t s);
// Row groups whose column sums the norm's gradient keeps in its workspace,
// for `rows` rows and at most.
int mlpc_norm_parts(int64_t rows, int H, int cus);
int mlpc_norm_max_parts(int H, int cus);

// Tile configurations (linear_configs.h): their number, sizes, whether a pass
// has them, and one launch.
int mlpc_linear_num_configs();
mlpc::LinearCfgInfo mlpc_linear_config(int cfg);
bool mlpc_linear_has(int cfg, int pass);
hipError_t mlpc_gemm(const mlpc::GemmArgs& a, int cfg, int pass, int dtype, hipStream_t s);
// Both products of the gradient in one launch, with the sums of dz's partial
// column sums unless dz.db is nullptr.
hipError_t mlpc_gemm_both(const mlpc::GemmArgs& dx, const mlpc::GemmArgs& dw, const mlpc::DzArgs& dz, int cfg, int dtype,
                          hipStream_t s);
// Sum the parts of a split product and finish its outputs (linear_reduce.hip).
hipError_t mlpc_gemm_reduce(const mlpc::GemmArgs& a, int dtype, hipStream_t s);
// dz and its column sums; with more than one row group `join` adds the groups'
// in a second kernel, else they are left in a.part.
hipError_t mlpc_dz(const mlpc::DzArgs& a, int dtype, bool join, hipStream_t s);
int mlpc_dz_parts(int64_t rows);
int mlpc_dz_max_parts();

// norm_kernels.hip -- layer norm, forward and backward (include/mlp_block.h
// has the formulas).
#include <hip/hip_runtime.h>

#include "block_launch.h"
#include "chain_device.hpp"

namespace mlpc {

template <int DT>
__device__ __forceinline__ float widen(uint16_t v) {
    if constexpr (DT == DT_F16) return (float)__builtin_bit_cast(_Float16, v);
    else return __builtin_bit_cast(float, (uint32_t)v << 16);
}

constexpr int NORM_NT = 256;

// Sum over the workgroup, the same bits in every thread.
__device__ __forceinline__ float block_sum(float v, float* s) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < NORM_NT / 64; ++i) t += s[i];
    return t;
}

// One workgroup per row, any H and strides: three passes over the row, the
// second and third from the caches.
template <int DT>
__global__ __launch_bounds__(NORM_NT) void norm_forward_kernel(NormArgs a) {
    __shared__ float s[NORM_NT / 64];
    const size_t r = blockIdx.x;
    const uint16_t* x = a.x + r * a.ldx;
    float t = 0.f;
    for (int c = threadIdx.x; c < a.H; c += NORM_NT) t += widen<DT>(x[c]);
    const float mean = block_sum(t, s) / a.H;
    t = 0.f;
    for (int c = threadIdx.x; c < a.H; c += NORM_NT) {
        const float d = widen<DT>(x[c]) - mean;
        t += d * d;
    }
    const float rstd = 1.0f / sqrtf(block_sum(t, s) / a.H + a.eps);
    for (int c = threadIdx.x; c < a.H; c += NORM_NT) {
        float v = (widen<DT>(x[c]) - mean) * rstd;
        if (a.weight) v *= widen<DT>(a.weight[c]);
        if (a.bias) v += widen<DT>(a.bias[c]);
        a.y[r * a.ldy + c] = to_storage<DT>(v);
    }
    if (threadIdx.x == 0) {
        if (a.mean) a.mean[r] = mean;
        if (a.rstd) a.rstd[r] = rstd;
    }
}

// dx of one row per workgroup.
template <int DT>
__global__ __launch_bounds__(NORM_NT) void norm_dx_kernel(NormArgs a) {
    __shared__ float s[NORM_NT / 64];
    const size_t r = blockIdx.x;
    const uint16_t* x = a.x + r * a.ldx;
    const uint16_t* dy = a.dy + r * a.lddy;
    const float mean = a.mean[r], rstd = a.rstd[r];
    float t0 = 0.f, t1 = 0.f;
    for (int c = threadIdx.x; c < a.H; c += NORM_NT) {
        const float g = widen<DT>(dy[c]) * (a.weight ? widen<DT>(a.weight[c]) : 1.f);
        t0 += g;
        t1 += g * ((widen<DT>(x[c]) - mean) * rstd);
    }
    const float m0 = block_sum(t0, s) / a.H, m1 = block_sum(t1, s) / a.H;
    for (int c = threadIdx.x; c < a.H; c += NORM_NT) {
        const float g = widen<DT>(dy[c]) * (a.weight ? widen<DT>(a.weight[c]) : 1.f);
        float v = rstd * (g - m0 - (widen<DT>(x[c]) - mean) * rstd * m1);
        if (a.dres) v += widen<DT>(a.dres[r * a.lddres + c]);
        a.dx[r * a.lddx + c] = to_storage<DT>(v);
    }
}

// Column sums of dy xhat and dy over row group blockIdx.y, one column per
// thread.
template <int DT>
__global__ __launch_bounds__(NORM_NT) void norm_cols_kernel(NormArgs a) {
    const int c = blockIdx.x * NORM_NT + threadIdx.x;
    if (c >= a.H) return;
    const int64_t r0 = a.rows * blockIdx.y / a.parts, r1 = a.rows * (blockIdx.y + 1) / a.parts;
    float tw = 0.f, tb = 0.f;
    for (int64_t r = r0; r < r1; ++r) {
        const float dy = widen<DT>(a.dy[r * a.lddy + c]);
        tw += dy * ((widen<DT>(a.x[r * a.ldx + c]) - a.mean[r]) * a.rstd[r]);
        tb += dy;
    }
    float* p = a.part + (size_t)blockIdx.y * 2 * a.H + c;
    p[0] = tw;
    p[a.H] = tb;
}

// The row groups' column sums added in group order.
template <int DT>
__global__ __launch_bounds__(NORM_NT) void norm_cols_sum_kernel(NormArgs a) {
    const int c = blockIdx.x * NORM_NT + threadIdx.x;
    if (c >= a.H) return;
    float tw = 0.f, tb = 0.f;
    for (int p = 0; p < a.parts; ++p) {
        tw += a.part[(size_t)p * 2 * a.H + c];
        tb += a.part[((size_t)p * 2 + 1) * a.H + c];
    }
    if (a.dweight) a.dweight[c] = to_storage<DT>(tw);
    if (a.dbias) a.dbias[c] = to_storage<DT>(tb);
}

template <int DT>
static hipError_t norm_forward_t(const NormArgs& a, hipStream_t s) {
    hipLaunchKernelGGL(norm_forward_kernel<DT>, dim3((unsigned)a.rows), dim3(NORM_NT), 0, s, a);
    return hipGetLastError();
}

template <int DT>
static hipError_t norm_backward_t(const NormArgs& a, hipStream_t s) {
    const unsigned cols = (unsigned)((a.H + NORM_NT - 1) / NORM_NT);
    if (a.dweight || a.dbias) {
        if (a.parts > 0) hipLaunchKernelGGL(norm_cols_kernel<DT>, dim3(cols, a.parts), dim3(NORM_NT), 0, s, a);
        hipLaunchKernelGGL(norm_cols_sum_kernel<DT>, dim3(cols), dim3(NORM_NT), 0, s, a);
    }
    if (a.rows > 0) hipLaunchKernelGGL(norm_dx_kernel<DT>, dim3((unsigned)a.rows), dim3(NORM_NT), 0, s, a);
    return hipGetLastError();
}

}  // namespace mlpc

using namespace mlpc;

int mlpc_norm_max_parts() { return 64; }

int mlpc_norm_parts(int64_t rows) { return (int)(rows < 64 ? rows : 64); }

hipError_t mlpc_norm_forward(const NormArgs& a, int dtype, hipStream_t s) {
    return dtype == DT_F16 ? norm_forward_t<DT_F16>(a, s) : norm_forward_t<DT_BF16>(a, s);
}

hipError_t mlpc_norm_backward(const NormArgs& a, int dtype, hipStream_t s) {
    return dtype == DT_F16 ? norm_backward_t<DT_F16>(a, s) : norm_backward_t<DT_BF16>(a, s);
}

// dz_kernels.hip -- the activation's gradient dz = dy act'(z) of the linear
// layer and the column sums of dz, its bias's gradient.
#include <hip/hip_runtime.h>

#include "block_launch.h"
#include "chain_device.hpp"
#include "linear_device.hpp"

namespace mlpc {

// d/dz of gelu(z) = z s, s = 1 / (1 + exp(-2u)), u = sqrt(2/pi) (z + 0.044715 z^3):
// s + z s (1 - s) 2 u'.  Beyond |z| = 12 it is 0 or 1 to the last fp32 bit;
// the clamp keeps z^3 finite.
__device__ __forceinline__ float gelu_tanh_grad(float z) {
    const float c = 0.7978845608028654f, k = 0.044715f;
    const float t = fminf(fmaxf(z, -12.f), 12.f);
    const float u = c * (t + k * (t * t * t));
    const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(u * -2.8853900817779268f));
    const float d = s + t * s * (1.f - s) * (2.f * c) * (1.f + 3.f * k * (t * t));
    return z != z ? z : d;
}

// dz and the column sums of row group blockIdx.y, one dy column per thread.
template <int DT>
__global__ __launch_bounds__(256) void dz_kernel(DzArgs a) {
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= a.N) return;
    const int64_t r0 = a.rows * blockIdx.y / a.parts, r1 = a.rows * (blockIdx.y + 1) / a.parts;
    float t0 = 0.f, t1 = 0.f;
    for (int64_t r = r0; r < r1; ++r) {
        const float dy = widen<DT>(a.dy[r * a.lddy + c]);
        float d0 = dy, d1 = 0.f;
        if (a.act == ACT_GELU_TANH) d0 = dy * gelu_tanh_grad(widen<DT>(a.z[r * a.ldz + c]));
        if (a.act == ACT_SWIGLU) {
            const float gate = widen<DT>(a.z[r * a.ldz + c]), u = widen<DT>(a.z[r * a.ldz + a.N + c]);
            const float s = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(gate * -1.4426950408889634f));
            d0 = dy * u * (s + gate * s * (1.f - s));
            d1 = dy * gate * s;
            a.dz[r * a.lddz + a.N + c] = to_storage<DT>(d1);
        }
        if (a.dz) a.dz[r * a.lddz + c] = to_storage<DT>(d0);
        t0 += d0;
        t1 += d1;
    }
    if (!a.db) return;
    const int gN = a.act == ACT_SWIGLU ? 2 * a.N : a.N;
    a.part[(size_t)blockIdx.y * gN + c] = t0;
    if (gN > a.N) a.part[(size_t)blockIdx.y * gN + a.N + c] = t1;
}

// The row groups' column sums added in group order.
template <int DT>
__global__ __launch_bounds__(256) void db_kernel(DzArgs a) {
    const int gN = a.act == ACT_SWIGLU ? 2 * a.N : a.N;
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= gN) return;
    float t = 0.f;
    for (int p = 0; p < a.parts; ++p) t += a.part[(size_t)p * gN + c];
    a.db[c] = to_storage<DT>(t);
}

template <int DT>
static hipError_t dz_t(const DzArgs& a, hipStream_t s) {
    const int gN = a.act == ACT_SWIGLU ? 2 * a.N : a.N;
    if (a.parts > 0)
        hipLaunchKernelGGL(dz_kernel<DT>, dim3((a.N + 255) / 256, a.parts), dim3(256), 0, s, a);
    if (a.db) hipLaunchKernelGGL(db_kernel<DT>, dim3((gN + 255) / 256), dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace mlpc

using namespace mlpc;

hipError_t mlpc_dz(const DzArgs& a, int dtype, hipStream_t s) {
    return dtype == DT_F16 ? dz_t<DT_F16>(a, s) : dz_t<DT_BF16>(a, s);
}

int mlpc_dz_max_parts() { return 64; }

int mlpc_dz_parts(int64_t rows) { return (int)(rows < 64 ? rows : 64); }

// linear_reduce.hip -- the second kernel of a split product: the parts'
// partials are added in part order and finished like an unsplit tile's
// accumulators.
#include <hip/hip_runtime.h>

#include "linear_device.hpp"

namespace mlpc {

// Eight output columns per thread.  A kernel of its own rather than the last
// part of each tile: it needs no counters and no agent-scope fences, and the
// whole chip reads the partials.
template <int DT>
__global__ __launch_bounds__(256) void linear_reduce_kernel(GemmArgs p) {
    const int chunks = p.N / 8;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= (int64_t)p.M * chunks) return;
    const int64_t r = i / chunks;
    const int n = (int)(i % chunks) * 8;
    const int64_t ld = p.N + p.up, plane = p.M * ld;
    const f32x4* src = reinterpret_cast<const f32x4*>(p.part + r * ld + n);
    const u32x4 res = p.res ? ld16(p.res + (size_t)r * p.ldr + n) : u32x4{};
    float b[8] = {}, bu[8] = {}, v[8], u[8];
    if (p.bias) {
        widen8<DT>(ld16(p.bias + n), b);
        if (p.up) widen8<DT>(ld16(p.bias + p.up + n), bu);
    }
    auto sum = [&](const f32x4* q, float (&t)[8]) {
        // eight parts' loads in flight, added in part order
        f32x4 lo = {}, hi = {};
        for (uint32_t s0 = 0; s0 < p.S; s0 += 8) {
            f32x4 l[8], h[8];
#pragma unroll
            for (uint32_t k = 0; k < 8; ++k) {
                if (s0 + k >= p.S) continue;
                l[k] = q[(s0 + k) * (size_t)(plane / 4)];
                h[k] = q[(s0 + k) * (size_t)(plane / 4) + 1];
            }
#pragma unroll
            for (uint32_t k = 0; k < 8; ++k) {
                if (s0 + k >= p.S) continue;
                lo = lo + l[k];
                hi = hi + h[k];
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            t[k] = lo[k];
            t[4 + k] = hi[k];
        }
    };
    sum(src, v);
    if (p.up) sum(src + p.up / 4, u);
    finish8<DT>(p, r, n, v, u, b, bu, res);
}

}  // namespace mlpc

using namespace mlpc;

hipError_t mlpc_gemm_reduce(const GemmArgs& a, int dtype, hipStream_t s) {
    const dim3 grid((unsigned)(((int64_t)a.M * (a.N / 8) + 255) / 256));
    if (dtype == DT_F16) hipLaunchKernelGGL(linear_reduce_kernel<DT_F16>, grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL(linear_reduce_kernel<DT_BF16>, grid, dim3(256), 0, s, a);
    return hipGetLastError();
}

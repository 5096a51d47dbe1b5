// linear_reduce.hip -- the second kernel of a split product: the parts'
// partials are added in part order and finished like an unsplit tile's
// accumulators.
#include <hip/hip_runtime.h>

#include "linear_device.hpp"

namespace mlpc {

constexpr int RNT = 64;     // small workgroups spread evenly over the CUs

// A workgroup takes 64 chunks of eight output columns of one split tile.  A
// kernel of its own rather than the last part of each tile: it needs no
// counters and no agent-scope fences, and the whole chip reads the partials
// (x W, both kernels: 128 rows 12288 x 6144 54 -> 46 us, 300 rows 98 -> 78, one
// row 37.7 -> 32.4 against the last part of each tile adding the others').
// Bound by latency: 4.8 us for one row, 6.4 us for 20 MB of partials.
template <int DT>
__global__ __launch_bounds__(RNT) void linear_reduce_kernel(GemmArgs p, int per_tile) {
    const uint32_t tile = blockIdx.x / per_tile;
    const int chunk = (int)(blockIdx.x % per_tile) * RNT + threadIdx.x;
    const int width = p.up ? p.BN / 2 : p.BN, row = chunk / (width / 8), oc = chunk % (width / 8) * 8;
    uint32_t mb, nb;
    tile_at(p, p.direct + tile, mb, nb);
    const int r = mb * p.BM + row, n = nb * width + oc;
    if (row >= p.BM || r >= p.M || n >= p.N) return;
    const size_t plane = (size_t)p.BM * p.BN / 4;
    // gate and up columns alternate in 16s
    const int col = p.up ? (oc >> 4) * 32 + (oc & 15) : oc;
    const f32x4* src = reinterpret_cast<const f32x4*>(p.part) + tile * p.S * plane + (row * p.BN + col) / 4;
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
                l[k] = q[(s0 + k) * plane];
                h[k] = q[(s0 + k) * plane + 1];
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
    if (p.up) sum(src + 4, u);
    finish8<DT>(p, r, n, v, u, b, bu, res);
}

}  // namespace mlpc

using namespace mlpc;

hipError_t mlpc_gemm_reduce(const GemmArgs& a, int dtype, hipStream_t s) {
    // (rows past M, as in the one tile row of a short product, are not launched)
    const int rows = a.M < a.BM ? a.M : a.BM, chunks = rows * ((a.up ? a.BN / 2 : a.BN) / 8);
    const int per_tile = (chunks + RNT - 1) / RNT;
    const dim3 grid((a.Mt * a.Nt - a.direct) * per_tile);
    return launch(dtype == DT_F16 ? linear_reduce_kernel<DT_F16> : linear_reduce_kernel<DT_BF16>, grid, RNT, s, a, per_tile);
}

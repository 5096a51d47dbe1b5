// loss_rows.hip -- the row work around the cross entropy's products: packing
// the rows that count, joining the tiles' softmax sums, and dx from its sums.
#include <hip/hip_runtime.h>

#include "loss_device.hpp"

namespace mlpc {

constexpr int PNT = 1024;

// Places of the rows that count, in order, by one workgroup: 1024 rows at a
// time, places from the waves' ballots.  Backward also what dz needs of each
// row.  (4096 rows 4 to 6 us, with the gradient's 7 to 11, 65536 rows 56 and 105:
// what one CU moves.  It is 0.1% of the large cases and 1% of 65536 x 1024 x 32000;
// four rows per thread at a time took as long.)
template <bool GRAD, int DT>
__global__ __launch_bounds__(PNT) void loss_pack_kernel(LossArgs a) {
    __shared__ int count[PNT / 64];
    __shared__ float largest[PNT / 64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    auto counts = [&](int64_t r) {
        const int64_t t = r < a.rows ? a.target[r] : -1;
        return t >= 0 && t < a.V;
    };
    float unit = 1.f;
    if constexpr (GRAD) {
        float top = 0.f;
        for (int64_t r = threadIdx.x; r < a.rows; r += PNT) {
            if (!counts(r)) continue;
            top = fmaxf(top, largest_coefficient(a.dloss ? a.dloss[r] : 1.f, a.dlse ? a.dlse[r] : 0.f));
        }
        top = wave_max(top);
        if (lane == 0) largest[wave] = top;
        __syncthreads();
        top = largest[lane & (PNT / 64 - 1)];
        top = wave_max(top);
        unit = dz_unit<DT>(top);
    }
    int n = 0;
    for (int64_t r0 = 0; r0 < a.rows; r0 += PNT) {
        const int64_t r = r0 + threadIdx.x;
        const bool in = counts(r);
        const uint64_t mask = __ballot(in);
        __syncthreads();
        if (lane == 0) count[wave] = __popcll(mask);
        __syncthreads();
        int at = n + __popcll(mask & ((1ull << lane) - 1));
#pragma unroll
        for (int w = 0; w < PNT / 64; ++w) {
            if (w < wave) at += count[w];
            n += count[w];
        }
        if (r < a.rows) a.place[r] = in ? at : -1;
        if (!in) continue;
        LossRow q{};
        q.target = (int)a.target[r];
        if constexpr (GRAD) {
            const float d = a.dloss ? a.dloss[r] : 1.f, l = a.dlse ? a.dlse[r] : 0.f;
            q.lse = a.lse_in[r];
            q.a = (d + l) / unit;
            q.b = d / unit;
        }
        a.row[at] = q;
    }
    if (threadIdx.x == 0) *a.info = LossInfo{n, unit, n < (int)a.rows};
}

// The packed rows of x, unless every row counts: 3700 of 4096 x 8192 in 24 us, 5.1
// TB/s.  The products save what it copies: a tenth of a call's rows is a tenth of
// its time.
__global__ __launch_bounds__(256) void loss_gather_kernel(LossArgs a) {
    if (!a.info->copied) return;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const int at = a.place[r];
        if (at < 0) continue;
        const uint16_t* from = a.x + r * a.ldx;
        uint16_t* to = a.packed + (size_t)at * a.H;
        for (int c = threadIdx.x * 8; c < a.H; c += 256 * 8) st16(to + c, ld16(from + c));
    }
}

// loss and lse of a row by one wave, from its tiles' maxima and sums (4096 rows of
// 500 tiles 10 us; few rows 3 to 5, a launch).
__global__ __launch_bounds__(256) void loss_join_kernel(LossArgs a) {
    const int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    if (r >= a.rows) return;
    const int64_t t = a.target[r];
    if (t < 0 || t >= a.V) {
        if (lane == 0) {
            const float v = t < 0 ? 0.f : NAN;
            if (a.loss) a.loss[r] = v;
            a.lse[r] = v;
        }
        return;
    }
    const int64_t at = a.packing ? a.place[r] : r;
    float m = -INFINITY, s = 0.f;
    for (int i = lane; i < a.tiles; i += 64) {
        const float2 v = a.part[(size_t)at * a.tiles + i];
        softmax_join(m, s, v.x, v.y);
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const float m2 = __shfl_xor(m, d), s2 = __shfl_xor(s, d);
        // (both lanes of a pair add in the same order)
        if (lane & d) {
            float mm = m2, ss = s2;
            softmax_join(mm, ss, m, s);
            m = mm;
            s = ss;
        } else {
            softmax_join(m, s, m2, s2);
        }
    }
    if (lane != 0) return;
    // (the loss is not taken from the rounded lse: a confident row's is far smaller)
    const float rest = logf(s);
    a.lse[r] = m + rest;
    if (a.loss) a.loss[r] = rest + (m - a.picked[at]);
}

// dx = unit (sum of the parts), rows that are left out 0.  (4096 x 8192 38 us, 5.0
// TB/s: one read of fp32 sums and one write, however many pieces there were.)
template <int DT>
__global__ __launch_bounds__(256) void loss_dx_kernel(LossArgs a) {
    const int per_row = a.H / 8;
    const int64_t chunks = a.rows * per_row;
    const float unit = a.info->unit;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < chunks; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / per_row;
        const int c = (int)(i % per_row) * 8;
        const int at = a.place[r];
        float v[8] = {};
        if (at >= 0) {
            f32x4 lo = {}, hi = {};
            for (uint32_t s = 0; s < a.S; ++s) {
                const f32x4* q = reinterpret_cast<const f32x4*>(a.sums + ((size_t)s * a.rows + at) * a.H + c);
                lo = lo + q[0];
                hi = hi + q[1];
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                v[k] = lo[k] * unit;
                v[4 + k] = hi[k] * unit;
            }
        }
        st16(a.dx + r * a.lddx + c, narrow8<DT>(v));
    }
}

}  // namespace mlpc

using namespace mlpc;

hipError_t mlpc_loss_rows(const LossArgs& a, bool backward, int dtype, hipStream_t s) {
    const dim3 one(1);
    hipError_t e = !backward            ? launch(loss_pack_kernel<false, DT_F16>, one, PNT, s, a)
                   : dtype == DT_F16 ? launch(loss_pack_kernel<true, DT_F16>, one, PNT, s, a)
                                     : launch(loss_pack_kernel<true, DT_BF16>, one, PNT, s, a);
    if (e == hipSuccess && a.rows > 0) e = launch(loss_gather_kernel, dim3(a.rows < 2048 ? a.rows : 2048), 256, s, a);
    return e;
}

hipError_t mlpc_loss_join(const LossArgs& a, hipStream_t s) {
    return launch(loss_join_kernel, dim3((a.rows + 3) / 4), 256, s, a);
}

hipError_t mlpc_loss_dx(const LossArgs& a, int dtype, hipStream_t s) {
    const int64_t n = (a.rows * (a.H / 8) + 255) / 256;
    const dim3 grid(n < 4096 ? n : 4096);
    return launch(dtype == DT_F16 ? loss_dx_kernel<DT_F16> : loss_dx_kernel<DT_BF16>, grid, 256, s, a);
}

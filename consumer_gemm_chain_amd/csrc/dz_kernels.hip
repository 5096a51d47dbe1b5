// dz_kernels.hip -- the activation's gradient dz = dy act'(z) of the linear
// layer and the column sums of dz, its bias's gradient.  Bound by memory: dy
// and z are read once, dz is written once for the two products that read it
// (2048 x 6144 gelu 18.6 us, 4.2 TB/s; 1000 x 3584 swiglu 10.0 us, 3.6 TB/s).
// dz is rounded to the storage type because the matrix cores take 16 bits: the
// relative error of dx and dW is 2.9e-4 (fp16) and 2.3e-3 (bf16) where that of
// one rounding is 2.1e-4 and 1.7e-3.  A second 16-bit term for what the rounding
// leaves would double both products' matrix work, which is nearly all of their
// time.  dz's column sums are those of the unrounded values.
#include <hip/hip_runtime.h>

#include "block_launch.h"
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

// A workgroup takes COLS columns (8 per thread) of one row group, ROWS rows at
// a time, with the columns' sums in registers: 256 columns by 8 rows, or 64 by
// 32 where one row group is the whole (short) batch.
constexpr int DZ_NT = 256;
constexpr int DZ_PARTS = 64;

template <int DT, int ACT, int COLS>
__global__ __launch_bounds__(DZ_NT) void dz_kernel(DzArgs a) {
    constexpr int LANES = COLS / 8, ROWS = DZ_NT / LANES;
    constexpr int G = ACT == ACT_SWIGLU ? 2 : 1;
    __shared__ float s[ROWS][COLS];
    const int lane = threadIdx.x % LANES, sub = threadIdx.x / LANES;
    const int c = blockIdx.x * COLS + lane * 8;
    const bool in = c < a.N;
    const int64_t r0 = a.rows * blockIdx.y / a.parts, r1 = a.rows * (blockIdx.y + 1) / a.parts;
    float sum[G][8] = {};
    if (in) {
        for (int64_t r = r0 + sub; r < r1; r += ROWS) {
            float d[G][8];
            widen8<DT>(ld16(a.dy + r * a.lddy + c), d[0]);
            if constexpr (ACT == ACT_GELU_TANH) {
                float z[8];
                widen8<DT>(ld16(a.z + r * a.ldz + c), z);
#pragma unroll
                for (int k = 0; k < 8; ++k) d[0][k] *= gelu_tanh_grad(z[k]);
            }
            if constexpr (ACT == ACT_SWIGLU) {
                float gate[8], up[8];
                widen8<DT>(ld16(a.z + r * a.ldz + c), gate);
                widen8<DT>(ld16(a.z + r * a.ldz + a.N + c), up);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float dy = d[0][k], q = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(gate[k] * -1.4426950408889634f));
                    d[0][k] = dy * up[k] * (q + gate[k] * q * (1.f - q));
                    d[1][k] = dy * gate[k] * q;
                }
            }
#pragma unroll
            for (int g = 0; g < G; ++g) {
                if constexpr (ACT != ACT_NONE) st16(a.dz + r * a.lddz + g * a.N + c, narrow8<DT>(d[g]));
#pragma unroll
                for (int k = 0; k < 8; ++k) sum[g][k] += d[g][k];
            }
        }
    }
    if (!a.db) return;
    const int j = threadIdx.x, col = blockIdx.x * COLS + j;
#pragma unroll
    for (int g = 0; g < G; ++g) {
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 8; ++k) s[sub][lane * 8 + k] = sum[g][k];
        __syncthreads();
        if (j >= COLS || col >= a.N) continue;
        float t = s[0][j];
#pragma unroll 8
        for (int k = 1; k < ROWS; ++k) t += s[k][j];
        if (a.parts == 1) a.db[g * a.N + col] = to_storage<DT>(t);
        else a.part[(size_t)blockIdx.y * G * a.N + g * a.N + col] = t;
    }
}

// The row groups' column sums added in a fixed order: 32 columns by 8 groups
// of row groups, joined through LDS.  Where both products follow, their launch
// adds them instead.
template <int DT>
__global__ __launch_bounds__(256) void db_kernel(DzArgs a, int n) {
    __shared__ float s[8][33];
    const int lane = threadIdx.x & 31, group = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float v[DZ_PARTS / 8], sum = 0.f;
#pragma unroll
    for (int k = 0; k < DZ_PARTS / 8; ++k) {
        const int p = k * 8 + group;
        v[k] = p < a.parts && c < n ? a.part[(size_t)p * n + c] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < DZ_PARTS / 8; ++k) sum += v[k];
    s[group][lane] = sum;
    __syncthreads();
    if (group != 0 || c >= n) return;
    sum = 0.f;
#pragma unroll
    for (int g = 0; g < 8; ++g) sum += s[g][lane];
    a.db[c] = to_storage<DT>(sum);
}

template <int DT, int ACT>
static hipError_t dz_launch(const DzArgs& a, hipStream_t s) {
    if (a.parts == 1) return launch(dz_kernel<DT, ACT, 64>, dim3((a.N + 63) / 64), DZ_NT, s, a);
    return launch(dz_kernel<DT, ACT, 256>, dim3((a.N + 255) / 256, a.parts), DZ_NT, s, a);
}

template <int DT>
static hipError_t dz_t(const DzArgs& a, bool join, hipStream_t s) {
    hipError_t e = hipSuccess;
    if (a.parts > 0) {
        if (a.act == ACT_NONE) e = dz_launch<DT, ACT_NONE>(a, s);
        else if (a.act == ACT_GELU_TANH) e = dz_launch<DT, ACT_GELU_TANH>(a, s);
        else e = dz_launch<DT, ACT_SWIGLU>(a, s);
    }
    if (e == hipSuccess && a.db && join && a.parts != 1) {
        const int n = a.act == ACT_SWIGLU ? 2 * a.N : a.N;
        e = launch(db_kernel<DT>, dim3((n + 31) / 32), 256, s, a, n);
    }
    return e;
}

}  // namespace mlpc

using namespace mlpc;

int mlpc_dz_max_parts() { return DZ_PARTS; }

// Row groups: one up to 128 rows (the column sums then need no second kernel,
// and its launch costs more than the few rows per thread), else groups of
// about 32 rows.
int mlpc_dz_parts(int64_t rows) {
    if (rows <= 128) return rows > 0 ? 1 : 0;
    const int64_t p = (rows + 31) / 32;
    return (int)(p < DZ_PARTS ? p : DZ_PARTS);
}

hipError_t mlpc_dz(const DzArgs& a, int dtype, bool join, hipStream_t s) {
    return dtype == DT_F16 ? dz_t<DT_F16>(a, join, s) : dz_t<DT_BF16>(a, join, s);
}

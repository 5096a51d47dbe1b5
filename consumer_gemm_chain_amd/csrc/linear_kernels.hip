// linear_kernels.hip -- the products of the linear layer and the activation's
// gradient (include/mlp_block.h has the formulas).
#include <hip/hip_runtime.h>

#include "block_launch.h"
#include "chain_device.hpp"

namespace mlpc {

template <int DT>
__device__ __forceinline__ float widen(uint16_t v) {
    if constexpr (DT == DT_F16) return (float)__builtin_bit_cast(_Float16, v);
    else return __builtin_bit_cast(float, (uint32_t)v << 16);
}

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

constexpr int BT = 64;      // output rows and B columns of a tile
constexpr int KT = 32;      // reduction per step
constexpr int LDT = KT + 8; // padded LDS row

// One 64 x 64 tile per workgroup of four 32 x 32 waves; both operands are
// brought into LDS element by element with the reduction contiguous, so one
// kernel serves every layout.  For swiglu the tile's 16-column fragments
// alternate gate / up.
template <int DT, int PASS>
__global__ __launch_bounds__(256) void gemm_kernel(GemmArgs a) {
    __shared__ __attribute__((aligned(16))) uint16_t sa[BT * LDT], sb[BT * LDT];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = wave >> 1, wn = wave & 1, g = lane >> 4, jj = lane & 15;
    const int width = a.up ? BT / 2 : BT;
    const int nt = (a.N + width - 1) / width;
    const int m0 = (int)(blockIdx.x / nt) * BT, n0 = (int)(blockIdx.x % nt) * width;
    f32x4 acc[2][2] = {};
    for (int k0 = 0; k0 < a.K; k0 += KT) {
        __syncthreads();
        for (int i = tid; i < BT * KT; i += 256) {
            // neighbouring threads follow the operand's contiguous direction
            const int rA = PASS == PASS_DW ? i % BT : i / KT, kA = PASS == PASS_DW ? i / BT : i % KT;
            uint16_t v = 0;
            if (m0 + rA < a.M && k0 + kA < a.K)
                v = PASS == PASS_DW ? a.a[(size_t)(k0 + kA) * a.lda + m0 + rA] : a.a[(size_t)(m0 + rA) * a.lda + k0 + kA];
            sa[rA * LDT + kA] = v;
            const int cB = PASS == PASS_DX ? i / KT : i % BT, kB = PASS == PASS_DX ? i % KT : i / BT;
            const int oc = a.up ? n0 + (cB >> 5) * 16 + (cB & 15) : n0 + cB;
            const int col = a.up ? oc + ((cB >> 4) & 1) * a.up : oc;
            uint16_t w = 0;
            if (oc < a.N && k0 + kB < a.K)
                w = PASS == PASS_DX ? a.b[(size_t)col * a.ldb + k0 + kB] : a.b[(size_t)(k0 + kB) * a.ldb + col];
            sb[cB * LDT + kB] = w;
        }
        __syncthreads();
        u32x4 fa[2], fb[2];
#pragma unroll
        for (int f = 0; f < 2; ++f) {
            fa[f] = *reinterpret_cast<const u32x4*>(&sa[(wm * 32 + f * 16 + jj) * LDT + g * 8]);
            fb[f] = *reinterpret_cast<const u32x4*>(&sb[(wn * 32 + f * 16 + jj) * LDT + g * 8]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) acc[i][j] = mfma16x16x32<DT>(fa[i], fb[j], acc[i][j]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int m = m0 + wm * 32 + i * 16 + g * 4 + q;
            if (m >= a.M) continue;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                if (a.up && j == 1) continue;
                const int n = a.up ? n0 + wn * 16 + jj : n0 + wn * 32 + j * 16 + jj;
                if (n >= a.N) continue;
                float v = acc[i][j][q] + (a.bias ? widen<DT>(a.bias[n]) : 0.f);
                if (a.z) a.z[(size_t)m * a.ldz + n] = to_storage<DT>(v);
                if (a.act == ACT_GELU_TANH) v = gelu_tanh(v);
                if (a.act == ACT_SWIGLU) {
                    const float u = acc[i][1][q] + (a.bias ? widen<DT>(a.bias[n + a.up]) : 0.f);
                    if (a.z) a.z[(size_t)m * a.ldz + n + a.up] = to_storage<DT>(u);
                    v = silu(v) * u;
                }
                if (a.res) v += widen<DT>(a.res[(size_t)m * a.ldr + n]);
                a.d[(size_t)m * a.ldd + n] = to_storage<DT>(v);
            }
        }
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
static hipError_t gemm_t(const GemmArgs& a, int pass, hipStream_t s) {
    const int width = a.up ? BT / 2 : BT;
    const dim3 grid((unsigned)((a.M + BT - 1) / BT) * (unsigned)((a.N + width - 1) / width));
    switch (pass) {
    case PASS_FWD: hipLaunchKernelGGL((gemm_kernel<DT, PASS_FWD>), grid, dim3(256), 0, s, a); break;
    case PASS_DX: hipLaunchKernelGGL((gemm_kernel<DT, PASS_DX>), grid, dim3(256), 0, s, a); break;
    default: hipLaunchKernelGGL((gemm_kernel<DT, PASS_DW>), grid, dim3(256), 0, s, a);
    }
    return hipGetLastError();
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

hipError_t mlpc_gemm(const GemmArgs& a, int pass, int dtype, hipStream_t s) {
    return dtype == DT_F16 ? gemm_t<DT_F16>(a, pass, s) : gemm_t<DT_BF16>(a, pass, s);
}

hipError_t mlpc_dz(const DzArgs& a, int dtype, hipStream_t s) {
    return dtype == DT_F16 ? dz_t<DT_F16>(a, s) : dz_t<DT_BF16>(a, s);
}

int mlpc_dz_max_parts() { return 64; }

int mlpc_dz_parts(int64_t rows) { return (int)(rows < 64 ? rows : 64); }

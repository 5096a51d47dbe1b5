// optim_kernels.hip -- the norm of all gradients and the AdamW step, over
// tables of tensors that travel with the launch.
#include <hip/hip_runtime.h>

#include "linear_device.hpp"
#include "train_launch.h"

namespace mlpc {

constexpr int ONT = 256;

// Elements need no more than their own alignment: gfx950 loads and stores 8 or
// 16 bytes at any address.
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));

// The entry of a table whose chunks begin at first[i] that chunk c belongs to
// (scalar): lanes compare, their ballot counts.
__device__ __forceinline__ int entry_of(const uint32_t* first, int count, uint32_t c) {
    const int lane = threadIdx.x & 63;
    int t = 0;
    for (int i = 0; i < count; i += 64) t += __popcll(__ballot(i + lane < count && first[i + lane] <= c));
    return __builtin_amdgcn_readfirstlane(t - 1);
}

// ---------------------------------------------------------------------- norm

// Sum over a wave in a fixed order.
__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d);
    return v;
}

// A workgroup's share of the launch's chunks, neighbours, to its partial sum.
// Reading the gradients bounds it: 302 MB of bf16 in 54 us (5.6 TB/s; 50 us where
// part of them is still in the Infinity Cache), 101 MB of fp16 in 144 tensors in 27.
// A square of 16 bits is exact in 64, and gradients of 1e-25 or 1e30 neither vanish
// nor overflow, so no scaling pass is needed; the products in 64 bits stay hidden
// behind the loads.
template <int DT>
__global__ __launch_bounds__(ONT) void norm_sum_kernel(NormTable a) {
    __shared__ double s[ONT / 64];
    const uint32_t c0 = (uint32_t)((uint64_t)a.chunks * blockIdx.x / gridDim.x);
    const uint32_t c1 = (uint32_t)((uint64_t)a.chunks * (blockIdx.x + 1) / gridDim.x);
    double sum = 0.0;
    for (uint32_t c = c0; c < c1; ++c) {
        const int i = entry_of(a.first, a.count, c);
        const int64_t n = a.n[i], at = (int64_t)(c - a.first[i]) * NORM_CHUNK;
        const uint16_t* g = a.grad[i];
#pragma unroll
        for (int k = 0; k < NORM_CHUNK / (8 * ONT); ++k) {
            const int64_t e = at + (k * ONT + threadIdx.x) * 8;
            if (e + 8 <= n) {
                float f[8];
                widen8<DT>(*reinterpret_cast<const u32x4_any*>(g + e), f);
#pragma unroll
                for (int j = 0; j < 8; ++j) sum = __builtin_fma((double)f[j], (double)f[j], sum);
            } else {
                for (int64_t j = e; j < n; ++j) {
                    const double f = widen<DT>(g[j]);
                    sum = __builtin_fma(f, f, sum);
                }
            }
        }
    }
    sum = wave_sum64(sum);
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = sum;
    __syncthreads();
    if (threadIdx.x != 0) return;
    sum = (s[0] + s[1]) + (s[2] + s[3]);
    a.part[blockIdx.x] = a.add ? a.part[blockIdx.x] + sum : sum;
}

// The partial sums to the norm and the gradients' scale: 16 KB, 4 us, nearly all
// of it the launch and two dependent trips to memory.
__global__ __launch_bounds__(ONT) void norm_join_kernel(NormJoin a) {
    __shared__ double s[ONT / 64];
    double p[NORM_PARTS / ONT], sum = 0.0;
#pragma unroll
    for (int k = 0; k < NORM_PARTS / ONT; ++k) p[k] = k * ONT + threadIdx.x < a.parts ? a.part[k * ONT + threadIdx.x] : 0.0;
#pragma unroll
    for (int k = 0; k < NORM_PARTS / ONT; ++k) sum += p[k];
    sum = wave_sum64(sum);
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = sum;
    __syncthreads();
    if (threadIdx.x != 0) return;
    const double norm = fabs(a.unscale) * sqrt((s[0] + s[1]) + (s[2] + s[3]));
    *a.norm = (float)norm;
    if (!a.scale) return;
    const double clip = norm > a.max_norm ? a.max_norm / norm : 1.0;
    *a.scale = (float)norm < INFINITY ? (float)(a.unscale * clip) : NAN;
}

// --------------------------------------------------------------------- adamw

// 32 well mixed bits of 32: two rounds of shift, xor and product with an odd
// number (the fraction bits of the square roots of 2 and 3).
__device__ __forceinline__ uint32_t mix(uint32_t x) {
    x = (x ^ (x >> 16)) * 0x6A09E667u;
    x = (x ^ (x >> 15)) * 0xBB67AE85u;
    return x ^ (x >> 16);
}

// What every workgroup of the step needs, once: its number, the bias
// corrections in 64 bits, and whether it is left out.
__global__ __launch_bounds__(64) void adamw_begin_kernel(AdamBegin a) {
    if (threadIdx.x != 0) return;
    const float scale = a.scale ? *a.scale : 1.f;
    AdamStep q{};
    q.run = fabsf(scale) < INFINITY;
    if (q.run) {
        const int64_t t = *a.t + 1;
        *a.t = t;
        const double lr = a.lr * (a.lr_scale ? (double)*a.lr_scale : 1.0);
        q.scale = scale;
        q.lr = lr;
        q.size = (float)(lr / (1.0 - pow(a.beta1, (double)t)));
        q.root = (float)(1.0 / sqrt(1.0 - pow(a.beta2, (double)t)));
        q.key = mix((uint32_t)t + a.seed);
    }
    *a.step = q;
}

// sqrt of a number that may be too small for the hardware's.
__device__ __forceinline__ float root_of(float v) {
    const bool small = v < 0x1p-96f;
    const float r = __builtin_amdgcn_sqrtf(small ? v * 0x1p64f : v);
    return small ? r * 0x1p-32f : r;
}

// Largest of a block of 32 lanes, in all of them: rotations within rows of 16
// lanes, then a swap between rows.
__device__ __forceinline__ uint32_t block_max(uint32_t v) {
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xf, 0xf, false));      // row_ror:8
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x124, 0xf, 0xf, false));
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x122, 0xf, 0xf, false));
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x121, 0xf, 0xf, false));
    const auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    const uint32_t p0 = p[0], p1 = p[1];
    return max(p0, p1);
}

// The power of two with which `top` (its bits) stays within a type whose
// largest number is 1.75 2^EXP, and its inverse.
template <int EXP>
__device__ __forceinline__ float block_scale(uint32_t top, float& inverse) {
    int e = (int)(top >> 23) - EXP + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = max(e, 1);
    if (top == 0) e = 127;
    inverse = __builtin_bit_cast(float, (uint32_t)(254 - e) << 23);
    return __builtin_bit_cast(float, (uint32_t)e << 23);
}

__device__ __forceinline__ uint32_t bits_of(float v) { return __builtin_bit_cast(uint32_t, v); }

constexpr uint32_t INF_BITS = 0x7f800000u;

// AdamW of one chunk of a tensor: 8 elements per thread, so that each access has
// 16 bytes (8-bit states: 8).  One pass over memory bounds it.  An element moves
// 28 bytes with 32-bit states and master weights (151 million of them 779 us, 5.4
// TB/s, a copy's rate) and 16 with 8-bit ones (117 million 352 us, 5.4 TB/s).  A
// chunk has 2048 elements, eight blocks of 8-bit states, whose largest magnitude 32
// lanes find among themselves: no LDS and no barrier.
template <int DT, int BITS, bool WHOLE>
__device__ __forceinline__ void adamw_chunk(const AdamTable& a, const AdamStep& q, int i, uint32_t c) {
    const int64_t n = a.n[i], e = (int64_t)c * ADAM_CHUNK + threadIdx.x * 8;
    const int left = WHOLE ? 8 : (int)(n - e < 0 ? 0 : n - e < 8 ? n - e : 8);
    const uint16_t* grad = a.grad[i] + e;
    uint16_t* w16 = a.w[i] + e;
    float* master = a.master[i] ? a.master[i] + e : nullptr;
    float g[8], w[8], m[8], v[8];
    auto load = [&](const float* p, float (&f)[8]) {
        if (left == 8) {
            const f32x4 lo = reinterpret_cast<const f32x4_any*>(p)[0], hi = reinterpret_cast<const f32x4_any*>(p)[1];
#pragma unroll
            for (int k = 0; k < 4; ++k) f[k] = lo[k], f[4 + k] = hi[k];
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) f[k] = k < left ? p[k] : 0.f;
        }
    };
    auto load16 = [&](const uint16_t* p, float (&f)[8]) {
        if (left == 8) widen8<DT>(*reinterpret_cast<const u32x4_any*>(p), f);
        else {
#pragma unroll
            for (int k = 0; k < 8; ++k) f[k] = k < left ? widen<DT>(p[k]) : 0.f;
        }
    };
    auto load8 = [&](const uint8_t* p) {
        uint64_t b = 0;
        if (left == 8) {
            const u32x2_any t = *reinterpret_cast<const u32x2_any*>(p);
            return u32x2{t[0], t[1]};
        }
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < left) b |= (uint64_t)p[k] << (8 * k);
        return u32x2{(uint32_t)b, (uint32_t)(b >> 32)};
    };
    auto store = [&](float* p, const float (&f)[8]) {
        if (left == 8) {
            reinterpret_cast<f32x4_any*>(p)[0] = f32x4{f[0], f[1], f[2], f[3]};
            reinterpret_cast<f32x4_any*>(p)[1] = f32x4{f[4], f[5], f[6], f[7]};
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < left) p[k] = f[k];
        }
    };
    auto store8 = [&](uint8_t* p, u32x2 t) {
        if (left == 8) {
            *reinterpret_cast<u32x2_any*>(p) = u32x2_any{t[0], t[1]};
            return;
        }
        const uint64_t b = (uint64_t)t[1] << 32 | t[0];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < left) p[k] = (uint8_t)(b >> (8 * k));
    };
    load16(grad, g);
    if (master) load(master, w);
    else load16(w16, w);
    const int64_t block = e / 256;
    float b1 = a.beta1, b2 = a.beta2;
    if constexpr (BITS == 32) {
        load(static_cast<const float*>(a.m[i]) + e, m);
        load(static_cast<const float*>(a.v[i]) + e, v);
    } else {
        const u32x2 mc = load8(static_cast<const uint8_t*>(a.m[i]) + e), vc = load8(static_cast<const uint8_t*>(a.v[i]) + e);
        // (scales are powers of two: taken with beta, they round nothing)
        b1 *= left ? a.m_scale[i][block] : 0.f;
        b2 *= left ? a.v_scale[i][block] : 0.f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const auto m0 = __builtin_amdgcn_cvt_pk_f32_fp8(mc[k], false), m1 = __builtin_amdgcn_cvt_pk_f32_fp8(mc[k], true);
            const auto v0 = __builtin_amdgcn_cvt_pk_f32_bf8(vc[k], false), v1 = __builtin_amdgcn_cvt_pk_f32_bf8(vc[k], true);
            m[4 * k] = m0[0], m[4 * k + 1] = m0[1], m[4 * k + 2] = m1[0], m[4 * k + 3] = m1[1];
            v[4 * k] = v0[0], v[4 * k + 1] = v0[1], v[4 * k + 2] = v1[0], v[4 * k + 3] = v1[1];
        }
    }
    const float decay = (float)(q.lr * a.decay[i]);
    auto update = [&](auto root) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float s = g[k] * q.scale;
            m[k] = m[k] * b1 + s * a.rest1;
            v[k] = v[k] * b2 + (s * s) * a.rest2;
            // (hardware root and reciprocal: ulps of the step's change; the decay is part of the change, because a factor of
            // 1 - 1e-6 rounded to fp32 decays by 1.3% more than that at every step)
            w[k] -= __builtin_fmaf(decay, w[k], q.size * (m[k] * __builtin_amdgcn_rcpf(root(v[k]) * q.root + a.eps)));
        }
    };
    // the hardware's root takes subnormal v as 0: beside an eps of 2^-39 and more that changes nothing
    if (a.eps >= 0x1p-39f) update([](float x) { return __builtin_amdgcn_sqrtf(x); });
    else update([](float x) { return root_of(x); });
    if (master) store(master, w);
    if (left == 8) *reinterpret_cast<u32x4_any*>(w16) = narrow8<DT>(w);
    else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < left) w16[k] = to_storage<DT>(w[k]);
    }
    if constexpr (BITS == 32) {
        store(static_cast<float*>(a.m[i]) + e, m);
        store(static_cast<float*>(a.v[i]) + e, v);
    } else {
        // magnitudes compare like their bits; elements that are not there are 0
        uint32_t mt = 0, vt = 0, low = ~0u;     // low: of the smallest m but 0, less 1
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint32_t mb = bits_of(m[k]) & 0x7fffffffu;
            mt = max(mt, mb), low = min(low, mb - 1u), vt = max(vt, bits_of(v[k]) & 0x7fffffffu);
        }
        const bool numbers = !__any(max(mt, vt) >= INF_BITS);
        if (!numbers) {
            // what is no number leaves the scale alone and becomes NaN
            mt = vt = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                uint32_t mb = bits_of(m[k]) & 0x7fffffffu, vb = bits_of(v[k]) & 0x7fffffffu;
                pin(mb), pin(vb);       // (the branch is hardly ever taken: nothing of it before it)
                if (mb < INF_BITS) mt = max(mt, mb);
                else m[k] = NAN;
                if (vb < INF_BITS) vt = max(vt, vb);
            }
        }
        float mi, vi;
        const float ms = block_scale<8>(block_max(mt), mi), vs = block_scale<15>(block_max(vt), vi);
        u32x2 mc = {0, 0}, vc = {0, 0};
        const uint32_t key = mix(q.key + 0x9E3779B9u * (uint32_t)(a.number + i)) + (uint32_t)(e >> 1);
        // v in units of its scale (which may underflow), at least the smallest number unless it is 0
        auto unit = [&](float x) {
            return fmaxf(x * vi, x > 0.f ? 0x1p-16f : 0.f);
        };
        static_for<0, 4>([&](auto j) {
            constexpr int K = decltype(j)::value * 2, W = K / 4, B = K % 4;
            const uint32_t r = mix(key + K / 2);
            vc[W] = __builtin_amdgcn_cvt_sr_bf8_f32(unit(v[K]), r << 16, vc[W], B);
            vc[W] = __builtin_amdgcn_cvt_sr_bf8_f32(unit(v[K + 1]), r & 0xffff0000u, vc[W], B + 1);
            mc[W] = __builtin_amdgcn_cvt_pk_fp8_f32(m[K] * mi, m[K + 1] * mi, mc[W], B != 0);
        });
        // Where a step moves m by less than half a code, rounding to nearest would leave it
        // as it was for good: with a large beta1 (chance) anywhere, with any below the
        // normal numbers (of codes up to 4 a beta1 of 0.9 takes less than half of one).
        // There m is rounded by chance, with the random bits of its neighbour's v.  (An m
        // that was 0 stays 0 below half a code, to nearest: that moves no weight.)
        // (Off the common path, and with m's codes read again: kept, they cost a wave of
        // seven per SIMD, and 50 million elements in 144 tensors took 112 us, not 107.)
        if (a.chance || __any(low < bits_of(0x1p-6f * ms) - 1u)) {
            const u32x2 old = load8(static_cast<const uint8_t*>(a.m[i]) + e);
            const float old_unit = (left ? a.m_scale[i][block] : 0.f) * mi;
            static_for<0, 8>([&](auto j) {
                constexpr int K = decltype(j)::value, W = K / 4, B = K % 4;
                const uint32_t r = mix(key + K / 2), bits = K % 2 == 0 ? r & 0xffff0000u : r << 16, code = mc[W] >> (8 * B) & 0x7fu;
                const auto was = __builtin_amdgcn_cvt_pk_f32_fp8(old[W], B >= 2);
                const float y = m[K] * mi;
                // (a subnormal code is its number in units of 2^-9)
                const bool stays = fabsf(y) < 0x1p-6f && code != 0 && fabsf(was[K % 2]) * old_unit == (float)code * 0x1p-9f;
                if (a.chance || stays) mc[W] = __builtin_amdgcn_cvt_sr_fp8_f32(y, bits, mc[W], B);
            });
        }
        if (!numbers) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                uint32_t vb = bits_of(v[k]) & 0x7fffffffu;
                pin(vb);
                if (vb >= INF_BITS) vc[k / 4] |= 0x7fu << (8 * (k % 4));
            }
        }
        store8(static_cast<uint8_t*>(a.m[i]) + e, mc);
        store8(static_cast<uint8_t*>(a.v[i]) + e, vc);
        if ((threadIdx.x & 31) == 0 && left) {
            a.m_scale[i][block] = ms;
            a.v_scale[i][block] = vs;
        }
    }
}

template <int DT, int BITS>
__global__ __launch_bounds__(ONT) void adamw_kernel(AdamTable a) {
    const AdamStep q = *a.step;
    if (!q.run) return;
    const int i = entry_of(a.first, a.count, blockIdx.x);
    const uint32_t c = blockIdx.x - a.first[i];
    if ((int64_t)(c + 1) * ADAM_CHUNK <= a.n[i]) adamw_chunk<DT, BITS, true>(a, q, i, c);
    else adamw_chunk<DT, BITS, false>(a, q, i, c);
}

}  // namespace mlpc

using namespace mlpc;

hipError_t mlpc_norm_sum(const NormTable& a, int dtype, int parts, hipStream_t s) {
    return launch(dtype == DT_F16 ? norm_sum_kernel<DT_F16> : norm_sum_kernel<DT_BF16>, dim3(parts), ONT, s, a);
}

hipError_t mlpc_norm_join(const NormJoin& a, hipStream_t s) { return launch(norm_join_kernel, dim3(1), ONT, s, a); }

hipError_t mlpc_adamw_begin(const AdamBegin& a, hipStream_t s) { return launch(adamw_begin_kernel, dim3(1), 64, s, a); }

hipError_t mlpc_adamw(const AdamTable& a, int dtype, int bits, hipStream_t s) {
    if (bits == 32) return launch(dtype == DT_F16 ? adamw_kernel<DT_F16, 32> : adamw_kernel<DT_BF16, 32>, dim3(a.chunks), ONT, s, a);
    return launch(dtype == DT_F16 ? adamw_kernel<DT_F16, 8> : adamw_kernel<DT_BF16, 8>, dim3(a.chunks), ONT, s, a);
}

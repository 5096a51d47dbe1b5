// norm_kernels.hip -- layer norm, forward and backward (include/mlp_block.h
// has the formulas).
//
// Rows of up to 16384 elements are held in registers: a group of threads
// takes a row, V chunks of 8 elements each, so x (and dy) is read once, the
// variance comes from centred values and the row is written from registers.
// Both passes are bound by memory.  Longer rows, and those of fewer
// than 8, take kernels that read a row once per sweep over it.
//
// Rows need only 2-byte alignment: gfx950 loads and stores 16 bytes at any
// address, so a row stride or width that is no multiple of 8 costs the extra
// cache lines it touches.  (Values stay packed between the sweeps over the registers, behind
// an empty asm each time: the compiler would otherwise keep their fp32 copies
// and halve the waves per CU.)
#include <hip/hip_runtime.h>

#include "block_launch.h"
#include "chain_device.hpp"
#include "linear_device.hpp"

namespace mlpc {

typedef u32x4 u32x4_any __attribute__((aligned(2)));

// Where chunk c (a multiple of 8, c < H) of a row is moved: at c, or where H
// is no multiple of 8 (RAGGED) and the row ends inside it, at the row's last
// 8 elements.  The first c - place of those belong to the chunk before: they
// add nothing to sums and are not stored.
template <bool RAGGED>
__device__ __forceinline__ int place(int c, int H) {
    if constexpr (RAGGED) return min(c, H - 8);
    else return c;
}

// (`row` is wave-uniform: a scalar base and a 32-bit lane offset.)
__device__ __forceinline__ u32x4 load8(const uint16_t* row, int c) {
    return *reinterpret_cast<const u32x4_any*>(row + (uint32_t)c);
}

// The last 8 - skip of eight elements.
template <bool RAGGED>
__device__ __forceinline__ void store8(uint16_t* row, int c, int skip, u32x4 v) {
    if (!RAGGED || skip == 0) {
        *reinterpret_cast<u32x4_any*>(row + (uint32_t)c) = v;
        return;
    }
#pragma unroll
    for (int i = 1; i < 8; ++i)
        if (i >= skip) row[(uint32_t)c + i] = (uint16_t)(v[i >> 1] >> (16 * (i & 1)));
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ float uniform(float v) { return __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, v))); }

// v + v rotated by N lanes within each row of 16.
template <int N>
__device__ __forceinline__ float add_rotated(float v) {
    const int r = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x120 + N, 0xf, 0xf, false);
    return v + __builtin_bit_cast(float, r);
}

// Sum over the wave, the same bits in every lane: rotations within rows of 16
// lanes, then swaps between rows (no LDS).
__device__ __forceinline__ float wave_sum(float v) {
    v = add_rotated<1>(add_rotated<2>(add_rotated<4>(add_rotated<8>(v))));
    uint32_t u = __builtin_bit_cast(uint32_t, v);
    const auto p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    const uint32_t p0 = p[0], p1 = p[1];
    v = __builtin_bit_cast(float, p0) + __builtin_bit_cast(float, p1);
    u = __builtin_bit_cast(uint32_t, v);
    const auto q = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const uint32_t q0 = q[0], q1 = q[1];
    return __builtin_bit_cast(float, q0) + __builtin_bit_cast(float, q1);
}

// ------------------------------------------------------------------- forward

constexpr int FWD_NT = 256;

// TR (64 or 256) threads per row, V chunks per thread.  A workgroup keeps
// weight and bias in registers over the rows it takes.  Bound by memory: 8192 x
// 8192 bf16 51.5 us, 5.2 TB/s (a 1 GiB copy reaches 5.17); 2048 x 12288 f16
// 22.3 us, 4.5 TB/s (too few rows for a second per workgroup); 1 x 512 1.8 us.
template <int DT, int TR, int V, bool RAGGED>
__global__ __launch_bounds__(FWD_NT, V <= 2 ? 8 : V <= 4 ? 5 : 4) void norm_forward_kernel(NormArgs a) {
    constexpr int RPW = FWD_NT / TR;
    __shared__ float s[2][FWD_NT / 64];
    const int t = threadIdx.x % TR, sub = uniform((int)(threadIdx.x / TR));
    u32x4 w[V], b[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = (i * TR + (int)fresh(t)) * 8;
        if (c < a.H) {
            if (a.weight) w[i] = load8(a.weight, place<RAGGED>(c, a.H));
            if (a.bias) b[i] = load8(a.bias, place<RAGGED>(c, a.H));
        }
    }
    const float inv = 1.0f / a.H;
    // zeroes what chunk i shares with the chunk before
    auto mask = [&](int i, float (&f)[8]) {
        if constexpr (RAGGED) {
            // (recomputed at each use: kept, the conditions of every chunk take too many registers)
            const int skip = (i * TR + (int)fresh(t)) * 8 - (a.H - 8);
#pragma unroll
            for (int k = 0; k < 7; ++k) f[k] = k < skip ? 0.f : f[k];
        }
    };
    auto row_sum = [&](float v, int k) {
        v = wave_sum(v);
        if constexpr (TR == 64) return v;
        if ((threadIdx.x & 63) == 0) s[k][threadIdx.x >> 6] = v;
        __syncthreads();
        return (s[k][0] + s[k][1]) + (s[k][2] + s[k][3]);
    };
    // (whole workgroups leave the loop together: the sums meet at barriers)
    for (int64_t r0 = (int64_t)blockIdx.x * RPW; r0 < a.rows; r0 += (int64_t)gridDim.x * RPW) {
        const int64_t r = r0 + sub < a.rows ? r0 + sub : a.rows - 1;
        const uint16_t* x = a.x + r * a.ldx;
        u32x4 v[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (i * TR + (int)fresh(t)) * 8;
            v[i] = c < a.H ? load8(x, place<RAGGED>(c, a.H)) : u32x4{0, 0, 0, 0};
        }
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float f[8];
            widen8<DT>(v[i], f);
            mask(i, f);
            sum += ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
        }
        const float mean = row_sum(sum, 0) * inv;
        float var = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if ((i * TR + (int)fresh(t)) * 8 >= a.H) continue;
            float f[8];
            pin(v[i]);
            widen8<DT>(v[i], f);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                f[k] -= mean;
                f[k] *= f[k];
            }
            mask(i, f);
            var += ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
        }
        const float rstd = 1.0f / sqrtf(row_sum(var, 1) * inv + a.eps);
        if (r0 + sub >= a.rows) continue;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (i * TR + (int)fresh(t)) * 8;
            if (c >= a.H) continue;
            float f[8], p[8];
            pin(v[i]);
            widen8<DT>(v[i], f);
#pragma unroll
            for (int k = 0; k < 8; ++k) f[k] = (f[k] - mean) * rstd;
            if (a.weight) {
                pin(w[i]);
                widen8<DT>(w[i], p);
#pragma unroll
                for (int k = 0; k < 8; ++k) f[k] *= p[k];
            }
            if (a.bias) {
                pin(b[i]);
                widen8<DT>(b[i], p);
#pragma unroll
                for (int k = 0; k < 8; ++k) f[k] += p[k];
            }
            const int at = place<RAGGED>(c, a.H);
            store8<RAGGED>(a.y + r * a.ldy, at, c - at, narrow8<DT>(f));
        }
        if (t == 0) {
            if (a.mean) a.mean[r] = mean;
            if (a.rstd) a.rstd[r] = rstd;
        }
    }
}

// ------------------------------------------------------------------ backward

constexpr int MAX_PARTS = 256;      // workgroups that keep column sums: one per CU

// TR threads per row (whole waves, a divisor of NT), V chunks per thread, NT / TR rows at a time.  A workgroup walks the rows with its
// columns' sums in registers and the next rows' loads in flight, and leaves
// one row of partial sums: large workgroups, one per CU, keep those
// partials (8 H bytes each) small against the rows.  A row needs the sums of g
// and g xhat; xhat itself is kept, for with (x - mean) and a factor of rstd^2
// rows with an rstd past 1.8e19 would overflow.  Bound by memory, the partials included: with
// dres, 8192 x 8192 bf16 102 us, 5.3 TB/s of the operands; 2048 x 12288 f16
// 44.6 us for 201 MB of operands and 25 MB of partials, 5.1 TB/s; 1000 x 8192
// 16.6 us (four rows per workgroup, whose loads are a chain).
template <int DT, int NT, int V, bool RAGGED, bool ALONE>
__global__ __launch_bounds__(NT) void norm_backward_kernel(NormArgs a, int TR) {
    __shared__ float s[2][NT / 64][2];
    __shared__ float cols[NT * 8];      // one chunk of every thread's column sums
    const int sub = uniform((int)(threadIdx.x / TR)), rpw = NT / TR;
    const uint32_t t = threadIdx.x - sub * TR;
    const int wave = threadIdx.x >> 6, first = sub * (TR / 64), waves = TR / 64;
    const float inv = 1.0f / a.H;
    const uint32_t one = DT == DT_F16 ? 0x3c003c00u : 0x3f803f80u;     // 1, 1: no weight
    u32x4 w[V];
    float sw[V][8] = {}, sb[V][8] = {};
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = (i * TR + (int)fresh(t)) * 8;
        w[i] = a.weight && c < a.H ? load8(a.weight, place<RAGGED>(c, a.H)) : u32x4{one, one, one, one};
    }
    // the next row's dres too, requested with x and dy: 2048 x 12288 47 -> 44
    // us; 16 waves' registers hold it only beside one chunk (with two they spill)
    constexpr bool EARLY = V == 1 || NT <= 768;
    u32x4 x[V], dy[V], dn[V];
    float mean = 0.f, rstd = 0.f;
    // row r's x, dy and statistics; a group past the last row takes that row's
    // x with dy = 0, which adds nothing to any sum
    auto fetch = [&](int64_t r) {
        const bool live = r < a.rows;
        if (!live) r = a.rows - 1;
        mean = a.mean[r];
        rstd = a.rstd[r];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (i * TR + (int)fresh(t)) * 8;
            x[i] = dy[i] = u32x4{0, 0, 0, 0};
            if (c < a.H) {
                x[i] = load8(a.x + r * a.ldx, place<RAGGED>(c, a.H));
                if (live) dy[i] = load8(a.dy + r * a.lddy, place<RAGGED>(c, a.H));
                if (EARLY && a.dres && live) dn[i] = load8(a.dres + r * a.lddres, place<RAGGED>(c, a.H));
            }
        }
    };
    const int64_t step = (int64_t)gridDim.x * rpw;
    int64_t r0 = (int64_t)blockIdx.x * rpw;
    fetch(r0 + sub);
    for (int buf = 0; r0 < a.rows; r0 += step, buf ^= 1) {
        const int64_t r = r0 + sub;
        const bool live = r < a.rows;
        u32x4 cx[V], cdy[V], dr[V];
        const float m = uniform(mean), rs = uniform(rstd);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            cx[i] = x[i];
            cdy[i] = dy[i];
            if constexpr (EARLY) {
                dr[i] = dn[i];
            } else {
                const int c = (i * TR + (int)fresh(t)) * 8;
                if (a.dres && live && c < a.H) dr[i] = load8(a.dres + r * a.lddres, place<RAGGED>(c, a.H));
            }
        }
        if (r0 + step < a.rows) fetch(r + step);
        // dy, g and xhat of chunk i (where dy = 0, past the row or shared with
        // the chunk before, so is all that is summed)
        auto terms = [&](int i, float (&e)[8], float (&g)[8], float (&xhat)[8]) {
            pin(cdy[i]);
            pin(cx[i]);
            widen8<DT>(cdy[i], e);
            widen8<DT>(cx[i], xhat);
            if constexpr (RAGGED) {
                const int skip = (i * TR + (int)fresh(t)) * 8 - (a.H - 8);
#pragma unroll
                for (int k = 0; k < 7; ++k) e[k] = k < skip ? 0.f : e[k];
            }
            pin(w[i]);
            widen8<DT>(w[i], g);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                g[k] *= e[k];
                xhat[k] = (xhat[k] - m) * rs;
            }
        };
        float t0 = 0.f, t1 = 0.f;
        float g[V][8], xhat[V][8];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float e[8], u0 = 0.f, u1 = 0.f;
            terms(i, e, g[i], xhat[i]);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                // (two chains each)
                float& v0 = k & 1 ? u0 : t0;
                float& v1 = k & 1 ? u1 : t1;
                v0 += g[i][k];
                v1 = __builtin_fmaf(g[i][k], xhat[i][k], v1);
                sb[i][k] += e[k];
                sw[i][k] = __builtin_fmaf(e[k], xhat[i][k], sw[i][k]);
            }
            t0 += u0;
            t1 += u1;
            __builtin_amdgcn_sched_barrier(0);      // one chunk's fp32 values at a time
        }
        t0 = wave_sum(t0);
        t1 = wave_sum(t1);
        if (waves > 1) {
            // (two sets of sums: a wave writes its next row's only after this row's barrier)
            if ((threadIdx.x & 63) == 0) {
                s[buf][wave][0] = t0;
                s[buf][wave][1] = t1;
            }
            __syncthreads();
            t0 = t1 = 0.f;
#pragma unroll 4
            for (int k = 0; k < waves; ++k) {
                t0 += s[buf][first + k][0];
                t1 += s[buf][first + k][1];
            }
        }
        if (!live) continue;
        const float b0 = -rs * (t0 * inv), b1 = -rs * (t1 * inv);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (i * TR + (int)fresh(t)) * 8;
            if (c >= a.H) continue;
            float e[8];
            // 16 waves' registers do not hold two chunks' fp32 values beside
            // the sums: taken again from the packed ones
            if constexpr (V > 1 && NT > 768) terms(i, e, g[i], xhat[i]);
#pragma unroll
            for (int k = 0; k < 8; ++k) e[k] = __builtin_fmaf(xhat[i][k], b1, __builtin_fmaf(g[i][k], rs, b0));
            if (a.dres) {
                float q[8];
                widen8<DT>(dr[i], q);
#pragma unroll
                for (int k = 0; k < 8; ++k) e[k] += q[k];
            }
            const int at = place<RAGGED>(c, a.H);
            store8<RAGGED>(a.dx + r * a.lddx, at, c - at, narrow8<DT>(e));
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    if (!a.dweight && !a.dbias) return;
    // the row groups' sums, chunk by chunk through LDS, added in group order
    // and written as the workgroup's row of partials, or as the gradients
    // themselves by one that has every row (ALONE; as a branch on a.parts it cost
    // 2048 x 12288 1 us)
    float* part = a.part + (size_t)blockIdx.x * 2 * a.H;
    auto join = [&](float (&v)[8], int i, float* row, uint16_t* out) {
        if (ALONE && !out) return;
        const int c = (i * TR + (int)t) * 8, at = c < a.H ? place<RAGGED>(c, a.H) : c;
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (!RAGGED || at + e >= c) cols[(sub * TR - i * TR) * 8 + at + e] = v[e];
        __syncthreads();
        for (int j = threadIdx.x; j < TR * 8; j += NT) {
            if (i * TR * 8 + j >= a.H) continue;
            float sum = cols[j];
#pragma unroll 4
            for (int k = 1; k < rpw; ++k) sum += cols[k * TR * 8 + j];
            if constexpr (ALONE) out[i * TR * 8 + j] = to_storage<DT>(sum);
            else row[i * TR * 8 + j] = sum;
        }
    };
#pragma unroll
    for (int i = 0; i < V; ++i) {
        join(sw[i], i, part, a.dweight);
        join(sb[i], i, part + a.H, a.dbias);
    }
}

// The workgroups' partial column sums added in a fixed order: 32 columns by
// 32 groups of parts, every part's load of a thread in flight at once, the
// groups joined through LDS.  256 parts of 12288: 5.9 us, 4.3 TB/s (14-16 us
// with 16 loads one after the other in each thread).
template <int DT>
__global__ __launch_bounds__(1024) void norm_cols_sum_kernel(NormArgs a) {
    __shared__ float s[32][33];
    const int64_t n = 2 * (int64_t)a.H;
    const int lane = threadIdx.x & 31, group = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    float v[MAX_PARTS / 32], sum = 0.f;
#pragma unroll
    for (int k = 0; k < MAX_PARTS / 32; ++k) {
        const int p = k * 32 + group;
        v[k] = p < a.parts && c < n ? a.part[(size_t)p * n + c] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < MAX_PARTS / 32; ++k) sum += v[k];
    s[group][lane] = sum;
    __syncthreads();
    if (group != 0 || c >= n) return;
    sum = 0.f;
#pragma unroll 8
    for (int g = 0; g < 32; ++g) sum += s[g][lane];
    if (c < a.H) {
        if (a.dweight) a.dweight[c] = to_storage<DT>(sum);
    } else if (a.dbias) {
        a.dbias[c - a.H] = to_storage<DT>(sum);
    }
}

// ------------------------------- rows of fewer than 8 or more than 16384

// Right for every size, not fast: bound by the latency of 2-byte accesses.  Whole
// calls, forward and gradient, f16: 2048 x 20000 145 and 240 us (floors 32 and 63),
// 256 x 40000 146 and 249 (8 and 16), 8192 x 4 8.8 and 23.

constexpr int LONG_ROW = 16384;
static bool held(int H) { return H >= 8 && H <= LONG_ROW; }
constexpr int SWEEP_NT = 256;

// Sum over the workgroup, the same bits in every thread.
__device__ __forceinline__ float block_sum(float v, float* s) {
    v = wave_sum(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
    return (s[0] + s[1]) + (s[2] + s[3]);
}

struct Two {
    float a, b;
};

// Sums of both values of f over first, first + step, .. below end, in chains of
// 64 additions: with one chain of 16384 over a row of 2^22, whose mean is 1000
// times its spread, rstd is off by 3e-5.
template <class I, class F>
__device__ __forceinline__ Two chained_sum(I first, I end, int step, F f) {
    Two t = {0.f, 0.f};
    for (I b = first; b < end; b += 64 * step) {
        Two u = {0.f, 0.f};
        const I stop = min(b + 64 * step, end);
        for (I i = b; i < stop; i += step) {
            const Two v = f(i);
            u.a += v.a;
            u.b += v.b;
        }
        t.a += u.a;
        t.b += u.b;
    }
    return t;
}

// At most this many workgroups, which then walk the rows: a launch of one per
// row would pass HIP's limit of 2^32 threads at 2^24 rows.
constexpr int64_t SWEEP_GRID = 1 << 16;
static dim3 sweep_grid(int64_t rows) { return dim3((unsigned)(rows < SWEEP_GRID ? rows : SWEEP_GRID)); }

// One workgroup per row: three sweeps, the second and third from the caches.
template <int DT>
__global__ __launch_bounds__(SWEEP_NT) void norm_forward_sweep_kernel(NormArgs a) {
    __shared__ float s[SWEEP_NT / 64];
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const uint16_t* x = a.x + r * a.ldx;
        const Two sum = chained_sum((int)threadIdx.x, a.H, SWEEP_NT, [&](int c) { return Two{widen<DT>(x[c]), 0.f}; });
        const float mean = block_sum(sum.a, s) / a.H;
        const Two var = chained_sum((int)threadIdx.x, a.H, SWEEP_NT, [&](int c) {
            const float d = widen<DT>(x[c]) - mean;
            return Two{d * d, 0.f};
        });
        const float rstd = 1.0f / sqrtf(block_sum(var.a, s) / a.H + a.eps);
        for (int c = threadIdx.x; c < a.H; c += SWEEP_NT) {
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
}

// dx of one row per workgroup.
template <int DT>
__global__ __launch_bounds__(SWEEP_NT) void norm_dx_sweep_kernel(NormArgs a) {
    __shared__ float s[SWEEP_NT / 64];
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const uint16_t* x = a.x + r * a.ldx;
        const uint16_t* dy = a.dy + r * a.lddy;
        const float mean = a.mean[r], rstd = a.rstd[r];
        const Two sum = chained_sum((int)threadIdx.x, a.H, SWEEP_NT, [&](int c) {
            const float g = widen<DT>(dy[c]) * (a.weight ? widen<DT>(a.weight[c]) : 1.f);
            return Two{g, g * ((widen<DT>(x[c]) - mean) * rstd)};
        });
        const float m0 = block_sum(sum.a, s) / a.H, m1 = block_sum(sum.b, s) / a.H;
        for (int c = threadIdx.x; c < a.H; c += SWEEP_NT) {
            const float g = widen<DT>(dy[c]) * (a.weight ? widen<DT>(a.weight[c]) : 1.f);
            float v = rstd * (g - m0 - (widen<DT>(x[c]) - mean) * rstd * m1);
            if (a.dres) v += widen<DT>(a.dres[r * a.lddres + c]);
            a.dx[r * a.lddx + c] = to_storage<DT>(v);
        }
    }
}

// Column sums of dy xhat and dy over row group blockIdx.y, one column per
// thread.
template <int DT>
__global__ __launch_bounds__(SWEEP_NT) void norm_cols_sweep_kernel(NormArgs a) {
    const int c = blockIdx.x * SWEEP_NT + threadIdx.x;
    if (c >= a.H) return;
    const int64_t r0 = a.rows * blockIdx.y / a.parts, r1 = a.rows * (blockIdx.y + 1) / a.parts;
    const Two sum = chained_sum(r0, r1, 1, [&](int64_t r) {
        const float dy = widen<DT>(a.dy[r * a.lddy + c]);
        return Two{dy * ((widen<DT>(a.x[r * a.ldx + c]) - a.mean[r]) * a.rstd[r]), dy};
    });
    float* p = a.part + (size_t)blockIdx.y * 2 * a.H + c;
    p[0] = sum.a;
    p[a.H] = sum.b;
}

// ---------------------------------------------------------------------- host

template <int DT, int TR, int V>
static hipError_t forward_v(const NormArgs& a, int cus, hipStream_t s) {
    // up to eight workgroups per CU, so that long batches reuse their weights
    const int64_t groups = (a.rows + FWD_NT / TR - 1) / (FWD_NT / TR), most = (int64_t)cus * 8;
    const dim3 grid((unsigned)(groups < most ? groups : most));
    if (a.H % 8) return launch(norm_forward_kernel<DT, TR, V, true>, grid, FWD_NT, s, a);
    return launch(norm_forward_kernel<DT, TR, V, false>, grid, FWD_NT, s, a);
}

template <int DT>
static hipError_t forward_sweep(const NormArgs& a, hipStream_t s) {
    return launch(norm_forward_sweep_kernel<DT>, sweep_grid(a.rows), SWEEP_NT, s, a);
}

template <int DT>
static hipError_t forward_t(const NormArgs& a, int cus, hipStream_t s) {
    // a wave per row while four chunks per lane hold it, then a workgroup
    if (a.H < 8) return forward_sweep<DT>(a, s);
    if (a.H <= 512) return forward_v<DT, 64, 1>(a, cus, s);
    if (a.H <= 1024) return forward_v<DT, 64, 2>(a, cus, s);
    if (a.H <= 2048) return forward_v<DT, 64, 4>(a, cus, s);
    if (a.H <= 4096) return forward_v<DT, 256, 2>(a, cus, s);
    if (a.H <= 8192) return forward_v<DT, 256, 4>(a, cus, s);
    if (a.H <= 12288) return forward_v<DT, 256, 6>(a, cus, s);
    if (a.H <= LONG_ROW) return forward_v<DT, 256, 8>(a, cus, s);
    return forward_sweep<DT>(a, s);
}

// The register-held backward's workgroup, threads per row and chunks per
// thread: one chunk each from a wave per row up to 1024 threads, then two; 768
// threads while they hold the row, whose larger register budget keeps every
// fp32 value of a row (whole calls with dres: 2048 x 12288 50.4 us, with 1024
// threads 72; 2048 x 9216 40.1 and 59.9).  Two chunks in 1024 threads spill up
// to 12 registers (2048 x 16384 90 us).
struct BackwardShape {
    int nt, tr, v;
};

static BackwardShape backward_shape(int H) {
    if (H > 12288) return {1024, 1024, 2};
    if (H > 8192) return {768, 768, 2};
    int tr = 64;
    while (tr * 8 < H) tr *= 2;
    return {1024, tr, 1};
}

template <int DT, int NT, int V, bool ALONE>
static hipError_t backward_v(const NormArgs& a, int tr, hipStream_t s) {
    if (a.H % 8) return launch(norm_backward_kernel<DT, NT, V, true, ALONE>, dim3(a.parts), NT, s, a, tr);
    return launch(norm_backward_kernel<DT, NT, V, false, ALONE>, dim3(a.parts), NT, s, a, tr);
}

template <int DT, bool ALONE>
static hipError_t backward_held(const NormArgs& a, hipStream_t s) {
    const BackwardShape b = backward_shape(a.H);
    if (b.v == 1) return backward_v<DT, 1024, 1, ALONE>(a, b.tr, s);
    if (b.nt == 768) return backward_v<DT, 768, 2, ALONE>(a, b.tr, s);
    return backward_v<DT, 1024, 2, ALONE>(a, b.tr, s);
}

template <int DT>
static hipError_t backward_t(const NormArgs& a, hipStream_t s) {
    const bool sums = a.dweight || a.dbias;
    hipError_t e = hipSuccess;
    if (held(a.H)) {
        if (a.parts == 1) return backward_held<DT, true>(a, s);
        if (a.parts > 1) e = backward_held<DT, false>(a, s);
    } else if (a.parts > 0) {
        if (sums) e = launch(norm_cols_sweep_kernel<DT>, dim3((a.H + SWEEP_NT - 1) / SWEEP_NT, a.parts), SWEEP_NT, s, a);
        if (e == hipSuccess) e = launch(norm_dx_sweep_kernel<DT>, sweep_grid(a.rows), SWEEP_NT, s, a);
    }
    if (e == hipSuccess && sums) e = launch(norm_cols_sum_kernel<DT>, dim3((2 * a.H + 31) / 32), 1024, s, a);
    return e;
}

}  // namespace mlpc

using namespace mlpc;

// Partial rows of column sums: the workgroups of the register-held kernel, or
// the row groups of the sweeping column kernel.  A single workgroup, which
// needs no second kernel, takes up to three steps where a thread holds one
// chunk (whole calls, 3 steps, then 5: 512 columns 8.1 and 10.1 us, 8192
// columns 10.2 and 13.5; with a workgroup per step and the second kernel 10.7).
constexpr int ALONE_STEPS = 3;

int mlpc_norm_parts(int64_t rows, int H, int cus) {
    const int64_t per = held(H) ? backward_shape(H).nt / backward_shape(H).tr : 1;
    const int64_t groups = (rows + per - 1) / per;
    if (held(H) && groups > 0 && groups <= (backward_shape(H).v == 1 ? ALONE_STEPS : 1)) return 1;
    const int64_t most = held(H) ? (cus < MAX_PARTS ? cus : MAX_PARTS) : 64;
    return (int)(groups < most ? groups : most);
}

int mlpc_norm_max_parts(int H, int cus) { return mlpc_norm_parts((int64_t)1 << 32, H, cus); }

hipError_t mlpc_norm_forward(const NormArgs& a, int dtype, int cus, hipStream_t s) {
    return dtype == DT_F16 ? forward_t<DT_F16>(a, cus, s) : forward_t<DT_BF16>(a, cus, s);
}

hipError_t mlpc_norm_backward(const NormArgs& a, int dtype, hipStream_t s) {
    return dtype == DT_F16 ? backward_t<DT_F16>(a, s) : backward_t<DT_BF16>(a, s);
}

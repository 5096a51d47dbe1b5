// loss_device.hpp -- the products of a vocabulary head's cross entropy on
// gfx950, on the linear layer's tiles (linear_device.hpp): z = x W^T with a
// softmax's maximum and sum, or its gradient dz, in the epilogue, and the
// products dz W and dz^T x of a piece of dz.
//
//   z     x [n, H] and W [V, H] both have the reduction contiguous
//   dx    dz [n, vn] contiguous, W [vn, H] across rows; fp32 sums over the
//         pieces of the vocabulary (and parts of a piece) stay in the workspace
//   dW    dz and x both across rows (the n packed rows); one output of V rows
//
// The number n of rows that count is known on the device alone: the grid is
// for every row, and tiles past n end at once.  Rows are packed by kernels of
// their own (loss_rows.hip) before the products, but where all rows fit one
// tile each workgroup finds out about them by itself.
#pragma once

#include "linear_device.hpp"
#include "train_launch.h"

namespace mlpc {

constexpr float LOG2E = 1.4426950408889634f;

// Rows to reduce or multiply, as a scalar.
__device__ __forceinline__ int packed_rows(const LossArgs& p) {
    return p.packing ? __builtin_amdgcn_readfirstlane(p.info->n) : (int)p.rows;
}

__device__ __forceinline__ const uint16_t* packed_x(const LossArgs& p, bool copied, int64_t& ld) {
    ld = copied ? p.H : p.ldx;
    return copied ? p.packed : p.x;
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) v = fmaxf(v, __shfl_xor(v, d));
    return v;
}

// The largest coefficient in a row of dz, for its unit; 0 if it is not finite
// (whatever the unit, that row's gradients are not, and the other rows' are not
// to suffer).
__device__ __forceinline__ float largest_coefficient(float dloss, float dlse) {
    const float top = fmaxf(fabsf(dloss), fabsf(dloss + dlse));
    return top < INFINITY ? top : 0.f;
}

// dz's unit from the call's largest coefficient.  The matrix cores take dz in
// 16 bits.  Where all rows have the same dloss (a mean), a target of probability
// p has dz = p - 1 units: exact to within p / 2, so dx of a wide vocabulary is as
// good as from an unrounded dz.  With few rows and a narrow one that rounding
// shows beside the outputs' own (one row, 711 words, bf16: relative error 3.0e-3,
// 1.7e-3 from an unrounded dz).  A second 16-bit term would cure that at twice
// the products' work.  (fp16 has few small numbers: 2^14 makes room below)
template <int DT>
__device__ __forceinline__ float dz_unit(float top) {
    return top > 0.f ? fmaxf(DT == DT_F16 ? top * 0x1p-14f : top, 0x1p-126f) : 1.f;
}

// A configuration whose waves multiply F fragments of 16 rows: tiles of 32 F
// rows.  Each wave requests as many rows as the others, so the DMA brings 192
// rows for 5 and 6 fragments and 256 for 7 (8192 -> 32000 bf16 on 160- and
// 192-row tiles, with 256 rows for all of them against this: 320 rows z 223 ->
// 214 us, gradient 715 -> 692; 384 rows 234 -> 225, 735 -> 713; 1100 rows 584 ->
// 559, 1627 -> 1602.  With one line requested for all of the last 32 rows of 7
// fragments: no difference).
template <class C, int F>
struct Shorter : C {
    static constexpr int FM = F, NF = F * C::FN, WTM = 16 * F;
    static constexpr int A_PER_WAVE = (32 * F * C::KS / 512 + C::NW - 1) / C::NW, LPS = A_PER_WAVE + C::B_PER_WAVE;
};

// Rows of a tile.
template <class C>
constexpr int tile_rows = C::WM * C::WTM;

// Rows of tiles of n rows.
template <class C>
struct RowTiles {
    static constexpr bool TALL = C::FM == 8;
    Fragments fragments;
    uint32_t Mt;

    __device__ __forceinline__ RowTiles(int n, uint32_t columns, uint32_t cus) {
        if constexpr (TALL) fragments = fragments_for(n, columns, cus);
        Mt = TALL ? fragments.tiles : (n + C::BM - 1) / C::BM;
    }

    // f(C with the fragments of row mb, its first row).
    template <class F>
    __device__ __forceinline__ void take(uint32_t mb, F&& f) const {
        if constexpr (TALL) {
            const int extra = min((int)mb, fragments.extra), k = fragments.base + ((int)mb < fragments.extra ? 1 : 0);
            const int m0 = 32 * ((int)mb * fragments.base + extra);
            if (k == 7) return f(Shorter<C, 7>{}, m0);
            if (k == 6) return f(Shorter<C, 6>{}, m0);
            if (k == 5) return f(Shorter<C, 5>{}, m0);
            f(C{}, m0);
        } else {
            f(C{}, (int)mb * C::BM);
        }
    }
};

// The reduction of a tile: stages k0 .. k1 of `slabs` whole slabs and the one
// that ends past K, for the last part.
template <class C, int DT, int PASS>
__device__ __forceinline__ void loss_reduce(f32x4 (&acc)[C::FM][C::FN], const LinTile<C, PASS>& t, const GemmArgs& g, int k0,
                                            int k1, bool last) {
    const int slabs = g.K / BK;
    const bool tail = last && g.K % BK;
    if (k1 > k0) t.template kloop<DT>(acc, k0 * C::SPS, k1 * C::SPS, tail ? slabs : -1, g);
    else if (tail) t.template only_tail<DT>(acc, slabs, g);
    ring_barrier<0>();          // no DMA in flight, and the ring is free
}

// Maximum and sum of exp(z - maximum), joined.
__device__ __forceinline__ void softmax_join(float& m, float& s, float m2, float s2) {
    const float top = fmaxf(m, m2);
    // (of nothing but -inf: no exponential of inf - inf)
    const float at = top == -INFINITY ? 0.f : top;
    s = s * __builtin_amdgcn_exp2f((m - at) * LOG2E) + s2 * __builtin_amdgcn_exp2f((m2 - at) * LOG2E);
    m = top;
}

// The tile's rows: maximum and sum of exp over its columns, and z at the
// target.  A lane holds 4 FN columns of FM rows; lanes 16 apart share a row,
// and so do the WN waves of a row of waves, which join through LDS.
template <class C>
__device__ __forceinline__ void softmax_epilogue(const f32x4 (&acc)[C::FM][C::FN], const LossArgs& p, int n, uint32_t nb, int m0,
                                                 int n0) {
    const int lane = threadIdx.x & 63, wave = uniform_wave(), g = lane >> 4;
    const int row = wave / C::WN * C::WTM + (lane & 15), col = n0 + wave % C::WN * C::WTN + g * 4;
    float2* s = reinterpret_cast<float2*>(linear_ring<C>());      // [BM][WN]
#pragma unroll
    for (int f = 0; f < C::FM; ++f) {
        const int r = m0 + row + f * 16;
        int target = -1;
        if (r < n) {
            if (p.packing) target = p.row[r].target;
            else {
                const int64_t t = p.target[r];
                target = t >= 0 && t < p.V ? (int)t : -1;
            }
        }
        float top = -INFINITY;
#pragma unroll
        for (int c = 0; c < C::FN; ++c)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (col + c * 16 + k < p.vn) {
                    top = fmaxf(top, acc[f][c][k]);
                    if (col + c * 16 + k == target) p.picked[r] = acc[f][c][k];
                }
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const float at = top == -INFINITY ? 0.f : top;
        float sum = 0.f;
#pragma unroll
        for (int c = 0; c < C::FN; ++c)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (col + c * 16 + k < p.vn) sum += __builtin_amdgcn_exp2f((acc[f][c][k] - at) * LOG2E);
        sum += __shfl_xor(sum, 16);
        sum += __shfl_xor(sum, 32);
        if (g == 0) s[(row + f * 16) * C::WN + wave % C::WN] = make_float2(top, sum);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < tile_rows<C>; i += C::NT) {
        if (m0 + i >= n) break;
        float2 t = s[i * C::WN];
#pragma unroll
        for (int w = 1; w < C::WN; ++w) softmax_join(t.x, t.y, s[i * C::WN + w].x, s[i * C::WN + w].y);
        p.part[(size_t)(m0 + i) * p.tiles + nb] = t;
    }
}

// What dz needs of the rows, where they fit one tile: a row per thread, loaded
// before the reduction and brought to LDS after it.
template <class C, int DT>
struct RowsOfTile {
    int64_t target;
    float d, l, lse;

    __device__ __forceinline__ void load(const LossArgs& p) {
        const int r = threadIdx.x;
        const bool in = r < (int)p.rows;
        target = in ? p.target[r] : -1;
        d = in && p.dloss ? p.dloss[r] : 1.f;
        l = in && p.dlse ? p.dlse[r] : 0.f;
        lse = in ? p.lse_in[r] : 0.f;
    }

    // Returns whether a row is left out.
    __device__ __forceinline__ bool store(const LossArgs& p) {
        static_assert(C::NT >= C::BM, "a row per thread");
        LossRow* row = reinterpret_cast<LossRow*>(linear_ring<C>());            // [BM]
        float* largest = reinterpret_cast<float*>(row + C::BM);                 // [NW]
        const int r = threadIdx.x, lane = r & 63;
        const bool counts = target >= 0 && target < p.V;
        const float top = wave_max(counts ? largest_coefficient(d, l) : 0.f);
        if (lane == 0) largest[r >> 6] = top;
        const bool out = __syncthreads_or(r < (int)p.rows && !counts);
        float all = largest[0];
#pragma unroll
        for (int w = 1; w < C::NW; ++w) all = fmaxf(all, largest[w]);
        const float unit = dz_unit<DT>(all);
        if (r < C::BM) row[r] = counts ? LossRow{lse, (d + l) / unit, d / unit, (int)target} : LossRow{0.f, 0.f, 0.f, -1};
        if (blockIdx.x == 0 && p.first) {
            if (r < (int)p.rows) p.place[r] = counts ? r : -1;
            if (r == 0) *p.info = LossInfo{(int)p.rows, unit, out};
        }
        __syncthreads();
        return out;
    }
};

// dW's x where a row is left out (its x may hold anything): the workgroups
// share the copy.
__device__ __forceinline__ void copy_rows(const LossArgs& p, int threads) {
    const int per_row = p.H / 8, chunks = (int)p.rows * per_row;
    for (int i = blockIdx.x * threads + threadIdx.x; i < chunks; i += gridDim.x * threads) {
        const int r = i / per_row, c = i % per_row * 8;
        const int64_t t = p.target[r];
        st16(p.packed + (size_t)r * p.H + c, t >= 0 && t < p.V ? ld16(p.x + r * p.ldx + c) : u32x4{});
    }
}

// dz of the tile, rounded to the storage type; columns between V and the next
// multiple of 8 are zeros, which the products read.
template <class C, int DT>
__device__ __forceinline__ void dz_epilogue(const f32x4 (&acc)[C::FM][C::FN], const LossArgs& p, int n, int m0, int n0) {
    const int lane = threadIdx.x & 63, wave = uniform_wave(), g = lane >> 4;
    const int row = wave / C::WN * C::WTM + (lane & 15);
    const int col = n0 + wave % C::WN * C::WTN + (g & 1) * 16 + (g >> 1) * 8;
#pragma unroll
    for (int f = 0; f < C::FM; ++f) {
        const int r = m0 + row + f * 16;
        LossRow q = {};
        if (!p.packing) q = reinterpret_cast<const LossRow*>(linear_ring<C>())[row + f * 16];
        else if (r < n) q = p.row[r];
        const int target = q.target - p.v0;
        static_for<0, C::FN / 2>([&](auto i) {
            constexpr int I = decltype(i)::value;
            float v[8];
            pair8(acc[f][2 * I], acc[f][2 * I + 1], v);
            const int c = col + I * 32;
            if (r >= n || c >= p.vn) return;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                v[k] = q.a * __builtin_amdgcn_exp2f((v[k] - q.lse) * LOG2E);
                if (c + k == target) v[k] -= q.b;
                if (c + k >= p.vn || q.target < 0) v[k] = 0.f;
            }
            st16(p.dz + (size_t)r * p.lddz + c, narrow8<DT>(v));
        });
    }
}

// A tile of z = x W^T.  With one or two rows of tiles, reading W bounds it, and
// tiles of different words then begin at different places of a long reduction:
// rows of W whose length is a power of two would otherwise have all workgroups
// read the same few memory channels at a time (48 x 8192 x 32000 121 -> 95 us,
// 4.3 -> 5.5 TB/s of W).
template <class C, int DT, bool GRAD>
__device__ __forceinline__ void loss_logits_tile(const LossArgs& p, const GemmArgs& g, int n, int m0, uint32_t nb,
                                                 RowsOfTile<C, DT>& rows) {
    const int n0 = nb * C::BN;
    f32x4 acc[C::FM][C::FN] = {};
    LinTile<C, PASS_DX> t;
    t.a.init(g.a, g.lda, m0, n, 0);
    t.b.init(g.b, g.ldb, n0, p.vn, 0);
    const int slabs = p.H / BK, turn = g.Mt <= 2 && slabs >= 32 ? (int)((uint64_t)nb * slabs / g.Nt) : 0;
    loss_reduce<C, DT>(acc, t, g, turn, slabs, true);
    if (turn > 0) loss_reduce<C, DT>(acc, t, g, 0, turn, false);
    if constexpr (GRAD) {
        const bool out = !p.packing && rows.store(p);
        dz_epilogue<C, DT>(acc, p, n, m0, n0);
        if (out && p.first && p.dw) copy_rows(p, C::NT);
    } else {
        softmax_epilogue<C>(acc, p, n, nb, m0, n0);
    }
}

// z = x W^T, and from the accumulators either a maximum and a sum per row and tile
// (softmax_epilogue; 8 bytes for BN logits) or dz in 16 bits (dz_epilogue): the
// logits themselves never leave the registers.  48 x 8192 x 32000 takes 89 us, 6.0
// TB/s of W.  3700 x 8192 x 128000 takes 6.14 ms (1.26 PFLOP/s, matrix cores
// 67% busy at 1.77 GHz), most of it the tiles' way from L2 to LDS: 64 KB per
// stage take 0.84 us where 112 CUs ask for them, 1.29 for 224, 1.56 for 256 (11
// TB/s over all), and 1.42 with an x and a W of zeros, whose products cost no power.
// Rows further apart, requests spread over both halves of a stage and lines brought
// to L2 ahead of them changed nothing.
template <class C, int DT, bool GRAD>
__global__ __launch_bounds__(C::NT, C::OCC) void loss_logits_kernel(LossArgs p) {
    const int n = packed_rows(p);
    GemmArgs g{};
    g.a = packed_x(p, p.packing && n < (int)p.rows, g.lda);
    g.b = p.w + (size_t)p.v0 * p.ldw;
    g.ldb = p.ldw;
    g.K = p.H;
    g.zero = p.zero;
    g.Nt = p.Nt;
    if (p.packing) {
        const RowTiles<C> rows(n, p.Nt, p.cus);
        g.Mt = rows.Mt;
        if (blockIdx.x >= g.Mt * g.Nt) return;
        uint32_t mb, nb;
        tile_at(g, xcd_chunked(blockIdx.x, g.Mt * g.Nt), mb, nb);
        rows.take(mb, [&](auto c, int m0) {
            RowsOfTile<decltype(c), DT> none;
            loss_logits_tile<decltype(c), DT, GRAD>(p, g, n, m0, nb, none);
        });
        return;
    }
    g.Mt = 1;
    RowsOfTile<C, DT> rows;
    if (GRAD) rows.load(p);
    loss_logits_tile<C, DT, GRAD>(p, g, n, 0, xcd_chunked(blockIdx.x, g.Nt), rows);
}

// The tile's rows below `rows` and columns below `cols`, times `unit`, rounded;
// rows whose place (unless nullptr) is -1 are zeros.
template <class C, int DT>
__device__ __forceinline__ void store_scaled(const f32x4 (&acc)[C::FM][C::FN], uint16_t* d, int64_t ld, int m0, int rows, int n0,
                                             int cols, float unit, const int* place) {
    const int lane = threadIdx.x & 63, wave = uniform_wave(), g = lane >> 4;
    const int row = m0 + wave / C::WN * C::WTM + (lane & 15);
    const int col = n0 + wave % C::WN * C::WTN + (g & 1) * 16 + (g >> 1) * 8;
    static_for<0, C::FN / 2>([&](auto i) {
        constexpr int I = decltype(i)::value;
#pragma unroll
        for (int f = 0; f < C::FM; ++f) {
            float v[8];
            pair8(acc[f][2 * I], acc[f][2 * I + 1], v);
            const int r = row + f * 16, c = col + I * 32;
            if (r >= rows || c >= cols) continue;
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] *= unit;
            st16(d + (size_t)r * ld + c, place && place[r] < 0 ? u32x4{} : narrow8<DT>(v));
        }
    });
}

// A part of a tile of dz W: added to the sums of the pieces before.
template <class C, int DT>
__device__ __forceinline__ void loss_dx_tile(const LossArgs& p, const LossInfo& info, const GemmArgs& g, int n, int m0, uint32_t nb,
                                             uint32_t part) {
    const int n0 = nb * C::BN, slabs = p.vn / BK;
    f32x4 acc[C::FM][C::FN] = {};
    {
        LinTile<C, PASS_FWD> t;
        t.a.init(g.a, g.lda, m0, n, 0);
        t.b.init(g.b, g.ldb, n0, p.H, 0);
        const int k0 = min((int)(part * p.ksp), slabs), k1 = min(k0 + (int)p.ksp, slabs);
        loss_reduce<C, DT>(acc, t, g, k0, k1, part + 1 == p.S);
    }
    const int lane = threadIdx.x & 63, wave = uniform_wave();
    if (p.direct) {
        store_scaled<C, DT>(acc, p.dx, p.lddx, m0, n, n0, p.H, info.unit, p.place);
        return;
    }
    const int row = m0 + wave / C::WN * C::WTM + (lane & 15), col = n0 + wave % C::WN * C::WTN + (lane >> 4) * 4;
    float* sums = p.sums + (size_t)part * p.rows * p.H;
#pragma unroll
    for (int f = 0; f < C::FM; ++f) {
        const int r = row + f * 16;
        if (r >= n) continue;
#pragma unroll
        for (int c = 0; c < C::FN; ++c) {
            if (col + c * 16 >= p.H) continue;
            f32x4* at = reinterpret_cast<f32x4*>(sums + (size_t)r * p.H + col + c * 16);
            *at = p.first ? acc[f][c] : *at + acc[f][c];
        }
    }
}

// A tile of dz^T x.
template <class C, int DT>
__device__ __forceinline__ void loss_dw_tile(const LossArgs& p, const LossInfo& info, int n, uint32_t block) {
    GemmArgs g{};
    g.a = p.dz;
    g.lda = p.lddz;
    g.b = packed_x(p, info.copied, g.ldb);
    g.K = n;
    g.zero = p.zero;
    g.Mt = p.dwMt;
    g.Nt = p.dwNt;
    uint32_t mb, nb;
    tile_at(g, xcd_chunked(block, g.Mt * g.Nt), mb, nb);
    const int m0 = mb * C::BM, n0 = nb * C::BN;
    f32x4 acc[C::FM][C::FN] = {};
    {
        LinTile<C, PASS_DW> t;
        t.a.init(g.a, g.lda, m0, (p.vn + 7) & ~7, 0);
        t.b.init(g.b, g.ldb, n0, p.H, 0);
        loss_reduce<C, DT>(acc, t, g, 0, n / BK, true);
    }
    store_scaled<C, DT>(acc, p.dw + (size_t)p.v0 * p.lddw, p.lddw, m0, p.vn, n0, p.H, info.unit, nullptr);
}

// Both products of a piece: the first dx_blocks workgroups (a multiple of 8,
// the XCDs that the others are dealt to) dz W, the others dz^T x.  dx has few
// tiles with a long reduction, dW many with a short one, which fill the round
// that dx's leave open (667 x 12288 x 50001: one launch 1655 us, dx alone 1038, dW
// alone 925).  3700 x 8192 x 32000 takes 2.95 ms (1.31 PFLOP/s, matrix cores 68%
// busy at 1.84 GHz); 667 x 12288 x 50001 reaches 0.98 PFLOP/s: dW's tiles
// have ten slabs each between filling the ring and storing 128 KB.
// With a few rows W's second reading and dW's writing bound it (48 x 8192 x 32000:
// 262 us for 1.05 GB; a kernel of its own for dW of up to 128 rows, x in registers
// and dz turned around in LDS, took 251 us for a call without dx, which 128 x 128
// tiles reach as well (245 to 251), and 392 with it: dropped).
template <class C, int DT>
__global__ __launch_bounds__(C::NT, C::OCC) void loss_products_kernel(LossArgs p, uint32_t dx_blocks) {
    // Loaded once, ahead: a tile that asks for the unit before its stores waits for
    // it (48 x 8192 x 32000 389 -> 357 us, 1 row 367 -> 318, 667 x 12288 x 50001
    // 2647 -> 2602; dW alone of 48 x 8192 x 32000 324 -> 332, of other sizes 2 to 6%
    // less).
    const LossInfo info = {__builtin_amdgcn_readfirstlane(p.info->n),
                           __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, p.info->unit))),
                           __builtin_amdgcn_readfirstlane(p.info->copied)};
    const int n = p.packing ? info.n : (int)p.rows;
    if (blockIdx.x >= dx_blocks) return loss_dw_tile<C, DT>(p, info, n, blockIdx.x - dx_blocks);
    const RowTiles<C> rows(n, 1, 0);
    GemmArgs g{};
    g.a = p.dz;
    g.lda = p.lddz;
    g.b = p.w + (size_t)p.v0 * p.ldw;
    g.ldb = p.ldw;
    g.K = p.vn;
    g.zero = p.zero;
    g.Mt = rows.Mt;
    g.Nt = p.dxNt;
    const uint32_t blocks = g.Mt * g.Nt * p.S;
    if (blockIdx.x >= blocks) return;
    const uint32_t q = xcd_chunked(blockIdx.x, blocks), part = q % p.S;
    uint32_t mb, nb;
    tile_at(g, q / p.S, mb, nb);
    rows.take(mb, [&](auto c, int m0) { loss_dx_tile<decltype(c), DT>(p, info, g, n, m0, nb, part); });
}

}  // namespace mlpc

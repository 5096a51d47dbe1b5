// linear_device.hpp -- one tile of a product of the linear layer on gfx950:
// D(m, n) = sum_k A(m, k) B(k, n) with either operand stored with the
// reduction contiguous ("KC": rows of k) or with it across rows ("KR": a row
// per k).  Forward x W is KC x KR, dz W^T is KC x KC and x^T dz is KR x KR,
// so nothing is ever transposed in memory.
//
//   * Operands go from global memory into a ring of NS LDS stages of KS
//     reduction elements (global_load_lds_dwordx4), NS - 1 of them in flight
//     while one is multiplied; the DMA of a stage is spread over the MFMAs.
//   * A KC operand is read as MFMA fragments with ds_read_b128, a KR operand
//     with the transpose read ds_read_b64_tr_b16, both from XOR-swizzled
//     16-byte chunks; the next half step's fragments are read during this
//     one's MFMAs.
//   * The MFMAs take B as their first operand, so a lane's accumulators are
//     four neighbouring columns of one row, and one v_permlane16_swap per
//     register pair makes them eight: the epilogue adds the bias and the
//     residual and stores 16 bytes per lane without going through LDS.
//   * Rows and columns past the matrices are clamped to the last row or
//     8-column chunk (their results are not stored).  A slab that ends past K
//     (K % 64 != 0) takes its out-of-range chunks from a zero page.
//
// What bounds it: with 500 rows and more the chip's power (the matrix cores
// 50-60% busy at 1.8-2.1 GHz on random operands, no LDS bank conflict): a call
// of 2048 x 12288 x 6144 fp16 with the planned tiles took 272-290 us for x W,
// 265-285 for dz W^T and 270-277 for x^T dz on three cards (1.07-1.17 PFLOP/s),
// 8192 x 4096 x 4096 224-235 us (1.17-1.22).  Single tokens stream W at 5.4
// TB/s (1 x 12288 x 6144: 27.8 us in the kernel).  In between, rows padded to
// the tile, the partials of split tiles and the memory's latency under two or
// three stages in flight share the loss: 300 x 8192 x 5504 takes 45-48 us in
// the kernel for 27 GFLOP and 95 MB of operands.
#pragma once

#include "block_launch.h"
#include "chain_device.hpp"

namespace mlpc {

template <int BM_, int BN_, int WM_, int WN_, int NS_, int KS_, int OCC_, int EARLY_ = 0>
struct LinCfg {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NS = NS_, KS = KS_, OCC = OCC_;
    static constexpr int NW = WM * WN, NT = 64 * NW;
    static constexpr int WTM = BM / WM, WTN = BN / WN;
    static constexpr int FM = WTM / 16, FN = WTN / 16, NF = FM * FN;
    static constexpr int EARLY = EARLY_;                    // rows of A fragments with registers of their own for the next ones
    static constexpr int HP = KS / 32;                      // 32-deep half steps per stage
    static constexpr int SPS = BK / KS;                     // stages per slab
    static constexpr int A_BYTES = BM * KS * 2, STAGE = A_BYTES + BN * KS * 2, RING = NS * STAGE;
    static constexpr int A_PER_WAVE = BM * KS / 512 / NW, B_PER_WAVE = BN * KS / 512 / NW;
    static constexpr int LPS = A_PER_WAVE + B_PER_WAVE;     // DMA instructions per wave per stage
    static_assert(KS == 32 || KS == 64, "stages of half a slab or a slab");
    static_assert(A_PER_WAVE * NW * 512 == BM * KS && B_PER_WAVE * NW * 512 == BN * KS, "DMA split across waves");
    static_assert(FN % 4 == 0, "16-byte epilogue chunks, gate / up pairs");
    static_assert(LPS * (NS - 1) <= 63, "vmcnt range");
};

template <int BYTES>
__device__ __forceinline__ char* ring_bytes() {
    __shared__ __attribute__((aligned(1024))) char buf[BYTES];
    return buf;
}

// (one for all configurations of its size that a kernel takes)
template <class C>
__device__ __forceinline__ char* linear_ring() {
    return ring_bytes<C::RING>();
}

// How a pass stores its operands.
template <int PASS> struct Layout { static constexpr bool a_kr = PASS == PASS_DW, b_kr = PASS != PASS_DX; };

// Physical chunk of logical chunk c in k row `k` of a KR stage of CPR chunks
// per row.  A transpose read covers, per 32 lanes, 8 k rows and two chunks of
// each; the XOR gives those rows 8 distinct chunk pairs.
template <int CPR>
__device__ __forceinline__ int kr_chunk(int k, int c) {
    return c ^ ((2 * ((k & 3) | (((k >> 3) & 1) << 2))) & (CPR - 1));
}

// Physical chunk of logical chunk c in row r of a KC stage.  32-deep rows have
// four chunks, so rows r, r + 4, r + 8, r + 12 share banks: the XOR gives them
// 0, 2, 3, 1, which keeps them apart whether they are read at one chunk or, as
// the 16 lanes that ds_read_b128 serves together take them, two of them at a
// chunk and the other two at its neighbour.  With the chain's a_chunk32, which
// gives those rows 0, 1, 2, 3, conflicts take 0.17 (x W) and 0.26 (dz W^T) of
// the busy cycles on 256 x 256 tiles, with these none; the times, which power
// bounds, are the same (2048 x 12288 x 6144: x W 280 us, dz W^T 316 either way).
template <int KS>
__device__ __forceinline__ int kc_chunk(int r, int c) {
    if constexpr (KS == 64) return a_chunk(r, c);
    else return c ^ (((r >> 3) & 1) | ((((r >> 2) ^ (r >> 3)) & 1) << 1));
}

// One operand of a tile: `lim` rows (KC) or columns (KR) from `r0` on.
template <class C, bool IS_A, bool KR>
struct Operand {
    static constexpr int EXT = IS_A ? C::BM : C::BN;        // tile extent across the reduction
    static constexpr int PER_WAVE = IS_A ? C::A_PER_WAVE : C::B_PER_WAVE;
    static constexpr int CPR = KR ? EXT / 8 : C::KS / 8;    // 16-byte chunks per LDS row
    static constexpr int FRAGS = IS_A ? C::FM : C::FN;
    static constexpr int READS = KR ? 2 : 1;                // LDS reads per fragment
    static constexpr int NBASE = KR ? FRAGS : C::HP;        // per-lane fragment addresses

    const char* base;       // first element of the tile's rows / columns at k = 0 (wave-uniform)
    size_t step;            // bytes from a stage to the next
    uint32_t off[PER_WAVE]; // each DMA chunk's offset from the stage's base
    uint32_t frag[NBASE];   // LDS addresses of the first fragments in stage 0

    // Global column (KR) of tile column chunk c: for swiglu's B, 16-column
    // fragments alternate gate and up (`up` columns apart).
    static __device__ __forceinline__ int column(int r0, int lim, int up, int c) {
        if (!IS_A && up) return min(r0 + (c >> 2) * 16 + (c & 1) * 8, lim - 8) + ((c >> 1) & 1) * up;
        return min(r0 + c * 8, lim - 8);
    }

    __device__ __forceinline__ void init(const uint16_t* p, int64_t ld, int r0, int lim, int up) {
        const int lane = threadIdx.x & 63, wave = uniform_wave();
        if constexpr (KR) {
            base = reinterpret_cast<const char*>(p);
            step = (size_t)ld * (C::KS * 2);
        } else {
            base = reinterpret_cast<const char*>(p + (size_t)r0 * ld);
            step = C::KS * 2;
        }
#pragma unroll
        for (int q = 0; q < PER_WAVE; ++q) {
            const int L = (wave * PER_WAVE + q) * 64 + lane, r = L / CPR, c = L % CPR;
            if constexpr (KR)
                off[q] = ((uint32_t)r * (uint32_t)ld + (uint32_t)column(r0, lim, up, kr_chunk<CPR>(r, c))) * 2u;
            else
                off[q] = (uint32_t)(min(r0 + r, lim - 1) - r0) * (uint32_t)ld * 2u + (uint32_t)kc_chunk<C::KS>(r, c) * 16u;
        }
        const uint32_t ring = lds_addr(linear_ring<C>()) + (IS_A ? 0 : C::A_BYTES);
        const int w = IS_A ? wave / C::WN * C::WTM : wave % C::WN * C::WTN;
        const int g = lane >> 4, jj = lane & 15;
        if constexpr (KR) {
            // lane (g, jj): k row 8g + jj / 4 (+4: the upper rows), columns 4 (jj % 4) .. +3 of the fragment
            const int k = g * 8 + (jj >> 2);
#pragma unroll
            for (int f = 0; f < FRAGS; ++f) {
                const int col = w + f * 16 + (jj & 3) * 4;
                frag[f] = ring + (k * CPR + kr_chunk<CPR>(k, col >> 3)) * 16 + (col & 7) * 2;
            }
        } else {
#pragma unroll
            for (int h = 0; h < C::HP; ++h)
                frag[h] = ring + ((w + jj) * CPR + kc_chunk<C::KS>(w + jj, h * 4 + g)) * 16;
        }
    }

    static __device__ __forceinline__ char* dst(int stage, int q) {
        return linear_ring<C>() + stage * C::STAGE + (IS_A ? 0 : C::A_BYTES) + (uniform_wave() * PER_WAVE + q) * 1024;
    }

    // DMA instruction q of reduction stage h into ring stage `stage`.
    __device__ __forceinline__ void issue(int h, int stage, int q) const {
        dma16(base + (size_t)h * step + fresh(off[q]), dst(stage, q));
    }

    // The same for a stage that ends past K: chunks out of range come from the zero page.
    __device__ __forceinline__ void issue_tail(int h, int stage, int q, int64_t ld, int K, const void* zero) const {
        const int L = (uniform_wave() * PER_WAVE + q) * 64 + (threadIdx.x & 63), r = L / CPR, c = L % CPR;
        const int k = h * C::KS + (KR ? r : kc_chunk<C::KS>(r, c) * 8);
        const char* src = base + (size_t)h * step + off[q];
        dma16(k < K ? src : static_cast<const char*>(zero), dst(stage, q));
    }

    // LDS read R (fragment R / READS) of half step H of the stage at offset `so`.
    template <int H, int R>
    __device__ __forceinline__ void read(uint32_t so, u32x4 (&f)[FRAGS]) const {
        constexpr int F = R / READS;
        if constexpr (KR) {
            const u32x2 v = ds_read_tr16_b64<(H * 32 + 4 * (R % 2)) * CPR * 16>(frag[F] + so);
            f[F][2 * (R % 2)] = v[0];
            f[F][2 * (R % 2) + 1] = v[1];
        } else {
            f[F] = ds_read_b128<F * 16 * CPR * 16>(frag[H] + so);
        }
    }
};

template <class C>
struct LinFrags {
    u32x4 a[C::FM], b[C::FN];
    __device__ __forceinline__ void ready() {
        lgkm_wait<0>();
#pragma unroll
        for (int i = 0; i < C::FM; ++i) pin(a[i]);
#pragma unroll
        for (int i = 0; i < C::FN; ++i) pin(b[i]);
    }
};

// A tile's operands and its reduction.  The next half step's LDS reads go among
// this one's MFMAs (row-major over the fragments): an A fragment's reads after
// the last MFMA of its row, when its registers are free, and one B read after
// each other MFMA; B reads left over follow the block.  The last rows' reads
// would then have no MFMAs left to wait behind: those of the last EARLY rows go
// among an earlier row's, into registers of their own.
template <class C, int PASS>
struct LinTile {
    using A = Operand<C, true, Layout<PASS>::a_kr>;
    using B = Operand<C, false, Layout<PASS>::b_kr>;
    A a;
    B b;

    template <int H>
    __device__ __forceinline__ void read_all(uint32_t so, LinFrags<C>& f) const {
        static_for<0, C::FM * A::READS>([&](auto r) { a.template read<H, decltype(r)::value>(so, f.a); });
        static_for<0, C::FN * B::READS>([&](auto r) { b.template read<H, decltype(r)::value>(so, f.b); });
    }

    // The reads of A fragment M.
    template <int H, int M>
    __device__ __forceinline__ void read_a(uint32_t so, LinFrags<C>& f) const {
        static_for<0, A::READS>([&](auto r) { a.template read<H, M * A::READS + decltype(r)::value>(so, f.a); });
    }

    // DMA instruction Q of LPS of a stage, B's first.
    template <int Q>
    __device__ __forceinline__ void issue(int h, int stage) const {
        if constexpr (Q < C::B_PER_WAVE) b.issue(h, stage, Q);
        else a.issue(h, stage, Q - C::B_PER_WAVE);
    }

    // The MFMAs of `cur`, with the reads of half step H at `so` into `nxt`
    // and, if DMA, the requests of reduction stage `h` into ring stage
    // `stage` among them.
    template <int DT, int H, bool DMA>
    __device__ __forceinline__ void multiply(f32x4 (&acc)[C::FM][C::FN], const LinFrags<C>& cur, uint32_t so,
                                             LinFrags<C>& nxt, int h, int stage) const {
        constexpr int GAP = C::NF / C::LPS >= 2 ? 2 : 1;
        constexpr int SLOTS = C::NF - C::FM, NB = C::FN * B::READS, LATE = C::FM - C::EARLY;
        static_assert(C::EARLY < C::FN && (C::EARLY == 0 || LATE >= 2), "slots of one row");
        static_for<0, C::NF>([&](auto i) {
            constexpr int I = decltype(i)::value, M = I / C::FN, N = I % C::FN;
            acc[M][N] = mfma16x16x32<DT>(cur.b[N], cur.a[M], acc[M][N]);
            if constexpr (N == C::FN - 1) {
                if constexpr (M < LATE) read_a<H, M>(so, nxt);
            } else {
                constexpr int R = I - M;      // B slots before this one
                if constexpr (R < NB) b.template read<H, R>(so, nxt.b);
                if constexpr (M == LATE - 2 && N < C::EARLY) read_a<H, LATE + N>(so, nxt);
            }
            if constexpr (DMA && I % GAP == 0 && I / GAP < C::LPS) issue<I / GAP>(h, stage);
            __builtin_amdgcn_sched_barrier(0);
        });
        if constexpr (SLOTS < NB) static_for<SLOTS, NB>([&](auto r) { b.template read<H, decltype(r)::value>(so, nxt.b); });
        constexpr int DONE = (C::NF + GAP - 1) / GAP;
        if constexpr (DMA && DONE < C::LPS) static_for<DONE, C::LPS>([&](auto q) { issue<decltype(q)::value>(h, stage); });
    }

    // Reduction stages h0 .. h1-1 (a whole number of slabs, at least one),
    // after the stages of slab `tail` (>= 0) that ends past K: taken first, it
    // arrives with the ring's first fill and costs no wait of its own.  Stage
    // i of the sequence lives in ring stage i % NS.  Before the last half of a
    // stage's MFMAs every wave has read all of it and the next stage has
    // landed (barrier); the freed ring stage then takes stage i + NS.  Past
    // the end the last stage is requested again, into ring stages that are
    // not read, so the number of requests in flight at a barrier is fixed.
    template <int DT>
    __device__ __forceinline__ void kloop(f32x4 (&acc)[C::FM][C::FN], int h0, int h1, int tail, const GemmArgs& p) const {
        static_assert(C::NS > C::SPS, "the tail's stages are requested by the first fill");
#pragma unroll
        for (int i = 0; i < C::NS; ++i) {
            if (i < C::SPS && tail >= 0) issue_tail(tail * C::SPS + i, i, p);
            else {
                const int h = min(h0 + i - (tail >= 0 ? C::SPS : 0), h1 - 1);
                static_for<0, C::LPS>([&](auto q) { issue<decltype(q)::value>(h, i); });
            }
        }
        if (tail >= 0) h0 -= C::SPS;
        LinFrags<C> f, g;
        ring_barrier<C::LPS * (C::NS - 1)>();
        read_all<0>(0, f);
        __builtin_amdgcn_sched_barrier(0);
        int st = 0;
        auto last_half = [&](int h, LinFrags<C>& cur, LinFrags<C>& nxt) {
            const int sn = st + 1 == C::NS ? 0 : st + 1;
            cur.ready();
            ring_barrier<C::LPS * (C::NS - 2)>();
            multiply<DT, 0, true>(acc, cur, (uint32_t)sn * C::STAGE, nxt, min(h + C::NS, h1 - 1), st);
            __builtin_amdgcn_sched_barrier(0);
            st = sn;
        };
        if constexpr (C::HP == 2) {
            for (int h = h0; h < h1; ++h) {
                f.ready();
                multiply<DT, 1, false>(acc, f, (uint32_t)st * C::STAGE, g, 0, 0);
                __builtin_amdgcn_sched_barrier(0);
                last_half(h, g, f);
            }
        } else {
            for (int h = h0; h < h1; h += 2) {
                last_half(h, f, g);
                last_half(h + 1, g, f);
            }
        }
        f.ready();       // the last reads land before their registers are reused
    }

    // A stage of the slab that ends past K.
    __device__ __forceinline__ void issue_tail(int h, int stage, const GemmArgs& p) const {
#pragma unroll
        for (int q = 0; q < C::B_PER_WAVE; ++q) b.issue_tail(h, stage, q, p.ldb, p.K, p.zero);
#pragma unroll
        for (int q = 0; q < C::A_PER_WAVE; ++q) a.issue_tail(h, stage, q, p.lda, p.K, p.zero);
    }

    // The slab that ends past K alone (a reduction of fewer than 64).
    template <int DT>
    __device__ __forceinline__ void only_tail(f32x4 (&acc)[C::FM][C::FN], int slab, const GemmArgs& p) const {
#pragma unroll
        for (int i = 0; i < C::SPS; ++i) issue_tail(slab * C::SPS + i, i, p);
        ring_barrier<0>();
        static_for<0, 2>([&](auto s) {
            constexpr int S = decltype(s)::value;
            LinFrags<C> f;
            read_all<C::HP == 2 ? S : 0>(C::HP == 2 ? 0 : S * C::STAGE, f);
            f.ready();
#pragma unroll
            for (int m = 0; m < C::FM; ++m)
#pragma unroll
                for (int n = 0; n < C::FN; ++n) acc[m][n] = mfma16x16x32<DT>(f.b[n], f.a[m], acc[m][n]);
        });
    }
};

template <int DT>
__device__ __forceinline__ float widen(uint32_t v) {
    if constexpr (DT == DT_F16) return (float)__builtin_bit_cast(_Float16, (uint16_t)v);
    else return __builtin_bit_cast(float, v << 16);
}

// Eight storage values to fp32 and back.
template <int DT>
__device__ __forceinline__ void widen8(u32x4 v, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = widen<DT>(v[i] & 0xffffu);
        if constexpr (DT == DT_F16) f[2 * i + 1] = widen<DT>(v[i] >> 16);
        else f[2 * i + 1] = __builtin_bit_cast(float, v[i] & 0xffff0000u);
    }
}

// (The empty asm statements pin the values in fp32: see to_storage.)
template <int DT>
__device__ __forceinline__ u32x4 narrow8(const float (&f)[8]) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo = f[2 * i], hi = f[2 * i + 1];
        pin(lo);
        pin(hi);
        if constexpr (DT == DT_F16) v[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{lo, hi}), f16x2));
        else v[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{lo, hi}), bf16x2));
    }
    return v;
}

// Two fragments of one row of fragments, four columns per lane each, to eight
// neighbouring columns of one of them: lane group g gets columns
// 8 (g / 2) .. +7 of fragment g % 2.
__device__ __forceinline__ void pair8(const f32x4& x, const f32x4& y, float (&v)[8]) {
    // (whole vectors are cast: a bit cast of one element reads element 0)
    const u32x4 a = __builtin_bit_cast(u32x4, x), b = __builtin_bit_cast(u32x4, y);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t ai = a[i], bi = b[i];
        const auto s = __builtin_amdgcn_permlane16_swap(ai, bi, false, false);
        const uint32_t lo = s[0], hi = s[1];
        v[i] = __builtin_bit_cast(float, lo);
        v[4 + i] = __builtin_bit_cast(float, hi);
    }
}

// Eight columns n .. n+7 of row r: v + bias (gate; u and bu: up) to z, the
// activation, the residual, one rounding and the store.
template <int DT>
__device__ __forceinline__ void finish8(const GemmArgs& p, int64_t r, int n, float (&v)[8], float (&u)[8],
                                        const float (&b)[8], const float (&bu)[8], u32x4 res) {
    const bool gated = p.act == ACT_SWIGLU;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += b[i];
    if (gated) {
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] += bu[i];
    }
    if (p.z) {
        st16(p.z + (size_t)r * p.ldz + n, narrow8<DT>(v));
        if (gated) st16(p.z + (size_t)r * p.ldz + p.up + n, narrow8<DT>(u));
    }
    if (gated) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = silu(v[i]) * u[i];
    } else if (p.act == ACT_GELU_TANH) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = gelu_tanh(v[i]);
    }
    if (p.res) {
        float t[8];
        widen8<DT>(res, t);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += t[i];
    }
    st16(p.d + (size_t)r * p.ldd + n, narrow8<DT>(v));
}

// bias, activation, residual, rounding and stores of a tile's accumulators.
template <class C, int DT, int PASS>
__device__ __forceinline__ void linear_epilogue(const f32x4 (&acc)[C::FM][C::FN], const GemmArgs& p, int m0, int n0) {
    const int lane = threadIdx.x & 63, wave = uniform_wave();
    const int g = lane >> 4;
    const int m = m0 + wave / C::WN * C::WTM + (lane & 15);
    const int col = (g & 1) * 16 + (g >> 1) * 8;
    if (PASS == PASS_FWD && p.act == ACT_SWIGLU) {
        static_for<0, C::FN / 4>([&](auto q) {
            constexpr int Q = decltype(q)::value;
            const int n = n0 + wave % C::WN * (C::WTN / 2) + Q * 32 + col;
            const bool in = n < p.N;
            float bg[8] = {}, bu[8] = {};
            if (in && p.bias) {
                widen8<DT>(ld16(p.bias + n), bg);
                widen8<DT>(ld16(p.bias + p.up + n), bu);
            }
#pragma unroll
            for (int f = 0; f < C::FM; ++f) {
                const int r = m + f * 16;
                float vg[8], vu[8];
                pair8(acc[f][4 * Q], acc[f][4 * Q + 2], vg);
                pair8(acc[f][4 * Q + 1], acc[f][4 * Q + 3], vu);
                if (!in || r >= p.M) continue;
                finish8<DT>(p, r, n, vg, vu, bg, bu, p.res ? ld16(p.res + (size_t)r * p.ldr + n) : u32x4{});
            }
        });
        return;
    }
    static_for<0, C::FN / 2>([&](auto q) {
        constexpr int Q = decltype(q)::value;
        const int n = n0 + wave % C::WN * C::WTN + Q * 32 + col;
        const bool in = n < p.N;
        float b[8] = {};
        u32x4 res[C::FM];
        if (PASS == PASS_FWD && in) {
            if (p.bias) widen8<DT>(ld16(p.bias + n), b);
            // every residual chunk is requested before the first store
            if (p.res) {
#pragma unroll
                for (int f = 0; f < C::FM; ++f)
                    if (m + f * 16 < p.M) res[f] = ld16(p.res + (size_t)(m + f * 16) * p.ldr + n);
            }
        }
#pragma unroll
        for (int f = 0; f < C::FM; ++f) {
            const int r = m + f * 16;
            float v[8];
            pair8(acc[f][2 * Q], acc[f][2 * Q + 1], v);
            if (!in || r >= p.M) continue;
            if constexpr (PASS == PASS_FWD) {
                float none[8] = {};
                finish8<DT>(p, r, n, v, none, b, none, res[f]);
            } else {
                st16(p.d + (size_t)r * p.ldd + n, narrow8<DT>(v));
            }
        }
    });
}

// A part's fp32 accumulators to its tile of the partials, columns in the
// order of the tile's B columns.
template <class C>
__device__ __forceinline__ void store_part(const f32x4 (&acc)[C::FM][C::FN], const GemmArgs& p, int m0, int n0,
                                           uint32_t slot) {
    const int lane = threadIdx.x & 63, wave = uniform_wave();
    const int g = lane >> 4, row = wave / C::WN * C::WTM + (lane & 15), col = wave % C::WN * C::WTN + g * 4;
    float* part = p.part + (size_t)slot * C::BM * C::BN;
#pragma unroll
    for (int f = 0; f < C::FN; ++f) {
        const int frag = wave % C::WN * C::FN + f;
        if ((p.up ? n0 + (frag >> 1) * 16 : n0 + frag * 16) + g * 4 >= p.N) continue;
#pragma unroll
        for (int i = 0; i < C::FM; ++i)
            if (m0 + row + i * 16 < p.M)
                *reinterpret_cast<f32x4*>(part + (row + i * 16) * C::BN + col + f * 16) = acc[i][f];
    }
}

// Tile i of the order -> tile row and column: patches of PATCH row blocks,
// column by column, so the ~32 tiles an XCD runs at a time share few operand
// panels in its L2 (2048 x 6144 x 12288, x W / x^T dz in us: patches of 1
// 291 / 293, 2 281 / 281, 4 278 / 273, 8 283 / 276, 32 281 / 290).
constexpr uint32_t PATCH = 4;

__device__ __forceinline__ void tile_at(const GemmArgs& p, uint32_t i, uint32_t& mb, uint32_t& nb) {
    const uint32_t band = i / (PATCH * p.Nt), j = i - band * PATCH * p.Nt;
    const uint32_t h = p.Mt - band * PATCH < PATCH ? p.Mt - band * PATCH : PATCH;
    mb = band * PATCH + j % h;
    nb = j / h;
}

// Workgroup b -> tile of the order and part (whole tiles first).  The
// dispatcher deals workgroups to the 8 XCDs in turn; each XCD gets one
// contiguous chunk of the order.
__device__ __forceinline__ uint32_t tile_of(const GemmArgs& p, uint32_t b, uint32_t& s) {
    s = 0;
    if (b < p.direct) return xcd_chunked(b, p.direct);
    const uint32_t q = xcd_chunked(b - p.direct, (p.Mt * p.Nt - p.direct) * p.S);
    s = q % p.S;
    return p.direct + q / p.S;
}

template <class C, int DT, int PASS>
__device__ __forceinline__ void linear_tile(const GemmArgs& p, uint32_t block) {
    uint32_t mb, nb, s;
    const uint32_t i = tile_of(p, block, s);
    tile_at(p, i, mb, nb);
    const bool whole = i < p.direct || p.S == 1;
    const int m0 = mb * C::BM, n0 = nb * (p.up ? C::BN / 2 : C::BN);
    f32x4 acc[C::FM][C::FN] = {};
    {
        LinTile<C, PASS> t;
        t.a.init(p.a, p.lda, m0, p.M, 0);
        t.b.init(p.b, p.ldb, n0, p.N, p.up);
        const int slabs = p.K / BK;
        const int k0 = whole ? 0 : min((int)(s * p.ksp), slabs), k1 = whole ? slabs : min(k0 + (int)p.ksp, slabs);
        const bool tail = (whole || s + 1 == p.S) && p.K % BK;
        if (k1 > k0) t.template kloop<DT>(acc, k0 * C::SPS, k1 * C::SPS, tail ? slabs : -1, p);
        else if (tail) t.template only_tail<DT>(acc, slabs, p);
        ring_barrier<0>();      // no DMA in flight when the workgroup ends
    }
    if (whole) linear_epilogue<C, DT, PASS>(acc, p, m0, n0);
    else store_part<C>(acc, p, m0, n0, (i - p.direct) * p.S + s);
}

template <class C, int DT, int PASS>
__global__ __launch_bounds__(C::NT, C::OCC) void linear_kernel(GemmArgs p) {
    linear_tile<C, DT, PASS>(p, blockIdx.x);
}

// Both products of the gradient: the first `dx_blocks` workgroups dz W^T, the
// others x^T dz.  They depend on dz alone, so one launch fills the chip with
// the tiles of both and waits for one last round instead of two (fp16, both
// products, launches of their own against this: 64 x 512 x 2048 13.0 -> 8.9 us,
// 1365 x 1688 x 616 26 -> 15, 128 x 8192 x 5504 84 -> 66, 1000 x 12288 x 4096
// 220 -> 192, 2048 x 12288 x 6144 539 -> 528).
// The first `db_blocks` workgroups add the column sums of dz's row groups, one
// column per thread, in db_kernel's order (a launch of its own less: 300 x 1024
// x 1024 gelu 15.4 -> 13.5 us).
template <class C, int DT>
__global__ __launch_bounds__(C::NT, C::OCC) void linear_both_kernel(GemmArgs dx, GemmArgs dw, DzArgs dz, uint32_t db_blocks,
                                                                    uint32_t dx_blocks) {
    if (blockIdx.x < db_blocks) {
        const int n = dw.N, c = blockIdx.x * C::NT + threadIdx.x;
        if (c >= n) return;
        float s[8] = {}, sum = 0.f;
#pragma unroll 2
        for (int p = 0; p < dz.parts; p += 8) {
            float v[8];
#pragma unroll
            for (int g = 0; g < 8; ++g) v[g] = p + g < dz.parts ? dz.part[(size_t)(p + g) * n + c] : 0.f;
#pragma unroll
            for (int g = 0; g < 8; ++g) s[g] += v[g];
        }
#pragma unroll
        for (int g = 0; g < 8; ++g) sum += s[g];
        dz.db[c] = to_storage<DT>(sum);
        return;
    }
    const uint32_t b = blockIdx.x - db_blocks;
    if (b < dx_blocks) linear_tile<C, DT, PASS_DX>(dx, b);
    else linear_tile<C, DT, PASS_DW>(dw, b - dx_blocks);
}

}  // namespace mlpc

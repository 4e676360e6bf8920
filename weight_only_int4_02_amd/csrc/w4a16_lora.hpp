// The GEMM kernels' extension that adds low-rank adapters to their fp32
// accumulators (w4a16_gemm_lora): Y[m] += S[m] . B_a^T, a the row's adapter, S the
// low-rank values already formed (and scaled) by lora_shrink_kernel.
//
// S reaches the second product as hi + lo pairs of 16-bit values, so that it
// runs on the 16-bit matrix instructions with the adapters as they are and
// keeps 16 (bf16) or 22 (fp16) bits of each sum.  fp16 has too small a range
// for sums that B may bring back into it, so each row's 32 ranks are stored
// times a power of two that puts their largest into [2^14, 2^15), and F holds
// the inverse, multiplied back in 32 bits.
//
// Rows are kept apart: what an adapter holds (infinities and NaN included)
// reaches only the rows that name it, so no product of a masked row's zero
// with another adapter's B is ever added.
#pragma once
#include <hip/hip_runtime.h>

#include <type_traits>

#include "w4a16_device.hpp"
#include "w4a16_routed.hpp"

namespace w4a16 {

// The plain GEMM: nothing is added.
struct NoExt {
    static constexpr bool on = false;
};

struct LoraExt {
    static constexpr bool on = true;
    LoraArgs l;
};

__device__ __forceinline__ int lora_part(const LoraArgs &l, int n) {
    int p = 0;
    while (p + 1 < l.parts && n >= l.part_end[p])
        p++;
    return p;
}

// The low-rank values of 16 rows and 32 ranks (block jb) as the A operand of an
// MFMA, hi + lo in the 16-bit type: lane r + 16 i holds row m + r, ranks 8 i
// .. 8 i + 7, and in f the factors of its results' rows 4 i .. 4 i + 3.  Rows
// without an adapter hold whatever the memory does: each row of an MFMA's
// result has its own row of A alone, and theirs are not used.
struct LoraS {
    u4_t hi, lo;
    f4_t f;
};
template <bool BF>
__device__ __forceinline__ LoraS lora_s(const LoraArgs &l, int M, int jb, int m, int lane) {
    const int row = min(m + (lane & 15), M - 1);
    const int64_t at = ((int64_t)jb * M + row) * 32 + 8 * (lane >> 4);
    LoraS o;
    o.hi = *(const u4_t *)(l.S_hi + at);
    o.lo = *(const u4_t *)(l.S_lo + at);
    o.f = f4_t{1.f, 1.f, 1.f, 1.f};
    if constexpr (!BF)   // (F's rows are padded to whole tiles; past the last tile: any)
        o.f = *(const f4_t *)(l.F + (int64_t)jb * l.f_pitch + min((int64_t)m, l.f_pitch - 16) +
                              4 * (lane >> 4));
    return o;
}

// S B of 16 rows and 16 columns, before the factors.
template <bool BF>
__device__ __forceinline__ f4_t lora_mfma(const LoraS &s, u4_t w) {
    const f4_t zero = {0.f, 0.f, 0.f, 0.f};
    if constexpr (BF) {
        const bf8_t b = __builtin_bit_cast(bf8_t, w);
        return mfma16x16x32_bf16(__builtin_bit_cast(bf8_t, s.lo), b,
                                 mfma16x16x32_bf16(__builtin_bit_cast(bf8_t, s.hi), b, zero));
    } else {
        const h8_t b = __builtin_bit_cast(h8_t, w);
        return mfma16x16x32(__builtin_bit_cast(h8_t, s.lo), b,
                            mfma16x16x32(__builtin_bit_cast(h8_t, s.hi), b, zero));
    }
}

// acc += f v in the rows of the mask (bit e: this lane's row 4 i + e) where col.
__device__ __forceinline__ void lora_select(f4_t &acc, f4_t v, f4_t f, uint32_t rows, bool col) {
#pragma unroll
    for (int e = 0; e < 4; e++)
        acc[e] += col && (rows >> e & 1) ? f[e] * v[e] : 0.f;
}

// The adapters of one 16-row tile (LoraList), through the scalar cache: the
// list is uniform, and its loads do not wait in line with the kernel's own.
struct LoraTile {
    const __attribute__((address_space(4))) LoraList *l;
    int count;
};
__device__ __forceinline__ LoraTile lora_tile(const LoraArgs &a, int M, int m) {
    LoraTile t;
    t.l = (const __attribute__((address_space(4))) LoraList *)(uintptr_t)(a.lists + m / 16);
    t.count = m < M ? t.l->count : 0;
    return t;
}

// The small-M kernels: adds the adapters to one wave's part acc of the results
// of 16 MT rows from m_base and 16 NB columns from n_base.  The work is cut
// into items -- one adapter of one 16-row tile, and P blocks of 32 ranks of one
// part -- which the W waves of a workgroup take in turn; their parts are
// summed at the end like the rest.  P is 2 for ranks above 32, so that both
// halves of B's 128-byte lines are read at once.
//
// begin() issues the loads of the wave's first items, before the ring's first
// stage, and finish() adds them and takes the others: the first items cost the
// wave no latency that the stage's own loads do not have.
template <bool BF, int W, int NB, int MT, int P>
struct LoraPart {
    // items in flight: as many as their registers (8 P S values, 4 P NB of B)
    // leave room for
    static_assert(MT <= 2, "an item's row tile is 0 or 1");
    static constexpr int BATCH = P * NB <= 2 ? 4 : P * NB <= 6 ? 2 : 1;
    struct Item {
        int t;             // row tile, -1: none
        uint32_t rows;
        int c_lo, c_hi;    // columns of the part
        LoraS s[P];
        u4_t w[P][NB];
    };
    const LoraArgs &l;
    int M, N, m_base, n_base, lane;
    LoraTile tile[MT];
    int per, items, next, p0, steps;
    Item it[BATCH];

    __device__ __forceinline__ LoraPart(const LoraArgs &l_, int M_, int N_, int m_base_, int n_base_,
                                        int wave, int lane_)
        : l(l_), M(M_), N(N_), m_base(m_base_), n_base(n_base_), lane(lane_) {
        per = 0;
#pragma unroll
        for (int t = 0; t < MT; t++) {
            tile[t] = lora_tile(l, M, m_base + 16 * t);
            per += tile[t].count;
        }
        p0 = lora_part(l, min(n_base, N - 1));
        const int p1 = lora_part(l, min(N, n_base + 16 * NB) - 1);
        steps = (l.blocks + P - 1) / P;
        items = n_base < N ? per * steps * (p1 - p0 + 1) : 0;
        next = wave;
    }
    __device__ __forceinline__ void load(Item &x) {
        x.t = -1;
        if (next >= items)
            return;
        const int ps = next / per, k = next - ps * per;
        const int p = p0 + ps / steps, jb = (ps % steps) * P;
        next += W;
        x.t = MT == 2 && k >= tile[0].count ? 1 : 0;
        const int at = x.t ? k - tile[0].count : k;
        const LoraTile &tl = tile[MT == 2 ? x.t : 0];
        const int a = tl.l->adapter[at];
        x.rows = tl.l->rows[at];
        x.c_lo = p ? l.part_end[p - 1] : 0;
        x.c_hi = l.part_end[p];
        const int r = lane & 15, i = lane >> 4;
#pragma unroll
        for (int h = 0; h < P; h++) {
            // (the last pair of an odd number of blocks: the last block again,
            // against a B of zeros)
            const int b32 = min(jb + h, l.blocks - 1);
            x.s[h] = lora_s<BF>(l, M, p * l.blocks + b32, m_base + 16 * x.t, lane);
            const int j = 32 * (jb + h) + 8 * i;
#pragma unroll
            for (int b = 0; b < NB; b++) {
                const int n = n_base + 16 * b + r;
                x.w[h][b] = u4_t{0u, 0u, 0u, 0u};
                if (n >= x.c_lo && n < x.c_hi && j < l.r)
                    x.w[h][b] = *(const u4_t *)(l.B + ((int64_t)a * N + n) * l.r + j);
            }
        }
    }
    __device__ __forceinline__ void add(const Item &x, f4_t (&acc)[NB][MT]) {
#pragma unroll
        for (int t = 0; t < MT; t++) {
            if (x.t != t)
                continue;
#pragma unroll
            for (int b = 0; b < NB; b++) {
                const int n = n_base + 16 * b + (lane & 15);
#pragma unroll
                for (int h = 0; h < P; h++)
                    lora_select(acc[b][t], lora_mfma<BF>(x.s[h], x.w[h][b]), x.s[h].f,
                                x.rows >> (4 * (lane >> 4)), n >= x.c_lo && n < x.c_hi);
            }
        }
    }
    __device__ __forceinline__ void begin() {
#pragma unroll
        for (int u = 0; u < BATCH; u++)
            load(it[u]);
        __builtin_amdgcn_sched_barrier(0);
    }
    __device__ __forceinline__ void finish(f4_t (&acc)[NB][MT]) {
        while (it[0].t >= 0) {
#pragma unroll
            for (int u = 0; u < BATCH; u++)
                add(it[u], acc);
            begin();
        }
    }
};

// A wave's 16 TM x 16 TN tile of results at row m_base, column n_base (the
// large-M kernel).  The distinct adapters of the tile's rows are taken one
// after the other: one in a prompt's tile, whose B tiles are then loaded once,
// and up to 16 TM where every row has its own.
template <bool BF, int TM, int TN>
__device__ __forceinline__ void lora_add_tile(const LoraArgs &l, int M, int N, int m_base,
                                              int n_base, int lane, f4_t (&acc)[TM][TN]) {
    static_assert(TM <= 8, "two rows per lane at most");
    const int r = lane & 15, i = lane >> 4;
    if (n_base >= N)
        return;
    // lane's rows: lane, lane + 64
    auto id_of = [&](int row) __attribute__((always_inline)) {
        const int m = m_base + row;
        const int id = row < 16 * TM && m < M ? l.ids[m] : -1;
        return id < l.n ? id : -1;
    };
    const int id0 = id_of(lane), id1 = TM > 4 ? id_of(lane + 64) : -1;
    uint64_t todo0 = __ballot(id0 >= 0), todo1 = __ballot(id1 >= 0);
    const int p0 = lora_part(l, n_base), p1 = lora_part(l, min(N, n_base + 16 * TN) - 1);
    while (todo0 | todo1) {
        const int a = todo0 ? __builtin_amdgcn_readlane(id0, __builtin_ctzll(todo0))
                            : __builtin_amdgcn_readlane(id1, __builtin_ctzll(todo1));
        const uint64_t in0 = __ballot(id0 == a), in1 = TM > 4 ? __ballot(id1 == a) : 0;
        todo0 &= ~in0;
        todo1 &= ~in1;
        for (int p = p0; p <= p1; p++) {
            const int c_lo = p ? l.part_end[p - 1] : 0, c_hi = l.part_end[p];
            for (int jb = 0; jb < l.blocks; jb++) {
                const int j = 32 * jb + 8 * i;
                u4_t w[TN];
#pragma unroll
                for (int t = 0; t < TN; t++) {
                    const int n = n_base + 16 * t + r;
                    w[t] = u4_t{0u, 0u, 0u, 0u};
                    if (n >= c_lo && n < c_hi && j < l.r)
                        w[t] = *(const u4_t *)(l.B + ((int64_t)a * N + n) * l.r + j);
                }
                constexpr int H = TM < 4 ? TM : 4;   // row tiles whose loads are in flight together
                LoraS s[H];
#pragma unroll
                for (int mi = 0; mi < TM; mi++) {
                    if (mi % H == 0) {
#pragma unroll
                        for (int h = 0; h < H; h++)
                            s[h] = lora_s<BF>(l, M, p * l.blocks + jb, m_base + 16 * (mi + h), lane);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                    const uint32_t rows = (uint32_t)((mi < 4 ? in0 : in1) >> (16 * (mi & 3))) & 0xFFFFu;
                    if (!rows)
                        continue;
#pragma unroll
                    for (int t = 0; t < TN; t++) {
                        const int n = n_base + 16 * t + r;
                        lora_select(acc[mi][t], lora_mfma<BF>(s[mi % H], w[t]), s[mi % H].f,
                                    rows >> (4 * i), n >= c_lo && n < c_hi);
                    }
                }
            }
        }
    }
}

}  // namespace w4a16

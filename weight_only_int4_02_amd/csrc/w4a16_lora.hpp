// The GEMM kernels' extension that adds low-rank adapters to their fp32
// results (w4a16_gemm_lora): Y[m] += S[m] . B_a^T, a the row's adapter, S the
// low-rank values already formed (and scaled) by lora_shrink_kernel.
//
// Rows are kept apart: what an adapter holds (infinities and NaN included)
// reaches only the rows that name it, so no product of a masked row's zero
// with another adapter's B is ever added.
#pragma once
#include <hip/hip_runtime.h>

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

// Four rows m0 .. m0 + 3 of column n, by plain fp32 multiply-adds: rank r
// terms for each result, against K of them in the GEMM.
template <bool BF>
__device__ __forceinline__ void lora_add4(const LoraArgs &l, int M, int N, int m0, int n, f4_t &v) {
    const int off = lora_part(l, n) * l.r;
#pragma unroll
    for (int rr = 0; rr < 4; rr++) {
        const int m = m0 + rr;
        if (m >= M)
            continue;
        const int a = l.ids[m];
        if (a < 0 || a >= l.n)
            continue;
        const float *s = l.S + (int64_t)m * l.pr + off;
        const uint16_t *b = l.B + ((int64_t)a * N + n) * l.r;
        float sum = 0.f;
        for (int j = 0; j < l.r; j += 8) {
            const u4_t w = *(const u4_t *)(b + j);
            const f4_t s0 = *(const f4_t *)(s + j), s1 = *(const f4_t *)(s + j + 4);
#pragma unroll
            for (int c = 0; c < 4; c++) {
                float lo, hi;
                if constexpr (BF) {
                    lo = bf16_bits_to_float(w[c] & 0xFFFFu);
                    hi = bf16_bits_to_float(w[c] >> 16);
                } else {
                    const h2_t h = as_h2(w[c]);
                    lo = (float)h.x;
                    hi = (float)h.y;
                }
                sum += lo * (c < 2 ? s0[2 * c] : s1[2 * c - 4]);
                sum += hi * (c < 2 ? s0[2 * c + 1] : s1[2 * c - 3]);
            }
        }
        v[rr] += sum;
    }
}

// v as hi + lo, two bf16 (16 bits of its significand; all 11 of an fp16
// value).  Where hi is not finite, lo is 0.
struct Bf16Pair {
    __bf16 hi, lo;
};
__device__ __forceinline__ Bf16Pair bf16_pair(float v) {
    Bf16Pair p;
    p.hi = (__bf16)v;
    const float h = (float)p.hi;
    p.lo = __builtin_isfinite(h) ? (__bf16)(v - h) : (__bf16)0.f;
    return p;
}

// A wave's 16 TM x 16 TN tile of results at row m_base, column n_base, by bf16
// MFMA.  S goes in as hi + lo pairs (bf16 has fp32's range, so no value
// overflows where an fp16 operand would), an fp16 B as an exact hi + lo pair:
// S B = Shi Bhi + Slo Bhi + Shi Blo, what is left out is below 2^-17 |S B|.
// The distinct adapters of the tile's rows are taken one after the other:
// one in a prompt's tile, up to 16 TM where every row has its own.
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
            for (int j0 = 0; j0 < l.r; j0 += 32) {
                const int j = j0 + 8 * i;
                bf8_t bh[TN], bl[TN];
#pragma unroll
                for (int t = 0; t < TN; t++) {
                    const int n = n_base + 16 * t + r;
                    u4_t w = {0u, 0u, 0u, 0u};
                    if (n >= c_lo && n < c_hi && j < l.r)
                        w = *(const u4_t *)(l.B + ((int64_t)a * N + n) * l.r + j);
                    if constexpr (BF) {
                        bh[t] = __builtin_bit_cast(bf8_t, w);
                    } else {
                        const h8_t h = __builtin_bit_cast(h8_t, w);
#pragma unroll
                        for (int c = 0; c < 8; c++) {
                            const Bf16Pair q = bf16_pair((float)h[c]);
                            bh[t][c] = q.hi;
                            bl[t][c] = q.lo;
                        }
                    }
                }
#pragma unroll
                for (int mi = 0; mi < TM; mi++) {
                    const uint32_t rows = (uint32_t)((mi < 4 ? in0 : in1) >> (16 * (mi & 3))) & 0xFFFFu;
                    if (!rows)
                        continue;
                    f4_t s0 = {0.f, 0.f, 0.f, 0.f}, s1 = s0;
                    if ((rows >> r & 1) && j < l.r) {
                        const float *s = l.S + (int64_t)(m_base + 16 * mi + r) * l.pr + p * l.r + j;
                        s0 = *(const f4_t *)s;
                        s1 = *(const f4_t *)(s + 4);
                    }
                    bf8_t sh, sl;
#pragma unroll
                    for (int c = 0; c < 8; c++) {
                        const Bf16Pair q = bf16_pair(c < 4 ? s0[c] : s1[c - 4]);
                        sh[c] = q.hi;
                        sl[c] = q.lo;
                    }
#pragma unroll
                    for (int t = 0; t < TN; t++) {
                        f4_t v = mfma16x16x32_bf16(sh, bh[t], f4_t{0.f, 0.f, 0.f, 0.f});
                        v = mfma16x16x32_bf16(sl, bh[t], v);
                        if constexpr (!BF)
                            v = mfma16x16x32_bf16(sh, bl[t], v);
                        // (this lane's results: column n_base + 16 t + r, rows 4 i ..)
                        const int n = n_base + 16 * t + r;
                        const bool col = n >= c_lo && n < c_hi;
#pragma unroll
                        for (int e = 0; e < 4; e++)
                            acc[mi][t][e] += col && (rows >> (4 * i + e) & 1) ? v[e] : 0.f;
                    }
                }
            }
        }
    }
}

}  // namespace w4a16

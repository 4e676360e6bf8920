// Device helpers shared by the experts' kernels.
#pragma once
#include "w4a16_gemm_kernels.hpp"
#include "w4a16_routed.hpp"

namespace w4a16 {

// v / (1 + exp(-v)).  exp2 and the reciprocal by the hardware's instructions,
// each good to one step of 32 bits (2 units of 2^-24); log2(e) and its product
// with v are rounded before the exp2 (2 |v| units), the sum and the last product
// after it (one each): off by at most (2 |v| + 8) 2^-24 of itself down to v = -87
// -- nothing beside the rounding of h to 16 bits.  Below, where it is less than
// 2^-119, the reciprocal's result is subnormal and may be flushed: -0.
__device__ __forceinline__ float silu(float v) {
    return v * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.44269504088896341f * v));
}

template <bool BF>
__device__ __forceinline__ void store_buffer16(__amdgpu_buffer_rsrc_t rsrc, uint32_t at, float v) {
    if constexpr (BF)
        __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, (__bf16)v), rsrc, (int)at, 0, 0);
    else
        __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, (_Float16)v), rsrc, (int)at, 0, 0);
}

// bf16 weights by one fma each: (q - z) s = q s - z s, exact in fp32 (q s and z s
// have at most 12 significant bits, the result 13), then one rounding to bf16.
// Eight instructions of 31 less per word than dequant_word_bf16, which is what
// the bf16 kernels are made of.  It gives +0 where that gives -0 (q = z, s < 0),
// which no sum notices, and needs |s| < 2^124 (z s in range).
struct Bf16Fma {
    float s, nzs;   // s, -(z s)
};
__device__ __forceinline__ Bf16Fma bf16_fma(uint32_t sbits, uint32_t z) {
    const float s = bf16_bits_to_float(sbits);
    return {s, -((float)z * s)};
}

__device__ __forceinline__ bf8_t dequant_word_bf16_fma(uint32_t w, Bf16Fma g) {
    const uint32_t lo = w & 0x0F0F0F0Fu, hi = (w >> 4) & 0x0F0F0F0Fu;
    const float q[8] = {(float)(lo & 0xFFu),         (float)((lo >> 16) & 0xFFu),
                        (float)(hi & 0xFFu),         (float)((hi >> 16) & 0xFFu),
                        (float)((lo >> 8) & 0xFFu),  (float)(lo >> 24),
                        (float)((hi >> 8) & 0xFFu),  (float)(hi >> 24)};
    u4_t o;
#pragma unroll
    for (int p = 0; p < 4; p++) {
        const float a = __builtin_fmaf(q[2 * p], g.s, g.nzs), b = __builtin_fmaf(q[2 * p + 1], g.s, g.nzs);
        o[p] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f2_t{a, b}, bf2_t));
    }
    return __builtin_bit_cast(bf8_t, o);
}

// One MFMA of 16 x 16 results with the weight operand formed from a packed word.
template <bool BF>
__device__ __forceinline__ f4_t expert_mfma(u4_t x, uint32_t word, uint32_t z, uint32_t sbits,
                                            uint32_t magic, f4_t c) {
    if constexpr (BF) {
        return mfma16x16x32_bf16(__builtin_bit_cast(bf8_t, x),
                                 dequant_word_bf16_fma(word, bf16_fma(sbits, z)), c);
    } else {
        return mfma16x16x32(__builtin_bit_cast(h8_t, x),
                            dequant_word(word, zero_pair(z), scale_pair(sbits), magic), c);
    }
}

// mfma8_dequant_bf16 with that form: eight MFMAs with the next word's
// dequantization between them, four vector instructions after each of the
// first six, and the same FORMs and hazards.
#define W4E_M(n) "v_mfma_f32_16x16x32_bf16 %[c" #n "], %[a" #n "], %[b], %[c" #n "]\n"
#define W4E_BLOCK(P0, S0, P1, S1, P2, S2, P3, S3, P4, S4, P5, S5, P6, S6, P7, S7)                  \
    asm volatile(P0 W4E_M(0) S0                                                                  \
                 "v_and_b32 %[lo], %[m], %[w]\n"                                                 \
                 "v_lshrrev_b32 %[hi], 4, %[w]\n"                                                \
                 "v_and_b32 %[hi], %[m], %[hi]\n"                                                \
                 "v_cvt_f32_ubyte0 %[f0], %[lo]\n" P1 W4E_M(1) S1                                \
                 "v_cvt_f32_ubyte2 %[f1], %[lo]\n"                                               \
                 "v_cvt_f32_ubyte0 %[f2], %[hi]\n"                                               \
                 "v_cvt_f32_ubyte2 %[f3], %[hi]\n"                                               \
                 "v_cvt_f32_ubyte1 %[f4], %[lo]\n" P2 W4E_M(2) S2                                \
                 "v_cvt_f32_ubyte3 %[f5], %[lo]\n"                                               \
                 "v_cvt_f32_ubyte1 %[f6], %[hi]\n"                                               \
                 "v_cvt_f32_ubyte3 %[f7], %[hi]\n"                                               \
                 "v_fma_f32 %[f0], %[f0], %[s], %[zs]\n" P3 W4E_M(3) S3                          \
                 "v_fma_f32 %[f1], %[f1], %[s], %[zs]\n"                                         \
                 "v_fma_f32 %[f2], %[f2], %[s], %[zs]\n"                                         \
                 "v_fma_f32 %[f3], %[f3], %[s], %[zs]\n"                                         \
                 "v_fma_f32 %[f4], %[f4], %[s], %[zs]\n" P4 W4E_M(4) S4                          \
                 "v_fma_f32 %[f5], %[f5], %[s], %[zs]\n"                                         \
                 "v_fma_f32 %[f6], %[f6], %[s], %[zs]\n"                                         \
                 "v_fma_f32 %[f7], %[f7], %[s], %[zs]\n" P5 W4E_M(5) S5                          \
                 "v_cvt_pk_bf16_f32 %[bn0], %[f0], %[f1]\n"                                      \
                 "v_cvt_pk_bf16_f32 %[bn1], %[f2], %[f3]\n"                                      \
                 "v_cvt_pk_bf16_f32 %[bn2], %[f4], %[f5]\n"                                      \
                 "v_cvt_pk_bf16_f32 %[bn3], %[f6], %[f7]\n" P6 W4E_M(6) S6 P7 W4E_M(7) S7        \
                 : [c0] "+v"(c0), [c1] "+v"(c1), [c2] "+v"(c2), [c3] "+v"(c3), [c4] "+v"(c4),    \
                   [c5] "+v"(c5), [c6] "+v"(c6), [c7] "+v"(c7), [bn0] "=&v"(bn0),                \
                   [bn1] "=&v"(bn1), [bn2] "=&v"(bn2), [bn3] "=&v"(bn3), [lo] "=&v"(lo),         \
                   [hi] "=&v"(hi), [f0] "=&v"(f0), [f1] "=&v"(f1), [f2] "=&v"(f2),               \
                   [f3] "=&v"(f3), [f4] "=&v"(f4), [f5] "=&v"(f5), [f6] "=&v"(f6),               \
                   [f7] "=&v"(f7), [a0] "+v"(a[0]), [a1] "+v"(a[1]), [a2] "+v"(a[2]),            \
                   [a3] "+v"(a[3]), [a4] "+v"(a[4]), [a5] "+v"(a[5]), [a6] "+v"(a[6]),           \
                   [a7] "+v"(a[7])                                                               \
                 : [b] "v"(b), [w] "v"(w), [zs] "v"(g.nzs), [s] "v"(g.s), [m] "s"(m),            \
                   [ln] "v"(lds_next))
#define W4E_PF(m, off) "ds_read_b128 %[a" #m "], %[ln] offset:" #off "\n"
#define W4E_WT(n) "s_waitcnt lgkmcnt(" #n ")\n"
template <int FORM>
__device__ __forceinline__ h8_t mfma8_dequant_bf16_fma(f4_t &c0, f4_t &c1, f4_t &c2, f4_t &c3,
                                                         f4_t &c4, f4_t &c5, f4_t &c6, f4_t &c7,
                                                         h8_t (&a)[8], h8_t b, uint32_t w, Bf16Fma g,
                                                         uint32_t m, uint32_t lds_next) {
    uint32_t bn0, bn1, bn2, bn3, lo, hi;
    float f0, f1, f2, f3, f4, f5, f6, f7;
    if constexpr (FORM == 0)
        W4E_BLOCK("", "", "", "", "", "", "", "", "", "", "", "", "", "", "", "");
    else if constexpr (FORM == 3)
        W4E_BLOCK("s_nop 1\n", "", "", "", "", "", "", "", "", "", "", "", "", "", "", "");
    else if constexpr (FORM == 1)
        W4E_BLOCK(W4E_WT(7), "", W4E_WT(6), "", W4E_WT(5), "", W4E_WT(4), "", W4E_WT(3), "",
                  W4E_WT(2), "", W4E_WT(1), "", W4E_WT(0), "");
    else
        W4E_BLOCK("", W4E_PF(0, 0), "", W4E_PF(1, 4096), "", W4E_PF(2, 8192), "",
                  W4E_PF(3, 12288), "", W4E_PF(4, 16384), "", W4E_PF(5, 20480), "",
                  W4E_PF(6, 24576), "", W4E_PF(7, 28672));
    return __builtin_bit_cast(h8_t, u4_t{bn0, bn1, bn2, bn3});
}
#undef W4E_PF
#undef W4E_WT
#undef W4E_BLOCK
#undef W4E_M

// ---------------------------------------------------------------------------
// h = silu(gate) up beyond 65504 does not fit the fp16 operand of the second
// product: it is stored as infinity, and every result of that row comes out
// infinite or NaN.  Whoever rounds the results sees that and forms them again
// here, with each infinite h in 32 bits (from its two rows of the first
// product) and plain fp32 sums.  Rows without such a value cost a test of
// their results.  One token through two experts of the 7B MLP's size, 34 us,
// takes 0.8 ms with a few such columns and 20 ms with a sixth of them; 4096
// tokens over 64 experts with one such row 1.2 and 7 ms instead of 0.5.  A
// scale for each row instead would have to be known before the first column of
// h is stored, and the row's columns are formed by different workgroups.
// ---------------------------------------------------------------------------

// One expert's matrices (uniform), addressed by 32-bit offsets from their first
// tile, and the scale bits and zero of the group of columns 8 q .. of row r of a
// tile.
struct ExpertBase {
    const uint32_t *q, *z;
    const uint16_t *s;
};
__device__ __forceinline__ ExpertBase expert_base(const ExpertsArgs &a, int e, int parts) {
    const int64_t tile = (int64_t)e * parts * a.NT;
    return {(const uint32_t *)a.qd + tile * a.KT * 256, a.sym ? nullptr : (const uint32_t *)a.zd + tile * a.GW * 16,
            (const uint16_t *)a.sd + tile * a.G * 16};
}
struct RowGroup {
    uint32_t s, z;
};
__device__ __forceinline__ RowGroup row_group(const ExpertsArgs &a, const ExpertBase &b, uint32_t tile, uint32_t r,
                                              int q) {
    const uint32_t grp = (uint32_t)min((8 * q) >> a.lg, a.G - 1);
    const uint32_t s = b.s[(tile * a.G + grp) * 16 + r];
    const uint32_t z = a.sym ? 8u : (b.z[(tile * a.GW + (grp >> 3)) * 16 + r] >> (4 * (grp & 7))) & 0xFu;
    return {s, z};
}

// Column i of h for row t of X and expert e, in 32 bits; the whole wave together.
__device__ __forceinline__ float wide_h(const ExpertsArgs &gu, int64_t t, int e, int i, int lane) {
    const ExpertBase b = expert_base(gu, e, 2);
    const uint32_t tile = (uint32_t)i >> 4, r = i & 15;   // (up's: NT further)
    const uint16_t *x_row = gu.X + t * gu.K;
    float sum[2] = {0.f, 0.f};
    for (int q = lane; 8 * q < gu.K; q += 64) {
        const h8_t x = *(const h8_t *)(x_row + 8 * q);
#pragma unroll
        for (int p = 0; p < 2; p++) {
            const uint32_t tp = tile + p * gu.NT;
            const RowGroup g = row_group(gu, b, tp, r, q);
            const uint32_t word = b.q[((tp * gu.KT + (q >> 4)) * 64 + r + 16 * (q & 3)) * 4 + ((q >> 2) & 3)];
            const h8_t w = dequant_word(word, zero_pair(g.z), scale_pair(g.s));
#pragma unroll
            for (int k = 0; k < 8; k++)
                sum[p] = fmaf((float)x[k], (float)w[k], sum[p]);
        }
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        sum[0] += __shfl_xor(sum[0], d);
        sum[1] += __shfl_xor(sum[1], d);
    }
    return silu(sum[0]) * sum[1];
}

// Whether a stored row of h holds an infinity (else what is not finite in its
// results came from elsewhere, a NaN in X say, and they stand); the whole wave.
__device__ __forceinline__ bool row_overflowed(const ExpertsArgs &dn, int64_t row, int lane) {
    bool inf = false;
    for (int i = 8 * lane; i < dn.K; i += 512) {
        const h8_t h = *(const h8_t *)(dn.X + row * dn.K + i);
#pragma unroll
        for (int k = 0; k < 8; k++)
            inf = inf || __builtin_isinf((float)h[k]);
    }
    return __any(inf);
}

// Columns of h that a wave holds in LDS at once, in 32 bits.
constexpr int kWideColumns = 1024;

// out += weight h . Wdown for columns n .. n + C - 1 (each lane its own n), h being
// row `row` of the stored ones; the whole wave together, hs its own LDS.
template <int C>
__device__ __forceinline__ void wide_dot(const ExpertsArgs &gu, const ExpertsArgs &dn, int64_t t, int64_t row,
                                         int e, float weight, int n, int lane, float *hs, float (&out)[C]) {
    const ExpertBase b = expert_base(dn, e, 1);
#pragma nounroll
    for (int i0 = 0; i0 < dn.K; i0 += kWideColumns) {
#pragma nounroll
        for (int at = 8 * lane; at < kWideColumns; at += 512) {
            h8_t stored = {};
            if (i0 + at < dn.K)
                stored = *(const h8_t *)(dn.X + row * dn.K + i0 + at);
            uint32_t inf = 0;
#pragma unroll
            for (int k = 0; k < 8; k++) {
                hs[at + k] = (float)stored[k];
                inf |= __builtin_isinf((float)stored[k]) ? 1u << k : 0u;
            }
            // one by one, the whole wave on each
            for (uint64_t lanes = __ballot(inf != 0); lanes; lanes &= lanes - 1) {
                const int from = __builtin_ctzll(lanes);
                const int base = at - 8 * lane + 8 * from;
                for (uint32_t bits = __builtin_amdgcn_readlane(inf, from); bits; bits &= bits - 1) {
                    const int i = base + __builtin_ctz(bits);
                    const float v = wide_h(gu, t, e, __builtin_amdgcn_readfirstlane(i0 + i), lane);
                    if (lane == from)
                        hs[i] = v;
                }
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        const int kt1 = min(dn.KT, (i0 + kWideColumns) >> 7);
#pragma nounroll
        for (int kt = i0 >> 7; kt < kt1; kt++) {
#pragma nounroll
            for (int c = 0; c < C; c++) {
                const uint32_t tile = (uint32_t)(n + c) >> 4, r = (n + c) & 15;
                float part = 0.f;
#pragma nounroll
                for (int i = 0; i < 4; i++) {
                    const u4_t word = ((const u4_t *)b.q)[(tile * dn.KT + kt) * 64 + r + 16 * i];
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        // (a word at a time: the next one's values only after this
                        // one's sum, or they would take all registers)
                        uint32_t at = (uint32_t)(kt * 128 - i0 + 32 * j + 8 * i), wd = word[j];
                        asm volatile("" : "+v"(at), "+v"(wd), "+v"(part));
                        const RowGroup g = row_group(dn, b, tile, r, 16 * kt + 4 * j);
                        const h8_t w = dequant_word(wd, zero_pair(g.z), scale_pair(g.s));
                        const f4_t h0 = *(const f4_t *)&hs[at], h1 = *(const f4_t *)&hs[at + 4];
#pragma unroll
                        for (int k = 0; k < 4; k++) {
                            part = fmaf(h0[k], (float)w[k], part);
                            part = fmaf(h1[k], (float)w[4 + k], part);
                        }
                    }
                }
#pragma unroll
                for (int k = 0; k < C; k++)
                    out[k] += k == c ? weight * part : 0.f;
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // (before the next columns)
    }
}

}  // namespace w4a16

// Products with MXFP4 weights for few rows (memory-bound).
//
// A workgroup takes NB column tiles of 16 and MT row tiles of 16, its KS waves
// (or, of one wave along K, four workgroups' worth of columns side by side)
// each every KS-th 128-column tile of K.  A weight tile is one 16-byte load a
// lane, straight into the operand registers (block b of row r in lane 16 b + r).
// The weights are the first operand, so a lane
// holds four neighbouring columns of one row's results.  With 16-bit
// activations, word j of a lane's block multiplies the same eight columns of its
// row of X, a matrix instruction of 16 x 16 x 32 for each j: the order of K
// inside an instruction is free as long as both operands have it.
#include <hip/hip_runtime.h>

#include "w4a16_mx_device.hpp"

namespace w4a16 {

namespace {

__device__ __forceinline__ u4_t load16(__amdgpu_buffer_rsrc_t r, uint32_t v, uint32_t s) {
    return __builtin_bit_cast(u4_t, __builtin_amdgcn_raw_buffer_load_b128(r, (int)v, (int)s, 0));
}
__device__ __forceinline__ uint32_t load4(__amdgpu_buffer_rsrc_t r, uint32_t v, uint32_t s) {
    return (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(r, (int)v, (int)s, 0);
}

// Words j of the four lane groups become group j's four words: in lanes 16 i + r
// word j is then word i of block j.
__device__ __forceinline__ u4_t transpose_words(u4_t w) {
    const auto a = __builtin_amdgcn_permlane16_swap(w.x, w.y, false, false);
    const auto b = __builtin_amdgcn_permlane16_swap(w.z, w.w, false, false);
    const auto c = __builtin_amdgcn_permlane32_swap(a[0], b[0], false, false);
    const auto d = __builtin_amdgcn_permlane32_swap(a[1], b[1], false, false);
    return u4_t{c[0], d[0], c[1], d[1]};
}

// One 128-column tile's operands of a wave.
template <int XT, int MT, int NB>
struct Stage {
    u4_t w[NB], x[MT][XT == MX_X_FP4 ? 1 : 4];
    uint32_t ws[NB], xs[MT];
};

// WAVES: of the workgroup; KS of them along K, the others on further columns.
template <int XT, int MT, int NB, int WAVES, int KS, int DEPTH, bool GROUPED>
__global__ __launch_bounds__(WAVES * 64) void mx_small_kernel(MxArgs a, int blocks_n, bool ybf) {
    constexpr bool FP4 = XT == MX_X_FP4;
    constexpr int NW = WAVES / KS;
    // column tiles whose sums lie in LDS at a time (at most 64 KiB)
    constexpr int NP = WAVES * MT * NB <= 64 ? NB : 64 / (WAVES * MT);
    __shared__ f4_t sums[KS > 1 ? WAVES * MT * NP * 64 : 1];
    const int lane = threadIdx.x & 63, r = lane & 15, kb = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int ks = wave % KS, nw = wave / KS;

    const int tile = blockIdx.x / blocks_n, block = blockIdx.x - tile * blocks_n;
    MxTile t;
    if constexpr (GROUPED) {
        t = mx_find_tile<16 * MT>(a, tile, lane);
        if (t.count == 0)
            return;
    } else {
        t = MxTile{0, 0, (int)a.R, 1};
        t.take(tile, 16 * MT);
    }
    const int nt0 = (block * NW + nw) * NB;

    // (a column tile past the last one reads zeros: its offset is past the matrix)
    const uint32_t wbytes = (uint32_t)a.NT * (uint32_t)a.KT * 1024u, sbytes = (uint32_t)a.NT * (uint32_t)a.KG * 256u;
    const __amdgpu_buffer_rsrc_t rw = make_rsrc((const char *)a.qd + (int64_t)t.e * wbytes, wbytes);
    const __amdgpu_buffer_rsrc_t rs = make_rsrc((const char *)a.sd + (int64_t)t.e * sbytes, sbytes);
    const uint32_t xrow = FP4 ? 128u : (uint32_t)a.K * 2u;
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.X, (uint32_t)(a.T * (FP4 ? a.KG * 256 : a.K * 2)));
    const __amdgpu_buffer_rsrc_t rxs = make_rsrc(a.xs, FP4 ? (uint32_t)(a.T * a.KG * 16) : 0u);
    const uint32_t wo = (uint32_t)(kb >> 1) * (uint32_t)a.NT * 512u + 256u * (kb & 1) + 16u * r;
    uint32_t xo[MT], xso[MT];
#pragma unroll
    for (int m = 0; m < MT; m++) {
        const int i = 16 * m + r;
        uint32_t row = (uint32_t)(t.row0 + i);
        if (GROUPED && a.rows)
            row = i < t.rows ? (uint32_t)a.rows[t.row0 + i] : ~0u;
        const bool in = i < t.rows && row < (uint32_t)a.T;
        xo[m] = in ? row * xrow + 16u * kb : kOutOfRange;
        xso[m] = in ? row * 16u : kOutOfRange;
    }

    f4_t acc[MT][NB];
#pragma unroll
    for (int m = 0; m < MT; m++)
#pragma unroll
        for (int n = 0; n < NB; n++)
            acc[m][n] = f4_t{0.f, 0.f, 0.f, 0.f};

    Stage<XT, MT, NB> st[DEPTH];
    auto load = [&](Stage<XT, MT, NB> &s, int kt) __attribute__((always_inline)) {
        const bool in = kt < a.KT;      // (past the last tile: zeros)
#pragma unroll
        for (int n = 0; n < NB; n++) {
            const bool here = in && nt0 + n < a.NT;
            s.w[n] = load16(rw, here ? wo : kOutOfRange, here ? (uint32_t)(2 * kt * a.NT + nt0 + n) * 512u : 0u);
            s.ws[n] = load4(rs, here ? 16u * r : kOutOfRange,
                            here ? (uint32_t)((kt >> 2) * a.NT + nt0 + n) * 256u + 4u * (kt & 3) : 0u);
        }
#pragma unroll
        for (int m = 0; m < MT; m++) {
            if constexpr (FP4) {
                s.x[m][0] = load16(rx, in ? xo[m] : kOutOfRange, in ? (uint32_t)(kt >> 1) * (uint32_t)a.T * 128u + 64u * (kt & 1) : 0u);
                s.xs[m] = load4(rxs, in ? xso[m] : kOutOfRange,
                                in ? (uint32_t)(kt >> 2) * (uint32_t)a.T * 16u + 4u * (kt & 3) : 0u);
            } else {
#pragma unroll
                for (int j = 0; j < 4; j++)
                    s.x[m][j] = load16(rx, kt * 128 + 32 * j + 8 * kb < a.K ? xo[m] : kOutOfRange,
                                       in ? 256u * kt + 64u * j : 0u);
            }
        }
    };
    auto compute = [&](const Stage<XT, MT, NB> &s) __attribute__((always_inline)) {
        if constexpr (FP4) {
            uint32_t xs[MT];
#pragma unroll
            for (int m = 0; m < MT; m++)
                xs[m] = s.xs[m] >> (8 * kb);
#pragma unroll
            for (int n = 0; n < NB; n++) {
                const uint32_t ws = s.ws[n] >> (8 * kb);
#pragma unroll
                for (int m = 0; m < MT; m++)
                    acc[m][n] = mx_mfma16(s.w[n], s.x[m][0], acc[m][n], ws, xs[m]);
            }
        } else {
#pragma unroll
            for (int n = 0; n < NB; n++) {
                const u4_t words = transpose_words(s.w[n]);
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const u4_t w = mx_decode<XT == MX_X_BF16>(words[j], mx_scale(s.ws[n], j));
#pragma unroll
                    for (int m = 0; m < MT; m++) {
                        if constexpr (XT == MX_X_BF16)
                            acc[m][n] = mfma16x16x32_bf16(__builtin_bit_cast(bf8_t, w),
                                                          __builtin_bit_cast(bf8_t, s.x[m][j]), acc[m][n]);
                        else
                            acc[m][n] = mfma16x16x32(__builtin_bit_cast(h8_t, w),
                                                     __builtin_bit_cast(h8_t, s.x[m][j]), acc[m][n]);
                    }
                }
            }
        }
    };
#pragma unroll
    for (int d = 0; d < DEPTH; d++)
        load(st[d], ks + d * KS);
    for (int kt = ks; kt < a.KT; kt += DEPTH * KS) {
#pragma unroll
        for (int d = 0; d < DEPTH; d++) {
            compute(st[d]);
            load(st[d], kt + (DEPTH + d) * KS);
        }
    }

    // the waves' sums, added in their order; tile (m, n) by wave (m NB + n) mod KS
    const auto store = [&](int m, int n, f4_t v) __attribute__((always_inline)) {
        if (16 * m + r < t.rows)
            mx_store4((uint16_t *)a.Y + (int64_t)(t.row0 + 16 * m + r) * a.N, (nt0 + n) * 16 + 4 * kb, a.N,
                      FP4 ? ybf : XT == MX_X_BF16, v[0], v[1], v[2], v[3]);
    };
    if constexpr (KS > 1) {
        // (NP column tiles a pass)
#pragma unroll
        for (int n0 = 0; n0 < NB; n0 += NP) {
            if (n0)
                __syncthreads();
#pragma unroll
            for (int m = 0; m < MT; m++)
#pragma unroll
                for (int n = n0; n < n0 + NP && n < NB; n++)
                    sums[((nw * MT * NP + m * NP + n - n0) * KS + ks) * 64 + lane] = acc[m][n];
            __syncthreads();
#pragma unroll
            for (int m = 0; m < MT; m++)
#pragma unroll
                for (int n = n0; n < n0 + NP && n < NB; n++)
                    if ((m * NP + n - n0) % KS == ks) {
                        const f4_t *from = &sums[(nw * MT * NP + m * NP + n - n0) * KS * 64 + lane];
                        f4_t v = from[0];
#pragma unroll
                        for (int k = 1; k < KS; k++)
                            v += from[64 * k];
                        store(m, n, v);
                    }
        }
    } else {
#pragma unroll
        for (int m = 0; m < MT; m++)
#pragma unroll
            for (int n = 0; n < NB; n++)
                store(m, n, acc[m][n]);
    }
}

template <int XT, int MT, int NB, int WAVES, int KS, int DEPTH, bool GROUPED>
int launch_inst(const MxArgs &a, bool ybf, hipStream_t st) {
    constexpr int cols = NB * (WAVES / KS);
    const int64_t blocks = (a.NT + cols - 1) / cols;
    // sum over the matrices with rows of ceil(rows / (16 MT)), at most
    const int64_t used = a.R < a.E ? a.R : a.E;
    const int64_t tiles = GROUPED ? used + (a.R - used) / (16 * MT) : (a.R + 16 * MT - 1) / (16 * MT);
    if (tiles * blocks * WAVES * 64 >= (int64_t(1) << 32))
        return (int)hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((mx_small_kernel<XT, MT, NB, WAVES, KS, DEPTH, GROUPED>),
                       dim3((unsigned)(tiles * blocks)), dim3(WAVES * 64), 0, st, a, (int)blocks, ybf);
    return (int)hipGetLastError();
}

template <int XT, int MT, int NB, int DEPTH>
int launch_ks(const MxArgs &a, const MxPlan &p, bool ybf, hipStream_t st) {
    if constexpr (MT == 1)      // (plan_mx: one row tile for matrices of few rows each)
        if (a.offsets)
            switch (p.ks) {
            case 1: return launch_inst<XT, MT, NB, 4, 1, DEPTH, true>(a, ybf, st);
            case 2: return launch_inst<XT, MT, NB, 4, 2, DEPTH, true>(a, ybf, st);
            case 4: return launch_inst<XT, MT, NB, 4, 4, DEPTH, true>(a, ybf, st);
            default: return launch_inst<XT, MT, NB, 8, 8, DEPTH, true>(a, ybf, st);
            }
    switch (p.ks) {
    case 1: return launch_inst<XT, MT, NB, 4, 1, DEPTH, false>(a, ybf, st);
    case 2: return launch_inst<XT, MT, NB, 4, 2, DEPTH, false>(a, ybf, st);
    case 4: return launch_inst<XT, MT, NB, 4, 4, DEPTH, false>(a, ybf, st);
    default: return launch_inst<XT, MT, NB, 8, 8, DEPTH, false>(a, ybf, st);
    }
}

template <int XT>
int launch_mt(const MxArgs &a, const MxPlan &p, bool ybf, hipStream_t st) {
    constexpr bool FP4 = XT == MX_X_FP4;
    if (p.mt == 2)
        switch (p.nb) {
        case 1: return launch_ks<XT, 2, 1, 4>(a, p, ybf, st);
        case 2: return launch_ks<XT, 2, 2, FP4 ? 4 : 3>(a, p, ybf, st);
        default: return launch_ks<XT, 2, 3, FP4 ? 4 : 3>(a, p, ybf, st);
        }
    switch (p.nb) {
    case 1: return launch_ks<XT, 1, 1, 4>(a, p, ybf, st);
    case 2: return launch_ks<XT, 1, 2, 4>(a, p, ybf, st);
    case 3: return launch_ks<XT, 1, 3, 4>(a, p, ybf, st);
    default: return launch_ks<XT, 1, 4, FP4 ? 4 : 3>(a, p, ybf, st);
    }
}

}  // namespace

int launch_mx_small(const MxArgs &a, const MxPlan &p, int x, bool ybf, void *stream) {
    hipStream_t st = (hipStream_t)stream;
    if (x == MX_X_F16)
        return launch_mt<MX_X_F16>(a, p, ybf, st);
    if (x == MX_X_BF16)
        return launch_mt<MX_X_BF16>(a, p, ybf, st);
    return launch_mt<MX_X_FP4>(a, p, ybf, st);
}

}  // namespace w4a16

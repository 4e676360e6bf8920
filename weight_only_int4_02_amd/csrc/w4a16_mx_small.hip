// Products with MXFP4 weights for few rows (memory-bound).
//
// A workgroup takes NB column tiles of 16 and MT row tiles of 16, its KS waves
// (or, of one wave along K, four workgroups' worth of columns side by side)
// each every KS-th 128-column tile of K.  A weight tile is one 16-byte load a
// lane, straight into the operand registers: the device layout is the lanes'
// order, block 4 of a row in lanes 16 b + r.  The weights are the first operand, so a lane
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

// One 128-column tile's operands of a wave.
template <int XT, int MT, int NB>
struct Stage {
    u4_t w[NB], x[MT][XT == MX_X_FP4 ? 1 : 4];
    uint32_t ws[NB], xs[MT];
};

// WAVES: of the workgroup; KS of them along K, the others on further columns.
template <int XT, bool YBF, int MT, int NB, int WAVES, int KS, int DEPTH, bool GROUPED>
__global__ __launch_bounds__(WAVES * 64) void mx_small_kernel(MxArgs a, int blocks_n) {
    constexpr bool FP4 = XT == MX_X_FP4;
    constexpr int NW = WAVES / KS;
    __shared__ f4_t sums[KS > 1 ? WAVES * MT * NB * 64 : 1];
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
    const uint32_t xrow = FP4 ? (uint32_t)a.KT * 64u : (uint32_t)a.K * 2u;
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.X, (uint32_t)(a.T * xrow));
    const __amdgpu_buffer_rsrc_t rxs = make_rsrc(a.xs, FP4 ? (uint32_t)(a.T * a.KT * 4) : 0u);
    uint32_t xo[MT], xso[MT];
#pragma unroll
    for (int m = 0; m < MT; m++) {
        const int i = 16 * m + r;
        uint32_t row = (uint32_t)(t.row0 + i);
        if (GROUPED && a.rows)
            row = i < t.rows ? (uint32_t)a.rows[t.row0 + i] : ~0u;
        const bool in = i < t.rows && row < (uint32_t)a.T;
        xo[m] = in ? row * xrow + (FP4 ? 16u * kb : 64u * kb) : kOutOfRange;
        xso[m] = in ? row * (uint32_t)a.KT * 4u : kOutOfRange;
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
            s.w[n] = load16(rw, here ? 16u * lane : kOutOfRange, here ? (uint32_t)((nt0 + n) * a.KT + kt) * 1024u : 0u);
            s.ws[n] = load4(rs, here ? 16u * r : kOutOfRange,
                            here ? (uint32_t)((nt0 + n) * a.KG + (kt >> 2)) * 256u + 4u * (kt & 3) : 0u);
        }
#pragma unroll
        for (int m = 0; m < MT; m++) {
            if constexpr (FP4) {
                s.x[m][0] = load16(rx, in ? xo[m] : kOutOfRange, in ? 64u * kt : 0u);
                s.xs[m] = load4(rxs, in ? xso[m] : kOutOfRange, in ? 4u * kt : 0u);
            } else {
#pragma unroll
                for (int j = 0; j < 4; j++)
                    s.x[m][j] = load16(rx, kt * 128 + 32 * kb + 8 * j < a.K ? xo[m] : kOutOfRange,
                                       in ? 256u * kt + 16u * j : 0u);
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
                const float ws = mx_scale(s.ws[n], kb);
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const u4_t w = mx_decode<XT == MX_X_BF16>(s.w[n][j], ws);
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
            mx_store4<YBF>((uint16_t *)a.Y + (int64_t)(t.row0 + 16 * m + r) * a.N, (nt0 + n) * 16 + 4 * kb,
                           a.N, v[0], v[1], v[2], v[3]);
    };
    if constexpr (KS > 1) {
#pragma unroll
        for (int m = 0; m < MT; m++)
#pragma unroll
            for (int n = 0; n < NB; n++)
                sums[((nw * MT * NB + m * NB + n) * KS + ks) * 64 + lane] = acc[m][n];
        __syncthreads();
#pragma unroll
        for (int m = 0; m < MT; m++)
#pragma unroll
            for (int n = 0; n < NB; n++)
                if ((m * NB + n) % KS == ks) {
                    f4_t v = sums[((nw * MT * NB + m * NB + n) * KS) * 64 + lane];
#pragma unroll
                    for (int k = 1; k < KS; k++)
                        v += sums[((nw * MT * NB + m * NB + n) * KS + k) * 64 + lane];
                    store(m, n, v);
                }
    } else {
#pragma unroll
        for (int m = 0; m < MT; m++)
#pragma unroll
            for (int n = 0; n < NB; n++)
                store(m, n, acc[m][n]);
    }
}

template <int XT, bool YBF, int MT, int NB, int WAVES, int KS, bool GROUPED>
int launch_inst(const MxArgs &a, hipStream_t st) {
    constexpr int cols = NB * (WAVES / KS), DEPTH = MT == 4 && XT != MX_X_FP4 ? 2 : 4;
    const int64_t blocks = (a.NT + cols - 1) / cols;
    // sum over the matrices with rows of ceil(rows / (16 MT)), at most
    const int64_t used = a.R < a.E ? a.R : a.E;
    const int64_t tiles = GROUPED ? used + (a.R - used) / (16 * MT) : (a.R + 16 * MT - 1) / (16 * MT);
    if (tiles * blocks * WAVES * 64 >= (int64_t(1) << 32))
        return (int)hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((mx_small_kernel<XT, YBF, MT, NB, WAVES, KS, DEPTH, GROUPED>),
                       dim3((unsigned)(tiles * blocks)), dim3(WAVES * 64), 0, st, a, (int)blocks);
    return (int)hipGetLastError();
}

template <int XT, bool YBF, int MT, int NB>
int launch_ks(const MxArgs &a, const MxPlan &p, hipStream_t st) {
    if (a.offsets) {
        switch (p.ks) {
        case 1: return launch_inst<XT, YBF, MT, NB, 4, 1, true>(a, st);
        case 2: return launch_inst<XT, YBF, MT, NB, 4, 2, true>(a, st);
        case 4: return launch_inst<XT, YBF, MT, NB, 4, 4, true>(a, st);
        default: return launch_inst<XT, YBF, MT, NB, 8, 8, true>(a, st);
        }
    }
    switch (p.ks) {
    case 1: return launch_inst<XT, YBF, MT, NB, 4, 1, false>(a, st);
    case 2: return launch_inst<XT, YBF, MT, NB, 4, 2, false>(a, st);
    case 4: return launch_inst<XT, YBF, MT, NB, 4, 4, false>(a, st);
    default: return launch_inst<XT, YBF, MT, NB, 8, 8, false>(a, st);
    }
}

template <int XT, bool YBF>
int launch_mt(const MxArgs &a, const MxPlan &p, hipStream_t st) {
    switch (p.mt) {
    case 1: return launch_ks<XT, YBF, 1, 1>(a, p, st);
    case 2: return launch_ks<XT, YBF, 2, 2>(a, p, st);
    default: return launch_ks<XT, YBF, 4, 2>(a, p, st);
    }
}

}  // namespace

int launch_mx_small(const MxArgs &a, const MxPlan &p, int x, bool ybf, void *stream) {
    hipStream_t st = (hipStream_t)stream;
    if (x == MX_X_F16)
        return launch_mt<MX_X_F16, false>(a, p, st);
    if (x == MX_X_BF16)
        return launch_mt<MX_X_BF16, true>(a, p, st);
    return ybf ? launch_mt<MX_X_FP4, true>(a, p, st) : launch_mt<MX_X_FP4, false>(a, p, st);
}

}  // namespace w4a16

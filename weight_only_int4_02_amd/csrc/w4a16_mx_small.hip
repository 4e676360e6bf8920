// Products with MXFP4 weights for few rows (memory-bound).
//
// A workgroup takes MT row tiles of 16 and, for each of its WAVES / KS groups of
// KS waves, NB column tiles of 16; the waves of a group take every KS-th tile of
// 128 columns of K each, and their sums are added through LDS at the end.  A weight
// tile is one 16-byte load a lane, straight into the operand registers (block b
// of row r in lane 16 b + r).  The weights are the first operand, so that a lane
// holds four neighbouring columns of one row's results.
//
// Activations go through LDS: a wave copies its tiles' rows into a ring of its own
// by buffer-to-LDS DMA, whole runs of a row at a time, and reads the operands from
// there (loaded straight into operand registers, a lane's 16 bytes lie a row away
// from its neighbours' and are a request of their own: 32 x 12288 x 4096 in bf16
// took 16.4 us so, of which 5.8 were those loads; now 10.2).  A row's blocks of
// 16 bytes stand in an order that gives the lanes of a read (one block of 16 rows)
// different banks.  No wave waits for another before the sums.
//
// With 16-bit activations, a lane's four code words are exchanged with those of the
// other three lane groups, so that word j of lane 16 i + r holds columns 32 j + 8 i
// .. + 7 of row r: the order in which a matrix instruction takes K from two
// operands of 16 x 32 values, and in which a row of X is one run of 64 bytes.
//
// All loads are untracked (see load_b128_so): a stage is waited for by counting.
//
// Bound by the weights' bytes where there are many: two experts of 22016 x 4096, one
// row each, 20.5 us (4.7 TB/s), 64 of 2048 x 1408, 1.5 rows each, 15.5 (5.0).  Below
// that launch and latency count: 4096 x 4096, one row, 5.3 (1.7), 12288 x 4096, 32 rows,
// 10.2 (2.6), whose workgroups read 67 MB of activations out of L2 beside 27 of weights.
// LDS is busy 0.05 .. 0.08 of the time, without bank conflicts, the matrix cores
// 0.05 .. 0.14.
#include <hip/hip_runtime.h>

#include "w4a16_mx_device.hpp"

namespace w4a16 {

namespace {

// Words j of the four lane groups become group j's four words: in lanes 16 i + r
// word j is then word i of block j.
__device__ __forceinline__ u4_t transpose_words(u4_t w) {
    const auto a = __builtin_amdgcn_permlane16_swap(w.x, w.y, false, false);
    const auto b = __builtin_amdgcn_permlane16_swap(w.z, w.w, false, false);
    const auto c = __builtin_amdgcn_permlane32_swap(a[0], b[0], false, false);
    const auto d = __builtin_amdgcn_permlane32_swap(a[1], b[1], false, false);
    return u4_t{c[0], d[0], c[1], d[1]};
}

// load_b128_so and load_u32_so with the five wait states that they need after a
// vector instruction wrote one of their scalar registers (a spilled one's reload).
__device__ __forceinline__ u4_t load16_nops(i4_t desc, uint32_t voffset, uint32_t soffset) {
    u4_t v;
    asm volatile("s_nop 4\n\tbuffer_load_dwordx4 %0, %1, %2, %3 offen"
                 : "=v"(v) : "v"(voffset), "s"(desc), "s"(soffset));
    return v;
}
__device__ __forceinline__ uint32_t load4_nops(i4_t desc, uint32_t voffset, uint32_t soffset) {
    uint32_t v;
    asm volatile("s_nop 4\n\tbuffer_load_dword %0, %1, %2, %3 offen"
                 : "=v"(v) : "v"(voffset), "s"(desc), "s"(soffset));
    return v;
}

template <int XT, int MT, int NB, int WAVES, int KS, int DEPTH, bool GROUPED>
__global__ __launch_bounds__(WAVES * 64) void mx_small_kernel(MxArgs a, int blocks_n, bool ybf) {
    constexpr bool FP4 = XT == MX_X_FP4;
    constexpr int XROW = FP4 ? 64 : 256, XC = FP4 ? 1 : 4;   // copies of 1 KiB a row tile
    constexpr int LPS = NB * 2 + MT * (FP4 ? 2 : XC);        // loads of a stage
    static_assert((DEPTH - 1) * LPS < 64, "counted by vmcnt");
    constexpr int SLOT = MT * XC * 1024;
    // column tiles summed at a time (in at most 64 KiB)
    constexpr int NP = WAVES * MT * NB <= 64 ? NB : 64 / (WAVES * MT);
    constexpr int RING = WAVES * DEPTH * SLOT, SUMS = KS > 1 ? WAVES * MT * NP * 1024 : 0;
    __shared__ __attribute__((aligned(1024))) char lds[RING > SUMS ? RING : SUMS];
    const int lane = threadIdx.x & 63, r = lane & 15, kb = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int ks = wave % KS, nw = wave / KS;

    const int tile = blockIdx.x / blocks_n, block = blockIdx.x - tile * blocks_n;
    MxTile t;
    if constexpr (GROUPED) {
        t = mx_find_tile<16 * MT>(a, (uint32_t)tile, lane);
        if (t.count == 0)
            return;
    } else {
        t = MxTile{0, 0, (int)a.R, 1};
        t.take(tile, 16 * MT);
    }
    const int nt0 = (block * (WAVES / KS) + nw) * NB;

    const uint32_t wbytes = (uint32_t)a.NT * (uint32_t)a.KT * 1024u, sbytes = (uint32_t)a.NT * (uint32_t)a.KG * 256u;
    const i4_t dw = make_desc((const char *)a.qd + (int64_t)t.e * wbytes, wbytes);
    const i4_t ds = make_desc((const char *)a.sd + (int64_t)t.e * sbytes, sbytes);
    const i4_t dx = make_desc(a.X, (uint32_t)(a.T * (FP4 ? a.KG * 256 : a.K * 2)));
    const i4_t dxs = make_desc(a.xs, FP4 ? (uint32_t)(a.T * a.KG * 16) : 0u);
    // the lane's part of the offsets: weights and scales of each column tile (past
    // the last one: nothing), activations of each copy
    const uint32_t wo = (uint32_t)(kb >> 1) * (uint32_t)a.NT * 512u + 256u * (kb & 1) + 16u * r;
    auto source_row = [&](int i) __attribute__((always_inline)) {
        uint32_t row = (uint32_t)t.row0 + (uint32_t)i;
        if (GROUPED && a.rows)
            row = i < t.rows ? (uint32_t)a.rows[t.row0 + i] : ~0u;
        return i < t.rows && row < (uint32_t)a.T ? row : ~0u;
    };
    uint32_t xo[MT][XC], xcol[XC], xso[MT];
#pragma unroll
    for (int c = 0; c < XC; c++) {
        const int row = FP4 ? lane / 4 : 4 * c + lane / 16;      // of the tile
        const uint32_t b = FP4 ? (uint32_t)(lane % 4) ^ ((row >> 1) & 3) ^ ((row >> 3) & 1) : (uint32_t)(lane % 16 ^ row);
        xcol[c] = 8 * b;
#pragma unroll
        for (int m = 0; m < MT; m++) {
            const uint32_t i = source_row(16 * m + row);
            xo[m][c] = i != ~0u ? i * (FP4 ? 64u : (uint32_t)a.K * 2u) + 16u * b : kOutOfRange;
        }
    }
#pragma unroll
    for (int m = 0; m < MT; m++) {
        const uint32_t i = FP4 ? source_row(16 * m + r) : ~0u;
        xso[m] = i != ~0u ? i * 16u : kOutOfRange;
    }

    const uint32_t ring = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)lds + (uint32_t)(wave * DEPTH * SLOT);
    const char *const mine = lds + wave * DEPTH * SLOT;
    struct {
        u4_t w[NB];
        uint32_t ws[NB], xs[MT];
    } st[DEPTH];
    auto load = [&](int d, int kt) __attribute__((always_inline)) {
        const bool in = kt < a.KT;      // (past the last tile: zeros)
#pragma unroll
        for (int m = 0; m < MT; m++) {
#pragma unroll
            for (int c = 0; c < XC; c++)
                copy16(dx, ring + (uint32_t)(d * SLOT + (m * XC + c) * 1024),
                       in && (FP4 || (int)xcol[c] < a.K - kt * 128) ? xo[m][c] : kOutOfRange,
                       !in ? 0u : FP4 ? (uint32_t)kt * (uint32_t)a.T * 64u : 256u * kt);
            if constexpr (FP4)
                st[d].xs[m] = load4_nops(dxs, in ? xso[m] : kOutOfRange,
                                             in ? (uint32_t)(kt >> 2) * (uint32_t)a.T * 16u + 4u * (kt & 3) : 0u);
        }
#pragma unroll
        for (int n = 0; n < NB; n++) {
            const bool here = in && nt0 + n < a.NT;
            st[d].w[n] = load16_nops(dw, here ? wo : kOutOfRange,
                                         here ? (uint32_t)(2 * kt * a.NT + nt0 + n) * 512u : 0u);
            st[d].ws[n] = load4_nops(ds, here ? 16u * r : kOutOfRange,
                                         here ? (uint32_t)((kt >> 2) * a.NT + nt0 + n) * 256u + 4u * (kt & 3) : 0u);
        }
    };
    auto fence = [&](int d) __attribute__((always_inline)) {
#pragma unroll
        for (int n = 0; n < NB; n++) {
            reg_fence(st[d].w[n]);
            reg_fence(st[d].ws[n]);
        }
        if constexpr (FP4)
#pragma unroll
            for (int m = 0; m < MT; m++)
                reg_fence(st[d].xs[m]);
    };
    f4_t acc[MT][NB];
#pragma unroll
    for (int m = 0; m < MT; m++)
#pragma unroll
        for (int n = 0; n < NB; n++)
            acc[m][n] = f4_t{0.f, 0.f, 0.f, 0.f};
    auto compute = [&](int d) __attribute__((always_inline)) {
        const char *x = mine + d * SLOT + r * XROW;
        if constexpr (FP4) {
            u4_t xa[MT];
            uint32_t xs[MT];
#pragma unroll
            for (int m = 0; m < MT; m++) {
                xa[m] = *(const u4_t *)(x + m * 1024 + 16 * (kb ^ ((r >> 1) & 3) ^ ((r >> 3) & 1)));
                xs[m] = st[d].xs[m] >> (8 * kb);
            }
#pragma unroll
            for (int n = 0; n < NB; n++) {
                const uint32_t ws = st[d].ws[n] >> (8 * kb);
#pragma unroll
                for (int m = 0; m < MT; m++)
                    acc[m][n] = mx_mfma16(st[d].w[n], xa[m], acc[m][n], ws, xs[m]);
            }
        } else {
            u4_t xa[MT][4];
#pragma unroll
            for (int m = 0; m < MT; m++)
#pragma unroll
                for (int j = 0; j < 4; j++)
                    xa[m][j] = *(const u4_t *)(x + m * 4096 + 16 * ((4 * j + kb) ^ r));
#pragma unroll
            for (int n = 0; n < NB; n++) {
                const u4_t words = transpose_words(st[d].w[n]);
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const u4_t w = mx_decode<XT == MX_X_BF16>(words[j], mx_scale(st[d].ws[n], j));
#pragma unroll
                    for (int m = 0; m < MT; m++) {
                        if constexpr (XT == MX_X_BF16)
                            acc[m][n] = mfma16x16x32_bf16(__builtin_bit_cast(bf8_t, w),
                                                          __builtin_bit_cast(bf8_t, xa[m][j]), acc[m][n]);
                        else
                            acc[m][n] = mfma16x16x32(__builtin_bit_cast(h8_t, w), __builtin_bit_cast(h8_t, xa[m][j]),
                                                     acc[m][n]);
                    }
                }
            }
        }
    };
#pragma unroll
    for (int d = 0; d < DEPTH; d++)
        load(d, ks + d * KS);
    for (int kt = ks; kt < a.KT; kt += DEPTH * KS) {
#pragma unroll
        for (int d = 0; d < DEPTH; d++) {
            wait_vmcnt<(DEPTH - 1) * LPS>();
            fence(d);
            compute(d);
            // (its reads of the slot are done before the next copies there)
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            load(d, kt + (DEPTH + d) * KS);
        }
    }
    wait_vmcnt<0>();
#pragma unroll
    for (int d = 0; d < DEPTH; d++)
        fence(d);

    const auto store = [&](int m, int n, f4_t v) __attribute__((always_inline)) {
        if (16 * m + r < t.rows)
            mx_store4((uint16_t *)a.Y + (int64_t)(t.row0 + 16 * m + r) * a.N, (nt0 + n) * 16 + 4 * kb, a.N,
                      FP4 ? ybf : XT == MX_X_BF16, v[0], v[1], v[2], v[3]);
    };
    if constexpr (KS == 1) {
#pragma unroll
        for (int m = 0; m < MT; m++)
#pragma unroll
            for (int n = 0; n < NB; n++)
                store(m, n, acc[m][n]);
        return;
    }
    // the waves' sums, added in their order; tile (m, n) by wave (m NP + n) mod KS
    f4_t *const sums = (f4_t *)lds + nw * MT * NP * KS * 64;
#pragma unroll
    for (int n0 = 0; n0 < NB; n0 += NP) {
        __syncthreads();       // (the rings, then the pass before, are used up)
#pragma unroll
        for (int m = 0; m < MT; m++)
#pragma unroll
            for (int n = n0; n < n0 + NP && n < NB; n++)
                sums[((m * NP + n - n0) * KS + ks) * 64 + lane] = acc[m][n];
        __syncthreads();
#pragma unroll
        for (int m = 0; m < MT; m++)
#pragma unroll
            for (int n = n0; n < n0 + NP && n < NB; n++)
                if ((m * NP + n - n0) % KS == ks) {
                    const f4_t *from = &sums[(m * NP + n - n0) * KS * 64 + lane];
                    f4_t v = from[0];
#pragma unroll
                    for (int k = 1; k < KS; k++)
                        v += from[64 * k];
                    store(m, n, v);
                }
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

// Stages of the rings: few where that lets more workgroups share a compute unit
// (64 experts of 2048 x 1408, 16 tokens in bf16, four stages 20.5 us, two 18.8), as
// many as LDS holds where one fills it.  The forms are those that plan_mx has.
template <int XT, int NB>
int launch_plain(const MxArgs &a, const MxPlan &p, bool ybf, hipStream_t st) {
    constexpr bool FP4 = XT == MX_X_FP4;
    if (p.mt == 1) {
        if constexpr (NB == 1)
            if (p.ks == 8)
                return launch_inst<XT, 1, 1, 8, 8, 2, false>(a, ybf, st);
        return launch_inst<XT, 1, NB, 4, 4, 2, false>(a, ybf, st);
    }
    if (p.mt == 2) {
        if constexpr (!FP4 || NB == 1)
            if (p.ks == 8)
                return launch_inst<XT, 2, NB, 8, 8, FP4 ? 4 : 2, false>(a, ybf, st);
        if constexpr (FP4)
            return launch_inst<XT, 2, NB, 4, 4, 4, false>(a, ybf, st);
    }
    return p.mt == 3 ? launch_inst<XT, 3, NB, 4, 4, FP4 ? 3 : 2, false>(a, ybf, st)
                     : launch_inst<XT, 4, NB, 4, 4, FP4 ? 3 : 2, false>(a, ybf, st);
}

template <int XT>
int launch_mt(const MxArgs &a, const MxPlan &p, bool ybf, hipStream_t st) {
    if (a.offsets) {
        if constexpr (XT != MX_X_FP4)
            if (p.mt == 2)
                return launch_inst<XT, 2, 4, 4, 2, 4, true>(a, ybf, st);
        return p.ks == 1   ? launch_inst<XT, 1, 4, 4, 1, 2, true>(a, ybf, st)
               : p.ks == 2 ? launch_inst<XT, 1, 4, 4, 2, 2, true>(a, ybf, st)
                           : launch_inst<XT, 1, 4, 4, 4, 2, true>(a, ybf, st);
    }
    return p.nb == 1   ? launch_plain<XT, 1>(a, p, ybf, st)
           : p.nb == 2 ? launch_plain<XT, 2>(a, p, ybf, st)
                       : launch_plain<XT, 3>(a, p, ybf, st);
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

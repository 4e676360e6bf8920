// Products with MXFP4 weights for many rows (compute-bound).
//
// A workgroup's waves form a BM x BN tile of Y, WM x WN of it each, from stages
// of K in a ring in LDS (128 columns of MXFP4 activations, 64 of 16-bit ones: 64
// and 128 bytes of a row).  Every wave copies its share of a stage by
// buffer-to-LDS DMA, NBUF - 1 stages ahead of the products; the copies are inline
// assembly that the compiler does not count, so that it never waits for one by
// itself.  A stage holds the activation rows (gathered, if an index is given: a
// lane of a copy has its own address), the weights' 16 x 128 tiles as they lie,
// and the scale words of both.
//
// Matrix instructions of 32 x 32, the weights first, so that a lane ends with
// four neighbouring columns of one row.  A lane's operand is 16 bytes, one block of
// 32 codes of one row: as MXFP4 it enters one 32 x 32 x 64 instruction with its
// scale; beside 16-bit activations its four words are decoded (one conversion
// a pair, the scale with it) for four 32 x 32 x 16 instructions, whose columns of
// K are the same eight for both operands.
//
// LDS: the weights' 16-byte blocks lie in the order in which lanes read them.  A
// row of activations is 4 (or 8) blocks of 16 bytes, stored at the block's number
// XOR a function of the row, so that the lanes of a read (one block of
// consecutive rows) reach all banks.
#include <hip/hip_runtime.h>

#include "w4a16_mx_device.hpp"

namespace w4a16 {

namespace {

constexpr int kXcds = 8;  // MI355X: 8 XCDs, workgroups dealt round-robin

// Copies 16 (4) bytes a lane to LDS at lds + 16 (4) lane; lds is the same in
// all lanes.  Out of range: zeros.  (M0, which the compiler uses for nothing else
// in these kernels, holds the address.)
__device__ __forceinline__ void copy16(i4_t desc, uint32_t lds, uint32_t voffset, uint32_t soffset) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :: "s"(lds), "v"(voffset), "s"(desc), "s"(soffset) : "memory");
}
__device__ __forceinline__ void copy4(i4_t desc, uint32_t lds, uint32_t voffset, uint32_t soffset) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds"
                 :: "s"(lds), "v"(voffset), "s"(desc), "s"(soffset) : "memory");
}

// Every wave's reads of the stage before are done, and its copies of this one.
template <int N>
__device__ __forceinline__ void stage_ready() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// Where block `b` of row `row` stands among the row's 4 or 8: any 8 or 16
// consecutive rows' blocks of one number lie in different banks.
template <bool FP4>
__device__ __forceinline__ uint32_t swizzle(uint32_t row, uint32_t b) {
    return FP4 ? b ^ ((row >> 1) & 3) ^ ((row >> 3) & 1) : b ^ (row & 7) ^ ((row >> 3) & 1);
}

template <int XT, bool YBF, int BM, int BN, int WM, int WN, int NBUF, int OCC, bool GROUPED>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * 64, OCC * (BM / WM) * (BN / WN) / 4)
void mx_large_kernel(MxArgs a, int blocks_n) {
    constexpr bool FP4 = XT == MX_X_FP4;
    constexpr int WAVES_M = BM / WM, WAVES = WAVES_M * (BN / WN);
    constexpr int TM = WM / 32, TN = WN / 32;
    constexpr int XROW = FP4 ? 64 : 128;             // bytes of a stage's row
    constexpr int XCH = BM * XROW / 1024;            // copies of a stage: activations,
    constexpr int WCH = BN * (FP4 ? 64 : 32) / 1024; // weights,
    constexpr int SW = BN / 64, SX = FP4 ? BM / 64 : 0;   // scale words
    static_assert(XCH % WAVES == 0 && WCH % WAVES == 0, "copies split evenly over the waves");
    constexpr int KX = XCH / WAVES, KW = WCH / WAVES, KSC = (SW + SX + WAVES - 1) / WAVES;
    constexpr int CPW = KX + KW + KSC;               // copies of a wave and stage
    static_assert((NBUF - 1) * CPW < 64, "counted by vmcnt");
    constexpr int STAGE = (XCH + WCH) * 1024 + KSC * WAVES * 256;
    __shared__ __attribute__((aligned(1024))) char lds[NBUF * STAGE];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave % WAVES_M, wn = wave / WAVES_M;
    const int h = lane >> 5, l32 = lane & 31;

    // this workgroup's tile: the XCDs take equal runs of them, column block by
    // column block of a matrix, its row tiles one after the other, so that
    // neighbours in time share the weights of a column block in their L2
    const uint32_t xcd = blockIdx.x % kXcds, at = blockIdx.x / kXcds;
    uint32_t tiles;
    if constexpr (GROUPED)
        tiles = (uint32_t)mx_count_tiles<BM>(a, lane);
    else
        tiles = (uint32_t)((a.R + BM - 1) / BM);
    const uint32_t items = tiles * (uint32_t)blocks_n;
    const uint32_t first = items / kXcds * xcd + min(items % kXcds, xcd);
    if (at >= items / kXcds + (items % kXcds > xcd ? 1 : 0))
        return;
    const uint32_t item = first + at;
    MxTile t;
    int nb;
    if constexpr (GROUPED) {
        const uint32_t any = item / (uint32_t)blocks_n;
        t = mx_find_tile<BM>(a, (int)any, lane);
        if (t.count == 0)
            return;
        // (within the matrix: column block, then row tile)
        const uint32_t within = item - (any - (uint32_t)t.mt) * (uint32_t)blocks_n;
        nb = (int)(within / (uint32_t)t.count);
        t.take((int)(within - (uint32_t)nb * (uint32_t)t.count), BM);
    } else {
        nb = (int)(item / tiles);
        t = MxTile{0, 0, (int)a.R, (int)tiles};
        t.take((int)(item - (uint32_t)nb * tiles), BM);
    }

    const uint32_t wbytes = (uint32_t)a.NT * (uint32_t)a.KT * 1024u, sbytes = (uint32_t)a.NT * (uint32_t)a.KG * 256u;
    const i4_t dw = make_desc((const char *)a.qd + (int64_t)t.e * wbytes, wbytes);
    const i4_t ds = make_desc((const char *)a.sd + (int64_t)t.e * sbytes, sbytes);
    const uint32_t xrow = FP4 ? (uint32_t)a.KT * 64u : (uint32_t)a.K * 2u;
    const i4_t dx = make_desc(a.X, (uint32_t)(a.T * xrow));
    const i4_t dxs = make_desc(a.xs, FP4 ? (uint32_t)(a.T * a.KT * 4) : 0u);

    // the copies' per-lane offsets
    auto source_row = [&](int i) __attribute__((always_inline)) {
        uint32_t row = (uint32_t)(t.row0 + i);
        if (GROUPED && a.rows)
            row = i < t.rows ? (uint32_t)a.rows[t.row0 + i] : ~0u;
        return i < t.rows && row < (uint32_t)a.T ? row : ~0u;
    };
    constexpr int RPC = 1024 / XROW;     // rows of an activation copy
    constexpr int LPR = 64 / RPC;        // and lanes of a row
    uint32_t xo[KX], xcol = 0, wo[KW], so[KSC];
#pragma unroll
    for (int k = 0; k < KX; k++) {
        const int i = (wave + k * WAVES) * RPC + lane / LPR;
        const uint32_t row = source_row(i), b = swizzle<FP4>((uint32_t)i, (uint32_t)(lane % LPR));
        xo[k] = row != ~0u ? row * xrow + 16u * b : kOutOfRange;
        // (8 columns a block of 16-bit activations; the same for every k: the
        // copies are 32 rows apart or more, and the order goes by the row's number below 16)
        static_assert(WAVES * RPC % 16 == 0, "a lane's copies have one order of blocks");
        xcol = 8u * b;
    }
    const int nt0 = nb * (BN / 16);
#pragma unroll
    for (int k = 0; k < KW; k++) {
        // FP4: one tile a copy; else the same half of two
        const int c = wave + k * WAVES;
        const int nt = nt0 + (FP4 ? c : 2 * c + (lane >> 5));
        wo[k] = nt < a.NT ? (uint32_t)nt * (uint32_t)a.KT * 1024u + 16u * (FP4 ? lane : lane & 31) : kOutOfRange;
    }
#pragma unroll
    for (int k = 0; k < KSC; k++) {
        // 64 columns' (or rows') words a copy
        const int c = wave + k * WAVES;
        const int nt = nt0 + 4 * c + (lane >> 4);
        so[k] = kOutOfRange;
        if (c < SW) {
            if (nt < a.NT)
                so[k] = (uint32_t)nt * (uint32_t)a.KG * 256u + 16u * (lane & 15);
        } else if (FP4 && c < SW + SX) {
            const uint32_t row = source_row((c - SW) * 64 + lane);
            if (row != ~0u)
                so[k] = row * (uint32_t)a.KT * 4u;
        }
    }
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)lds;
    const int stages = FP4 ? a.KT : (a.K + 63) / 64;
    auto issue = [&](int s, int buf) __attribute__((always_inline)) {
        const uint32_t to = lds0 + (uint32_t)(buf * STAGE);
        const int kt = FP4 ? s : s >> 1;
#pragma unroll
        for (int k = 0; k < KX; k++)
            copy16(dx, to + (uint32_t)(wave + k * WAVES) * 1024u,
                   FP4 || (int)xcol < a.K - s * 64 ? xo[k] : kOutOfRange, (uint32_t)(s * XROW));
#pragma unroll
        for (int k = 0; k < KW; k++)
            copy16(dw, to + (uint32_t)(XCH + wave + k * WAVES) * 1024u, wo[k],
                   (uint32_t)kt * 1024u + (FP4 ? 0u : 512u * (s & 1)));
#pragma unroll
        for (int k = 0; k < KSC; k++) {
            const int c = wave + k * WAVES;
            const uint32_t l = to + (uint32_t)(XCH + WCH) * 1024u + (uint32_t)c * 256u;
            if (!FP4 || c < SW)
                copy4(ds, l, so[k], (uint32_t)(kt >> 2) * 256u + 4u * (uint32_t)(kt & 3));
            else
                copy4(dxs, l, so[k], 4u * (uint32_t)kt);
        }
    };

    f16_t acc[TM][TN];
#pragma unroll
    for (int m = 0; m < TM; m++)
#pragma unroll
        for (int n = 0; n < TN; n++)
#pragma unroll
            for (int i = 0; i < 16; i++)
                acc[m][n][i] = 0.f;

    auto compute = [&](int s, int buf) __attribute__((always_inline)) {
        const char *st = lds + buf * STAGE;
        const char *x = st + (wm * WM + l32) * XROW;
        const char *w = st + XCH * 1024 + (wn * (WN / 16) + (l32 >> 4)) * (FP4 ? 1024 : 512) + h * 256 + (l32 & 15) * 16;
        const uint32_t *sw = (const uint32_t *)(st + (XCH + WCH) * 1024) + wn * WN + l32;
        const uint32_t *sx = (const uint32_t *)(st + (XCH + WCH) * 1024) + SW * 64 + wm * WM + l32;
        if constexpr (FP4) {
            uint32_t xs[TM], ws[TN];
#pragma unroll
            for (int m = 0; m < TM; m++)
                xs[m] = sx[32 * m] >> (8 * h);
#pragma unroll
            for (int n = 0; n < TN; n++)
                ws[n] = sw[32 * n] >> (8 * h);
#pragma unroll
            for (int j = 0; j < 2; j++) {
                u4_t xa[TM], wa[TN];
#pragma unroll
                for (int m = 0; m < TM; m++)
                    xa[m] = *(const u4_t *)(x + m * 32 * XROW + 16 * swizzle<true>((uint32_t)l32, (uint32_t)(2 * j + h)));
#pragma unroll
                for (int n = 0; n < TN; n++)
                    wa[n] = *(const u4_t *)(w + n * 2048 + j * 512);
#pragma unroll
                for (int n = 0; n < TN; n++)
#pragma unroll
                    for (int m = 0; m < TM; m++)
                        acc[m][n] = j == 0 ? mx_mfma32<0>(wa[n], xa[m], acc[m][n], ws[n], xs[m])
                                           : mx_mfma32<2>(wa[n], xa[m], acc[m][n], ws[n], xs[m]);
            }
        } else {
            float ws[TN];
            u4_t wa[TN];
#pragma unroll
            for (int n = 0; n < TN; n++) {
                ws[n] = mx_scale(sw[32 * n], (uint32_t)(2 * (s & 1) + h));
                wa[n] = *(const u4_t *)(w + n * 1024);
            }
#pragma unroll
            for (int j = 0; j < 4; j++) {
                u4_t xa[TM];
#pragma unroll
                for (int m = 0; m < TM; m++)
                    xa[m] = *(const u4_t *)(x + m * 32 * XROW + 16 * swizzle<false>((uint32_t)l32, (uint32_t)(4 * h + j)));
#pragma unroll
                for (int n = 0; n < TN; n++) {
                    const u4_t v = mx_decode<XT == MX_X_BF16>(wa[n][j], ws[n]);
#pragma unroll
                    for (int m = 0; m < TM; m++) {
                        if constexpr (XT == MX_X_BF16)
                            acc[m][n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                                __builtin_bit_cast(bf8_t, v), __builtin_bit_cast(bf8_t, xa[m]), acc[m][n], 0, 0, 0);
                        else
                            acc[m][n] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
                                __builtin_bit_cast(h8_t, v), __builtin_bit_cast(h8_t, xa[m]), acc[m][n], 0, 0, 0);
                    }
                }
            }
        }
    };

#pragma unroll
    for (int s = 0; s < NBUF - 1; s++)
        if (s < stages)
            issue(s, s);
    int buf = 0;
    for (int s = 0; s < stages; s++) {
        // (copies of the NBUF - 2 stages after this one may be under way)
        if (s + NBUF - 2 < stages)
            stage_ready<(NBUF - 2) * CPW>();
        else
            stage_ready<0>();
        if (s + NBUF - 1 < stages)
            issue(s + NBUF - 1, buf == 0 ? NBUF - 1 : buf - 1);
        compute(s, buf);
        buf = buf + 1 < NBUF ? buf + 1 : 0;
    }

#pragma unroll
    for (int m = 0; m < TM; m++) {
        const int i = wm * WM + 32 * m + l32;
        if (i >= t.rows)
            continue;
        uint16_t *y = (uint16_t *)a.Y + (int64_t)(t.row0 + i) * a.N;
#pragma unroll
        for (int n = 0; n < TN; n++)
#pragma unroll
            for (int q = 0; q < 4; q++)
                mx_store4<YBF>(y, nb * BN + wn * WN + 32 * n + 8 * q + 4 * h, a.N, acc[m][n][4 * q],
                               acc[m][n][4 * q + 1], acc[m][n][4 * q + 2], acc[m][n][4 * q + 3]);
    }
}

template <int XT, bool YBF, int BM, int BN, int WM, int WN, int NBUF, int OCC>
int launch_inst(const MxArgs &a, hipStream_t st) {
    const int64_t blocks = (a.N + BN - 1) / BN;
    const int64_t used = a.R < a.E ? a.R : a.E;
    const int64_t tiles = a.offsets ? used + (a.R - used) / BM : (a.R + BM - 1) / BM;
    const int64_t grid = (tiles * blocks + kXcds - 1) / kXcds * kXcds;
    constexpr int threads = (BM / WM) * (BN / WN) * 64;
    if (grid * threads >= (int64_t(1) << 32))
        return (int)hipErrorInvalidConfiguration;
    if (a.offsets)
        hipLaunchKernelGGL((mx_large_kernel<XT, YBF, BM, BN, WM, WN, NBUF, OCC, true>), dim3((unsigned)grid),
                           dim3(threads), 0, st, a, (int)blocks);
    else
        hipLaunchKernelGGL((mx_large_kernel<XT, YBF, BM, BN, WM, WN, NBUF, OCC, false>), dim3((unsigned)grid),
                           dim3(threads), 0, st, a, (int)blocks);
    return (int)hipGetLastError();
}

template <int XT, bool YBF>
int launch_shape(const MxArgs &a, const MxPlan &p, hipStream_t st) {
    (void)p;
    return launch_inst<XT, YBF, 128, 256, 64, 128, 3, 2>(a, st);
}

}  // namespace

int launch_mx_large(const MxArgs &a, const MxPlan &p, int x, bool ybf, void *stream) {
    hipStream_t st = (hipStream_t)stream;
    if (x == MX_X_F16)
        return launch_shape<MX_X_F16, false>(a, p, st);
    if (x == MX_X_BF16)
        return launch_shape<MX_X_BF16, true>(a, p, st);
    return ybf ? launch_shape<MX_X_FP4, true>(a, p, st) : launch_shape<MX_X_FP4, false>(a, p, st);
}

}  // namespace w4a16

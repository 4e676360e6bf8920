// Products with MXFP4 weights for many rows (compute-bound).
//
// A workgroup's waves form a BM x BN tile of Y, WM x WN of it each, from stages
// of KC columns of K in a ring in LDS: 256 or 128 of MXFP4, 64 of a 16-bit type
// (128 or 64 bytes of a row of activations).  Every wave copies its share of a stage by
// buffer-to-LDS DMA, NBUF - 1 stages ahead of the products; the copies are inline
// assembly that the compiler does not count, so that it never waits for one by
// itself.  A stage holds the activation rows (gathered, if an index is given: a
// lane of a copy has its own address) and the weights' 16 x 64 tiles as they lie.
// Scales are copied a slab of 512 columns at a time, 16 bytes a row, when the
// slab's first stage is.
//
// Matrix instructions of 32 x 32, the weights first, so that a lane ends with
// four neighbouring columns of one row.  A lane's operand is 16 bytes, one block of
// 32 codes of one row: as MXFP4 it enters one 32 x 32 x 64 instruction with its
// scale; beside 16-bit activations its four words are decoded (one conversion
// a pair, the scale with it) for four 32 x 32 x 16 instructions, whose columns of
// K are the same eight for both operands.
//
// LDS: the weights' 16-byte blocks lie in the order in which lanes read them.  A
// row of activations is 4 (MXFP4) or 8 blocks of 16 bytes, stored at the block's
// number XOR a function of the row, so that the lanes of a read (one block of
// consecutive rows) reach all banks.  Results leave through LDS too, 32 rows of a
// wave at a time, so that a store writes whole runs of a row.  Reads of scales, whose
// rows lie 16 bytes apart, and writes of results do conflict: 0.15 .. 0.22 of the
// cycles that LDS is busy, which are 0.20 .. 0.28 of all.
//
// The largest tiles stay: as many workgroups as compute units, each taking tile
// after tile of its XCD's run, whose stages are one stream, so that the copies of
// the next tile run while results leave (2048 x 22016 x 4096 in bf16 295 -> 281 us,
// quantized 106 -> 104; 4096 tokens over 64 experts quantized 135 -> 128).
//
// Beside 16-bit activations the matrix cores are nearest to what bounds it where there
// are many rows: 2048 x 4096 x 11008 in bf16 159 us, 1.16 PFLOP/s (a large library
// product on this card: 1.39), busy 0.63 of the cycles; 2048 tokens over two of eight
// experts of 22016 x 4096 614, 1.20, busy 0.73.  Quantized they wait for stages, which
// have the time of one to land in: 2048 x 22016 x 4096 103, 3.6 (operands of random
// codes, from registers alone: 6.6 at the power limit), busy 0.43; 4096 tokens over six
// of 64 experts of 2816 x 2048 125, 2.3, busy 0.28: their last tiles are padding, and a
// tile has eight stages only.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "w4a16_mx_device.hpp"

namespace w4a16 {

namespace {

constexpr int kXcds = 8;  // MI355X: 8 XCDs, workgroups dealt round-robin
constexpr int kCus = 256;
constexpr int kMaxMatrices = 1024;

// A value that is the same in all lanes, in a scalar register.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Every wave's reads of the stage before are done, and its copies of this one.
template <int N>
__device__ __forceinline__ void stage_ready() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// Every wave's reads of the last stage are done (and its copies, if ALL).
template <bool ALL>
__device__ __forceinline__ void used_up() {
    if constexpr (ALL)
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    else
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// Where block `b` of row `row` stands among the row's 4 (MXFP4) or 8: any 8 or 16
// consecutive rows' blocks of one number lie in different banks.
template <bool FP4>
__device__ __forceinline__ uint32_t swizzle(uint32_t row, uint32_t b) {
    return FP4 ? b ^ ((row >> 1) & 3) ^ ((row >> 3) & 1) : b ^ (row & 7) ^ ((row >> 3) & 1);
}

// f with 0 .. N - 1, known when it is compiled (N 2 or 4).
template <int N, typename F>
__device__ __forceinline__ void steps(F f) {
    f(std::integral_constant<int, 0>{});
    f(std::integral_constant<int, 1>{});
    if constexpr (N == 4) {
        f(std::integral_constant<int, 2>{});
        f(std::integral_constant<int, 3>{});
    }
}

template <int XT, int KC, int BM, int BN, int WM, int WN, int NBUF, int OCC, bool STAY, bool GROUPED>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * 64, OCC * (BM / WM) * (BN / WN) / 4)
void mx_large_kernel(MxArgs a, int blocks_n, bool ybf) {
    constexpr bool FP4 = XT == MX_X_FP4;
    constexpr bool SPLIT = !STAY && !GROUPED;        // K may be split over workgroups
    constexpr int WAVES_N = BN / WN, WAVES = BM / WM * WAVES_N;
    constexpr int TM = WM / 32, TN = WN / 32;
    static_assert(FP4 ? KC == 128 || KC == 256 : KC == 64, "columns of a stage");
    constexpr int KQ = KC / 64;                      // of 64 columns each
    constexpr int H = FP4 ? KC / 128 : 1;            // parts of a stage's rows: 128 columns of
    constexpr int XROW = FP4 ? 64 : 128;             // MXFP4 or 64 of 16 bits, in bytes
    constexpr int RPC = 1024 / XROW, LPR = XROW / 16;    // rows of a copy, lanes of a row
    constexpr int SPS = 512 / KC;                    // stages of a slab
    constexpr int XPH = BM / RPC, XCH = H * XPH;     // copies of 1 KiB of a stage: activations,
    constexpr int WCH = KQ * BN / 32;                // weights;
    constexpr int SX = FP4 ? BM / 64 : 0, SCH = BN / 64 + SX;   // of a slab: scales
    static_assert(XCH % WAVES == 0 && WCH % WAVES == 0, "copies split evenly over the waves");
    constexpr int KX = XCH / WAVES, KW = WCH / WAVES, KSC = (SCH + WAVES - 1) / WAVES;
    constexpr int CPW = KX + KW;                     // copies of a wave and stage
    static_assert((NBUF - 1) * (CPW + KSC) < 64, "counted by vmcnt");
    constexpr int STAGE = (XCH + WCH) * 1024, SLAB = KSC * WAVES * 1024;
    // slabs that the stages of the ring can belong to: of one tile; of tiles of one
    // stage each; of tiles of two and more, a ring of four reaches three at most
    constexpr int NSLAB = !STAY ? (NBUF - 2) / SPS + 2 : NBUF < 4 ? NBUF : 3;
    constexpr int OUT = 32 * (WN > 64 ? WN : 64) * 2;    // a wave's results on their way
    // (through the ring's stages that are free, or a place of their own)
    constexpr bool OWN = WAVES * OUT > (STAY ? 1 : NBUF) * STAGE;
    constexpr int TABLE = STAY && GROUPED ? kMaxMatrices * 4 : 0;
    __shared__ __attribute__((aligned(1024))) char lds[NBUF * STAGE + NSLAB * SLAB + TABLE + (OWN ? WAVES * OUT : 0)];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WAVES_N, wn = wave % WAVES_N;
    const int h = lane >> 5, l32 = lane & 31;

    // this workgroup's tiles (one, unless STAY): the XCDs take equal runs of them,
    // column block by column block of a matrix, its row tiles one after the other,
    // so that neighbours in time share the weights of a column block in their L2
    const uint32_t xcd = blockIdx.x % kXcds, wg = blockIdx.x / kXcds, wgs = gridDim.x / kXcds;
    uint32_t *const table = (uint32_t *)(lds + NBUF * STAGE + NSLAB * SLAB);   // tiles up to each matrix
    uint32_t tiles;
    if constexpr (!GROUPED) {
        tiles = (uint32_t)((a.R + BM - 1) / BM);
    } else if constexpr (STAY) {
        if (wave == 0)
            mx_tile_table<BM>(a, table, lane);
        __syncthreads();
        tiles = (uint32_t)__builtin_amdgcn_readfirstlane((int)table[a.E - 1]);
    } else {
        tiles = mx_count_tiles<BM>(a, lane);
    }
    const uint32_t whole = tiles * (uint32_t)blocks_n, items = SPLIT ? whole * (uint32_t)a.splits : whole;
    const uint32_t first = items / kXcds * xcd + min(items % kXcds, xcd);
    const uint32_t run = items / kXcds + (items % kXcds > xcd ? 1 : 0);
    // (round by round, each one on from the last: a matrix's last tiles have less work,
    // and would fall to the same workgroups again and again)
    const uint32_t rounds = run / wgs;
    const uint32_t mine = (uint32_t)uniform((int)(rounds + ((wg + rounds) % wgs < run % wgs ? 1 : 0)));
    if (mine == 0)
        return;
    struct Item {
        MxTile t;
        int nb, split;
    };
    auto find = [&](uint32_t k) __attribute__((always_inline)) {
        Item it;
        const uint32_t at = first + k * wgs + (wg + k) % wgs;
        it.split = SPLIT ? uniform((int)(at / whole)) : 0;
        const uint32_t item = at - (uint32_t)it.split * whole;
        if constexpr (GROUPED) {
            const uint32_t any = (uint32_t)uniform((int)(item / (uint32_t)blocks_n));
            it.t = STAY ? mx_table_tile<BM>(a, table, any, lane) : mx_find_tile<BM>(a, any, lane);
            // (within the matrix: column block, then row tile)
            const uint32_t within = item - (any - (uint32_t)it.t.mt) * (uint32_t)blocks_n;
            it.nb = uniform((int)(within / (uint32_t)it.t.count));
            it.t.take((int)(within - (uint32_t)it.nb * (uint32_t)it.t.count), BM);
        } else {
            it.nb = uniform((int)(item / tiles));
            it.t = MxTile{0, 0, (int)a.R, (int)tiles};
            it.t.take((int)(item - (uint32_t)it.nb * tiles), BM);
        }
        return it;
    };

    const uint32_t wbytes = (uint32_t)a.NT * (uint32_t)a.KT * 1024u, sbytes = (uint32_t)a.NT * (uint32_t)a.KG * 256u;
    const uint32_t xrow = FP4 ? 64u : (uint32_t)a.K * 2u;
    const i4_t dx = make_desc(a.X, (uint32_t)(a.T * (FP4 ? a.KG * 256 : a.K * 2)));
    const i4_t dxs = make_desc(a.xs, FP4 ? (uint32_t)(a.T * a.KG * 16) : 0u);

    // The rows of X that a lane copies in a tile, as the index has them: of RPC a copy,
    // and of 64 a copy of scales.  (They are looked at when the tile's copies begin:
    // until then they may be on their way.)
    static_assert(XPH % WAVES == 0, "the same rows in every part");
    constexpr int KR = XPH / WAVES;
    struct Rows {
        uint32_t x[KR], s[KSC];
    };
    auto source_row = [&](const MxTile &t, int i) __attribute__((always_inline)) {
        uint32_t row = (uint32_t)t.row0 + (uint32_t)i;
        if (GROUPED && a.rows)
            row = i < t.rows ? (uint32_t)a.rows[t.row0 + i] : ~0u;
        return i < t.rows ? row : ~0u;
    };
    auto source_rows = [&](const MxTile &t) __attribute__((always_inline)) {
        Rows r;
#pragma unroll
        for (int k = 0; k < KR; k++)
            r.x[k] = source_row(t, (wave + k * WAVES) * RPC + lane / LPR);
#pragma unroll
        for (int k = 0; k < KSC; k++) {
            const int c = wave + k * WAVES - BN / 64;
            r.s[k] = FP4 && c >= 0 && c < SX ? source_row(t, c * 64 + lane) : ~0u;
        }
        return r;
    };
    // A lane's block of an activation row is the same in all of a wave's copies
    // (which are 16 rows apart or a multiple, and the order of blocks goes by the
    // row's number below 16).
    static_assert(WAVES * RPC % 16 == 0, "a lane's copies have one order of blocks");
    const uint32_t xblock = swizzle<FP4>((uint32_t)(wave * RPC + lane / LPR), (uint32_t)(lane % LPR));
    // the tile whose stages are being copied, and its copies' offsets
    i4_t dw, ds;
    uint32_t xo[KR], so[KSC];
    int nt0;
    auto begin = [&](const Item &it, const Rows &rows) __attribute__((always_inline)) {
        dw = make_desc((const char *)a.qd + (int64_t)it.t.e * wbytes, wbytes);
        ds = make_desc((const char *)a.sd + (int64_t)it.t.e * sbytes, sbytes);
#pragma unroll
        for (int k = 0; k < KR; k++)
            xo[k] = rows.x[k] < (uint32_t)a.T ? rows.x[k] * xrow + 16u * xblock : kOutOfRange;
        nt0 = it.nb * (BN / 16);
#pragma unroll
        for (int k = 0; k < KSC; k++) {
            // the scales of 64 columns (or rows) a copy
            const int c = wave + k * WAVES;
            so[k] = kOutOfRange;
            if (c < BN / 64) {
                const int nt = nt0 + 4 * c + (lane >> 4);
                if (nt < a.NT)
                    so[k] = (uint32_t)nt * 256u + 16u * (lane & 15);
            } else if (rows.s[k] < (uint32_t)a.T) {
                so[k] = rows.s[k] * 16u;
            }
        }
    };
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)lds;
    // the stages of a split
    const int all = (a.K + KC - 1) / KC;
    auto stage_from = [&](int split) __attribute__((always_inline)) {
        return SPLIT ? uniform(all * split / a.splits) : split * all;
    };
    // the copies of stage s of the current tile: the scales of its slab, to `place`,
    auto issue_slab = [&](int s, int place) __attribute__((always_inline)) {
        const uint32_t slab = (uint32_t)(s / SPS);
        const uint32_t at = lds0 + (uint32_t)(NBUF * STAGE + place * SLAB);
#pragma unroll
        for (int k = 0; k < KSC; k++) {
            const int c = wave + k * WAVES;
            if (!FP4 || c < BN / 64)
                copy16(ds, at + 1024u * (uint32_t)c, so[k], slab * (uint32_t)a.NT * 256u);
            else
                copy16(dxs, at + 1024u * (uint32_t)c, so[k], slab * (uint32_t)a.T * 16u);
        }
    };
    // and copies k0 .. k1 - 1 of the wave's CPW: activations, then weights, two tiles'
    // 64 columns a copy, 1 KiB as they lie.  (Past the last tile of rows the last one
    // again, whose results nobody stores; past the last of K, and where `none` is not
    // 0, zeros: of vector offsets past the descriptor, beside scalar offsets that are
    // within it, so that they do not rest on how the range check takes the two together.)
    auto issue = [&](int s, int buf, uint32_t none, auto k0_c, auto k1_c) __attribute__((always_inline)) {
        constexpr int k0 = decltype(k0_c)::value, k1 = decltype(k1_c)::value;
        const uint32_t to = lds0 + (uint32_t)(buf * STAGE);
        const int sx = none ? 0 : s;
#pragma unroll
        for (int k = k0; k < (k1 < KX ? k1 : KX); k++)
            copy16(dx, to + (uint32_t)(wave + k * WAVES) * 1024u,
                   none | (FP4 || (int)(8 * xblock) < a.K - s * 64 ? xo[k % KR] : kOutOfRange),
                   FP4 ? (uint32_t)(sx * H + k / KR) * (uint32_t)a.T * 64u : (uint32_t)(sx * XROW));
#pragma unroll
        for (int k = (k0 > KX ? k0 - KX : 0); k < k1 - KX; k++) {
            const int c = wave + k * WAVES;
            const int kq = KQ * s + c / (BN / 32), two = nt0 + 2 * (c % (BN / 32));
            const int nt = two < a.NT ? two : a.NT - 1;
            const bool in = !none && (!FP4 || kq < 2 * a.KT);
            copy16(dw, to + (uint32_t)(XCH + c) * 1024u,
                   in ? 16u * (nt + 1 < a.NT ? lane : lane & 31) : kOutOfRange,
                   in ? (uint32_t)(kq * a.NT + nt) * 512u : 0u);
        }
    };

    f16_t acc[TM][TN];
    // stage s of the wave's first MU row tiles; `between` is called in each of its parts
    auto compute = [&](int s, int buf, int place, auto mu, auto between) __attribute__((always_inline)) {
        constexpr int MU = decltype(mu)::value;
        const char *st = lds + buf * STAGE;
        const char *x = st + (wm * WM + l32) * XROW;      // (part 0)
        const char *w = st + XCH * 1024 + (wn * (WN / 16) + (l32 >> 4)) * 512 + h * 256 + (l32 & 15) * 16;
        const char *slab = lds + NBUF * STAGE + place * SLAB;
        const char *sw = slab + (wn * WN + l32) * 16, *sx = slab + (BN + wm * WM + l32) * 16;
        if constexpr (MU == 0) {
            steps<FP4 ? KQ : 4>(between);
        } else if constexpr (FP4) {
            // of a row's scale words of the stage, the lane's blocks in bytes 0 and 2
            uint32_t xs[MU][H], ws[TN][H];
            auto scales = [&](const char *from, uint32_t (&to)[H]) __attribute__((always_inline)) {
                from += 4 * H * (s % SPS);
                if constexpr (H == 2) {
                    const u2_t v = *(const u2_t *)from >> (uint32_t)(8 * h);
                    to[0] = v.x;
                    to[1] = v.y;
                } else {
                    to[0] = *(const uint32_t *)from >> (8 * h);
                }
            };
#pragma unroll
            for (int m = 0; m < MU; m++)
                scales(sx + 512 * m, xs[m]);
#pragma unroll
            for (int n = 0; n < TN; n++)
                scales(sw + 512 * n, ws[n]);
            u4_t xa[2][MU], wa[2][TN];        // (the next 64 columns are read during these)
            auto read = [&](int j) __attribute__((always_inline)) {
#pragma unroll
                for (int m = 0; m < MU; m++)
                    xa[j & 1][m] = *(const u4_t *)(x + (j / 2 * BM + m * 32) * XROW +
                                                   16 * swizzle<true>((uint32_t)l32, (uint32_t)(2 * (j & 1) + h)));
#pragma unroll
                for (int n = 0; n < TN; n++)
                    wa[j & 1][n] = *(const u4_t *)(w + n * 1024 + j * (BN * 32));
            };
            read(0);
            steps<KQ>([&](auto jc) __attribute__((always_inline)) {     // 64 columns each
                constexpr int j = decltype(jc)::value;
                if (j < KQ - 1)
                    read(j + 1);
#pragma unroll
                for (int n = 0; n < TN; n++) {
#pragma unroll
                    for (int m = 0; m < MU; m++)
                        acc[m][n] = j % 2 == 0
                            ? mx_mfma32<0>(wa[j & 1][n], xa[j & 1][m], acc[m][n], ws[n][j / 2], xs[m][j / 2])
                            : mx_mfma32<2>(wa[j & 1][n], xa[j & 1][m], acc[m][n], ws[n][j / 2], xs[m][j / 2]);
                    if (n == 0)
                        between(jc);
                }
                __builtin_amdgcn_sched_barrier(0);
            });
        } else {
            float ws[TN];
            u4_t wa[TN];
#pragma unroll
            for (int n = 0; n < TN; n++) {
                // (the slab's scale of block 2 s + h)
                ws[n] = __builtin_bit_cast(float, (uint32_t)*(const uint8_t *)(sw + 512 * n + 2 * (s % SPS) + h) << 23);
                wa[n] = *(const u4_t *)(w + n * 1024);
            }
            u4_t xa[2][MU];
            auto read = [&](int j) __attribute__((always_inline)) {
#pragma unroll
                for (int m = 0; m < MU; m++)
                    xa[j & 1][m] = *(const u4_t *)(x + m * 32 * XROW + 16 * swizzle<false>((uint32_t)l32, (uint32_t)(4 * h + j)));
            };
            read(0);
            steps<4>([&](auto jc) __attribute__((always_inline)) {
                constexpr int j = decltype(jc)::value;
                if (j < 3)
                    read(j + 1);
#pragma unroll
                for (int n = 0; n < TN; n++) {
                    const u4_t v = mx_decode<XT == MX_X_BF16>(wa[n][j], ws[n]);
#pragma unroll
                    for (int m = 0; m < MU; m++) {
                        if constexpr (XT == MX_X_BF16)
                            acc[m][n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                                __builtin_bit_cast(bf8_t, v), __builtin_bit_cast(bf8_t, xa[j & 1][m]), acc[m][n], 0, 0, 0);
                        else
                            acc[m][n] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
                                __builtin_bit_cast(h8_t, v), __builtin_bit_cast(h8_t, xa[j & 1][m]), acc[m][n], 0, 0, 0);
                    }
                    if (n == 0)
                        between(jc);
                }
                __builtin_amdgcn_sched_barrier(0);
            });
        }
    };

    // The stages of all tiles are one stream.  The copies run NBUF - 1 stages ahead,
    // into the next tile while this one's results are stored: `i` has the place of
    // the copies, `next` what the tile after theirs needs.
    struct {
        int s, s1, buf, place;
        uint32_t k;
    } i;
    Item now = find(0), next = now;
    Rows rows = source_rows(now.t);
    uint32_t known = 0;                 // the tile that `next` and `rows` are of
    begin(now, rows);
    i = {stage_from(now.split), stage_from(now.split + 1), 0, 0, 0};
    bool fresh = true;                  // i.s is its tile's first
    auto look_ahead = [&]() __attribute__((always_inline)) {
        if (STAY && known == i.k && i.k + 1 < mine) {
            known = i.k + 1;
            next = find(known);
            if constexpr (GROUPED)
                rows = source_rows(next.t);
        }
    };
    // goes on to the next stage to copy, its tile's offsets and its slab; whether
    // there is one
    auto next_stage = [&]() __attribute__((always_inline)) {
        if (i.s == i.s1) {
            if (!STAY || i.k + 1 >= mine)
                return false;
            look_ahead();
            i.k++;
            if constexpr (GROUPED)
                begin(next, rows);
            else
                begin(next, source_rows(next.t));
            i.s = stage_from(next.split);
            i.s1 = stage_from(next.split + 1);
            fresh = true;
        }
        if (fresh || i.s % SPS == 0) {
            i.place = i.place + 1 < NSLAB ? i.place + 1 : 0;
            issue_slab(i.s, i.place);
        }
        fresh = false;
        return true;
    };
#pragma unroll
    for (int k = 0; k < NBUF - 1; k++) {
        const uint32_t none = next_stage() ? 0u : kOutOfRange;
        issue(i.s, i.buf, none, std::integral_constant<int, 0>{}, std::integral_constant<int, CPW>{});
        i.s += none ? 0 : 1;
        i.buf = i.buf + 1 < NBUF ? i.buf + 1 : 0;
    }
    int buf = 0, place = 0;
    for (uint32_t k = 0; k < mine; k++) {
        const int s0 = stage_from(now.split), s1 = stage_from(now.split + 1);
#pragma unroll
        for (int m = 0; m < TM; m++)
#pragma unroll
            for (int n = 0; n < TN; n++)
#pragma unroll
                for (int e = 0; e < 16; e++)
                    acc[m][n][e] = 0.f;
        // Of a matrix's last tile a wave may have few rows or none, and leaves out their
        // products: whole halves of its rows (4096 tokens over 64 experts of 2816 x
        // 2048 quantized, with the order of tiles above, 136 -> 130 us; 1000 tokens
        // 61 -> 59; 2048 over 8 of 22016 x 4096 282 -> 275).
        auto stages = [&](auto mu) __attribute__((always_inline)) {
            for (int s = s0; s < s1; s++) {
                // (copies of the NBUF - 2 stages after this one may be under way)
                stage_ready<(NBUF - 2) * CPW>();
                // (Behind the last stage of all, copies of nothing: zeros, read by nobody.)
                const uint32_t none = next_stage() ? 0u : kOutOfRange;
                if (s == s0)
                    look_ahead();
                if (s == s0 || s % SPS == 0)
                    place = place + 1 < NSLAB ? place + 1 : 0;
                if constexpr (NBUF == 2) {
                    // the copies have to land within this stage: all at once
                    issue(i.s, i.buf, none, std::integral_constant<int, 0>{}, std::integral_constant<int, CPW>{});
                    compute(s, buf, place, mu, [](auto) {});
                } else {
                    // a quarter at a time between the products: all at once they fill the
                    // memory pipeline's queue and hold the waves up (2048 x 22016 x 4096 in
                    // bf16 293 -> 288 us)
                    compute(s, buf, place, mu, [&](auto j) __attribute__((always_inline)) {
                        constexpr int at = decltype(j)::value, parts = FP4 ? KQ : 4;
                        issue(i.s, i.buf, none, std::integral_constant<int, CPW * at / parts>{},
                              std::integral_constant<int, CPW * (at + 1) / parts>{});
                    });
                }
                i.s += none ? 0 : 1;
                i.buf = i.buf + 1 < NBUF ? i.buf + 1 : 0;
                buf = buf + 1 < NBUF ? buf + 1 : 0;
            }
        };
        if constexpr (GROUPED) {
            const int rows_of_wave = now.t.rows - wm * WM;
            if (rows_of_wave <= 0)
                stages(std::integral_constant<int, 0>{});
            else if (TM > 1 && rows_of_wave <= WM / 2)
                stages(std::integral_constant<int, (TM + 1) / 2>{});
            else
                stages(std::integral_constant<int, TM>{});
        } else {
            stages(std::integral_constant<int, TM>{});
        }
        // the results, 32 rows of the wave's at a time through its part of the stage
        // just used (the next copy there is issued after the next stage's barrier)
        used_up<!STAY>();
        const MxTile t = now.t;
        const int split = now.split, n0 = now.nb * BN + wn * WN;
        char *out = lds + wave * OUT + (OWN    ? NBUF * STAGE + NSLAB * SLAB + TABLE
                                        : STAY ? (buf == 0 ? NBUF - 1 : buf - 1) * STAGE
                                               : 0);
#pragma unroll
        for (int m = 0; m < TM; m++) {
            const int i0 = wm * WM + 32 * m;
            if (i0 >= t.rows)
                break;
            const int rows_here = t.rows - i0 < 32 ? t.rows - i0 : 32;
            if (SPLIT && a.splits > 1) {
                // fp32 sums of this split (rows of whole groups of four columns), 32
                // columns at a time
                float *part = a.part + ((int64_t)split * a.R + t.row0 + i0) * a.NP + n0;
                const int g = lane % 8;
#pragma unroll
                for (int n = 0; n < TN; n++) {
#pragma unroll
                    for (int q = 0; q < 4; q++)
                        *(f4_t *)(out + l32 * 128 + 16 * ((2 * q + h) ^ (l32 & 7))) =
                            f4_t{acc[m][n][4 * q], acc[m][n][4 * q + 1], acc[m][n][4 * q + 2], acc[m][n][4 * q + 3]};
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        const int r = 8 * k + lane / 8;
                        const f4_t v = *(const f4_t *)(out + r * 128 + 16 * (g ^ (r & 7)));
                        if (r < rows_here && n0 + 32 * n + 4 * g < a.N)
                            *(f4_t *)(part + (int64_t)r * a.NP + 32 * n + 4 * g) = v;
                    }
                }
                continue;
            }
            constexpr int G = WN / 8, X = G < 8 ? G - 1 : 7;
            const bool bf = FP4 ? ybf : XT == MX_X_BF16;
#pragma unroll
            for (int n = 0; n < TN; n++)
#pragma unroll
                for (int q = 0; q < 4; q++)
                    *(u2_t *)(out + l32 * (WN * 2) + 16 * ((4 * n + q) ^ (l32 & X)) + 8 * h) =
                        mx_pack4(bf, acc[m][n][4 * q], acc[m][n][4 * q + 1], acc[m][n][4 * q + 2], acc[m][n][4 * q + 3]);
            uint16_t *y = (uint16_t *)a.Y + (int64_t)(t.row0 + i0) * a.N + n0;
            // (a row of Y starts at a multiple of 16, 4 or 2 bytes)
            if ((a.N & 7) == 0) {
                const int g = lane % G;
#pragma unroll
                for (int k = 0; k < 32 * G / 64; k++) {
                    const int r = k * (64 / G) + lane / G;
                    const u4_t v = *(const u4_t *)(out + r * (WN * 2) + 16 * (g ^ (r & X)));
                    if (r < rows_here && n0 + 8 * g < a.N)
                        *(u4_t *)(y + (int64_t)r * a.N + 8 * g) = v;
                }
            } else if ((a.N & 1) == 0) {
                constexpr int P = WN / 2;                // pairs of columns a row
                const int c = 2 * (lane % P);
                for (int r = lane / P; r < rows_here; r += 64 / P)
                    if (n0 + c < a.N)
                        *(uint32_t *)(y + (int64_t)r * a.N + c) =
                            *(const uint32_t *)(out + r * (WN * 2) + 16 * ((c >> 3) ^ (r & X)) + 2 * (c & 7));
            } else {
                for (int at = lane; at < rows_here * WN; at += 64) {
                    const int r = at / WN, c = at % WN;
                    if (n0 + c < a.N)
                        y[(int64_t)r * a.N + c] =
                            *(const uint16_t *)(out + r * (WN * 2) + 16 * ((c >> 3) ^ (r & X)) + 2 * (c & 7));
                }
            }
        }
        if constexpr (!STAY)
            return;
        if (k + 1 < mine)
            now = find(k + 1);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // (copies of nothing: the LDS is still ours)
}

// The splits' sums, in their order, rounded: four columns a thread.
constexpr int kSumThreads = 256;
__global__ __launch_bounds__(kSumThreads) void mx_sum_kernel(MxArgs a, int64_t groups, bool ybf) {
    const int per = a.NP / 4;
    for (int64_t i = (int64_t)blockIdx.x * kSumThreads + threadIdx.x; i < groups;
         i += (int64_t)gridDim.x * kSumThreads) {
        const int64_t row = i / per;
        const int n = (int)(i - row * per) * 4;
        f4_t v = *(const f4_t *)(a.part + 4 * i);
        for (int k = 1; k < a.splits; k++)
            v += *(const f4_t *)(a.part + (int64_t)k * a.R * a.NP + 4 * i);
        mx_store4((uint16_t *)a.Y + row * a.N, n, a.N, ybf, v[0], v[1], v[2], v[3]);
    }
}

template <int XT, int KC, int BM, int BN, int WM, int WN, int NBUF, int OCC, bool STAY, bool GROUPED>
int launch_inst(const MxArgs &a, bool ybf, hipStream_t st) {
    const int64_t blocks = (a.N + BN - 1) / BN;
    // sum over the matrices with rows of ceil(rows / BM), at most
    const int64_t used = a.R < a.E ? a.R : a.E;
    const int64_t tiles = GROUPED ? used + (a.R - used) / BM : (a.R + BM - 1) / BM;
    const int64_t items = tiles * blocks * a.splits, most = STAY && items > kCus ? kCus : items;
    const int64_t grid = (most + kXcds - 1) / kXcds * kXcds;
    constexpr int threads = (BM / WM) * (BN / WN) * 64;
    if (items >= (int64_t(1) << 31) || grid * threads >= (int64_t(1) << 32))
        return (int)hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((mx_large_kernel<XT, KC, BM, BN, WM, WN, NBUF, OCC, STAY, GROUPED>), dim3((unsigned)grid),
                       dim3(threads), 0, st, a, (int)blocks, ybf);
    const int e = (int)hipGetLastError();
    if (e || a.splits == 1)
        return e;
    const int64_t groups = a.R * (a.NP / 4), wgs = (groups + kSumThreads - 1) / kSumThreads;
    hipLaunchKernelGGL(mx_sum_kernel, dim3((unsigned)(wgs < (1 << 20) ? wgs : 1 << 20)), dim3(kSumThreads), 0, st, a,
                       groups, XT == MX_X_FP4 ? ybf : XT == MX_X_BF16);
    return (int)hipGetLastError();
}

template <int XT, bool GROUPED>
int launch_shape(const MxArgs &a, const MxPlan &p, bool ybf, hipStream_t st) {
    if constexpr (XT == MX_X_FP4) {
        switch (p.shape) {
        case MX_64x128: return launch_inst<XT, 256, 64, 128, 32, 64, 3, 2, false, GROUPED>(a, ybf, st);
        case MX_128x128: return launch_inst<XT, 256, 128, 128, 64, 64, 2, 2, false, GROUPED>(a, ybf, st);
        case MX_128x256:
            // (four stages of 128 columns where an expert's weights come from memory:
            // 1000 tokens over 64 experts of 2816 x 2048 63 -> 56 us; two of 256 where they
            // stay in the caches: 2048 x 22016 x 4096 128 -> 116)
            if constexpr (GROUPED)
                return launch_inst<XT, 128, 128, 256, 64, 64, 4, 1, true, GROUPED>(a, ybf, st);
            else
                return launch_inst<XT, 256, 128, 256, 64, 64, 2, 1, true, GROUPED>(a, ybf, st);
        default: return launch_inst<XT, 256, 256, 256, 128, 64, 2, 1, true, GROUPED>(a, ybf, st);
        }
    } else {
        switch (p.shape) {
        case MX_64x128: return launch_inst<XT, 64, 64, 128, 32, 64, 3, 3, false, GROUPED>(a, ybf, st);
        case MX_64x256: return launch_inst<XT, 64, 64, 256, 64, 64, 4, 2, false, GROUPED>(a, ybf, st);
        case MX_128x128: return launch_inst<XT, 64, 128, 128, 64, 64, 3, 2, false, GROUPED>(a, ybf, st);
        case MX_128x256: return launch_inst<XT, 64, 128, 256, 128, 64, 3, 2, false, GROUPED>(a, ybf, st);
        default: return launch_inst<XT, 64, 256, 256, 128, 64, 3, 1, true, GROUPED>(a, ybf, st);
        }
    }
}

template <int XT>
int launch_any(const MxArgs &a, const MxPlan &p, bool ybf, hipStream_t st) {
    return a.offsets ? launch_shape<XT, true>(a, p, ybf, st) : launch_shape<XT, false>(a, p, ybf, st);
}

}  // namespace

int launch_mx_large(const MxArgs &a, const MxPlan &p, int x, bool ybf, void *stream) {
    hipStream_t st = (hipStream_t)stream;
    if (x == MX_X_F16)
        return launch_any<MX_X_F16>(a, p, ybf, st);
    if (x == MX_X_BF16)
        return launch_any<MX_X_BF16>(a, p, ybf, st);
    return launch_any<MX_X_FP4>(a, p, ybf, st);
}

}  // namespace w4a16

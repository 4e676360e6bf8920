// Low-rank adapters: the first product, S[m] = scale_a X[m] . A_a^T, and the
// launch of the GEMM with the second one in its epilogue.
#include <hip/hip_runtime.h>

#include "w4a16_gemm_kernels.hpp"
#include "w4a16_kernels.hpp"
#include "w4a16_lora.hpp"

namespace w4a16 {

namespace {

// A workgroup takes a tile of 16 rows and a block of 32 ranks of one part over
// all of K, and of the distinct adapters of its rows every `lanes`-th: with few row
// tiles each adapter of a tile has a workgroup of its own (rows of 16
// different adapters read 16 of them at once), with many two workgroups do
// them all, since a run of rows with one adapter (a prompt) has only one, and
// a workgroup that finds nothing to do still costs its launch (measured: 1920
// of 16 waves 0.1 us each).  Rows in any order need no sort.
//
// The waves split K in runs of 128 columns and are summed in LDS.  Each wave
// copies its runs' 16 rows of X and of A into a ring of its own in LDS by
// buffer-to-LDS DMA, whole 256-byte pieces of rows, and reads the MFMA
// operands there (as the XL form of gemm_small_m_kernel, so no barrier): loaded
// straight into operands, each lane of a load touches another row's cache
// line, and a compute unit takes in 16 bytes a clock instead of 64 (measured:
// one adapter of rank 16 at K = 4096 7.6 us, down at M = 2048 56 us).
// The first wave stores the sums as the second product reads them (LoraS).  K is
// not split across workgroups: the second product would have to add the
// slices, and its latency is on the GEMM's own path (measured at four slices:
// qkv at M = 32 20.1 us for the GEMM with adapters, 13.2 without).
constexpr int kShrinkWaves = 4;

// NB: 16-rank tiles, 1 where the rank is at most 16 (the block's other half is
// stored as zeros).
template <int NB, bool BF>
__global__ __launch_bounds__(kShrinkWaves * 64) void lora_shrink_kernel(LoraShrinkArgs a) {
    constexpr int D = NB == 1 ? 4 : 3;       // ring slots: 128 or 144 KiB in all
    constexpr int SLOT = (1 + NB) * 256;     // u4_t: 16 rows x 128 columns of X, then of A
    __shared__ u4_t ring[kShrinkWaves][D * SLOT];
    __shared__ f4_t red[kShrinkWaves][NB * 64];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    const int r = lane & 15, i = lane >> 4;
    const int64_t m0 = (int64_t)(blockIdx.x / a.lanes) * 16;
    const int turn = (int)(blockIdx.x % a.lanes);
    int id = lane < 16 && m0 + lane < a.M ? a.ids[m0 + lane] : -1;
    id = id < a.n ? id : -1;
    uint32_t todo = (uint32_t)__ballot(id >= 0);
    const int block = (int)blockIdx.y;                     // p blocks + jb
    const int part = block / a.blocks, c0 = (block - part * a.blocks) * 32;
    const int tile_rows = (int)(a.M - m0 < 16 ? a.M - m0 : 16);
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.X + m0 * a.K, (uint32_t)(tile_rows * a.K * 2));
    const int runs = (a.K + 127) / 128;
    const int mine = runs > wave ? (runs - wave + kShrinkWaves - 1) / kShrinkWaves : 0;
    if (turn == 0 && block == 0 && wave == 0) {
        // the list of the tile's adapters
        LoraList &list = a.lists[m0 / 16];
        uint32_t rest = todo;
        int count = 0;
        for (; rest; count++) {
            const int ad = __builtin_amdgcn_readlane(id, __builtin_ctz(rest));
            const uint32_t rows = (uint32_t)__ballot(id == ad);
            rest &= ~rows;
            if (lane == 0) {
                list.adapter[count] = ad;
                list.rows[count] = rows;
            }
        }
        if (lane == 0)
            list.count = count;
    }
    for (int k = 0; todo; k++) {
        const int ad = __builtin_amdgcn_readlane(id, __builtin_ctz(todo));
        const uint32_t rows = (uint32_t)__ballot(id == ad);
        todo &= ~rows;
        if (k % a.lanes != turn)
            continue;
        const __amdgpu_buffer_rsrc_t ra = make_rsrc(
            a.A + ((int64_t)ad * a.parts + part) * a.r * a.K, (uint32_t)(a.r * a.K * 2));
        const float scale = a.scales[ad];
        // copy c: rows 4 c .. 4 c + 3, lane L row 4 c + L / 16, the chunk its
        // position L % 16 holds; rows of other adapters, and ranks past the
        // last, out of range (zeros)
        int col[4];
        uint32_t ox[4], oa[NB][4];
#pragma unroll
        for (int c = 0; c < 4; c++) {
            const int row = 4 * c + (lane >> 4);
            col[c] = 8 * ((lane & 15) ^ row);
            ox[c] = rows >> row & 1 ? (uint32_t)((row * a.K + col[c]) * 2) : kOutOfRange;
#pragma unroll
            for (int b = 0; b < NB; b++) {
                const int rank = c0 + 16 * b + row;
                oa[b][c] = rank < a.r ? (uint32_t)((rank * a.K + col[c]) * 2) : kOutOfRange;
            }
        }
        f4_t acc[NB];
#pragma unroll
        for (int b = 0; b < NB; b++)
            acc[b] = f4_t{0.f, 0.f, 0.f, 0.f};
        // (columns past K, and runs past the last: out of range too)
        auto load = [&](int slot, int k) __attribute__((always_inline)) {
            const int q = wave + kShrinkWaves * k;
            const int left = k < mine ? a.K - 128 * q : 0;
            u4_t *at = ring[wave] + slot * SLOT;
#pragma unroll
            for (int c = 0; c < 4; c++) {
                const bool in = col[c] < left;
                lds_dma16_so(rx, at + 64 * c, in ? ox[c] : kOutOfRange, 256u * (uint32_t)q);
#pragma unroll
                for (int b = 0; b < NB; b++)
                    lds_dma16_so(ra, at + (1 + b) * 256 + 64 * c, in ? oa[b][c] : kOutOfRange,
                                 256u * (uint32_t)q);
            }
        };
        auto multiply = [&](int slot) __attribute__((always_inline)) {
            const u4_t *at = ring[wave] + slot * SLOT + r * 16;
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const u4_t x = at[(4 * j + i) ^ r];
#pragma unroll
                for (int b = 0; b < NB; b++) {
                    const u4_t w = at[(1 + b) * 256 + ((4 * j + i) ^ r)];
                    if constexpr (BF)
                        acc[b] = mfma16x16x32_bf16(__builtin_bit_cast(bf8_t, x),
                                                   __builtin_bit_cast(bf8_t, w), acc[b]);
                    else
                        acc[b] = mfma16x16x32(__builtin_bit_cast(h8_t, x),
                                              __builtin_bit_cast(h8_t, w), acc[b]);
                }
            }
        };
        // D - 1 runs in flight behind the one multiplied
        constexpr int LPS = 4 * (1 + NB);
#pragma unroll
        for (int p = 0; p < D - 1; p++)
            load(p, p);
        auto turn_of = [&](int s, auto slot_c) __attribute__((always_inline)) {
            constexpr int slot = decltype(slot_c)::value;
            load((slot + D - 1) % D, s + D - 1);
            wait_vmcnt<(D - 1) * LPS>();
            multiply(slot);
        };
        for (int s = 0; s < mine; s += D)
            ring_pass<D>(s, mine, turn_of);
        wait_vmcnt<0>();   // (the runs past the last write zeros)
#pragma unroll
        for (int b = 0; b < NB; b++)
            red[wave][b * 64 + lane] = acc[b];
        __syncthreads();
        if (wave == 0) {
            f4_t v[2];
            v[1] = f4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int b = 0; b < NB; b++) {
                v[b] = red[0][b * 64 + lane];
#pragma unroll
                for (int w = 1; w < kShrinkWaves; w++)
                    v[b] += red[w][b * 64 + lane];
                v[b] *= scale;
            }
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const int row = 4 * i + e;
                if (!(rows >> row & 1))
                    continue;
                const int64_t at = ((int64_t)block * a.M + m0 + row) * 32 + r;
                if constexpr (BF) {
#pragma unroll
                    for (int b = 0; b < 2; b++) {
                        const __bf16 hi = (__bf16)v[b][e];
                        const float h = (float)hi;
                        ((__bf16 *)a.S_hi)[at + 16 * b] = hi;
                        ((__bf16 *)a.S_lo)[at + 16 * b] =
                            __builtin_isfinite(h) ? (__bf16)(v[b][e] - h) : (__bf16)0.f;
                    }
                } else {
                    // the largest of the row's 32 values: lanes r = 0 .. 15
                    // (the branch is uniform over them)
                    float top = fmaxf(fabsf(v[0][e]), fabsf(v[1][e]));
#pragma unroll
                    for (int d = 1; d < 16; d *= 2)
                        top = fmaxf(top, __shfl_xor(top, d));
                    // (0, infinity and NaN stay as they are; ilogb of a
                    // finite value is -149 .. 127)
                    const int up = top > 0.f && __builtin_isfinite(top) ? max(ilogbf(top) - 14, -100) : 0;
                    if (r == 0)
                        a.F[(int64_t)block * a.f_pitch + m0 + row] = ldexpf(1.f, up);
#pragma unroll
                    for (int b = 0; b < 2; b++) {
                        const float x = ldexpf(v[b][e], -up);
                        const _Float16 hi = (_Float16)x;
                        const float h = (float)hi;
                        ((_Float16 *)a.S_hi)[at + 16 * b] = hi;
                        ((_Float16 *)a.S_lo)[at + 16 * b] =
                            __builtin_isfinite(h) ? (_Float16)(x - h) : (_Float16)0.f;
                    }
                }
            }
        }
        __syncthreads();   // before the next adapter's sums
    }
}

template <bool BF>
void launch_shrink(const LoraShrinkArgs &a, hipStream_t st) {
    const dim3 grid((unsigned)((a.M + 15) / 16 * a.lanes), (unsigned)(a.parts * a.blocks));
    const dim3 block(kShrinkWaves * 64);
    if (a.r <= 16)
        hipLaunchKernelGGL((lora_shrink_kernel<1, BF>), grid, block, 0, st, a);
    else
        hipLaunchKernelGGL((lora_shrink_kernel<2, BF>), grid, block, 0, st, a);
}

}  // namespace

int launch_lora_shrink(const LoraShrinkArgs &a, void *stream) {
    if (a.bf16)
        launch_shrink<true>(a, (hipStream_t)stream);
    else
        launch_shrink<false>(a, (hipStream_t)stream);
    return (int)hipGetLastError();
}

int launch_gemm_lora(const uint16_t *X, const void *q_dev, const void *s_dev, const void *z_dev,
                     const Geom &geo, const GemmPlan &plan, const LoraArgs &lora, uint16_t *Y,
                     void *workspace, void *stream) {
    const GemmArgs a = gemm_args(X, q_dev, s_dev, z_dev, geo, plan, Y, workspace);
    const hipStream_t st = (hipStream_t)stream;
    LoraExt x;
    x.l = lora;
    int e;
    if (plan.path == PATH_SMALL) {
        const SmallPlan p = small_plan(plan);
        if (a.g == 32)
            e = a.bf16 ? launch_small_m_jpg1_bf16_lora(a, p, x, st) : launch_small_m_jpg1_lora(a, p, x, st);
        else if (a.g == 64)
            e = a.bf16 ? launch_small_m_jpg2_bf16_lora(a, p, x, st) : launch_small_m_jpg2_lora(a, p, x, st);
        else
            e = a.bf16 ? launch_small_m_jpg4_bf16_lora(a, p, x, st) : launch_small_m_jpg4_lora(a, p, x, st);
        return e || a.splits == 1 ? e : launch_splitk_reduce(a, st);
    }
    LargePlan lp;
    lp.shape = plan.large_shape;
    return a.bf16 ? launch_large_m_bf16_lora(a, lp, x, st) : launch_large_m_lora(a, lp, x, st);
}

}  // namespace w4a16

// Low-rank adapters: the first product, S[m] = scale_a X[m] . A_a^T, and the
// launch of the GEMM with the second one in its epilogue.
#include <hip/hip_runtime.h>

#include "w4a16_gemm_kernels.hpp"
#include "w4a16_kernels.hpp"
#include "w4a16_lora.hpp"

namespace w4a16 {

namespace {

// One workgroup for each (row, block of 16 NB ranks); it does the work of its
// 16-row tile for its row's adapter, and nothing unless its row is the first
// of the tile with that adapter.  So rows in any order need no sort, a run of
// rows with one adapter takes one MFMA tile per 16, and rows of 16 different
// adapters take 16 workgroups that each read one adapter.
// The W waves split K (32-column MFMA steps, in turn) and are summed in LDS.
constexpr int kShrinkWaves = 16;

template <int NB, bool BF>
__global__ __launch_bounds__(kShrinkWaves * 64) void lora_shrink_kernel(LoraShrinkArgs a) {
    __shared__ f4_t red[kShrinkWaves][NB * 64];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    const int r = lane & 15, i = lane >> 4;
    const int64_t m = blockIdx.x, m0 = m & ~(int64_t)15;
    const int ad = a.ids[m];
    if (ad < 0 || ad >= a.n)
        return;
    const bool mine = lane < 16 && m0 + lane < a.M && a.ids[m0 + lane] == ad;
    const uint32_t rows = (uint32_t)__ballot(mine);
    if (__builtin_ctz(rows) != (int)(m - m0))
        return;
    const int c0 = (int)blockIdx.y * NB * 16;   // first rank of the workgroup

    const int tile_rows = (int)(a.M - m0 < 16 ? a.M - m0 : 16);
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.X + m0 * a.K, (uint32_t)(tile_rows * a.K * 2));
    const __amdgpu_buffer_rsrc_t ra =
        make_rsrc(a.A + (int64_t)ad * a.pr * a.K, (uint32_t)(a.pr * a.K * 2));
    const uint32_t ox = rows >> r & 1 ? (uint32_t)((r * a.K + 8 * i) * 2) : kOutOfRange;
    uint32_t oa[NB];
#pragma unroll
    for (int b = 0; b < NB; b++)
        oa[b] = c0 + 16 * b + r < a.pr ? (uint32_t)(((c0 + 16 * b + r) * a.K + 8 * i) * 2) : kOutOfRange;

    f4_t acc[NB];
#pragma unroll
    for (int b = 0; b < NB; b++)
        acc[b] = f4_t{0.f, 0.f, 0.f, 0.f};
    const int steps = (a.K + 31) / 32;
    constexpr int U = 4;   // steps whose loads are issued together
    for (int s0 = wave; s0 < steps; s0 += kShrinkWaves * U) {
        u4_t x[U], w[U][NB];
#pragma unroll
        for (int u = 0; u < U; u++) {
            // columns past K: out of range, both operands read 0
            const int s = s0 + kShrinkWaves * u;
            const bool in = 32 * s + 8 * i < a.K;
            x[u] = __builtin_bit_cast(u4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                                rx, (int)(in ? ox + 64u * s : kOutOfRange), 0, 0));
#pragma unroll
            for (int b = 0; b < NB; b++)
                w[u][b] = __builtin_bit_cast(
                    u4_t, __builtin_amdgcn_raw_buffer_load_b128(
                              ra, (int)(in ? oa[b] + 64u * s : kOutOfRange), 0, 0));
        }
#pragma unroll
        for (int u = 0; u < U; u++)
#pragma unroll
            for (int b = 0; b < NB; b++) {
                if constexpr (BF)
                    acc[b] = mfma16x16x32_bf16(__builtin_bit_cast(bf8_t, x[u]),
                                               __builtin_bit_cast(bf8_t, w[u][b]), acc[b]);
                else
                    acc[b] = mfma16x16x32(__builtin_bit_cast(h8_t, x[u]),
                                          __builtin_bit_cast(h8_t, w[u][b]), acc[b]);
            }
    }
#pragma unroll
    for (int b = 0; b < NB; b++)
        red[wave][b * 64 + lane] = acc[b];
    __syncthreads();
    const float scale = a.scales[ad];
    for (int idx = threadIdx.x; idx < NB * 64; idx += kShrinkWaves * 64) {
        f4_t v = red[0][idx];
#pragma unroll
        for (int w = 1; w < kShrinkWaves; w++)
            v += red[w][idx];
        const int l = idx & 63, c = c0 + (idx >> 6) * 16 + (l & 15);
        if (c >= a.pr)
            continue;
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const int row = 4 * (l >> 4) + e;
            if (rows >> row & 1)
                a.S[(m0 + row) * a.pr + c] = scale * v[e];
        }
    }
}

template <bool BF>
void launch_shrink(const LoraShrinkArgs &a, hipStream_t st) {
    const dim3 block(kShrinkWaves * 64);
    if (a.pr <= 16)
        hipLaunchKernelGGL((lora_shrink_kernel<1, BF>), dim3((unsigned)a.M), block, 0, st, a);
    else
        hipLaunchKernelGGL((lora_shrink_kernel<2, BF>),
                           dim3((unsigned)a.M, (unsigned)((a.pr + 31) / 32)), block, 0, st, a);
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

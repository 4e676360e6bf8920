// Pure host logic of the routed operators: argument checks, plans and
// workspace sizes.  No HIP call is made here.
#include <math.h>
#include <stdint.h>

#include "w4a16_routed.h"
#include "w4a16_routed.hpp"

namespace w4a16 {

namespace {

bool aligned(const void *p, uintptr_t to) { return ((uintptr_t)p & (to - 1)) == 0; }

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

bool overlap(const void *a, int64_t a_bytes, const void *b, int64_t b_bytes) {
    const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
    return a0 < b0 + (uintptr_t)b_bytes && b0 < a0 + (uintptr_t)a_bytes;
}

constexpr uint32_t kWeightFlags = W4A16_SYMMETRIC | W4A16_PARTIAL_LAST_GROUP | W4A16_BF16;

// Shape, group and flag rules of an experts call (w4a16_repack_size has the
// rules of one matrix).
int32_t check_experts_shape(int64_t T, int32_t k, int64_t K, int64_t I, int64_t D, int64_t E,
                            int32_t g, uint32_t flags) {
    if (flags & ~kWeightFlags)
        return W4A16_ERR_FLAGS;
    if (T <= 0 || T > (int64_t(1) << 20) || k <= 0 || k > 32 || E <= 0 || E > kMaxExperts ||
        T * k > (int64_t(1) << 22))
        return W4A16_ERR_SHAPE;
    size_t q, s, z;
    int32_t st = w4a16_repack_size(I, K, g, flags, &q, &s, &z);
    if (!st)
        st = w4a16_repack_size(D, I, g, flags, &q, &s, &z);
    if (st)
        return st;
    // the kernels address one expert's matrices, and X, with 31-bit byte offsets
    const Geom gu = make_geom(T, I, K, g, flags), dn = make_geom(T, D, I, g, flags);
    if (2 * gu.NT * gu.KT * 1024 >= (int64_t(1) << 31) ||
        dn.NT * dn.KT * 1024 >= (int64_t(1) << 31) || T * K * 2 >= (int64_t(1) << 31))
        return W4A16_ERR_SHAPE;
    // a tile's rows of h and P too
    if (128 * I * 2 >= (int64_t(1) << 31) || 128 * D * 4 >= (int64_t(1) << 31))
        return W4A16_ERR_SHAPE;
    return W4A16_OK;
}

int32_t check_lora_shape(int64_t N, int64_t K, int64_t n, int32_t r, int32_t n_parts) {
    if (n <= 0 || n > 65536 || r <= 0 || r > 256 || r % 8 != 0 || n_parts <= 0 ||
        n_parts > W4A16_LORA_MAX_PARTS || n_parts > N)
        return W4A16_ERR_SHAPE;
    // one adapter's A is addressed with 31-bit byte offsets
    if ((int64_t)n_parts * r * K * 2 >= (int64_t(1) << 31))
        return W4A16_ERR_SHAPE;
    return W4A16_OK;
}

}  // namespace

// Rows per tile: 16 (one MFMA row tile, the memory-bound kernel) while an
// expert has few rows on average, then 64 and 128 rows of the compute-bound
// kernel.
ExpertsPlan plan_experts(int64_t T, int k, int64_t K, int64_t I, int64_t D, int64_t E, int32_t g,
                         uint32_t flags) {
    ExpertsPlan p;
    const int64_t R = T * k;
    // One token's activations, scales and zero words stay in LDS (1 KiB
    // chunks, of every slot in the second product) where they leave room for
    // two workgroups on a compute unit.
    const Geom gu = make_geom(1, I, K, g, flags), dn = make_geom(1, D, I, g, flags);
    auto image = [](const Geom &q, int tiles) {
        return (q.KT * 256 + 1023) / 1024 +
               tiles * ((q.G * 32 + 1023) / 1024 + (q.sym ? 0 : (q.GW * 64 + 1023) / 1024));
    };
    p.one = T == 1 && image(gu, 2) <= 72 && k * image(dn, 1) <= 72;
    p.direct = R <= kDirectRows;
    p.mt = R <= 16 * E ? 1 : 4;
    p.large = !p.direct && R > 16 * E;
    p.bm = !p.large ? 16 * p.mt : R <= 64 * E ? 64 : 128;
    // sum over the experts with rows of ceil(rows / bm), at most
    const int64_t used = R < E ? R : E;
    p.tiles = p.direct ? R : used + (R - used) / p.bm;
    size_t at = 0;
    p.used_off = at;
    at += p.direct ? 0 : 256;
    p.tiles_off = at;
    at += p.direct ? 0 : up256((size_t)p.tiles * sizeof(ExpertTile));
    p.perm_off = at;
    at += p.direct ? 0 : up256((size_t)R * 4);
    p.place_off = at;
    at += p.direct ? 0 : up256((size_t)R * 4);
    p.h_off = at;
    at += up256((size_t)R * (size_t)I * 2);
    p.p_off = at;
    at += up256((size_t)R * (size_t)D * 4);
    p.ws_bytes = at;
    return p;
}

// Up to 16 row tiles, each adapter of a tile has a workgroup in the first
// product, above two share them (see lora_shrink_kernel): one for most tiles
// of a prompt, the second for those where two prompts meet (six prompts at M =
// 2048, K = 11008: 29.7 us with one, 17.1 for a single prompt).
LoraPlan plan_lora(int64_t M, int parts, int r, bool bf16) {
    LoraPlan p;
    p.blocks = (r + 31) / 32;
    p.lanes = M > 256 ? 2 : M < 16 ? (int)M : 16;
    p.f_pitch = (M + 15) / 16 * 16;
    const size_t values = (size_t)parts * (size_t)p.blocks * (size_t)M * 32 * 2;
    p.s_hi_off = up256((size_t)(p.f_pitch / 16) * sizeof(LoraList));
    p.s_lo_off = p.s_hi_off + up256(values);
    p.f_off = p.s_lo_off + up256(values);
    p.bytes = p.f_off + (bf16 ? 0 : (size_t)parts * (size_t)p.blocks * (size_t)p.f_pitch * 4);
    return p;
}

}  // namespace w4a16

using namespace w4a16;

extern "C" {

int32_t w4a16_check_route_args(const void *logits, int32_t logits_dtype, int64_t T, int64_t E,
                               const float *bias, int32_t k, int32_t n_groups,
                               int32_t topk_groups, int32_t group_top, float scale,
                               uint32_t flags, const int32_t *ids, const float *weights) {
    if (flags & ~(W4A16_ROUTE_SIGMOID | W4A16_ROUTE_RENORMALIZE))
        return W4A16_ERR_FLAGS;
    if (!logits || !ids || !weights)
        return W4A16_ERR_NULL;
    if (logits_dtype < W4A16_LOGITS_F16 || logits_dtype > W4A16_LOGITS_F32 || T <= 0 ||
        T > (int64_t(1) << 24) || E <= 0 || E > kMaxExperts || n_groups <= 0 || n_groups > 64 ||
        E % n_groups != 0 || topk_groups <= 0 || topk_groups > n_groups || group_top < 1 ||
        group_top > 2 || k <= 0 || k > 32 || k > topk_groups * (E / n_groups) || !isfinite(scale))
        return W4A16_ERR_SHAPE;
    if (!aligned(logits, logits_dtype == W4A16_LOGITS_F32 ? 4 : 2) || !aligned(bias, 4) ||
        !aligned(ids, 4) || !aligned(weights, 4))
        return W4A16_ERR_ALIGN;
    return W4A16_OK;
}

int32_t w4a16_experts_workspace_size(int64_t T, int32_t k, int64_t K, int64_t I, int64_t D,
                                     int64_t E, int32_t g, uint32_t flags, size_t *bytes) {
    if (!bytes)
        return W4A16_ERR_NULL;
    const int32_t st = check_experts_shape(T, k, K, I, D, E, g, flags);
    if (st)
        return st;
    *bytes = plan_experts(T, k, K, I, D, E, g, flags).ws_bytes;
    return W4A16_OK;
}

int32_t w4a16_check_experts_args(const uint16_t *X, int64_t T, int64_t K, const int32_t *ids,
                                 const float *weights, int32_t k, int64_t E,
                                 const void *gate_up_q, const void *gate_up_s,
                                 const void *gate_up_z, int64_t I, const void *down_q,
                                 const void *down_s, const void *down_z, int64_t D, int32_t g,
                                 uint32_t flags, const uint16_t *Y, const void *workspace,
                                 size_t workspace_bytes) {
    int32_t st = check_experts_shape(T, k, K, I, D, E, g, flags);
    if (st)
        return st;
    const bool sym = (flags & W4A16_SYMMETRIC) != 0;
    if (!X || !ids || !weights || !gate_up_q || !gate_up_s || !down_q || !down_s || !Y ||
        !workspace || (!sym && (!gate_up_z || !down_z)))
        return W4A16_ERR_NULL;
    if (!aligned(X, 16) || !aligned(gate_up_q, 16) || !aligned(gate_up_s, 16) ||
        !aligned(down_q, 16) || !aligned(down_s, 16) || !aligned(Y, 16) ||
        !aligned(workspace, 16) || (!sym && (!aligned(gate_up_z, 16) || !aligned(down_z, 16))) ||
        !aligned(ids, 4) || !aligned(weights, 4))
        return W4A16_ERR_ALIGN;
    const ExpertsPlan p = plan_experts(T, k, K, I, D, E, g, flags);
    if (workspace_bytes < p.ws_bytes)
        return W4A16_ERR_WORKSPACE;
    // Y is written while ids and weights are still read
    if (overlap(X, T * K * 2, Y, T * D * 2) || overlap(ids, T * k * 4, Y, T * D * 2) ||
        overlap(weights, T * k * 4, Y, T * D * 2))
        return W4A16_ERR_SHAPE;
    return W4A16_OK;
}

int32_t w4a16_gemm_lora_workspace_size(int64_t M, int64_t N, int64_t K, int32_t g,
                                       uint32_t flags, int32_t n_parts, int32_t r,
                                       size_t *bytes) {
    if (!bytes)
        return W4A16_ERR_NULL;
    size_t gemm = 0;
    int32_t st = w4a16_gemm_workspace_size(M, N, K, g, flags, &gemm);
    if (!st)
        st = check_lora_shape(N, K, 1, r, n_parts);
    if (st)
        return st;
    *bytes = up256(gemm) + plan_lora(M, n_parts, r, (flags & W4A16_BF16) != 0).bytes;
    return W4A16_OK;
}

int32_t w4a16_check_gemm_lora_args(const uint16_t *X, int64_t M, int64_t K, const void *q_dev,
                                   const void *s_dev, const void *z_dev, int64_t N, int32_t g,
                                   uint32_t flags, const uint16_t *A, const uint16_t *B,
                                   const float *scales, int64_t n, int32_t r, int32_t n_parts,
                                   const int64_t *part_sizes, const int32_t *adapter_ids,
                                   const uint16_t *Y, const void *workspace,
                                   size_t workspace_bytes) {
    size_t need = 0;
    int32_t st = w4a16_gemm_lora_workspace_size(M, N, K, g, flags, n_parts, r, &need);
    if (!st)
        st = check_lora_shape(N, K, n, r, n_parts);
    if (st)
        return st;
    if (!A || !B || !scales || !part_sizes || !adapter_ids || !workspace)
        return W4A16_ERR_NULL;
    int64_t sum = 0;
    for (int p = 0; p < n_parts; p++) {
        if (part_sizes[p] <= 0 || part_sizes[p] > N)
            return W4A16_ERR_SHAPE;
        sum += part_sizes[p];
    }
    if (sum != N)
        return W4A16_ERR_SHAPE;
    if (!aligned(A, 16) || !aligned(B, 16) || !aligned(scales, 4) || !aligned(adapter_ids, 4))
        return W4A16_ERR_ALIGN;
    if (workspace_bytes < need)
        return W4A16_ERR_WORKSPACE;
    // (the rules of w4a16_gemm; the GEMM's own part of the workspace comes first)
    st = w4a16_check_gemm_args(X, M, K, q_dev, s_dev, z_dev, N, g, flags, Y, workspace,
                               workspace_bytes);
    if (st)
        return st;
    if (!aligned(workspace, 16))
        return W4A16_ERR_ALIGN;
    if (overlap(adapter_ids, M * 4, Y, M * N * 2))
        return W4A16_ERR_SHAPE;
    return W4A16_OK;
}

}  // extern "C"

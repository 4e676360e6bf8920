// C ABI of the routed operators (declared in include/w4a16_routed.h): host
// checks, the gfx950 gate, and launches on the caller's stream.
#include <hip/hip_runtime.h>

#include "w4a16_routed.h"
#include "w4a16_routed.hpp"

using namespace w4a16;

namespace {

// One grouped product's geometry; expert_stride arguments are derived from it
// by the kernel.
ExpertsArgs product(const uint16_t *X, int64_t x_rows, int64_t K, const void *q, const void *s,
                    const void *z, int64_t N, int32_t g, uint32_t flags) {
    const Geom geo = make_geom(x_rows, N, K, g, flags);
    ExpertsArgs a = {};
    a.X = X;
    a.x_rows = x_rows;
    a.qd = q;
    a.sd = s;
    a.zd = z;
    a.N = (int)N;
    a.K = (int)K;
    a.g = g;
    a.lg = __builtin_ctz((unsigned)g);
    a.G = (int)geo.G;
    a.GW = (int)geo.GW;
    a.KT = (int)geo.KT;
    a.NT = (int)geo.NT;
    a.sym = geo.sym ? 1 : 0;
    return a;
}

}  // namespace

extern "C" {

int32_t w4a16_route(const void *logits, int32_t logits_dtype, int64_t T, int64_t E,
                    const float *bias, int32_t k, int32_t n_groups, int32_t topk_groups,
                    int32_t group_top, float scale, uint32_t flags, int32_t *ids, float *weights,
                    void *stream) {
    int32_t st = w4a16_check_route_args(logits, logits_dtype, T, E, bias, k, n_groups,
                                        topk_groups, group_top, scale, flags, ids, weights);
    if (st)
        return st;
    if ((st = arch_gate()))
        return st;
    (void)hipGetLastError();
    RouteArgs a;
    a.logits = logits;
    a.bias = bias;
    a.ids = ids;
    a.weights = weights;
    a.T = (int)T;
    a.E = (int)E;
    a.k = k;
    a.n_groups = n_groups;
    a.topk_groups = topk_groups;
    a.group_top = group_top;
    a.scale = scale;
    a.dtype = logits_dtype;
    a.sigmoid = (flags & W4A16_ROUTE_SIGMOID) ? 1 : 0;
    a.renormalize = (flags & W4A16_ROUTE_RENORMALIZE) ? 1 : 0;
    return finish_launch("w4a16_route", launch_route(a, stream));
}

int32_t w4a16_experts(const uint16_t *X, int64_t T, int64_t K, const int32_t *ids,
                      const float *weights, int32_t k, int64_t E, const void *gate_up_q,
                      const void *gate_up_s, const void *gate_up_z, int64_t I,
                      const void *down_q, const void *down_s, const void *down_z, int64_t D,
                      int32_t g, uint32_t flags, uint16_t *Y, void *workspace,
                      size_t workspace_bytes, void *stream) {
    int32_t st = w4a16_check_experts_args(X, T, K, ids, weights, k, E, gate_up_q, gate_up_s,
                                          gate_up_z, I, down_q, down_s, down_z, D, g, flags, Y,
                                          workspace, workspace_bytes);
    if (st)
        return st;
    if ((st = arch_gate()))
        return st;
    (void)hipGetLastError();
    const ExpertsPlan p = plan_experts(T, k, K, I, D, E, g, flags);
    char *ws = (char *)workspace;
    ExpertTile *tiles = (ExpertTile *)(ws + p.tiles_off);
    int32_t *used = (int32_t *)(ws + p.used_off);
    int32_t *perm = (int32_t *)(ws + p.perm_off);
    int32_t *place = (int32_t *)(ws + p.place_off);
    uint16_t *h = (uint16_t *)(ws + p.h_off);
    float *P = (float *)(ws + p.p_off);
    const int R = (int)(T * k);
    const bool bf = (flags & W4A16_BF16) != 0;
    int e = 0;
    if (!p.direct)
        e = launch_expert_plan(ids, R, (int)E, p.bm, (int)p.tiles, tiles, used, perm, place, stream);
    ExpertsArgs gu = product(X, T, K, gate_up_q, gate_up_s, gate_up_z, I, g, flags);
    ExpertsArgs dn = product(h, R, I, down_q, down_s, down_z, D, g, flags);
    gu.Y = h;
    dn.Y = P;
    for (ExpertsArgs *a : {&gu, &dn}) {
        a->ids = ids;
        a->perm = perm;
        a->tiles = tiles;
        a->tiles_used = used;
        a->R = R;
        a->E = (int)E;
        a->k = k;
        a->direct = p.direct;
    }
    if (p.one) {
        const auto one = bf ? launch_experts_one_bf16 : launch_experts_one;
        dn.Y = Y;
        e = one(gu, gu, weights, true, stream);
        if (!e)
            e = one(dn, gu, weights, false, stream);
        return finish_launch("w4a16_experts", e);
    }
    const auto launch = p.large ? (bf ? launch_experts_large_bf16 : launch_experts_large)
                                : (bf ? launch_experts_small_bf16 : launch_experts_small);
    if (!e)
        e = launch(gu, p, true, stream);
    if (!e)
        e = launch(dn, p, false, stream);
    if (!e) {
        CombineArgs c;
        c.P = P;
        c.ids = ids;
        c.weights = weights;
        c.place = p.direct ? nullptr : place;
        c.Y = Y;
        c.T = T;
        c.D = D;
        c.k = k;
        c.E = (int)E;
        c.bf16 = bf ? 1 : 0;
        c.gu = gu;
        c.dn = dn;
        e = launch_experts_combine(c, stream);
    }
    return finish_launch("w4a16_experts", e);
}

int32_t w4a16_gemm_lora(const uint16_t *X, int64_t M, int64_t K, const void *q_dev,
                        const void *s_dev, const void *z_dev, int64_t N, int32_t g,
                        uint32_t flags, const uint16_t *A, const uint16_t *B,
                        const float *scales, int64_t n, int32_t r, int32_t n_parts,
                        const int64_t *part_sizes, const int32_t *adapter_ids, uint16_t *Y,
                        void *workspace, size_t workspace_bytes, void *stream) {
    int32_t st = w4a16_check_gemm_lora_args(X, M, K, q_dev, s_dev, z_dev, N, g, flags, A, B,
                                            scales, n, r, n_parts, part_sizes, adapter_ids, Y,
                                            workspace, workspace_bytes);
    if (st)
        return st;
    if ((st = arch_gate()))
        return st;
    (void)hipGetLastError();
    const Geom geo = make_geom(M, N, K, g, flags);
    const GemmPlan plan = plan_gemm(geo, flags);
    const LoraPlan lp = plan_lora(M, n_parts, r, geo.bf16);
    char *ws = (char *)workspace + ((plan.ws_bytes + 255) & ~(size_t)255);
    LoraShrinkArgs sh;
    sh.X = X;
    sh.A = A;
    sh.scales = scales;
    sh.ids = adapter_ids;
    sh.lists = (LoraList *)ws;
    sh.S_hi = (uint16_t *)(ws + lp.s_hi_off);
    sh.S_lo = (uint16_t *)(ws + lp.s_lo_off);
    sh.F = (float *)(ws + lp.f_off);
    sh.M = M;
    sh.f_pitch = lp.f_pitch;
    sh.K = (int)K;
    sh.n = (int)n;
    sh.r = r;
    sh.parts = n_parts;
    sh.blocks = lp.blocks;
    sh.lanes = lp.lanes;
    sh.bf16 = geo.bf16 ? 1 : 0;
    LoraArgs lo;
    lo.S_hi = sh.S_hi;
    lo.S_lo = sh.S_lo;
    lo.F = sh.F;
    lo.B = B;
    lo.lists = sh.lists;
    lo.ids = adapter_ids;
    lo.n = (int)n;
    lo.f_pitch = lp.f_pitch;
    lo.r = r;
    lo.blocks = lp.blocks;
    lo.parts = n_parts;
    int64_t end = 0;
    for (int p = 0; p < kMaxParts; p++) {
        end += p < n_parts ? part_sizes[p] : 0;
        lo.part_end[p] = (int)end;
    }
    int e = launch_lora_shrink(sh, stream);
    if (!e)
        e = launch_gemm_lora(X, q_dev, s_dev, z_dev, geo, plan, lo, Y, workspace, stream);
    return finish_launch("w4a16_gemm_lora", e);
}

}  // extern "C"

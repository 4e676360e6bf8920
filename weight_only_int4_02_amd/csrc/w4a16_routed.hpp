// Internal interface of the routed operators (include/w4a16_routed.h): plans,
// kernel arguments and launchers.  Plain C++ (no HIP types), shared with the
// pure-host checks.
#pragma once
#include <stddef.h>
#include <stdint.h>

#include "w4a16_internal.hpp"

namespace w4a16 {

// ---- routing ---------------------------------------------------------------
struct RouteArgs {
    const void *logits;
    const float *bias;
    int32_t *ids;
    float *weights;
    int T, E, k, n_groups, topk_groups, group_top;
    float scale;
    int sigmoid, renormalize, dtype;
};
int launch_route(const RouteArgs &a, void *stream);

// ---- experts ---------------------------------------------------------------
// Rows (t, j) of the [T][k] slots are numbered flat, t k + j.  A tile is up to
// `bm` rows of one expert.  Up to kDirectRows rows, the workgroups find their
// tile from the ids themselves: slot y is a tile if it is the first, (bm +
// 1)-th, ... slot of its expert.  Above, a plan kernel sorts the rows by expert
// and lists the tiles.
constexpr int kDirectRows = 64;
constexpr int kMaxExperts = 1024;

struct ExpertTile {
    int32_t expert, row0, rows;   // rows row0 .. of the sorted order
    int32_t first, count;         // the expert's tiles: first .. first + count - 1
    int32_t unused[3];
};

struct ExpertsPlan {
    int one;             // a single token: the kernels of w4a16_experts_one.inc
    int direct;          // no plan kernel
    int large;           // the compute-bound kernel
    int mt;              // small kernel: 16-row activation tiles per workgroup
    int bm;              // rows per tile
    int64_t tiles;       // tiles launched (an upper bound)
    size_t used_off, tiles_off, perm_off, place_off, h_off, p_off, ws_bytes;
};
ExpertsPlan plan_experts(int64_t T, int k, int64_t K, int64_t I, int64_t D, int64_t E, int32_t g,
                         uint32_t flags);

// One grouped product.  Weight pointers are those of expert 0; `parts`
// matrices of NT 16-row tiles for each expert.
struct ExpertsArgs {
    const uint16_t *X;      // 16-bit rows of K
    const void *qd, *sd, *zd;
    void *Y;                // gated: h, 16-bit [T k][N]; else P, fp32 [T k][N]; rows in the
                            // plan's order (direct: by their flat numbers)
    const int32_t *ids;     // [R]
    const int32_t *perm;    // sorted position -> flat row (plan)
    const ExpertTile *tiles;  // (plan)
    const int32_t *tiles_used;  // (plan) how many
    int64_t x_rows;         // rows of X
    int R, E, k, direct;
    int N, K, g, G, GW, KT, NT, lg, sym;
};

struct CombineArgs {
    const float *P;         // [T k][D]
    const int32_t *ids;
    const int32_t *place;   // flat row -> its row of P (plan), or null: the same
    const float *weights;
    uint16_t *Y;            // [T][D]
    int64_t T, D;
    int k, E, bf16;
    ExpertsArgs gu, dn;     // the two products (fp16: rows whose h overflowed)
};

int launch_expert_plan(const int32_t *ids, int R, int E, int bm, int tiles_max, ExpertTile *tiles,
                       int32_t *tiles_used, int32_t *perm, int32_t *place, void *stream);
int launch_experts_small(const ExpertsArgs &a, const ExpertsPlan &p, bool gated, void *stream);
int launch_experts_small_bf16(const ExpertsArgs &a, const ExpertsPlan &p, bool gated, void *stream);
int launch_experts_large(const ExpertsArgs &a, const ExpertsPlan &p, bool gated, void *stream);
int launch_experts_large_bf16(const ExpertsArgs &a, const ExpertsPlan &p, bool gated, void *stream);
// (gu: the first product, whichever is launched)
int launch_experts_one(const ExpertsArgs &a, const ExpertsArgs &gu, const float *weights, bool gated,
                       void *stream);
int launch_experts_one_bf16(const ExpertsArgs &a, const ExpertsArgs &gu, const float *weights, bool gated,
                            void *stream);
int launch_experts_combine(const CombineArgs &a, void *stream);

// ---- adapters ----------------------------------------------------------------
constexpr int kMaxParts = 8;

// The low-rank values S of every row, in blocks of 32 ranks of one part (the
// last block of a part filled up with zeros): hi + lo in the 16-bit type,
// [parts blocks][M][32] each, and (fp16) the rows' factors [parts blocks][f_pitch].
// The distinct adapters of each 16-row tile are listed too.
struct LoraList {
    int32_t count, unused[3];
    int32_t adapter[16];
    uint32_t rows[16];       // bit j: row j of the tile names it
};
struct LoraPlan {
    int blocks;              // of 32 ranks, per part
    int lanes;               // first product: workgroups for the adapters of a row tile
    int64_t f_pitch;         // M in whole row tiles
    size_t s_hi_off, s_lo_off, f_off, bytes;   // (the lists come first)
};
LoraPlan plan_lora(int64_t M, int parts, int r, bool bf16);

// What the GEMM kernels need to add the adapters.
struct LoraArgs {
    const uint16_t *S_hi, *S_lo;
    const float *F;
    const LoraList *lists;   // [row tiles]
    const uint16_t *B;       // [n][N][r]
    const int32_t *ids;      // [M]
    int64_t f_pitch;
    int n, r, blocks, parts;
    int part_end[kMaxParts]; // first column after part p
};
struct LoraShrinkArgs {
    const uint16_t *X, *A;   // A [n][parts r][K]
    const float *scales;
    const int32_t *ids;
    uint16_t *S_hi, *S_lo;
    float *F;
    LoraList *lists;
    int64_t M, f_pitch;
    int K, n, r, parts, blocks, lanes, bf16;
};
int launch_lora_shrink(const LoraShrinkArgs &a, void *stream);
int launch_gemm_lora(const uint16_t *X, const void *q_dev, const void *s_dev, const void *z_dev,
                     const Geom &geo, const GemmPlan &plan, const LoraArgs &lora, uint16_t *Y,
                     void *workspace, void *stream);

// w4a16_api.hip: the architecture gate and the error text of this host thread
int32_t arch_gate();
int32_t finish_launch(const char *what, int err);

}  // namespace w4a16

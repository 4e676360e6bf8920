// Pure host logic of the microscaled 4-bit operators: argument checks and
// plans.  No HIP call is made here.
#include <stdint.h>

#include "w4a16_mx.h"
#include "w4a16_mx.hpp"

namespace w4a16 {

namespace {

bool aligned(const void *p, uintptr_t to) { return ((uintptr_t)p & (to - 1)) == 0; }

bool overlap(const void *a, int64_t a_bytes, const void *b, int64_t b_bytes) {
    const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
    return a0 < b0 + (uintptr_t)b_bytes && b0 < a0 + (uintptr_t)a_bytes;
}

int64_t ktiles(int64_t K) { return (K + 127) / 128; }
int64_t kslabs(int64_t K) { return (K + 511) / 512; }

int32_t check_rows(int64_t M, int64_t K, int32_t dtype) {
    if (M <= 0 || M >= (int64_t(1) << 31) || K <= 0 || K > (int64_t(1) << 24) || K % 8 != 0 ||
        M * kslabs(K) * 4 >= (int64_t(1) << 31) || dtype < W4A16_MX_F16 || dtype > W4A16_MX_F32)
        return W4A16_ERR_SHAPE;
    return W4A16_OK;
}

int32_t check_weight_shape(int64_t E, int64_t N, int64_t K) {
    if (E <= 0 || E > 1024 || N <= 0 || N >= (int64_t(1) << 22) || K <= 0 ||
        K > (int64_t(1) << 20) || K % 8 != 0)
        return W4A16_ERR_SHAPE;
    // the kernels address one matrix with 31-bit byte offsets
    if ((N + 15) / 16 * ktiles(K) * 1024 >= (int64_t(1) << 31))
        return W4A16_ERR_SHAPE;
    return W4A16_OK;
}

int64_t weight_q_bytes(int64_t E, int64_t N, int64_t K) { return E * ((N + 15) / 16) * ktiles(K) * 1024; }
int64_t weight_s_bytes(int64_t E, int64_t N, int64_t K) { return E * ((N + 15) / 16) * kslabs(K) * 256; }

bool overlaps_weight(const void *p, int64_t bytes, const void *q_dev, const void *s_dev, int64_t E, int64_t N,
                     int64_t K) {
    return overlap(p, bytes, q_dev, weight_q_bytes(E, N, K)) || overlap(p, bytes, s_dev, weight_s_bytes(E, N, K));
}

// The rules that a product has with and without experts.
int32_t check_product(const void *X, const uint8_t *x_scales, int32_t x_dtype, int64_t T,
                      int64_t K, int64_t R, int64_t E, const void *q_dev, const void *s_dev,
                      int64_t N, int32_t y_dtype, const void *Y) {
    const int32_t st = check_weight_shape(E, N, K);
    if (st)
        return st;
    if (T <= 0 || R <= 0 || T >= (int64_t(1) << 31) || R >= (int64_t(1) << 31) ||
        (y_dtype != W4A16_MX_F16 && y_dtype != W4A16_MX_BF16) || (!x_scales && x_dtype != y_dtype))
        return W4A16_ERR_SHAPE;
    // the activations too are addressed with 31-bit byte offsets
    const int64_t x_bytes = x_scales ? T * kslabs(K) * 256 : T * K * 2;
    if (x_bytes >= (int64_t(1) << 31))
        return W4A16_ERR_SHAPE;
    if (!X || !q_dev || !s_dev || !Y)
        return W4A16_ERR_NULL;
    if (!aligned(X, 16) || !aligned(q_dev, 16) || !aligned(s_dev, 16) || !aligned(Y, 16) ||
        !aligned(x_scales, 16))
        return W4A16_ERR_ALIGN;
    if (overlap(X, x_bytes, Y, R * N * 2) ||
        (x_scales && overlap(x_scales, T * kslabs(K) * 16, Y, R * N * 2)) ||
        overlaps_weight(Y, R * N * 2, q_dev, s_dev, E, N, K))
        return W4A16_ERR_SHAPE;
    return W4A16_OK;
}

}  // namespace

bool weight_overlaps(const void *codes, const void *scales, int64_t E, int64_t N, int64_t K,
                     const void *q_dev, const void *s_dev) {
    const int64_t rows = E * N * kslabs(K);
    return overlaps_weight(codes, rows * 256, q_dev, s_dev, E, N, K) ||
           overlaps_weight(scales, rows * 16, q_dev, s_dev, E, N, K) ||
           overlap(q_dev, weight_q_bytes(E, N, K), s_dev, weight_s_bytes(E, N, K));
}

// The large kernel's output tiles: workgroups that share a compute unit, whether K
// may be split over workgroups, and microseconds: of a stage (64 columns of
// 16-bit activations, 256 of MXFP4) what a workgroup needs at least (`alone`: the
// copies' latency) and what each adds to a busy compute unit (`work`), and what a
// tile takes besides (`tile`: its results' way out).  Fitted to 2048 x 22016 x
// 4096, 61 .. 512 rows of the 7B model's projections, and 4096 tokens over 64 experts.
struct MxTileCost {
    int shape, bm, bn, occ, split;
    double alone, work, tile;
};
const MxTileCost kTiles16[] = {{MX_64x128, 64, 128, 3, 1, 0.40, 0.25, 1.0}, {MX_64x256, 64, 256, 2, 1, 0.52, 0.44, 1.0},
                               {MX_128x128, 128, 128, 2, 1, 0.55, 0.47, 1.5}, {MX_128x256, 128, 256, 2, 1, 0.92, 0.81, 1.0},
                               {MX_256x256, 256, 256, 1, 0, 1.5, 1.5, 2.8}};
const MxTileCost kTiles4[] = {{MX_64x128, 64, 128, 2, 1, 0.57, 0.30, 2.5}, {MX_128x128, 128, 128, 2, 1, 0.84, 0.45, 3.9},
                              {MX_128x256, 128, 256, 1, 0, 0.98, 0.98, 6.7}, {MX_256x256, 256, 256, 1, 0, 1.87, 1.87, 5.0}};

MxPlan plan_mx(int64_t R, int64_t E, int64_t N, int64_t K, bool fp4, bool grouped) {
    MxPlan p = {};
    const int64_t hit = R < E ? R : E;      // matrices with rows, if the rows are spread evenly,
    const double per = (double)R / (double)hit;   // and the rows of each
    const int64_t nt = (N + 15) / 16, kt = ktiles(K);
    p.splits = 1;
    // Few rows: the memory-bound kernel, as far as its traffic of activations (all
    // rows once for every nb column tiles) stays beside that of the weights.  Both
    // measured at 48 and 61 rows: 4096 x 4096 8.7 .. 10.2 us against 13.8 .. 14.5 in
    // bf16, 22016 x 4096 24.1 .. 28.7 against 26.0 .. 26.3; quantized 6.3 .. 7.3 against
    // 10.0 .. 11.8 and 17.2 .. 18.9 against 13.5.  A long K leaves more to the splits of
    // the large kernel (61 x 4096 x 11008: 23.4 against 20.0).
    if (grouped) {
        // (8 experts of 4000 x 4096, 10 rows each in bf16: 22 us against 33)
        p.large = per > (fp4 ? 6 : 8) && (fp4 || per > 24 || hit * nt > 4096);
        p.mt = per > 8 ? 2 : 1;
        p.nb = 4;
        const int64_t blocks = (nt + 3) / 4 * hit;
        p.ks = blocks < 1000 && p.mt == 1 ? 4 : blocks < 4096 ? 2 : 1;
    } else {
        p.large = R > 64 || (R > 32 && ((double)R * nt * kt > (fp4 ? 1.6e6 : 2.1e6) || (R > 48 && kt > 64)));
        p.mt = (int)((R + 15) / 16);
        p.nb = nt <= 256 ? 1 : nt <= 512 ? 2 : 3;
        p.ks = p.mt <= 2 && ((p.mt == 2 && !fp4) || (p.nb == 1 && kt >= 64)) ? 8 : 4;
    }
    if (!p.large)
        return p;
    const int64_t stages = fp4 ? (K + 255) / 256 : (K + 63) / 64;
    const double most_bytes = 512.0 * (1 << 20);   // of splits' sums
    double best = 1e30;
    const MxTileCost *tiles = fp4 ? kTiles4 : kTiles16;
    const int n = fp4 ? 4 : 5;
    for (int k = 0; k < n; k++) {
        const MxTileCost &t = tiles[k];
        if (fp4 && grouped && t.shape == MX_128x256 && kt < 2)
            continue;    // (its ring of four stages has scales of three slabs only)
        // (a matrix's last tile is half full on average)
        const double rows = grouped ? hit * (per <= t.bm / 2 ? 1.0 : per / t.bm + 0.5) : (double)((R + t.bm - 1) / t.bm);
        const double items = rows * (double)((N + t.bn - 1) / t.bn);
        for (int64_t sp = 1; sp <= 16; sp++) {
            const double sum_bytes = (double)sp * R * N * 8;
            if (sp > 1 && (grouped || !t.split || sp * 2 > stages || sum_bytes > 2 * most_bytes))
                break;
            const double each = (double)((stages + sp - 1) / sp);
            const double rounds = (int64_t)((items * sp + 256 * t.occ - 1) / (256 * t.occ));
            const double fill = items * sp / 256;
            // (workgroups that share a compute unit take up its idle ends)
            const double deep = fill <= t.occ || t.occ == 1 ? (double)(int64_t)(fill + 0.999) : fill + 0.25;
            // (finding an expert's tile, where workgroups do not stay)
            const double tile = !grouped ? t.tile : t.shape == MX_128x256 && fp4 ? 5.5 : t.split ? t.tile + 1.5 : t.tile;
            const double alone = (each * t.alone + tile) * rounds, work = (each * t.work + tile) * deep;
            double us = alone > work ? alone : work;
            if (sp > 1)
                us += 2.0 + sum_bytes / 6e6;
            if (us < best) {
                best = us;
                p.shape = t.shape;
                p.splits = (int)sp;
            }
        }
    }
    p.ws_bytes = p.splits > 1 ? (size_t)(p.splits * R * ((N + 3) / 4 * 4) * 4) : 0;
    return p;
}

}  // namespace w4a16

using namespace w4a16;

extern "C" {

int32_t w4a16_mx_check_quantize_args(const void *X, int32_t dtype, int64_t M, int64_t K,
                                     const uint8_t *codes, const uint8_t *scales) {
    const int32_t st = check_rows(M, K, dtype);
    if (st)
        return st;
    if (!X || !codes || !scales)
        return W4A16_ERR_NULL;
    if (!aligned(X, 16) || !aligned(codes, 16) || !aligned(scales, 16))
        return W4A16_ERR_ALIGN;
    const int64_t x_bytes = M * K * (dtype == W4A16_MX_F32 ? 4 : 2), slabs = M * kslabs(K);
    if (overlap(X, x_bytes, codes, slabs * 256) || overlap(X, x_bytes, scales, slabs * 16) ||
        overlap(codes, slabs * 256, scales, slabs * 16))
        return W4A16_ERR_SHAPE;
    return W4A16_OK;
}

int32_t w4a16_mx_check_dequantize_args(const uint8_t *codes, const uint8_t *scales, int64_t M,
                                       int64_t K, int32_t dtype, const void *Y) {
    return w4a16_mx_check_quantize_args(Y, dtype, M, K, codes, scales);
}

int32_t w4a16_mx_weight_size(int64_t E, int64_t N, int64_t K, size_t *q_bytes, size_t *s_bytes) {
    if (!q_bytes || !s_bytes)
        return W4A16_ERR_NULL;
    const int32_t st = check_weight_shape(E, N, K);
    if (st)
        return st;
    *q_bytes = (size_t)weight_q_bytes(E, N, K);
    *s_bytes = (size_t)weight_s_bytes(E, N, K);
    return W4A16_OK;
}

int32_t w4a16_mx_check_weight_args(const uint8_t *codes, const uint8_t *scales, int64_t E,
                                   int64_t N, int64_t K, const void *q_dev, const void *s_dev) {
    const int32_t st = check_weight_shape(E, N, K);
    if (st)
        return st;
    if (!codes || !scales || !q_dev || !s_dev)
        return W4A16_ERR_NULL;
    if (!aligned(codes, 16) || !aligned(scales, 16) || !aligned(q_dev, 16) || !aligned(s_dev, 16))
        return W4A16_ERR_ALIGN;
    return W4A16_OK;
}

int32_t w4a16_mx_check_gemm_args(const void *X, const uint8_t *x_scales, int32_t x_dtype,
                                 int64_t M, int64_t K, const void *q_dev, const void *s_dev,
                                 int64_t N, int32_t y_dtype, const void *Y,
                                 const void *workspace, size_t workspace_bytes) {
    const int32_t st = check_product(X, x_scales, x_dtype, M, K, M, 1, q_dev, s_dev, N, y_dtype, Y);
    if (st)
        return st;
    const size_t need = plan_mx(M, 1, N, K, x_scales != nullptr, false).ws_bytes;
    if (!need)
        return W4A16_OK;
    if (!workspace)
        return W4A16_ERR_NULL;
    if (!aligned(workspace, 16))
        return W4A16_ERR_ALIGN;
    if (workspace_bytes < need)
        return W4A16_ERR_WORKSPACE;
    const int64_t ws = (int64_t)need, x_bytes = x_scales ? M * kslabs(K) * 256 : M * K * 2;
    if (overlap(workspace, ws, X, x_bytes) || overlap(workspace, ws, Y, M * N * 2) ||
        (x_scales && overlap(workspace, ws, x_scales, M * kslabs(K) * 16)) ||
        overlaps_weight(workspace, ws, q_dev, s_dev, 1, N, K))
        return W4A16_ERR_SHAPE;
    return W4A16_OK;
}

int32_t w4a16_mx_gemm_workspace_size(int64_t M, int64_t N, int64_t K, int32_t quantized,
                                     size_t *bytes) {
    if (!bytes)
        return W4A16_ERR_NULL;
    const int32_t st = check_weight_shape(1, N, K);
    if (st || M <= 0 || M >= (int64_t(1) << 31))
        return st ? st : W4A16_ERR_SHAPE;
    *bytes = plan_mx(M, 1, N, K, quantized != 0, false).ws_bytes;
    return W4A16_OK;
}

int32_t w4a16_mx_kernel(int64_t R, int64_t E, int64_t N, int64_t K, int32_t quantized,
                        int32_t grouped, int32_t *form) {
    if (!form)
        return W4A16_ERR_NULL;
    const int32_t st = check_weight_shape(E, N, K);
    if (st || R <= 0 || R >= (int64_t(1) << 31) || (!grouped && E != 1))
        return st ? st : W4A16_ERR_SHAPE;
    const MxPlan p = plan_mx(R, E, N, K, quantized != 0, grouped != 0);
    form[0] = p.large;
    form[1] = p.large ? p.shape : p.mt;
    form[2] = p.large ? p.splits : p.nb;
    form[3] = p.large ? 0 : p.ks;
    return W4A16_OK;
}

int32_t w4a16_mx_check_grouped_gemm_args(const void *X, const uint8_t *x_scales, int32_t x_dtype,
                                         int64_t T, int64_t K, const int32_t *rows, int64_t R,
                                         const int32_t *offsets, int64_t E, const void *q_dev,
                                         const void *s_dev, int64_t N, int32_t y_dtype,
                                         const void *Y) {
    const int32_t st = check_product(X, x_scales, x_dtype, T, K, R, E, q_dev, s_dev, N, y_dtype, Y);
    if (st)
        return st;
    if (!offsets)
        return W4A16_ERR_NULL;
    if (!rows && T != R)
        return W4A16_ERR_SHAPE;
    if (!aligned(rows, 4) || !aligned(offsets, 4))
        return W4A16_ERR_ALIGN;
    if ((rows && overlap(rows, R * 4, Y, R * N * 2)) || overlap(offsets, (E + 1) * 4, Y, R * N * 2))
        return W4A16_ERR_SHAPE;
    return W4A16_OK;
}

}  // extern "C"

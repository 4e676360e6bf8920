// C ABI of the microscaled 4-bit operators (declared in include/w4a16_mx.h):
// host checks, the gfx950 gate, and launches on the caller's stream.
#include <hip/hip_runtime.h>

#include "w4a16_mx.h"
#include "w4a16_mx.hpp"
#include "w4a16_routed.hpp"

using namespace w4a16;

namespace {

// Runs `launch` where the host checks passed (their status `st`) on a gfx950.
template <typename F>
int32_t enqueue(const char *what, int32_t st, F launch) {
    if (st || (st = arch_gate()))
        return st;
    (void)hipGetLastError();
    return finish_launch(what, launch());
}

int run_product(const void *X, const uint8_t *x_scales, int32_t x_dtype, int64_t T, int64_t K,
                const int32_t *rows, int64_t R, const int32_t *offsets, int64_t E,
                const void *q_dev, const void *s_dev, int64_t N, int32_t y_dtype, void *Y,
                void *workspace, void *stream) {
    MxArgs a;
    a.X = X;
    a.xs = x_scales;
    a.rows = rows;
    a.offsets = offsets;
    a.qd = q_dev;
    a.sd = s_dev;
    a.Y = Y;
    a.T = T;
    a.R = R;
    a.E = (int)E;
    a.N = (int)N;
    a.K = (int)K;
    a.KT = (int)((K + 127) / 128);
    a.NT = (int)((N + 15) / 16);
    a.KG = (a.KT + 3) / 4;
    const MxPlan p = plan_mx(R, E, N, K, x_scales != nullptr, offsets != nullptr);
    a.part = (float *)workspace;
    a.splits = p.splits;
    a.NP = (int)((N + 3) / 4 * 4);
    const int x = x_scales ? MX_X_FP4 : x_dtype == W4A16_MX_BF16 ? MX_X_BF16 : MX_X_F16;
    const bool ybf = y_dtype == W4A16_MX_BF16;
    return p.large ? launch_mx_large(a, p, x, ybf, stream) : launch_mx_small(a, p, x, ybf, stream);
}

}  // namespace

extern "C" {

int32_t w4a16_mx_quantize(const void *X, int32_t dtype, int64_t M, int64_t K, uint8_t *codes,
                          uint8_t *scales, void *stream) {
    return enqueue("w4a16_mx_quantize", w4a16_mx_check_quantize_args(X, dtype, M, K, codes, scales),
                   [&] { return launch_mx_quantize(X, dtype, M, K, codes, scales, stream); });
}

int32_t w4a16_mx_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t M, int64_t K,
                            int32_t dtype, void *Y, void *stream) {
    return enqueue("w4a16_mx_dequantize",
                   w4a16_mx_check_dequantize_args(codes, scales, M, K, dtype, Y),
                   [&] { return launch_mx_dequantize(codes, scales, M, K, dtype, Y, stream); });
}

int32_t w4a16_mx_weight(const uint8_t *codes, const uint8_t *scales, int64_t E, int64_t N,
                        int64_t K, void *q_dev, void *s_dev, void *stream) {
    int32_t st = w4a16_mx_check_weight_args(codes, scales, E, N, K, q_dev, s_dev);
    if (!st && weight_overlaps(codes, scales, E, N, K, q_dev, s_dev))
        st = W4A16_ERR_SHAPE;
    return enqueue("w4a16_mx_weight", st,
                   [&] { return launch_mx_weight(codes, scales, E, N, K, q_dev, s_dev, stream); });
}

int32_t w4a16_mx_gemm(const void *X, const uint8_t *x_scales, int32_t x_dtype, int64_t M,
                      int64_t K, const void *q_dev, const void *s_dev, int64_t N,
                      int32_t y_dtype, void *Y, void *workspace, size_t workspace_bytes,
                      void *stream) {
    return enqueue("w4a16_mx_gemm",
                   w4a16_mx_check_gemm_args(X, x_scales, x_dtype, M, K, q_dev, s_dev, N, y_dtype, Y,
                                            workspace, workspace_bytes),
                   [&] {
                       return run_product(X, x_scales, x_dtype, M, K, nullptr, M, nullptr, 1, q_dev,
                                          s_dev, N, y_dtype, Y, workspace, stream);
                   });
}

int32_t w4a16_mx_grouped_gemm(const void *X, const uint8_t *x_scales, int32_t x_dtype, int64_t T,
                              int64_t K, const int32_t *rows, int64_t R, const int32_t *offsets,
                              int64_t E, const void *q_dev, const void *s_dev, int64_t N,
                              int32_t y_dtype, void *Y, void *stream) {
    return enqueue("w4a16_mx_grouped_gemm",
                   w4a16_mx_check_grouped_gemm_args(X, x_scales, x_dtype, T, K, rows, R, offsets, E,
                                                    q_dev, s_dev, N, y_dtype, Y),
                   [&] {
                       return run_product(X, x_scales, x_dtype, T, K, rows, R, offsets, E, q_dev,
                                          s_dev, N, y_dtype, Y, nullptr, stream);
                   });
}

}  // extern "C"

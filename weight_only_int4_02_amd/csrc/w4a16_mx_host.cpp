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

int32_t check_rows(int64_t M, int64_t K, int32_t dtype) {
    if (M <= 0 || M >= (int64_t(1) << 31) || K <= 0 || K > (int64_t(1) << 24) || K % 8 != 0 ||
        M * ktiles(K) >= (int64_t(1) << 31) || dtype < W4A16_MX_F16 || dtype > W4A16_MX_F32)
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
    const int64_t x_bytes = x_scales ? T * ktiles(K) * 64 : T * K * 2;
    if (x_bytes >= (int64_t(1) << 31))
        return W4A16_ERR_SHAPE;
    if (!X || !q_dev || !s_dev || !Y)
        return W4A16_ERR_NULL;
    if (!aligned(X, 16) || !aligned(q_dev, 16) || !aligned(s_dev, 16) || !aligned(Y, 16) ||
        !aligned(x_scales, 4))
        return W4A16_ERR_ALIGN;
    if (overlap(X, x_bytes, Y, R * N * 2) ||
        (x_scales && overlap(x_scales, T * ktiles(K) * 4, Y, R * N * 2)))
        return W4A16_ERR_SHAPE;
    return W4A16_OK;
}

}  // namespace

MxPlan plan_mx(int64_t R, int64_t E, int64_t N, int64_t K, bool fp4) {
    (void)fp4;
    MxPlan p = {};
    const int64_t per = (R + E - 1) / E;   // rows per matrix, on average
    const int64_t nt = (N + 15) / 16, kt = ktiles(K);
    p.large = per > (E > 1 ? 32 : 64);
    p.mt = per > 32 ? 4 : per > 16 ? 2 : 1;
    p.nb = p.mt == 1 ? 1 : 2;
    // waves along K until the chip has about 16 waves a compute unit
    const int64_t hit = R < E ? R : E;
    const int64_t waves = (nt + p.nb - 1) / p.nb * hit;
    p.ks = 1;
    while (p.ks < 8 && waves * p.ks < 4096 && p.ks * 4 <= kt)
        p.ks *= 2;
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
    if (!aligned(X, 16) || !aligned(codes, 16) || !aligned(scales, 4))
        return W4A16_ERR_ALIGN;
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
    const int64_t nt = (N + 15) / 16, kt = ktiles(K);
    *q_bytes = (size_t)(E * nt * kt * 1024);
    *s_bytes = (size_t)(E * nt * ((kt + 3) / 4) * 256);
    return W4A16_OK;
}

int32_t w4a16_mx_check_weight_args(const uint8_t *codes, const uint8_t *scales, int64_t E,
                                   int64_t N, int64_t K, const void *q_dev, const void *s_dev) {
    const int32_t st = check_weight_shape(E, N, K);
    if (st)
        return st;
    if (!codes || !scales || !q_dev || !s_dev)
        return W4A16_ERR_NULL;
    if (!aligned(codes, 16) || !aligned(scales, 4) || !aligned(q_dev, 16) || !aligned(s_dev, 16))
        return W4A16_ERR_ALIGN;
    return W4A16_OK;
}

int32_t w4a16_mx_check_gemm_args(const void *X, const uint8_t *x_scales, int32_t x_dtype,
                                 int64_t M, int64_t K, const void *q_dev, const void *s_dev,
                                 int64_t N, int32_t y_dtype, const void *Y) {
    return check_product(X, x_scales, x_dtype, M, K, M, 1, q_dev, s_dev, N, y_dtype, Y);
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

/*
 * w4a16_mx.h -- C ABI of the microscaled 4-bit operators of libw4a16.so:
 * quantization to MXFP4, products of activations with MXFP4 weights, and
 * products grouped by expert.  Conventions and status codes are those of
 * w4a16.h (the caller owns every buffer, arguments are checked on the host
 * before any launch, work is enqueued on `stream`, nothing is allocated).
 *
 * MXFP4 (Open Compute Project, "Microscaling Formats", version 1.0): blocks of
 * 32 consecutive columns of a row.  An element is E2M1 (sign, and one of 0, 0.5,
 * 1, 1.5, 2, 3, 4, 6 by its number 0..7), a block's scale E8M0: byte b stands
 * for 2^(b - 127), 255 for NaN.  A value is element times scale.
 *
 * Rows are held in whole slabs of 512 columns, KG = ceil(K / 512):
 *   codes   uint8 [4 KG][rows][64], of 128 columns the 64 bytes of a row, two
 *           columns a byte, the first in the low half;
 *   scales  uint8 [KG][rows][16], the slab's 16 blocks of a row.
 * Columns from K on hold zeros (their scales: any but 255).  K is a multiple of
 * 8 (the last block may be partial).
 *
 * The device layout of a weight of N rows, NT = ceil(N / 16), KT = ceil(K / 128):
 *   codes   [2 KT][NT][2][16][16]: of 64 columns and 16 rows, the 16 bytes of
 *           each row's first block, then of its second;
 *   scales  [KG][16 NT][16]: of 512 columns the 16 scales of each row.
 * (What a tile of the products takes of 64 columns is one run of memory.)
 * Rows past N and columns past K hold zeros (scales: 127).
 */
#ifndef W4A16_MX_H
#define W4A16_MX_H

#include "w4a16.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of plain tensors. */
#define W4A16_MX_F16  0
#define W4A16_MX_BF16 1
#define W4A16_MX_F32  2

/* X [M][K] -> codes, scales.  A block of largest magnitude a has the scale
 * 2^e, e = floor(log2 a) - 2, held within -127 .. 127 (a = 0: -127); its
 * elements are x / 2^e rounded to the nearest E2M1 value, of two to the one
 * with the even number, a magnitude beyond 6 to 6.  The sign of a zero is
 * kept.  A block that holds an infinity or a NaN is NaN throughout: scale 255,
 * codes 0.
 * Limits: M < 2^31, K <= 2^24, 4 M KG < 2^31.
 * Errors: W4A16_ERR_NULL, W4A16_ERR_SHAPE (also where two of the buffers
 * overlap), W4A16_ERR_ALIGN (16 bytes each), W4A16_ERR_ARCH, W4A16_ERR_HIP. */
int32_t w4a16_mx_quantize(const void *X, int32_t dtype, int64_t M, int64_t K, uint8_t *codes,
                          uint8_t *scales, void *stream);
int32_t w4a16_mx_check_quantize_args(const void *X, int32_t dtype, int64_t M, int64_t K,
                                     const uint8_t *codes, const uint8_t *scales);

/* codes, scales -> Y [M][K], each value rounded once to Y's type (exact in bf16
 * and fp32 but for magnitudes past the type's largest, which are infinite).
 * Limits and errors as w4a16_mx_quantize. */
int32_t w4a16_mx_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t M, int64_t K,
                            int32_t dtype, void *Y, void *stream);
int32_t w4a16_mx_check_dequantize_args(const uint8_t *codes, const uint8_t *scales, int64_t M,
                                       int64_t K, int32_t dtype, const void *Y);

/* E matrices [N][K] (codes and scales as above, of E N rows) -> the device
 * layout, one matrix after the other; w4a16_mx_weight_size has the bytes of all E.
 * Limits: 1 <= E <= 1024, N < 2^22, K <= 2^20, one matrix's codes below 2 GiB.
 * A result that overlaps the other or an input is refused too (W4A16_ERR_SHAPE),
 * by w4a16_mx_weight itself: w4a16_mx_check_weight_args does not look at that. */
int32_t w4a16_mx_weight_size(int64_t E, int64_t N, int64_t K, size_t *q_bytes, size_t *s_bytes);
int32_t w4a16_mx_weight(const uint8_t *codes, const uint8_t *scales, int64_t E, int64_t N,
                        int64_t K, void *q_dev, void *s_dev, void *stream);
int32_t w4a16_mx_check_weight_args(const uint8_t *codes, const uint8_t *scales, int64_t E,
                                   int64_t N, int64_t K, const void *q_dev, const void *s_dev);

/* Y [M][N] = X [M][K] . W^T, with fp32 sums, rounded once.
 *   x_scales NULL: X is 16-bit (x_dtype), and a weight enters as its value
 *     rounded to that type (exact in bf16 but for magnitudes past its largest; in
 *     fp16 for scales of 2^-23 .. 2^13, infinite for larger values than it has);
 *   else X and x_scales are MXFP4 rows, multiplied by the matrix cores' scaled
 *     instruction.
 * y_dtype: fp16 or bf16; of a 16-bit X, its own.
 * workspace: w4a16_mx_gemm_workspace_size bytes (no fill needed, NULL where
 * that is 0; quantized: x_scales given): fp32 sums of parts of K.  Calls that may
 * run at the same time need separate ones.
 * Limits: those of w4a16_mx_weight, M < 2^31, X below 2 GiB.
 * Errors: W4A16_ERR_NULL, W4A16_ERR_SHAPE (also where Y or the workspace
 * overlaps the other, X with its scales or the weight), W4A16_ERR_ALIGN (16 bytes
 * each), W4A16_ERR_WORKSPACE, W4A16_ERR_ARCH, W4A16_ERR_HIP. */
int32_t w4a16_mx_gemm_workspace_size(int64_t M, int64_t N, int64_t K, int32_t quantized,
                                     size_t *bytes);
int32_t w4a16_mx_gemm(const void *X, const uint8_t *x_scales, int32_t x_dtype, int64_t M,
                      int64_t K, const void *q_dev, const void *s_dev, int64_t N,
                      int32_t y_dtype, void *Y, void *workspace, size_t workspace_bytes,
                      void *stream);
int32_t w4a16_mx_check_gemm_args(const void *X, const uint8_t *x_scales, int32_t x_dtype,
                                 int64_t M, int64_t K, const void *q_dev, const void *s_dev,
                                 int64_t N, int32_t y_dtype, const void *Y, const void *workspace,
                                 size_t workspace_bytes);

/* The products of E experts over rows that lie sorted by expert:
 *   Y[i] = X[rows[i]] . W_e^T   for offsets[e] <= i < offsets[e + 1]
 * with rows NULL: X[i].  X [T][K] as in w4a16_mx_gemm, rows int32 [R],
 * offsets int32 [E + 1], Y [R][N]; with rows NULL, T = R.
 * offsets rise from 0 or more to R or less.  Rows of Y before the first and
 * from the last offset on stay as they are.  An index outside 0 .. T - 1 counts
 * as a row of zeros (NaN comes of it where the weight is not finite).  Offsets live on the device and are not checked: values
 * outside 0 .. R are taken as 0 or R, and where they fall, which rows are
 * written, and with what, is not defined (nothing outside Y is).
 * Limits: those of w4a16_mx_gemm, R < 2^31.
 * Errors: as w4a16_mx_gemm (rows and offsets aligned to 4 bytes, and Y must
 * not overlap them). */
int32_t w4a16_mx_grouped_gemm(const void *X, const uint8_t *x_scales, int32_t x_dtype, int64_t T,
                              int64_t K, const int32_t *rows, int64_t R, const int32_t *offsets,
                              int64_t E, const void *q_dev, const void *s_dev, int64_t N,
                              int32_t y_dtype, void *Y, void *stream);
int32_t w4a16_mx_check_grouped_gemm_args(const void *X, const uint8_t *x_scales, int32_t x_dtype,
                                         int64_t T, int64_t K, const int32_t *rows, int64_t R,
                                         const int32_t *offsets, int64_t E, const void *q_dev,
                                         const void *s_dev, int64_t N, int32_t y_dtype,
                                         const void *Y);

/* The kernel that a product of R rows runs (pure host): form[0] 0 the one for few
 * rows, then form[1..3] its row tiles of 16, column tiles of 16 and waves along K;
 * 1 the one for many, then form[1] its output tile (0 64 x 128, 1 64 x 256, 2
 * 128 x 128, 3 128 x 256, 4 256 x 256) and form[2] the parts of K.  quantized:
 * MXFP4 activations; grouped: w4a16_mx_grouped_gemm over E matrices (else E = 1). */
int32_t w4a16_mx_kernel(int64_t R, int64_t E, int64_t N, int64_t K, int32_t quantized,
                        int32_t grouped, int32_t *form);

#ifdef __cplusplus
}
#endif
#endif /* W4A16_MX_H */

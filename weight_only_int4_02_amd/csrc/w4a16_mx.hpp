// Internal interface of the microscaled 4-bit operators (include/w4a16_mx.h):
// plans, kernel arguments and launchers.  Plain C++ (no HIP types), shared
// with the pure-host checks.
#pragma once
#include <stddef.h>
#include <stdint.h>

namespace w4a16 {

// What the activations are.
enum MxX { MX_X_F16 = 0, MX_X_BF16 = 1, MX_X_FP4 = 2 };

// One product: E matrices, rows sorted by matrix (a plain product has E = 1 and
// no offsets).
struct MxArgs {
    const void *X;            // 16-bit [T][K], or codes [4 KG][T][64]
    const uint8_t *xs;        // scales [KG][T][16] (codes only)
    const int32_t *rows;      // [R], or null: row i
    const int32_t *offsets;   // [E + 1], or null
    const void *qd, *sd;      // device layout, matrix 0
    void *Y;                  // [R][N]
    float *part;              // splits' sums [splits][R][NP] (splits > 1)
    int64_t T, R;
    int E, N, K, KT, NT, KG;
    int splits, NP;           // NP: N in whole groups of 4
};

// Output tiles of the large kernel.
enum MxShape { MX_64x128, MX_64x256, MX_128x128, MX_128x256, MX_256x256 };

struct MxPlan {
    int large;    // the compute-bound kernel
    // small kernel: row tiles of 16, column tiles of 16, waves along K
    int mt, nb, ks;
    int shape;    // large kernel: output tile (MxShape),
    int splits;   // and workgroups along K
    size_t ws_bytes;
};
MxPlan plan_mx(int64_t R, int64_t E, int64_t N, int64_t K, bool fp4, bool grouped);

// Whether a result of w4a16_mx_weight overlaps the other or an input.
bool weight_overlaps(const void *codes, const void *scales, int64_t E, int64_t N, int64_t K,
                     const void *q_dev, const void *s_dev);

int launch_mx_quantize(const void *X, int dtype, int64_t M, int64_t K, uint8_t *codes,
                       uint8_t *scales, void *stream);
int launch_mx_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t M, int64_t K,
                         int dtype, void *Y, void *stream);
int launch_mx_weight(const uint8_t *codes, const uint8_t *scales, int64_t E, int64_t N, int64_t K,
                     void *q_dev, void *s_dev, void *stream);
// x: an MxX; ybf: bf16 results (of 16-bit activations, their own type)
int launch_mx_small(const MxArgs &a, const MxPlan &p, int x, bool ybf, void *stream);
int launch_mx_large(const MxArgs &a, const MxPlan &p, int x, bool ybf, void *stream);

}  // namespace w4a16

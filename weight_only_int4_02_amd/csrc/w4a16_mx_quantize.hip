// MXFP4 quantization, its inverse, and the weights' device layout.  All three
// move bytes and are bound by memory.
#include <hip/hip_runtime.h>

#include "w4a16_mx_device.hpp"

namespace w4a16 {

namespace {

constexpr int kThreads = 256;
// A launch holds fewer than 2^32 threads: beyond so many workgroups they take
// several places each.
constexpr int64_t kMaxGroups = int64_t(1) << 23;

unsigned groups(int64_t places) {
    const int64_t n = (places + kThreads - 1) / kThreads;
    return (unsigned)(n < kMaxGroups ? n : kMaxGroups);
}

// Eight values as fp32.  DT: 0 fp16, 1 bf16, 2 fp32.
template <int DT>
__device__ __forceinline__ void load8(const void *x, int64_t at, float (&v)[8]) {
    if constexpr (DT == 2) {
        const f4_t a = *(const f4_t *)((const float *)x + at), b = *(const f4_t *)((const float *)x + at + 4);
#pragma unroll
        for (int i = 0; i < 4; i++)
            v[i] = a[i], v[4 + i] = b[i];
    } else {
        const u4_t w = *(const u4_t *)((const uint16_t *)x + at);
        if constexpr (DT == 1) {
#pragma unroll
            for (int i = 0; i < 4; i++) {
                v[2 * i] = __builtin_bit_cast(float, w[i] << 16);
                v[2 * i + 1] = __builtin_bit_cast(float, w[i] & 0xFFFF0000u);
            }
        } else {
            const h8_t h = __builtin_bit_cast(h8_t, w);
#pragma unroll
            for (int i = 0; i < 8; i++)
                v[i] = (float)h[i];
        }
    }
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}

// Sixteen lanes take a tile of 128 columns of one row, eight columns each; four
// neighbours share a block.  The largest magnitude is found on the bits (whose
// order is that of the magnitudes, NaN above infinity above numbers): its
// exponent field less two is the scale byte.
template <int DT>
__global__ __launch_bounds__(kThreads) void mx_quantize_kernel(const void *__restrict__ X,
                                                               uint32_t tiles, uint32_t KT, uint32_t K,
                                                               uint32_t *__restrict__ codes,
                                                               uint32_t *__restrict__ scales) {
    const uint32_t l = threadIdx.x & 15;
    // (a group of 16 lanes leaves the loop as a whole)
    for (uint32_t tile = blockIdx.x * (kThreads / 16) + threadIdx.x / 16; tile < tiles;
         tile += gridDim.x * (kThreads / 16)) {
    const uint32_t row = tile / KT, col = (tile - row * KT) * 128 + 8 * l;
    float v[8] = {};
    if (col < K)
        load8<DT>(X, (int64_t)row * K + col, v);
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const uint32_t a = __builtin_bit_cast(uint32_t, v[i]) & 0x7FFFFFFFu;
        top = a > top ? a : top;
    }
    uint32_t o = dpp<0xB1>(top);   // the neighbour, then the other pair
    top = o > top ? o : top;
    o = dpp<0x4E>(top);
    top = o > top ? o : top;
    const uint32_t field = top >> 23;
    const uint32_t byte = field == 255 ? 255 : field > 2 ? field - 2 : 0;
    const float s = __builtin_bit_cast(float, byte << 23);
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], s, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], s, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], s, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], s, 3);
    codes[(int64_t)tile * 16 + l] = byte == 255 ? 0 : w;
    // the tile's four scale bytes in one word
    uint32_t b = byte << (8 * (l >> 2));
    b |= dpp<0x124>(b);            // rotated by 4 and by 8 lanes of 16
    b |= dpp<0x128>(b);
    if (l == 0)
        scales[tile] = b;
    }
}

// The inverse: eight values a lane.
template <int DT>
__global__ __launch_bounds__(kThreads) void mx_dequantize_kernel(const uint32_t *__restrict__ codes,
                                                                 const uint32_t *__restrict__ scales,
                                                                 uint32_t tiles, uint32_t KT, uint32_t K,
                                                                 void *__restrict__ Y) {
    const uint32_t l = threadIdx.x & 15;
    for (uint32_t tile = blockIdx.x * (kThreads / 16) + threadIdx.x / 16; tile < tiles;
         tile += gridDim.x * (kThreads / 16)) {
    const uint32_t row = tile / KT, col = (tile - row * KT) * 128 + 8 * l;
    if (col >= K)
        continue;
    const uint32_t w = codes[(int64_t)tile * 16 + l];
    const float s = mx_scale(scales[tile], l >> 2);
    const int64_t at = (int64_t)row * K + col;
    if constexpr (DT == 2) {
        const f2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 0),
                   b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 1),
                   c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 2),
                   d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 3);
        *(f4_t *)((float *)Y + at) = f4_t{a.x, a.y, b.x, b.y};
        *(f4_t *)((float *)Y + at + 4) = f4_t{c.x, c.y, d.x, d.y};
    } else {
        *(u4_t *)((uint16_t *)Y + at) = mx_decode<DT == 1>(w, s);
    }
    }
}

// Rows to the device layout: one thread a block of 16 code bytes (and every
// fourth the tile's scale word), in the order of the result.
__global__ __launch_bounds__(kThreads) void mx_weight_kernel(const u4_t *__restrict__ codes,
                                                             const uint32_t *__restrict__ scales,
                                                             int64_t blocks, int N, int KT, int NT,
                                                             int KG, u4_t *__restrict__ q,
                                                             uint32_t *__restrict__ s) {
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < blocks;
         i += (int64_t)gridDim.x * kThreads) {
    const int lane = (int)(i & 63), r = lane & 15, kb = lane >> 4;
    const int64_t tile = i >> 6;                 // (e NT + nt) KT + kt
    const int64_t group = tile / KT;             // e NT + nt
    const int kt = (int)(tile - group * KT);
    const int64_t e = group / NT;
    const int n = (int)(group - e * NT) * 16 + r;
    const int64_t from = (e * N + n) * KT + kt;
    q[i] = n < N ? codes[from * 4 + kb] : u4_t{0u, 0u, 0u, 0u};
    if (kb == 0) {
        s[((group * KG + (kt >> 2)) * 16 + r) * 4 + (kt & 3)] = n < N ? scales[from] : 0x7F7F7F7Fu;
        if (kt == KT - 1)
            for (int k = kt + 1; k < 4 * KG; k++)
                s[((group * KG + (k >> 2)) * 16 + r) * 4 + (k & 3)] = 0x7F7F7F7Fu;
    }
    }
}

template <int DT>
int quantize_as(const void *X, uint32_t tiles, uint32_t KT, uint32_t K, uint8_t *codes,
                uint8_t *scales, hipStream_t st) {
    hipLaunchKernelGGL((mx_quantize_kernel<DT>), dim3(groups((int64_t)tiles * 16)), dim3(kThreads), 0, st, X,
                       tiles, KT, K, (uint32_t *)codes, (uint32_t *)scales);
    return (int)hipGetLastError();
}

template <int DT>
int dequantize_as(const uint8_t *codes, const uint8_t *scales, uint32_t tiles, uint32_t KT, uint32_t K,
                  void *Y, hipStream_t st) {
    hipLaunchKernelGGL((mx_dequantize_kernel<DT>), dim3(groups((int64_t)tiles * 16)), dim3(kThreads), 0, st,
                       (const uint32_t *)codes, (const uint32_t *)scales, tiles, KT, K, Y);
    return (int)hipGetLastError();
}

}  // namespace

int launch_mx_quantize(const void *X, int dtype, int64_t M, int64_t K, uint8_t *codes,
                       uint8_t *scales, void *stream) {
    const uint32_t KT = (uint32_t)((K + 127) / 128), tiles = (uint32_t)M * KT;
    hipStream_t st = (hipStream_t)stream;
    return dtype == 0   ? quantize_as<0>(X, tiles, KT, (uint32_t)K, codes, scales, st)
           : dtype == 1 ? quantize_as<1>(X, tiles, KT, (uint32_t)K, codes, scales, st)
                        : quantize_as<2>(X, tiles, KT, (uint32_t)K, codes, scales, st);
}

int launch_mx_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t M, int64_t K,
                         int dtype, void *Y, void *stream) {
    const uint32_t KT = (uint32_t)((K + 127) / 128), tiles = (uint32_t)M * KT;
    hipStream_t st = (hipStream_t)stream;
    return dtype == 0   ? dequantize_as<0>(codes, scales, tiles, KT, (uint32_t)K, Y, st)
           : dtype == 1 ? dequantize_as<1>(codes, scales, tiles, KT, (uint32_t)K, Y, st)
                        : dequantize_as<2>(codes, scales, tiles, KT, (uint32_t)K, Y, st);
}

int launch_mx_weight(const uint8_t *codes, const uint8_t *scales, int64_t E, int64_t N, int64_t K,
                     void *q_dev, void *s_dev, void *stream) {
    const int KT = (int)((K + 127) / 128), NT = (int)((N + 15) / 16), KG = (KT + 3) / 4;
    const int64_t blocks = E * NT * KT * 64;
    hipLaunchKernelGGL(mx_weight_kernel, dim3(groups(blocks)), dim3(kThreads), 0, (hipStream_t)stream,
                       (const u4_t *)codes, (const uint32_t *)scales, blocks, (int)N, KT, NT, KG,
                       (u4_t *)q_dev, (uint32_t *)s_dev);
    return (int)hipGetLastError();
}

}  // namespace w4a16

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

unsigned groups(int64_t n) { return (unsigned)(n < kMaxGroups ? n : kMaxGroups); }

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

// A workgroup takes four rows of a slab of 512 columns: a wave 128 columns of
// each, a lane eight of one row, so that reads are runs of 1 KiB (16 bits) and the
// codes of a wave one run of 256 bytes (22016 x 4096 in bf16 47 us, 4.8 TB/s, its
// inverse 33, 6.9 with codes that the caches still hold; with four tiles of one row a
// wave 88 together).  Four neighbouring
// lanes share a block.  The largest magnitude is found on the bits (whose order is
// that of the magnitudes, NaN above infinity above numbers): its exponent field
// less two is the scale byte.
struct Place {
    uint32_t row, kt;
    bool in;
};
__device__ __forceinline__ Place place_of(uint32_t group, uint32_t M, uint32_t KG) {
    const uint32_t rows = group / KG, slab = group - rows * KG, row = 4 * rows + ((threadIdx.x >> 4) & 3);
    return {row, 4 * slab + (threadIdx.x >> 6), row < M};
}

template <int DT>
__global__ __launch_bounds__(kThreads) void mx_quantize_kernel(const void *__restrict__ X, uint32_t M,
                                                               uint32_t KG, uint32_t K, uint32_t n_groups,
                                                               uint32_t *__restrict__ codes,
                                                               uint32_t *__restrict__ scales) {
    const uint32_t l = threadIdx.x & 15;
    for (uint32_t group = blockIdx.x; group < n_groups; group += gridDim.x) {
        const Place p = place_of(group, M, KG);
        if (!p.in)                  // (whole groups of 16 lanes)
            continue;
        const uint32_t row = p.row, kt = p.kt, col = kt * 128 + 8 * l;
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
        codes[((int64_t)kt * M + row) * 16 + l] = byte == 255 ? 0 : w;
        // the tile's four scale bytes in one word
        uint32_t b = byte << (8 * (l >> 2));
        b |= dpp<0x124>(b);            // rotated by 4 and by 8 lanes of 16
        b |= dpp<0x128>(b);
        if (l == 0)
            scales[((int64_t)(kt >> 2) * M + row) * 4 + (kt & 3)] = b;
    }
}

// The inverse: eight values a lane.
template <int DT>
__global__ __launch_bounds__(kThreads) void mx_dequantize_kernel(const uint32_t *__restrict__ codes,
                                                                 const uint32_t *__restrict__ scales,
                                                                 uint32_t M, uint32_t KG, uint32_t K,
                                                                 uint32_t n_groups, void *__restrict__ Y) {
    const uint32_t l = threadIdx.x & 15;
    for (uint32_t group = blockIdx.x; group < n_groups; group += gridDim.x) {
        const Place p = place_of(group, M, KG);
        const uint32_t row = p.row, kt = p.kt, col = kt * 128 + 8 * l;
        if (!p.in || col >= K)
            continue;
        const uint32_t w = codes[((int64_t)kt * M + row) * 16 + l];
        const float s = mx_scale(scales[((int64_t)(kt >> 2) * M + row) * 4 + (kt & 3)], l >> 2);
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

// Rows to the device layout: one thread a block of 16 code bytes (and the scale
// word of every four blocks), in the order of the result.
__global__ __launch_bounds__(kThreads) void mx_weight_kernel(const u4_t *__restrict__ codes,
                                                             const uint32_t *__restrict__ scales,
                                                             int64_t blocks, int64_t rows, int N, int KT,
                                                             int NT, int KG, u4_t *__restrict__ q,
                                                             uint32_t *__restrict__ s) {
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < blocks;
         i += (int64_t)gridDim.x * kThreads) {
        // ((e 2 KT + k) NT + nt) 2 + b) 16 + r: block 2 k + b of row 16 nt + r of matrix e
        const int r = (int)(i & 15), b = (int)((i >> 4) & 1);
        const int64_t piece = i >> 5;                // (e 2 KT + k) NT + nt
        const int64_t slab = piece / NT;             // e 2 KT + k
        const int nt = (int)(piece - slab * NT), n = nt * 16 + r;
        const int64_t e = slab / (2 * KT), row = e * N + n;
        const int k = (int)(slab - e * 2 * KT), kt = k >> 1;
        q[i] = n < N ? codes[(kt * rows + row) * 4 + (k & 1) * 2 + b] : u4_t{0u, 0u, 0u, 0u};
        if (b == 0 && (k & 1) == 0) {
            uint32_t *to = s + (e * KG * NT * 16 + n) * 4;
            const int64_t step = (int64_t)NT * 64;
            to[(kt >> 2) * step + (kt & 3)] = n < N ? scales[((kt >> 2) * rows + row) * 4 + (kt & 3)] : 0x7F7F7F7Fu;
            if (kt == KT - 1)
                for (int j = kt + 1; j < 4 * KG; j++)
                    to[(j >> 2) * step + (j & 3)] = 0x7F7F7F7Fu;
        }
    }
}

template <int DT>
int quantize_as(const void *X, uint32_t M, uint32_t K, uint8_t *codes, uint8_t *scales, hipStream_t st) {
    const uint32_t KG = (K + 511) / 512, n = (M + 3) / 4 * KG;
    hipLaunchKernelGGL((mx_quantize_kernel<DT>), dim3(groups(n)), dim3(kThreads), 0, st, X, M, KG, K, n,
                       (uint32_t *)codes, (uint32_t *)scales);
    return (int)hipGetLastError();
}

template <int DT>
int dequantize_as(const uint8_t *codes, const uint8_t *scales, uint32_t M, uint32_t K, void *Y,
                  hipStream_t st) {
    const uint32_t KG = (K + 511) / 512, n = (M + 3) / 4 * KG;
    hipLaunchKernelGGL((mx_dequantize_kernel<DT>), dim3(groups(n)), dim3(kThreads), 0, st,
                       (const uint32_t *)codes, (const uint32_t *)scales, M, KG, K, n, Y);
    return (int)hipGetLastError();
}

}  // namespace

int launch_mx_quantize(const void *X, int dtype, int64_t M, int64_t K, uint8_t *codes,
                       uint8_t *scales, void *stream) {
    const uint32_t m = (uint32_t)M, k = (uint32_t)K;
    hipStream_t st = (hipStream_t)stream;
    return dtype == 0   ? quantize_as<0>(X, m, k, codes, scales, st)
           : dtype == 1 ? quantize_as<1>(X, m, k, codes, scales, st)
                        : quantize_as<2>(X, m, k, codes, scales, st);
}

int launch_mx_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t M, int64_t K,
                         int dtype, void *Y, void *stream) {
    const uint32_t m = (uint32_t)M, k = (uint32_t)K;
    hipStream_t st = (hipStream_t)stream;
    return dtype == 0   ? dequantize_as<0>(codes, scales, m, k, Y, st)
           : dtype == 1 ? dequantize_as<1>(codes, scales, m, k, Y, st)
                        : dequantize_as<2>(codes, scales, m, k, Y, st);
}

int launch_mx_weight(const uint8_t *codes, const uint8_t *scales, int64_t E, int64_t N, int64_t K,
                     void *q_dev, void *s_dev, void *stream) {
    const int KT = (int)((K + 127) / 128), NT = (int)((N + 15) / 16), KG = (KT + 3) / 4;
    const int64_t blocks = E * NT * KT * 64;
    hipLaunchKernelGGL(mx_weight_kernel, dim3(groups((blocks + kThreads - 1) / kThreads)), dim3(kThreads), 0, (hipStream_t)stream,
                       (const u4_t *)codes, (const uint32_t *)scales, blocks, E * N, (int)N, KT, NT, KG,
                       (u4_t *)q_dev, (uint32_t *)s_dev);
    return (int)hipGetLastError();
}

}  // namespace w4a16

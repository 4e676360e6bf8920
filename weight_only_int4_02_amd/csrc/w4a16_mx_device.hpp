// Device helpers shared by the microscaled 4-bit kernels.
//
// gfx950 converts between E2M1 and wider types in one instruction per pair of
// values, with the scale applied: v_cvt_scalef32_* take the scale's power of two
// from the exponent field of an fp32 register (0 there means 2^-127, 255 NaN), so
// an E8M0 byte moved to bits 23..30 is that register.  They round to nearest
// even and saturate where E2M1 is the result.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "w4a16_gemm_kernels.hpp"
#include "w4a16_mx.hpp"

namespace w4a16 {

typedef int32_t i8_t __attribute__((ext_vector_type(8)));
typedef float f16_t __attribute__((ext_vector_type(16)));
typedef uint32_t u2_t __attribute__((ext_vector_type(2)));

// Copies 16 bytes a lane to LDS at lds + 16 lane; lds is the same in all lanes.
// Out of range: zeros.  (M0 holds the address.  Its write and the s_nop are the five
// wait states that the load needs after a vector instruction wrote a scalar
// register it reads, a spilled one's reload among them.  The block names no memory:
// what it writes is read behind the barrier of a later stage only, and reads of the
// present stage may be moved past it.)
__device__ __forceinline__ void copy16(i4_t desc, uint32_t lds, uint32_t voffset, uint32_t soffset) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :: "s"(lds), "v"(voffset), "s"(desc), "s"(soffset) : "m0");
}

// Byte `b` of a register of four scales as the scale operand of a conversion.
__device__ __forceinline__ float mx_scale(uint32_t scales, uint32_t b) {
    return __builtin_bit_cast(float, ((scales >> (8 * b)) & 0xFFu) << 23);
}

// The eight values of a code word times the scale, in the 16-bit type.
template <bool BF>
__device__ __forceinline__ u4_t mx_decode(uint32_t w, float s) {
    u4_t o;
    if constexpr (BF) {
        o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0));
        o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1));
        o.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2));
        o.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3));
    } else {
        o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 0));
        o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 1));
        o.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 2));
        o.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 3));
    }
    return o;
}

// 16 x 16 results of 128 columns of two MXFP4 operands; byte 0 of sa and sb is
// the scale of the lane's block.
__device__ __forceinline__ f4_t mx_mfma16(u4_t a, u4_t b, f4_t c, uint32_t sa, uint32_t sb) {
    const i8_t A = {(int)a.x, (int)a.y, (int)a.z, (int)a.w}, B = {(int)b.x, (int)b.y, (int)b.z, (int)b.w};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(A, B, c, 4, 4, 0, (int)sa, 0, (int)sb);
}

// 32 x 32 results of 64 columns; byte SEL of sa and sb.
template <int SEL>
__device__ __forceinline__ f16_t mx_mfma32(u4_t a, u4_t b, f16_t c, uint32_t sa, uint32_t sb) {
    const i8_t A = {(int)a.x, (int)a.y, (int)a.z, (int)a.w}, B = {(int)b.x, (int)b.y, (int)b.z, (int)b.w};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(A, B, c, 4, 4, SEL, (int)sa, SEL, (int)sb);
}

template <bool BF>
__device__ __forceinline__ uint32_t mx_pack2(float a, float b) {
    if constexpr (BF)
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(f2_t{a, b}, bf2_t));
    else
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(f2_t{a, b}, h2_t));
}

__device__ __forceinline__ u2_t mx_pack4(bool bf, float v0, float v1, float v2, float v3) {
    return bf ? u2_t{mx_pack2<true>(v0, v1), mx_pack2<true>(v2, v3)}
              : u2_t{mx_pack2<false>(v0, v1), mx_pack2<false>(v2, v3)};
}

// Four neighbouring results of one row, rounded and stored: columns n .. n + 3
// of the row at y (of N columns); n is a multiple of 4.
__device__ __forceinline__ void mx_store4(uint16_t *y, int n, int N, bool bf, float v0, float v1, float v2,
                                          float v3) {
    const u2_t v = mx_pack4(bf, v0, v1, v2, v3);
    if ((N & 3) == 0) {     // (rows are aligned to 8 bytes)
        if (n < N)
            *(u2_t *)(y + n) = v;
    } else {
        if (n < N)
            y[n] = (uint16_t)v.x;
        if (n + 1 < N)
            y[n + 1] = (uint16_t)(v.x >> 16);
        if (n + 2 < N)
            y[n + 2] = (uint16_t)v.y;
        if (n + 3 < N)
            y[n + 3] = (uint16_t)(v.y >> 16);
    }
}

// A row tile of a product: matrix e has the rows from `start` on, `total` of
// them, in `count` tiles of BM; the tile is the mt-th, rows row0 .. row0 + rows - 1.
// All are held within 0 .. R.
struct MxTile {
    int e, start, total, count;
    int mt, row0, rows;
    __device__ __forceinline__ void take(int tile, int bm) {
        mt = tile;
        row0 = start + tile * bm;
        rows = total - tile * bm < bm ? total - tile * bm : bm;
    }
};

// Rows of matrix e: offsets outside 0 .. R are taken as the ends.
__device__ __forceinline__ int mx_offset(const MxArgs &a, int e) {
    const int o = a.offsets[e];
    return o < 0 ? 0 : o > (int)a.R ? (int)a.R : o;
}

// Sum over the wave's lanes up to the own one.
__device__ __forceinline__ uint32_t wave_scan(uint32_t v, int lane) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const uint32_t o = __shfl_up(v, d);
        v += lane >= d ? o : 0;
    }
    return v;
}

__device__ __forceinline__ uint32_t last_lane(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// Tiles of BM rows of matrix e, whose first row goes to `start` and rows to `total`.
// (R may be 2^31 - 1: nothing is added to a number of rows.)
template <int BM>
__device__ __forceinline__ uint32_t mx_tiles_of(const MxArgs &a, int e, int &start, int &total) {
    start = mx_offset(a, e);
    total = mx_offset(a, e + 1) - start;
    return total > 0 ? (uint32_t)(total - 1) / BM + 1 : 0;
}

// The tiles that all matrices have together at most.  Where offsets fall, their
// ranges overlap and would have more: what is past these is left out, so that a sum
// of tiles stays within 32 bits (64 matrices' 2^25 tiles of 64 rows each and these)
// and the work within what the launch is for.
template <int BM>
__device__ __forceinline__ uint32_t mx_most_tiles(const MxArgs &a) {
    const uint32_t R = (uint32_t)a.R, used = min(R, (uint32_t)a.E);
    return used + (R - used) / BM;
}

// How many tiles of BM rows all matrices have together (by one wave).
template <int BM>
__device__ __forceinline__ uint32_t mx_count_tiles(const MxArgs &a, int lane) {
    const uint32_t most = mx_most_tiles<BM>(a);
    uint32_t total = 0;
    for (int base = 0; base < a.E; base += 64) {
        const int e = base + lane;
        int start, rows;
        const uint32_t n = e < a.E ? mx_tiles_of<BM>(a, e, start, rows) : 0;
        total = min(total + last_lane(wave_scan(n, lane)), most);
    }
    return total;
}

// Tile `t` of all matrices' (by one wave; t is the same in all lanes); count 0
// where there are not so many.
template <int BM>
__device__ __forceinline__ MxTile mx_find_tile(const MxArgs &a, uint32_t t, int lane) {
    const uint32_t most = mx_most_tiles<BM>(a);
    MxTile out = {};
    uint32_t before = 0;
    for (int base = 0; base < a.E; base += 64) {
        const int e = base + lane;
        int start = 0, total = 0;
        const uint32_t n = e < a.E ? mx_tiles_of<BM>(a, e, start, total) : 0;
        const uint32_t incl = min(before + wave_scan(n, lane), most);
        const uint64_t past = __ballot(incl > t);
        if (past) {
            const int l = __builtin_ctzll(past);
            out.e = base + l;
            out.start = __builtin_amdgcn_readlane(start, l);
            out.total = __builtin_amdgcn_readlane(total, l);
            out.count = __builtin_amdgcn_readlane((int)n, l);
            out.take((int)t - (__builtin_amdgcn_readlane((int)incl, l) - out.count), BM);
            return out;
        }
        before = last_lane(incl);
    }
    return out;
}

// The same from a table in LDS of the tiles up to and with each matrix, made
// once by one wave.
template <int BM>
__device__ __forceinline__ void mx_tile_table(const MxArgs &a, uint32_t *table, int lane) {
    const uint32_t most = mx_most_tiles<BM>(a);
    uint32_t before = 0;
    for (int base = 0; base < a.E; base += 64) {
        const int e = base + lane;
        int start, total;
        const uint32_t n = e < a.E ? mx_tiles_of<BM>(a, e, start, total) : 0;
        const uint32_t incl = min(before + wave_scan(n, lane), most);
        if (e < a.E)
            table[e] = incl;
        before = last_lane(incl);
    }
}

template <int BM>
__device__ __forceinline__ MxTile mx_table_tile(const MxArgs &a, const uint32_t *table, uint32_t t, int lane) {
    MxTile out = {};
    for (int base = 0; base < a.E; base += 64) {
        const int e = base + lane;
        const uint64_t past = __ballot(e < a.E && table[e < a.E ? e : 0] > t);
        if (past) {
            out.e = base + __builtin_ctzll(past);
            break;
        }
    }
    const int before = __builtin_amdgcn_readfirstlane(out.e ? (int)table[out.e - 1] : 0);
    out.count = __builtin_amdgcn_readfirstlane((int)table[out.e]) - before;
    // (scalar loads: a vector load would wait for the copies under way)
    const auto *offsets = (const __attribute__((address_space(4))) int *)(uintptr_t)a.offsets;
    const int R = (int)a.R, o = offsets[out.e], p = offsets[out.e + 1];
    out.start = o < 0 ? 0 : o > R ? R : o;
    out.total = (p < 0 ? 0 : p > R ? R : p) - out.start;
    out.take((int)t - before, BM);
    return out;
}

}  // namespace w4a16

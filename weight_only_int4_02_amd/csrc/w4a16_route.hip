// Routing to experts (w4a16_route), and the two small kernels around the
// experts' products: the plan that sorts the rows by expert, and the weighted
// sum over a row's slots.
#include <hip/hip_runtime.h>

#include <math.h>

#include "w4a16_kernels.hpp"
#include "w4a16_routed.h"
#include "w4a16_routed.hpp"

namespace w4a16 {

namespace {

// ---------------------------------------------------------------------------
// w4a16_route: one wave per row; lane l holds experts l, l + 64, ...
//
// Which expert is larger must not hang on the rounding of an exponential:
// without a bias, and with groups judged by their best expert alone, the
// order of the scores is the order of the logits (softmax and sigmoid both
// rise), and the keys are the logits themselves.  Otherwise (WIDE) scores and
// keys are formed in 64 bits.
//
// The k largest are taken one at a time: a wave-wide maximum of the keys (DPP
// moves, no LDS), then the first lane and slot that holds it -- expert l + 64
// v, so the lowest slot with a holder, and in it the lowest lane, is the
// lowest index.  A taken or excluded expert's key is -infinity.
// ---------------------------------------------------------------------------
template <int CTRL>
__device__ __forceinline__ int dpp(int v) {
    return __builtin_amdgcn_update_dpp(v, v, CTRL, 0xF, 0xF, false);
}
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __builtin_bit_cast(float, dpp<CTRL>(__builtin_bit_cast(int, v)));
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)dpp<CTRL>((int)(uint32_t)b);
    const uint32_t hi = (uint32_t)dpp<CTRL>((int)(uint32_t)(b >> 32));
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ float lane_value(float v, int l) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), l));
}
__device__ __forceinline__ double lane_value(double v, int l) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, l);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), l);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
template <typename T, typename F>
__device__ __forceinline__ T wave_reduce(T v, F op) {
    v = op(v, dpp<0xB1>(v));   // lanes 1 apart
    v = op(v, dpp<0x4E>(v));   // 2 apart
    v = op(v, dpp<0x141>(v));  // mirrored within 8
    v = op(v, dpp<0x140>(v));  // mirrored within 16: every lane has its 16's
    return op(op(lane_value(v, 0), lane_value(v, 16)), op(lane_value(v, 32), lane_value(v, 48)));
}
__device__ __forceinline__ float vmax(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ double vmax(double a, double b) { return fmax(a, b); }

template <int DT>
__device__ __forceinline__ float load_logit(const void *p, int64_t at) {
    if constexpr (DT == W4A16_LOGITS_F32)
        return ((const float *)p)[at];
    else if constexpr (DT == W4A16_LOGITS_BF16)
        return bf16_bits_to_float(((const uint16_t *)p)[at]);
    else
        return (float)((const _Float16 *)p)[at];
}

constexpr int kRouteWaves = 4;

template <int V, bool WIDE, int DT>
__global__ __launch_bounds__(kRouteWaves * 64) void route_kernel(RouteArgs a) {
    using Key = std::conditional_t<WIDE, double, float>;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int t = (int)blockIdx.x * kRouteWaves + wave;
    if (t >= a.T)
        return;
    const Key none = -(Key)INFINITY;
    float l[V];
    float top = -INFINITY;
#pragma unroll
    for (int v = 0; v < V; v++) {
        const int e = lane + 64 * v;
        const float x = e < a.E ? load_logit<DT>(a.logits, (int64_t)t * a.E + e) : -INFINITY;
        l[v] = x != x ? -INFINITY : fminf(x, 3.402823466e38f);
        top = fmaxf(top, l[v]);
    }
    top = wave_reduce(top, [](float x, float y) { return fmaxf(x, y); });
    // scores: softmax's numerator, or sigmoid; a row with nothing has none
    const bool sig = a.sigmoid != 0;
    Key s[V], key[V];
    Key sum = 0;
#pragma unroll
    for (int v = 0; v < V; v++) {
        if constexpr (WIDE) {
            s[v] = l[v] == -INFINITY ? 0.0
                   : sig             ? 1.0 / (1.0 + exp(-(double)l[v]))
                                     : exp((double)l[v] - (double)top);
        } else {
            s[v] = l[v] == -INFINITY ? 0.f : sig ? 1.f / (1.f + expf(-l[v])) : expf(l[v] - top);
        }
        sum += s[v];
    }
    if (!sig) {
        sum = wave_reduce(sum, [](Key x, Key y) { return x + y; });
        const Key inv = sum > 0 ? 1 / sum : 0;
#pragma unroll
        for (int v = 0; v < V; v++)
            s[v] *= inv;
    }
#pragma unroll
    for (int v = 0; v < V; v++) {
        if constexpr (WIDE) {
            const int e = lane + 64 * v;
            key[v] = s[v];
            if (a.bias && e < a.E) {
                key[v] += (double)a.bias[e];
                key[v] = key[v] != key[v] ? none : key[v];
            }
            if (l[v] == -INFINITY)
                key[v] = none;
        } else {
            key[v] = l[v];
        }
    }

    if (a.topk_groups < a.n_groups) {
        // the keys go through LDS, so that lane q can walk group q; only this
        // wave reads what it wrote
        __shared__ Key ks[kRouteWaves][V * 64];
#pragma unroll
        for (int v = 0; v < V; v++)
            ks[wave][lane + 64 * v] = key[v];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        const int size = a.E / a.n_groups;
        Key best = none, second = none;
        if (lane < a.n_groups) {
            for (int i = 0; i < size; i++) {
                const Key x = ks[wave][lane * size + i];
                second = vmax(second, x < best ? x : best);
                best = vmax(best, x);
            }
        }
        Key value = best;
        if (a.group_top == 2 && second != none)
            value += second;
        uint64_t keep = 0;
        for (int i = 0; i < a.topk_groups; i++) {
            const Key m = wave_reduce(value, [](Key x, Key y) { return vmax(x, y); });
            const uint64_t at = __ballot(value == m && lane < a.n_groups && !(keep >> lane & 1));
            const int q = __builtin_ctzll(at);
            keep |= 1ull << q;
            value = lane == q ? none : value;
        }
#pragma unroll
        for (int v = 0; v < V; v++) {
            const int q = (lane + 64 * v) / size;
            if (q >= 64 || !(keep >> q & 1))
                key[v] = none;
        }
    }

    int id = -1;      // lane j: slot j
    Key weight = 0, total = 0;
    for (int j = 0; j < a.k; j++) {
        Key m = key[0];
#pragma unroll
        for (int v = 1; v < V; v++)
            m = vmax(m, key[v]);
        m = wave_reduce(m, [](Key x, Key y) { return vmax(x, y); });
        if (m == none)
            break;
        bool found = false;
#pragma unroll
        for (int v = 0; v < V; v++) {
            const uint64_t at = __ballot(key[v] == m);
            if (!found && at) {
                found = true;
                const int q = __builtin_ctzll(at);
                const Key w = lane_value(s[v], q);
                total += w;
                if (lane == j) {
                    id = q + 64 * v;
                    weight = w;
                }
                key[v] = lane == q ? none : key[v];
            }
        }
    }
    if (lane < a.k) {
        if (a.renormalize)
            weight = total > 0 ? weight / total : 0;
        a.ids[(int64_t)t * a.k + lane] = id;
        a.weights[(int64_t)t * a.k + lane] = id < 0 ? 0.f : (float)(weight * (Key)a.scale);
    }
}

template <int V, bool WIDE>
void launch_route_typed(const RouteArgs &a, int dt, unsigned blocks, hipStream_t st) {
    const dim3 grid(blocks), block(kRouteWaves * 64);
    if (dt == W4A16_LOGITS_F32)
        hipLaunchKernelGGL((route_kernel<V, WIDE, W4A16_LOGITS_F32>), grid, block, 0, st, a);
    else if (dt == W4A16_LOGITS_BF16)
        hipLaunchKernelGGL((route_kernel<V, WIDE, W4A16_LOGITS_BF16>), grid, block, 0, st, a);
    else
        hipLaunchKernelGGL((route_kernel<V, WIDE, W4A16_LOGITS_F16>), grid, block, 0, st, a);
}

template <int V>
void launch_route_wide(const RouteArgs &a, int dt, bool wide, unsigned blocks, hipStream_t st) {
    if (wide)
        launch_route_typed<V, true>(a, dt, blocks, st);
    else
        launch_route_typed<V, false>(a, dt, blocks, st);
}

// ---------------------------------------------------------------------------
// The plan: rows sorted by expert, in their own order within an expert, and
// the list of tiles.  One workgroup per expert, each with its own count of
// all experts (integer adds in LDS: their order changes nothing).  Each wave
// takes a run of rows, counts its expert's in it, and after the one barrier
// that shares the counts writes their places in order; no workgroup waits for
// another.  (With a barrier for every 1024 rows: 32 us for 24576 rows.)
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 1024, kPlanWaves = kPlanThreads / 64;

__global__ __launch_bounds__(kPlanThreads) void expert_plan_kernel(
    const int32_t *__restrict__ ids, int R, int E, int bm, int tiles_max,
    ExpertTile *__restrict__ tiles, int32_t *__restrict__ tiles_used, int32_t *__restrict__ perm,
    int32_t *__restrict__ place) {
    __shared__ int count[kMaxExperts];
    __shared__ int part[kPlanWaves][3];
    __shared__ int wave_n[kPlanWaves];
    const int e = blockIdx.x, tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    static_assert(kPlanThreads == kMaxExperts, "one thread per expert");
    count[tid] = 0;
    __syncthreads();
    // the wave's rows: blocks of 64, eight of them loaded at once
    constexpr int U = 8;
    const int blocks = (R + 63) / 64, per = (blocks + kPlanWaves - 1) / kPlanWaves;
    const int b0 = min(blocks, wave * per), b1 = min(blocks, b0 + per);
    auto each_block = [&](auto &&f) __attribute__((always_inline)) {
        for (int b = b0; b < b1; b += U) {
            int id[U];
#pragma unroll
            for (int u = 0; u < U; u++) {
                const int i = (b + u) * 64 + lane;
                id[u] = b + u < b1 && i < R ? ids[i] : -1;
            }
#pragma unroll
            for (int u = 0; u < U; u++)
                f(id[u], (b + u) * 64 + lane);
        }
    };
    int hits = 0;
    each_block([&](int id, int) {
        if (id >= 0 && id < E)
            atomicAdd(&count[id], 1);
        hits += __popcll(__ballot(id == e));
    });
    if (lane == 0)
        wave_n[wave] = hits;
    __syncthreads();
    // rows and tiles of the experts before this one, and tiles of all
    {
        const int c = count[tid], n = (c + bm - 1) / bm;
        int rows = tid < e ? c : 0, before = tid < e ? n : 0, all = n;
        for (int d = 32; d; d >>= 1) {
            rows += __shfl_xor(rows, d);
            before += __shfl_xor(before, d);
            all += __shfl_xor(all, d);
        }
        if (lane == 0) {
            part[wave][0] = rows;
            part[wave][1] = before;
            part[wave][2] = all;
        }
    }
    __syncthreads();
    int row0 = 0, tile0 = 0, used = 0, at = 0;
    for (int w = 0; w < kPlanWaves; w++) {
        row0 += part[w][0];
        tile0 += part[w][1];
        used += part[w][2];
        at += w < wave ? wave_n[w] : 0;
    }
    const int mine = count[e];
    for (int i = tid; i * bm < mine; i += kPlanThreads)
        if (tile0 + i < tiles_max)
            tiles[tile0 + i] = ExpertTile{e,     row0 + i * bm,         min(bm, mine - i * bm),
                                          tile0, (mine + bm - 1) / bm,  {0, 0, 0}};
    if (e == E - 1) {
        for (int i = used + tid; i < tiles_max; i += kPlanThreads)
            tiles[i] = ExpertTile{0, 0, 0, 0, 0, {0, 0, 0}};
        if (tid == 0)
            *tiles_used = used;
    }
    if (hits == 0)
        return;
    at += row0;
    each_block([&](int id, int i) {
        const uint64_t b = __ballot(id == e);
        if (id == e) {
            const int p = at + __popcll(b & ((1ull << lane) - 1));
            perm[p] = i;
            place[i] = p;
        }
        at += __popcll(b);
    });
}

// ---------------------------------------------------------------------------
// Y[t] = RNE(sum over the slots with an expert of weights[t][j] P[t][j]), in
// slot order; slots without an expert have no row of P.  Four
// columns per thread where D is a multiple of 4.
// ---------------------------------------------------------------------------
// Columns are cut into blocks of 256 C; a workgroup takes one block of a row.
template <bool BF, int C>
__global__ __launch_bounds__(256) void experts_combine_kernel(CombineArgs a) {
    const int64_t d = ((int64_t)blockIdx.x * 256 + threadIdx.x) * C;
    if (d >= a.D)
        return;
    for (int64_t t = blockIdx.y; t < a.T; t += gridDim.y) {
        float acc[C];
#pragma unroll
        for (int c = 0; c < C; c++)
            acc[c] = 0.f;
        // (the slots' numbers are the same for the whole workgroup)
        constexpr int U = 4;   // slots whose loads are in flight together
        for (int j0 = 0; j0 < a.k; j0 += U) {
            float w[U], v[U][C];
            bool in[U];
#pragma unroll
            for (int u = 0; u < U; u++) {
                const int64_t s = t * a.k + j0 + u;
                in[u] = j0 + u < a.k;
                const int id = in[u] ? a.ids[s] : -1;
                in[u] = id >= 0 && id < a.E;
                if (in[u]) {
                    w[u] = a.weights[s];
                    const float *p = a.P + (a.place ? (int64_t)a.place[s] : s) * a.D + d;
                    if constexpr (C == 4) {
                        const f4_t x = *(const f4_t *)p;
#pragma unroll
                        for (int c = 0; c < C; c++)
                            v[u][c] = x[c];
                    } else {
                        v[u][0] = *p;
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < U; u++)
                if (in[u]) {
#pragma unroll
                    for (int c = 0; c < C; c++)
                        acc[c] += w[u] * v[u][c];
                }
        }
        uint16_t out[C];
#pragma unroll
        for (int c = 0; c < C; c++) {
            if constexpr (BF)
                out[c] = __builtin_bit_cast(uint16_t, (__bf16)acc[c]);
            else
                out[c] = __builtin_bit_cast(uint16_t, (_Float16)acc[c]);
        }
        uint16_t *y = a.Y + t * a.D + d;
        if constexpr (C == 4) {
            typedef uint32_t u2_t __attribute__((ext_vector_type(2)));
            *(u2_t *)y = u2_t{out[0] | (uint32_t)out[1] << 16, out[2] | (uint32_t)out[3] << 16};
        } else {
            y[0] = out[0];
        }
    }
}

template <bool BF>
void launch_combine(const CombineArgs &a, hipStream_t st) {
    const int c = (a.D & 3) == 0 ? 4 : 1;
    const dim3 grid((unsigned)((a.D + 256 * c - 1) / (256 * c)),
                    (unsigned)(a.T < 32768 ? a.T : 32768));
    if (c == 4)
        hipLaunchKernelGGL((experts_combine_kernel<BF, 4>), grid, dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL((experts_combine_kernel<BF, 1>), grid, dim3(256), 0, st, a);
}

}  // namespace

int launch_route(const RouteArgs &a, int logits_dtype, void *stream) {
    const hipStream_t st = (hipStream_t)stream;
    const unsigned blocks = (unsigned)((a.T + kRouteWaves - 1) / kRouteWaves);
    const bool wide = a.bias != nullptr || (a.topk_groups < a.n_groups && a.group_top == 2);
    if (a.E <= 64)
        launch_route_wide<1>(a, logits_dtype, wide, blocks, st);
    else if (a.E <= 128)
        launch_route_wide<2>(a, logits_dtype, wide, blocks, st);
    else if (a.E <= 256)
        launch_route_wide<4>(a, logits_dtype, wide, blocks, st);
    else if (a.E <= 512)
        launch_route_wide<8>(a, logits_dtype, wide, blocks, st);
    else
        launch_route_wide<16>(a, logits_dtype, wide, blocks, st);
    return (int)hipGetLastError();
}

int launch_expert_plan(const int32_t *ids, int R, int E, int bm, int tiles_max, ExpertTile *tiles,
                       int32_t *tiles_used, int32_t *perm, int32_t *place, void *stream) {
    hipLaunchKernelGGL(expert_plan_kernel, dim3((unsigned)E), dim3(kPlanThreads), 0,
                       (hipStream_t)stream, ids, R, E, bm, tiles_max, tiles, tiles_used, perm, place);
    return (int)hipGetLastError();
}

int launch_experts_combine(const CombineArgs &a, void *stream) {
    if (a.bf16)
        launch_combine<true>(a, (hipStream_t)stream);
    else
        launch_combine<false>(a, (hipStream_t)stream);
    return (int)hipGetLastError();
}

}  // namespace w4a16

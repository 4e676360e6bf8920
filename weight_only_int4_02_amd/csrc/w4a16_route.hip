// Routing to experts (w4a16_route), and the two small kernels around the
// experts' products: the plan that sorts the rows by expert, and the weighted
// sum over a row's slots.
#include <hip/hip_runtime.h>

#include <math.h>

#include "w4a16_experts.hpp"
#include "w4a16_kernels.hpp"
#include "w4a16_routed.h"
#include "w4a16_routed.hpp"

namespace w4a16 {

namespace {

// ---------------------------------------------------------------------------
// w4a16_route.  A row takes L = 16 or 64 lanes; lane l holds the V experts from
// l V on.
//
// Which expert is larger must not hang on the rounding of an exponential:
// without a bias, and with groups judged by their best expert alone, the
// order of the scores is the order of the logits (softmax and sigmoid both
// rise), and the keys are the logits themselves.  Otherwise (WIDE) scores and
// keys are formed in 64 bits.
//
// The k largest are taken one at a time: the maximum over the row's lanes by
// DPP moves, then the lowest expert that holds it.  A taken or excluded
// expert's key is -infinity.  The chosen experts' scores are formed anew from
// their logits at the end, one lane a slot, in 64 bits.
//
// The kernel is bound by its instructions and their latency, not its bytes
// (8192 rows of 256 experts, 9 MB: 15.9 us, most of it the eight selections).  Few
// rows take a wave each, for the latency; many share waves, since the
// reductions are the same work for all of a row's lanes.
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
// op of the values D = 16 or 32 lanes apart: gfx950's swap of two registers'
// odd and even halves, given the same register twice, leaves the even halves in
// one result and the odd ones in the other.
template <int D>
__device__ __forceinline__ void halves(uint32_t v, uint32_t &even, uint32_t &odd) {
    const auto r = D == 16 ? __builtin_amdgcn_permlane16_swap(v, v, false, false)
                           : __builtin_amdgcn_permlane32_swap(v, v, false, false);
    even = r[0];
    odd = r[1];
}
template <int D, typename T, typename F>
__device__ __forceinline__ T op_rows(T v, F op) {
    if constexpr (sizeof(T) == 4) {
        uint32_t e, o;
        halves<D>(__builtin_bit_cast(uint32_t, v), e, o);
        return op(__builtin_bit_cast(T, e), __builtin_bit_cast(T, o));
    } else {
        const uint64_t b = __builtin_bit_cast(uint64_t, v);
        uint32_t el, ol, eh, oh;
        halves<D>((uint32_t)b, el, ol);
        halves<D>((uint32_t)(b >> 32), eh, oh);
        return op(__builtin_bit_cast(T, (uint64_t)eh << 32 | el),
                  __builtin_bit_cast(T, (uint64_t)oh << 32 | ol));
    }
}
// op over the L lanes of a row; every lane gets the result.
template <int L, typename T, typename F>
__device__ __forceinline__ T row_reduce(T v, F op) {
    v = op(v, dpp<0xB1>(v));   // lanes 1 apart
    v = op(v, dpp<0x4E>(v));   // 2 apart
    v = op(v, dpp<0x141>(v));  // mirrored within 8
    v = op(v, dpp<0x140>(v));  // mirrored within 16
    if constexpr (L == 64) {
        v = op_rows<16>(v, op);
        v = op_rows<32>(v, op);
    }
    return v;
}
__device__ __forceinline__ float vmax(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ double vmax(double a, double b) { return fmax(a, b); }

__device__ __forceinline__ float load_logit(const RouteArgs &a, int64_t at) {
    if (a.dtype == W4A16_LOGITS_F32)
        return ((const float *)a.logits)[at];
    if (a.dtype == W4A16_LOGITS_BF16)
        return bf16_bits_to_float(((const uint16_t *)a.logits)[at]);
    return (float)((const _Float16 *)a.logits)[at];
}
__device__ __forceinline__ float clean_logit(float x) {
    return x != x ? -INFINITY : fminf(x, 3.402823466e38f);
}

// exp(x) for x <= 0 in 64 bits, without the branches of a library's.  Cody and
// Waite's reduction: x = n ln 2 + r with |r| <= ln 2 / 2, ln 2 in two parts, so
// that n times the first is exact; then the exponential's series to r^13 / 13!
// (the next term is below 2^-57), times 2^n.  Below -745, where the result
// would round to less than the smallest subnormal, it is 0.
__device__ __forceinline__ double exp_series(double arg) {
    const double x = fmax(arg, -745.0);
    const double n = __builtin_rint(x * 1.4426950408889634);
    const double r = fma(n, -1.9082149292705877e-10, fma(n, -0.6931471803691238, x));
    double y = 1.0 / 6227020800.0;
    constexpr double over[13] = {1.0 / 479001600.0, 1.0 / 39916800.0, 1.0 / 3628800.0, 1.0 / 362880.0,
                                 1.0 / 40320.0,     1.0 / 5040.0,     1.0 / 720.0,     1.0 / 120.0,
                                 1.0 / 24.0,        1.0 / 6.0,        0.5,             1.0,
                                 1.0};
#pragma unroll
    for (int k = 0; k < 13; k++)
        y = fma(y, r, over[k]);
    y = ldexp(y, (int)n);
    return arg < -745.0 ? 0.0 : y;
}
// 1 / v for 1 <= v <= 2, by two steps of Newton's from the hardware's estimate.
__device__ __forceinline__ double reciprocal(double v) {
    double y = __builtin_amdgcn_rcp(v);
    y = fma(y, fma(-v, y, 1.0), y);
    y = fma(y, fma(-v, y, 1.0), y);
    return y;
}

// A logit's score in 64 bits: sigmoid, or softmax's numerator.  The sigmoid is
// formed from e = exp(-|l|), as 1 / (1 + e) or e / (1 + e), so that nothing
// overflows and the score of a very negative logit keeps its bits (a row may
// have no others, and is then divided by their sum).  -infinity has none.
__device__ __forceinline__ double score_of(float l, float top, bool sigmoid) {
    const double e = exp_series(sigmoid ? -fabs((double)l) : (double)l - (double)top);
    const double s = sigmoid ? (l < 0 ? e : 1.0) * reciprocal(1.0 + e) : e;
    return l == -INFINITY ? 0 : s;
}

constexpr int kRouteThreads = 256;

template <int V, int L, bool WIDE>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(RouteArgs a) {
    using Key = std::conditional_t<WIDE, double, float>;
    constexpr int ROWS = kRouteThreads / L;
    constexpr int NQ = 64 / L;       // groups of experts per lane, at most
    constexpr int none_index = 1 << 30;
    const int l = threadIdx.x % L, row = threadIdx.x / L;
    // (rows past the last repeat it, and store nothing: every lane stays
    // active for the moves between lanes)
    const int64_t t_own = (int64_t)blockIdx.x * ROWS + row;
    const int64_t t = t_own < a.T ? t_own : a.T - 1;
    const int64_t base = t * a.E;
    const Key none = -(Key)INFINITY;
    const bool sig = a.sigmoid != 0;
    const auto larger = [](auto x, auto y) { return vmax(x, y); };
    float lg[V];
    float top = -INFINITY;
    const int own = a.E - l * V;      // the lane's experts that there are
    auto load_as = [&](auto of) __attribute__((always_inline)) {
        if (a.E == V * L) {
#pragma unroll
            for (int v = 0; v < V; v++)
                lg[v] = of(base + l * V + v);
        } else {
            // (past the row's end, its last logit is loaded and dropped)
#pragma unroll
            for (int v = 0; v < V; v++) {
                const float x = of(base + min(l * V + v, a.E - 1));
                lg[v] = v < own ? x : -INFINITY;
            }
        }
    };
    if (a.dtype == W4A16_LOGITS_F32)
        load_as([&](int64_t at) { return ((const float *)a.logits)[at]; });
    else if (a.dtype == W4A16_LOGITS_BF16)
        load_as([&](int64_t at) { return bf16_bits_to_float(((const uint16_t *)a.logits)[at]); });
    else
        load_as([&](int64_t at) { return (float)((const _Float16 *)a.logits)[at]; });
#pragma unroll
    for (int v = 0; v < V; v++) {
        lg[v] = clean_logit(lg[v]);
        top = fmaxf(top, lg[v]);
    }
    // softmax's denominator, and the keys
    Key key[V], inv = 1;
    if (!sig || WIDE) {
        if (!sig)
            top = row_reduce<L>(top, larger);
        Key sum = 0;
#pragma unroll
        for (int v = 0; v < V; v++) {
            if constexpr (WIDE)
                key[v] = score_of(lg[v], top, sig);
            else
                key[v] = lg[v] == -INFINITY ? 0.f : expf(lg[v] - top);
            sum += key[v];
        }
        if (!sig) {
            sum = row_reduce<L>(sum, [](Key x, Key y) { return x + y; });
            inv = sum > 0 ? 1 / sum : 0;
        }
    }
#pragma unroll
    for (int v = 0; v < V; v++) {
        if constexpr (WIDE) {
            key[v] *= inv;
            if (a.bias) {
                key[v] += (double)a.bias[min(l * V + v, a.E - 1)];
                key[v] = key[v] != key[v] ? none : key[v];
            }
            key[v] = lg[v] == -INFINITY ? none : key[v];
        } else {
            key[v] = lg[v];
        }
    }

    if (a.topk_groups < a.n_groups) {
        const int size = a.E / a.n_groups;
        // the two best keys of each group; value[q] of lane l: group l + q L
        Key value[NQ];
        const auto take = [&](Key &best, Key &second, Key x) {
            second = vmax(second, x < best ? x : best);
            best = vmax(best, x);
        };
        __shared__ Key ks[ROWS][V * L + V * L / 16];
        if (size % V == 0) {
            // a group is n whole lanes' keys: after the step of d lanes, a
            // lane holds the two best of its 2 d and those behind them in its
            // group, and lane q fetches group q's value from its first lane
            // (8192 rows of 512 experts in 8 groups, through LDS as below:
            // 41.6 us, so 29.2; 61 rows of 160 in 8: 7.1, 5.0)
            const int n = size / V, behind = n - 1 - l % n;
            Key best = none, second = none;
#pragma unroll
            for (int v = 0; v < V; v++)
                take(best, second, key[v]);
            for (int d = 1; d < n; d *= 2) {
                const Key b2 = __shfl_down(best, d), s2 = __shfl_down(second, d);
                take(best, second, d <= behind ? b2 : none);
                take(best, second, d <= behind ? s2 : none);
            }
            const Key x = a.group_top == 2 && second != none ? best + second : best;
            const Key y = __shfl(x, (int)(threadIdx.x & (64 - L)) + min(l * n, L - 1));
            value[0] = l < a.n_groups ? y : none;
#pragma unroll
            for (int q = 1; q < NQ; q++)
                value[q] = none;
        } else {
            // the keys go through LDS, so that lane q can walk groups q, q +
            // L, ...; a row's lanes are one wave's, so no barrier.  One place
            // in 17 is left out, or the walks of groups of 32 would meet in
            // one bank.
#pragma unroll
            for (int v = 0; v < V; v++) {
                const int e = l * V + v;
                ks[row][e + e / 16] = key[v];
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
            for (int q = 0; q < NQ; q++) {
                Key best = none, second = none;
                const int grp = l + q * L;
                const int n = grp < a.n_groups ? size : 0;
                for (int i0 = 0; i0 < n; i0 += 8) {
                    Key x[8];
#pragma unroll
                    for (int i = 0; i < 8; i++) {
                        const int e = grp * size + min(i0 + i, size - 1);
                        x[i] = ks[row][e + e / 16];
                    }
#pragma unroll
                    for (int i = 0; i < 8; i++)
                        take(best, second, i0 + i < size ? x[i] : none);
                }
                value[q] = a.group_top == 2 && second != none ? best + second : best;
            }
        }
        uint64_t keep = 0;
        for (int i = 0; i < a.topk_groups; i++) {
            Key m = value[0];
#pragma unroll
            for (int q = 1; q < NQ; q++)
                m = vmax(m, value[q]);
            m = row_reduce<L>(m, larger);
            int at = none_index;
#pragma unroll
            for (int q = NQ - 1; q >= 0; q--) {
                const int grp = l + q * L;
                at = value[q] == m && grp < a.n_groups && !(keep >> grp & 1) ? grp : at;
            }
            at = row_reduce<L>(at, [](int x, int y) { return x < y ? x : y; });
            keep |= 1ull << (at & 63);
#pragma unroll
            for (int q = 0; q < NQ; q++)
                value[q] = l + q * L == at ? none : value[q];
        }
        int grp = l * V / size, rest = l * V - grp * size;   // of the lane's experts
#pragma unroll
        for (int v = 0; v < V; v++) {
            if (grp >= a.n_groups || !(keep >> grp & 1))
                key[v] = none;
            if (++rest == size) {
                rest = 0;
                grp++;
            }
        }
    }

    // slots l and l + L (k is at most 32)
    constexpr int NS = L == 16 ? 2 : 1;
    int id[NS];
#pragma unroll
    for (int n = 0; n < NS; n++)
        id[n] = -1;
    for (int j = 0; j < a.k; j++) {
        Key m = key[0];
#pragma unroll
        for (int v = 1; v < V; v++)
            m = vmax(m, key[v]);
        m = row_reduce<L>(m, larger);
        int at = none_index;
#pragma unroll
        for (int v = V - 1; v >= 0; v--)
            at = key[v] == m ? v : at;
        at += l * V;
        at = row_reduce<L>(at, [](int x, int y) { return x < y ? x : y; });
        at = m == none ? -1 : at;
        const int mine = at - l * V;
#pragma unroll
        for (int v = 0; v < V; v++)
            key[v] = v == mine ? none : key[v];
#pragma unroll
        for (int n = 0; n < NS; n++)
            id[n] = j == l + n * L ? at : id[n];
    }

    // in 64 bits whatever the keys are: a chosen sigmoid may be far below what
    // 32 bits hold, and one lane a slot costs next to nothing
    double w[NS], total = 0;
#pragma unroll
    for (int n = 0; n < NS; n++) {
        const float x =
            id[n] < 0 ? -INFINITY : clean_logit(load_logit(a, base + id[n]));
        w[n] = score_of(x, top, sig) * inv;
        total += w[n];
    }
    if (a.renormalize) {
        total = row_reduce<L>(total, [](double x, double y) { return x + y; });
#pragma unroll
        for (int n = 0; n < NS; n++)
            w[n] = total > 0 ? w[n] / total : 0;
    }
#pragma unroll
    for (int n = 0; n < NS; n++) {
        const int j = l + n * L;
        if (t_own < a.T && j < a.k) {
            a.ids[t * a.k + j] = id[n];
            a.weights[t * a.k + j] = id[n] < 0 ? 0.f : (float)(w[n] * (double)a.scale);
        }
    }
}

template <int V, int L>
void launch_route_rows(const RouteArgs &a, bool wide, hipStream_t st) {
    constexpr int ROWS = kRouteThreads / L;
    const dim3 grid((unsigned)((a.T + ROWS - 1) / ROWS)), block(kRouteThreads);
    if (wide)
        hipLaunchKernelGGL((route_kernel<V, L, true>), grid, block, 0, st, a);
    else
        hipLaunchKernelGGL((route_kernel<V, L, false>), grid, block, 0, st, a);
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
// Columns d .. d + C - 1 of row t once more, where an h beyond fp16 (or a routing
// weight, X or W that is not finite) left one without a finite sum: the slots
// whose h overflowed with it in 32 bits.  Stored where `in`; the whole wave
// together.
// The kernel's arguments are read again from their own memory, behind a pointer
// that the compiler knows nothing about: in registers from the start they would
// cost the kernel waves.
template <int C>
__device__ __forceinline__ void combine_wide(int64_t t, int64_t d, bool in) {
    uint64_t args = (uint64_t)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(args));
    const CombineArgs &a = *(const CombineArgs *)(const __attribute__((address_space(4))) CombineArgs *)args;
    __shared__ __align__(16) float hs[4][kWideColumns];
    const int lane = threadIdx.x & 63;
    float sum[C];
#pragma unroll
    for (int c = 0; c < C; c++)
        sum[c] = 0.f;
#pragma nounroll
    for (int j = 0; j < a.k; j++) {
        const int64_t s = t * a.k + j;
        const int id = __builtin_amdgcn_readfirstlane(a.ids[s]);
        if (id < 0 || id >= a.E)
            continue;
        const int64_t row = a.place ? (int64_t)__builtin_amdgcn_readfirstlane(a.place[s]) : s;
        const float weight = a.weights[s];
        const float *p = a.P + row * a.D + d;
        bool whole = true;
#pragma unroll
        for (int c = 0; c < C; c++)
            whole = whole && __builtin_isfinite(p[c]);
        if (__any(!whole) && row_overflowed(a.dn, row, lane))
            wide_dot<C>(a.gu, a.dn, t, row, id, weight, (int)d, lane, hs[threadIdx.x >> 6], sum);
        else
#pragma unroll
            for (int c = 0; c < C; c++)
                sum[c] += weight * p[c];
    }
#pragma unroll
    for (int c = 0; c < C; c++)
        if (in)
            a.Y[t * a.D + d + c] = __builtin_bit_cast(uint16_t, (_Float16)sum[c]);
}

// Columns are cut into blocks of 256 C; a workgroup takes one block of a row.
constexpr int kCombineRows = 32768;   // rows along a grid's y, at most
template <bool BF, int C>
__global__ __launch_bounds__(256) void experts_combine_kernel(CombineArgs a) {
    // (threads past the last column form the first ones again and store nothing:
    // every lane stays active for wide_dot)
    const int64_t d_own = ((int64_t)blockIdx.x * 256 + threadIdx.x) * C;
    const int64_t d = d_own < a.D ? d_own : 0;
    // (one row a workgroup: a loop over rows would hold the arguments in registers
    // over the rare path below)
    const int64_t t = (int64_t)blockIdx.z * kCombineRows + blockIdx.y;
    if (t >= a.T)
        return;
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
    if constexpr (!BF) {
        bool finite = true;
#pragma unroll
        for (int c = 0; c < C; c++)
            finite = finite && __builtin_isfinite(acc[c]);
        if (__builtin_expect(__any(!finite), 0)) {
            combine_wide<C>(t, d, d_own < a.D);
            return;
        }
    }
    if (d_own >= a.D)
        return;
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

template <bool BF>
void launch_combine(const CombineArgs &a, hipStream_t st) {
    const int c = (a.D & 3) == 0 ? 4 : 1;
    const unsigned rows = (unsigned)(a.T < kCombineRows ? a.T : kCombineRows);
    const dim3 grid((unsigned)((a.D + 256 * c - 1) / (256 * c)), rows, (unsigned)((a.T + rows - 1) / rows));
    if (c == 4)
        hipLaunchKernelGGL((experts_combine_kernel<BF, 4>), grid, dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL((experts_combine_kernel<BF, 1>), grid, dim3(256), 0, st, a);
}

}  // namespace

int launch_route(const RouteArgs &a, void *stream) {
    const hipStream_t st = (hipStream_t)stream;
    const bool wide = a.bias != nullptr || (a.topk_groups < a.n_groups && a.group_top == 2);
    // Up to two waves a SIMD, a wave to a row: 2048 rows of 256 experts in
    // groups, with a bias, 8.6 us, 12.3 with 16 lanes a row; of 64 experts 6.7
    // either way.  Above, 16 lanes: 4096 rows of 64 experts 6.9 us, 9.8 with a
    // wave a row; 8192 of 256 experts 17 us, 21 with 32 lanes, 23 with 64.
    const bool few = a.T <= 2048;
    if (a.E <= 256 && !few)
        a.E <= 16    ? launch_route_rows<1, 16>(a, wide, st)
        : a.E <= 64  ? launch_route_rows<4, 16>(a, wide, st)
        : a.E <= 128 ? launch_route_rows<8, 16>(a, wide, st)
                     : launch_route_rows<16, 16>(a, wide, st);
    else if (a.E <= 64)
        launch_route_rows<1, 64>(a, wide, st);
    else if (a.E <= 128)
        launch_route_rows<2, 64>(a, wide, st);
    else if (a.E <= 256)
        launch_route_rows<4, 64>(a, wide, st);
    else if (a.E <= 512)
        launch_route_rows<8, 64>(a, wide, st);
    else
        launch_route_rows<16, 64>(a, wide, st);
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

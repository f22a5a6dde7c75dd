// routing.hpp -- what stands around the products grouped by expert: the router's choice, the
// sort of the places by expert, and the rows to their places and back.
#pragma once

#include "grouped.hpp"
#include "sg_device.hpp"

namespace sg {

enum : int { ROUTE_SOFTMAX = 0, ROUTE_SIGMOID = 1 };

struct RouteParams {
    const void* X;
    int64_t ldx;
    int T, E, top_k, scoring, groups, top_groups, group_top, renormalize;
    float scale;
    const float* bias;
    const uint8_t* mask;
    int32_t* ids;
    float* weights;
    // backward
    const int32_t* chosen;
    const float* dweights;
    void* dX;
    int64_t lddx;
};

// x moved between lanes by a data-parallel move; lanes without a source (rows left out) get `none`.
// Every lane of the wave takes part: none of these may stand in an operand that only some evaluate.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t moved(uint32_t x, uint32_t none) {
    return (uint32_t)__builtin_amdgcn_update_dpp((int)none, (int)x, CTRL, ROWS, 0xf, false);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ int moved(int x, int none) {
    return (int)moved<CTRL, ROWS>((uint32_t)x, (uint32_t)none);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ float moved(float x, float none) {
    return __builtin_bit_cast(float, moved<CTRL, ROWS>(__builtin_bit_cast(uint32_t, x),
                                                       __builtin_bit_cast(uint32_t, none)));
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double moved(double x, double none) {
    const u32x2 v = __builtin_bit_cast(u32x2, x), n = __builtin_bit_cast(u32x2, none);
    return __builtin_bit_cast(
        double, u32x2{moved<CTRL, ROWS>((uint32_t)v.x, (uint32_t)n.x),
                      moved<CTRL, ROWS>((uint32_t)v.y, (uint32_t)n.y)});
}
__device__ __forceinline__ int from_lane(int x, int lane) {
    return __builtin_amdgcn_readlane(x, lane);
}
__device__ __forceinline__ float from_lane(float x, int lane) {
    return __builtin_bit_cast(float, from_lane(__builtin_bit_cast(int, x), lane));
}
__device__ __forceinline__ double from_lane(double x, int lane) {
    const u32x2 v = __builtin_bit_cast(u32x2, x);
    return __builtin_bit_cast(double, u32x2{(uint32_t)from_lane((int)v.x, lane),
                                            (uint32_t)from_lane((int)v.y, lane)});
}
// f over the lanes of a wave, the same in every lane: neighbours, pairs, mirrored halves of a row of
// 16, then the rows' last lanes to the rows behind.
template <typename T, typename F>
__device__ __forceinline__ T wave_reduce(T x, T none, F f) {
    x = f(x, moved<0xB1, 0xf>(x, none));         // quad_perm 1 0 3 2
    x = f(x, moved<0x4E, 0xf>(x, none));         // quad_perm 2 3 0 1
    x = f(x, moved<0x141, 0xf>(x, none));        // row_half_mirror
    x = f(x, moved<0x140, 0xf>(x, none));        // row_mirror
    x = f(x, moved<0x142, 0xa>(x, none));        // row_bcast:15
    x = f(x, moved<0x143, 0xc>(x, none));        // row_bcast:31
    return from_lane(x, 63);
}
__device__ __forceinline__ float wave_sum(float x) {
    return wave_reduce(x, 0.0f, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ double wave_sum(double x) {
    return wave_reduce(x, 0.0, [](double a, double b) { return a + b; });
}
__device__ __forceinline__ float wave_max(float x) {
    return wave_reduce(x, -__builtin_huge_valf(), [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ double wave_max(double x) {
    return wave_reduce(x, -__builtin_huge_val(), [](double a, double b) { return fmax(a, b); });
}
__device__ __forceinline__ int wave_min(int x) {
    return wave_reduce(x, 0x7FFFFFFF, [](int a, int b) { return min(a, b); });
}

// log of a score, up to what renormalising over the chosen cancels
__device__ __forceinline__ float log_score(int scoring, float x) {
    return scoring == ROUTE_SOFTMAX ? x : fminf(x, 0.0f) - log1pf(expf(-fabsf(x)));
}
__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

constexpr double kNone = -__builtin_huge_val();
constexpr double kNanKey = -1e300;        // a NaN logit: behind every number, in front of none

// Lane j < top_k holds place j of token t: its expert (-1: none) and logit x; top and total: the row's
// largest logit and the sum of e^(x - top), where softmax is not renormalised.
__device__ __forceinline__ void route_finish(const RouteParams& p, int t, int lane, int id, float x,
                                             float top, float total, bool bad) {
    float w;
    if (p.renormalize) {
        const float inf = __builtin_huge_valf(), l = id < 0 ? -inf : log_score(p.scoring, x);
        const float most = wave_max(l);
        const float a = id < 0 ? 0.0f : expf(l - most);
        w = a / wave_sum(a);
    } else {
        w = p.scoring == ROUTE_SOFTMAX ? expf(x - top) / total : sigmoid(x);
    }
    if (lane < p.top_k) {
        p.ids[(int64_t)t * p.top_k + lane] = id;
        p.weights[(int64_t)t * p.top_k + lane] =
            id < 0 ? 0.0f : bad ? __builtin_nanf("") : p.scale * w;
    }
}

// One token by one wave, every comparison in 64 bits; lane l holds experts l, l + 64, ...  The choices
// follow one another, each a maximum over the wave, which bounds it: 16384 tokens of 512 experts, 10
// choices 35 us; of 1024, 32 choices 161 us (fp32, MI355X).
// lds: 64 NV values for this wave.
template <int DT, int NV>
__device__ __forceinline__ void route_token(const RouteParams& p, int t, int lane, double* lds) {
    int32_t* ids = p.ids + (int64_t)t * p.top_k;
    float* weights = p.weights + (int64_t)t * p.top_k;
    if (p.mask && p.mask[t] == 0) {
        if (lane < p.top_k) {
            ids[lane] = -1;
            weights[lane] = 0.0f;
        }
        return;
    }
    const char* row = reinterpret_cast<const char*>(p.X) +
                      (int64_t)t * p.ldx * (DT == DT_F32 ? 4 : 2);
    const float inf = __builtin_huge_valf();
    float x[NV];
    bool bad = false;
    float top = -inf;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = lane + 64 * i;
        x[i] = e < p.E ? load_elem<DT>(row, e) : -inf;
        bad |= x[i] != x[i] || (p.scoring == ROUTE_SOFTMAX && x[i] == inf);
        top = fmaxf(top, x[i]);
    }
    bad = __any(bad);
    top = wave_max(top);
    // key: what the choice compares
    double key[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) key[i] = x[i] != x[i] ? kNanKey : (double)x[i];
    if (p.bias || p.groups > 1) {
        // scores of the row without its NaN logits; infinite ones share softmax's whole
        double c[NV];
        if (p.scoring == ROUTE_SOFTMAX) {
            double sum = 0.0;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                c[i] = !(x[i] > -inf) ? 0.0
                       : top == inf   ? (double)(x[i] == inf)
                                      : exp((double)x[i] - (double)top);
                sum += c[i];
            }
            sum = wave_sum(sum);
#pragma unroll
            for (int i = 0; i < NV; ++i) c[i] /= sum;
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i) c[i] = 1.0 / (1.0 + exp(-(double)x[i]));
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = lane + 64 * i;
            if (x[i] != x[i]) c[i] = 0.0;
            if (p.bias && e < p.E) c[i] += (double)p.bias[e];
            if (x[i] == -inf || c[i] != c[i]) c[i] = kNone;
            if (x[i] != x[i] && c[i] != kNone) c[i] = kNanKey;
            if (p.bias) key[i] = c[i];
        }
        if (p.groups > 1) {
#pragma unroll
            for (int i = 0; i < NV; ++i) lds[lane + 64 * i] = c[i];
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
            const int per = p.E / p.groups;
            double value = kNone;
            if (lane < p.groups) {
                double a = kNone, b = kNone;          // the two best
                for (int i = 0; i < per; ++i) {
                    const double v = lds[lane * per + i];
                    b = fmax(b, fmin(a, v));
                    a = fmax(a, v);
                }
                value = p.group_top == 2 && b > kNanKey ? a + b : a;
            }
            int rank = 0;
            for (int g = 0; g < p.groups; ++g) {
                const double v = from_lane(value, g);
                rank += v > value || (v == value && g < lane);
            }
            const uint64_t kept = __ballot(lane < p.groups && rank < p.top_groups);
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (!(kept >> min((lane + 64 * i) / per, 63) & 1)) key[i] = kNone;
        }
    }
    // the top_k: the largest key, of equal ones the lowest index, one after the other
    int id = -1;
    float mine = -inf;
    for (int j = 0; j < p.top_k; ++j) {
        double best = kNone;
        int e = 1 << 20;
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (key[i] > best) {
                best = key[i];
                e = lane + 64 * i;
                v = x[i];
            }
        const double most = wave_max(best);
        if (most == kNone) break;
        e = wave_min(best == most ? e : 1 << 20);
        v = from_lane(v, e & 63);
        if (lane == j) {
            id = e;
            mine = v;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (lane + 64 * i == e) key[i] = kNone;
    }
    float total = 0.0f;
    if (!p.renormalize && p.scoring == ROUTE_SOFTMAX) {
#pragma unroll
        for (int i = 0; i < NV; ++i) total += x[i] == -inf ? 0.0f : expf(x[i] - top);
        total = wave_sum(total);
    }
    route_finish(p, t, lane, id, mine, top, total, bad);
}

template <int DT, int NV>
__global__ void __launch_bounds__(256) route_kernel(const RouteParams p) {
    __shared__ double lds[4][NV * 64];
    const int wave = threadIdx.x >> 6;
    const int t = blockIdx.x * 4 + wave;
    if (t < p.T) route_token<DT, NV>(p, t, threadIdx.x & 63, lds[wave]);
}

// ---------------------------------------------------------------------------
// The usual case, at most 256 experts and 8 choices: L lanes a token (64 / L tokens a wave) hold V
// neighbouring experts each.  Keys of 32 bits carry the value in front of the inverted index, so
// the eight largest come out of sorting networks of integer maxima and minima: within a lane, then
// between lanes, whose sorted lists a and b join as max(a[i], b[7 - i]).
//   16-bit logits without a bias: the value is the logit itself, in an order of unsigned numbers.
//   Otherwise 24 bits from the row's largest value down to its smallest (at most 64 below), of
//   scores in fp32.  Where two values that decide are closer than what they may be off by (of the
//   scores 2^-21 for sigmoid and 2^-18 of the largest for softmax), equal ones among them, the few
//   that are in question are compared in 64 bits, one a lane, a token after the other: 0.1 % of the
//   tokens with random fp32 logits, but 22 % (64 experts) and 39 % (256) with fp32 logits cast from
//   bf16.  Groups that close and everything unusual (NaN, too few experts left) go through route_token.
// What bounds it is the vector unit, not memory: 16384 tokens, top 8 (MI355X, in a graph), fp32 logits:
//   64 experts 4.3 us, 0.9 TB/s;
//   256 experts 7.8 us, 2.2 TB/s: 819 vector instructions a wave, 13100 cycles of each SIMD, 5.5 us;
//     cast from bf16 20 us: 1573 and 42 of LDS, most of them for tokens redone;
//   256 experts in 8 groups, sigmoid and bias 14.2 to 16.8 us: 1287 instructions, 20600 cycles, 8.6 us;
//     the unit is busy for 0.7 of the time that waves run, which wait for a third of theirs.
// 1 token of 64 experts 3.3 us, nearly all of it the launch; 77 tokens of 256 in groups 5.8 us, the
// latency of one wave's steps, more than half of it waits.
// ---------------------------------------------------------------------------
template <int S>
__device__ __forceinline__ uint32_t lane_swap(uint32_t x) {
    constexpr int ctrl = S == 1 ? 0xB1 : S == 2 ? 0x4E : S == 4 ? 0x141 : 0x140;
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)x, ctrl, 0xf, 0xf, true);
}
template <int S>
__device__ __forceinline__ float lane_swap(float x) {
    return __builtin_bit_cast(float, lane_swap<S>(__builtin_bit_cast(uint32_t, x)));
}
// f over the L lanes of a token; every lane gets the result.  (Lanes of a half that S = 4 or 8 mirrors
// onto hold the same value already.)
template <int L, typename T, typename F>
__device__ __forceinline__ T lanes_reduce(T x, F f) {
    if constexpr (L > 1) x = f(x, lane_swap<1>(x));
    if constexpr (L > 2) x = f(x, lane_swap<2>(x));
    if constexpr (L > 4) x = f(x, lane_swap<4>(x));
    if constexpr (L > 8) x = f(x, lane_swap<8>(x));
    return x;
}

__device__ __forceinline__ void order_pair(uint32_t& a, uint32_t& b) {
    const uint32_t hi = max(a, b);
    b = min(a, b);
    a = hi;
}
// Eight values, the largest first: Batcher's odd-even merge sort.
__device__ __forceinline__ void sort8(uint32_t (&v)[8]) {
    order_pair(v[0], v[1]), order_pair(v[2], v[3]), order_pair(v[4], v[5]), order_pair(v[6], v[7]);
    order_pair(v[0], v[2]), order_pair(v[1], v[3]), order_pair(v[4], v[6]), order_pair(v[5], v[7]);
    order_pair(v[1], v[2]), order_pair(v[5], v[6]);
    order_pair(v[0], v[4]), order_pair(v[1], v[5]), order_pair(v[2], v[6]), order_pair(v[3], v[7]);
    order_pair(v[2], v[4]), order_pair(v[3], v[5]);
    order_pair(v[1], v[2]), order_pair(v[3], v[4]), order_pair(v[5], v[6]);
}
// The eight largest of two sorted lists (b the other one, its last first): bitonic, then sorted.
__device__ __forceinline__ void join8(uint32_t (&v)[8], const uint32_t (&b)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = max(v[i], b[i]);
#pragma unroll
    for (int d = 4; d > 0; d /= 2)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (!(i & d)) order_pair(v[i], v[i + d]);
}
template <int S>
__device__ __forceinline__ void join_lanes(uint32_t (&v)[8]) {
    uint32_t b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = lane_swap<S>(v[7 - i]);
    join8(v, b);
}
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}
// e^d and 1 / (1 + e^-x) from the hardware's exp2 and reciprocal
__device__ __forceinline__ float fast_exp(float d) {
    return __builtin_amdgcn_exp2f(d * 1.44269504088896341f);
}

template <int DT, int L, int V>
__global__ void __launch_bounds__(256) route_lanes_kernel(const RouteParams p) {
    constexpr int TOKENS = 64 / L, NV = L * V > 64 ? L * V / 64 : 1;
    constexpr int ROW = L * V + 1;                      // odd: tokens' rows start in other banks
    constexpr int GROUPS = L * V < 64 ? L * V : 64;
    struct Wave {
        union {
            float c[TOKENS * ROW];
            double exact[NV * 64];
        };
        float value[TOKENS * GROUPS];
        uint8_t kept[TOKENS * GROUPS];
        float edge[TOKENS][2];                          // the lowest group kept, the best one not
        uint16_t list[64];                              // candidates, then the chosen ones
        float logit[64];
        double exact_value[64];
    };
    __shared__ Wave lds[4];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, li = lane % L, lt = lane / L;
    Wave& w = lds[wave];
    const int t0 = (blockIdx.x * 4 + wave) * TOKENS, t = t0 + lt;
    if (t0 >= p.T) return;
    const float inf = __builtin_huge_valf();
    const bool here = t < p.T, live = here && !(p.mask && p.mask[t] == 0);
    const char* row = reinterpret_cast<const char*>(p.X) +
                      (int64_t)(here ? t : t0) * p.ldx * (DT == DT_F32 ? 4 : 2);
    const int e0 = li * V;
    float x[V];
    if (live && e0 + V <= p.E) {
#pragma unroll
        for (int i = 0; i < V; i += 8) {
            Raw8<DT> raw;
            float v[8];
            raw.load(row, e0 + i, p.E);
            raw.get(v);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[i + j] = v[j];
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = live && e0 + i < p.E ? load_elem<DT>(row, e0 + i) : -inf;
    }
    float bias[V];
    if (p.bias) {
        if (e0 + V <= p.E) {
#pragma unroll
            for (int i = 0; i < V; i += 4) {
                const f32x4 b = *reinterpret_cast<const f32x4_any*>(p.bias + e0 + i);
#pragma unroll
                for (int j = 0; j < 4; ++j) bias[i + j] = b[j];
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) bias[i] = e0 + i < p.E ? p.bias[e0 + i] : 0.0f;
        }
    }
    float top = -inf;
    // unusual: for route_token; unsure: the order of a few has to be looked at in 64 bits
    bool unusual = false, unsure = false;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        top = fmaxf(top, x[i]);
        unusual |= x[i] != x[i];
    }
    top = lanes_reduce<L>(top, [](float a, float b) { return fmaxf(a, b); });
    unusual |= p.scoring == ROUTE_SOFTMAX && top == inf;
    const bool softmax = p.scoring == ROUTE_SOFTMAX, groups = p.groups > 1;
    // scores, where they decide or are needed for the weights
    float c[V], total = 0.0f, off = 0.0f;
    if (softmax && (p.bias || groups || !p.renormalize)) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            c[i] = x[i] == -inf ? 0.0f : fast_exp(x[i] - top);
            total += c[i];
        }
        total = lanes_reduce<L>(total, [](float a, float b) { return a + b; });
        const float f = __builtin_amdgcn_rcpf(total);
#pragma unroll
        for (int i = 0; i < V; ++i) c[i] *= f;
        off = 0x1p-23f + 0x1p-18f * f;                  // f: the largest score
    } else if (p.bias || groups) {
#pragma unroll
        for (int i = 0; i < V; ++i) c[i] = __builtin_amdgcn_rcpf(1.0f + fast_exp(-x[i]));
        off = 0x1p-21f;
    }
    float hi = -inf, lo = inf;
    if (p.bias || groups) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (p.bias) c[i] += bias[i];
            if (x[i] == -inf || c[i] != c[i]) c[i] = -inf;
            hi = fmaxf(hi, c[i]);
            lo = fminf(lo, c[i] == -inf ? inf : c[i]);
        }
        hi = lanes_reduce<L>(hi, [](float a, float b) { return fmaxf(a, b); });
        lo = lanes_reduce<L>(lo, [](float a, float b) { return fminf(a, b); });
        off += 0x1p-23f * fmaxf(fabsf(hi), fabsf(lo));
    }
    bool in[V];
#pragma unroll
    for (int i = 0; i < V; ++i) in[i] = p.bias ? c[i] != -inf : x[i] != -inf;
    if (groups) {
        const int per = p.E / p.groups, work = TOKENS * p.groups, wide = per / V;
        if (per % V == 0 && (wide == 1 || wide == 2 || wide == 4 || wide == 8)) {
            // a group is 1, 2, 4 or 8 lanes: its best two by data-parallel moves
            float a = -inf, b = -inf;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                b = fmaxf(b, fminf(a, c[i]));
                a = fmaxf(a, c[i]);
            }
            auto with = [&](float a2, float b2) {
                b = fmaxf(fminf(a, a2), fmaxf(b, b2));
                a = fmaxf(a, a2);
            };
            if (wide > 1) with(lane_swap<1>(a), lane_swap<1>(b));
            if (wide > 2) with(lane_swap<2>(a), lane_swap<2>(b));
            if (wide > 4) with(lane_swap<4>(a), lane_swap<4>(b));
            const float v = p.group_top == 2 && b != -inf ? a + b : a;
            const int g = li / wide;
            if (li % wide == 0 && g < p.groups) w.value[lt * p.groups + g] = v;
            wave_sync();
            int rank = 0;
#pragma unroll 8
            for (int h = 0; h < p.groups; ++h) {
                const float o = w.value[lt * p.groups + h];
                rank += o > v || (o == v && h < g);
            }
            const bool is = g < p.groups, keep = is && rank < p.top_groups;
            const float low = lanes_reduce<L>(keep ? v : inf,
                                              [](float a, float b) { return fminf(a, b); });
            const float high = lanes_reduce<L>(is && !keep ? v : -inf,
                                               [](float a, float b) { return fmaxf(a, b); });
            // a sum of two is off by twice what a score is, and so is the other
            unusual |= low - high <= 5.0f * off;
#pragma unroll
            for (int i = 0; i < V; ++i) in[i] = in[i] && keep;
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) w.c[lt * ROW + e0 + i] = c[i];
            wave_sync();
            // one lane a token's group: its best two; each starts elsewhere, for the banks
            for (int k = lane; k < work; k += 64) {
                const int tt = k / p.groups, g = k - tt * p.groups;
                const float* from = w.c + tt * ROW + g * per;
                float a = -inf, b = -inf;
#pragma unroll 8
                for (int i = 0, j = g % per; i < per; ++i) {
                    const float v = from[j];
                    b = fmaxf(b, fminf(a, v));
                    a = fmaxf(a, v);
                    j = j + 1 == per ? 0 : j + 1;
                }
                w.value[k] = p.group_top == 2 && b != -inf ? a + b : a;
            }
            wave_sync();
            for (int k = lane; k < work; k += 64) {
                const int tt = k / p.groups, g = k - tt * p.groups;
                const float v = w.value[k];
                int rank = 0;
#pragma unroll 4
                for (int h = 0; h < p.groups; ++h) {
                    const float o = w.value[tt * p.groups + h];
                    rank += o > v || (o == v && h < g);
                }
                w.kept[k] = rank < p.top_groups;
                if (rank == p.top_groups - 1) w.edge[tt][0] = v;
                if (rank == p.top_groups) w.edge[tt][1] = v;
            }
            wave_sync();
            unusual |= w.edge[lt][0] - w.edge[lt][1] <= 5.0f * off;
            int g = e0 / per, r = e0 - g * per;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                in[i] = in[i] && g < p.groups && w.kept[lt * p.groups + min(g, p.groups - 1)];
                if (++r == per) {
                    r = 0;
                    ++g;
                }
            }
        }
    }
    // keys
    const bool whole = DT != DT_F32 && !p.bias;          // a 16-bit logit whole
    uint32_t key[V], band = 0;
    if (whole) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            uint32_t h = __builtin_bit_cast(uint32_t, x[i]);
            if constexpr (DT == DT_F16) h = (uint32_t)from_f32<DT_F16>(x[i]) << 16;
            if (h == 0x80000000u) h = 0;                 // -0 is 0
            h = (h ^ (h >> 31 ? 0xFFFF0000u : 0x80000000u)) & 0xFFFF0000u;
            key[i] = in[i] ? h | (0xFFFFu - (e0 + i)) : 0;
        }
    } else {
        if (!p.bias) {
            hi = top;
            lo = inf;
#pragma unroll
            for (int i = 0; i < V; ++i) lo = fminf(lo, x[i] == -inf ? inf : x[i]);
            lo = lanes_reduce<L>(lo, [](float a, float b) { return fminf(a, b); });
            off = 0.0f;
        }
        lo = fmaxf(lo, hi - 64.0f);
        const float scale = hi > lo ? 16770000.0f / (hi - lo) : 0.0f;
        // The steps from value to key keep the order, so of exact values only equal keys are in
        // doubt; else both ends of a difference may be off, and the key by a step of rounding each.
        const float wide = off > 0.0f ? 2.0f + 2.0f * off * scale : 0.0f;
        unusual |= !(wide < 4000.0f);
        band = (uint32_t)fminf(wide, 4000.0f);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float d = fmaxf((p.bias ? c[i] : x[i]) - lo, 0.0f);
            key[i] = in[i] ? (4096u + (uint32_t)fminf(d * scale, 16770000.0f)) << 8 | (255u - (e0 + i))
                           : 0;
        }
    }
    uint32_t best[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) best[i] = key[i];
    sort8(best);
    if constexpr (V == 16) {
        uint32_t more[8], back[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) more[i] = key[8 + i];
        sort8(more);
#pragma unroll
        for (int i = 0; i < 8; ++i) back[i] = more[7 - i];
        join8(best, back);
    }
    if constexpr (L > 1) join_lanes<1>(best);
    if constexpr (L > 2) join_lanes<2>(best);
    if constexpr (L > 4) join_lanes<4>(best);
    if constexpr (L > 8) join_lanes<8>(best);
    // the last one chosen, and how far behind it the next key is
    uint32_t end = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j == p.top_k - 1) end = best[j];
    unusual |= end == 0;
    if (!whole) {
        uint32_t gap = ~0u;
#pragma unroll
        for (int i = 0; i < V; ++i) gap = min(gap, end - 1 - key[i]);
        gap = lanes_reduce<L>(gap, [](uint32_t a, uint32_t b) { return min(a, b); });
        unsure |= gap >> 8 <= band;
#pragma unroll
        for (int j = 0; j < 7; ++j)
            if (j + 1 < p.top_k) unsure |= (best[j] >> 8) - (best[j + 1] >> 8) <= band;
    }
    const uint64_t mine = ((uint64_t)1 << L) - 1;         // the lanes of the token at bit 0
    const uint64_t fully = __ballot(unusual && live), closely = __ballot(unsure && live);
    const bool redo = ((fully | closely) >> (lt * L) & mine) != 0;
    // weights: lane li has places li, li + L, ...
    constexpr int PLACES = L < 8 ? 8 / L : 1;
    int id[PLACES];
    float v[PLACES], most = -inf;
#pragma unroll
    for (int k = 0; k < PLACES; ++k) {
        uint32_t kk = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (li + L * k == j && j < p.top_k) kk = best[j];
        id[k] = kk == 0 ? -1 : (int)(whole ? 0xFFFFu - (kk & 0xFFFFu) : 255u - (kk & 255u));
        v[k] = id[k] < 0 ? -inf : load_elem<DT>(row, id[k]);
    }
    if (p.renormalize) {
#pragma unroll
        for (int k = 0; k < PLACES; ++k) {
            v[k] = id[k] < 0 ? -inf : log_score(p.scoring, v[k]);
            most = fmaxf(most, v[k]);
        }
        most = lanes_reduce<L>(most, [](float a, float b) { return fmaxf(a, b); });
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < PLACES; ++k) {
            v[k] = id[k] < 0 ? 0.0f : expf(v[k] - most);
            sum += v[k];
        }
        sum = lanes_reduce<L>(sum, [](float a, float b) { return a + b; });
#pragma unroll
        for (int k = 0; k < PLACES; ++k) v[k] /= sum;
    } else {
#pragma unroll
        for (int k = 0; k < PLACES; ++k) v[k] = softmax ? expf(v[k] - top) / total : sigmoid(v[k]);
    }
    if (here && !redo)
#pragma unroll
        for (int k = 0; k < PLACES; ++k) {
            const int j = li + L * k;
            if (j < p.top_k) {
                p.ids[(int64_t)t * p.top_k + j] = live ? id[k] : -1;
                p.weights[(int64_t)t * p.top_k + j] = live ? p.scale * v[k] : 0.0f;
            }
        }
    for (uint64_t left = fully | closely; left;) {
        const int tt = __builtin_ctzll(left) / L;
        left &= ~(mine << (tt * L));
        wave_sync();
        // every key that may belong in front of the last one chosen, one a lane, in 64 bits
        int n = 64 + 1;
        if ((fully >> (tt * L) & mine) == 0) {
            const uint32_t from = (end >> 8) - min(end >> 8, band + 2);
            n = 0;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const bool is = lt == tt && key[i] != 0 && key[i] >> 8 >= from;
                const uint64_t all = __ballot(is);
                const int at = n + __popcll(all & (((uint64_t)1 << lane) - 1));
                if (is && at < 64) w.list[at] = (uint16_t)(e0 + i);
                n += __popcll(all);
            }
        }
        if (n > 64) {
            route_token<DT, NV>(p, t0 + tt, lane, w.exact);
            continue;
        }
        wave_sync();
        const char* its = reinterpret_cast<const char*>(p.X) +
                          (int64_t)(t0 + tt) * p.ldx * (DT == DT_F32 ? 4 : 2);
        const float its_top = from_lane(top, tt * L), its_total = from_lane(total, tt * L);
        const int e = lane < n ? w.list[lane] : 0;
        const float its_x = load_elem<DT>(its, e);
        double exact = its_x;
        if (p.bias) {
            if (softmax) {
                double sum = 0.0;
                for (int i = lane; i < p.E; i += 64)
                    sum += exp((double)load_elem<DT>(its, i) - (double)its_top);
                exact = exp(exact - (double)its_top) / wave_sum(sum);
            } else {
                exact = 1.0 / (1.0 + exp(-exact));
            }
            exact += (double)p.bias[e];
        }
        w.exact_value[lane] = exact;
        wave_sync();
        int rank = 0;
#pragma unroll 4
        for (int j = 0; j < n; ++j) {
            const double o = w.exact_value[j];
            rank += (int)(o > exact) | ((int)(o == exact) & (int)(w.list[j] < e));
        }
        wave_sync();
        if (lane < n && rank < p.top_k) {
            w.list[rank] = (uint16_t)e;
            w.logit[rank] = its_x;
        }
        wave_sync();
        const int id = lane < p.top_k ? w.list[lane] : -1;
        route_finish(p, t0 + tt, lane, id, w.logit[lane], its_top, its_total, false);
    }
}

// ---------------------------------------------------------------------------
// dX of a token by one wave, from the choice: with l the chosen logs of scores, q = softmax(l) and
// G = scale * dweights, dl = q (G - sum G q) (for sigmoid times dl/dx = 1 - s); not renormalised, the
// softmax's own product dx = s (G - sum G s) over the row, or G s (1 - s).  One read of what it needs
// of X (renormalised: the chosen alone), one write of dX.  A lane has NV experts in registers and the
// choices are added to them in order, so that the same expert twice adds up the same each time.
// Measured (MI355X, bf16, 16384 tokens, top 8): 64 experts 6.3 us, softmax not renormalised 6.4 us;
// 256 experts 9.1 and 11.8 us (8 MB written; 17 MB moved, 1.4 TB/s): the walk over the choices bounds it,
// 269 vector instructions a wave, which keep the unit busy for 0.9 of the time.
// ---------------------------------------------------------------------------
template <int DT, int NV>
__global__ void __launch_bounds__(256) route_bwd_kernel(const RouteParams p) {
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int t = blockIdx.x * 4 + wave;
    if (t >= p.T) return;
    constexpr int ESZ = DT == DT_F32 ? 4 : 2;
    const char* row = reinterpret_cast<const char*>(p.X) + (int64_t)t * p.ldx * ESZ;
    char* out = reinterpret_cast<char*>(p.dX) + (int64_t)t * p.lddx * ESZ;
    const float inf = __builtin_huge_valf();
    int id = -1;
    float G = 0.0f;
    if (lane < p.top_k) {
        id = p.chosen[(int64_t)t * p.top_k + lane];
        if (id < 0 || id >= p.E) id = -1;
        else G = p.scale * p.dweights[(int64_t)t * p.top_k + lane];
    }
    float d[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) d[i] = 0.0f;
    if (__any(id >= 0)) {
        float v = 0.0f;
        if (p.renormalize) {
            const float x = id < 0 ? 0.0f : load_elem<DT>(row, id);
            const float l = id < 0 ? -inf : log_score(p.scoring, x);
            const float most = wave_max(l);
            const float a = id < 0 ? 0.0f : expf(l - most);
            const float q = a / wave_sum(a);
            v = q * (G - wave_sum(G * q));
            if (p.scoring == ROUTE_SIGMOID) v *= sigmoid(-x);
        } else if (p.scoring == ROUTE_SIGMOID) {
            const float x = id < 0 ? 0.0f : load_elem<DT>(row, id);
            v = G * (sigmoid(x) * sigmoid(-x));
        } else {
            v = G;
        }
        for (int j = 0; j < p.top_k; ++j) {
            const int e = from_lane(id, j);
            const float g = from_lane(v, j);
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (lane + 64 * i == e) d[i] += g;
        }
        if (!p.renormalize && p.scoring == ROUTE_SOFTMAX) {
            float x[NV], top = -inf, sum = 0.0f, dot = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                x[i] = lane + 64 * i < p.E ? load_elem<DT>(row, lane + 64 * i) : -inf;
                top = fmaxf(top, x[i]);
            }
            top = wave_max(top);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                x[i] = x[i] == -inf ? 0.0f : expf(x[i] - top);
                sum += x[i];
                dot += d[i] * x[i];
            }
            sum = wave_sum(sum);
            dot = wave_sum(dot) / sum;
#pragma unroll
            for (int i = 0; i < NV; ++i) d[i] = x[i] / sum * (d[i] - dot);
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (lane + 64 * i < p.E) put_elem<DT>(out, lane + 64 * i, d[i]);
}

// ---------------------------------------------------------------------------
// The places sorted by expert.  Work-group e < experts counts the ids below e, which is its first
// row, and writes the rows and places of its own; the last one does the same for the ids of no
// expert, which behave as expert `experts`.  Every work-group reads all ids: no second launch, no
// table between work-groups and no atomics.  Wave w owns one run of the ids, in order, so the
// ranks are the order of the places.  Grid y divides the second walk, the one that writes.
// What bounds it is the latency of one work-group's walk over all ids (of a wave's cycles six in ten wait;
// the vector unit is busy for four): 64 experts (MI355X): 1024 ids 2.9 us, 16384 5.0 us, 65536 9.4 us
// (0.2 us for the 0.8 MB at the rate of a copy, and the launch).
// ---------------------------------------------------------------------------
typedef int32_t i32x4_any __attribute__((ext_vector_type(4), aligned(4)));

struct SortParams {
    const int32_t* ids;
    int n, experts;
    int32_t *offsets, *order, *place;
};

// Four ids of a lane of each of DEEP pieces of 256, ids past the end as expert ~0 and those of no
// expert as expert `none`.  Whole pieces load 16 bytes a lane, all of them before the first is used.
template <int DEEP>
__device__ __forceinline__ void sort_load(const SortParams& p, int i, int lane, int last,
                                          uint32_t none, uint32_t (&v)[DEEP][4]) {
    const int at = i + 4 * lane;
    i32x4_any x[DEEP];
    if (i + 256 * DEEP <= last) {
#pragma unroll
        for (int d = 0; d < DEEP; ++d)
            x[d] = *reinterpret_cast<const i32x4_any*>(p.ids + at + 256 * d);
#pragma unroll
        for (int d = 0; d < DEEP; ++d)
#pragma unroll
            for (int j = 0; j < 4; ++j) v[d][j] = min((uint32_t)x[d][j], none);
        return;
    }
#pragma unroll
    for (int d = 0; d < DEEP; ++d) {
        const int32_t* ids = p.ids + at + 256 * d;
        if (i + 256 * (d + 1) <= last) {
            x[d] = *reinterpret_cast<const i32x4_any*>(ids);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) x[d][j] = at + 256 * d + j < last ? ids[j] : 0;
        }
    }
#pragma unroll
    for (int d = 0; d < DEEP; ++d)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[d][j] = at + 256 * d + j < last ? min((uint32_t)x[d][j], none) : ~0u;
}

// A wave counts COUNT pieces of 256 ids at a time and writes DEEP, so that as many loads are under way
// (65536 ids of 64 experts: 4 and 2 9.4 us, 4 and 4 10.1 us, 16 and 4 10.1 us).
template <int WAVES, int DEEP, int COUNT>
__global__ void __launch_bounds__(64 * WAVES) sort_kernel(const SortParams p) {
    __shared__ int below[WAVES], equal[WAVES];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const uint32_t e = blockIdx.x, none = p.experts;
    const int64_t run = ((int64_t)p.n + WAVES * 256 - 1) / (WAVES * 256) * 256;
    const int first = (int)min((int64_t)p.n, wave * run), last = (int)min((int64_t)p.n, first + run);
    // this work-group's part of the run, in whole steps
    constexpr int STEP = 256 * DEEP;
    const int steps = (last - first + STEP - 1) / STEP, parts = gridDim.y;
    const int begin = first + (int)((int64_t)steps * blockIdx.y / parts) * STEP;
    const int end = min(last, first + (int)((int64_t)steps * (blockIdx.y + 1) / parts) * STEP);
    // counts of each lane: two vector instructions an id and count, where a ballot and its bits
    // counted keep the scalar unit busy (65536 ids of 64 experts: 20.9 us)
    int lt = 0, eq = 0, ahead = 0;
    for (int i = first; i < last; i += 256 * COUNT) {
        uint32_t v[COUNT][4];
        sort_load<COUNT>(p, i, lane, last, none, v);
#pragma unroll
        for (int d = 0; d < COUNT; ++d) {
            if (d % DEEP == 0 && i + 256 * d == begin) ahead = eq;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                lt += v[d][j] < e;
                eq += v[d][j] == e;
            }
        }
    }
    lt = __builtin_amdgcn_readlane(lane_scan(lt), 63);
    eq = __builtin_amdgcn_readlane(lane_scan(eq), 63);
    ahead = __builtin_amdgcn_readlane(lane_scan(ahead), 63);
    if (lane == 0) {
        below[wave] = lt;
        equal[wave] = eq;
    }
    __syncthreads();
    int at = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
        at += below[w];
        if (w < wave) at += equal[w];
    }
    if (threadIdx.x == 0 && blockIdx.y == 0) {
        int row = 0;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) row += below[w];
        p.offsets[e] = row;
    }
    if (eq == 0) return;
    at = __builtin_amdgcn_readfirstlane(at + ahead);
    const uint64_t before = ((uint64_t)1 << lane) - 1;
    for (int i = begin; i < end; i += STEP) {
        uint32_t v[DEEP][4];
        sort_load<DEEP>(p, i, lane, last, none, v);
#pragma unroll
        for (int d = 0; d < DEEP; ++d) {
            uint64_t m[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) m[j] = __ballot(v[d][j] == e);
            if ((m[0] | m[1] | m[2] | m[3]) == 0) continue;
            int r = at;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                r += __popcll(m[j] & before);
                at += __popcll(m[j]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (v[d][j] == e) {
                    const int place = i + 256 * d + 4 * lane + j;
                    if (p.order) p.order[r] = e < none ? place : -1;
                    if (p.place) p.place[place] = e < none ? r : -1;
                    ++r;
                }
        }
    }
}

// ---------------------------------------------------------------------------
// Rows to their places and back.  Eight elements a thread; `lanes` threads (a power of two up to
// 256) walk a row, 256 / lanes tokens share a work-group, grid y divides long rows.  Memory bounds
// all three, and each byte is moved once: a token's row is read once for its top_k places, and its sum
// stays in registers.  Measured (MI355X, bf16, memory cold, all bytes read and written):
//   spread    4096 x 4096 to 8 places  302 MB  61.5 us  4.9 TB/s;  128 x 4096 5.8 us;  1 x 4096 4.7 us
//   combine   4096 x 4096 of 8 places  302 MB  62 us    4.9 TB/s;  128 x 4096 5.5 us;  1 x 4096 4.3 us
//   combine's gradient, 16384 x 2048 of 4 places, 604 MB with Z read for the weights' dots: 131 us,
//   4.6 TB/s (a copy of 4 GiB: 4.75 TB/s); of 65536 places 64 wide 19 us, 1.3 TB/s, where a wave a place
//   has work for 8 lanes and the vector unit, 129 instructions a wave, is busy for 0.87 of the time
// ---------------------------------------------------------------------------
struct RowsParams {
    const void *X, *Z, *R;       // spread: X; combine: Z, R; backward: X = dOut, Z
    void *Y, *dZ;                // spread, combine: Y
    int64_t ldx, ldz, ldr, ldy;  // backward: ldy of dZ
    int T, M, D, top_k, lanes;
    const int32_t* place;
    const float* weights;
    float* dweights;
};

template <int DT>
__global__ void __launch_bounds__(256) spread_kernel(const RowsParams p) {
    constexpr int ESZ = DT == DT_F32 ? 4 : 2;
    const int per = 256 / p.lanes, lx = threadIdx.x % p.lanes;
    const int64_t t = (int64_t)blockIdx.x * per + threadIdx.x / p.lanes;
    if (t >= p.T) return;
    const char* row = reinterpret_cast<const char*>(p.X) + t * p.ldx * ESZ;
    const int32_t* place = p.place + t * p.top_k;
    for (int64_t c = 8 * ((int64_t)blockIdx.y * p.lanes + lx); c < p.D;
         c += 8 * (int64_t)gridDim.y * p.lanes) {
        float v[8];
        load8<DT>(row, (int)c, p.D, v);
        for (int j = 0; j < p.top_k; ++j) {
            const uint32_t r = place[j];
            if (r >= (uint32_t)p.M) continue;
            char* y = reinterpret_cast<char*>(p.Y) + (int64_t)r * p.ldy * ESZ;
            if (p.weights) {
                const float w = p.weights[t * p.top_k + j];
                float s[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) s[i] = w * v[i];
                store8<DT>(y, (int)c, p.D, s);
            } else {
                store8<DT>(y, (int)c, p.D, v);
            }
        }
    }
}

// Rows are loaded four places at a time, so that their latencies overlap.
template <int DT>
__global__ void __launch_bounds__(256) combine_kernel(const RowsParams p) {
    constexpr int ESZ = DT == DT_F32 ? 4 : 2;
    const int per = 256 / p.lanes, lx = threadIdx.x % p.lanes;
    const int64_t t = (int64_t)blockIdx.x * per + threadIdx.x / p.lanes;
    if (t >= p.T) return;
    const int32_t* place = p.place + t * p.top_k;
    const float* weights = p.weights + t * p.top_k;
    const char* Z = reinterpret_cast<const char*>(p.Z);
    for (int64_t c = 8 * ((int64_t)blockIdx.y * p.lanes + lx); c < p.D;
         c += 8 * (int64_t)gridDim.y * p.lanes) {
        float acc[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
        if (p.R) load8<DT>(reinterpret_cast<const char*>(p.R) + t * p.ldr * ESZ, (int)c, p.D, acc);
        for (int j = 0; j < p.top_k; j += 4) {
            uint32_t r[4];
            float w[4];
            Raw8<DT> raw[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                r[i] = j + i < p.top_k ? (uint32_t)place[j + i] : ~0u;
                w[i] = p.weights && j + i < p.top_k ? weights[j + i] : 1.0f;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (r[i] < (uint32_t)p.M) raw[i].load(Z + (int64_t)r[i] * p.ldz * ESZ, (int)c, p.D);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (r[i] < (uint32_t)p.M) {
                    float v[8];
                    raw[i].get(v);
#pragma unroll
                    for (int k = 0; k < 8; ++k) acc[k] = __builtin_fmaf(w[i], v[k], acc[k]);
                }
        }
        store8<DT>(reinterpret_cast<char*>(p.Y) + t * p.ldy * ESZ, (int)c, p.D, acc);
    }
}

// One wave a place: its row of dZ, and the dot product for its weight, whose order of summing is fixed.
template <int DT>
__global__ void __launch_bounds__(256) combine_bwd_kernel(const RowsParams p) {
    constexpr int ESZ = DT == DT_F32 ? 4 : 2;
    const int lane = threadIdx.x & 63;
    const int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (i >= (int64_t)p.T * p.top_k) return;
    const uint32_t r = p.place[i];
    if (r >= (uint32_t)p.M) {
        if (p.dweights && lane == 0) p.dweights[i] = 0.0f;
        return;
    }
    const char* dout = reinterpret_cast<const char*>(p.X) + i / p.top_k * p.ldx * ESZ;
    const char* z = reinterpret_cast<const char*>(p.Z) + (int64_t)r * p.ldz * ESZ;
    char* dz = reinterpret_cast<char*>(p.dZ) + (int64_t)r * p.ldy * ESZ;
    const float w = p.weights[i];
    float dot = 0.0f;
    for (int64_t c = 8 * lane; c < p.D; c += 512) {
        float g[8], v[8];
        load8<DT>(dout, (int)c, p.D, g);
        if (p.dweights) {
            load8<DT>(z, (int)c, p.D, v);
#pragma unroll
            for (int k = 0; k < 8; ++k) dot = __builtin_fmaf(g[k], v[k], dot);
        }
        if (p.dZ) {
#pragma unroll
            for (int k = 0; k < 8; ++k) g[k] *= w;
            store8<DT>(dz, (int)c, p.D, g);
        }
    }
    if (p.dweights) {
        dot = wave_sum(dot);
        if (lane == 0) p.dweights[i] = dot;
    }
}

}  // namespace sg

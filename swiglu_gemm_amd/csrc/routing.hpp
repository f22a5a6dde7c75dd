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

template <typename T, typename F>
__device__ __forceinline__ T wave_reduce(T x, F f) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) x = f(x, __shfl_xor(x, d));
    return x;
}
__device__ __forceinline__ float wave_sum(float x) {
    return wave_reduce(x, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ double wave_sum(double x) {
    return wave_reduce(x, [](double a, double b) { return a + b; });
}
__device__ __forceinline__ float wave_max(float x) {
    return wave_reduce(x, [](float a, float b) { return fmaxf(a, b); });
}

// log of a score, up to what renormalising over the chosen cancels
__device__ __forceinline__ float log_score(int scoring, float x) {
    return scoring == ROUTE_SOFTMAX ? x : fminf(x, 0.0f) - log1pf(expf(-fabsf(x)));
}
__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

constexpr double kNone = -__builtin_huge_val();
constexpr double kNanKey = -1e300;        // a NaN logit: behind every number

// One wave a token; lane l holds experts l, l + 64, ...
template <int DT, int NV>
__global__ void __launch_bounds__(256) route_kernel(const RouteParams p) {
    __shared__ double lds[4][NV * 64];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int t = blockIdx.x * 4 + wave;
    if (t >= p.T) return;
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
    const bool scores = (p.bias || p.groups > 1) && !bad;
    if (scores || p.groups > 1) {
        double c[NV];
        if (scores) {
            if (p.scoring == ROUTE_SOFTMAX) {
                double sum = 0.0;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    c[i] = x[i] == -inf ? 0.0 : exp((double)x[i] - (double)top);
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
                if (p.bias && e < p.E) c[i] += (double)p.bias[e];
                if (x[i] == -inf || c[i] != c[i]) c[i] = kNone;
                if (p.bias) key[i] = c[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i) c[i] = key[i];
        }
        if (p.groups > 1) {
#pragma unroll
            for (int i = 0; i < NV; ++i) lds[wave][lane + 64 * i] = c[i];
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
            const int per = p.E / p.groups;
            double value = kNone;
            if (lane < p.groups) {
                double a = kNone, b = kNone;          // the two best
                for (int i = 0; i < per; ++i) {
                    const double v = lds[wave][lane * per + i];
                    b = fmax(b, fmin(a, v));
                    a = fmax(a, v);
                }
                value = p.group_top == 2 && b != kNone ? a + b : a;
            }
            int rank = 0;
            for (int g = 0; g < p.groups; ++g) {
                const double v = __shfl(value, g);
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
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const double b = __shfl_xor(best, d);
            const int f = __shfl_xor(e, d);
            const float w = __shfl_xor(v, d);
            if (b > best || (b == best && f < e)) {
                best = b;
                e = f;
                v = w;
            }
        }
        if (best == kNone) break;
        if (lane == j) {
            id = e;
            mine = v;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (lane + 64 * i == e) key[i] = kNone;
    }
    float w;
    if (p.renormalize) {
        const float l = id < 0 ? -inf : log_score(p.scoring, mine);
        const float m = wave_max(l);
        const float a = id < 0 ? 0.0f : expf(l - m);
        w = a / wave_sum(a);
    } else if (p.scoring == ROUTE_SOFTMAX) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) sum += x[i] == -inf ? 0.0f : expf(x[i] - top);
        w = expf(mine - top) / wave_sum(sum);
    } else {
        w = sigmoid(mine);
    }
    if (lane < p.top_k) {
        ids[lane] = id;
        weights[lane] = id < 0 ? 0.0f : bad ? __builtin_nanf("") : p.scale * w;
    }
}

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
            const float a = id < 0 ? 0.0f : expf(l - wave_max(l));
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
            const int e = __shfl(id, j);
            const float g = __shfl(v, j);
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

// A wave takes DEEP pieces of 256 ids at a time, so that as many loads are under way.
template <int WAVES, int DEEP>
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
    for (int i = first; i < last; i += STEP) {
        uint32_t v[DEEP][4];
        if (i == begin) ahead = eq;
        sort_load<DEEP>(p, i, lane, last, none, v);
#pragma unroll
        for (int d = 0; d < DEEP; ++d)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                lt += v[d][j] < e;
                eq += v[d][j] == e;
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
// 256) walk a row, 256 / lanes tokens share a work-group, grid y divides long rows of few tokens.
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

typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));

// Eight elements from column c of a row of D, as loaded; zeros behind the row.
template <int DT>
struct Raw8 {
    u32x4 a;
    __device__ __forceinline__ void load(const char* row, int c, int D) {
        if (c + 8 <= D) {
            a = *reinterpret_cast<const u32x4_any*>(row + (int64_t)c * 2);
        } else {
            const uint16_t* p = reinterpret_cast<const uint16_t*>(row) + c;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                a[i] = (c + 2 * i < D ? p[2 * i] : 0u) |
                       (c + 2 * i + 1 < D ? (uint32_t)p[2 * i + 1] << 16 : 0u);
        }
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = to_f32<DT>((uint16_t)a[i]);
            v[2 * i + 1] = to_f32<DT>((uint16_t)(a[i] >> 16));
        }
    }
};
template <>
struct Raw8<DT_F32> {
    f32x4 a, b;
    __device__ __forceinline__ void load(const char* row, int c, int D) {
        const float* p = reinterpret_cast<const float*>(row) + c;
        if (c + 8 <= D) {
            a = *reinterpret_cast<const f32x4_any*>(p);
            b = *reinterpret_cast<const f32x4_any*>(p + 4);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a[i] = c + i < D ? p[i] : 0.0f;
                b[i] = c + 4 + i < D ? p[4 + i] : 0.0f;
            }
        }
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = a[i];
            v[4 + i] = b[i];
        }
    }
};
template <int DT>
__device__ __forceinline__ void load8(const char* row, int c, int D, float (&v)[8]) {
    Raw8<DT> raw;
    raw.load(row, c, D);
    raw.get(v);
}
template <int DT>
__device__ __forceinline__ void store8(char* row, int c, int D, const float (&v)[8]) {
    if (c + 8 <= D) {
        if constexpr (DT == DT_F32) {
            *reinterpret_cast<f32x4_any*>(row + (int64_t)c * 4) = f32x4{v[0], v[1], v[2], v[3]};
            *reinterpret_cast<f32x4_any*>(row + (int64_t)c * 4 + 16) = f32x4{v[4], v[5], v[6], v[7]};
        } else {
            u32x4 a;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                a[i] = from_f32<DT>(v[2 * i]) | (uint32_t)from_f32<DT>(v[2 * i + 1]) << 16;
            *reinterpret_cast<u32x4_any*>(row + (int64_t)c * 2) = a;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < D) put_elem<DT>(row, c + i, v[i]);
    }
}

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

// One wave a place: its row of dZ, and the dot product for its weight.
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

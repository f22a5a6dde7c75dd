// api_routing.hip -- the C ABI of the routing to experts: argument checks and launches on the
// caller's stream.  Declarations and contracts are in include/swiglu_gemm.h.  Nothing here
// allocates or keeps a workspace.
#include <hip/hip_runtime.h>

#include "abi_checks.hpp"
#include "routing.hpp"
#include "swiglu_gemm.h"

using namespace sg;

namespace {

// Work-groups of 256 threads along one side of a grid: a launch has fewer than 2^32 threads there.
constexpr int64_t kMaxSide = ((int64_t)1 << 24) - 1;

#define SG_LAUNCH(KERNEL, GRID, BLOCK, ST, P) hipLaunchKernelGGL((KERNEL), GRID, BLOCK, 0, ST, P)

// Up to 256 experts and 8 choices several tokens share a wave; else each has one.  fp32 logits, 8
// choices: 1 token of 64 experts 3.3 against 3.4 us for one wave each, 16384 tokens 4.3 and 17.1 us, of
// 256 experts 7.7 and 21.7 us, of 256 in 8 groups with a bias 14.2 and 36.1 us.  That is for logits
// that differ.  Tokens whose order the lanes leave to 64 bits, or that have fewer than top_k experts
// left, hold up their wave one after the other, which the sizes do not show: logits cast from
// bf16 to fp32, 16384 tokens of 64 experts 13.3 and 18.5 us, of 256 experts 20.6 and 22.5 us, but 77 tokens
// 12.7 and 5.3 us; 8 choices with 6 experts left, 16384 tokens of 256 30 and 20 us, of 8 131 and 17 us.
template <int DT>
void launch_route(const RouteParams& p, hipStream_t st) {
    const dim3 block(256);
    auto waves = [&](int64_t tokens) { return dim3((unsigned)cdiv(p.T, 4 * tokens)); };
    if (p.E <= 256 && p.top_k <= 8) {
#define SG_ROUTE_LANES(L, V)                                                     \
    if (p.E <= L * V) {                                                          \
        SG_LAUNCH((route_lanes_kernel<DT, L, V>), waves(64 / L), block, st, p);  \
        return;                                                                  \
    }
        SG_ROUTE_LANES(1, 8)
        SG_ROUTE_LANES(2, 8)
        SG_ROUTE_LANES(4, 8)
        SG_ROUTE_LANES(8, 8)
        SG_ROUTE_LANES(16, 8)
        SG_ROUTE_LANES(16, 16)
#undef SG_ROUTE_LANES
    }
#define SG_ROUTE(NV)                                                     \
    if (p.E <= 64 * NV) {                                                \
        SG_LAUNCH((route_kernel<DT, NV>), waves(1), block, st, p);       \
        return;                                                          \
    }
    SG_ROUTE(1)
    SG_ROUTE(2)
    SG_ROUTE(4)
    SG_ROUTE(8)
    SG_ROUTE(16)
#undef SG_ROUTE
}

template <int DT>
void launch_route_bwd(const RouteParams& p, hipStream_t st) {
    const dim3 grid((unsigned)cdiv(p.T, 4)), block(256);
#define SG_ROUTE(NV)                                                     \
    if (p.E <= 64 * NV) {                                                \
        SG_LAUNCH((route_bwd_kernel<DT, NV>), grid, block, st, p);       \
        return;                                                          \
    }
    SG_ROUTE(1)
    SG_ROUTE(2)
    SG_ROUTE(4)
    SG_ROUTE(8)
    SG_ROUTE(16)
#undef SG_ROUTE
}

int run_route(bool bwd, int dtype, const RouteParams& p, hipStream_t st) {
    if (cdiv(p.T, 4) > kMaxSide) return status_of(hipErrorInvalidConfiguration);
    describe(bwd ? "route_experts_bwd" : "route_experts", -2, "");
    if (dtype == SG_F32) bwd ? launch_route_bwd<DT_F32>(p, st) : launch_route<DT_F32>(p, st);
    else if (dtype == SG_F16) bwd ? launch_route_bwd<DT_F16>(p, st) : launch_route<DT_F16>(p, st);
    else bwd ? launch_route_bwd<DT_BF16>(p, st) : launch_route<DT_BF16>(p, st);
    return status_of(hipGetLastError());
}

bool float_type(int dtype) { return dtype == SG_F32 || dtype == SG_F16 || dtype == SG_BF16; }

// Threads of a row and the grid: rows of up to 2048 elements share a work-group, longer ones are
// divided over grid y (bf16, 8 places: spreading 1 row of 4096 4.8 us, 6.4 us by one work-group; 4096
// rows of 4096 61.4 and 66.1 us; 4096 elements by 64 threads 76.9 us).
dim3 rows_grid(RowsParams& p) {
    const int64_t pieces = cdiv(p.D, 8);
    p.lanes = 1;
    while (p.lanes < 256 && p.lanes < pieces) p.lanes *= 2;
    const int64_t x = cdiv(p.T, 256 / p.lanes), y = cdiv(pieces, p.lanes);
    return dim3((unsigned)x, (unsigned)(y < 65535 ? y : 65535));
}

enum { SPREAD, COMBINE, COMBINE_BWD };
template <int DT>
void launch_rows(int what, const dim3& grid, const RowsParams& p, hipStream_t st) {
    if (what == SPREAD) SG_LAUNCH(spread_kernel<DT>, grid, dim3(256), st, p);
    else if (what == COMBINE) SG_LAUNCH(combine_kernel<DT>, grid, dim3(256), st, p);
    else SG_LAUNCH(combine_bwd_kernel<DT>, grid, dim3(256), st, p);
}
int run_rows(const char* name, int what, int dtype, const dim3& grid, const RowsParams& p,
             hipStream_t st) {
    describe(name, -2, "");
    if (dtype == SG_F32) launch_rows<DT_F32>(what, grid, p, st);
    else if (dtype == SG_F16) launch_rows<DT_F16>(what, grid, p, st);
    else launch_rows<DT_BF16>(what, grid, p, st);
    return status_of(hipGetLastError());
}

}  // namespace

extern "C" {

int sg_route_experts(const void* X, int64_t ldx, int64_t T, int64_t E, int dtype, int64_t top_k,
                     int scoring, const float* bias, int64_t groups, int64_t top_groups,
                     int group_top, int renormalize, float scale, const uint8_t* mask,
                     int32_t* ids, float* weights, void* stream) {
    if (T > 0 && !X) return -1;
    if (ldx < E) return -2;
    if (T < 0 || T > kMaxDim) return -3;
    if (E < 1 || E > SG_ROUTE_MAX_EXPERTS) return -4;
    if (!float_type(dtype)) return -5;
    if (top_k < 1 || top_k > E || top_k > SG_ROUTE_MAX_TOP_K) return -6;
    if (scoring != SG_ROUTE_SOFTMAX && scoring != SG_ROUTE_SIGMOID) return -7;
    if (groups < 1 || groups > 64 || E % groups != 0) return -9;
    if (top_groups < 1 || top_groups > groups) return -10;
    if (group_top != 1 && group_top != 2) return -11;
    if (renormalize != 0 && renormalize != 1) return -12;
    if (!std::isfinite(scale)) return -13;
    if (T > 0 && !ids) return -15;
    if (T > 0 && !weights) return -16;
    if (T == 0) return 0;
    RouteParams p{};
    p.X = X;
    p.ldx = ldx;
    p.T = (int)T;
    p.E = (int)E;
    p.top_k = (int)top_k;
    p.scoring = scoring;
    p.groups = top_groups == groups ? 1 : (int)groups;      // all of them: no choice of groups
    p.top_groups = (int)top_groups;
    p.group_top = group_top;
    p.renormalize = renormalize;
    p.scale = scale;
    p.bias = bias;
    p.mask = mask;
    p.ids = ids;
    p.weights = weights;
    return run_route(false, dtype, p, static_cast<hipStream_t>(stream));
}

int sg_route_experts_bwd(const void* X, int64_t ldx, int64_t T, int64_t E, int dtype,
                         int64_t top_k, int scoring, int renormalize, float scale,
                         const int32_t* ids, const float* dweights, void* dX, int64_t lddx,
                         void* stream) {
    if (T > 0 && !X) return -1;
    if (ldx < E) return -2;
    if (T < 0 || T > kMaxDim) return -3;
    if (E < 1 || E > SG_ROUTE_MAX_EXPERTS) return -4;
    if (!float_type(dtype)) return -5;
    if (top_k < 1 || top_k > E || top_k > SG_ROUTE_MAX_TOP_K) return -6;
    if (scoring != SG_ROUTE_SOFTMAX && scoring != SG_ROUTE_SIGMOID) return -7;
    if (renormalize != 0 && renormalize != 1) return -8;
    if (!std::isfinite(scale)) return -9;
    if (T > 0 && !ids) return -10;
    if (T > 0 && !dweights) return -11;
    if (T > 0 && !dX) return -12;
    if (lddx < E) return -13;
    if (T == 0) return 0;
    RouteParams p{};
    p.X = X;
    p.ldx = ldx;
    p.T = (int)T;
    p.E = (int)E;
    p.top_k = (int)top_k;
    p.scoring = scoring;
    p.renormalize = renormalize;
    p.scale = scale;
    p.chosen = ids;
    p.dweights = dweights;
    p.dX = dX;
    p.lddx = lddx;
    return run_route(true, dtype, p, static_cast<hipStream_t>(stream));
}

int sg_sort_experts(const int32_t* ids, int64_t n, int64_t experts, int32_t* offsets,
                    int32_t* order, int32_t* place, void* stream) {
    if (n > 0 && !ids) return -1;
    if (n < 0 || n > kMaxDim) return -2;
    if (experts < 1 || experts > kMaxExperts) return -3;
    if (!offsets) return -4;
    SortParams p{ids, (int)n, (int)experts, offsets, order, place};
    hipStream_t st = static_cast<hipStream_t>(stream);
    // Four waves up to 4096 ids (64 experts, 1024 ids: 2.9 us, 4.1 us with 16 waves; 4096: 4.7 and 5.6
    // us; 8192: 7.2 and 5.2 us).  The walk that writes is divided from 16384 ids on while the
    // work-groups fit the CUs one each (64 experts, 16384 ids in 3 parts 5.0 us, in one 5.7 us; 65536
    // in 3 parts 9.4 us, in one 13.8 us, in 4 12.0 us; of 8 experts in 8 parts 7.4 us, in one 15.4 us;
    // 8192 ids: no part helps).
    const int64_t fit = 256 / (experts + 1), parts = n < 16384 || fit < 1 ? 1 : fit < 8 ? fit : 8;
    const dim3 grid((unsigned)experts + 1, (unsigned)parts);
    describe("sort_experts", -2, "");
    if (n <= 4096) SG_LAUNCH((sort_kernel<4, 1, 1>), grid, dim3(256), st, p);
    else SG_LAUNCH((sort_kernel<16, 2, 4>), grid, dim3(1024), st, p);
    return status_of(hipGetLastError());
}

int sg_spread_rows(const void* X, int64_t ldx, int64_t T, int64_t D, int dtype,
                   const int32_t* place, int64_t top_k, const float* weights, int64_t M, void* Y,
                   int64_t ldy, void* stream) {
    const bool any = T > 0 && D > 0 && M > 0;
    if (any && !X) return -1;
    if (ldx < (D > 1 ? D : 1)) return -2;
    if (T < 0 || T > kMaxDim) return -3;
    if (D < 0 || D > kMaxDim) return -4;
    if (!float_type(dtype)) return -5;
    if (any && !place) return -6;
    if (top_k < 1 || top_k > 65536) return -7;
    if (M < 0 || M > kMaxDim) return -9;
    if (any && !Y) return -10;
    if (ldy < (D > 1 ? D : 1)) return -11;
    if (!any) return 0;
    RowsParams p{};
    p.X = X;
    p.ldx = ldx;
    p.T = (int)T;
    p.D = (int)D;
    p.place = place;
    p.top_k = (int)top_k;
    p.weights = weights;
    p.M = (int)M;
    p.Y = Y;
    p.ldy = ldy;
    const dim3 grid = rows_grid(p);
    if (grid.x > kMaxSide) return status_of(hipErrorInvalidConfiguration);
    return run_rows("spread_rows", SPREAD, dtype, grid, p, static_cast<hipStream_t>(stream));
}

int sg_combine_rows(const void* Z, int64_t ldz, int64_t M, int64_t D, int64_t T, int dtype,
                    const int32_t* place, int64_t top_k, const float* weights,
                    const void* residual, int64_t ldr, void* out, int64_t ldo, void* stream) {
    const bool any = T > 0 && D > 0;
    const int64_t row = D > 1 ? D : 1;
    if (any && M > 0 && !Z) return -1;
    if (ldz < row) return -2;
    if (M < 0 || M > kMaxDim) return -3;
    if (D < 0 || D > kMaxDim) return -4;
    if (T < 0 || T > kMaxDim) return -5;
    if (!float_type(dtype)) return -6;
    if (any && !place) return -7;
    if (top_k < 1 || top_k > 65536) return -8;
    if (residual && ldr < row) return -11;
    if (any && !out) return -12;
    if (ldo < row) return -13;
    if (!any) return 0;
    RowsParams p{};
    p.Z = Z;
    p.ldz = ldz;
    p.M = (int)M;
    p.D = (int)D;
    p.T = (int)T;
    p.place = place;
    p.top_k = (int)top_k;
    p.weights = weights;
    p.R = residual;
    p.ldr = ldr;
    p.Y = out;
    p.ldy = ldo;
    const dim3 grid = rows_grid(p);
    if (grid.x > kMaxSide) return status_of(hipErrorInvalidConfiguration);
    return run_rows("combine_rows", COMBINE, dtype, grid, p, static_cast<hipStream_t>(stream));
}

int sg_combine_rows_bwd(const void* dOut, int64_t lddo, const void* Z, int64_t ldz, int64_t M,
                        int64_t D, int64_t T, int dtype, const int32_t* place, int64_t top_k,
                        const float* weights, void* dZ, int64_t lddz, float* dweights,
                        void* stream) {
    const bool any = T > 0 && (dZ || dweights);
    const bool reads = any && D > 0 && M > 0;
    const int64_t row = D > 1 ? D : 1;
    if (reads && !dOut) return -1;
    if (lddo < row) return -2;
    if (reads && dweights && !Z) return -3;
    if (ldz < row) return -4;
    if (M < 0 || M > kMaxDim) return -5;
    if (D < 0 || D > kMaxDim) return -6;
    if (T < 0 || T > kMaxDim) return -7;
    if (!float_type(dtype)) return -8;
    if (any && !place) return -9;
    if (top_k < 1 || top_k > 65536) return -10;
    if (any && !weights) return -11;
    if (dZ && lddz < row) return -13;
    if (!any) return 0;
    const int64_t blocks = cdiv(T * top_k, 4);
    if (blocks > kMaxSide) return status_of(hipErrorInvalidConfiguration);
    RowsParams p{};
    p.X = dOut;
    p.ldx = lddo;
    p.Z = Z;
    p.ldz = ldz;
    p.M = (int)M;
    p.D = (int)D;
    p.T = (int)T;
    p.place = place;
    p.top_k = (int)top_k;
    p.weights = weights;
    p.dZ = dZ;
    p.ldy = lddz;
    p.dweights = dweights;
    return run_rows("combine_rows_bwd", COMBINE_BWD, dtype, dim3((unsigned)blocks), p,
                    static_cast<hipStream_t>(stream));
}

}  // extern "C"

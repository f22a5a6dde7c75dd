// grouped.hpp -- matrix products grouped by expert: the rows of A are sorted by
// expert, expert e owning rows [offsets[e], offsets[e+1]), and every expert has a
// weight of its own:
//
//   rows (TA = false)   C[r] = alpha * scale[e] * A[r] * op(B_e) + beta * C[r]
//                       or the SwiGLU of the same product, or its backward
//   depth (TA = true)   C_e = alpha * A[rows of e]^T * D[rows of e] + beta * C_e, the
//                       gradient of the weight: the ragged dimension is summed
//
// The offsets live on the device, so the host knows neither an expert's rows nor the
// number of tiles.  It launches an upper bound of the tiles; each work-group reads the
// offsets, finds its own (expert, tile) by a scan over the experts' tile counts, and
// leaves if there is none.  No second launch, no workspace, nothing shared between
// work-groups: concurrent calls and captured graphs cannot disturb one another.
// Offsets are clamped to [0, M] where they are read, so a bad table gives wrong rows
// but no access outside A and C.
#pragma once

#include <type_traits>

#include "epilogue16.hpp"
#include "sg_device.hpp"

namespace sg {

// Epilogues of the grouped kernels beside EPI_GEMM and EPI_SWIGLU.
enum : int {
    EPI_GEMM_F32 = 6,     // EPI_GEMM into an fp32 C
    EPI_SWIGLU_BWD = 7    // the gradient of SwiGLU's two arguments from dY
};

struct GroupedParams {
    Gemm16Params g;           // M: rows of all experts (rows) or of C (depth); K: depth (rows)
    const int32_t* offsets;   // experts + 1 row numbers; nullptr: one expert owns every row
    const float* scale;       // nullptr, or one factor for each expert (rows)
    const void* dY;           // EPI_SWIGLU_BWD: M x N/2 (N: the fused width), contiguous
    int experts;
    int rows;                 // rows of A in all (depth: the summed dimension)
    int64_t sB, sC;           // bytes from one expert's B (rows) or C (depth) to the next
};

__device__ __forceinline__ int group_offset(const GroupedParams& q, int e) {
    return min(max(q.offsets[e], 0), q.rows);
}

// The work of one work-group: expert e, whose rows are [row0, row0 + rows), and the rows from
// m0 on and columns from tile tn of its product; half: only half of the tile's rows.
struct GroupItem {
    int e, row0, rows, m0, tn;
    bool half;
};

// The item of work-group `bid` among `total`: consecutive items share an XCD (as xcd_remap).
// OCC > 0 (the work-groups of a CU, for kernels that have a tile of half the rows): where the
// items of an XCD leave its last round at most half full, that round's items are split into
// two halves each, which finish it in 0.6 of the time (4-bit, 8 experts of 1024 rows, 4096 x
// 4096: 109 -> 98 us).  The launch has room for them: group_blocks().
constexpr int kXcds = 8, kXcdCus = 32;
template <int OCC>
__device__ __forceinline__ bool xcd_item(int bid, int total, int& lid, int& part) {
    part = -1;
    if (total < kXcds) {
        lid = bid;
        return bid < total;
    }
    const int x = bid % kXcds, i = bid / kXcds, per = total / kXcds, rem = total % kXcds;
    const int n = per + (x < rem), first = x * per + min(x, rem);
    int split = 0;
    if constexpr (OCC > 0) {
        constexpr int slots = kXcdCus * OCC;
        split = n % slots;
        if (n <= slots || 2 * split > slots) split = 0;
    }
    const int j = i - (n - split);
    if (j >= 2 * split) return false;
    lid = first + (j < 0 ? i : n - split + j / 2);
    if (j >= 0) part = j & 1;
    return true;
}
inline int64_t group_blocks(int64_t items, int occ) { return items + kXcds * kXcdCus * occ / 2; }

// The sum of x over the lanes up to and including this one: data-parallel moves within rows of
// 16 lanes (row_shr), then the rows' last values to the rows behind (row_bcast).
template <int CTRL, int ROWS, int BANKS>
__device__ __forceinline__ int lane_moved(int x) {
    return __builtin_amdgcn_update_dpp(0, x, CTRL, ROWS, BANKS, false);
}
__device__ __forceinline__ int lane_scan(int x) {
    x += lane_moved<0x111, 0xf, 0xf>(x);       // row_shr:1
    x += lane_moved<0x112, 0xf, 0xf>(x);       // row_shr:2
    x += lane_moved<0x114, 0xf, 0xe>(x);       // row_shr:4
    x += lane_moved<0x118, 0xf, 0xc>(x);       // row_shr:8
    x += lane_moved<0x142, 0xa, 0xf>(x);       // row_bcast:15
    x += lane_moved<0x143, 0xc, 0xf>(x);       // row_bcast:31
    return x;
}

// Finds the item of work-group `bid` for products over an expert's rows in tiles of BM
// rows; false if there are fewer items.  Every lane of a wave calls it and gets the same
// answer in scalar registers: lane l counts the tiles of experts [l*P, (l+1)*P), P =
// ceil(experts / 64), a scan over the lanes finds the one that holds the item, and its
// experts are walked.  Consecutive items share an XCD, and an expert's items follow one
// another, so that its weight is read while it is in that XCD's L2.
template <int BM, int OCC = 0>
__device__ __forceinline__ bool find_rows(const GroupedParams& q, int bid, int lane,
                                          GroupItem& it) {
    const int tiles_n = q.g.tiles_n;
    int tm, lid, part;
    if (!q.offsets) {
        const int tiles_m = (q.rows + BM - 1) / BM;
        if (!xcd_item<OCC>(bid, tiles_m * tiles_n, lid, part)) return false;
        it.e = 0;
        it.row0 = 0;
        it.rows = q.rows;
        tile_coords(lid, tiles_m, tiles_n, q.g.group_m, tm, it.tn);
        it.m0 = tm * BM + (part > 0 ? BM / 2 : 0);
        it.half = part >= 0;
        return it.m0 < it.rows;
    }
    const int per = (q.experts + 63) / 64;
    int mine = 0, row = 0, len = 0;                // row, len: the lane's expert where per is 1
    for (int j = 0; j < per; ++j) {
        const int e = lane * per + j;
        if (e >= q.experts) break;
        row = group_offset(q, e);
        len = group_offset(q, e + 1) - row;
        if (len > 0) mine += (len + BM - 1) / BM;
    }
    const int incl = lane_scan(mine);
    const int total = __builtin_amdgcn_readlane(incl, 63) * tiles_n;
    if (!xcd_item<OCC>(bid, total, lid, part)) return false;
    const uint64_t past = __ballot(incl * tiles_n > lid);
    if (past == 0) return false;
    const int owner = __builtin_ctzll(past);
    int first = __builtin_amdgcn_readlane(incl - mine, owner) * tiles_n;
    const int last = min(q.experts, (owner + 1) * per) - 1;
    int e = owner * per;
    int row0 = __builtin_amdgcn_readlane(row, owner), n = __builtin_amdgcn_readlane(len, owner);
    int tiles_m = n > 0 ? (n + BM - 1) / BM : 0;
    if (per > 1) {
        for (;; ++e) {
            row0 = __builtin_amdgcn_readfirstlane(group_offset(q, e));
            n = __builtin_amdgcn_readfirstlane(group_offset(q, e + 1)) - row0;
            tiles_m = n > 0 ? (n + BM - 1) / BM : 0;
            if (lid < first + tiles_m * tiles_n || e >= last) break;
            first += tiles_m * tiles_n;
        }
    }
    // a table that does not ascend can count more tiles than an int holds: no item then
    if (lid < first || lid - first >= tiles_m * tiles_n) return false;
    it.e = e;
    it.row0 = row0;
    it.rows = n;
    tile_coords(lid - first, tiles_m, tiles_n, q.g.group_m, tm, it.tn);
    it.m0 = tm * BM + (part > 0 ? BM / 2 : 0);
    it.half = part >= 0;
    return it.m0 < n;
}

// The same for products that sum over an expert's rows: tiles_m x tiles_n tiles of C for
// every expert, whatever its rows.  An item's work goes with its expert's rows, so each
// expert's tiles are dealt to all XCDs (a compact block of them to each), and the experts
// come in order of their rows, the longest first, so that short items end the launch.  (Up to
// 64 experts, one a lane; more come in their own order.)
template <int BM>
__device__ __forceinline__ bool find_depth(const GroupedParams& q, int bid, int lane,
                                           GroupItem& it) {
    const int per = q.g.tiles_m * q.g.tiles_n;
    if (bid >= per * q.experts) return false;
    const int place = bid / per;
    int n;
    if (q.experts <= 64) {
        const int e = min(lane, q.experts - 1), row = group_offset(q, e);
        const int rows = lane < q.experts ? group_offset(q, e + 1) - row : -1;
        int before = 0;
        for (int j = 0; j < q.experts; ++j) {
            const int other = __builtin_amdgcn_readlane(rows, j);
            before += other > rows || (other == rows && j < lane);
        }
        it.e = __builtin_ctzll(__ballot(lane < q.experts && before == place));
        it.row0 = __builtin_amdgcn_readlane(row, it.e);
        n = __builtin_amdgcn_readlane(rows, it.e);
    } else {
        it.e = place;
        it.row0 = __builtin_amdgcn_readfirstlane(group_offset(q, place));
        n = __builtin_amdgcn_readfirstlane(group_offset(q, place + 1)) - it.row0;
    }
    it.rows = n > 0 ? n : 0;
    int tm;
    tile_coords(xcd_remap(bid - place * per, per), q.g.tiles_m, q.g.tiles_n, q.g.group_m, tm,
                it.tn);
    it.m0 = tm * BM;
    return true;
}

// The expert's own problem: operands, output and sizes from the item.  ESZ: bytes of an
// operand element; CSZ: of an output element.  Depth: an expert without rows has no products,
// and alpha, which may be infinite, does not count.
template <bool TA, int ESZ, int CSZ>
__device__ __forceinline__ Gemm16Params group_problem(const GroupedParams& q,
                                                      const GroupItem& it) {
    Gemm16Params p = q.g;
    const char* A = reinterpret_cast<const char*>(q.g.A);
    const char* B = reinterpret_cast<const char*>(q.g.B);
    p.A = reinterpret_cast<const uint16_t*>(A + (int64_t)it.row0 * p.lda * ESZ);
    if constexpr (TA) {
        p.B = reinterpret_cast<const uint16_t*>(B + (int64_t)it.row0 * p.ldb * ESZ);
        p.C = reinterpret_cast<char*>(q.g.C) + it.e * q.sC;
        p.K = it.rows;
        if (it.rows == 0) p.alpha = 0.0f;
    } else {
        p.B = reinterpret_cast<const uint16_t*>(B + it.e * q.sB);
        p.C = reinterpret_cast<char*>(q.g.C) + (int64_t)it.row0 * p.ldc * CSZ;
        p.M = it.rows;
        p.tiles_m = 0;
        if (q.scale) p.alpha *= q.scale[it.e];
    }
    return p;
}

// d/dg and d/du of SiLU(g) * u, times dy.  With s = 1/(1 + e^-g): SiLU = g s and
// SiLU' = s (1 + g (1 - s)).
// The two leave in dy's 16-bit type, rounded once (bf16: by at most 2^-8 of the value), because the
// products that take them next read 16-bit operands: gradients of 8192 rows of 16 experts, 2048 x 2
// x 1408, are then off by 0.0023 in relative 2-norm, 0.0017 if dH stays fp32.
__device__ __forceinline__ void swiglu_grad(float g, float u, float dy, float& dg, float& du) {
    const float s =
        __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.44269504088896341f));
    dg = dy * u * s * (1.0f + g * (1.0f - s));
    du = dy * g * s;
}

// Four consecutive columns n .. n+3 of row m from their sums, element by element: any
// alignment, columns past N left out.
template <int DT_OUT, int EPI, bool SCALED>
__device__ __forceinline__ void group_store(const Gemm16Params& p, const uint16_t* dy_row, int m,
                                            int n, const float (&a)[4]) {
    if constexpr (EPI == EPI_GEMM || EPI == EPI_GEMM_F32) {
        const EpiEx none{};
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (n + e < p.N)
                store_elem<EPI == EPI_GEMM_F32 ? DT_F32 : DT_OUT>(
                    p.C, (int64_t)m * p.ldc + n + e, n + e, p.alpha * a[e], p.beta, none);
    } else if constexpr (EPI == EPI_SWIGLU) {
        uint16_t* y = reinterpret_cast<uint16_t*>(p.C) + (int64_t)m * p.ldc + (n >> 1);
#pragma unroll
        for (int e = 0; e < 4; e += 2)
            if (n + e + 1 < p.N)
                y[e >> 1] = from_f32<DT_OUT>(
                    SCALED ? silu(p.alpha * a[e]) * (p.alpha * a[e + 1]) : silu(a[e]) * a[e + 1]);
    } else {
        uint16_t* dh = reinterpret_cast<uint16_t*>(p.C) + (int64_t)m * p.ldc + n;
#pragma unroll
        for (int e = 0; e < 4; e += 2)
            if (n + e + 1 < p.N) {
                float dg, du;
                swiglu_grad(a[e], a[e + 1], to_f32<DT_OUT>(dy_row[(n + e) >> 1]), dg, du);
                dh[e] = from_f32<DT_OUT>(dg);
                dh[e + 1] = from_f32<DT_OUT>(du);
            }
    }
}

// ---------------------------------------------------------------------------
// The kernel for every stride and alignment: 64 x 64 tiles, four waves of one 32 x 32
// accumulator each, depth 32 at a time staged through LDS element by element (zeros past
// the edges, nothing read there).  e4m3 codes are widened to bf16 on the way, which holds
// every one of them exactly.
// ---------------------------------------------------------------------------
template <int DT>
__device__ __forceinline__ uint16_t group_elem(const void* base, int64_t i) {
    if constexpr (DT == DT_E4M3) {
        const uint32_t c = reinterpret_cast<const uint8_t*>(base)[i];
        return from_f32<DT_BF16>(__builtin_amdgcn_cvt_f32_fp8((int)c, 0));
    } else {
        return reinterpret_cast<const uint16_t*>(base)[i];
    }
}

template <int DT, bool TA, bool TB, int EPI>
__global__ void __launch_bounds__(256) grouped_any_kernel(const GroupedParams q) {
    constexpr int ESZ = DT == DT_E4M3 ? 1 : 2, CSZ = EPI == EPI_GEMM_F32 ? 4 : 2;
    constexpr int DT_OUT = DT == DT_E4M3 ? DT_BF16 : DT;
    constexpr int T = 64, BK = 32, LD = BK + 8;
    __shared__ __attribute__((aligned(16))) uint16_t As[T * LD], Bs[T * LD];
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    GroupItem it;
    if constexpr (TA) {
        if (!find_depth<T>(q, blockIdx.x, lane, it)) return;
    } else {
        if (!find_rows<T>(q, blockIdx.x, lane, it)) return;
    }
    const Gemm16Params p = group_problem<TA, ESZ, CSZ>(q, it);
    const int m0 = it.m0, n0 = it.tn * T;
    f32x16 acc;
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[e] = 0.0f;
    for (int k0 = 0; k0 < p.K; k0 += BK) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < T * BK / 256; ++i) {
            const int x = tid + i * 256;
            {   // op(A): consecutive threads along the stored row
                const int r = TA ? x % T : x / BK, k = TA ? x / T : x % BK;
                const bool in = m0 + r < p.M && k0 + k < p.K;
                const int64_t at = TA ? (int64_t)(k0 + k) * p.lda + m0 + r
                                      : (int64_t)(m0 + r) * p.lda + k0 + k;
                As[r * LD + k] = in ? group_elem<DT>(p.A, at) : (uint16_t)0;
            }
            {
                const int r = TB ? x / BK : x % T, k = TB ? x % BK : x / T;
                const bool in = n0 + r < p.N && k0 + k < p.K;
                const int64_t at = TB ? (int64_t)(n0 + r) * p.ldb + k0 + k
                                      : (int64_t)(k0 + k) * p.ldb + n0 + r;
                Bs[r * LD + k] = in ? group_elem<DT>(p.B, at) : (uint16_t)0;
            }
        }
        __syncthreads();
        const int at = (lane & 31) * LD + 8 * (lane >> 5);
#pragma unroll
        for (int s = 0; s < BK; s += 16) {
            const u32x4 b = *reinterpret_cast<const u32x4*>(Bs + (wave >> 1) * 32 * LD + at + s);
            const u32x4 a = *reinterpret_cast<const u32x4*>(As + (wave & 1) * 32 * LD + at + s);
            acc = mfma16<DT_OUT>(b, a, acc);
        }
    }
    const int m = m0 + (wave & 1) * 32 + (lane & 31);
    if (m >= p.M) return;
    const uint16_t* dy = nullptr;
    if constexpr (EPI == EPI_SWIGLU_BWD)
        dy = reinterpret_cast<const uint16_t*>(q.dY) + (int64_t)(it.row0 + m) * (p.N >> 1);
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        const int n = n0 + (wave >> 1) * 32 + 8 * g + 4 * (lane >> 5);
        const float a[4] = {acc[4 * g], acc[4 * g + 1], acc[4 * g + 2], acc[4 * g + 3]};
        group_store<DT_OUT, EPI, DT == DT_E4M3>(p, dy, m, n, a);
    }
}

// Launches the kernels of one operand type: epi as above, ta: depth; cfg < 0: the kernel
// for every alignment.  blocks: the host's upper bound of the items.
template <int DT>
hipError_t launch_grouped(int epi, bool ta, bool tb, int cfg, const GroupedParams& q,
                          unsigned blocks, hipStream_t st);

}  // namespace sg

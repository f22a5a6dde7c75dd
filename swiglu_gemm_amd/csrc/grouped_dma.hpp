// grouped_dma.hpp -- the grouped products on the direct-to-LDS tile loop of
// gemm16_dma.hpp: a work-group finds its item (grouped.hpp) and runs the loop and the
// epilogue on the expert's own problem.  Operands 16-byte aligned, rows and expert strides
// 16-byte multiples.
#pragma once

#include "gemm16_dma.hpp"
#include "grouped.hpp"

namespace sg {

// C in fp32: C = alpha * acc + beta * C_old.  As epilogue_gemm_rows_beta_lds, with 16-byte
// pieces of four outputs: one 32-row block of every wave row and CW wave columns at a time
// pass through LDS, so that C is read and written along its rows.
template <int FM, int FN, int BM, int BN, int WN, int NT, int LDSB>
__device__ __forceinline__ void epilogue_f32_rows_lds(const Gemm16Params& p, f32x16 (&acc)[FN][FM],
                                                      char* smem, int m0, int n0, int rb, int wn,
                                                      int lane) {
    constexpr int TN = BN / WN, CW = staged_wave_cols<BM, BN, FM, WN, LDSB, 0>();
    static_assert(CW > 0, "one wave column of fp32 rows fits the LDS ring");
    constexpr int TS = CW * TN, ROW = 4 * TS + 16, CPR = TS / 4;
    constexpr int PB = BM / (32 * FM) * 32 * CPR;
    const int lm = lane & 31, lq = (lane >> 5) * 4, wr = rb / (32 * FM);
    const float alpha = p.alpha, beta = p.beta;
    float* C = reinterpret_cast<float*>(p.C);
    const bool vec = (reinterpret_cast<uintptr_t>(C) & 15) == 0 && (p.ldc & 3) == 0;
#pragma unroll
    for (int tm = 0; tm < FM; ++tm) {
#pragma unroll
        for (int h = 0; h < WN / CW; ++h) {
            __syncthreads();
            if (wn / CW == h) {
                char* row = smem + (wr * 32 + lm) * ROW + 4 * (wn % CW) * TN;
#pragma unroll
                for (int tn = 0; tn < FN; ++tn)
#pragma unroll
                    for (int g = 0; g < 4; ++g)
                        *reinterpret_cast<f32x4*>(row + 4 * (tn * 32 + 8 * g + lq)) =
                            f32x4{alpha * acc[tn][tm][4 * g], alpha * acc[tn][tm][4 * g + 1],
                                  alpha * acc[tn][tm][4 * g + 2], alpha * acc[tn][tm][4 * g + 3]};
            }
            __syncthreads();
            for (int i = threadIdx.x; i < PB; i += NT) {
                const int rr = i / CPR, c = i - rr * CPR;
                const int m = m0 + (rr >> 5) * (32 * FM) + tm * 32 + (rr & 31);
                const int n = n0 + h * TS + c * 4;
                if (m >= p.M || n >= p.N) continue;
                f32x4 v = *reinterpret_cast<const f32x4*>(smem + rr * ROW + c * 16);
                float* cp = C + (int64_t)m * p.ldc + n;
                if (vec && n + 4 <= p.N) {
                    if (beta != 0.0f) {
                        const f32x4 old = *reinterpret_cast<const f32x4*>(cp);
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[e] = __builtin_fmaf(beta, old[e], v[e]);
                    }
                    *reinterpret_cast<f32x4*>(cp) = v;
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (n + e < p.N)
                            cp[e] = beta != 0.0f ? __builtin_fmaf(beta, cp[e], v[e]) : v[e];
                }
            }
        }
    }
}

// The gradient of gate and up from dY, staged the same way: eight interleaved columns (four
// pairs) a piece meet four values of dY and leave as one 16-byte store.  dy: the expert's
// first row of dY.
template <int DT, int FM, int FN, int BM, int BN, int WN, int NT, int LDSB>
__device__ __forceinline__ void epilogue_swiglu_bwd_lds(const Gemm16Params& p, const uint16_t* dy,
                                                        f32x16 (&acc)[FN][FM], char* smem, int m0,
                                                        int n0, int rb, int wn, int lane) {
    constexpr int TN = BN / WN, CW = staged_wave_cols<BM, BN, FM, WN, LDSB, 0>();
    static_assert(CW > 0, "one wave column of fp32 rows fits the LDS ring");
    constexpr int TS = CW * TN, ROW = 4 * TS + 16, CPR = TS / 8;
    constexpr int PB = BM / (32 * FM) * 32 * CPR;
    const int lm = lane & 31, lq = (lane >> 5) * 4, wr = rb / (32 * FM);
    const int nout = p.N >> 1;
    uint16_t* H = reinterpret_cast<uint16_t*>(p.C);
    const bool vec = (reinterpret_cast<uintptr_t>(H) & 15) == 0 &&
                     (reinterpret_cast<uintptr_t>(dy) & 7) == 0 && (nout & 3) == 0;
#pragma unroll
    for (int tm = 0; tm < FM; ++tm) {
#pragma unroll
        for (int h = 0; h < WN / CW; ++h) {
            __syncthreads();
            if (wn / CW == h) {
                char* row = smem + (wr * 32 + lm) * ROW + 4 * (wn % CW) * TN;
#pragma unroll
                for (int tn = 0; tn < FN; ++tn)
#pragma unroll
                    for (int g = 0; g < 4; ++g)
                        *reinterpret_cast<f32x4*>(row + 4 * (tn * 32 + 8 * g + lq)) =
                            f32x4{acc[tn][tm][4 * g], acc[tn][tm][4 * g + 1],
                                  acc[tn][tm][4 * g + 2], acc[tn][tm][4 * g + 3]};
            }
            __syncthreads();
            for (int i = threadIdx.x; i < PB; i += NT) {
                const int rr = i / CPR, c = i - rr * CPR;
                const int m = m0 + (rr >> 5) * (32 * FM) + tm * 32 + (rr & 31);
                const int n = n0 + h * TS + c * 8;
                if (m >= p.M || n >= p.N) continue;
                const char* src = smem + rr * ROW + c * 32;
                const f32x4 lo = *reinterpret_cast<const f32x4*>(src);
                const f32x4 hi = *reinterpret_cast<const f32x4*>(src + 16);
                const float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
                const uint16_t* d = dy + (int64_t)m * nout + (n >> 1);
                uint16_t* out = H + (int64_t)m * p.ldc + n;
                const bool whole = vec && n + 8 <= p.N;
                uint16_t dv[4] = {0, 0, 0, 0};
                if (whole) {
                    const u32x2 w = *reinterpret_cast<const u32x2*>(d);
                    dv[0] = (uint16_t)w.x, dv[1] = (uint16_t)(w.x >> 16);
                    dv[2] = (uint16_t)w.y, dv[3] = (uint16_t)(w.y >> 16);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (n + 2 * j < p.N) dv[j] = d[j];
                }
                float o[8];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    swiglu_grad(v[2 * j], v[2 * j + 1], to_f32<DT>(dv[j]), o[2 * j], o[2 * j + 1]);
                if (whole) {
                    __builtin_nontemporal_store(
                        u32x4{pack2<DT>(o[0], o[1]), pack2<DT>(o[2], o[3]), pack2<DT>(o[4], o[5]),
                              pack2<DT>(o[6], o[7])},
                        reinterpret_cast<u32x4*>(out));
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (n + e < p.N) out[e] = from_f32<DT>(o[e]);
                }
            }
        }
    }
}

// Whether the partial K tile at the end of a tile's loop may be read whole: everything it would
// load behind K, rows clamped to the tile's own, lies in front of `end`, the row behind the last
// expert's, and inside the experts' matrices.  Rows of no expert and gaps between the matrices are
// not read; what lies between one row's end and the next row may be, and the fragments are cut so
// that none of it counts.
template <bool TA, bool TB, int BM, int BN, int BK, int ESZ>
__host__ __device__ inline bool tail_readable(const GroupedParams& q, const GroupItem& it,
                                              const Gemm16Params& p, int end, int m0, int n0,
                                              int nkt) {
    const int past = (nkt + 1) * BK;                     // the whole tile's last k, plus 1
    if constexpr (TA) {
        // k are rows of A and D; past the expert's rows come the next expert's
        return it.row0 + past <= end;
    } else {
        // A: k run along a row, so past K comes the next row, if there is one
        const int rows = m0 + BM < p.M ? m0 + BM : p.M;
        const bool a_in = it.row0 + rows < end && past <= q.g.lda + p.K;
        const bool more = it.e + 1 < q.experts && q.sB == (int64_t)(TB ? p.N : p.K) * p.ldb * ESZ;
        const bool b_in = TB ? (more || n0 + BN < p.N) && past <= p.ldb + p.K
                             : more && past - p.K <= p.K;
        return a_in && b_in;
    }
}

template <int DT, bool TA, bool TB, int EPI, int BM, int BN, int BK, int S, int WM, int WN>
__device__ __forceinline__ void grouped_tile(const GroupedParams& q, const GroupItem& it,
                                             const Gemm16Params& p, char* smem, int wave,
                                             int lane) {
    using D = DmaShape<DT, TA, TB, EPI, BM, BN, BK, S, WM, WN>;
    const int m0 = it.m0, n0 = it.tn * BN;
    const int nkt = p.K / BK, ktail = p.K - nkt * BK;
    typename D::Acc acc;
#pragma unroll
    for (int i = 0; i < D::FN; ++i)
#pragma unroll
        for (int j = 0; j < D::FM; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
    bool ring_tail = false;
    if (ktail > 0) {
        const int end = __builtin_amdgcn_readfirstlane(group_offset(q, q.experts));
        ring_tail = tail_readable<TA, TB, BM, BN, BK, D::ESZ>(q, it, p, end, m0, n0, nkt);
    }
    dma_mainloop<DT, TA, TB, EPI, BM, BN, BK, S, WM, WN, true>(p, smem, m0, n0, 0, nkt, ktail, acc,
                                                               wave, lane, ring_tail);
    const int wm = wave % WM, wn = wave / WM;
    if constexpr (EPI == EPI_GEMM_F32)
        epilogue_f32_rows_lds<D::FM, D::FN, BM, BN, WN, 64 * WM * WN, D::LDS>(
            p, acc, smem, m0, n0, wm * D::TM, wn, lane);
    else if constexpr (EPI == EPI_SWIGLU_BWD)
        epilogue_swiglu_bwd_lds<D::DT_OUT, D::FM, D::FN, BM, BN, WN, 64 * WM * WN, D::LDS>(
            p, reinterpret_cast<const uint16_t*>(q.dY) + (int64_t)it.row0 * (p.N >> 1), acc, smem,
            m0, n0, wm * D::TM, wn, lane);
    else
        dma_epilogue<DT, TA, TB, EPI, BM, BN, BK, S, WM, WN>(p, acc, smem, m0, n0, wave, lane);
}

// Two work-groups a CU where the ring takes at most half of its LDS.
constexpr int group_occ(int lds) { return lds <= 80 * 1024 ? 2 : 1; }

// The height on which a tile of products over rows runs an expert's last rows where they fit
// (same columns, same number of waves), 0: none.  Half of the height takes 0.6 of the time of a
// whole one (64 of 192 rows for 48 experts of 250 rows in the mean, e4m3: 142 -> 137 us).
constexpr int group_low(bool ta, int bm, int bn, int wm, int wn) {
    if (ta) return 0;
    if (bm == 256 && wm * wn == 8) return 128;
    if (bm == 192 && wm * wn == 8) return 64;
    return bm == 128 && bn == 256 && wm * wn == 4 ? 64 : 0;
}

template <int DT, bool TA, bool TB, int EPI, int BM, int BN, int BK, int S, int WM, int WN>
__global__ void __launch_bounds__(
    64 * WM * WN, group_occ(DmaShape<DT, TA, TB, EPI, BM, BN, BK, S, WM, WN>::LDS))
    grouped_dma_kernel(const GroupedParams q) {
    using D = DmaShape<DT, TA, TB, EPI, BM, BN, BK, S, WM, WN>;
    constexpr int LOW = group_low(TA, BM, BN, WM, WN);
    constexpr int S2 = BM == 256 ? 3 : S, WM2 = WM * WN == 8 ? 2 : 1, WN2 = 4;
    constexpr int LDS_LOW = LOW > 0 ? S2 * (LOW + BN) * BK * D::ESZ : 0;
    __shared__ __attribute__((aligned(1024))) char smem[LDS_LOW > D::LDS ? LDS_LOW : D::LDS];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    GroupItem it;
    if constexpr (TA) {
        if (!find_depth<BM>(q, blockIdx.x, lane, it)) return;
    } else {
        if (!find_rows<BM, 2 * LOW == BM ? group_occ(D::LDS) : 0>(q, blockIdx.x, lane, it)) return;
    }
    const Gemm16Params p = group_problem<TA, D::ESZ, EPI == EPI_GEMM_F32 ? 4 : 2>(q, it);
    if constexpr (LOW > 0) {
        if (it.half || it.rows - it.m0 <= LOW) {
            grouped_tile<DT, TA, TB, EPI, LOW, BN, BK, S2, WM2, WN2>(q, it, p, smem, wave, lane);
            return;
        }
    }
    grouped_tile<DT, TA, TB, EPI, BM, BN, BK, S, WM, WN>(q, it, p, smem, wave, lane);
}

// Tiles of the grouped products.  Index = configuration id (SG_FORCE_GROUPED=<id> overrides
// the choice; -1: the kernel for every alignment).  rate and fixed are the cost model's: TFLOP/s
// of a CU and the time a tile costs beside its products (_d: products that sum over rows; 0:
// not for these).  They were fitted, near the rates of single tiles, to every tile forced on
// 38 problems (1 to 64 experts, 1 to 16384 rows, K and N 724 to 5000) for each layout, SwiGLU
// and the weight gradient; the model's choice is 1.6 % above the best tile in the mean for
// 16-bit and 1.1 % for e4m3 rows, 2.5 % for weight gradients.
//
// What the tiles are for (MI355X, bf16, weights cold): 32 x 128, which streams a weight for a
// few rows: 64 experts of 4 rows, 2048 x 1536: 72 us, 76-81 us on the wider ones; 32 x 64 where
// even those leave CUs idle: 2 rows, 896 x 1792: 10.2 against 13.1 us.  128 x 256 with a
// 32-deep ring, two work-groups a CU that fill each other's gaps: 32 uneven experts of 512
// rows in the mean, 2048 x 2048: 158 us against 190 us for 256 x 256 (one work-group a CU,
// whole rounds of long tiles) and 172 us for the 64-deep 128 x 256, which is ahead where its
// tiles make about one round (16 experts of 128 rows, 2048 x 2816: 44 against 52 us); 256 x 256
// where experts are long: 4096 rows of one 64 us against 68 and 70 us.  e4m3: 192 x 128, two a
// CU: 48 experts of 250 rows, 1536 x 4096: 130 us against 142 us on 128 x 128, 137 us on
// 128 x 256 and 139 us on 256 x 256.
struct GroupCfg {
    int e4m3, BM, BN, BK, S, WM, WN;
    double rate, fixed, rate_d, fixed_d;
    const char* name;
};
constexpr GroupCfg kGroupCfg[] = {
    {0, 32, 64, 64, 6, 1, 2, 1.18, 1.44, 0.0, 0.0, "32x64x64 s6 1x2w"},
    {0, 32, 128, 64, 4, 1, 4, 2.49, 2.02, 0.0, 0.0, "32x128x64 s4 1x4w"},
    {0, 128, 128, 64, 2, 2, 4, 0.0, 0.0, 4.0, 2.96, "128x128x64 s2 2x4w"},
    {0, 128, 256, 64, 3, 2, 4, 4.47, 2.8, 0.0, 0.0, "128x256x64 s3 2x4w"},
    {0, 128, 256, 32, 3, 2, 2, 5.0, 2.94, 4.3, 2.03, "128x256x32 s3 2x2w"},
    {0, 256, 256, 64, 2, 4, 2, 4.89, 4.07, 5.17, 5.06, "256x256x64 s2 4x2w"},
    {1, 32, 128, 128, 4, 1, 4, 3.67, 2.76, 0.0, 0.0, "e4m3 32x128x128 s4 1x4w"},
    {1, 128, 128, 128, 2, 2, 4, 6.94, 2.01, 0.0, 0.0, "e4m3 128x128x128 s2 2x4w"},
    {1, 192, 128, 128, 2, 2, 4, 8.28, 3.16, 0.0, 0.0, "e4m3 192x128x128 s2 2x4w"},
};
constexpr int kNumGroupCfg = sizeof(kGroupCfg) / sizeof(kGroupCfg[0]);
constexpr int kFewRows = 1, kTwoPerCu = 4;       // 16-bit: 32 x 128; 128 x 256, 32 deep
static_assert(kGroupCfg[kFewRows].BM == 32 && kGroupCfg[kFewRows].BN == 128 &&
                  kGroupCfg[kTwoPerCu].BN == 256 && kGroupCfg[kTwoPerCu].BK == 32,
              "the tiles the choice names");

#define SG_GROUPED_16(X)          \
    X(0, 32, 64, 64, 6, 1, 2)     \
    X(1, 32, 128, 64, 4, 1, 4)    \
    X(3, 128, 256, 64, 3, 2, 4)   \
    X(4, 128, 256, 32, 3, 2, 2)   \
    X(5, 256, 256, 64, 2, 4, 2)
#define SG_GROUPED_DEPTH(X)       \
    X(2, 128, 128, 64, 2, 2, 4)   \
    X(4, 128, 256, 32, 3, 2, 2)   \
    X(5, 256, 256, 64, 2, 4, 2)
#define SG_GROUPED_8(X)           \
    X(6, 32, 128, 128, 4, 1, 4)   \
    X(7, 128, 128, 128, 2, 2, 4)  \
    X(8, 192, 128, 128, 2, 2, 4)

constexpr bool group_row(int id, bool depth, int bm, int bn, int bk, int s, int wm, int wn) {
    const GroupCfg& c = kGroupCfg[id];
    return c.BM == bm && c.BN == bn && c.BK == bk && c.S == s && c.WM == wm && c.WN == wn &&
           (depth ? c.rate_d : c.rate) > 0.0;
}
#define SG_GROUP_ROW(ID, BM, BN, BK, S, WM, WN) \
    static_assert(group_row(ID, false, BM, BN, BK, S, WM, WN), "grouped row " #ID);
#define SG_GROUP_ROW_D(ID, BM, BN, BK, S, WM, WN) \
    static_assert(group_row(ID, true, BM, BN, BK, S, WM, WN), "grouped row " #ID);
SG_GROUPED_16(SG_GROUP_ROW)
SG_GROUPED_8(SG_GROUP_ROW)
SG_GROUPED_DEPTH(SG_GROUP_ROW_D)
#undef SG_GROUP_ROW
#undef SG_GROUP_ROW_D

}  // namespace sg

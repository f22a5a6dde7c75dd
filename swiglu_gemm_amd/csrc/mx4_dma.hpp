// mx4_dma.hpp -- the 4-bit product on a direct-to-LDS ring of K tiles, as gemm16_dma.hpp
// runs the 16-bit one.  A K tile is 128 bytes of every row (256 elements, 8 blocks) and the
// matching tiles of scales; codes are moved as the 16-bit kernels move 64-deep tiles, the
// scales of 32 rows as one 256-byte line.
//
// MFMA step s of a tile takes blocks s (lanes 0..31) and 4 + s (lanes 32..63), so that the
// four scales a lane needs in a tile are the bytes of one dword of the tile of scales, step s
// selecting byte s.  One ds_read_b32 a fragment and K tile then feeds the scales of four
// MFMAs.
//
// A row may end inside a K tile: the ring loads the row's last chunk again for the chunks
// past its end, and the tile is finished apart from the loop with those chunks of A as zero
// codes and both scales 1, so neither stray codes nor padding of the scales count.
//
// Large products are bound by the matrix cores and power: 8192^3 258 us, 4.3 PFLOP/s.  A tile
// of K = 2048 is 8 K tiles, so its fill and epilogue show: 16384 rows of 32 uneven experts,
// 2048 x 2 x 1408 with SwiGLU, 81 us, 2.3 PFLOP/s.  Few rows are bound by reading the weights
// and by latency: 8 rows, 4096 x 11008 (24 MB), 8.8 us.
#pragma once

#include "gemm16_dma.hpp"
#include "grouped_dma.hpp"
#include "mx4.hpp"

namespace sg {

template <int BM, int BN, int S, int WM, int WN>
struct MxShape {
    static constexpr int BK = 64;                        // 16-bit units of a row in a K tile
    static constexpr int KS = 4;                         // MFMA steps of a K tile
    static constexpr int NW = WM * WN, NT = 64 * NW;
    static constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 32, FN = TN / 32;
    using TA = DmaTile<true, BM, BK, 2>;
    using TB = DmaTile<true, BN, BK, 2>;
    static constexpr int NG = (BM + BN) / 32;            // 32-row groups of scales
    static constexpr int NIS = (NG + NW - 1) / NW;       // their loads per wave
    static constexpr int SCALES = TA::BYTES + TB::BYTES; // offset of the scales in a stage
    static constexpr int STAGE = SCALES + NG * kMxTileBytes;
    static constexpr int LDS = S * STAGE;
    static_assert(LDS <= 160 * 1024, "LDS budget");
    static constexpr int NL = TA::BLOCKS / NW + TB::BLOCKS / NW + NIS;
    static_assert((S - 2) * NL < 64, "vmcnt range");
    using Acc = f32x16[FN][FM];
};

// The lane's codes of MFMA step s: block 4*(lane/32) + s of row rbase + lane%32.
template <int R>
__device__ __forceinline__ u32x4 mx_frag(const char* tile, int rbase, int s, int lane) {
    using T = DmaTile<true, R, 64, 2>;
    const int row = rbase + (lane & 31), chunk = 4 * (lane >> 5) + s;
    return *reinterpret_cast<const u32x4*>(tile + row * T::ROW_BYTES + ((chunk ^ T::swz(row)) << 4));
}

template <int SEL>
__device__ __forceinline__ f32x16 mx_mfma(const u32x4& b, uint32_t sb, const u32x4& a, uint32_t sa,
                                          const f32x16& c) {
    const i32x8 vb = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
    const i32x8 va = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
    // format 4 = e2m1 for both; byte SEL of each scale register
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(vb, va, c, 4, 4, SEL, (int)sb, SEL,
                                                           (int)sa);
}

template <int BM, int BN, int S, int WM, int WN>
__device__ __forceinline__ void mx_mainloop(const MxParams& x, const GroupItem& it,
                                            const Gemm16Params& p, char* smem, int m0, int n0,
                                            typename MxShape<BM, BN, S, WM, WN>::Acc& acc,
                                            int wave, int lane) {
    using D = MxShape<BM, BN, S, WM, WN>;
    constexpr int FM = D::FM, FN = D::FN, KS = D::KS, NW = D::NW, NL = D::NL;
    const int wm = wave % WM, wn = wave / WM;
    const int nkt = p.K / 8, nbt = p.K - nkt * 8;        // whole K tiles; blocks behind them
    const int nt = nkt + (nbt > 0 ? 1 : 0);

    DmaStream<true, BM, D::BK, 2, NW> da;
    DmaStream<true, BN, D::BK, 2, NW> db;
    da.init(p.A, p.lda / 2, m0, p.M, 0, wave, lane);
    db.init(p.B, p.ldb / 2, n0, p.N, 0, wave, lane);
    // scales: the lane's dword of each of the wave's groups, from a base of the tile's own
    const int64_t row_of_tiles = (int64_t)x.tiles_k * kMxTileBytes;
    const int ra0 = it.row0 + m0;
    const char* sa0 = reinterpret_cast<const char*>(x.As) + (ra0 >> 5) * row_of_tiles;
    const char* sb0 = reinterpret_cast<const char*>(x.Bs) + it.e * x.sBs + (n0 >> 5) * row_of_tiles;
    uint32_t soff[D::NIS];
    bool s_of_b[D::NIS];
#pragma unroll
    for (int i = 0; i < D::NIS; ++i) {
        const int g = min(wave + i * NW, D::NG - 1);
        s_of_b[i] = g >= BM / 32;
        const int r = s_of_b[i]
                          ? min(n0 + (g - BM / 32) * 32 + (lane & 31), p.N - 1) - (n0 & ~31)
                          : it.row0 + min(m0 + g * 32 + (lane & 31), p.M - 1) - (ra0 & ~31);
        soff[i] = (uint32_t)((r >> 5) * row_of_tiles + (lane >> 5) * 128 + (r & 31) * 4);
    }
    auto issue = [&](int t) __attribute__((always_inline)) {
        char* st = smem + (t % S) * D::STAGE;
        if (t < nkt) {
            da.issue(st, t, wave);
            db.issue(st + D::TA::BYTES, t, wave);
        } else {
            // the row ends in this tile: the last chunk again past the end
            auto ends = [&](auto s, const void* base, int64_t ld, int r0, int rows)
                __attribute__((always_inline)) {
                using T = typename decltype(s)::T;
                s.base = reinterpret_cast<const char*>(base) + (int64_t)r0 * ld;
                s.step = D::BK * 2;
#pragma unroll
                for (int i = 0; i < decltype(s)::NI; ++i) {
                    const int chunk = (wave + i * NW) * 64 + lane;
                    const int row = chunk / T::SLOTS, c = (chunk % T::SLOTS) ^ T::swz(row);
                    s.off[i] = (uint32_t)((min(r0 + row, rows - 1) - r0) * ld + min(c, nbt - 1) * 16);
                }
                return s;
            };
            ends(da, p.A, p.lda, m0, p.M).issue(st, t, wave);
            ends(db, p.B, p.ldb, n0, p.N).issue(st + D::TA::BYTES, t, wave);
        }
#pragma unroll
        for (int i = 0; i < D::NIS; ++i) {
            const int g = min(wave + i * NW, D::NG - 1);
            const char* src = (s_of_b[i] ? sb0 : sa0) + (int64_t)t * kMxTileBytes;
            const uint32_t lds = (uint32_t)(uintptr_t)(
                (__attribute__((address_space(3))) char*)(st + D::SCALES + g * kMxTileBytes));
            asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2"
                         :: "s"(lds), "v"(soff[i]), "s"(src) : "memory", "m0");
        }
    };

    u32x4 fa[2][FM], fb[2][FN];
    uint32_t sa[FM], sb[FN], na[FM], nb[FN];
    auto read_all = [&](const char* st, int s, u32x4 (&af)[FM], u32x4 (&bf)[FN])
        __attribute__((always_inline)) {
#pragma unroll
        for (int tm = 0; tm < FM; ++tm) af[tm] = mx_frag<BM>(st, wm * D::TM + tm * 32, s, lane);
#pragma unroll
        for (int tn = 0; tn < FN; ++tn)
            bf[tn] = mx_frag<BN>(st + D::TA::BYTES, wn * D::TN + tn * 32, s, lane);
    };
    auto read_scales = [&](const char* st, uint32_t (&a)[FM], uint32_t (&b)[FN])
        __attribute__((always_inline)) {
        const char* sc = st + D::SCALES + lane * 4;
#pragma unroll
        for (int tm = 0; tm < FM; ++tm)
            a[tm] = *reinterpret_cast<const uint32_t*>(sc + (wm * FM + tm) * kMxTileBytes);
#pragma unroll
        for (int tn = 0; tn < FN; ++tn)
            b[tn] =
                *reinterpret_cast<const uint32_t*>(sc + (BM / 32 + wn * FN + tn) * kMxTileBytes);
    };
    auto mfma_all = [&](auto step, const u32x4 (&af)[FM], const u32x4 (&bf)[FN])
        __attribute__((always_inline)) {
        constexpr int s = decltype(step)::value;
#pragma unroll
        for (int tn = 0; tn < FN; ++tn)
#pragma unroll
            for (int tm = 0; tm < FM; ++tm)
                acc[tn][tm] = mx_mfma<s>(bf[tn], sb[tn], af[tm], sa[tm], acc[tn][tm]);
    };

    if (nt == 0) return;
#pragma unroll
    for (int i = 0; i < S - 1; ++i)
        if (i < nt) issue(i);
    if (nt >= S - 1) wait_vmcnt<(S - 2) * NL>();
    else wait_vmcnt<0>();
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    read_scales(smem, sa, sb);
    read_all(smem, 0, fa[0], fb[0]);
    for (int t = 0; t < nkt; ++t) {
        const char* cur = smem + (t % S) * D::STAGE;
        const char* nxt = smem + ((t + 1) % S) * D::STAGE;
        const bool ahead = t + S - 1 < nt;
        if (ahead) issue(t + S - 1);
        static_for<0, KS - 1>([&](auto step) __attribute__((always_inline)) {
            constexpr int s = decltype(step)::value;
            read_all(cur, s + 1, fa[(s + 1) & 1], fb[(s + 1) & 1]);
            mfma_all(step, fa[s & 1], fb[s & 1]);
            sched_interleave<FM * FN, FM + FN, 0, 0>();
            __builtin_amdgcn_sched_barrier(0);
        });
        if (ahead) wait_vmcnt<(S - 2) * NL>();
        else wait_vmcnt<0>();
        stage_barrier();
        // the next tile's scales and first codes under this tile's last MFMAs (after the
        // last tile: a stale stage, unused)
        read_scales(nxt, na, nb);
        read_all(nxt, 0, fa[0], fb[0]);
        mfma_all(std::integral_constant<int, KS - 1>{}, fa[(KS - 1) & 1], fb[(KS - 1) & 1]);
        sched_interleave<FM * FN, 2 * (FM + FN), 0, 0>();
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int tm = 0; tm < FM; ++tm) sa[tm] = na[tm];
#pragma unroll
        for (int tn = 0; tn < FN; ++tn) sb[tn] = nb[tn];
    }
    if (nbt > 0) {
        const char* st = smem + (nkt % S) * D::STAGE;
        // the lane's blocks 4h .. 4h+3: scales past the row's end become 1, codes 0
        const int n = min(max(nbt - 4 * (lane >> 5), 0), 4);
        const uint32_t keep = n == 4 ? 0xffffffffu : (1u << (8 * n)) - 1u;
#pragma unroll
        for (int tm = 0; tm < FM; ++tm) sa[tm] = (sa[tm] & keep) | (0x7f7f7f7fu & ~keep);
#pragma unroll
        for (int tn = 0; tn < FN; ++tn) sb[tn] = (sb[tn] & keep) | (0x7f7f7f7fu & ~keep);
        static_for<0, KS>([&](auto step) __attribute__((always_inline)) {
            constexpr int s = decltype(step)::value;
            if (s >= nbt) return;                        // neither half has this block
            read_all(st, s, fa[0], fb[0]);
#pragma unroll
            for (int tm = 0; tm < FM; ++tm)
#pragma unroll
                for (int d = 0; d < 4; ++d) fa[0][tm][d] = s < n ? fa[0][tm][d] : 0u;
            mfma_all(step, fa[0], fb[0]);
        });
    }
}

template <int DT_OUT, int EPI, int BM, int BN, int S, int WM, int WN>
__device__ __forceinline__ void mx_tile(const MxParams& x, const GroupItem& it,
                                        const Gemm16Params& p, char* smem, int wave, int lane) {
    using D = MxShape<BM, BN, S, WM, WN>;
    const int m0 = it.m0, n0 = it.tn * BN;
    typename D::Acc acc;
#pragma unroll
    for (int i = 0; i < D::FN; ++i)
#pragma unroll
        for (int j = 0; j < D::FM; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
    mx_mainloop<BM, BN, S, WM, WN>(x, it, p, smem, m0, n0, acc, wave, lane);

    constexpr int FM = D::FM, FN = D::FN, NT = D::NT, LDS = D::LDS;
    const int wm = wave % WM, wn = wave / WM;
    if constexpr (EPI == EPI_SWIGLU) {
        static_assert(BM * (BN + 8) <= LDS, "staged SwiGLU tile fits the LDS ring");
        epilogue_swiglu_lds<DT_OUT, FM, FN, BM, BN, NT, false, false>(p, acc, smem, m0, n0,
                                                                      wm * D::TM, wn * D::TN, lane);
    } else if constexpr (EPI == EPI_GEMM_F32) {
        epilogue_f32_rows_lds<FM, FN, BM, BN, WN, NT, LDS>(p, acc, smem, m0, n0, wm * D::TM, wn,
                                                           lane);
    } else {
        if ((reinterpret_cast<uintptr_t>(p.C) & 15) == 0 && (p.ldc & 7) == 0)
            epilogue_gemm_rows_beta_lds<DT_OUT, FM, FN, BM, BN, WN, NT, LDS>(
                p, acc, smem, m0, n0, wm * D::TM, wn, lane);
        else
            epilogue16<DT_OUT, EPI_GEMM, FM, FN>(p, acc, m0, n0, BM, BN, m0 + wm * D::TM,
                                                 n0 + wn * D::TN, lane);
    }
}

// The last rows of a run go on half of the tile's height where that holds them, as in
// grouped_dma_kernel.
template <int DT_OUT, int EPI, int BM, int BN, int S, int WM, int WN>
__global__ void __launch_bounds__(64 * WM * WN, group_occ(MxShape<BM, BN, S, WM, WN>::LDS))
    mx_dma_kernel(const MxParams x) {
    using D = MxShape<BM, BN, S, WM, WN>;
    constexpr bool HALF = BM >= 128;
    constexpr int S2 = BM == 256 ? 3 : S;
    constexpr int LDS_HALF = HALF ? MxShape<(HALF ? BM / 2 : 64), BN, S2, 2, 4>::LDS : 0;
    __shared__ __attribute__((aligned(1024))) char smem[LDS_HALF > D::LDS ? LDS_HALF : D::LDS];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    GroupItem it;
    if (!find_rows<BM, HALF ? group_occ(D::LDS) : 0>(x.q, blockIdx.x, lane, it)) return;
    const Gemm16Params p = group_problem<false, 1, EPI == EPI_GEMM_F32 ? 4 : 2>(x.q, it);
    if constexpr (HALF) {
        static_assert(WM * WN == 8, "the half tile's waves");
        if (it.half || it.rows - it.m0 <= BM / 2) {
            mx_tile<DT_OUT, EPI, BM / 2, BN, S2, 2, 4>(x, it, p, smem, wave, lane);
            return;
        }
    }
    mx_tile<DT_OUT, EPI, BM, BN, S, WM, WN>(x, it, p, smem, wave, lane);
}

// Tiles of the 4-bit product; SG_FORCE_MX4=<id> overrides the choice.
struct MxCfg {
    int BM, BN, S, WM, WN;
    const char* name;
};
constexpr MxCfg kMxCfg[] = {
    {32, 64, 6, 1, 2, "32x64 s6 1x2w"},
    {32, 128, 3, 1, 4, "32x128 s3 1x4w"},
    {128, 128, 2, 2, 4, "128x128 s2 2x4w"},
    {256, 256, 2, 4, 2, "256x256 s2 4x2w"},
};
constexpr int kNumMxCfg = sizeof(kMxCfg) / sizeof(kMxCfg[0]);
#define SG_MX_CONFIGS(X)     \
    X(0, 32, 64, 6, 1, 2)    \
    X(1, 32, 128, 3, 1, 4)   \
    X(2, 128, 128, 2, 2, 4)  \
    X(3, 256, 256, 2, 4, 2)
#define SG_MX_ROW(ID, BM_, BN_, S_, WM_, WN_)                                             \
    static_assert(kMxCfg[ID].BM == BM_ && kMxCfg[ID].BN == BN_ && kMxCfg[ID].S == S_ &&   \
                      kMxCfg[ID].WM == WM_ && kMxCfg[ID].WN == WN_,                       \
                  "4-bit row " #ID);
SG_MX_CONFIGS(SG_MX_ROW)
#undef SG_MX_ROW

}  // namespace sg

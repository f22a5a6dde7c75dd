// int4.hpp -- products with weights of 4-bit integers that share a scale (and a zero point) in
// groups of 32, 64 or 128 along K:  W[n, k] = scale[n, g] * (code[n, k] - zero[n, g]).
//
// Codes lie in tiles of 16 rows x 128 columns (1024 bytes) in the order in which a wave's lanes
// feed them to the 16 x 16 x 32 matrix instruction: lane 16 q + r loads 16 bytes, and dword s of
// them holds W[r, 32 s + 8 q .. + 7], element i in nibble i/2 + 4 (i % 2), so that masking out
// one nibble of each half gives two neighbours of k.  A tile is one 1024-byte load of a wave.
//
// The codes meet the activations unscaled: a group's sum over k of a * (code - zero) is taken in
// fp32 accumulators, then multiplied by the group's scale and added to the running sum, so
// neither the weights nor the groups' sums are rounded to 16 bits.
//   fp16: 0x6400 | code is 1024 + code; adding -(1024 + zero) leaves code - zero exactly.
//   bf16: there is no packed bf16 subtraction, so 0x4180 | code << 3, which is 16 + code, goes
//         into the product as it is, and (16 + zero) * sum of a is taken out afterwards, the sum
//         of a from a product with ones (it stands in the same registers as the group's sums).
//         The fp32 sums then hold numbers up to 31 / |code - zero| times larger: still 2^-24 of
//         them, far below the 2^-9 of a bf16 output.
#pragma once

#include <type_traits>

#include "grouped.hpp"
#include "sg_device.hpp"

namespace sg {

struct Int4Params {
    GroupedParams q;          // g.A, g.lda: activations; g.C, g.ldc; g.N: rows of the weight
    const int32_t* order;     // nullptr: row r of C is row r of A
    int top_k, T;             // row of A: order[r] / top_k, of T
    const uint8_t* codes;
    const uint16_t* scales;
    const uint8_t* zeros;     // nullptr: 8
    int64_t s_codes, s_scales;   // codes' bytes and scales' elements of one expert
    int tiles_k, tiles_g;     // tiles along K of codes (128) and of scales (4 groups)
    int swiglu, c_f32;
};

inline int64_t int4_tiles_k(int64_t K) { return (K + 127) / 128; }
inline int64_t int4_tiles_g(int64_t K, int64_t group) {
    return ((K + group - 1) / group + 3) / 4;
}

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));

template <int DT>
__device__ __forceinline__ f32x4 mfma_16x16x32(const u32x4& a, const u32x4& b, const f32x4& c) {
    if constexpr (DT == DT_F16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                      __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                       __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// x & mask | magic in one instruction: kept in registers, the two constants leave it the one form
// that takes both.  fp16 has a second mask, for the codes in the upper halves of bytes: 0x6400 |
// code << 4 is 1024 + 16 code, of which one multiply-add makes code - zero, without a shift.
struct Int4Magic {
    uint32_t mask, high, magic;
};
template <int DT>
__device__ __forceinline__ Int4Magic int4_magic() {
    Int4Magic m = {DT == DT_F16 ? 0x000F000Fu : 0x00780078u, 0x00F000F0u,
                   DT == DT_F16 ? 0x64006400u : 0x41804180u};
    asm("" : "+v"(m.mask));
    if constexpr (DT == DT_F16) asm("" : "+v"(m.high));
    asm("" : "+s"(m.magic));
    return m;
}

// The zero point as int4_operand takes it: fp16: -(1024 + zero) and -(64 + zero), both twice, and
// 2^-4 twice.  All three are exact, and so is code - zero.
struct Int4Zero {
    f16x2 low, high, scale;
};
__device__ __forceinline__ Int4Zero int4_zero(float z) {
    const _Float16 l = (_Float16)(-1024.0f - z), h = (_Float16)(-64.0f - z), f = (_Float16)0.0625f;
    return Int4Zero{{l, l}, {h, h}, {f, f}};
}

// Eight codes as an operand: fp16: code - zero; bf16: 16 + code.
template <int DT>
__device__ __forceinline__ u32x4 int4_operand(uint32_t w, const Int4Zero& z, const Int4Magic& m) {
    u32x4 o;
    if constexpr (DT == DT_F16) {
#pragma unroll
        for (int p = 0; p < 4; p += 2) {
            const uint32_t v = w >> (4 * p);
            const uint32_t a = (v & m.mask) | m.magic, b = (v & m.high) | m.magic;
            o[p] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, a) + z.low);
            o[p + 1] = __builtin_bit_cast(
                uint32_t, __builtin_elementwise_fma(__builtin_bit_cast(f16x2, b), z.scale, z.high));
        }
    } else {
        o[0] = (w << 3 & m.mask) | m.magic;
#pragma unroll
        for (int p = 1; p < 4; ++p) o[p] = (w >> (4 * p - 3) & m.mask) | m.magic;
    }
    return o;
}

// Eight activations from column k on of a row of K; zeros behind it, nothing read there.
__device__ __forceinline__ u32x4 int4_act(const uint16_t* row, int k, int K) {
    if (k + 8 <= K) return *reinterpret_cast<const u32x4_a2*>(row + k);
    u32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (k + i < K) v[i / 2] |= (uint32_t)row[k + i] << (16 * (i % 2));
    return v;
}

// One tile of 16 x 128 codes with its scales and zeros (PER groups of a row side by side), as
// loaded.
template <int GROUP, bool ZEROS>
struct Int4Tile {
    static constexpr int PER = 128 / GROUP;
    u32x4 w;
    uint32_t f[PER == 4 ? 2 : 1], z;

    template <int DT>
    __device__ __forceinline__ float scale(int p) const {
        return to_f32<DT>((uint16_t)(f[p / 2] >> (16 * (p % 2))));
    }
    __device__ __forceinline__ float zero(int p) const {
        return ZEROS ? (float)(z >> (8 * p) & 0xFFu) : 8.0f;
    }
    // the tile that holds column K of a row: groups wholly behind it have no scale
    __device__ __forceinline__ void cut(int columns) {
#pragma unroll
        for (int p = 1; p < PER; ++p)
            if (p * GROUP >= columns) f[p / 2] &= p % 2 ? 0x0000FFFFu : 0u;
    }
};
// A strip of 16 columns.  For few rows: the same addresses in every lane, so that a load takes its
// base from scalar registers and only the lane's offset from a vector one.
struct Int4Strip {
    const uint8_t *codes, *zeros;
    const uint16_t* scales;
};
template <int GROUP, bool ZEROS>
__device__ __forceinline__ void int4_load(Int4Tile<GROUP, ZEROS>& t, const Int4Strip& s,
                                          uint32_t lane, int kt) {
    constexpr int PER = 128 / GROUP;
    const int g = kt * PER, at = g / 4 * 64 + g % 4;
    const uint32_t l = 4 * (lane & 15);
    t.w = *reinterpret_cast<const u32x4*>(s.codes + (int64_t)kt * 1024 + 16 * lane);
    const uint16_t* f = s.scales + at + l;
    if constexpr (PER == 4) {
        const u32x2 v = *reinterpret_cast<const u32x2*>(f);
        t.f[0] = v.x;
        t.f[1] = v.y;
    } else if constexpr (PER == 2) {
        t.f[0] = *reinterpret_cast<const uint32_t*>(f);
    } else {
        t.f[0] = *f;
    }
    if constexpr (ZEROS) {
        const uint8_t* z = s.zeros + at + l;
        t.z = PER == 4   ? *reinterpret_cast<const uint32_t*>(z)
              : PER == 2 ? *reinterpret_cast<const uint16_t*>(z)
                         : *z;
    }
}

// The activations of 16 MT rows and 128 columns from tile kt on.
template <int MT, bool TAIL>
__device__ __forceinline__ void int4_rows(u32x4 (&a)[MT][4], const uint16_t* const (&row)[MT],
                                          int lane, int kt, int K) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int k = kt * 128 + 32 * s + 8 * (lane >> 4);
            a[i][s] = TAIL ? int4_act(row[i], k, K)
                           : *reinterpret_cast<const u32x4_a2*>(row[i] + k);
        }
}

// bf16: the sums of the activations over each group, in every column of a 16 x 16 tile.
template <int DT, int GROUP, int MT>
__device__ __forceinline__ void int4_row_sums(f32x4 (&asum)[MT][128 / GROUP],
                                              const u32x4 (&a)[MT][4]) {
    if constexpr (DT == DT_BF16) {
        constexpr int STEPS = GROUP / 32;
        const uint32_t one = 0x3F803F80u;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int p = 0; p < 128 / GROUP; ++p) {
                asum[i][p] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int s = 0; s < STEPS; ++s)
                    asum[i][p] = mfma_16x16x32<DT>(a[i][p * STEPS + s], u32x4{one, one, one, one},
                                                   asum[i][p]);
            }
    }
}

// Adds the products of the activations with one tile of codes.
template <int DT, int GROUP, bool ZEROS, int MT>
__device__ __forceinline__ void int4_add(f32x4 (&sum)[MT], const u32x4 (&a)[MT][4],
                                         const f32x4 (&asum)[MT][128 / GROUP],
                                         const Int4Tile<GROUP, ZEROS>& t,
                                         const Int4Magic& magic) {
    constexpr int STEPS = GROUP / 32;
#pragma unroll
    for (int p = 0; p < 128 / GROUP; ++p) {
        const float f = t.template scale<DT>(p), z = t.zero(p);
        Int4Zero zero{};
        if constexpr (DT == DT_F16) zero = int4_zero(z);
        f32x4 acc[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[i] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const u32x4 b = int4_operand<DT>(t.w[p * STEPS + s], zero, magic);
#pragma unroll
            for (int i = 0; i < MT; ++i)
                acc[i] = mfma_16x16x32<DT>(a[i][p * STEPS + s], b, acc[i]);
        }
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                float v = acc[i][r];
                if constexpr (DT == DT_BF16) v = __builtin_fmaf(-16.0f - z, asum[i][p][r], v);
                sum[i][r] = __builtin_fmaf(f, v, sum[i][r]);
            }
    }
}

// Stores columns n (even) and n + 1 of the row that starts `row` elements into C.
template <int DT>
__device__ __forceinline__ void int4_put(const Int4Params& x, int64_t row, int n, float u, float v) {
    const Gemm16Params& g = x.q.g;
    if (x.swiglu) {
        reinterpret_cast<uint16_t*>(g.C)[row + n / 2] = from_f32<DT>(silu(u) * v);
    } else if (x.c_f32) {
        float* c = reinterpret_cast<float*>(g.C) + row + n;
        c[0] = g.alpha * u;
        if (n + 1 < g.N) c[1] = g.alpha * v;
    } else {
        uint16_t* c = reinterpret_cast<uint16_t*>(g.C) + row + n;
        c[0] = from_f32<DT>(g.alpha * u);
        if (n + 1 < g.N) c[1] = from_f32<DT>(g.alpha * v);
    }
}

// One work-group: 16 MT rows x 16 NT columns of the product; its waves take every NW-th tile of
// 128 along K and their sums meet in LDS, in the order of the waves.  A wave keeps a tile of codes
// of each of its NT strips, and the activations of a tile, under way while it works on the one
// before.  For few rows: what bounds it is the codes from memory.  Measured (MI355X, kernel alone,
// weights cold): bf16, 1 x 4096 by 4096 5.0 us, most of it launch and one trip to memory; fp16, 16 x
// 4096 by 22016 (SwiGLU, groups of 128 with zero points) 14.2 us, 48 MB, 3.4 TB/s; bf16, 256 rows of
// 64 experts, 2048 by 2816 with zero points in groups of 64, 200 MB, 47.5 us in the mean, 44.6 at best,
// 4.2 to 4.5 TB/s (a plain read: 5.66 TB/s).
template <int DT, int GROUP, bool ZEROS, int MT, int NT, int NW>
__global__ void __launch_bounds__(64 * NW) int4_kernel(const Int4Params x) {
    constexpr int BM = 16 * MT, BN = 16 * NT, PER = 128 / GROUP;
    __shared__ float part[NW][BM * BN];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const GroupedParams& q = x.q;
    GroupItem it;
    if (!find_rows<BM>(q, blockIdx.x, lane, it)) return;
    const int N = q.g.N, K = q.g.K, n0 = it.tn * BN, lr = lane & 15, lq = lane >> 4;
    Int4Strip strip[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int tn = __builtin_amdgcn_readfirstlane(min(it.tn * NT + j, (N + 15) / 16 - 1));
        const int64_t at = it.e * x.s_scales + (int64_t)tn * x.tiles_g * 64;
        strip[j].codes = x.codes + it.e * x.s_codes + (int64_t)tn * x.tiles_k * 1024;
        strip[j].scales = x.scales + at;
        strip[j].zeros = x.zeros + at;
    }
    const Int4Magic magic = int4_magic<DT>();
    const int full = K / 128;
    int kt = wave;
    Int4Tile<GROUP, ZEROS> t[2][NT];
    if (kt < full)
#pragma unroll
        for (int j = 0; j < NT; ++j) int4_load(t[0][j], strip[j], lane, kt);
    const uint16_t* row[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        // rows past the expert's last one: that one again, their sums are not stored
        int r = it.row0 + min(it.m0 + 16 * i + lr, it.rows - 1);
        if (x.order) r = min(max(x.order[r] / x.top_k, 0), x.T - 1);
        row[i] = q.g.A + (int64_t)r * q.g.lda;
    }
    f32x4 sum[NT][MT];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < MT; ++i) sum[j][i] = f32x4{0, 0, 0, 0};
    u32x4 a[2][MT][4];
    f32x4 asum[MT][PER];
    // One tile of 128 along K: everything of the next one is loaded first, into registers of its
    // own.  The barrier keeps the loads there; the compiler would gather them at the end, with
    // nothing left to cover them.
    auto step = [&](auto from, auto more) {
        if constexpr (more) {
            int4_rows<MT, false>(a[1 - from], row, lane, kt + NW, K);
#pragma unroll
            for (int j = 0; j < NT; ++j) int4_load(t[1 - from][j], strip[j], lane, kt + NW);
            __builtin_amdgcn_sched_barrier(0);
        }
        int4_row_sums<DT, GROUP, MT>(asum, a[from]);
#pragma unroll
        for (int j = 0; j < NT; ++j)
            int4_add<DT, GROUP, ZEROS, MT>(sum[j], a[from], asum, t[from][j], magic);
        kt += NW;
    };
    constexpr std::integral_constant<int, 0> even{};
    constexpr std::integral_constant<int, 1> odd{};
    constexpr std::true_type more{};
    constexpr std::false_type last{};
    if (kt < full) {
        int4_rows<MT, false>(a[0], row, lane, kt, K);
        while (kt + 2 * NW < full) {
            step(even, more);
            step(odd, more);
        }
        if (kt + NW < full) {
            step(even, more);
            step(odd, last);
        } else {
            step(even, last);
        }
    }
    if (K % 128 != 0 && wave == full % NW) {
        int4_rows<MT, true>(a[0], row, lane, full, K);
        int4_row_sums<DT, GROUP, MT>(asum, a[0]);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            int4_load(t[0][j], strip[j], lane, full);
            t[0][j].cut(K - full * 128);
            int4_add<DT, GROUP, ZEROS, MT>(sum[j], a[0], asum, t[0][j], magic);
        }
    }
    // D[m][n]: lane 16 q + r holds rows 4 q .. 4 q + 3 of column r
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                part[wave][(16 * i + 4 * lq + r) * BN + 16 * j + lr] = sum[j][i][r];
    __syncthreads();
    for (int o = 2 * threadIdx.x; o < BM * BN; o += 128 * NW) {
        float u = 0.0f, v = 0.0f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            u += part[w][o];
            v += part[w][o + 1];
        }
        const int m = it.m0 + o / BN, n = n0 + o % BN;
        if (m >= it.rows || n >= N) continue;
        const int64_t r = (int64_t)(it.row0 + m) * q.g.ldc;
        int4_put<DT>(x, r, n, u, v);
    }
}

// ---------------------------------------------------------------------------
// Many rows: 32 MT rows x 128 columns a work-group, the columns divided over its four waves, so that
// each code is loaded and widened once and meets all rows, on 32 x 32 x 16 products: their operands
// keep the vector unit, which widens the codes, from issuing for less time than those of four times
// as many 16 x 16 x 32 ones.  A wave takes two strips of 16 columns together: lane 32 h + n loads
// the pieces q = h and q = 2 + h of row n of the two.  The activations pass through LDS, three tiles
// of 128 along K with one barrier a tile, their 16-byte pieces XOR-swizzled by row.  bf16: minus the
// sums of the activations over each group are taken one tile ahead, 16 rows by each wave; times
// scale * (16 + zero) they are a product along the groups, two at a time on the fp32 32 x 32 x 2
// matrix instruction.  (As the initial accumulators of each group's products they cost a read of LDS
// by every lane and, with zero points, a multiplication for each value: 256 x 4096 by 11008, groups
// of 64 with zero points, 57.6 us so and 52.3 us this way; 128 x 4096 by 11008, groups of 128, 33.2
// and 32.2; 512 rows of the latter and groups of 32 the same both ways.)
// KS = 2: eight waves, four for each half of K, joined through LDS, for grids that leave a CU one
// work-group, whose waves would wait for their own operands.
// Measured (MI355X, bf16, groups of 128): 512 x 4096 by 11008 62 us, 745 TFLOP/s (MT = 2; 103 us with
// 16-row strips); 256 x 4096 by 4096 19.1 us (MT = 1, KS = 2; 25.7 us with 16-row strips, 31.7 us with
// MT = 2, KS = 1).  What bounds it is issue, not memory or the matrix unit: with MT = 2 a wave's step is
// 18 products of 16 ns, 140 vector instructions and 20 KB read from LDS, none of which is hidden whole.
// Longer look-ahead on the codes and activations (2 tiles more: 5% faster alone on a CU, 8% slower
// shared), on LDS (3 products: slower) and 256 columns (spills) did not pay.
// ---------------------------------------------------------------------------
template <int DT, int GROUP, bool ZEROS, int MT, int KS>
__global__ void __launch_bounds__(256 * KS, 2) int4_tile_kernel(const Int4Params x) {
    constexpr int BM = 32 * MT, BN = 128, PIECES = BM / 16, PER = 128 / GROUP, STEPS = 2 * GROUP / 32;
    constexpr bool SUMS = DT == DT_BF16;
    typedef Int4Tile<GROUP, ZEROS> Tile;
    __shared__ u32x4 all_lds[KS][3][BM * 16];
    __shared__ f32x4 all_sums[KS][SUMS ? 4 : 1][SUMS ? PER * BM / 4 : 1];     // of tile kt at kt % 4
    const int lane = threadIdx.x & 63, tid = threadIdx.x & 255;
    const int part = __builtin_amdgcn_readfirstlane(threadIdx.x >> 8);
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    auto& lds = all_lds[part];
    auto& sums = all_sums[part];
    const GroupedParams& q = x.q;
    GroupItem it;
    if (!find_rows<BM>(q, blockIdx.x, lane, it)) return;
    const int N = q.g.N, K = q.g.K, lr = lane & 15, ln = lane & 31, lh = lane >> 5;
    const int n0 = it.tn * BN + wave * 32;
    const int tn = min(n0 / 16 + (ln >> 4), (N + 15) / 16 - 1);
    const int64_t at = it.e * x.s_scales + (int64_t)tn * x.tiles_g * 64 + 4 * lr;
    const Int4Strip strip = {
        x.codes + it.e * x.s_codes + (int64_t)tn * x.tiles_k * 1024 + 16 * (16 * lh + lr),
        x.zeros + at, x.scales + at};
    // this thread's piece of 8 columns in rows srow, srow + 16, ...
    const int srow = tid >> 4, spiece = tid & 15;
    const uint16_t* row[PIECES];
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
        int r = it.row0 + min(it.m0 + 16 * i + srow, it.rows - 1);
        if (x.order) r = min(max(x.order[r] / x.top_k, 0), x.T - 1);
        row[i] = q.g.A + (int64_t)r * q.g.lda + 8 * spiece;
    }
    const int spot = srow * 16 + (spiece ^ srow);
    const Int4Magic magic = int4_magic<DT>();
    f32x16 sum[MT] = {};
    u32x4 stage[PIECES];
    auto load_stage = [&](int kt) {
#pragma unroll
        for (int i = 0; i < PIECES; ++i)
            stage[i] = *reinterpret_cast<const u32x4_a2*>(row[i] + (int64_t)kt * 128);
    };
    auto store_stage = [&](u32x4* buf) {
#pragma unroll
        for (int i = 0; i < PIECES; ++i) buf[spot + 256 * i] = stage[i];
    };
    // t: pieces q = h; more: pieces q = 2 + h
    Tile t[2];
    u32x4 more[2];
    auto load_codes = [&](auto to, int kt) {
        int4_load(t[to], strip, 0, kt);
        more[to] = *reinterpret_cast<const u32x4*>(strip.codes + (int64_t)kt * 1024 + 512);
    };
    // Minus the group sums of this wave's 16 rows (32 rows: the first two waves').
    auto add_up = [&](f32x4* to, const u32x4* buf) {
        if (PIECES < 4 && wave >= PIECES) return;
        const uint32_t c = 0xBF80BF80u;                          // -1, twice
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            f32x4 d = {0, 0, 0, 0};
#pragma unroll
            for (int s = p * GROUP / 32; s < (p + 1) * GROUP / 32; ++s)
                d = mfma_16x16x32<DT>(buf[(16 * wave + lr) * 16 + ((4 * s + (lane >> 4)) ^ lr)],
                                      u32x4{c, c, c, c}, d);
            if (lr == 0) to[p * (BM / 4) + 4 * wave + (lane >> 4)] = d;
        }
    };
    // Eight steps of 16 along K.  While a step's products run, the next one's activations are read
    // and its codes widened; the barriers between steps keep the compiler from reading all of them
    // at once, which spills.
    auto compute = [&](const u32x4* buf, auto from) {
        const Tile& tile = t[from];
        f32x16 acc[MT];
        u32x4 a[2][MT], b[2];
        auto ready = [&](auto uc) {
            constexpr int u = uc, s = u / 2, p = u / STEPS;
            const int piece = (4 * s + 2 * (u % 2) + lh) ^ lr;
#pragma unroll
            for (int i = 0; i < MT; ++i) a[u % 2][i] = buf[(32 * i + ln) * 16 + piece];
            Int4Zero zero{};
            if constexpr (DT == DT_F16) zero = int4_zero(tile.zero(p));
            b[u % 2] = int4_operand<DT>(u % 2 ? more[from][s] : tile.w[s], zero, magic);
        };
        auto eighth = [&](auto uc) {
            constexpr int u = uc, p = u / STEPS;
#pragma unroll
            for (int i = 0; i < MT; ++i)
                acc[i] = mfma16<DT>(a[u % 2][i], b[u % 2], u % STEPS == 0 ? f32x16{} : acc[i]);
            if constexpr (u < 7) ready(std::integral_constant<int, u + 1>{});
            if constexpr (u % STEPS == STEPS - 1) {
                const float f = tile.template scale<DT>(p);
#pragma unroll
                for (int i = 0; i < MT; ++i) {
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        sum[i][r] = __builtin_fmaf(f, acc[i][r], sum[i][r]);
                    // here, not a tile later with both tiles' accumulators alive
                    asm volatile("" : "+v"(sum[i]));
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        ready(std::integral_constant<int, 0>{});
        eighth(std::integral_constant<int, 0>{});
        eighth(std::integral_constant<int, 1>{});
        eighth(std::integral_constant<int, 2>{});
        eighth(std::integral_constant<int, 3>{});
        eighth(std::integral_constant<int, 4>{});
        eighth(std::integral_constant<int, 5>{});
        eighth(std::integral_constant<int, 6>{});
        eighth(std::integral_constant<int, 7>{});
    };
    // Takes scale * (16 + zero) * the sums of two groups out of the sums of the products: lanes h of
    // `offset` hold it for the group whose sums are at of[h].
    auto offset_of = [&](const Tile& tile, int p) {
        return tile.template scale<DT>(p) * (16.0f + tile.zero(p));
    };
    auto take_out = [&](float offset, const f32x4* first, const f32x4* second, bool both) {
        const float* of = reinterpret_cast<const float*>(lh ? second : first);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const float s = both || lh == 0 ? of[32 * i + ln] : 0.0f;
            sum[i] = __builtin_amdgcn_mfma_f32_32x32x2f32(s, offset, sum[i], 0, 0, 0);
        }
    };
    // ... of a tile's own groups, where it has more than one
    auto take_out_pairs = [&](const Tile& tile, const f32x4* of) {
#pragma unroll
        for (int p = 0; p + 1 < PER; p += 2) {
            const float lo = offset_of(tile, p), hi = offset_of(tile, p + 1);
            take_out(lh ? hi : lo, of + p * (BM / 4), of + (p + 1) * (BM / 4), true);
        }
    };
    // The whole tiles along K: `most` for the first part, `mine` for this one, of which `common` are
    // every part's.  Step kt computes on buffer kt % 3 while the sums of tile kt + 1, whose
    // activations are in LDS, are taken.  At its end the codes of tile kt + 2 take the registers of
    // tile kt's, tile kt + 2 of the activations goes to LDS, and its registers get tile kt + 3.
    // Tiles past the last whole one are that one again: a load behind a branch would make the
    // compiler wait for all of them.  A partial tile comes last, by itself.
    constexpr std::integral_constant<int, 0> even{};
    constexpr std::integral_constant<int, 1> odd{};
    const int full = K / 128, common = full / KS, most = (full + KS - 1) / KS, base = part * most;
    const int mine = KS == 1 || part == 0 ? most : full - most;
    auto tile_at = [&](int kt) { return min(base + kt, full - 1); };
    int cur = 0;
    float before = 0.0f;                                // the even tile's offset (one group a tile)
    auto after = [](int i) { return i == 2 ? 0 : i + 1; };
    auto step = [&](auto from, int kt, bool active) {
        const int next = after(cur), free = after(next);
        if (active) compute(lds[cur], from);
        if constexpr (SUMS) {
            add_up(sums[(kt + 1) % 4], lds[next]);
            if (active) {
                if constexpr (PER > 1) {
                    take_out_pairs(t[from], sums[kt % 4]);
                } else if constexpr (from == 0) {
                    before = offset_of(t[0], 0);
                } else {
                    const float here = offset_of(t[1], 0);
                    take_out(lh ? here : before, sums[(kt + 3) % 4], sums[kt % 4], true);
                }
            }
        }
        load_codes(from, tile_at(kt + 2));
        store_stage(lds[free]);
        load_stage(tile_at(kt + 3));
        __syncthreads();
        cur = next;
    };
    if (full > 0) {
        load_stage(tile_at(0));
        load_codes(even, tile_at(0));
        store_stage(lds[0]);
        load_stage(tile_at(1));
        load_codes(odd, tile_at(1));
        store_stage(lds[1]);
        load_stage(tile_at(2));
        __syncthreads();
        if constexpr (SUMS) {
            add_up(sums[0], lds[0]);
            __syncthreads();
        }
        int kt = 0;
        for (; kt + 1 < common; kt += 2) {
            step(even, kt, true);
            step(odd, kt + 1, true);
        }
        if (kt < most) step(even, kt, kt < mine);
        if (KS > 1 && kt + 1 < most) step(odd, kt + 1, kt + 1 < mine);
        if constexpr (SUMS && PER == 1)
            if (mine % 2)
                take_out(lh ? 0.0f : before, sums[(mine - 1) % 4], sums[(mine - 1) % 4], false);
    }
    if (K % 128 != 0) {
        load_codes(even, full);
#pragma unroll
        for (int i = 0; i < PIECES; ++i)
            stage[i] = int4_act(row[i] - 8 * spiece, full * 128 + 8 * spiece, K);
        t[0].cut(K - full * 128);
        __syncthreads();                  // the sums of the last whole tile are read
        store_stage(lds[0]);
        __syncthreads();
        if constexpr (SUMS) {
            add_up(sums[0], lds[0]);
            __syncthreads();
        }
        if (part == KS - 1) {
            if constexpr (SUMS) {
                if constexpr (PER > 1) take_out_pairs(t[0], sums[0]);
                else take_out(lh ? 0.0f : offset_of(t[0], 0), sums[0], sums[0], false);
            }
            compute(lds[0], even);
        }
    }
    if constexpr (KS > 1) {
        // the second part's sums reach the first through LDS
        f32x4* pass = reinterpret_cast<f32x4*>(all_lds) + 4 * MT * (wave * 64) + lane;
        __syncthreads();
        if (part == 1)
#pragma unroll
            for (int v = 0; v < 4 * MT; ++v)
                pass[64 * v] = f32x4{sum[v / 4][4 * (v % 4)], sum[v / 4][4 * (v % 4) + 1],
                                     sum[v / 4][4 * (v % 4) + 2], sum[v / 4][4 * (v % 4) + 3]};
        __syncthreads();
        if (part == 1) return;
#pragma unroll
        for (int v = 0; v < 4 * MT; ++v) {
            const f32x4 d = pass[64 * v];
#pragma unroll
            for (int r = 0; r < 4; ++r) sum[v / 4][4 * (v % 4) + r] += d[r];
        }
    }
    // lane 32 h + n holds rows 8 g + 4 h .. + 3 of column n of each 32 x 32 tile; even columns and
    // the ones behind them meet in the even lanes
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const float u = sum[i][r];
            const float v = __builtin_bit_cast(
                float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, u), 0xB1, 0xf, 0xf, true));
            const int m = it.m0 + 32 * i + 8 * (r / 4) + 4 * lh + r % 4;
            const int n = n0 + ln;
            if ((ln & 1) || m >= it.rows || n >= N) continue;
            int4_put<DT>(x, (int64_t)(it.row0 + m) * q.g.ldc, n, u, v);
        }
}

// ---------------------------------------------------------------------------
// Quantisation, packing and the way back: one wave a tile of 16 x 128, each lane with the 32 codes
// that it holds in the products, so that codes move 1024 bytes at a time and a row's columns 64.
// A group's extremes meet over the four lanes of a row.  Quantising computes in fp32 what decides, and
// in 64 bits where the quotient is near a tie, so that codes are the formula's.  Measured (MI355X,
// 11008 x 4096, groups of 128): quantised from bf16 39 us, 2.9 TB/s (by one thread a group, with a
// division in 64 bits for each code: 986 us), bound by the vector unit: 822 instructions a wave, 70700
// cycles of each SIMD, busy for 0.85 of the time; packed 18.6 us, 3.6 TB/s, back to bf16 21 us, 5.4 TB/s.
// ---------------------------------------------------------------------------
struct Int4PackParams {
    const void* W;              // quantise
    const uint8_t *src, *src_zeros;    // pack
    const uint16_t* src_scales;
    int64_t ldw, sW;            // elements
    int N, K, group, scale_bf16;
    uint8_t* codes;
    uint16_t* scales;
    uint8_t* zeros;
    void* out;                  // dequantise
    int64_t s_codes, s_scales;
    int tiles_k, tiles_g;
    int across;                 // tiles of a strip that the waves walk
};
typedef uint32_t u32x2_a1 __attribute__((ext_vector_type(2), aligned(1)));

// Code i stands in nibble i / 2 + 4 (i % 2) of a dword.
__device__ __forceinline__ constexpr int int4_shift(int i) { return 4 * (i / 2 + 4 * (i % 2)); }
__device__ __forceinline__ float int4_scale(const Int4PackParams& p, uint16_t bits) {
    return p.scale_bf16 ? to_f32<DT_BF16>(bits) : to_f32<DT_F16>(bits);
}
template <typename F>
__device__ __forceinline__ float int4_over_row(float x, F f) {
    x = f(x, __shfl_xor(x, 16));
    return f(x, __shfl_xor(x, 32));
}

// Rows and columns past the matrix, up to whole tiles, get zeros.
template <int DT, int GROUP, bool PACK>
__global__ void __launch_bounds__(256) int4_pack_kernel(const Int4PackParams p) {
    constexpr int PER = 128 / GROUP, STEPS = GROUP / 32;
    const int64_t b = blockIdx.z;
    const int lane = threadIdx.x & 63, lr = lane & 15, lq = lane >> 4;
    const int real = (p.K + GROUP - 1) / GROUP;
    uint8_t* codes = p.codes + b * p.s_codes;
    uint16_t* scales = p.scales + b * p.s_scales;
    uint8_t* zeros = p.zeros ? p.zeros + b * p.s_scales : nullptr;
    const int64_t work = (int64_t)((p.N + 15) / 16) * p.across;
    for (int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); i < work;
         i += (int64_t)gridDim.x * 4) {
        const int tn = (int)(i / p.across), kt = (int)(i % p.across), r = 16 * tn + lr;
        const int from = min(r, p.N - 1);             // rows past the last one: read as that one
        u32x4 w = {0, 0, 0, 0};
        uint16_t scale[PER];
        int zero[PER];
        if constexpr (PACK) {
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                const int g = kt * PER + j;
                const int64_t at = (b * p.N + from) * real + min(g, real - 1);
                const bool in = r < p.N && g < real;
                scale[j] = in ? p.src_scales[at] : 0;
                zero[j] = in && p.src_zeros ? p.src_zeros[at] : 0;
            }
            const uint8_t* row = p.src + (b * p.N + from) * p.K;
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int c = 128 * kt + 32 * s + 8 * lq;
                u32x2_a1 x = {0, 0};
                if (c + 8 <= p.K)
                    x = *reinterpret_cast<const u32x2_a1*>(row + c);
                else
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (c + e < p.K) x[e / 4] |= (uint32_t)row[c + e] << (8 * (e % 4));
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    w[s] |= (x[e / 4] >> (8 * (e % 4)) & 15) << int4_shift(e);
                if (r >= p.N) w[s] = 0;
            }
        } else {
            const char* row = reinterpret_cast<const char*>(p.W) +
                              (b * p.sW + (int64_t)from * p.ldw) * (DT == DT_F32 ? 4 : 2);
            Raw8<DT> raw[4];
#pragma unroll
            for (int s = 0; s < 4; ++s) raw[s].load(row, 128 * kt + 32 * s + 8 * lq, p.K);
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                float v[STEPS][8], lo = 0.0f, hi = 0.0f;
#pragma unroll
                for (int s = 0; s < STEPS; ++s) {
                    raw[j * STEPS + s].get(v[s]);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        lo = fminf(lo, v[s][e]);
                        hi = fmaxf(hi, v[s][e] == v[s][e] ? v[s][e] : __builtin_huge_valf());
                    }
                }
                lo = int4_over_row(lo, [](float x, float y) { return fminf(x, y); });
                hi = int4_over_row(hi, [](float x, float y) { return fmaxf(x, y); });
                const bool in = r < p.N && kt * PER + j < real;
                float s = zeros ? (hi - lo) / 15.0f : fmaxf(hi, -lo) / 7.0f;
                uint16_t f = p.scale_bf16 ? from_f32<DT_BF16>(s) : from_f32<DT_F16>(s);
                s = int4_scale(p, f);
                if (!(s < __builtin_huge_valf())) {
                    f = p.scale_bf16 ? 0x7FC0 : 0x7E00;
                    s = 0.0f;
                }
                int z = 8;
                if (zeros && s > 0.0f)
                    z = (int)fmin(fmax(rint(-(double)lo / (double)s), 0.0), 15.0);
                scale[j] = in ? f : 0;
                zero[j] = in ? z : 0;
                // v / s from the hardware's reciprocal is off by less than 2^-16 up to 16; nearer to
                // a tie than that, or with a scale whose reciprocal may not be normal, it is divided
                const bool plain = s > 0x1p-100f && s < 0x1p100f;
                const float inv = __builtin_amdgcn_rcpf(s);
#pragma unroll
                for (int k = 0; k < STEPS; ++k)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float q = fminf(fmaxf(v[k][e] * inv, -32.0f), 32.0f);
                        float n = __builtin_rintf(q);
                        if (!plain || !(__builtin_fabsf(q - n) < 0.4999f))
                            n = s > 0.0f ? (float)fmin(fmax(rint((double)v[k][e] / (double)s), -32.0),
                                                       32.0)
                                         : 0.0f;
                        const int code = s > 0.0f ? min(max((int)n + z, 0), 15) : 8;
                        const bool at = in && 128 * kt + 32 * (j * STEPS + k) + 8 * lq + e < p.K;
                        w[j * STEPS + k] |= (at ? (uint32_t)code : 0u) << int4_shift(e);
                    }
            }
        }
        if (kt < p.tiles_k)
            *reinterpret_cast<u32x4*>(codes + ((int64_t)tn * p.tiles_k + kt) * 1024 + 16 * lane) = w;
        if (lq == 0) {
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                const int g = kt * PER + j;
                const int64_t at = ((int64_t)tn * p.tiles_g + g / 4) * 64 + 4 * lr + g % 4;
                scales[at] = scale[j];
                if (zeros) zeros[at] = (uint8_t)zero[j];
            }
        }
    }
}

template <int DT, int GROUP>
__global__ void __launch_bounds__(256) int4_dequantize_kernel(const Int4PackParams p) {
    constexpr int PER = 128 / GROUP;
    const int64_t b = blockIdx.z;
    const int lane = threadIdx.x & 63, lr = lane & 15, lq = lane >> 4;
    const uint8_t* codes = p.codes + b * p.s_codes;
    const uint16_t* scales = p.scales + b * p.s_scales;
    const uint8_t* zeros = p.zeros ? p.zeros + b * p.s_scales : nullptr;
    const int64_t work = (int64_t)((p.N + 15) / 16) * p.across;
    for (int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); i < work;
         i += (int64_t)gridDim.x * 4) {
        const int tn = (int)(i / p.across), kt = (int)(i % p.across), r = 16 * tn + lr;
        const u32x4 w = *reinterpret_cast<const u32x4*>(
            codes + ((int64_t)tn * p.tiles_k + kt) * 1024 + 16 * lane);
        float f[PER];
        int z[PER];
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int g = kt * PER + j;
            const int64_t at = ((int64_t)tn * p.tiles_g + g / 4) * 64 + 4 * lr + g % 4;
            f[j] = int4_scale(p, scales[at]);
            z[j] = zeros ? zeros[at] : 8;
        }
        if (r >= p.N) continue;
        char* row = reinterpret_cast<char*>(p.out) +
                    (b * p.sW + (int64_t)r * p.ldw) * (DT == DT_F32 ? 4 : 2);
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int j = s * 32 / GROUP;
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = f[j] * (float)((int)(w[s] >> int4_shift(e) & 15) - z[j]);
            store8<DT>(row, 128 * kt + 32 * s + 8 * lq, p.K, v);
        }
    }
}

// Configurations of the product: rows and columns of a work-group in tiles of 16, and its waves; then
// what one takes in us, for the choice: start + rounds * round + tiles of K * (first, where there is
// one round of 256 work-groups, else rounds * per + more).
// Index = configuration id (SG_FORCE_INT4=<id> overrides the choice).
struct Int4Cfg {
    int MT, NT, NW;
    double start, round, first, per, more;
    const char* name;
};
#define SG_INT4_FEW(X)                                \
    X(0, 1, 1, 8, 3.0, 0.5, 0.107, 0.107, 0.0)        \
    X(1, 1, 2, 8, 2.5, 1.0, 0.138, 0.138, 0.0)        \
    X(2, 1, 3, 8, 2.2, 1.4, 0.155, 0.155, 0.0)        \
    X(3, 1, 4, 4, 4.1, 0.4, 0.154, 0.154, 0.0)        \
    X(4, 1, 6, 4, 4.8, 0.5, 0.193, 0.193, 0.0)
#define SG_INT4_MANY(X)                               \
    X(5, 4, 8, 4, 6.0, 1.3, 0.79, 0.555, 0.0)         \
    X(6, 4, 8, 8, 7.2, 1.3, 0.60, 0.70, -0.08)        \
    X(7, 2, 8, 8, 5.6, 0.65, 0.40, 0.34, 0.03)        \
    X(8, 2, 8, 4, 5.0, 0.65, 0.545, 0.31, 0.10)
#define SG_INT4_ROW(ID, MT, NT, NW, START, ROUND, FIRST, PER, MORE) \
    {MT, NT, NW, START, ROUND, FIRST, PER, MORE, #MT "x" #NT " " #NW "w"},
constexpr Int4Cfg kInt4Cfg[] = {SG_INT4_FEW(SG_INT4_ROW) SG_INT4_MANY(SG_INT4_ROW)};
#undef SG_INT4_ROW
constexpr int kNumInt4Cfg = sizeof(kInt4Cfg) / sizeof(kInt4Cfg[0]);
constexpr int kNumInt4Few = 5;                           // those of SG_INT4_FEW

template <int DT, bool ZEROS>
hipError_t launch_int4(int group, int cfg, const Int4Params& x, unsigned blocks, hipStream_t st);

}  // namespace sg

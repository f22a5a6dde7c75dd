// api_int4.hip -- the C ABI of 4-bit integer weights: argument checks, kernel choice and launches
// on the caller's stream.  Declarations and contracts are in include/swiglu_gemm.h.  Nothing here
// allocates or keeps a workspace.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdlib>

#include "abi_checks.hpp"
#include "int4.hpp"
#include "swiglu_gemm.h"

using namespace sg;

namespace {

bool group_ok(int64_t group) { return group == 32 || group == 64 || group == 128; }
bool half_type(int dtype) { return dtype == SG_F16 || dtype == SG_BF16; }

// The configuration with the least time after the figures beside it (the rows of each expert are not
// known here: their mean stands for them, a run of n rows making n / bm + 1/2 tiles, at least one; a
// load that is not even can have a run many times the mean, whose weight 16-row strips read once for
// each 16 rows).  They were fitted to every configuration forced on some 120 products (MI355X, weights
// cold); on 48 products, most of them drawn at random, the choice takes 1.02 of the best in the mean, 1.19 at most (1000 rows of 64
// experts, fp16, 2048 by 2816: 54.9 us by 16-row strips of 64 columns, 46.4 by 32-row tiles; next 1.12).
// Both sides where it turns (us; bf16, groups of 128, rows x K by N):
//   strips of 16 or 32 columns: 1 x 4096 by 4096 4.9, 5.7;  32 x 4096 by 4096 11.6, 8.2
//   32 or 48: 1 x 4096 by 11008 8.2, 7.2;  48 or 64: 96 x 2048 by 2048 9.9, 6.8
//   64 or 96: 96 x 4096 by 4096 15.2, 18.2;  16 x 4096 by 22016 18.5, 14.7
//   16-row strips or 32-row tiles in two parts of K: 128 x 4096 by 4096 15.8, 18.5; 192 rows 21.1, 18.9;
//   those, or whole: 256 x 4096 by 4096 19.1, 23.1; 256 x 4096 by 11008 41.1, 39.3
//   32-row or 64-row tiles in two parts: 256 x 4096 by 4096 19.1, 26.3; 512 x 11008 by 4096 67.1, 60.7
//   32-row or 64-row tiles: 384 x 4096 by 11008 61.4, 58.3; 32 rows of each of 64 experts 66.0, 69.6
// Not fitted but measured: up to 16 rows in the mean no tile of more rows is taken (16 x 4096 by 22016
// 14.7, tiles 16.7), and 96-column strips only for one weight (98 rows of 32 experts, 1024 by 2816, 15.4
// by 64 columns and 23.7; 320 rows of 64, 4096 by 1024, 31.9 and 34.9).
int choose(const GroupedParams& q) {
    if (const char* s = std::getenv("SG_FORCE_INT4")) {
        const int c = std::atoi(s);
        if (*s && c >= 0 && c < kNumInt4Cfg) return c;
    }
    const double runs = q.experts < q.rows ? q.experts : q.rows, mean = q.rows / runs;
    const double tiles_k = (double)cdiv(q.g.K, 128);
    int best = 0;
    double least = INFINITY;
    for (int i = 0; i < (mean > 16.0 ? kNumInt4Cfg : kNumInt4Few); ++i) {
        const Int4Cfg& c = kInt4Cfg[i];
        if (c.NT == 6 && q.experts > 1) continue;
        const int bm = 16 * c.MT;
        const double high = q.experts == 1 ? (double)cdiv(q.rows, bm)
                                           : runs * std::fmax(1.0, mean / bm + 0.5);
        const double rounds = std::ceil(high * cdiv(q.g.N, 16 * c.NT) / 256.0);
        const double t = c.start + rounds * c.round +
                         tiles_k * (rounds > 1.0 ? rounds * c.per + c.more : c.first);
        if (t < least) {
            least = t;
            best = i;
        }
    }
    return best;
}

int run_product(const char* what, int64_t experts, const int32_t* offsets, const int32_t* order,
                int64_t top_k, int64_t T, int64_t M, int64_t N, int64_t K, int64_t group,
                const void* A, int64_t lda, const void* codes, const void* scales,
                const void* zeros, int dtype, Int4Params& x, void* stream) {
    x.q.g.A = static_cast<const uint16_t*>(A);
    x.q.g.lda = lda;
    x.q.g.N = (int)N;
    x.q.g.K = (int)K;
    x.q.g.group_m = 4;
    x.q.offsets = offsets;
    x.q.experts = (int)experts;
    x.q.rows = (int)M;
    x.order = order;
    x.top_k = (int)top_k;
    x.T = (int)T;
    x.codes = static_cast<const uint8_t*>(codes);
    x.scales = static_cast<const uint16_t*>(scales);
    x.zeros = static_cast<const uint8_t*>(zeros);
    x.s_codes = SG_INT4_CODE_BYTES(N, K);
    x.s_scales = SG_INT4_SCALES(N, K, group);
    x.tiles_k = (int)int4_tiles_k(K);
    x.tiles_g = (int)int4_tiles_g(K, group);
    const int cfg = choose(x.q);
    const int mt = kInt4Cfg[cfg].MT, nt = kInt4Cfg[cfg].NT;
    x.q.g.tiles_n = (int)cdiv(N, 16 * nt);
    const int64_t tiles_m = offsets ? most_row_tiles(M, experts, 16 * mt) : cdiv(M, 16 * mt);
    const int64_t blocks = tiles_m * x.q.g.tiles_n;
    if (blocks > kMaxBlocks) return status_of(hipErrorInvalidConfiguration);
    describe(what, cfg, kInt4Cfg[cfg].name);
    hipStream_t st = static_cast<hipStream_t>(stream);
    const unsigned b = (unsigned)blocks;
    const int g = (int)group;
    return status_of(dtype == SG_F16 ? zeros ? launch_int4<DT_F16, true>(g, cfg, x, b, st)
                                             : launch_int4<DT_F16, false>(g, cfg, x, b, st)
                     : zeros         ? launch_int4<DT_BF16, true>(g, cfg, x, b, st)
                                     : launch_int4<DT_BF16, false>(g, cfg, x, b, st));
}

enum { QUANTIZE, PACK, DEQUANTIZE };
template <int DT, int GROUP>
void launch_tiles(int what, const Int4PackParams& p, const dim3& grid, hipStream_t st) {
    const dim3 block(256);
    if (what == DEQUANTIZE)
        hipLaunchKernelGGL((int4_dequantize_kernel<DT, GROUP>), grid, block, 0, st, p);
    else if (what == QUANTIZE)
        hipLaunchKernelGGL((int4_pack_kernel<DT, GROUP, false>), grid, block, 0, st, p);
    else if constexpr (DT == DT_F32)                       // (packing reads no floats)
        hipLaunchKernelGGL((int4_pack_kernel<DT, GROUP, true>), grid, block, 0, st, p);
}
template <int DT>
void launch_tiles(int what, const Int4PackParams& p, const dim3& grid, hipStream_t st) {
    if (p.group == 32) launch_tiles<DT, 32>(what, p, grid, st);
    else if (p.group == 64) launch_tiles<DT, 64>(what, p, grid, st);
    else launch_tiles<DT, 128>(what, p, grid, st);
}
int run_tiles(const char* name, int what, Int4PackParams& p, int dtype, int64_t batch, void* stream) {
    // quantising and packing fill whole tiles of scales, which may reach past those of codes
    p.across = what == DEQUANTIZE ? p.tiles_k : p.tiles_g * 4 * p.group / 128;
    const int64_t blocks = cdiv(cdiv(p.N, 16) * p.across, 4);
    const dim3 grid((unsigned)(blocks < 65536 ? blocks : 65536), 1, (unsigned)batch);
    hipStream_t st = static_cast<hipStream_t>(stream);
    describe(name, -2, "");
    if (dtype == SG_F32) launch_tiles<DT_F32>(what, p, grid, st);
    else if (dtype == SG_F16) launch_tiles<DT_F16>(what, p, grid, st);
    else launch_tiles<DT_BF16>(what, p, grid, st);
    return status_of(hipGetLastError());
}

Int4PackParams pack_params(int64_t N, int64_t K, int64_t group, const void* codes,
                           const void* scales, const void* zeros) {
    Int4PackParams p{};
    p.N = (int)N;
    p.K = (int)K;
    p.group = (int)group;
    p.codes = static_cast<uint8_t*>(const_cast<void*>(codes));
    p.scales = static_cast<uint16_t*>(const_cast<void*>(scales));
    p.zeros = static_cast<uint8_t*>(const_cast<void*>(zeros));
    p.s_codes = SG_INT4_CODE_BYTES(N, K);
    p.s_scales = SG_INT4_SCALES(N, K, group);
    p.tiles_k = (int)int4_tiles_k(K);
    p.tiles_g = (int)int4_tiles_g(K, group);
    return p;
}

}  // namespace

extern "C" {

int sg_int4_quantize(const void* W, int64_t ldw, int64_t strideW, int64_t batch, int64_t N,
                     int64_t K, int dtype, int64_t group, void* codes, void* scales, void* zeros,
                     int scale_dtype, void* stream) {
    const bool any = batch > 0 && N > 0 && K > 0;
    if (any && !W) return -1;
    if (ldw < (K > 1 ? K : 1)) return -2;
    if (strideW < 0 || (batch > 1 && strideW > kMaxStride)) return -3;
    if (batch < 0 || batch > 65535) return -4;
    if (N < 0 || N > kMaxDim) return -5;
    if (K < 0 || K > kMaxDim) return -6;
    if (dtype != SG_F32 && !half_type(dtype)) return -7;
    if (!group_ok(group)) return -8;
    if (any && (!codes || !aligned(codes, 16))) return -9;
    if (any && (!scales || !aligned(scales, 8))) return -10;
    if (!aligned(zeros, 4)) return -11;
    if (!half_type(scale_dtype)) return -12;
    if (!any) return 0;
    Int4PackParams p = pack_params(N, K, group, codes, scales, zeros);
    p.W = W;
    p.ldw = ldw;
    p.sW = batch > 1 ? strideW : 0;
    p.scale_bf16 = scale_dtype == SG_BF16;
    return run_tiles("int4_quantize", QUANTIZE, p, dtype, batch, stream);
}

int sg_int4_pack(const void* src, const void* src_scales, const void* src_zeros, int64_t batch,
                 int64_t N, int64_t K, int64_t group, void* codes, void* scales, void* zeros,
                 void* stream) {
    const bool any = batch > 0 && N > 0 && K > 0;
    if (any && !src) return -1;
    if (any && (!src_scales || !aligned(src_scales, 2))) return -2;
    if (any && !src_zeros != !zeros) return -3;
    if (batch < 0 || batch > 65535) return -4;
    if (N < 0 || N > kMaxDim) return -5;
    if (K < 0 || K > kMaxDim) return -6;
    if (!group_ok(group)) return -7;
    if (any && (!codes || !aligned(codes, 16))) return -8;
    if (any && (!scales || !aligned(scales, 8))) return -9;
    if (!aligned(zeros, 4)) return -10;
    if (!any) return 0;
    Int4PackParams p = pack_params(N, K, group, codes, scales, zeros);
    p.src = static_cast<const uint8_t*>(src);
    p.src_scales = static_cast<const uint16_t*>(src_scales);
    p.src_zeros = static_cast<const uint8_t*>(src_zeros);
    return run_tiles("int4_pack", PACK, p, SG_F32, batch, stream);
}

int sg_int4_dequantize(const void* codes, const void* scales, const void* zeros, int scale_dtype,
                       int64_t batch, int64_t N, int64_t K, int64_t group, void* W, int64_t ldw,
                       int64_t strideW, int dtype, void* stream) {
    const bool any = batch > 0 && N > 0 && K > 0;
    if (any && (!codes || !aligned(codes, 16))) return -1;
    if (any && (!scales || !aligned(scales, 8))) return -2;
    if (!aligned(zeros, 4)) return -3;
    if (!half_type(scale_dtype)) return -4;
    if (batch < 0 || batch > 65535) return -5;
    if (N < 0 || N > kMaxDim) return -6;
    if (K < 0 || K > kMaxDim) return -7;
    if (!group_ok(group)) return -8;
    if (any && !W) return -9;
    if (ldw < (K > 1 ? K : 1)) return -10;
    if (strideW < 0) return -11;
    if (batch > 1 && any && (strideW > kMaxStride || !apart(strideW, N, ldw, K))) return -11;
    if (dtype != SG_F32 && !half_type(dtype)) return -12;
    if (!any) return 0;
    Int4PackParams p = pack_params(N, K, group, codes, scales, zeros);
    p.out = W;
    p.ldw = ldw;
    p.sW = batch > 1 ? strideW : 0;
    p.scale_bf16 = scale_dtype == SG_BF16;
    return run_tiles("int4_dequantize", DEQUANTIZE, p, dtype, batch, stream);
}

int sg_int4_gemm(int64_t experts, const int32_t* offsets, const int32_t* order, int64_t top_k,
                 int64_t T, int64_t M, int64_t N, int64_t K, int64_t group, float alpha,
                 const void* A, int64_t lda, const void* codes, const void* scales,
                 const void* zeros, void* C, int64_t ldc, int dtype, int c_dtype, void* stream) {
    if (experts < 1 || experts > kMaxExperts) return -1;
    if (!offsets && experts != 1) return -2;
    if (top_k < 1 || top_k > 65536 || (!order && top_k != 1)) return -4;
    if (M < 0 || M > kMaxDim) return -6;
    if (N < 0 || N > kMaxDim) return -7;
    if (K < 0 || K > kMaxDim) return -8;
    const bool reads = M > 0 && N > 0 && K > 0 && alpha != 0.0f;
    if (T < 0 || T > kMaxDim || (!order && T != M) || (reads && T == 0)) return -5;
    if (!group_ok(group)) return -9;
    if (reads && !A) return -11;
    if (lda < (K > 1 ? K : 1)) return -12;
    if (reads && (!codes || !aligned(codes, 16))) return -13;
    if (reads && (!scales || !aligned(scales, 8))) return -14;
    if (!aligned(zeros, 4)) return -15;
    if (M > 0 && N > 0 && !C) return -16;
    if (ldc < (N > 1 ? N : 1)) return -17;
    if (!half_type(dtype)) return -18;
    if (c_dtype != dtype && c_dtype != SG_F32) return -19;
    if (M == 0 || N == 0) return 0;
    Int4Params x{};
    x.q.g.C = C;
    x.q.g.ldc = ldc;
    x.q.g.alpha = reads ? alpha : 0.0f;
    x.c_f32 = c_dtype == SG_F32;
    return run_product("int4_gemm", experts, offsets, order, top_k, T, M, N, reads ? K : 0, group,
                       A, lda, codes, scales, zeros, dtype, x, stream);
}

int sg_int4_swiglu_gemm(int64_t experts, const int32_t* offsets, const int32_t* order,
                        int64_t top_k, int64_t T, int64_t M, int64_t N, int64_t K, int64_t group,
                        const void* A, int64_t lda, const void* codes, const void* scales,
                        const void* zeros, void* Y, int64_t ldy, int dtype, void* stream) {
    if (experts < 1 || experts > kMaxExperts) return -1;
    if (!offsets && experts != 1) return -2;
    if (top_k < 1 || top_k > 65536 || (!order && top_k != 1)) return -4;
    if (M < 0 || M > kMaxDim) return -6;
    if (N < 0 || N > kMaxDim / 2) return -7;
    if (K < 0 || K > kMaxDim) return -8;
    const bool reads = M > 0 && N > 0 && K > 0;
    if (T < 0 || T > kMaxDim || (!order && T != M) || (reads && T == 0)) return -5;
    if (!group_ok(group)) return -9;
    if (reads && !A) return -10;
    if (lda < (K > 1 ? K : 1)) return -11;
    if (reads && (!codes || !aligned(codes, 16))) return -12;
    if (reads && (!scales || !aligned(scales, 8))) return -13;
    if (!aligned(zeros, 4)) return -14;
    if (M > 0 && N > 0 && !Y) return -15;
    if (ldy < (N > 1 ? N : 1)) return -16;
    if (!half_type(dtype)) return -17;
    if (M == 0 || N == 0) return 0;
    Int4Params x{};
    x.q.g.C = Y;
    x.q.g.ldc = ldy;
    x.q.g.alpha = 1.0f;
    x.swiglu = 1;
    return run_product("int4_swiglu", experts, offsets, order, top_k, T, M, 2 * N, reads ? K : 0,
                       group, A, lda, codes, scales, zeros, dtype, x, stream);
}

}  // extern "C"

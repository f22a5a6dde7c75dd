// api_experts.hip -- the C ABI of the products grouped by expert and of microscaled 4-bit
// floating point: argument checks, kernel choice and launches on the caller's stream.
// Declarations and contracts are in include/swiglu_gemm.h.  Nothing here allocates or keeps
// a workspace.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstddef>
#include <cstdint>
#include <cstdlib>

#include "configs16.hpp"
#include "grouped.hpp"
#include "grouped_dma.hpp"
#include "mx4.hpp"
#include "mx4_dma.hpp"
#include "swiglu_gemm.h"

using namespace sg;

namespace sg {
void set_last_config(const char* text, size_t len);   // api.hip
}

namespace {

constexpr int64_t kMaxDim = (int64_t)1 << 30;
constexpr int64_t kMaxExperts = (int64_t)1 << 16;
// tile-rows of an expert walked together (2, 8 and 16 measured the same)
constexpr int kGroupM = 4;
constexpr int64_t kMaxBlocks = (int64_t)1 << 22;   // work-groups of one launch
// elements from one matrix to the next: with 65536 of them no offset in bytes passes 64 bits
constexpr int64_t kMaxStride = (int64_t)1 << 44;

bool aligned(const void* p, int bytes) { return ((uintptr_t)p % bytes) == 0; }
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
int status_of(hipError_t e) { return e == hipSuccess ? 0 : (int)e; }
// Whether matrices of `rows` rows, `stride` elements apart, do not reach into one another (no
// product is formed that could pass 64 bits).
bool apart(int64_t stride, int64_t rows, int64_t ld, int64_t cols) {
    return stride >= cols && (rows <= 1 || (stride - cols) / (rows - 1) >= ld);
}
bool finite_positive(float x) { return std::isfinite(x) && x > 0.0f; }

// Upper bound of the tiles of bm rows that `experts` runs of M rows in all can have: every
// run that is not empty rounds up once.
int64_t most_row_tiles(int64_t M, int64_t experts, int bm) {
    const int64_t runs = experts < M ? experts : M;
    return (M + runs * (bm - 1)) / bm;
}

// "<what> cfg=<id> <name>" for sg_last_config(); put together by hand: snprintf takes half a
// microsecond of calls that take eight.
void describe(const char* what, int cfg, const char* name) {
    char text[160];
    size_t n = 0;
    auto put = [&](const char* s) {
        while (*s && n + 1 < sizeof(text)) text[n++] = *s++;
    };
    put(what);
    if (cfg >= -1) {
        const char digits[] = {(char)('0' + cfg / 10), (char)('0' + cfg % 10), 0};
        put(" cfg=");
        put(cfg < 0 ? "-1" : cfg < 10 ? digits + 1 : digits);
        put(" ");
        put(name);
    }
    text[n] = 0;
    set_last_config(text, n);
}

hipError_t launch_dt(int dtype, int epi, bool ta, bool tb, int cfg, const GroupedParams& q,
                     int64_t blocks, hipStream_t st) {
    if (blocks > kMaxBlocks) return hipErrorInvalidConfiguration;
    const unsigned b = (unsigned)blocks;
    if (dtype == SG_F16) return launch_grouped<DT_F16>(epi, ta, tb, cfg, q, b, st);
    if (dtype == SG_BF16) return launch_grouped<DT_BF16>(epi, ta, tb, cfg, q, b, st);
    return launch_grouped<DT_E4M3>(epi, ta, tb, cfg, q, b, st);
}

// SG_FORCE_GROUPED=<id>: that tile for every call it can run (-1: the 64 x 64 tiles).
bool forced_group(int* cfg) {
    const char* s = std::getenv("SG_FORCE_GROUPED");
    if (!s || !*s) return false;
    *cfg = std::atoi(s);
    return true;
}

// Whether tile c can run the problem: 16-byte aligned operands, rows and expert strides,
// DMA-compatible tiles, and every lane's offset from its tile's base below 2^31 bytes.
bool group_cfg_ok(const GroupCfg& c, bool ta, bool tb, int esz, const GroupedParams& q) {
    if ((c.e4m3 != 0) != (esz == 1) || (ta ? c.rate_d : c.rate) <= 0.0) return false;
    if (!aligned(q.g.A, 16) || !aligned(q.g.B, 16)) return false;
    constexpr int64_t kLim = (int64_t)1 << 31;
    if (q.g.lda >= kLim || q.g.ldb >= kLim) return false;
    if (q.g.lda * esz % 16 != 0 || q.g.ldb * esz % 16 != 0 || q.sB % 16 != 0) return false;
    const int nw = c.WM * c.WN;
    if (!dma_tile_ok(!ta, c.BM, c.BK, esz, nw) || !dma_tile_ok(tb, c.BN, c.BK, esz, nw))
        return false;
    return ((ta ? c.BK : c.BM) * q.g.lda + 256) * esz < kLim &&
           ((tb ? c.BN : c.BK) * q.g.ldb + 256) * esz < kLim;
}

// Rounds of work-groups over the CUs, `occ` to a CU: whole ones while there are few and one
// work-group fills a CU, the mean when there are many or two share it (one that has a CU alone
// takes 0.62 of the time).
constexpr int kNumCU = 256;
double rounds_of(double w, int occ) {
    if (w <= 1.0) return occ == 1 || w > 0.5 ? 1.0 : 0.62;
    if (occ == 2) return w + 0.45;
    return w < 4.0 ? std::ceil(w - 0.06) : w + 0.4;
}

// Microseconds of `tiles` tiles of `flops` each that move `bytes` in all: never less than the
// bytes take.
double est_us(double tiles, int occ, double flops, double rate, double fixed, double bytes) {
    const double t =
        rounds_of(tiles / (kNumCU * occ), occ) * occ * (flops / (rate * 1e6) + fixed);
    const double m = bytes / 4.8e6;
    return std::fmax(t, m) + 0.15 * std::fmin(t, m);
}

// The rows of each expert are not known here, so their mean stands for them: a run of n rows is
// taken for n/BM + 1/2 tiles, never less than one; less where the tile has a low form (0.6 of
// the time of a whole one).
double est_rows(const GroupCfg& c, bool tb, int esz, const GroupedParams& q) {
    const double runs = q.experts < q.rows ? q.experts : q.rows, mean = q.rows / runs;
    const int low = group_low(false, c.BM, c.BN, c.WM, c.WN);
    double per = std::fmax(mean <= low ? 0.6 : 1.0, mean / c.BM + (low ? 0.35 : 0.5));
    if (q.experts == 1) {
        const int rest = q.rows % c.BM;
        per = q.rows / c.BM + (rest == 0 ? 0.0 : rest <= low ? 0.6 : 1.0);
    }
    const double bytes = (double)q.rows * q.g.K * esz + runs * q.g.K * (double)q.g.N * esz +
                         (double)q.rows * q.g.N * 2.0;
    const int occ = group_occ(c.S * (c.BM + c.BN) * c.BK * esz);
    // B stored N x K in a 32-deep ring is read in 64-byte pieces: 0.85 of the rate (16 experts of
    // 512 rows, K = 2816, N = 2048: 143 us on 128 x 256 x 32, 124 us on the 64-deep one)
    const double rate = c.rate * (tb && c.BK * esz < 128 ? 0.85 : 1.0);
    return est_us((double)cdiv(q.g.N, c.BN) * runs * per, occ, 2.0 * c.BM * c.BN * q.g.K, rate,
                  c.fixed, bytes);
}

double est_depth(const GroupCfg& c, const GroupedParams& q) {
    const double tiles = (double)q.experts * cdiv(q.g.M, c.BM) * cdiv(q.g.N, c.BN);
    const double bytes = (double)q.rows * (q.g.M + q.g.N) * 2.0 +
                         (double)q.experts * q.g.M * (double)q.g.N * 2.0;
    const int occ = group_occ(c.S * (c.BM + c.BN) * c.BK * 2);
    return est_us(tiles, occ, 2.0 * c.BM * c.BN * q.rows / q.experts, c.rate_d, c.fixed_d, bytes);
}

// The tile with the least estimated time, or -1: the kernel for every alignment.
int choose_group(bool depth, bool tb, int esz, const GroupedParams& q) {
    int cfg = -1;
    if (forced_group(&cfg))
        return cfg >= 0 && cfg < kNumGroupCfg && group_cfg_ok(kGroupCfg[cfg], depth, tb, esz, q)
                   ? cfg
                   : -1;
    double best = 0.0;
    for (int i = 0; i < kNumGroupCfg; ++i) {
        const GroupCfg& c = kGroupCfg[i];
        if (!group_cfg_ok(c, depth, tb, esz, q)) continue;
        const double t = depth ? est_depth(c, q) : est_rows(c, tb, esz, q);
        if (cfg < 0 || t < best) {
            cfg = i;
            best = t;
        }
    }
    // A few rows each against weights stored K x N: where 256-wide tiles make close to one round
    // (3/4 of the CUs to all), their 512-byte pieces of a weight's rows stream faster than twice
    // as many of 256 bytes.  Measured on 306 such calls (8 to 64 experts, N = 768 to 8192, K = 512
    // to 4096, 1 to 32 rows each, plain and SwiGLU), 256 wide over 128 wide: at 192 tiles 1.05 for
    // K = 512, 1.00 for 1024, 0.99 for 2048, 0.94 for 4096; at 256 tiles 0.94, 0.93, 0.91, 0.86
    // (K = 2048, 32 experts, N = 2048: 49.3 -> 46.5 us); all of them 0.95 in the mean, the worst
    // 1.10 (K = 512, 64 experts, N = 768: 12.8 -> 14.1 us).  With more tiles it loses: N = 2816,
    // 512 rows of 48 experts, 80.4 -> 89.8 us.
    if (cfg == kFewRows && !depth && !tb) {
        const int64_t runs = q.experts < q.rows ? q.experts : q.rows;
        const int64_t wide = runs * cdiv(q.g.N, kGroupCfg[kTwoPerCu].BN);
        if (4 * wide >= 3 * kNumCU && wide <= kNumCU && q.rows <= 32 * runs &&
            group_cfg_ok(kGroupCfg[kTwoPerCu], false, tb, esz, q))
            cfg = kTwoPerCu;
    }
    return cfg;
}

// Products over the rows of each expert: chooses the tile and launches.
int run_rows(const char* what, int epi, bool tb, int dtype, GroupedParams q, hipStream_t st) {
    const int esz = dtype == SG_F8E4M3 ? 1 : 2;
    const int cfg = q.g.K > 0 ? choose_group(false, tb, esz, q) : -1;
    const int bm = cfg < 0 ? 64 : kGroupCfg[cfg].BM, bn = cfg < 0 ? 64 : kGroupCfg[cfg].BN;
    q.g.group_m = kGroupM;
    q.g.tiles_n = (int)cdiv(q.g.N, bn);
    q.g.vec_c = aligned(q.g.C, 8) && q.g.ldc % 4 == 0;
    describe(what, cfg, cfg < 0 ? "any 64x64x32" : kGroupCfg[cfg].name);
    return status_of(launch_dt(
        dtype, epi, false, tb, cfg, q,
        group_blocks(most_row_tiles(q.rows, q.experts, bm) * q.g.tiles_n, 2), st));
}

// Products that sum over the rows of each expert.
int run_depth(const char* what, int epi, int dtype, GroupedParams q, hipStream_t st) {
    const int cfg = q.rows > 0 ? choose_group(true, false, 2, q) : -1;
    const int bm = cfg < 0 ? 64 : kGroupCfg[cfg].BM, bn = cfg < 0 ? 64 : kGroupCfg[cfg].BN;
    q.g.group_m = kGroupM;
    q.g.tiles_m = (int)cdiv(q.g.M, bm);
    q.g.tiles_n = (int)cdiv(q.g.N, bn);
    q.g.vec_c = aligned(q.g.C, 8) && q.g.ldc % 4 == 0 && q.sC % 8 == 0;
    describe(what, cfg, cfg < 0 ? "any 64x64x32" : kGroupCfg[cfg].name);
    return status_of(launch_dt(dtype, epi, true, false, cfg, q,
                               (int64_t)q.experts * q.g.tiles_m * q.g.tiles_n, st));
}

// Wide tiles where they fill the chip, 32-row ones for a few rows, the narrow ones of those where
// even they leave CUs idle.  Measured against every tile forced on 130 problems (one weight of 1 to
// 8192 rows, N = 2048 to 11008; 8 to 64 experts of 1 to 1024 rows, plain and SwiGLU; K = 2048 and
// 4096): the choice takes 1.03 of the best tile's time in the mean, at most 1.22.  32-row tiles are
// mostly ahead of 128 x 128 while there are fewer than 256 of the latter (one weight, 1024 rows,
// 2048 x 2048: 9.1 against 10.5 us; not so 256 rows, 2048 x 11008: 13.8 against 11.6 us), 256 x 256
// of 128 x 128 in long runs (32 experts of 512 rows, 2048 x 2 x 1408: 69 against 83 us).  It errs
// most where 128 x 128 runs what makes 150 to 512 tiles of 256 x 256 (64 experts of 256 rows, 2048 x
// 2048: 68 against 56 us).
int choose_mx4(const GroupedParams& q) {
    if (const char* s = std::getenv("SG_FORCE_MX4")) {
        const int c = std::atoi(s);
        if (*s && c >= 0 && c < kNumMxCfg) return c;
    }
    const int64_t runs = q.experts < q.rows ? q.experts : q.rows, mean = q.rows / runs;
    auto tiles = [&](int bm, int bn) { return runs * cdiv(mean, bm) * cdiv(q.g.N, bn); };
    if (mean >= 384 && tiles(256, 256) >= 400) return 3;
    if (mean > 32 && tiles(128, 128) >= 256) return 2;
    return tiles(32, 128) >= 256 ? 1 : 0;
}

int run_mx4(const char* what, int epi, int dtype, MxParams x, hipStream_t st) {
    GroupedParams& q = x.q;
    // a lane's offset from its tile's base stays below 2^31 bytes
    if (256 * q.g.lda + 256 >= (int64_t)1 << 31) return status_of(hipErrorInvalidConfiguration);
    const int cfg = choose_mx4(q);
    const MxCfg& c = kMxCfg[cfg];
    q.g.group_m = kGroupM;
    q.g.tiles_n = (int)cdiv(q.g.N, c.BN);
    q.g.vec_c = aligned(q.g.C, 8) && q.g.ldc % 4 == 0;
    const int64_t tiles_m = q.offsets ? most_row_tiles(q.rows, q.experts, c.BM) : cdiv(q.rows, c.BM);
    const int64_t blocks = group_blocks(tiles_m * q.g.tiles_n, 2);
    if (blocks > kMaxBlocks) return status_of(hipErrorInvalidConfiguration);
    describe(what, cfg, c.name);
    return status_of(launch_mx4(epi, dtype == SG_F16 ? DT_F16 : DT_BF16, cfg, x,
                                (unsigned)blocks, st));
}

}  // namespace

extern "C" {

int sg_grouped_gemm(char transB, int64_t experts, const int32_t* offsets, int64_t M, int64_t N,
                    int64_t K, float alpha, const float* scale, const void* A, int64_t lda,
                    const void* B, int64_t ldb, int64_t strideB, float beta, void* C,
                    int64_t ldc, int dtype, void* stream) {
    const bool tb = transB == 'T' || transB == 't';
    if (!tb && transB != 'N' && transB != 'n') return -1;
    if (experts < 1 || experts > kMaxExperts) return -2;
    if (!offsets) return -3;
    if (M < 0 || M > kMaxDim) return -4;
    if (N < 0 || N > kMaxDim) return -5;
    if (K < 0 || K > kMaxDim) return -6;
    const bool reads = M > 0 && N > 0 && K > 0 && alpha != 0.0f;
    if (reads && !A) return -9;
    if (lda < (K > 1 ? K : 1)) return -10;
    if (reads && !B) return -11;
    const int64_t brow = tb ? K : N;
    if (ldb < (brow > 1 ? brow : 1)) return -12;
    if (strideB < 0 || (experts > 1 && strideB > kMaxStride)) return -13;
    if (M > 0 && N > 0 && !C) return -15;
    if (ldc < (N > 1 ? N : 1)) return -16;
    if (dtype != SG_F16 && dtype != SG_BF16 && dtype != SG_F8E4M3) return -17;
    if (M == 0 || N == 0) return 0;
    const int esz = dtype == SG_F8E4M3 ? 1 : 2;
    GroupedParams q{};
    q.g.A = static_cast<const uint16_t*>(A);
    q.g.B = static_cast<const uint16_t*>(B);
    q.g.C = C;
    q.g.lda = lda;
    q.g.ldb = ldb;
    q.g.ldc = ldc;
    q.g.N = (int)N;
    q.g.K = reads ? (int)K : 0;
    q.g.alpha = reads ? alpha : 0.0f;    // no products: no factor of theirs, infinite or not
    q.g.beta = beta;
    q.offsets = offsets;
    q.scale = reads ? scale : nullptr;
    q.experts = (int)experts;
    q.rows = (int)M;
    q.sB = experts > 1 ? strideB * esz : 0;
    return run_rows("grouped_gemm", EPI_GEMM, tb, dtype, q, static_cast<hipStream_t>(stream));
}

int sg_grouped_gemm_wgrad(int64_t experts, const int32_t* offsets, int64_t M, int64_t N,
                          int64_t K, float alpha, const void* A, int64_t lda, const void* D,
                          int64_t ldd, float beta, void* C, int64_t ldc, int64_t strideC,
                          int dtype, int c_dtype, void* stream) {
    if (experts < 1 || experts > kMaxExperts) return -1;
    if (!offsets) return -2;
    if (M < 0 || M > kMaxDim) return -3;
    if (N < 0 || N > kMaxDim) return -4;
    if (K < 0 || K > kMaxDim) return -5;
    const bool reads = M > 0 && N > 0 && K > 0 && alpha != 0.0f;
    if (reads && !A) return -7;
    if (lda < (K > 1 ? K : 1)) return -8;
    if (reads && !D) return -9;
    if (ldd < (N > 1 ? N : 1)) return -10;
    if (N > 0 && K > 0 && !C) return -12;
    if (ldc < (N > 1 ? N : 1)) return -13;
    if (experts > 1 && N > 0 && K > 0 && (strideC > kMaxStride || !apart(strideC, K, ldc, N)))
        return -14;
    if (dtype != SG_F16 && dtype != SG_BF16) return -15;
    if (c_dtype != dtype && c_dtype != SG_F32) return -16;
    if (N == 0 || K == 0) return 0;
    const bool f32 = c_dtype == SG_F32;
    GroupedParams q{};
    q.g.A = static_cast<const uint16_t*>(A);
    q.g.B = static_cast<const uint16_t*>(D);
    q.g.C = C;
    q.g.lda = lda;
    q.g.ldb = ldd;
    q.g.ldc = ldc;
    q.g.M = (int)K;
    q.g.N = (int)N;
    q.g.alpha = alpha;
    q.g.beta = beta;
    q.offsets = offsets;
    q.experts = (int)experts;
    q.rows = reads ? (int)M : 0;      // nothing is summed, and nothing read, past row 0
    q.sC = experts > 1 ? strideC * (f32 ? 4 : 2) : 0;
    return run_depth("grouped_wgrad", f32 ? EPI_GEMM_F32 : EPI_GEMM, dtype, q,
                     static_cast<hipStream_t>(stream));
}

int sg_grouped_swiglu_gemm(int64_t experts, const int32_t* offsets, const void* A,
                           const void* Wfused, void* Y, int64_t M, int64_t N, int64_t K,
                           int dtype, float alpha, const float* scale, void* stream) {
    if (experts < 1 || experts > kMaxExperts) return -1;
    if (!offsets) return -2;
    const bool reads = M > 0 && N > 0 && K > 0;
    if (reads && !A) return -3;
    if (reads && !Wfused) return -4;
    if (M > 0 && N > 0 && !Y) return -5;
    if (M < 0 || M > kMaxDim) return -6;
    if (N < 0 || N > kMaxDim / 2) return -7;
    if (K < 0 || K > kMaxDim) return -8;
    if (dtype != SG_F16 && dtype != SG_BF16 && dtype != SG_F8E4M3) return -9;
    if (!finite_positive(alpha) || (dtype != SG_F8E4M3 && alpha != 1.0f)) return -10;
    if (scale && dtype != SG_F8E4M3) return -11;
    if (M == 0 || N == 0) return 0;
    GroupedParams q{};
    q.g.A = static_cast<const uint16_t*>(A);
    q.g.B = static_cast<const uint16_t*>(Wfused);
    q.g.C = Y;
    q.g.lda = K;
    q.g.ldb = 2 * N;
    q.g.ldc = N;
    q.g.N = (int)(2 * N);
    q.g.K = (int)K;
    q.g.alpha = alpha;
    q.g.epi_flags = aligned(Y, 16) && N % 8 == 0 ? EPI_Y16 : 0;
    q.offsets = offsets;
    q.scale = reads ? scale : nullptr;
    q.experts = (int)experts;
    q.rows = (int)M;
    q.sB = K * 2 * N * (dtype == SG_F8E4M3 ? 1 : 2);
    return run_rows("grouped_swiglu", EPI_SWIGLU, false, dtype, q,
                    static_cast<hipStream_t>(stream));
}

int sg_grouped_swiglu_gemm_bwd(int64_t experts, const int32_t* offsets, const void* A,
                               const void* Wfused, const void* dY, void* dH, int64_t M,
                               int64_t N, int64_t K, int dtype, void* stream) {
    if (experts < 1 || experts > kMaxExperts) return -1;
    if (!offsets) return -2;
    const bool reads = M > 0 && N > 0 && K > 0;
    if (reads && !A) return -3;
    if (reads && !Wfused) return -4;
    if (M > 0 && N > 0 && !dY) return -5;
    if (M > 0 && N > 0 && !dH) return -6;
    if (M < 0 || M > kMaxDim) return -7;
    if (N < 0 || N > kMaxDim / 2) return -8;
    if (K < 0 || K > kMaxDim) return -9;
    if (dtype != SG_F16 && dtype != SG_BF16) return -10;
    if (M == 0 || N == 0) return 0;
    GroupedParams q{};
    q.g.A = static_cast<const uint16_t*>(A);
    q.g.B = static_cast<const uint16_t*>(Wfused);
    q.g.C = dH;
    q.g.lda = K;
    q.g.ldb = 2 * N;
    q.g.ldc = 2 * N;
    q.g.N = (int)(2 * N);
    q.g.K = (int)K;
    q.g.alpha = 1.0f;
    q.offsets = offsets;
    q.dY = dY;
    q.experts = (int)experts;
    q.rows = (int)M;
    q.sB = K * 2 * N * 2;
    return run_rows("grouped_swiglu_bwd", EPI_SWIGLU_BWD, false, dtype, q,
                    static_cast<hipStream_t>(stream));
}

int sg_mxfp4_quantize(const void* X, int64_t ldx, int64_t strideX, int64_t batch, int64_t M,
                      int64_t K, int dtype, void* codes, void* scales, void* values,
                      void* stream) {
    if (M > 0 && K > 0 && batch > 0 && !X) return -1;
    if (ldx < (K > 1 ? K : 1)) return -2;
    if (strideX < 0 || (batch > 1 && strideX > kMaxStride)) return -3;
    if (batch < 0 || batch > 65535) return -4;
    if (M < 0 || M > kMaxDim) return -5;
    if (K < 0 || K > kMaxDim) return -6;
    if (dtype < SG_F32 || dtype > SG_BF16) return -7;
    if (!codes && !scales && !values) return -8;
    if (!aligned(codes, 4)) return -8;
    if (!aligned(scales, 4)) return -9;
    if (batch == 0 || M == 0 || K == 0) return 0;
    const int64_t blocks = cdiv(M, 32) * mx_tiles_k(K);
    if (blocks > kMaxBlocks) return status_of(hipErrorInvalidConfiguration);
    const int esz = dtype == SG_F32 ? 4 : 2;
    MxQuantParams p{};
    p.X = X;
    p.codes = static_cast<uint8_t*>(codes);
    p.scales = static_cast<uint8_t*>(scales);
    p.values = values;
    p.ldx = ldx;
    p.ldv = K;
    p.sX = batch > 1 ? strideX * esz : 0;
    p.sV = M * K * esz;
    p.M = (int)M;
    p.K = (int)K;
    p.vec_x = aligned(X, 16) && ldx % (16 / esz) == 0 && p.sX % 16 == 0;
    p.vec_v = aligned(values, 16) && K * esz % 16 == 0;
    const dim3 grid((unsigned)blocks, 1, (unsigned)batch);
    hipStream_t st = static_cast<hipStream_t>(stream);
    describe("mxfp4_quantize", -2, "");
    if (dtype == SG_F32)
        hipLaunchKernelGGL(mx_quantize_kernel<DT_F32>, grid, dim3(256), 0, st, p);
    else if (dtype == SG_F16)
        hipLaunchKernelGGL(mx_quantize_kernel<DT_F16>, grid, dim3(256), 0, st, p);
    else
        hipLaunchKernelGGL(mx_quantize_kernel<DT_BF16>, grid, dim3(256), 0, st, p);
    return status_of(hipGetLastError());
}

int sg_mxfp4_dequantize(const void* codes, const void* scales, int64_t batch, int64_t M,
                        int64_t K, void* X, int64_t ldx, int64_t strideX, int dtype,
                        void* stream) {
    const bool any = batch > 0 && M > 0 && K > 0;
    if (any && (!codes || !aligned(codes, 4))) return -1;
    if (any && !scales) return -2;
    if (batch < 0 || batch > 65535) return -3;
    if (M < 0 || M > kMaxDim) return -4;
    if (K < 0 || K > kMaxDim) return -5;
    if (any && !X) return -6;
    if (ldx < (K > 1 ? K : 1)) return -7;
    if (strideX < 0) return -8;
    if (batch > 1 && any && (strideX > kMaxStride || !apart(strideX, M, ldx, K))) return -8;
    if (dtype < SG_F32 || dtype > SG_BF16) return -9;
    if (!any) return 0;
    const int64_t blocks = cdiv(M, 32) * mx_tiles_k(K);
    if (blocks > kMaxBlocks) return status_of(hipErrorInvalidConfiguration);
    const int esz = dtype == SG_F32 ? 4 : 2;
    MxQuantParams p{};
    p.codes = const_cast<uint8_t*>(static_cast<const uint8_t*>(codes));
    p.scales = const_cast<uint8_t*>(static_cast<const uint8_t*>(scales));
    p.values = X;
    p.ldv = ldx;
    p.sV = batch > 1 ? strideX * esz : 0;
    p.M = (int)M;
    p.K = (int)K;
    p.vec_v = aligned(X, 16) && ldx % (16 / esz) == 0 && p.sV % 16 == 0;
    const dim3 grid((unsigned)blocks, 1, (unsigned)batch);
    hipStream_t st = static_cast<hipStream_t>(stream);
    describe("mxfp4_dequantize", -2, "");
    if (dtype == SG_F32)
        hipLaunchKernelGGL(mx_dequantize_kernel<DT_F32>, grid, dim3(256), 0, st, p);
    else if (dtype == SG_F16)
        hipLaunchKernelGGL(mx_dequantize_kernel<DT_F16>, grid, dim3(256), 0, st, p);
    else
        hipLaunchKernelGGL(mx_dequantize_kernel<DT_BF16>, grid, dim3(256), 0, st, p);
    return status_of(hipGetLastError());
}

int sg_mxfp4_tile_scales(const void* src, int64_t ld, int64_t stride, int64_t batch, int64_t M,
                         int64_t blocks, void* dst, void* stream) {
    const bool any = batch > 0 && M > 0 && blocks > 0;
    if (any && !src) return -1;
    if (ld < (blocks > 1 ? blocks : 1)) return -2;
    if (stride < 0 || (batch > 1 && stride > kMaxStride)) return -3;
    if (batch < 0 || batch > 65535) return -4;
    if (M < 0 || M > kMaxDim) return -5;
    if (blocks < 0 || blocks > kMaxDim / kMxBlock) return -6;
    if (any && (!dst || !aligned(dst, 4))) return -7;
    if (!any) return 0;
    const int64_t work = cdiv(cdiv(M, 32) * cdiv(blocks, 8) * (kMxTileBytes / 4), 256);
    const dim3 grid((unsigned)(work < 8192 ? work : 8192), 1, (unsigned)batch);
    describe("mxfp4_tile_scales", -2, "");
    hipLaunchKernelGGL(mx_tile_scales_kernel, grid, dim3(256), 0,
                       static_cast<hipStream_t>(stream), static_cast<const uint8_t*>(src), ld,
                       stride, static_cast<uint8_t*>(dst), (int)M, (int)blocks);
    return status_of(hipGetLastError());
}

int sg_mxfp4_gemm(int64_t experts, const int32_t* offsets, int64_t M, int64_t N, int64_t K,
                  float alpha, const void* A, const void* As, const void* B, const void* Bs,
                  void* C, int64_t ldc, int dtype, void* stream) {
    if (experts < 1 || experts > kMaxExperts) return -1;
    if (!offsets && experts != 1) return -2;
    if (M < 0 || M > kMaxDim) return -3;
    if (N < 0 || N > kMaxDim) return -4;
    if (K < 0 || K > kMaxDim) return -5;
    const bool reads = M > 0 && N > 0 && K > 0 && alpha != 0.0f;
    if (reads && (!A || !aligned(A, 16))) return -7;
    if (reads && (!As || !aligned(As, 4))) return -8;
    if (reads && (!B || !aligned(B, 16))) return -9;
    if (reads && (!Bs || !aligned(Bs, 4))) return -10;
    if (M > 0 && N > 0 && !C) return -11;
    if (ldc < (N > 1 ? N : 1)) return -12;
    if (dtype < SG_F32 || dtype > SG_BF16) return -13;
    if (M == 0 || N == 0) return 0;
    MxParams x{};
    x.q.g.A = static_cast<const uint16_t*>(A);
    x.q.g.B = static_cast<const uint16_t*>(B);
    x.q.g.C = C;
    x.q.g.lda = x.q.g.ldb = mx_row_bytes(K);
    x.q.g.ldc = ldc;
    x.q.g.N = (int)N;
    x.q.g.K = reads ? (int)mx_blocks(K) : 0;
    x.q.g.alpha = reads ? alpha : 0.0f;
    x.q.offsets = offsets;
    x.q.experts = (int)experts;
    x.q.rows = (int)M;
    x.q.sB = N * mx_row_bytes(K);
    x.As = static_cast<const uint8_t*>(As);
    x.Bs = static_cast<const uint8_t*>(Bs);
    x.sBs = mx_scale_bytes(N, K);
    x.tiles_k = (int)mx_tiles_k(K);
    return run_mx4("mxfp4_gemm", dtype == SG_F32 ? EPI_GEMM_F32 : EPI_GEMM, dtype, x,
                   static_cast<hipStream_t>(stream));
}

int sg_mxfp4_swiglu_gemm(int64_t experts, const int32_t* offsets, int64_t M, int64_t N,
                         int64_t K, const void* A, const void* As, const void* W,
                         const void* Ws, void* Y, int dtype, void* stream) {
    if (experts < 1 || experts > kMaxExperts) return -1;
    if (!offsets && experts != 1) return -2;
    if (M < 0 || M > kMaxDim) return -3;
    if (N < 0 || N > kMaxDim / 2) return -4;
    if (K < 0 || K > kMaxDim) return -5;
    const bool reads = M > 0 && N > 0 && K > 0;
    if (reads && (!A || !aligned(A, 16))) return -6;
    if (reads && (!As || !aligned(As, 4))) return -7;
    if (reads && (!W || !aligned(W, 16))) return -8;
    if (reads && (!Ws || !aligned(Ws, 4))) return -9;
    if (M > 0 && N > 0 && !Y) return -10;
    if (dtype != SG_F16 && dtype != SG_BF16) return -11;
    if (M == 0 || N == 0) return 0;
    MxParams x{};
    x.q.g.A = static_cast<const uint16_t*>(A);
    x.q.g.B = static_cast<const uint16_t*>(W);
    x.q.g.C = Y;
    x.q.g.lda = x.q.g.ldb = mx_row_bytes(K);
    x.q.g.ldc = N;
    x.q.g.N = (int)(2 * N);
    x.q.g.K = (int)mx_blocks(K);
    x.q.g.alpha = 1.0f;
    x.q.g.epi_flags = aligned(Y, 16) && N % 8 == 0 ? EPI_Y16 : 0;
    x.q.offsets = offsets;
    x.q.experts = (int)experts;
    x.q.rows = (int)M;
    x.q.sB = 2 * N * mx_row_bytes(K);
    x.As = static_cast<const uint8_t*>(As);
    x.Bs = static_cast<const uint8_t*>(Ws);
    x.sBs = mx_scale_bytes(2 * N, K);
    x.tiles_k = (int)mx_tiles_k(K);
    return run_mx4("mxfp4_swiglu", EPI_SWIGLU, dtype, x, static_cast<hipStream_t>(stream));
}

}  // extern "C"

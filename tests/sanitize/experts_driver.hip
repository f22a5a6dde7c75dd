// Host-only, under AddressSanitizer and UndefinedBehaviorSanitizer: the C ABI of the grouped and
// 4-bit operators (api_experts.hip) from the arguments to the launch.  Every invalid argument
// returns its status; valid calls of every size, up to the largest dimensions and strides, choose
// a tile and a number of work-groups, which stand-ins for the kernels' launchers look over in
// place of running them.  It needs no GPU.  Exit status 0: no finding and every status as
// documented.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <limits>

#include "grouped.hpp"
#include "grouped_dma.hpp"
#include "mx4.hpp"
#include "mx4_dma.hpp"
#include "swiglu_gemm.h"

using namespace sg;

static int failures = 0;
static long launches = 0;
#define EXPECT(call, want)                                                          \
    do {                                                                            \
        const int got_ = (call);                                                    \
        if (got_ != (want)) {                                                       \
            fprintf(stderr, "line %d: %s returned %d, want %d\n", __LINE__, #call,   \
                    got_, (int)(want));                                             \
            ++failures;                                                             \
        }                                                                           \
    } while (0)
#define CHECK(cond)                                                                 \
    do {                                                                            \
        if (!(cond)) {                                                              \
            fprintf(stderr, "line %d: not so: %s\n", __LINE__, #cond);              \
            ++failures;                                                             \
        }                                                                           \
    } while (0)

// The most tiles of bm rows that a table for q can hold, and the halves that the last round of
// each XCD may be split into.
static int64_t most_items(const GroupedParams& q, int bm, int bn) {
    const int64_t runs = q.experts < q.rows ? q.experts : q.rows;
    // all runs but one of one row, and the rest
    const int64_t rest = q.rows - (runs - 1);
    return (runs - 1 + (rest + bm - 1) / bm) * ((q.g.N + (int64_t)bn - 1) / bn);
}

static void look(bool ta, int cfg, int bm, int bn, const GroupedParams& q, unsigned blocks) {
    ++launches;
    CHECK(blocks > 0 && blocks <= 1u << 22);
    CHECK(q.g.tiles_n == (q.g.N + (int64_t)bn - 1) / bn);
    if (ta)
        CHECK((int64_t)blocks == (int64_t)q.experts * q.g.tiles_m * q.g.tiles_n);
    else
        CHECK((int64_t)blocks >= most_items(q, bm, bn) + kXcds * kXcdCus);
    (void)cfg;
}

namespace sg {
void set_last_config(const char* text, size_t len) {
    CHECK(len < 160 && std::strlen(text) == len);
}
template <int DT>
static hipError_t stand_in(bool ta, int cfg, const GroupedParams& q, unsigned blocks) {
    CHECK(cfg >= -1 && cfg < kNumGroupCfg);
    const GroupCfg any = {0, 64, 64};
    const GroupCfg& c = cfg < 0 ? any : kGroupCfg[cfg];
    if (cfg >= 0) {
        CHECK((c.e4m3 != 0) == (DT == DT_E4M3));
        CHECK((ta ? c.rate_d : c.rate) > 0.0);
        CHECK((uintptr_t)q.g.A % 16 == 0 && (uintptr_t)q.g.B % 16 == 0);
    }
    look(ta, cfg, c.BM, c.BN, q, blocks);
    return hipSuccess;
}
template <>
hipError_t launch_grouped<DT_F16>(int, bool ta, bool, int cfg, const GroupedParams& q, unsigned blocks,
                                  hipStream_t) {
    return stand_in<DT_F16>(ta, cfg, q, blocks);
}
template <>
hipError_t launch_grouped<DT_BF16>(int, bool ta, bool, int cfg, const GroupedParams& q,
                                   unsigned blocks, hipStream_t) {
    return stand_in<DT_BF16>(ta, cfg, q, blocks);
}
template <>
hipError_t launch_grouped<DT_E4M3>(int, bool ta, bool, int cfg, const GroupedParams& q,
                                   unsigned blocks, hipStream_t) {
    return stand_in<DT_E4M3>(ta, cfg, q, blocks);
}
hipError_t launch_mx4(int, int, int cfg, const MxParams& x, unsigned blocks, hipStream_t) {
    CHECK(cfg >= 0 && cfg < kNumMxCfg);
    look(false, cfg, kMxCfg[cfg].BM, kMxCfg[cfg].BN, x.q, blocks);
    return hipSuccess;
}
}  // namespace sg

static char memory[64] __attribute__((aligned(16)));

int main() {
    void* P = memory;                    // never dereferenced
    void* ODD = memory + 2;              // an element-aligned operand
    void* BAD = memory + 1;
    void* Z = nullptr;
    const int32_t* O = reinterpret_cast<const int32_t*>(memory);
    const float* S = reinterpret_cast<const float*>(memory);
    const int F16 = SG_F16, BF = SG_BF16, F8 = SG_F8E4M3, F32 = SG_F32;
    const int64_t FAR = std::numeric_limits<int64_t>::max(), BIG = (int64_t)1 << 30;
    const float inf = std::numeric_limits<float>::infinity();

    // ---- invalid arguments, in order
    EXPECT(sg_grouped_gemm('X', 2, O, 4, 8, 16, 1.f, nullptr, P, 16, P, 8, 128, 0.f, P, 8, BF, Z), -1);
    EXPECT(sg_grouped_gemm('N', 0, O, 4, 8, 16, 1.f, nullptr, P, 16, P, 8, 128, 0.f, P, 8, BF, Z), -2);
    EXPECT(sg_grouped_gemm('N', 65537, O, 4, 8, 16, 1.f, nullptr, P, 16, P, 8, 128, 0.f, P, 8, BF, Z), -2);
    EXPECT(sg_grouped_gemm('N', 2, nullptr, 4, 8, 16, 1.f, nullptr, P, 16, P, 8, 128, 0.f, P, 8, BF, Z), -3);
    EXPECT(sg_grouped_gemm('N', 2, O, -1, 8, 16, 1.f, nullptr, P, 16, P, 8, 128, 0.f, P, 8, BF, Z), -4);
    EXPECT(sg_grouped_gemm('N', 2, O, 4, BIG + 1, 16, 1.f, nullptr, P, 16, P, 8, 128, 0.f, P, 8, BF, Z), -5);
    EXPECT(sg_grouped_gemm('N', 2, O, 4, 8, -1, 1.f, nullptr, P, 16, P, 8, 128, 0.f, P, 8, BF, Z), -6);
    EXPECT(sg_grouped_gemm('N', 2, O, 4, 8, 16, 1.f, nullptr, Z, 16, P, 8, 128, 0.f, P, 8, BF, Z), -9);
    EXPECT(sg_grouped_gemm('N', 2, O, 4, 8, 16, 1.f, nullptr, P, 15, P, 8, 128, 0.f, P, 8, BF, Z), -10);
    EXPECT(sg_grouped_gemm('N', 2, O, 4, 8, 16, 1.f, nullptr, P, 16, Z, 8, 128, 0.f, P, 8, BF, Z), -11);
    EXPECT(sg_grouped_gemm('T', 2, O, 4, 8, 16, 1.f, nullptr, P, 16, P, 15, 128, 0.f, P, 8, BF, Z), -12);
    EXPECT(sg_grouped_gemm('N', 2, O, 4, 8, 16, 1.f, nullptr, P, 16, P, 8, -1, 0.f, P, 8, BF, Z), -13);
    EXPECT(sg_grouped_gemm('N', 2, O, 4, 8, 16, 1.f, nullptr, P, 16, P, 8, 128, 0.f, Z, 8, BF, Z), -15);
    EXPECT(sg_grouped_gemm('N', 2, O, 4, 8, 16, 1.f, nullptr, P, 16, P, 8, 128, 0.f, P, 7, BF, Z), -16);
    EXPECT(sg_grouped_gemm('N', 2, O, 4, 8, 16, 1.f, nullptr, P, 16, P, 8, 128, 0.f, P, 8, 7, Z), -17);
    EXPECT(sg_grouped_gemm('N', 2, O, 0, 8, 16, 1.f, nullptr, Z, 16, Z, 8, 128, 0.f, Z, 8, BF, Z), 0);
    EXPECT(sg_grouped_gemm_wgrad(0, O, 4, 8, 16, 1.f, P, 16, P, 8, 0.f, P, 8, 128, BF, F32, Z), -1);
    EXPECT(sg_grouped_gemm_wgrad(2, nullptr, 4, 8, 16, 1.f, P, 16, P, 8, 0.f, P, 8, 128, BF, F32, Z), -2);
    EXPECT(sg_grouped_gemm_wgrad(2, O, 4, 8, 16, 1.f, P, 15, P, 8, 0.f, P, 8, 128, BF, F32, Z), -8);
    EXPECT(sg_grouped_gemm_wgrad(2, O, 4, 8, 16, 1.f, P, 16, P, 7, 0.f, P, 8, 128, BF, F32, Z), -10);
    EXPECT(sg_grouped_gemm_wgrad(2, O, 4, 8, 16, 1.f, P, 16, P, 8, 0.f, P, 7, 128, BF, F32, Z), -13);
    EXPECT(sg_grouped_gemm_wgrad(2, O, 4, 8, 16, 1.f, P, 16, P, 8, 0.f, P, 8, 127, BF, F32, Z), -14);
    EXPECT(sg_grouped_gemm_wgrad(2, O, 4, 8, 16, 1.f, P, 16, P, 8, 0.f, P, FAR, FAR, BF, F32, Z), -14);
    EXPECT(sg_grouped_gemm_wgrad(2, O, 4, 8, 16, 1.f, P, 16, P, 8, 0.f, P, 8, 128, F8, F32, Z), -15);
    EXPECT(sg_grouped_gemm_wgrad(2, O, 4, 8, 16, 1.f, P, 16, P, 8, 0.f, P, 8, 128, BF, F16, Z), -16);
    EXPECT(sg_grouped_gemm_wgrad(2, O, 4, 0, 16, 1.f, P, 16, P, 8, 0.f, Z, 8, 128, BF, F32, Z), 0);
    EXPECT(sg_grouped_swiglu_gemm(2, O, P, P, P, 4, BIG, 16, BF, 1.f, nullptr, Z), -7);
    EXPECT(sg_grouped_swiglu_gemm(2, O, P, P, P, 4, 8, 16, BF, 2.f, nullptr, Z), -10);
    EXPECT(sg_grouped_swiglu_gemm(2, O, P, P, P, 4, 8, 16, F8, inf, nullptr, Z), -10);
    EXPECT(sg_grouped_swiglu_gemm(2, O, P, P, P, 4, 8, 16, BF, 1.f, S, Z), -11);
    EXPECT(sg_grouped_swiglu_gemm_bwd(2, O, P, P, Z, P, 4, 8, 16, BF, Z), -5);
    EXPECT(sg_grouped_swiglu_gemm_bwd(2, O, P, P, P, P, 4, 8, 16, F8, Z), -10);
    EXPECT(sg_mxfp4_quantize(Z, 64, 0, 1, 4, 64, BF, P, P, Z, Z), -1);
    EXPECT(sg_mxfp4_quantize(P, 63, 0, 1, 4, 64, BF, P, P, Z, Z), -2);
    EXPECT(sg_mxfp4_quantize(P, 64, 0, 65536, 4, 64, BF, P, P, Z, Z), -4);
    EXPECT(sg_mxfp4_quantize(P, 64, 0, 1, 4, 64, BF, BAD, P, Z, Z), -8);
    EXPECT(sg_mxfp4_quantize(P, 64, 0, 1, 4, 64, BF, Z, Z, Z, Z), -8);
    EXPECT(sg_mxfp4_quantize(P, 64, 0, 1, 4, 64, BF, P, BAD, Z, Z), -9);
    EXPECT(sg_mxfp4_quantize(P, BIG, 0, 1, BIG, BIG, BF, P, P, P, Z), hipErrorInvalidConfiguration);
    EXPECT(sg_mxfp4_quantize(P, 64, 0, 1, 0, 64, BF, P, P, Z, Z), 0);
    EXPECT(sg_mxfp4_dequantize(P, P, 2, 4, 64, P, 64, 255, BF, Z), -8);
    EXPECT(sg_mxfp4_dequantize(P, P, 2, 4, 64, P, FAR, FAR, BF, Z), -8);
    EXPECT(sg_mxfp4_dequantize(P, P, 1, BIG, BIG, P, BIG, 0, BF, Z), hipErrorInvalidConfiguration);
    EXPECT(sg_mxfp4_dequantize(Z, Z, 0, 4, 64, Z, 64, 0, BF, Z), 0);
    EXPECT(sg_mxfp4_tile_scales(P, 3, 16, 1, 4, 4, P, Z), -2);
    EXPECT(sg_mxfp4_tile_scales(P, 4, 16, 1, 4, 4, BAD, Z), -7);
    EXPECT(sg_mxfp4_tile_scales(Z, 4, 16, 1, 0, 4, Z, Z), 0);
    EXPECT(sg_mxfp4_gemm(2, nullptr, 4, 8, 64, 1.f, P, P, P, P, P, 8, BF, Z), -2);
    EXPECT(sg_mxfp4_gemm(1, nullptr, 4, 8, 64, 1.f, ODD, P, P, P, P, 8, BF, Z), -7);
    EXPECT(sg_mxfp4_gemm(1, nullptr, 4, 8, 64, 1.f, P, P, P, P, P, 7, BF, Z), -12);
    EXPECT(sg_mxfp4_gemm(1, nullptr, 4, 8, BIG, 1.f, P, P, P, P, P, 8, BF, Z),
           hipErrorInvalidConfiguration);
    EXPECT(sg_mxfp4_swiglu_gemm(1, nullptr, 4, 8, 64, P, P, P, P, P, F32, Z), -11);

    // ---- valid calls: every status is 0 or "too many work-groups", every launch is looked over
    const int64_t sizes[] = {1, 2, 7, 8, 33, 64, 100, 256, 1000, 2048, 16384, 1 << 20, BIG};
    const int64_t counts[] = {1, 3, 64, 65, 150, 65536};
    auto ok = [](int status, int far = 0) {
        if (far ? status != far : status != 0 && status != (int)hipErrorInvalidConfiguration) {
            fprintf(stderr, "a valid call returned %d\n", status);
            ++failures;
        }
    };
    for (int64_t E : counts)
        for (int64_t M : sizes)
            for (int64_t N : sizes)
                for (int64_t K : sizes) {
                    // matrices further apart than any memory reaches are refused
                    const bool far = E > 1 && N * K > (int64_t)1 << 44;
                    for (int dt : {F16, BF, F8})
                        for (char tb : {'N', 'T'}) {
                            const int64_t ldb = tb == 'T' ? K : N;
                            ok(sg_grouped_gemm(tb, E, O, M, N, K, 1.f, S, P, K, P, ldb, N * K, 1.f, P,
                                               N, dt, Z),
                               far ? -13 : 0);
                        }
                    ok(sg_grouped_gemm('N', E, O, M, N, K, 0.f, S, Z, K, Z, N, 0, 1.f, P, N, BF, Z));
                    ok(sg_grouped_gemm('T', E, O, M, N, K, inf, nullptr, ODD, K, ODD, K, 1, 0.f, P, N,
                                       BF, Z));
                    for (int cdt : {BF, F32})
                        ok(sg_grouped_gemm_wgrad(E, O, M, N, K, 1.f, P, K, P, N, 0.f, P, N, N * K, BF,
                                                 cdt, Z),
                           far ? -14 : 0);
                    ok(sg_mxfp4_gemm(E, O, M, N, K < 1 << 20 ? K : 1 << 20, 1.f, P, P, P, P, P, N, BF,
                                     Z));
                    if (N < BIG) {
                        ok(sg_grouped_swiglu_gemm(E, O, P, P, P, M, N, K, F8, 2.f, S, Z));
                        ok(sg_grouped_swiglu_gemm_bwd(E, O, P, P, P, P, M, N, K, BF, Z));
                        ok(sg_mxfp4_swiglu_gemm(E, O, M, N, K < 1 << 20 ? K : 1 << 20, P, P, P, P, P,
                                                BF, Z));
                    }
                }
    // ---- strides that no address is formed from: any value is allowed
    for (int dt : {F16, F8})
        for (char tb : {'N', 'T'}) {
            EXPECT(sg_grouped_gemm(tb, 1, O, 4, 8, 16, 1.f, S, P, 16, P, 16, FAR, 0.f, P, 8, dt, Z), 0);
            EXPECT(sg_grouped_gemm(tb, 1, O, 1, 1, 1, 1.f, S, P, FAR, P, FAR, FAR, 0.f, P, FAR, dt, Z), 0);
        }
    EXPECT(sg_grouped_gemm_wgrad(1, O, 4, 8, 16, 1.f, P, 16, P, 8, 0.f, P, 8, FAR, BF, F32, Z), 0);
    EXPECT(sg_grouped_gemm_wgrad(1, O, 1, 8, 1, 1.f, P, FAR, P, FAR, 0.f, P, FAR, FAR, BF, F32, Z), 0);
    EXPECT(sg_grouped_gemm_wgrad(2, O, 1, 8, 1, 1.f, P, FAR, P, FAR, 0.f, P, FAR, 8, BF, F32, Z), 0);
    EXPECT(sg_mxfp4_gemm(1, nullptr, 1, 8, 64, 1.f, P, P, P, P, P, FAR, F32, Z), 0);
    // (nothing of these two to do, so that no kernel is launched)
    EXPECT(sg_mxfp4_quantize(P, FAR, FAR, 1, 0, 64, BF, P, P, Z, Z), 0);
    EXPECT(sg_mxfp4_dequantize(P, P, 1, 0, 64, P, FAR, FAR, BF, Z), 0);

    if (failures) return 1;
    std::printf("ok: %ld launches\n", launches);
    return launches > 0 ? 0 : 1;
}

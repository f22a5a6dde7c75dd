// Host-only, under AddressSanitizer and UndefinedBehaviorSanitizer: the C ABI of the routing to
// experts and of 4-bit integer weights (api_routing.hip, api_int4.hip) from the arguments to the
// launch.  Invalid arguments and launches past the largest grid return their status, calls with
// nothing to do return 0; products of every size, up to the largest dimensions, choose a tile and
// a number of work-groups, which a stand-in for the kernels' launcher looks over in place of running
// them.  No other valid call is made, so no kernel runs.  Exit status 0: no finding.
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <limits>

#include "abi_checks.hpp"
#include "int4.hpp"
#include "swiglu_gemm.h"

using namespace sg;

static int failures = 0;
static long launches = 0;
#define EXPECT(call, want)                                                          \
    do {                                                                            \
        const int got_ = (call);                                                    \
        if (got_ != (int)(want)) {                                                  \
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

namespace sg {
void set_last_config(const char* text, size_t len) {
    CHECK(len < 160 && std::strlen(text) == len);
}
// Every tile that a table of the experts' rows can hold has a work-group.
static hipError_t look(bool zeros, int group, int cfg, const Int4Params& x, unsigned blocks) {
    ++launches;
    CHECK(cfg >= 0 && cfg < kNumInt4Cfg);
    CHECK(group == 32 || group == 64 || group == 128);
    const GroupedParams& q = x.q;
    const int64_t bm = 16 * kInt4Cfg[cfg].MT, bn = 16 * kInt4Cfg[cfg].NT;
    const int64_t runs = q.experts < q.rows ? q.experts : q.rows, rest = q.rows - (runs - 1);
    const int64_t tiles_n = cdiv(q.g.N, bn);
    CHECK(q.g.tiles_n == tiles_n);
    CHECK((int64_t)blocks >= (runs - 1 + cdiv(rest, bm)) * tiles_n);
    CHECK(blocks > 0 && (int64_t)blocks <= kMaxBlocks);
    CHECK(x.tiles_k == cdiv(q.g.K, 128) && x.tiles_g == cdiv(cdiv(q.g.K, group), 4));
    CHECK(zeros == (x.zeros != nullptr));
    CHECK(x.top_k >= 1 && x.T >= 0);
    return hipSuccess;
}
template <>
hipError_t launch_int4<DT_F16, false>(int g, int cfg, const Int4Params& x, unsigned b, hipStream_t) {
    return look(false, g, cfg, x, b);
}
template <>
hipError_t launch_int4<DT_F16, true>(int g, int cfg, const Int4Params& x, unsigned b, hipStream_t) {
    return look(true, g, cfg, x, b);
}
template <>
hipError_t launch_int4<DT_BF16, false>(int g, int cfg, const Int4Params& x, unsigned b, hipStream_t) {
    return look(false, g, cfg, x, b);
}
template <>
hipError_t launch_int4<DT_BF16, true>(int g, int cfg, const Int4Params& x, unsigned b, hipStream_t) {
    return look(true, g, cfg, x, b);
}
}  // namespace sg

static char memory[64] __attribute__((aligned(16)));

int main() {
    void* P = memory;                    // never dereferenced
    void* BAD = memory + 1;
    void* Z = nullptr;
    int32_t* I = reinterpret_cast<int32_t*>(memory);
    float* S = reinterpret_cast<float*>(memory);
    const int F16 = SG_F16, BF = SG_BF16, F32 = SG_F32;
    const int64_t FAR = std::numeric_limits<int64_t>::max(), BIG = (int64_t)1 << 30;
    const int64_t MANY = (int64_t)1 << 27;
    const int TOO_MANY = hipErrorInvalidConfiguration;

    // ---- routing
    EXPECT(sg_route_experts(P, FAR, MANY, 64, F32, 8, 0, S, 8, 4, 2, 1, 1.f, nullptr, I, S, Z), TOO_MANY);
    EXPECT(sg_route_experts(P, FAR, BIG, 1024, BF, 64, 1, S, 64, 64, 1, 0, 1.f, nullptr, I, S, Z), TOO_MANY);
    EXPECT(sg_route_experts(P, 8, 4, 8, F32, 2, 0, S, 64, 4, 2, 1, 1.f, nullptr, I, S, Z), -9);
    EXPECT(sg_route_experts(P, FAR, BIG + 1, 8, F32, 2, 0, S, 1, 1, 2, 1, 1.f, nullptr, I, S, Z), -3);
    EXPECT(sg_route_experts(Z, FAR, 0, 8, F32, 2, 0, S, 1, 1, 2, 1, 1.f, nullptr, nullptr, nullptr, Z), 0);
    EXPECT(sg_route_experts_bwd(P, FAR, MANY, 64, F16, 8, 1, 0, 1.f, I, S, P, FAR, Z), TOO_MANY);
    EXPECT(sg_route_experts_bwd(P, 64, 4, 64, F16, 65, 1, 0, 1.f, I, S, P, 64, Z), -6);
    EXPECT(sg_route_experts_bwd(Z, 64, 0, 64, F16, 8, 1, 0, 1.f, nullptr, nullptr, Z, FAR, Z), 0);
    EXPECT(sg_sort_experts(I, BIG + 1, 8, I, I, I, Z), -2);
    EXPECT(sg_sort_experts(nullptr, 8, 8, I, I, I, Z), -1);
    EXPECT(sg_sort_experts(I, 8, 65537, I, I, I, Z), -3);
    EXPECT(sg_spread_rows(P, FAR, BIG, 4096, BF, I, 65536, S, BIG, P, FAR, Z), TOO_MANY);
    EXPECT(sg_spread_rows(P, FAR, 4, 8, BF, I, 65537, S, 8, P, 8, Z), -7);
    EXPECT(sg_spread_rows(Z, 1, 4, 0, BF, nullptr, 8, S, 8, Z, 1, Z), 0);
    EXPECT(sg_combine_rows(P, FAR, BIG, BIG, BIG, F32, I, 65536, S, P, FAR, P, FAR, Z), TOO_MANY);
    EXPECT(sg_combine_rows(P, 8, 8, 8, 4, F32, I, 2, S, P, 7, P, 8, Z), -11);
    EXPECT(sg_combine_rows(Z, FAR, 8, 8, 0, F32, nullptr, 2, S, Z, 0, Z, FAR, Z), 0);
    EXPECT(sg_combine_rows_bwd(P, FAR, P, FAR, BIG, 8, BIG, F32, I, 65536, S, P, FAR, S, Z), TOO_MANY);
    EXPECT(sg_combine_rows_bwd(P, 8, Z, 8, 8, 8, 4, F32, I, 2, S, P, 8, S, Z), -3);
    EXPECT(sg_combine_rows_bwd(Z, 8, Z, 8, 8, 8, 4, F32, nullptr, 2, nullptr, Z, 8, nullptr, Z), 0);

    // ---- 4-bit weights
    EXPECT(sg_int4_quantize(P, FAR, ((int64_t)1 << 44) + 1, 2, 4, 64, BF, 64, P, P, Z, BF, Z), -3);
    EXPECT(sg_int4_quantize(P, 63, 0, 1, 4, 64, BF, 64, P, P, Z, BF, Z), -2);
    EXPECT(sg_int4_quantize(Z, FAR, FAR, 1, 0, 64, BF, 64, Z, Z, Z, BF, Z), 0);
    EXPECT(sg_int4_pack(P, P, P, 1, 4, 64, 64, P, P, Z, Z), -3);
    EXPECT(sg_int4_pack(P, BAD, Z, 1, 4, 64, 64, P, P, Z, Z), -2);
    EXPECT(sg_int4_pack(Z, Z, Z, 0, BIG, BIG, 32, Z, Z, Z, Z), 0);
    EXPECT(sg_int4_dequantize(P, P, Z, BF, 2, 4, 64, 64, P, FAR, FAR, BF, Z), -11);
    EXPECT(sg_int4_dequantize(P, P, Z, BF, 2, 4, 64, 64, P, 64, 255, BF, Z), -11);
    EXPECT(sg_int4_dequantize(Z, Z, Z, BF, 1, 0, 64, 64, Z, FAR, FAR, BF, Z), 0);
    EXPECT(sg_int4_gemm(1, nullptr, nullptr, 1, 4, 4, 8, 64, 64, 1.f, P, 64, BAD, P, Z, P, 8, BF, BF, Z), -13);
    EXPECT(sg_int4_gemm(1, nullptr, nullptr, 1, 0, 0, 8, 64, 64, 1.f, Z, 64, Z, Z, Z, Z, 8, BF, BF, Z), 0);
    EXPECT(sg_int4_swiglu_gemm(1, nullptr, nullptr, 1, 4, 4, BIG / 2 + 1, 64, 64, P, 64, P, P, Z, P, BIG, BF, Z),
           -7);

    // ---- valid products: every status is 0 or "too many work-groups"
    const int64_t sizes[] = {1, 2, 7, 16, 33, 64, 100, 256, 1000, 2048, 16384, 1 << 20, BIG};
    const int64_t counts[] = {1, 3, 64, 65, 150, 65536};
    auto ok = [](int status) {
        if (status != 0 && status != (int)hipErrorInvalidConfiguration) {
            fprintf(stderr, "a valid call returned %d\n", status);
            ++failures;
        }
    };
    for (int64_t E : counts)
        for (int64_t M : sizes)
            for (int64_t N : sizes)
                for (int64_t K : sizes)
                    for (int64_t group : {32, 64, 128})
                        for (int dt : {F16, BF}) {
                            void* zeros = (M + N + K) % 2 ? P : Z;
                            ok(sg_int4_gemm(E, I, nullptr, 1, M, M, N, K, group, 1.f, P, K, P, P, zeros, P,
                                            N, dt, dt, Z));
                            ok(sg_int4_gemm(E, I, I, 8, 5, M, N, K, group, 2.f, P, FAR, P, P, zeros, P,
                                            FAR, dt, F32, Z));
                            if (N <= BIG / 2)
                                ok(sg_int4_swiglu_gemm(E, I, I, 65536, BIG, M, N, K, group, P, K, P, P,
                                                       zeros, P, N, dt, Z));
                        }
    if (failures) return 1;
    std::printf("ok: %ld launches\n", launches);
    return launches > 0 ? 0 : 1;
}

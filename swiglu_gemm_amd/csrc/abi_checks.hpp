// abi_checks.hpp -- what the C ABI's entry points share on the host: limits, small arithmetic
// and the description of the last call.
#pragma once

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstddef>
#include <cstdint>

namespace sg {

void set_last_config(const char* text, size_t len);   // api.hip

constexpr int64_t kMaxDim = (int64_t)1 << 30;
constexpr int64_t kMaxExperts = (int64_t)1 << 16;
constexpr int64_t kMaxBlocks = (int64_t)1 << 22;   // work-groups of one launch
// elements from one matrix to the next: with 65536 of them no offset in bytes passes 64 bits
constexpr int64_t kMaxStride = (int64_t)1 << 44;

inline bool aligned(const void* p, int bytes) { return ((uintptr_t)p % bytes) == 0; }
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int status_of(hipError_t e) { return e == hipSuccess ? 0 : (int)e; }
// Whether matrices of `rows` rows, `stride` elements apart, do not reach into one another (no
// product is formed that could pass 64 bits).
inline bool apart(int64_t stride, int64_t rows, int64_t ld, int64_t cols) {
    return stride >= cols && (rows <= 1 || (stride - cols) / (rows - 1) >= ld);
}
inline bool finite_positive(float x) { return std::isfinite(x) && x > 0.0f; }

// Upper bound of the tiles of bm rows that `experts` runs of M rows in all can have: every
// run that is not empty rounds up once.
inline int64_t most_row_tiles(int64_t M, int64_t experts, int bm) {
    const int64_t runs = experts < M ? experts : M;
    return (M + runs * (bm - 1)) / bm;
}

// "<what> cfg=<id> <name>" for sg_last_config(); put together by hand: snprintf takes half a
// microsecond of calls that take eight.
inline void describe(const char* what, int cfg, const char* name) {
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

}  // namespace sg

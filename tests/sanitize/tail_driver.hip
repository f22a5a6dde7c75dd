// Host-only: every byte that the whole K tile at a tile's end would load, for small grouped
// problems with rows of no expert, padded rows and gaps between the experts' matrices, wherever
// tail_readable() lets it be read.  Prints the first byte that it must not load.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "grouped_dma.hpp"

using namespace sg;

static long checked = 0, let = 0;

static void fail(const char* what, long at) {
    std::printf("%s: loads element %ld\n", what, at);
    std::exit(1);
}

// elements [lo, hi) from the start of an operand, which owns the ranges of `own`
struct Range { long lo, hi; };
static void inside(const char* what, long lo, long hi, const std::vector<Range>& own) {
    for (long at = lo; at < hi; ++at) {
        bool ok = false;
        for (const Range& r : own) ok = ok || (at >= r.lo && at < r.hi);
        if (!ok) fail(what, at);
        ++checked;
    }
}

template <bool TA, bool TB, int BM, int BN, int BK>
static void problem(const std::vector<int>& off, int rows, int N, int K, int pada, int padb,
                    int gap) {
    const int E = (int)off.size() - 1, end = off[E];
    const long lda = K + pada, brow = TA ? N : TB ? K : N, ldb = brow + padb;
    const long bmat = (TB ? N : K) * ldb;                 // a matrix with its rows' padding
    GroupedParams q{};
    q.g.lda = lda;
    q.g.ldb = ldb;
    q.g.N = N;
    q.g.K = K;
    q.experts = E;
    q.rows = rows;
    q.sB = (bmat + gap) * 2;
    // depth: A and D are rows x K and rows x N, only the experts' rows are theirs
    const std::vector<Range> a_own = {{off[0] * lda, (end - 1) * lda + K}};
    std::vector<Range> b_own;
    if (TA) b_own.push_back({off[0] * ldb, (end - 1) * ldb + N});
    for (int e = 0; !TA && e < E; ++e) {
        const long at = e * (bmat + gap);
        // without a gap the padding of a matrix's last row runs into the next matrix
        b_own.push_back({at, gap || e + 1 == E ? at + bmat - padb : at + bmat});
    }
    for (int e = 0; e < E; ++e) {
        GroupItem it{};
        it.e = e;
        it.row0 = off[e];
        it.rows = off[e + 1] - off[e];
        if (it.rows <= 0) continue;
        Gemm16Params p = q.g;
        p.M = TA ? K : it.rows;
        p.K = TA ? it.rows : K;
        const int nkt = p.K / BK;
        if (p.K % BK == 0) continue;
        for (int m0 = 0; m0 < p.M; m0 += BM)
            for (int n0 = 0; n0 < N; n0 += BN) {
                if (!tail_readable<TA, TB, BM, BN, BK, 2>(q, it, p, end, m0, n0, nkt)) continue;
                ++let;
                const long k0 = (long)nkt * BK;
                if (TA) {
                    for (long k = k0; k < k0 + BK; ++k) {
                        const long r = it.row0 + k;
                        inside("A", r * lda + m0, r * lda + (m0 + BM < K ? m0 + BM : K), a_own);
                        inside("D", r * ldb + n0, r * ldb + (n0 + BN < N ? n0 + BN : N), b_own);
                    }
                    continue;
                }
                for (int i = 0; i < BM; ++i) {
                    const long r = it.row0 + (m0 + i < p.M ? m0 + i : p.M - 1);
                    inside("A", r * lda + k0, r * lda + k0 + BK, a_own);
                }
                const long b0 = e * (bmat + gap);
                if (TB) {
                    for (int i = 0; i < BN; ++i) {
                        const long r = n0 + i < N ? n0 + i : N - 1;
                        inside("B", b0 + r * ldb + k0, b0 + r * ldb + k0 + BK, b_own);
                    }
                } else {
                    for (long k = k0; k < k0 + BK; ++k) {
                        // the rows behind K are the next matrix's, without a gap
                        const long at = b0 + k * ldb;
                        inside("B", at + n0, at + (n0 + BN < N ? n0 + BN : N), b_own);
                    }
                }
            }
    }
}

template <int BM, int BN, int BK>
static void tile() {
    const std::vector<std::vector<int>> tables = {
        {0, 20, 20, 37}, {5, 6, 70, 71, 90}, {0, 33}, {7, 40, 41, 105}, {0, 64, 64}};
    for (const auto& off : tables)
        for (int behind : {0, 3, 40})
            for (int N : {8, 24, 72})
                for (int K : {8, 40, 72})
                    for (int pada : {0, 8})
                        for (int padb : {0, 8})
                            for (int gap : {0, 8, 200}) {
                                const int rows = off.back() + behind;
                                problem<false, false, BM, BN, BK>(off, rows, N, K, pada, padb, gap);
                                problem<false, true, BM, BN, BK>(off, rows, N, K, pada, padb, gap);
                                if (gap == 0)
                                    problem<true, false, BM, BN, BK>(off, rows, N, K, pada, padb, 0);
                            }
}

int main() {
    tile<16, 16, 16>();
    tile<32, 64, 64>();
    tile<128, 64, 32>();
    std::printf("ok: %ld tails read whole, %ld elements\n", let, checked);
    return let > 0 ? 0 : 1;
}

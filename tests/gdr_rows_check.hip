// Host check of the mapping from packed offsets to rows and chunk slots that the kernels use
// (gdr_sequence, gdr_chunk): every row and slot in range for any offsets, and for offsets in order
// every token in exactly one chunk of a slot of its own.  Prints the first failure and exits with 1.
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "../gated_delta_rule_31_amd/csrc/kda_gdr.h"

static std::mt19937_64 rng(5);
static int64_t below(int64_t n) { return (int64_t)(rng() % (uint64_t)n); }

static bool fail(const char *what, const kda::GdrArgs &a, const std::vector<int32_t> &cu) {
    printf("%s: T %lld, offsets", what, (long long)a.T);
    for (int32_t c : cu) printf(" %d", c);
    printf("\n");
    return false;
}

static bool check(int64_t T, const std::vector<int32_t> &cu) {
    constexpr int C = kda::GDR_C;
    kda::GdrArgs a{};
    a.T = T;
    a.N = (int)cu.size() - 1;
    a.cu = cu.data();
    a.slots = T / C + a.N;
    bool ordered = cu[0] >= 0 && cu[a.N] <= T;
    for (int n = 0; n < a.N; ++n) ordered = ordered && cu[n] <= cu[n + 1];
    std::vector<int> taken(a.slots, 0), seen(T, 0);
    int64_t row, len, slot, end = 0;
    for (int n = 0; n < a.N; ++n) {
        kda::gdr_sequence(a, n, row, len, slot);
        const int64_t chunks = (len + C - 1) / C;
        if (row < 0 || len < 0 || row + len > T || slot < 0 || (chunks > 0 && slot + chunks > a.slots)) return fail("a sequence out of range", a, cu);
        for (int64_t c = 0; c < chunks; ++c) {
            if (ordered && taken[slot + c]) return fail("a slot taken twice", a, cu);
            taken[slot + c] = 1;
        }
        end = row + len;
    }
    for (int64_t s = 0; s < a.slots; ++s) {
        int n;
        const bool there = kda::gdr_chunk(a, s, row, n);
        if (there && (row < 0 || n < 1 || n > C || row + n > T)) return fail("a chunk out of range", a, cu);
        if (ordered && there != (taken[s] != 0)) return fail("a chunk that is not found, or not there", a, cu);
        if (there && ordered)
            for (int i = 0; i < n; ++i) ++seen[row + i];
        // the rows behind the last sequence that this slot clears in the backward pass
        if (ordered)
            for (int64_t t = end + (a.slots - 1 - s) * C; t < end + (a.slots - s) * C && t < T; ++t) ++seen[t];
    }
    if (ordered)
        for (int64_t t = cu[0]; t < T; ++t)
            if (seen[t] != 1) return fail("a row that is not written once", a, cu);
    return true;
}

int main() {
    if (!check(6400, {0, 6400, 0, 6400}) || !check(64, {0, 64}) || !check(1, {0, 0})) return 1;
    for (int i = 0; i < 20000; ++i) {
        const int64_t T = 1 + below(i % 3 ? 200 : 3000);
        const int N = 1 + (int)below(i % 5 ? 6 : 80), kind = i % 4;
        std::vector<int32_t> cu(N + 1);
        for (auto &c : cu) c = kind == 3 ? (int32_t)rng() : kind == 2 ? (int32_t)(below(3 * T) - T) : (int32_t)below(T + 1);
        if (kind < 2) std::sort(cu.begin(), cu.end());
        if (kind == 0) cu[0] = 0;
        if (!check(T, cu)) return 1;
    }
    printf("ok\n");
    return 0;
}

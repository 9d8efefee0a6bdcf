// Host check of where sequences begin and end (struct Seqs of kda_rows.h): for any offsets every sequence's
// number and every row stay in range; for offsets in order the marks, the sequence of a row and its
// first row are those of a plain walk.
#include <cstdio>
#include <random>
#include <vector>

#include "../gated_delta_rule_31_amd/csrc/kda_rows.h"

static int fail(const char *what, int64_t t) {
    std::printf("%s at row %lld\n", what, (long long)t);
    return 1;
}

static int check(const kda::Seqs &s, const std::vector<int> &seq, const std::vector<int64_t> &begin, const std::vector<int64_t> &end, bool ordered) {
    const int64_t limit = s.limit();
    if (limit < 0 || limit > s.rows) return fail("limit", limit);
    for (int64_t t = 0; t < s.rows; ++t) {
        const int n = s.of(t);
        if (n < 0 || n >= s.N) return fail("sequence out of range", t);
        const int64_t b = s.begin(n, t);
        if (b < 0 || b > t) return fail("begin out of range", t);
        if (!ordered || t >= limit) continue;
        if (n != seq[t] || b != begin[t]) return fail("sequence", t);
    }
    for (int count : {1, 7, 8, 16, 35, 61, 64})
        for (int64_t t0 = 0; t0 < limit; t0 += count > 8 ? 5 : 1) {
            const int c = (int)(limit - t0 < count ? limit - t0 : count);
            uint64_t first, last;
            s.marks(t0, c, first, last);
            if (c < 64 && ((first | last) >> c)) return fail("mark behind the rows", t0);
            if (!ordered) continue;
            for (int u = 0; u < c; ++u) {
                const int64_t t = t0 + u;
                if ((first >> u & 1) != (uint64_t)(begin[t] == t)) return fail("first", t);
                if ((last >> u & 1) != (uint64_t)(end[t] == t + 1)) return fail("last", t);
            }
        }
    return 0;
}

int main() {
    std::mt19937 rng(5);
    for (int round = 0; round < 400; ++round) {
        const int N = 1 + rng() % 9;
        const bool packed = round % 2;
        std::vector<int64_t> lens(N);
        const int64_t T = 1 + rng() % 70;
        for (auto &l : lens) l = packed ? (rng() % 3 ? rng() % 60 : 0) : T;
        std::vector<int32_t> cu(N + 1, 0);
        for (int n = 0; n < N; ++n) cu[n + 1] = cu[n] + (int32_t)lens[n];
        const int64_t used = cu[N], rows = used + (packed ? rng() % 20 : 0);
        if (rows == 0) continue;
        std::vector<int> seq(rows, -1);
        std::vector<int64_t> begin(rows), end(rows);
        for (int n = 0; n < N; ++n)
            for (int64_t t = cu[n]; t < cu[n + 1]; ++t) {
                seq[t] = n;
                begin[t] = cu[n];
                end[t] = cu[n + 1];
            }
        kda::Seqs s{};
        s.T = T;
        s.rows = rows;
        s.N = N;
        s.cu = packed ? cu.data() : nullptr;
        if (check(s, seq, begin, end, true)) return 1;
        if (packed) {  // any numbers at all
            for (auto &c : cu) c = rng() % 4 ? (int32_t)(rng() % (rows + 10)) - 5 : (int32_t)rng();
            if (check(s, seq, begin, end, false)) return 1;
        }
    }
    std::puts("ok");
    return 0;
}

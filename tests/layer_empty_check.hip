// Host check of Seqs::marks (kda_rows.h) where very many sequences hold no row: the marks are those of a plain walk over the
// distinct offsets, and a lookup does not go through the empty sequences one by one.
#include <chrono>
#include <cstdio>
#include <random>
#include <vector>

#include "../gated_delta_rule_31_amd/csrc/kda_rows.h"

int main() {
    std::mt19937 rng(7);
    for (int round = 0; round < 60; ++round) {
        const int64_t rows = 200 + rng() % 300;
        std::vector<int32_t> cu{0};
        std::vector<char> at(rows + 1, 0);
        at[0] = 1;
        while (cu.back() < rows) {
            const int many = rng() % 3 ? rng() % 5 : round < 50 ? rng() % 3000 : 1 << 20;
            cu.insert(cu.end(), many, cu.back());
            const int32_t next = cu.back() + 1 + rng() % (round % 2 ? 12 : 150);
            cu.push_back(next < rows ? next : (int32_t)rows);
            at[cu.back()] = 1;
        }
        cu.insert(cu.end(), round < 50 ? rng() % 2000 : 1 << 20, (int32_t)rows);  // a batch padded to its largest count
        kda::Seqs s{};
        s.cu = cu.data();
        s.rows = rows;
        s.N = (int)cu.size() - 1;
        const auto begin = std::chrono::steady_clock::now();
        for (int again = 0; again < 20; ++again)
            for (int64_t t0 = 0; t0 < rows; ++t0) {
                const int count = (int)(rows - t0 < 64 ? rows - t0 : 64);
                uint64_t first, last, f = 0, l = 0;
                s.marks(t0, count, first, last);
                for (int u = 0; u < count; ++u) {
                    if (at[t0 + u]) f |= 1ull << u;
                    if (at[t0 + u + 1]) l |= 1ull << u;
                }
                if (f != first || l != last) {
                    std::printf("marks of row %lld\n", (long long)t0);
                    return 1;
                }
            }
        // up to 10000 lookups of at most 65 offsets and as many searches: far below a second; one by one, 10^10 steps
        if (std::chrono::steady_clock::now() - begin > std::chrono::seconds(2)) {
            std::puts("a lookup goes through the empty sequences one by one");
            return 1;
        }
    }
    std::puts("ok");
    return 0;
}

// Host check of how the gated linear recurrence joins stretches of tiles (join, both of kda_glr.h), in the order in
// which glr_carry_kernel does it: a group's tiles one after another, the groups of a wave by doubling distances, the
// waves in their order.  Words of one sequence that are not finite change no bit of the state in front of a tile of
// another, and are not forgotten in their own; finite ones give the state of a plain walk.
#include <cmath>
#include <cstdio>
#include <cstring>
#include <random>
#include <vector>

#include "../gated_delta_rule_31_amd/csrc/kda_glr.h"

struct Word {
    float a, h;
};

static std::vector<float> carry(const std::vector<Word> &w, int carry_c) {
    const int n = (int)w.size(), groups = 1024 / carry_c, in_wave = 64 / carry_c, each = (n + groups - 1) / groups;
    std::vector<float> A(groups, 1.f), H(groups, 0.f), front(n);
    auto lo = [&](int g) { return g * each < n ? g * each : n; };
    for (int g = 0; g < groups; ++g)
        for (int at = lo(g); at < lo(g + 1); ++at) {
            H[g] = kda::join(w[at].a, w[at].h, H[g]);
            A[g] = kda::both(A[g], w[at].a);
        }
    for (int d = 1; d < in_wave; d *= 2) {
        const std::vector<float> pa = A, ph = H;
        for (int g = 0; g < groups; ++g)
            if (g % in_wave >= d) {
                H[g] = kda::join(A[g], H[g], ph[g - d]);
                A[g] = kda::both(A[g], pa[g - d]);
            }
    }
    for (int g = 0; g < groups; ++g) {
        float x = 0.f;
        for (int v = 0; v < g / in_wave; ++v) x = kda::join(A[v * in_wave + in_wave - 1], H[v * in_wave + in_wave - 1], x);
        if (g % in_wave) x = kda::join(A[g - 1], H[g - 1], x);
        for (int at = lo(g); at < lo(g + 1); ++at) {
            front[at] = x;
            x = kda::join(w[at].a, w[at].h, x);
        }
    }
    return front;
}

static int fail(const char *what, int at, int round) {
    std::printf("%s, tile %d of round %d\n", what, at, round);
    return 1;
}

int main() {
    const float inf = INFINITY, nan = NAN;
    std::mt19937 rng(3);
    auto unit = [&] { return (float)(rng() >> 8) / (1 << 24); };
    for (int round = 0; round < 4000; ++round) {
        const int n = 17 + rng() % (round % 4 ? 120 : 6000), carry_c = round % 2 ? 4 : 16;
        const int per = 1 + rng() % (round % 3 ? 6 : 300);  // tiles between two that hold a beginning
        std::vector<Word> good(n);
        std::vector<int> seq(n);  // the sequence that the state in front of a tile belongs to
        int s = 0;
        for (int t = 0; t < n; ++t) {
            const bool cut = rng() % per == 0;
            good[t] = {cut ? kda::CUT : rng() % 9 ? unit() : 0.f, 2 * unit() - 1};
            seq[t] = s;
            s += cut;
        }
        const std::vector<float> want = carry(good, carry_c);
        double x = 0, size = 1;
        for (int t = 0; t < n; ++t) {
            // every join rounds once, and a state is at most the sum of what its tiles add
            if (std::fabs(want[t] - x) > 64 * size * 6e-8) return fail("state", t, round);
            const bool cut = kda::is_cut(good[t].a);
            x = cut ? good[t].h : (double)good[t].a * x + good[t].h;
            size = 1 + (cut ? 0 : good[t].a * size);
        }
        const int bad = rng() % (s + 1), kind = rng() % 4;
        std::vector<Word> w = good;
        bool any = false;
        for (int t = 0; t < n; ++t) {
            // tiles in which the bad sequence alone has rows behind the last beginning
            const bool behind = kda::is_cut(w[t].a) ? seq[t] + 1 == bad : seq[t] == bad;
            if (!behind || (any && rng() % 3)) continue;
            any = true;
            if (kind == 0) w[t] = {nan, nan};                                       // a gate
            else if (kind == 1) w[t].h = inf;                                       // an input
            else if (kind == 2) w[t].h = rng() % 2 ? nan : -inf;
            else if (t == 0 || kda::is_cut(w[t].a)) w[t].h = rng() % 2 ? inf : nan;  // an initial state, seen at the beginning alone
        }
        const std::vector<float> got = carry(w, carry_c);
        float plain = 0.f;
        for (int t = 0; t < n; ++t) {
            if (seq[t] != bad) {
                if (std::memcmp(&got[t], &want[t], 4)) return fail("another sequence", t, round);
            } else if (!std::isfinite(plain) && std::isfinite(got[t])) {
                return fail("forgotten", t, round);
            }
            plain = kda::join(w[t].a, w[t].h, plain);
        }
    }
    // minus zero beside everything
    for (float v : {1.f, 0.f, kda::CUT, inf, nan, -nan, 1e-40f})
        if (!kda::is_cut(kda::both(kda::CUT, v)) || !kda::is_cut(kda::both(v, kda::CUT))) return fail("both", 0, 0);
    if (kda::is_cut(kda::both(1e-30f, 1e-30f)) || kda::is_cut(kda::both(0.f, 1.f))) return fail("an underflow counts as a cut", 0, 0);
    std::puts("ok");
    return 0;
}

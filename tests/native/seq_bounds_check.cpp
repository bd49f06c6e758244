// The device functions that look up sequence bounds and slots (cut out of the kernels' sources into seq_bounds.inc),
// on bounds and slots outside their contract: whatever those hold, the places that the kernels index with
// stay inside the tensors, and every search ends.
#include <stdio.h>

#include <algorithm>
#include <random>
#include <vector>

#define __device__
#define __forceinline__ inline
using std::max;
using std::min;
struct SeqAxis {
    int S, T, L;
    const int* starts;
};
struct SeqSlots {
    const int* slots;
    long long count;
};
#include "seq_bounds.inc"

static long long bad = 0, checked = 0;
#define CHECK(c)                                                   \
    do {                                                           \
        ++checked;                                                 \
        if (!(c) && ++bad < 10) printf("%s: S %d T %d\n", #c, ax.S, ax.T); \
    } while (0)

int main() {
    std::mt19937_64 rng(1);
    auto below = [&](long long n) { return (long long)(rng() % (unsigned long long)n); };
    for (int round = 0; round < 40000; ++round) {
        const int S = 1 + (int)below(round % 3 ? 12 : 70), T = (int)below(90);
        std::vector<int> v(S + 1), slots(S);
        const int kind = (int)below(6);
        for (int i = 0; i <= S; ++i) {
            if (kind == 0) v[i] = (int)below(T + 1);                              // in range, in any order
            else if (kind == 1) v[i] = (int)below(2 * T + 3) - T / 2 - 1;           // before and behind the axis
            else if (kind == 2) v[i] = (int)rng();                                // anything
            else v[i] = i * T / S + (int)below(5) - 2;                            // nearly right
        }
        if (kind >= 4) std::sort(v.begin(), v.end());
        if (kind == 5) v[0] = 0;                                                   // (the end may still be wrong)
        for (int& s : slots) s = kind == 2 ? (int)rng() : (int)below(2 * S) - S / 2;
        const SeqAxis ax = {S, T, 0, v.data()};
        for (int t = 0; t < T; ++t) {
            Place q = place_of(ax, t);                     // convolution: the sequence of a run's first token,
            CHECK(q.s >= -1 && q.s < S && q.begin >= 0 && q.begin <= t && q.end > t && q.end <= T);
            for (int at = q.end, n = 0; at < T; at = q.end, ++n) {                  // and those that follow
                next_place(ax, at, q);
                CHECK(q.s >= 0 && q.s < S && q.begin == at && q.end > at && q.end <= T);
                if (q.end <= at || n > T) return 1;
            }
            const ScanPlace r = scan_place(ax, t);
            CHECK(r.s >= -1 && r.s < S && r.begin >= 0 && r.begin <= t && r.end > t && r.end <= T);
            const int f = seq_first_at(ax, t);
            CHECK(f >= 0 && f <= S);
            CHECK(seq_start(ax, f, t) >= t && seq_start(ax, f, t) <= T);
            const int g = seq_first_at(ax, t + 1);
            CHECK(min(t + 8, seq_start(ax, g, t + 1)) > t);                         // the tokens that a piece sends back
        }
        const SeqSlots sl = {slots.data(), (long long)S};
        for (int s = -1; s < S; ++s) {
            const long long slot = seq_slot(sl, s);
            CHECK(slot >= -1 && slot < S);
            if (s < 0) continue;
            const int begin = seq_start(ax, s, 0), end = seq_start(ax, s + 1, begin);
            CHECK(0 <= begin && begin <= end && end <= T);                         // the states left
        }
        CHECK(seq_start(ax, S, 0) == T);
    }
    printf("%lld checks, %lld wrong\n", checked, bad);
    return bad != 0;
}

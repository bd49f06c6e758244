// Where the delta rule's walks over pieces of the axis stand (cut_piece, mark_piece and walk_place, cut out of their sources into
// delta_place.inc).  With bounds in their contract: every piece that another of its sequence follows has one block that walks it first, a place of
// its own in what is kept by mark, and the second walks and the joining look it up there; every token is walked once.  With any bounds:
// nothing leads outside the tensors or what is kept.
#include <stdint.h>
#include <stdio.h>

#include <algorithm>
#include <random>
#include <set>
#include <vector>

#define __host__
#define __device__
#define __forceinline__ inline
using std::max;
using std::min;
struct {
    unsigned x;
} blockIdx;
struct SeqAxis {
    int S, T, L;
    const int* starts;
};
enum { DELTA_WHOLE = 0, DELTA_PIECES = 1, DELTA_JOINED = 2 };
constexpr int DELTA_CHUNK = 64, DC = DELTA_CHUNK;
struct SeqDeltaParams {
    SeqAxis ax;
    int Hv, run, pieces, marks;
};
#include "delta_place.inc"

static long long bad = 0, checked = 0;
#define CHECK(c)                                                                           \
    do {                                                                                   \
        ++checked;                                                                         \
        if (!(c) && ++bad < 10) printf("%s: S %d T %d L %d run %d\n", #c, p.ax.S, p.ax.T, p.ax.L, p.run); \
    } while (0)

int main() {
    std::mt19937_64 rng(1);
    auto below = [&](long long n) { return (long long)(rng() % (unsigned long long)n); };
    for (int round = 0; round < 300; ++round) {
        const int S = 1 + (int)below(round % 3 ? 9 : 60), kind = (int)below(5);
        int T = (int)below(round % 8 ? 2500 : 6000);
        std::vector<int> v(S + 1);
        SeqDeltaParams p = {};
        if (kind == 4) {                                   // equal lengths
            T = S * (1 + (int)below(900));
            p.ax = {S, T, T / S, nullptr};
            for (int i = 0; i <= S; ++i) v[i] = i * (T / S);
        } else {
            for (int i = 0; i <= S; ++i)
                v[i] = kind == 0 ? (int)rng() : kind == 1 ? (int)below(2 * T + 3) - T / 2 : (int)below(T + 1);
            if (kind >= 2) {
                std::sort(v.begin(), v.end());
                v[0] = 0;
                v[S] = T;
            }
            p.ax = {S, T, 0, v.data()};
        }
        const bool good = kind >= 2;
        p.Hv = 1;
        p.run = 1 + (int)below(12);
        const int len = p.run * DC;
        p.marks = (int)delta_marks(T, p.run);
        p.pieces = (int)cut_slots(S, T, p.ax.L, len);
        const long long slots = cut_slots(S, T, p.ax.L, DC);
        std::set<std::pair<int, int>> walked;              // sequence, first token
        std::vector<std::pair<int, int>> at(p.marks, {-1, -1});
        auto inside = [&](const WalkPlace& w) {
            return w.seq >= 0 && w.seq < S && w.t0 >= 0 && w.t1 >= w.t0 && w.t1 <= T && w.slot0 >= 0 && w.slot0 + w.chunks <= slots;
        };
        for (int b = 0; b < 2 * p.marks; ++b) {            // columns of values, and of the unit matrix
            blockIdx.x = (unsigned)b;
            const WalkPlace w = walk_place<DELTA_PIECES>(p, 1, 1);
            if (w.none) continue;
            CHECK(inside(w) && w.mark >= 0 && w.mark < p.marks && w.t1 - w.t0 == len);
            if (w.unit) {
                CHECK(!w.first);
                continue;
            }
            if (good) {
                CHECK(walked.insert({w.seq, w.t0}).second && w.mark == first_mark(v[w.seq], len) + (w.t0 - v[w.seq]) / len);
                at[w.mark] = {w.seq, w.t0};
            }
        }
        std::vector<int> seen(T, 0), states(S, 0);
        for (int b = 0; b < p.pieces; ++b) {
            blockIdx.x = (unsigned)b;
            const WalkPlace w = walk_place<DELTA_JOINED>(p, 1, 0);
            if (w.none) continue;
            CHECK(inside(w));
            const bool kept = !(w.first && w.last);
            if (kept) CHECK(w.mark >= 0 && w.mark < p.marks);
            if (!good) continue;
            for (int t = w.t0; t < w.t1; ++t) ++seen[t];
            if (w.last) ++states[w.seq];
            if (kept) CHECK(at[w.mark].first == w.seq && at[w.mark].second == (w.first ? w.t0 : w.t0 - len));
        }
        if (!good) continue;
        for (int t = 0; t < T; ++t) CHECK(seen[t] == 1);
        long long whole = 0;
        for (int s = 0; s < S; ++s) {
            CHECK(states[s] == 1);
            const int n = (v[s + 1] - v[s] + len - 1) / len;
            for (int i = 0; i < n - 1; ++i, ++whole) CHECK(walked.count({s, v[s] + i * len}));
        }
        CHECK((long long)walked.size() == whole);
        // the joining: by sequences, or by the marks of first pieces
        std::vector<int> joins(S, 0);
        for (long long b = 0; b < delta_joined(S, p.marks); ++b) {
            int s = (int)b;
            if (S > p.marks) {
                const MarkPiece c = mark_piece(p.ax, (int)b, len);
                CHECK(c.s >= 0 && c.s < S);
                if (c.index > 0) continue;
                s = c.s;
            }
            if (v[s + 1] - v[s] > len) ++joins[s];
        }
        for (int s = 0; s < S; ++s) CHECK(joins[s] == (v[s + 1] - v[s] > len));
    }
    printf("%lld checks, %lld wrong\n", checked, bad);
    return bad != 0;
}

// Which group norm calls let every block join its groups' entries itself (gn_shape and gn_self, cut out of their source into
// gnorm_join.inc): never more entries than a block's threads take a few each of, however the tokens lie in the sequences.
#include <stdio.h>

#include <initializer_list>

struct SeqAxis {
    int S, T, L;
};
struct SeqGnormParams {
    SeqAxis ax;
    int D, G, slab;
};
#include "gnorm_join.inc"

int main() {
    long long wrong = 0, cases = 0, self = 0;
    for (int S : {1, 2, 7, 150, 20000})
        for (int T : {100, 5003, 70000, 2000000})
            for (int D : {1, 32, 64, 512, 770, 4096})
                for (int G : {1, 2, 8, 32})
                    for (int slab : {16, 32, 200, 1024})
                        for (int V : {1, 2, 4, 8})
                            for (bool known : {false, true}) {
                                if (D % G || (known && T % S)) continue;
                                const SeqGnormParams p = {{S, T, known ? T / S : 0}, D, G, slab};
                                const GnShape s = gn_shape(D, D / G, V);
                                const long long longest = known ? T / S : T;      // all tokens may be one sequence's
                                const long long entries = (longest + slab - 1) / slab * (s.tx * V / (D / G));
                                ++cases;
                                if (gn_self(p, s, V)) {
                                    ++self;
                                    if (entries > 16 * GT) ++wrong;
                                }
                            }
    printf("%lld cases, %lld by themselves, %lld wrong\n", cases, self, wrong);
    return wrong != 0 || self == 0;
}

// What the delta rule's walks wait for before they give shared memory and TMEM back (struct Turns and settle, cut out of their
// sources into delta_settle.inc), on barriers whose phases complete some time later or never: nothing that was issued is on
// its way when they return, unless the limit has passed.
#include <stdint.h>
#include <stdio.h>

#include <random>

#define __device__
#define __forceinline__ inline
static void tc_fence_after() {}
static void tc_fence_before() {}
static void tmem_st_wait() {}
static void __syncwarp() {}
static void arrive_once(uint32_t) {}

// Three barriers: the copies of two stages (addresses 0 and 8) and the products (16).  Phase i of one completes at done[.][i].
static long long now;
static int begun[3];
static long long done[3][64];
static int completed(int b) {
    int n = 0;
    while (n < begun[b] && done[b][n] <= now) ++n;
    return n;
}
static bool mbar_try_wait(uint32_t bar, uint32_t parity) { return (completed(bar / 8) & 1) != (int)parity; }
static long long clock64() { return now += 20000; }
static bool wait_turn(uint32_t, uint32_t, volatile int*, unsigned*) { return true; }

#include "delta_settle.inc"

int main() {
    std::mt19937 rng(5);
    int wrong = 0, cases = 0;
    for (int round = 0; round < 2000; ++round) {
        const int sent = (int)(rng() % 20), products = (int)(rng() % 40);
        now = 0;
        begun[0] = (sent + 1) / 2;
        begun[1] = sent / 2;
        begun[2] = products;
        for (int b = 0; b < 3; ++b)              // all but the last are done; the last some time later, or never
            for (int i = 0; i < begun[b]; ++i) done[b][i] = i < begun[b] - 1 ? 0 : round % 10 == 9 ? (1ll << 60) : (long long)(rng() % 50000000);
        volatile int abort_flag = round & 1;
        Turns t = {};
        t.mma = 16;
        t.full = 0;
        t.abort_flag = &abort_flag;
        const long long from = now;
        t.settle_copies(sent);
        t.settle_products(products);
        const long long took = now - from;
        ++cases;
        const bool all = completed(0) == begun[0] && completed(1) == begun[1] && completed(2) == begun[2];
        const int open = (begun[0] > 0) + (begun[1] > 0) + (begun[2] > 0);
        if (round % 10 == 9 ? took > open * (WAIT_CYCLES + 40000) : !all || took > 3 * 60000000) ++wrong;
    }
    printf("%d cases, %d wrong\n", cases, wrong);
    return wrong != 0;
}

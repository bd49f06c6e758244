// The waits of the delta rule's tensor-core kernels (cut out of their sources into delta_wait.inc), run by 32 threads as the
// lanes of a warp.  Lanes need not see a barrier's phase at the same look: whatever each of them sees, all leave a wait together
// with one answer, and no vote is left waiting for a lane that has gone on.
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include <atomic>
#include <condition_variable>
#include <mutex>
#include <random>
#include <thread>
#include <vector>

#define __device__
#define __forceinline__ inline
enum : unsigned { ERR_WAIT_TIMEOUT = 1u };

constexpr int LANES = 32;
static thread_local int lane;
static std::vector<int> sees(LANES);        // the look of each lane that first sees the phase (-1: none does)
static std::vector<int> looks(LANES);
static std::vector<long long> now(LANES), tick(LANES);

// A meeting of all lanes.  `place` tells the warp's instructions apart: lanes that meet at different ones have split.
static std::mutex m;
static std::condition_variable cv;
static int met, open_place, round_;
static bool all_of, any_of, all_was, any_was;
[[noreturn]] static void split(const char* why) {
    printf("the warp split: %s\n", why);
    fflush(stdout);
    _Exit(1);
}
static void meet(int place, bool pred, bool& all, bool& any) {
    std::unique_lock<std::mutex> l(m);
    if (met == 0) {
        open_place = place;
        all_of = true;
        any_of = false;
    } else if (open_place != place) {
        split("lanes at different instructions");
    }
    all_of = all_of && pred;
    any_of = any_of || pred;
    const int mine = round_;
    if (++met == LANES) {
        met = 0;
        ++round_;
        all_was = all_of;
        any_was = any_of;
        cv.notify_all();
    } else if (!cv.wait_for(l, std::chrono::seconds(20), [&] { return round_ != mine; })) {
        split("a lane did not come");
    }
    all = all_was;
    any = any_was;
}
static int __all_sync(unsigned, int pred) {
    bool all, any;
    meet(1, pred != 0, all, any);
    return all;
}
static int __any_sync(unsigned, int pred) {
    bool all, any;
    meet(2, pred != 0, all, any);
    return any;
}
static bool mbar_try_wait(uint32_t, uint32_t) { return sees[lane] >= 0 && looks[lane]++ >= sees[lane]; }
static long long clock64() { return now[lane] += tick[lane]; }
static std::atomic<unsigned> error_word;
static void atomicOr(unsigned*, unsigned v) { error_word |= v; }

#include "delta_wait.inc"

int main() {
    std::mt19937 rng(3);
    int wrong = 0, cases = 0;
    for (int kind = 0; kind < 60; ++kind) {
        volatile int abort_flag = kind % 6 == 5;
        error_word = 0;
        const bool never = kind % 6 >= 4;
        for (int i = 0; i < LANES; ++i) {
            looks[i] = 0;
            now[i] = (long long)(rng() % 1000);
            tick[i] = never ? WAIT_CYCLES / 7 + (long long)(rng() % 1000000) : 30;
            sees[i] = never                ? (kind % 12 >= 10 ? -1 : (i == 3 ? 0 : -1))      // no lane, or one alone
                      : kind % 6 == 0      ? 0
                      : kind % 6 == 1      ? (i == 5 ? 1 : 0)
                      : kind % 6 == 2      ? (i == 5 ? 0 : 2)
                                           : (int)(rng() % 9);
        }
        std::vector<int> got(LANES, -1);
        std::vector<std::thread> t;
        unsigned err = 0;
        for (int i = 0; i < LANES; ++i)
            t.emplace_back([&, i] {
                lane = i;
                got[i] = wait_turn(0, 0, &abort_flag, &err);
                bool all, any;
                meet(3, true, all, any);               // the warp's next instruction
            });
        for (auto& x : t) x.join();
        for (int i = 0; i < LANES; ++i) {
            ++cases;
            if (got[i] != !never) ++wrong;
            if (!never && looks[i] <= sees[i]) ++wrong;  // it went on before it saw the phase
        }
        if (never && (!abort_flag || error_word != ERR_WAIT_TIMEOUT)) ++wrong;
        if (!never && (abort_flag || error_word)) ++wrong;
    }
    printf("%d answers, %d wrong\n", cases, wrong);
    return wrong != 0;
}

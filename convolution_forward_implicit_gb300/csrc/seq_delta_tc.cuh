// What the tcgen05 kernels of the gated delta rule share: K and Q in shared memory, descriptors, bounded waits.
#pragma once
#include "seq_delta.cuh"
#include "tc_common.cuh"

namespace convfwd {
namespace {

constexpr uint32_t ATOM = 128 * 128;          // 128 rows of 64 bf16
__device__ __forceinline__ uint64_t mn_desc(uint32_t saddr, uint32_t stride) {     // N side by side, blocks of 64 `stride` bytes apart
    uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)((stride >> 4) & 0x3FFFu) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}
// A wait of a converged warp for a barrier's phase, for about a second at most.  The limit goes by the SM's clock: reading the global
// timer between two looks costs more than a hand-off takes (8192 tokens, 32 heads of 128 x 128: the forward walk then took 449 us with it, 249 without).
constexpr long long WAIT_CYCLES = 2000000000ll;
// Every lane looks, and what follows is the warp's decision: lanes that look at once need not see the same, and one that went on
// alone would leave the others in a vote that it never joins.  The arrivals below are predicated: a branch that only one lane takes costs a few
// hundred cycles at each hand-off until its warp is together again (2048 x 16 heads: 233 us with them, 184 with the waits alone changed).
__device__ __forceinline__ bool wait_turn(uint32_t bar, uint32_t parity, volatile int* abort_flag, unsigned* err) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    const long long since = clock64();
    while (!__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) {
        if (__any_sync(0xffffffffu, *abort_flag != 0 || clock64() - since > WAIT_CYCLES)) {
            *abort_flag = 1;
            atomicOr(err, ERR_WAIT_TIMEOUT);
            return false;
        }
    }
    return true;
}
// By the one thread that issued copies or products, before it ends: the phase that the last of them complete, for about a second
// at most.  Shared memory and TMEM are then given back with nothing of its own on the way, also after a wait has run out.
__device__ __forceinline__ void settle(uint32_t bar, uint32_t parity) {
    const long long since = clock64();
    while (!mbar_try_wait(bar, parity) && clock64() - since < WAIT_CYCLES) {
    }
}
__device__ __forceinline__ void arrive_once(uint32_t bar) {       // one arrival of a converged warp
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];\n\t}" ::"r"(bar)
        : "memory");
}

// K and Q rows of a chunk to [K; Q] atoms in the 128-byte swizzle; rows at and behind n and columns behind the width are zero.
template <int KP, int THREADS>
__device__ __forceinline__ void load_kq(uint32_t to, const __nv_bfloat16* k, const __nv_bfloat16* q, long long k_ld, long long q_ld, int n, int width, int thread) {
    constexpr int CPR = KP / 8;                  // 16-byte pieces of a row
    for (int i = thread; i < 128 * CPR; i += THREADS) {
        const int row = i / CPR, c = i % CPR, r = row & 63;
        const bool there = r < n && c * 8 < width;
        const __nv_bfloat16* from = row < 64 ? k : q;
        const uint32_t step = (uint32_t)(row < 64 ? k_ld : q_ld);
        cp_async_16(to + (uint32_t)(c / 8) * ATOM + row * 128 + ((c % 8) ^ (row & 7)) * 16, there ? from + r * step + c * 8 : from, there ? 16 : 0);
    }
}

}  // namespace
}  // namespace convfwd

// What the kernels of the selective scan share: how states lie on threads, the sequence bounds
// inside a tile of tokens, and the layout of saved states.
#pragma once
#include "seq_common.cuh"
#include "seq_internal.h"

namespace convfwd {

// Saved and carried states: [row][quad of states][channel][4], so that neighbouring channels of a
// warp store neighbouring 16 bytes.
__device__ __forceinline__ long long scan_state_at(const SeqScanParams& p, long long row, int quad, int d) {
    return ((row * ((p.N + 3) >> 2) + quad) * p.D + d) * 4;
}

// Where sequences begin and end among the tokens t0 .. t0 + n - 1 of a tile: bit i of `first`
// (`last`) is set when token t0 + i is the first (last) of its sequence, seq[i].
struct ScanBounds {
    unsigned first, last;
    int seq[SCAN_TILE];
};
// Called by one whole warp.
__device__ __forceinline__ void scan_bounds(const SeqAxis& ax, int t0, int n, ScanBounds* out) {
    const int i = threadIdx.x & 31;
    bool f = false, l = false;
    if (i < n) {
        const int t = t0 + i;
        const int s = seq_first_at(ax, t + 1) - 1;
        f = s >= 0 && seq_start(ax, s, 0) == t;
        l = s >= 0 && seq_start(ax, s + 1, t + 1) == t + 1;
        out->seq[i] = s;
    }
    const unsigned mf = __ballot_sync(~0u, f), ml = __ballot_sync(~0u, l);
    if (i == 0) {
        out->first = mf;
        out->last = ml;
    }
}

// The states (d, n0 .. n0 + NPT - 1) of a row of h_in / h_out: D x N fp32 values.
template <int NPT>
__device__ __forceinline__ void scan_h_load(const SeqScanParams& p, const float* h, long long slot, int d, int n0, float (&v)[NPT]) {
#pragma unroll
    for (int k = 0; k < NPT; ++k) v[k] = h && slot >= 0 && n0 + k < p.N ? h[(slot * p.D + d) * p.N + n0 + k] : 0.f;
}
template <int NPT>
__device__ __forceinline__ void scan_h_store(const SeqScanParams& p, float* h, long long slot, int d, int n0, const float (&v)[NPT]) {
    if (!h || slot < 0) return;
#pragma unroll
    for (int k = 0; k < NPT; ++k)
        if (n0 + k < p.N) h[(slot * p.D + d) * p.N + n0 + k] = v[k];
}

}  // namespace convfwd

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

// The sequence at hand while a block walks the tokens of a piece, in either direction.  Every thread
// holds the same values.
struct ScanPlace {
    int s, begin, end;
};
__device__ __forceinline__ ScanPlace scan_place(const SeqAxis& ax, int t) {
    ScanPlace q;
    q.s = seq_first_at(ax, t + 1) - 1;       // the last sequence that starts at or before t
    q.begin = q.s < 0 ? 0 : seq_start(ax, q.s, 0);
    q.end = seq_start(ax, q.s + 1, t + 1);
    return q;
}
// Where sequences begin and end among the tokens t0 .. t0 + n - 1 of a tile: bit i of `first`
// (`last`) is set when token t0 + i is the first (last) of its sequence.  Most tiles lie within the
// sequence at hand and need no look at the bounds.
struct ScanMarks {
    unsigned first, last;
};
__device__ __forceinline__ ScanMarks scan_marks(const SeqAxis& ax, int t0, int n, ScanPlace& q) {
    ScanMarks m = {0u, 0u};
    if (t0 < q.begin || t0 >= q.end) q = scan_place(ax, t0);
    if (q.s >= 0 && q.begin == t0) m.first = 1u;
    if (t0 + n <= q.end) {
        if (q.s >= 0 && t0 + n == q.end) m.last = 1u << (n - 1);
        return m;
    }
    const int lane = threadIdx.x & 31;
    bool f = false, l = false;
    if (lane < n) {
        const ScanPlace r = scan_place(ax, t0 + lane);
        f = r.s >= 0 && r.begin == t0 + lane;
        l = r.s >= 0 && r.end == t0 + lane + 1;
    }
    m.first = __ballot_sync(~0u, f);
    m.last = __ballot_sync(~0u, l);
    return m;
}
// The slot of the sequence that token t belongs to.
__device__ __forceinline__ long long scan_slot(const SeqAxis& ax, const SeqSlots& sl, int t, const ScanPlace& q) {
    return seq_slot(sl, t >= q.begin && t < q.end ? q.s : seq_first_at(ax, t + 1) - 1);
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

// Packed fp32 pairs.  The compiler's own f32x2 operations on float2 keep a loop's values in place;
// the same instructions written as asm on 64-bit values cost a register move for each value carried
// from one token to the next (measured: 66 moves a token in the backward kernel).
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 sum2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 dup2(float a) { return make_float2(a, a); }
__device__ __forceinline__ float2 exp2_2(float2 v) { return make_float2(ex2_approx(v.x), ex2_approx(v.y)); }
// exp(delta A) of two states or channels, with A2 = A log2(e).  The special-function unit's 2^v lies low on
// average (measured over 1 M values an octave: 5e-9 to 1e-8 for |v| of 2^-9 to 2^-21, 2.7e-8 at 2^-7 and 2^-6, 5e-8 from
// 1 on), and a state multiplies about 1 / |v| such factors.  An offset of 1.5e-8 in the argument, where it costs nothing, leaves
// +5e-9 to 0 of it up to 2^-9, whose many factors add up most (2e-5 of a state after 4096 tokens; with 2.3e-8 +1e-8 a
// factor and 4e-5, with 1e-8 +2e-9), and -1.6e-8 at 2^-7 (2.3e-8: -1e-8, 1e-8: -1.9e-8).  (2^1.5e-8 is 1 in fp32: delta = 0 still changes nothing.)
__device__ __forceinline__ float2 decay2(float2 delta, float2 A2) { return exp2_2(fma2(delta, A2, dup2(1.5e-8f))); }
__device__ __forceinline__ void unpack(float2 v, float& a, float& b) {
    a = v.x;
    b = v.y;
}
// Two pairs from 16 bytes.
__device__ __forceinline__ void ld2(const float* p, float2& a, float2& b) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    a = make_float2(v.x, v.y);
    b = make_float2(v.z, v.w);
}
__device__ __forceinline__ void st2(float* p, float2 a, float2 b) { *reinterpret_cast<float4*>(p) = make_float4(a.x, a.y, b.x, b.y); }

// A2 = A log2(e) of states n0 .. n0 + NPT - 1 of channel d, as pairs; zero behind the last state.  Rows of
// whole aligned quads are read 16 bytes at a time.
template <int NPT>
__device__ __forceinline__ void scan_decays(const SeqScanParams& p, int d, int n0, float2 (&A2)[NPT / 2]) {
    const float* A = p.A + (long long)d * p.N + n0;
#pragma unroll
    for (int k = 0; k < NPT / 2; k += 2) {
        float4 q = make_float4(0.f, 0.f, 0.f, 0.f);
        if (p.quads) {
            if (n0 + 2 * k < p.N) q = *reinterpret_cast<const float4*>(A + 2 * k);
        } else {
            if (n0 + 2 * k < p.N) q.x = A[2 * k];
            if (n0 + 2 * k + 1 < p.N) q.y = A[2 * k + 1];
            if (n0 + 2 * k + 2 < p.N) q.z = A[2 * k + 2];
            if (n0 + 2 * k + 3 < p.N) q.w = A[2 * k + 3];
        }
        A2[k] = mul2(make_float2(q.x, q.y), dup2(LOG2E));
        A2[k + 1] = mul2(make_float2(q.z, q.w), dup2(LOG2E));
    }
}

}  // namespace convfwd

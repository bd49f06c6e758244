// What the kernels of the gated delta rule share: matrix products of a chunk on tensor cores, its rows in
// shared memory, and the factors of its rows.
//
// A chunk of C = 64 tokens, b_i the sum of g up to token i of the chunk, E_ij = exp(b_i - b_j), k and q
// normalised if wanted, h0 the state before it:
//   L_ij = beta_i E_ij k_i.k_j (j < i)      T = (I + L)^-1
//   A_ij = scale E_ij q_i.k_j  (j <= i)
//   R = beta (V - exp(b) K h0)              U = T R
//   Y = scale exp(b) Q h0 + A U             h = exp(b_C) h0 + (exp(b_C - b) K)^T U
// q and k stay as they came, as operands: all factors of a row (lengths, decay, beta, scale) go with the other operand or
// the result, so that bf16 rows are exact in a tf32 product.
#pragma once
#include "delta.h"
#include "seq_common.cuh"
#include "seq_internal.h"

namespace convfwd {

constexpr int DC = DELTA_CHUNK;
constexpr int DT = 256;              // threads of the chunk kernels
constexpr float QK_EPS = 1e-6f;

__device__ __forceinline__ void dep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void dep_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// ---- products ----
// Matrix products on mma.sync m16n8k8 (tf32 operands, fp32 sums).  An fp32 operand is two tf32 ones, hi = x rounded
// to 11 bits and lo = x - hi (read with 11 bits of its own): hi hi + hi lo + lo hi leaves 2^-22 of a product, about
// what fp32 products leave; an operand that holds bf16 values is exact in hi alone.  A product's k index is free
// to run in any order that both operands share: slots t and t + 4 of a step are columns 2t and 2t + 1, so that an
// operand whose k lies side by side is read in pairs.
__device__ __forceinline__ uint32_t tf32_of(float x) {
    uint32_t r;
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ void mma8(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// Operands in shared memory: the values of row (or column) i at k and k + 1, k even.
template <typename T>
struct Along {                       // k lies side by side: element (i, k) at p[i ld + k]
    const T* p;
    int ld;
    static constexpr bool EXACT = sizeof(T) == 2;
    __device__ __forceinline__ float2 get(int i, int k) const { return seq_ld2(p + i * ld + k); }
};
template <typename T>
struct Across {                      // element (i, k) at p[k ld + i]
    const T* p;
    int ld;
    static constexpr bool EXACT = sizeof(T) == 2;
    __device__ __forceinline__ float2 get(int i, int k) const { return make_float2(seq_ld(p + k * ld + i), seq_ld(p + (k + 1) * ld + i)); }
};
struct AcrossScaled {                // element (i, k) at p[k ld + i] times f[k]
    const float* p;
    int ld;
    const float* f;
    static constexpr bool EXACT = false;
    __device__ __forceinline__ float2 get(int i, int k) const {
        const float2 s = *reinterpret_cast<const float2*>(f + k);
        return make_float2(p[k * ld + i] * s.x, p[(k + 1) * ld + i] * s.y);
    }
};

template <bool EXACT, int N>
__device__ __forceinline__ void split(const float (&x)[N], uint32_t (&hi)[N], uint32_t (&lo)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        hi[i] = EXACT ? __float_as_uint(x[i]) : tf32_of(x[i]);
        lo[i] = EXACT ? 0u : __float_as_uint(x[i] - __uint_as_float(hi[i]));
    }
}

// acc += a b for rows m0 .. m0 + 15 of a and columns n0 .. n0 + 8 NT - 1 of b, k from k0 to k1, by one warp.  Lane
// (g, t) = (lane / 4, lane % 4) holds rows g and g + 8, columns 2t and 2t + 1 of each 8: acc[.][0, 1] and [2, 3].
// The instruction cuts its sums instead of rounding them, so the products with low parts have sums of their own: with one sum for all
// three, gradients were off by 1 to 2.8e-6 instead of 5 to 9e-7 (300 tokens, 128 x 128), and the fp32 prompt of 5003 tokens (6 heads of 48 x 80) took 254 us
// instead of 243.  A fresh sum each step added in fp32 is off by 2 to 5e-7, but takes 281 us.
template <int NT, typename A, typename B>
__device__ __forceinline__ void warp_mma(float (&acc)[NT][4], const A& a, const B& b, int m0, int n0, int k0, int k1) {
    const int g = (threadIdx.x & 31) >> 2, t2 = (threadIdx.x & 3) * 2;
    float low[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) low[n][0] = low[n][1] = low[n][2] = low[n][3] = 0.f;
#pragma unroll 4
    for (int k = k0; k < k1; k += 8) {
        const float2 r0 = a.get(m0 + g, k + t2), r1 = a.get(m0 + g + 8, k + t2);
        const float av[4] = {r0.x, r1.x, r0.y, r1.y};
        uint32_t ah[4], al[4];
        split<A::EXACT>(av, ah, al);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float2 c = b.get(n0 + 8 * n + g, k + t2);
            const float bv[2] = {c.x, c.y};
            uint32_t bh[2], bl[2];
            split<B::EXACT>(bv, bh, bl);
            if (!A::EXACT) mma8(low[n], al, bh);
            if (!B::EXACT) mma8(low[n], ah, bl);
            mma8(acc[n], ah, bh);
        }
    }
    if constexpr (!A::EXACT || !B::EXACT) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[n][e] += low[n][e];
    }
}
template <int N>
__device__ __forceinline__ void zero(float (&acc)[N][4]) {
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
}

// ---- rows in shared memory ----
// 64 rows of `width` elements (KP, a multiple of 8, at most) to shared memory rows of LD elements, by the block; rows at and behind
// n and columns behind the width become zero.  wide: as part of the copy group at hand; else done on return.
template <int KP, int LD, typename T>
__device__ __forceinline__ void load_rows(T* to, const T* from, long long ld, int n, int width, bool wide) {
    if (wide) {
        constexpr int E = 16 / sizeof(T), CPR = KP / E;
        for (int i = threadIdx.x; i < DC * CPR; i += DT) {
            const int r = i / CPR, c = i % CPR * E;
            const bool on = r < n && c < width;
            copy16_async(to + r * LD + c, on ? from + r * ld + c : from, on);
        }
    } else {
        for (int i = threadIdx.x; i < DC * KP; i += DT) {
            const int r = i / KP, c = i % KP;
            to[r * LD + c] = r < n && c < width ? from[r * ld + c] : T(0.f);
        }
    }
}
// 64 rows of 64 floats to rows of LD floats, as part of the copy group at hand.
template <int LD>
__device__ __forceinline__ void load_square(float* to, const float* from) {
    for (int i = threadIdx.x; i < DC * (DC / 4); i += DT) {
        const int r = i / (DC / 4), c = i % (DC / 4) * 4;
        copy16_async(to + r * LD + c, from + r * DC + c, true);
    }
}

// ---- factors of a chunk's rows ----
// In the workspace, by chunk and value head: RF_IN: beta exp(b) |k|^-1, RF_OUT: scale exp(b) |q|^-1, RF_END:
// exp(b_C - b) |k|^-1, RF_BETA: beta, 64 each, and exp(b_C) at RF_DECAY; for the gradients |q|^-1, |k|^-1 and b (float2).
constexpr int RF_IN = 0, RF_OUT = DC, RF_END = 2 * DC, RF_BETA = 3 * DC, RF_DECAY = 4 * DC, RF_RQ = DELTA_FACTORS, RF_RK = RF_RQ + DC,
              RF_B = RF_RK + DC;

// b of a chunk as two floats each (their sum is exact to 2^-48 or so): differences of neighbouring tokens keep
// their accuracy however much has decayed before them.  g below -200 counts as -200, whose exponential is zero too;
// minus infinity then gives no differences of infinities.  By one warp; lane i holds tokens 2i and 2i + 1.
__device__ __forceinline__ void chunk_decay(const float* g, long long ld, int n, float2 (&b)[2]) {
    const int lane = threadIdx.x & 31;
    double v[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float x = 2 * lane + i < n ? g[(2 * lane + i) * ld] : 0.f;
        v[i] = x < -200.f ? -200.0 : (double)x;
    }
    double sum = v[0] + v[1];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const double o = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += o;
    }
    const double at[2] = {sum - v[1], sum};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float hi = (float)at[i];
        b[i] = make_float2(hi, hi - hi == 0.f ? (float)(at[i] - (double)hi) : 0.f);
    }
}
// exp(b_i - b_j)
__device__ __forceinline__ float decay_between(float2 bi, float2 bj) { return expf((bi.x - bj.x) + (bi.y - bj.y)); }

// 1 / length of 64 rows of q and k in shared memory: two threads a row (threads 0..127: q, 128..255: k), the even
// one holds the result.
template <int KP, int LD, typename T>
__device__ __forceinline__ float row_length(const T* rows) {
    const int r = (threadIdx.x & 127) >> 1, half = threadIdx.x & 1;
    float s = 0.f;
#pragma unroll 8
    for (int c = half * 2; c < KP; c += 4) {
        const float2 v = seq_ld2(rows + r * LD + c);
        s = fmaf(v.x, v.x, fmaf(v.y, v.y, s));
    }
    s += __shfl_xor_sync(0xffffffffu, s, 1);
    return 1.f / sqrtf(s + QK_EPS);
}

// Two neighbouring values of a row, the first at column c of `width`; `pair`: rows lie in aligned pairs.
template <typename T>
__device__ __forceinline__ float2 load_pair(const T* at, int c, int width, bool pair) {
    if (pair) return c < width ? seq_ld2(at) : make_float2(0.f, 0.f);
    return make_float2(c < width ? seq_ld(at) : 0.f, c + 1 < width ? seq_ld(at + 1) : 0.f);
}
template <typename T>
__device__ __forceinline__ void store_pair(T* at, int c, int width, bool pair, float2 v) {
    if (pair) {
        if (c < width) seq_st2(at, v, true, true);
    } else {
        if (c < width) seq_st(at, v.x);
        if (c + 1 < width) seq_st(at + 1, v.y);
    }
}

// ---- a walk's place ----
// With few heads the chunks of a long sequence in order leave most SMs without work.  Its axis is then cut into pieces of p.run chunks, whose walks
// are: what a piece adds to a state (from zero; the first piece: from the sequence's state), and, as its columns, what becomes of the unit
// matrix with v = 0 (DELTA_PIECES, the last piece of a sequence needs neither); h = through h + added from piece to piece gives the states
// that they leave (delta_join_kernel); and the walks themselves from these (DELTA_JOINED).  The first of several starts from a copy of the
// sequence's state, which the joining puts where what the piece adds has been: the last one may be writing the state in its place.
// The piece whose mark is token m * len (see delta_marks): its sequence, index in it, and first token; `t1`: the sequence's end.
struct MarkPiece {
    int s, index, t0, t1;
};
__device__ __forceinline__ MarkPiece mark_piece(const SeqAxis& a, int m, int len) {
    const int t = m * len;           // (a token: below T)
    MarkPiece c;
    if (a.L > 0) {
        c.s = t / a.L;
    } else {
        int lo = 0, hi = a.S - 1;    // the last sequence that begins at or before the mark
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (seq_start(a, mid, 0) <= t) lo = mid; else hi = mid - 1;
        }
        c.s = lo;
    }
    const int begin = seq_start(a, c.s, 0);
    c.t1 = seq_start(a, c.s + 1, begin);
    c.index = t > begin ? (t - begin) / len : 0;
    c.t0 = begin + c.index * len;
    return c;
}
// The mark of the first piece of a sequence that begins at t0.
__device__ __forceinline__ int first_mark(int t0, int len) { return (int)(((long long)t0 + len - 1) / len); }
struct WalkPlace {
    int h, seq, dvb, t0, t1, chunks, slot0;
    int mark;                        // of the piece, or (DELTA_JOINED, but for the first) of the one before it
    bool first, last, unit;          // piece of its sequence; columns of the unit matrix
    bool none;                       // nothing to do
};
template <int MODE>
__device__ __forceinline__ WalkPlace walk_place(const SeqDeltaParams& p, int dvbs, int dkbs) {
    WalkPlace w;
    const int per = MODE == DELTA_PIECES ? dvbs + dkbs : dvbs, sh = blockIdx.x / per, piece = sh / p.Hv;
    w.dvb = blockIdx.x % per;
    w.unit = MODE == DELTA_PIECES && w.dvb >= dvbs;
    if (w.unit) w.dvb -= dvbs;
    w.h = sh % p.Hv;
    w.mark = 0;
    if (MODE == DELTA_WHOLE) {
        w.seq = piece;
        w.t0 = p.ax.L > 0 ? w.seq * p.ax.L : seq_start(p.ax, w.seq, 0);
        w.t1 = p.ax.L > 0 ? w.t0 + p.ax.L : seq_start(p.ax, w.seq + 1, w.t0);
        w.slot0 = cut_base(p.ax, w.seq, DC);
        w.first = w.last = true;
        w.none = false;
    } else if (MODE == DELTA_PIECES) {
        const int len = p.run * DC;
        const MarkPiece c = mark_piece(p.ax, piece, len);
        w.seq = c.s;
        w.mark = piece;
        w.t0 = c.t0;
        w.t1 = c.t0 + len;
        w.slot0 = cut_base(p.ax, w.seq, DC) + c.index * p.run;
        w.first = c.index == 0;
        w.last = w.t1 >= c.t1;
        w.none = w.last || (w.unit && w.first);
    } else {
        const int len = p.run * DC;
        const CutPiece c = cut_piece(p.ax, piece, len);
        w.seq = c.s;
        w.t0 = c.t0;
        w.t1 = c.t0 + max(c.n, 0);
        w.slot0 = cut_base(p.ax, w.seq, DC) + c.index * p.run;
        w.first = c.index == 0;
        const int begin = seq_start(p.ax, w.seq, 0);
        w.last = w.t1 >= seq_start(p.ax, w.seq + 1, begin);
        w.none = c.n <= 0 && !w.first;
        w.mark = first_mark(begin, len) + max(c.index - 1, 0);
    }
    w.chunks = (w.t1 - w.t0 + DC - 1) / DC;
    return w;
}

// T, A and the row factors of every chunk (the first kernel of a forward and of a backward call).
cudaError_t launch_seq_delta_chunks(const SeqDeltaParams& p, bool bf16, cudaStream_t stream);

}  // namespace convfwd

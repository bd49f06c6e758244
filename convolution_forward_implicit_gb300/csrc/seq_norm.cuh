// What the forward and backward kernels of the norm, gate and residual step share: a row's place
// in a thread block, its loads and stores, and its sums.
#pragma once
#include "seq_common.cuh"
#include "seq_internal.h"

namespace convfwd {

// A row of D values lies on TPR = blockDim.x threads (whole warps); a block holds blockDim.y rows at a
// time.  Thread i holds columns 8 (i + u TPR) .. + 7 for u < UPT, as 4 pairs each: the arithmetic between
// the sums is on packed pairs.
#define EACH_PAIR _Pragma("unroll") for (int u = 0; u < UPT; ++u) _Pragma("unroll") for (int e = 0; e < 4; ++e)

__device__ __forceinline__ float2 pmul(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 padd(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 pfma(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 pdup(float a) { return make_float2(a, a); }

// 8 values as loaded; `put` and `get` convert.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
    uint4 q;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { q = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void zero() { q = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void ones() { q = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u); }
    __device__ __forceinline__ void get(float2 (&v)[4]) const {
        bf2_unpack(q.x, v[0].x, v[0].y);
        bf2_unpack(q.y, v[1].x, v[1].y);
        bf2_unpack(q.z, v[2].x, v[2].y);
        bf2_unpack(q.w, v[3].x, v[3].y);
    }
};
template <>
struct Raw8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = reinterpret_cast<const float4*>(p)[0];
        b = reinterpret_cast<const float4*>(p)[1];
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void ones() { a = b = make_float4(1.f, 1.f, 1.f, 1.f); }
    __device__ __forceinline__ void get(float2 (&v)[4]) const {
        v[0] = make_float2(a.x, a.y);
        v[1] = make_float2(a.z, a.w);
        v[2] = make_float2(b.x, b.y);
        v[3] = make_float2(b.z, b.w);
    }
};

// A thread's columns of a row, as loaded (WIDE) or converted one by one; columns behind D are zero.
template <typename T, bool WIDE, int UPT>
struct RowIn {
    Raw8<T> raw[WIDE ? UPT : 1];
    float2 val[WIDE ? 1 : UPT][4];
    __device__ __forceinline__ void load(const void* base, long long off, int D) {
        const T* p = static_cast<const T*>(base) + off;
#pragma unroll
        for (int u = 0; u < UPT; ++u) {
            const int c = (threadIdx.x + u * blockDim.x) * 8;
            if constexpr (WIDE) {
                if (c < D) raw[u].load(p + c);
                else raw[u].zero();
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    val[u][e] = make_float2(c + 2 * e < D ? seq_ld(p + c + 2 * e) : 0.f, c + 2 * e + 1 < D ? seq_ld(p + c + 2 * e + 1) : 0.f);
            }
        }
    }
    __device__ __forceinline__ void get(float2 (&v)[UPT][4]) const {
#pragma unroll
        for (int u = 0; u < UPT; ++u) {
            if constexpr (WIDE) {
                raw[u].get(v[u]);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) v[u][e] = val[u][e];
            }
        }
    }
};
template <typename T, bool WIDE, int UPT>
__device__ __forceinline__ void row_load(const void* base, long long off, int D, float2 (&v)[UPT][4]) {
    RowIn<T, WIDE, UPT> in;
    in.load(base, off, D);
    in.get(v);
}
template <typename T, bool WIDE, int UPT>
__device__ __forceinline__ void row_store(void* base, long long off, int D, const float2 (&v)[UPT][4]) {
    T* p = static_cast<T*>(base) + off;
#pragma unroll
    for (int u = 0; u < UPT; ++u) {
        const int c = (threadIdx.x + u * blockDim.x) * 8;
        if constexpr (WIDE) {
            const float w[8] = {v[u][0].x, v[u][0].y, v[u][1].x, v[u][1].y, v[u][2].x, v[u][2].y, v[u][3].x, v[u][3].y};
            if (c < D) seq_stv<8>(p + c, w);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (c + 2 * e < D) seq_st(p + c + 2 * e, v[u][e].x);
                if (c + 2 * e + 1 < D) seq_st(p + c + 2 * e + 1, v[u][e].y);
            }
        }
    }
}
// A parameter of the columns, held in registers as loaded (KEEP) or loaded at each use; ones or zeros where there
// is none, so that its uses need no branch (a branch costs a register move for each value that it may change).
template <typename T, bool WIDE, int UPT, bool KEEP, bool ONES>
struct Column {
    RowIn<T, WIDE, UPT> in;
    const void* base;
    __device__ __forceinline__ void load(RowIn<T, WIDE, UPT>& to, int D) const {
        if (base) {
            to.load(base, 0, D);
        } else if constexpr (WIDE) {
#pragma unroll
            for (int u = 0; u < UPT; ++u) {
                if (ONES) to.raw[u].ones();
                else to.raw[u].zero();
            }
        } else {
            EACH_PAIR to.val[u][e] = pdup(ONES ? 1.f : 0.f);
        }
    }
    __device__ __forceinline__ void open(const void* from, int D) {
        base = from;
        if (KEEP) load(in, D);
    }
    __device__ __forceinline__ void get(int D, float2 (&w)[UPT][4]) const {
        if constexpr (KEEP) {
            in.get(w);
        } else {
            RowIn<T, WIDE, UPT> now;
            load(now, D);
            now.get(w);
        }
    }
    __device__ __forceinline__ void mul(int D, float2 (&v)[UPT][4]) const {
        float2 w[UPT][4];
        get(D, w);
        EACH_PAIR v[u][e] = pmul(v[u][e], w[u][e]);
    }
    __device__ __forceinline__ void add(int D, float2 (&v)[UPT][4]) const {
        float2 w[UPT][4];
        get(D, w);
        EACH_PAIR v[u][e] = padd(v[u][e], w[u][e]);
    }
};
// v *= the columns' parameter, v += the parameter (nothing where there is none).
template <typename T, bool WIDE, int UPT>
__device__ __forceinline__ void col_mul(const void* base, int D, float2 (&v)[UPT][4]) {
    if (!base) return;
    float2 w[UPT][4];
    row_load<T, WIDE, UPT>(base, 0, D, w);
    EACH_PAIR v[u][e] = pmul(v[u][e], w[u][e]);
}
template <typename T, bool WIDE, int UPT>
__device__ __forceinline__ void col_add(const void* base, int D, float2 (&v)[UPT][4]) {
    if (!base) return;
    float2 w[UPT][4];
    row_load<T, WIDE, UPT>(base, 0, D, w);
    EACH_PAIR v[u][e] = padd(v[u][e], w[u][e]);
}
__device__ __forceinline__ float2 silu2(float2 v) { return pmul(v, make_float2(sigmoid(v.x), sigmoid(v.y))); }

// Rows on their way through shared memory.  A thread copies exactly the columns that it will use (16 bytes
// a copy, copies of neighbouring threads side by side), so it only has to wait for its own copies: no
// barrier.  `at` is the thread's place in the tensor's part of a stage, row_bytes of THREADS threads.
template <typename T, int UPT, int THREADS>
__host__ __device__ constexpr int row_bytes() { return THREADS * UPT * 8 * (int)sizeof(T); }
template <typename T, int UPT, int THREADS>
__device__ __forceinline__ void row_copy(uint32_t at, const void* base, long long off, int D) {
    constexpr int H = sizeof(T) * 8 / 16;
    const T* p = static_cast<const T*>(base) + off + threadIdx.x * 8;
#pragma unroll
    for (int u = 0; u < UPT; ++u) {
        const bool on = (threadIdx.x + u * blockDim.x) * 8 < D;
        const T* q = on ? p + u * blockDim.x * 8 : static_cast<const T*>(base);
#pragma unroll
        for (int h = 0; h < H; ++h)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at + (u * H + h) * THREADS * 16), "l"(q + h * (16 / sizeof(T))),
                         "r"(on ? 16 : 0) : "memory");
    }
}
__device__ __forceinline__ uint4 shared_16(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
template <typename T, int UPT, int THREADS>
__device__ __forceinline__ void row_take(uint32_t at, float2 (&v)[UPT][4]) {
    constexpr int H = sizeof(T) * 8 / 16;
#pragma unroll
    for (int u = 0; u < UPT; ++u) {
        Raw8<T> raw;
        if constexpr (H == 1) {
            raw.q = shared_16(at + u * THREADS * 16);
        } else {
            const uint4 a = shared_16(at + u * 2 * THREADS * 16), b = shared_16(at + (u * 2 + 1) * THREADS * 16);
            raw.a = make_float4(__uint_as_float(a.x), __uint_as_float(a.y), __uint_as_float(a.z), __uint_as_float(a.w));
            raw.b = make_float4(__uint_as_float(b.x), __uint_as_float(b.y), __uint_as_float(b.z), __uint_as_float(b.w));
        }
        raw.get(v[u]);
    }
}

// Sums over the threads of a row.  A warp sums by shuffles, so that all of its lanes hold the same value and
// store it to the warp's slot (one store, no predicate); behind a barrier each thread reads the row's slots
// four at a time and adds them up, always in the same order.  Two halves of the buffer take turns, so one barrier a sum is
// enough.  Every thread of the block takes part.  THREADS: of the block at most.
struct NormSums {
    float v[2][4][64];       // turn, value, slot: a row has THREADS / 32 of them, or more threads in one row
    float n[64];             // columns of the slot's warp
};
template <int THREADS>
struct RowSums {
    static constexpr int SLOTS = (THREADS / 32 + 3) / 4 * 4;
    uint32_t put, half, get, counts;     // shared addresses: the warp's slot (and, for lanes 16 .. 31, the next value's)
    int turn;
    float n, inv_n;
    template <int UPT>
    __device__ __forceinline__ void init(NormSums& b, int D) {
        const int tid = threadIdx.y * blockDim.x + threadIdx.x, all = blockDim.x * blockDim.y;
        for (int i = tid; i < (int)(sizeof(NormSums) / 4); i += all) (&b.v[0][0][0])[i] = 0.f;
        __syncthreads();
        const int first = threadIdx.y * SLOTS, warp = threadIdx.x >> 5;
        int columns = 0;
#pragma unroll
        for (int u = 0; u < UPT; ++u) columns += max(0, min(256, D - (int)(warp * 32 + u * blockDim.x) * 8));
        n = (float)columns;
        inv_n = 1.0f / (float)max(columns, 1);
        b.n[first + warp] = n;           // (read behind a sum's barrier)
        get = (uint32_t)__cvta_generic_to_shared(&b.v[0][0][first]);
        counts = (uint32_t)__cvta_generic_to_shared(&b.n[first]);
        put = get + warp * 4;
        half = put + (threadIdx.x & 16) * 16;
        asm volatile("" : "+r"(put), "+r"(half), "+r"(get));       // (not to be worked out again at every use)
        turn = 4 * 64 * 4;
    }
    __device__ __forceinline__ void next() { put += turn, half += turn, get += turn, turn = -turn; }
    static __device__ __forceinline__ void store(uint32_t at, float v) { asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory"); }
    static __device__ __forceinline__ float4 four(uint32_t at) {
        float4 q;
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(q.x), "=f"(q.y), "=f"(q.z), "=f"(q.w) : "r"(at) : "memory");
        return q;
    }
    static __device__ __forceinline__ void barrier() {
        if (blockDim.x == 32) __syncwarp();
        else __syncthreads();
    }
    // of one value over the warp; of two, one in lanes 0 .. 15 and the other in 16 .. 31
    static __device__ __forceinline__ float warp(float a) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(~0u, a, o);
        return a;
    }
    static __device__ __forceinline__ float warp(float a, float b) {
        const bool up = threadIdx.x & 16;
        float v = (up ? b : a) + __shfl_xor_sync(~0u, up ? a : b, 16);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
        return v;
    }
    __device__ __forceinline__ float slots(int k) const {
        float2 s[SLOTS / 4];
#pragma unroll
        for (int w = 0; w < SLOTS / 4; ++w) {
            const float4 q = four(get + (k * 64 + 4 * w) * 4);
            s[w] = padd(make_float2(q.x, q.y), make_float2(q.z, q.w));
        }
#pragma unroll
        for (int o = SLOTS / 8; o > 0; o /= 2)
#pragma unroll
            for (int w = 0; w < o; ++w) s[w] = padd(s[w], s[w + o]);
        return s[0].x + s[0].y;
    }
    __device__ __forceinline__ float sum(float a) {
        store(put, warp(a));
        barrier();
        a = slots(0);
        next();
        return a;
    }
    __device__ __forceinline__ void sum(float& a, float& b) {
        store(half, warp(a, b));
        barrier();
        a = slots(0);
        b = slots(1);
        next();
    }
};
template <int UPT>
__device__ __forceinline__ float lane_total(const float2 (&v)[UPT][4]) {
    float2 s = make_float2(0.f, 0.f);
    EACH_PAIR s = padd(s, v[u][e]);
    return s.x + s.y;
}
template <int UPT>
__device__ __forceinline__ float lane_dot(const float2 (&v)[UPT][4], const float2 (&w)[UPT][4]) {
    float2 s = make_float2(0.f, 0.f);
    EACH_PAIR s = pfma(v[u][e], w[u][e], s);
    return s.x + s.y;
}
// v -= m in the row's columns
template <bool WIDE, int UPT>
__device__ __forceinline__ void row_shift(float2 (&v)[UPT][4], int D, float m) {
    EACH_PAIR {
        const int c = (threadIdx.x + u * blockDim.x) * 8;
        if constexpr (WIDE) {
            v[u][e] = padd(v[u][e], pdup(c < D ? -m : 0.f));
        } else {
            if (c + 2 * e < D) v[u][e].x -= m;
            if (c + 2 * e + 1 < D) v[u][e].y -= m;
        }
    }
}

// What a layer norm's row is made of, from its warps' parts: warp w has n_w columns of mean m_w, the sum Q_w of
// (v - m_w)^2, and (BACK) the sums P_w of e (v - m_w) and E_w of e.  With d_w = m_w - m_0,
//   mean = m_0 + sum n_w d_w / D,   sum (v - mean)^2 = sum (Q_w + n_w d_w^2) - (sum n_w d_w)^2 / D,
//   sum e (v - mean) = sum (P_w + d_w E_w) - (mean - m_0) sum E_w.
// Only differences of the warps' means are squared, so rows far from zero lose nothing.  (Values 0 .. 3: m, E, Q, P.)
template <bool BACK, int THREADS>
__device__ __forceinline__ void row_moments(const RowSums<THREADS>& s, float inv_D, float& mean, float& Q, float& P, float& E) {
    float a = 0.f, b = 0.f, m0 = 0.f;
    Q = P = E = 0.f;
#pragma unroll
    for (int w = 0; w < s.SLOTS; w += 4) {
        const float4 m = s.four(s.get + w * 4), q = s.four(s.get + (128 + w) * 4), n = s.four(s.counts + w * 4);
        if (w == 0) m0 = m.x;
        const float mm[4] = {m.x, m.y, m.z, m.w}, nn[4] = {n.x, n.y, n.z, n.w};
        float d[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            d[i] = mm[i] - m0;
            const float t = nn[i] * d[i];
            a += t;
            b = fmaf(t, d[i], b);
        }
        Q += (q.x + q.y) + (q.z + q.w);
        if (BACK) {
            const float4 e = s.four(s.get + (64 + w) * 4), p = s.four(s.get + (192 + w) * 4);
            E += (e.x + e.y) + (e.z + e.w);
            P += (p.x + p.y) + (p.z + p.w);
            P = fmaf(d[0], e.x, fmaf(d[1], e.y, fmaf(d[2], e.z, fmaf(d[3], e.w, P))));
        }
    }
    const float shift = a * inv_D;
    mean = m0 + shift;
    Q += fmaf(-shift, a, b);
    if (BACK) P = fmaf(-shift, E, P);
}

// 1 / sqrt(v); 0 in the place of a row behind the last one, which must add nothing to the parameters' sums even
// where eps is 0.
__device__ __forceinline__ float norm_factor(float v, bool there) { return there ? 1.0f / sqrtf(v) : 0.f; }
// v -> (v - mean) / sqrt(var + eps) (layer) or v / sqrt(mean(v^2) + eps) in place; returns the
// factor 1 / sqrt(...).  Columns at and behind D stay zero.  One barrier.
template <bool WIDE, int UPT, int THREADS>
__device__ __forceinline__ float row_norm(float2 (&v)[UPT][4], int D, bool layer, float eps, RowSums<THREADS>& s, bool there) {
    const float inv = 1.0f / (float)D;
    float q;
    if (layer) {
        const float m = s.warp(lane_total(v)) * s.inv_n;
        row_shift<WIDE>(v, D, m);
        s.store(s.put, m);
        s.store(s.put + 2 * 64 * 4, s.warp(lane_dot(v, v)));
        s.barrier();
        float mean, unused;
        row_moments<false>(s, inv, mean, q, unused, unused);
        s.next();
        row_shift<WIDE>(v, D, mean - m);
    } else {
        q = s.sum(lane_dot(v, v));
    }
    const float r = norm_factor(fmaf(q, inv, eps), there);
    EACH_PAIR v[u][e] = pmul(v[u][e], pdup(r));
    return r;
}

constexpr int NORM_RING = 2;                  // stages: a row in use and one on its way
constexpr int NORM_RING_MAX = 224 * 1024;     // bytes of a block's stages; wider rows are loaded directly
static_assert(NORM_RING_MAX + sizeof(NormSums) <= 227 * 1024, "a block's shared memory");

// Threads per row and rows per block: upt groups of 8 columns to a thread.
inline dim3 norm_block(int D, int upt) {
    const int tpr = (((D + 7) / 8 + upt - 1) / upt + 31) / 32 * 32;
    return dim3((unsigned)tpr, (unsigned)(tpr < 128 ? 128 / tpr : 1));
}

}  // namespace convfwd

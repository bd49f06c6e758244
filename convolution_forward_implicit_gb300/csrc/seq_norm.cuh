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
// A parameter of the columns, held in registers as loaded (KEEP) or loaded at each use.
template <typename T, bool WIDE, int UPT, bool KEEP>
struct Column {
    RowIn<T, WIDE, UPT> in;
    const void* base;
    __device__ __forceinline__ void open(const void* from, int D) {
        base = from;
        if (KEEP && base) in.load(base, 0, D);
    }
    __device__ __forceinline__ void get(int D, float2 (&w)[UPT][4]) const {
        if constexpr (KEEP) in.get(w);
        else row_load<T, WIDE, UPT>(base, 0, D, w);
    }
    // v *= it, v += it: nothing where there is none
    __device__ __forceinline__ void mul(int D, float2 (&v)[UPT][4]) const {
        if (!base) return;
        float2 w[UPT][4];
        get(D, w);
        EACH_PAIR v[u][e] = pmul(v[u][e], w[u][e]);
    }
    __device__ __forceinline__ void add(int D, float2 (&v)[UPT][4]) const {
        if (!base) return;
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

// Sums K values over the threads of a row; every thread of the block calls it together.  `turn`
// alternates between two halves of the shared buffer, so one barrier a call is enough.  The warps' sums lie
// in groups of four, which each thread reads at once and adds up in order.
struct NormSums {
    float v[2][2][32];       // turn, value, warp
};
template <int N>
struct NormGroups {
    static constexpr int n = N;
};
__device__ __forceinline__ void row_sum_init(NormSums& b) {
    for (int i = threadIdx.y * blockDim.x + threadIdx.x; i < 128; i += blockDim.x * blockDim.y) (&b.v[0][0][0])[i] = 0.f;
    __syncthreads();
}
template <int K>
__device__ __forceinline__ void row_sum(float (&v)[K], NormSums& b, int& turn) {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(~0u, v[k], o);
    const int wpr = blockDim.x >> 5;
    if (wpr == 1) return;
    const int fours = (wpr + 3) >> 2, first = threadIdx.y * fours * 4;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
        for (int k = 0; k < K; ++k) b.v[turn][k][first + (threadIdx.x >> 5)] = v[k];
    }
    __syncthreads();
    auto add = [&](auto groups) {                  // (slots behind the row's warps hold zeros)
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float4 q[decltype(groups)::n];
#pragma unroll
            for (int w = 0; w < decltype(groups)::n; ++w) q[w] = *reinterpret_cast<const float4*>(&b.v[turn][k][first + 4 * w]);
            v[k] = 0.f;
#pragma unroll
            for (int w = 0; w < decltype(groups)::n; ++w) v[k] += (q[w].x + q[w].y) + (q[w].z + q[w].w);
        }
    };
    if (fours == 1) add(NormGroups<1>());
    else if (fours == 2) add(NormGroups<2>());
    else if (fours <= 4) add(NormGroups<4>());
    else add(NormGroups<8>());
    turn ^= 1;
}
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

// v -> (v - mean) / sqrt(var + eps) (layer) or v / sqrt(mean(v^2) + eps) in place; returns the
// factor 1 / sqrt(...).  Columns at and behind D stay zero.  The variance is summed from the centred
// values, which keeps it exact for rows far from zero.
template <int UPT>
__device__ __forceinline__ float row_norm(float2 (&v)[UPT][4], int D, bool layer, float eps, NormSums& buf, int& turn) {
    const float inv = 1.0f / (float)D;
    float s[1];
    if (layer) {
        s[0] = lane_total(v);
        row_sum(s, buf, turn);
        const float mean = s[0] * inv;
        EACH_PAIR {
            const int c = (threadIdx.x + u * blockDim.x) * 8 + 2 * e;
            if (c < D) v[u][e].x -= mean;
            if (c + 1 < D) v[u][e].y -= mean;
        }
    }
    s[0] = lane_dot(v, v);
    row_sum(s, buf, turn);
    const float r = 1.0f / sqrtf(fmaf(s[0], inv, eps));
    EACH_PAIR v[u][e] = pmul(v[u][e], pdup(r));
    return r;
}

constexpr int NORM_RING = 2;                  // stages: a row in use and one on its way
constexpr int NORM_RING_MAX = 226 * 1024;     // bytes of a block's stages; wider rows are loaded directly

// Threads per row and rows per block: upt groups of 8 columns to a thread.
inline dim3 norm_block(int D, int upt) {
    const int tpr = (((D + 7) / 8 + upt - 1) / upt + 31) / 32 * 32;
    return dim3((unsigned)tpr, (unsigned)(tpr < 128 ? 128 / tpr : 1));
}

}  // namespace convfwd

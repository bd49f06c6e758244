// Device helpers of the sequence-mixing kernels: loads and stores of 1 or several elements of
// either type as fp32, and the scalar functions they share.
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

#include "gelu.cuh"

namespace convfwd {

__device__ __forceinline__ float seq_ld(const float* p) { return *p; }
__device__ __forceinline__ float seq_ld(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void seq_st(float* p, float v) { *p = v; }
__device__ __forceinline__ void seq_st(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ void bf2_unpack(uint32_t u, float& a, float& b) {
    a = __uint_as_float(u << 16);
    b = __uint_as_float(u & 0xffff0000u);
}
__device__ __forceinline__ uint32_t bf2_pack(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// V consecutive elements <-> fp32 registers; V > 1: whole
// 16-byte groups (or 8 bytes: 4 bf16) at an address aligned to them.
template <int V>
__device__ __forceinline__ void seq_ldv(const float* p, float (&v)[V]) {
    if constexpr (V % 4 == 0) {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            const float4 q = reinterpret_cast<const float4*>(p)[i];
            v[4 * i] = q.x; v[4 * i + 1] = q.y; v[4 * i + 2] = q.z; v[4 * i + 3] = q.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = p[i];
    }
}
template <int V>
__device__ __forceinline__ void seq_ldv(const __nv_bfloat16* p, float (&v)[V]) {
    if constexpr (V % 8 == 0) {
#pragma unroll
        for (int i = 0; i < V / 8; ++i) {
            const uint4 q = reinterpret_cast<const uint4*>(p)[i];
            bf2_unpack(q.x, v[8 * i], v[8 * i + 1]);
            bf2_unpack(q.y, v[8 * i + 2], v[8 * i + 3]);
            bf2_unpack(q.z, v[8 * i + 4], v[8 * i + 5]);
            bf2_unpack(q.w, v[8 * i + 6], v[8 * i + 7]);
        }
    } else if constexpr (V == 4) {
        const uint2 q = *reinterpret_cast<const uint2*>(p);
        bf2_unpack(q.x, v[0], v[1]);
        bf2_unpack(q.y, v[2], v[3]);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = __bfloat162float(p[i]);
    }
}
template <int V>
__device__ __forceinline__ void seq_stv(float* p, const float (&v)[V]) {
    if constexpr (V % 4 == 0) {
#pragma unroll
        for (int i = 0; i < V / 4; ++i)
            reinterpret_cast<float4*>(p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    } else if constexpr (V == 2) {
        *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = v[i];
    }
}
template <int V>
__device__ __forceinline__ void seq_stv(__nv_bfloat16* p, const float (&v)[V]) {
    if constexpr (V % 8 == 0) {
#pragma unroll
        for (int i = 0; i < V / 8; ++i)
            reinterpret_cast<uint4*>(p)[i] =
                make_uint4(bf2_pack(v[8 * i], v[8 * i + 1]), bf2_pack(v[8 * i + 2], v[8 * i + 3]),
                           bf2_pack(v[8 * i + 4], v[8 * i + 5]), bf2_pack(v[8 * i + 6], v[8 * i + 7]));
    } else if constexpr (V == 4) {
        *reinterpret_cast<uint2*>(p) = make_uint2(bf2_pack(v[0], v[1]), bf2_pack(v[2], v[3]));
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = __float2bfloat16_rn(v[i]);
    }
}

constexpr float LOG2E = 1.4426950408889634f;

// 2^v on the special-function unit.
__device__ __forceinline__ float ex2_approx(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
// 1 / (1 + e^-v).  For v below -88 the exponential overflows to infinity and the reciprocal is 0.
__device__ __forceinline__ float sigmoid(float v) { return rcp_approx(1.0f + ex2_approx(-LOG2E * v)); }
__device__ __forceinline__ float silu(float v) { return v * sigmoid(v); }
// d silu / dv = s (1 + v (1 - s)), s = sigmoid(v)
__device__ __forceinline__ float silu_grad(float v, float s) { return s * fmaf(v, 1.0f - s, 1.0f); }

// log(1 + e^v) = max(v, 0) + log1p(q), q = e^-|v| in (0, 1].  log1p(q) = 2 atanh(r), r = q / (2 + q)
// <= 1/3, by atanh's Taylor series r (1 + r^2/3 + r^4/5 + ...): the first term left out, r^16/17, is
// below 2e-9 relative, and small q keeps its relative accuracy (a step of 1e-3 is as exact as one of 1).
__device__ __forceinline__ float softplus(float v) {
    const float q = ex2_approx(-LOG2E * fabsf(v));
    const float r = q * rcp_approx(2.0f + q);
    const float r2 = r * r;
    float s = fmaf(r2, 1.0f / 15.0f, 1.0f / 13.0f);
    s = fmaf(r2, s, 1.0f / 11.0f);
    s = fmaf(r2, s, 1.0f / 9.0f);
    s = fmaf(r2, s, 1.0f / 7.0f);
    s = fmaf(r2, s, 1.0f / 5.0f);
    s = fmaf(r2, s, 1.0f / 3.0f);
    s = fmaf(r2, s, 1.0f);
    return fmaf(2.0f * r, s, fmaxf(v, 0.0f));
}

// Copies of 16 bytes from global to shared memory that run on while the thread goes on; `on` false:
// zeros, and no access to the source.
__device__ __forceinline__ void copy16_async(void* to, const void* from, bool on) {
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(to);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(from), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most N of this thread's latest groups are still on their way.
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// rows_to_shared for rows that are not whole 16-byte groups.  A thread stays in its columns and steps from row to
// row, so that a copy costs little more than one addition.
template <typename T, int ROWS, int W, int THREADS>
__device__ __noinline__ void rows_to_shared_odd(T (*to)[W], const T* from, long long ld, int n, int width, int grain) {
    if (grain == 4) {
        constexpr int E = 4 / sizeof(T), CPR = W / E, CPT = CPR > THREADS ? CPR / THREADS : 1;
        constexpr int STEP = CPR > THREADS ? 1 : THREADS / CPR, J = (ROWS + STEP - 1) / STEP;
        static_assert(CPR % THREADS == 0 || THREADS % CPR == 0, "whole columns to a thread");
        const int r0 = CPR >= THREADS ? 0 : threadIdx.x / CPR;
#pragma unroll
        for (int u = 0; u < CPT; ++u) {
            const int c = (threadIdx.x % CPR + u * THREADS) * E;
            const bool on = c < width;
            const T* at = on ? from + r0 * ld + c : from;
            const long long next = on ? STEP * ld : 0;
            uint32_t d = (uint32_t)__cvta_generic_to_shared(&to[r0][c]);
#pragma unroll
            for (int j = 0; j < J; ++j) {
                if (ROWS % STEP == 0 || r0 + j * STEP < ROWS) {
                    const bool there = on && r0 + j * STEP < n;
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(d + j * STEP * W * (int)sizeof(T)), "l"(there ? at : from),
                                 "r"(there ? 4 : 0) : "memory");
                }
                at += next;
            }
        }
    } else {
        constexpr int CPT = W > THREADS ? W / THREADS : 1, STEP = W > THREADS ? 1 : THREADS / W, J = (ROWS + STEP - 1) / STEP;
        static_assert(W % THREADS == 0 || THREADS % W == 0, "whole columns to a thread");
        const int r0 = W >= THREADS ? 0 : threadIdx.x / W;
#pragma unroll
        for (int u = 0; u < CPT; ++u) {
            const int c = threadIdx.x % W + u * THREADS;
            const bool on = c < width;
            const T* at = on ? from + r0 * ld + c : from;
            T v[J];
#pragma unroll
            for (int j = 0; j < J; ++j) {
                v[j] = on && r0 + j * STEP < n ? at[0] : T(0.f);
                at += STEP * ld;
            }
#pragma unroll
            for (int j = 0; j < J; ++j)
                if (ROWS % STEP == 0 || r0 + j * STEP < ROWS) to[r0 + j * STEP][c] = v[j];
        }
    }
}
// n rows of W elements (a multiple of 16 bytes), ROWS at most, to shared memory by the block's THREADS
// threads, as part of the copy group at hand.  Columns at and behind `width` and rows at and behind n
// become zero.  WIDE: rows are whole and aligned groups of 16 bytes.  Otherwise grain: 4 when they are such groups
// of 4 bytes; else 0: plain loads (2-byte elements at odd places), which are done on return.
template <typename T, int ROWS, int W, int THREADS, bool WIDE>
__device__ __forceinline__ void rows_to_shared(T (*to)[W], const T* from, long long ld, int n, int width, int grain) {
    if constexpr (WIDE) {
        constexpr int E = 16 / sizeof(T), CPR = W / E, ALL = ROWS * CPR;
        static_assert(W % E == 0, "rows of whole 16-byte groups");
#pragma unroll
        for (int j = 0; j < (ALL + THREADS - 1) / THREADS; ++j) {
            const int i = threadIdx.x + j * THREADS, r = i / CPR, c = i % CPR * E;
            if (ALL % THREADS == 0 || i < ALL) {
                const bool on = r < n && c < width;
                copy16_async(&to[r][c], on ? from + r * ld + c : from, on);
            }
        }
    } else {
        rows_to_shared_odd<T, ROWS, W, THREADS>(to, from, ld, n, width, grain);
    }
}

// Sum of the values at `rows` rows `step` apart, of 32 neighbouring columns (`src`: the column of lane
// threadIdx.x & 31) by a block of COLUMN_THREADS: warps take turns at the rows, then the first warp adds their
// sums in order and holds the result.  Called by the whole block.
// Eight loads a thread are on their way at once, in kernels of 32 registers (two blocks an SM) that spill a little (the norm's
// 136 bytes, the convolution's 24).  With 16 and their registers, one block an SM and few of them next to the kernel
// before: the norm's 6007 x 1280 training pass 80.8 us against 82.3, the convolution's 8 x 2048 x 4096 147 against 144.
constexpr int COLUMN_THREADS = 1024;
__device__ __forceinline__ float column_sum(const float* src, long long step, int rows, bool on) {
    constexpr int WARPS = COLUMN_THREADS / 32;
    __shared__ float part[WARPS][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float s[4] = {};
    if (on) {
        for (int r = warp; r < rows; r += 8 * WARPS) {         // 8 loads on their way at once
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = r + i * WARPS < rows ? src[(r + i * WARPS) * step] : 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) s[i & 3] += v[i];
        }
    }
    part[warp][lane] = (s[0] + s[1]) + (s[2] + s[3]);
    __syncthreads();
    float v = 0.f;
    if (warp == 0)
#pragma unroll
        for (int w = 0; w < WARPS; ++w) v += part[w][lane];
    return v;
}

// softplus and, if wanted, its derivative sigmoid(v) of two values: see softplus.
__device__ __forceinline__ float2 softplus2(float2 v, float2* slope) {
    const float2 q = make_float2(ex2_approx(-LOG2E * fabsf(v.x)), ex2_approx(-LOG2E * fabsf(v.y)));
    const float2 two = make_float2(2.f, 2.f);
    const float2 d = __fadd2_rn(two, q);
    const float2 r = __fmul2_rn(q, make_float2(rcp_approx(d.x), rcp_approx(d.y)));
    const float2 r2 = __fmul2_rn(r, r);
    auto step = [&](float2 s, float c) { return __ffma2_rn(r2, s, make_float2(c, c)); };
    float2 s = step(make_float2(1.0f / 15.0f, 1.0f / 15.0f), 1.0f / 13.0f);
    s = step(s, 1.0f / 11.0f);
    s = step(s, 1.0f / 9.0f);
    s = step(s, 1.0f / 7.0f);
    s = step(s, 1.0f / 5.0f);
    s = step(s, 1.0f / 3.0f);
    s = step(s, 1.0f);
    if (slope) {                     // 1 / (1 + e^-v) = (v < 0 ? q : 1) / (1 + q)
        slope->x = (v.x < 0.f ? q.x : 1.f) * rcp_approx(1.f + q.x);
        slope->y = (v.y < 0.f ? q.y : 1.f) * rcp_approx(1.f + q.y);
    }
    return __ffma2_rn(__fmul2_rn(two, r), s, make_float2(fmaxf(v.x, 0.f), fmaxf(v.y, 0.f)));
}

__device__ __forceinline__ float2 seq_ld2(const float* p) { return *reinterpret_cast<const float2*>(p); }
__device__ __forceinline__ float2 seq_ld2(const __nv_bfloat16* p) {
    float2 v;
    bf2_unpack(*reinterpret_cast<const uint32_t*>(p), v.x, v.y);
    return v;
}
// Two neighbouring values; `pair`: both are there and the address is aligned to both.
__device__ __forceinline__ void seq_st2(float* p, float2 v, bool pair, bool one) {
    if (pair) *reinterpret_cast<float2*>(p) = v;
    else if (one) *p = v.x;
}
__device__ __forceinline__ void seq_st2(__nv_bfloat16* p, float2 v, bool pair, bool one) {
    if (pair) *reinterpret_cast<uint32_t*>(p) = bf2_pack(v.x, v.y);
    else if (one) *p = __float2bfloat16_rn(v.x);
}

}  // namespace convfwd

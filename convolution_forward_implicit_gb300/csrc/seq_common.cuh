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

// V consecutive elements <-> fp32 registers; V > 1 needs V * sizeof(T) a multiple of 16 and the
// address 16-byte aligned.
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

}  // namespace convfwd

// What the forward and backward kernels of the norm, gate and residual step share: a row's place
// in a thread block, its loads and stores, and its sums.
#pragma once
#include "seq_common.cuh"
#include "seq_internal.h"

namespace convfwd {

// A row of D values lies on TPR = blockDim.x threads (whole warps); a block holds blockDim.y rows.
// Thread i holds columns 8 (i + u TPR) .. + 7 for u < UPT.
template <typename T, bool WIDE, int UPT>
__device__ __forceinline__ void row_load(const void* base, long long off, int D, float (&v)[UPT][8]) {
    const T* p = static_cast<const T*>(base) + off;
#pragma unroll
    for (int u = 0; u < UPT; ++u) {
        const int c = (threadIdx.x + u * blockDim.x) * 8;
        if (WIDE) {
            if (c < D) {
                seq_ldv<8>(p + c, v[u]);
                continue;
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) v[u][e] = !WIDE && c + e < D ? seq_ld(p + c + e) : 0.f;
    }
}
template <typename T, bool WIDE, int UPT>
__device__ __forceinline__ void row_store(void* base, long long off, int D, const float (&v)[UPT][8]) {
    T* p = static_cast<T*>(base) + off;
#pragma unroll
    for (int u = 0; u < UPT; ++u) {
        const int c = (threadIdx.x + u * blockDim.x) * 8;
        if (WIDE) {
            if (c < D) seq_stv<8>(p + c, v[u]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (c + e < D) seq_st(p + c + e, v[u][e]);
        }
    }
}
// A per-column parameter, or its neutral value where there is none.
template <typename T, bool WIDE, int UPT>
__device__ __forceinline__ void col_load(const void* base, float neutral, int D, float (&v)[UPT][8]) {
    if (base) {
        row_load<T, WIDE, UPT>(base, 0, D, v);
        return;
    }
#pragma unroll
    for (int u = 0; u < UPT; ++u)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[u][e] = neutral;
}

// Sums K values over the threads of a row; every thread of the block calls it together.  `turn`
// alternates between two halves of the shared buffer, so one barrier a call is enough.
template <int K>
__device__ __forceinline__ void row_sum(float (&v)[K], float (*buf)[32][2], int& turn) {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(~0u, v[k], o);
    const int wpr = blockDim.x >> 5;
    if (wpr == 1) return;
    const int warp = threadIdx.y * wpr + (threadIdx.x >> 5);
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
        for (int k = 0; k < K; ++k) buf[turn][warp][k] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = 0.f;
    for (int w = 0; w < wpr; ++w) {
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += buf[turn][threadIdx.y * wpr + w][k];
    }
    turn ^= 1;
}

// v -> (v - mean) / sqrt(var + eps) (layer) or v / sqrt(mean(v^2) + eps) in place; returns the
// factor 1 / sqrt(...).  Columns at and behind D stay zero.  The variance is summed from the centred
// values, which keeps it exact for rows far from zero.
template <int UPT>
__device__ __forceinline__ float row_norm(float (&v)[UPT][8], int D, bool layer, float eps, float (*buf)[32][2], int& turn) {
    const float inv = 1.0f / (float)D;
    float s[1];
    if (layer) {
        s[0] = 0.f;
#pragma unroll
        for (int u = 0; u < UPT; ++u)
#pragma unroll
            for (int e = 0; e < 8; ++e) s[0] += v[u][e];
        row_sum(s, buf, turn);
        const float mean = s[0] * inv;
#pragma unroll
        for (int u = 0; u < UPT; ++u)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if ((threadIdx.x + u * blockDim.x) * 8 + e < D) v[u][e] -= mean;
    }
    s[0] = 0.f;
#pragma unroll
    for (int u = 0; u < UPT; ++u)
#pragma unroll
        for (int e = 0; e < 8; ++e) s[0] = fmaf(v[u][e], v[u][e], s[0]);
    row_sum(s, buf, turn);
    const float r = 1.0f / sqrtf(fmaf(s[0], inv, eps));
#pragma unroll
    for (int u = 0; u < UPT; ++u)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[u][e] *= r;
    return r;
}

// Threads per row (a multiple of 32) and rows per block for rows of D values, UPT groups of 8 a thread.
inline dim3 norm_block(int D, int upt, int threads) {
    const int units = (D + 7) / 8;
    int tpr = ((units + upt - 1) / upt + 31) / 32 * 32;
    int rpb = threads / tpr;
    return dim3((unsigned)tpr, (unsigned)(rpb < 1 ? 1 : rpb));
}

}  // namespace convfwd

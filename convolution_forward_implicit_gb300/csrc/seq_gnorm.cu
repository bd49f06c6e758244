// Group norm with an activation, channels last: see gnorm.h for the formulas.  Bound by bytes.  Statistics
// cross the whole sequence, so a call reads its rows twice: a pass for the sums of every slab of tokens and channel, a
// small one that joins them to the groups' statistics (a warp or a block a sequence and group), and one that
// applies them, last slabs first, so that it finds in L2 what the first pass read last.
//
// A slab's statistics are means and sums of squared differences, joined pairwise: M2 = M2a + M2b + d^2 na nb / n.  A thread
// sums over differences from the first value it meets in a channel; that value is one of the data, so the
// variance it takes part in is at least (its distance from the mean)^2 / n, and the rounding of the sums stays below
// about n 2^-24 of the result for n tokens a thread, wherever the mean lies.
#include "gnorm.h"
#include "seq_common.cuh"
#include "seq_internal.h"

namespace convfwd {
namespace {

constexpr int GN_BLOCK = 256;        // threads a block at most (those of whole rows of threads)

// How the channels lie on a block's threads: tx threads of V channels in a row, ty rows; cblocks blocks for all channels.
struct GnShape {
    int tx, ty, cblocks;
};
GnShape gn_shape(int D, int V) {
    const int n = (D + V - 1) / V;
    GnShape s;
    s.cblocks = (n + GN_BLOCK - 1) / GN_BLOCK;
    s.tx = (n + s.cblocks - 1) / s.cblocks;
    s.ty = GN_BLOCK / s.tx;
    if (s.ty < 2 && s.cblocks == 1) s.ty = 2;         // (up to 512 threads)
    return s;
}

// act(z), and its slope if wanted
template <int ACT>
__device__ __forceinline__ float act_of(float z) {
    return ACT == SEQ_ACT_SILU ? silu(z) : ACT == SEQ_ACT_GELU ? gelu(z) : z;
}
// d gelu = Phi(z) + z phi(z).  Phi from A&S 7.1.28 as in gelu (y^-16 = erfc |z| / sqrt 2).
__device__ __forceinline__ float gelu_slope(float z) {
    const float u = fabsf(z) * 0.70710678118654752f;
    float y = fmaf(u, 0.0000430638f, 0.0002765672f);
    y = fmaf(u, y, 0.0001520143f);
    y = fmaf(u, y, 0.0092705272f);
    y = fmaf(u, y, 0.0422820123f);
    y = fmaf(u, y, 0.0705230784f);
    y = fmaf(u, y, 1.0f);
    y = y * y; y = y * y; y = y * y; y = y * y;
    const float tail = 0.5f * rcp_approx(y);
    const float phi = 0.39894228040143268f * ex2_approx(-0.5f * LOG2E * z * z);
    return fmaf(z, phi, z < 0.f ? tail : 1.f - tail);
}
template <int ACT>
__device__ __forceinline__ float slope_of(float z) {
    if (ACT == SEQ_ACT_SILU) return silu_grad(z, sigmoid(z));
    if (ACT == SEQ_ACT_GELU) return gelu_slope(z);
    return 1.f;
}

__device__ __forceinline__ void wait_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void launch_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// A thread's place: its channels c .. c + V - 1 and row of threads.
struct GnPlace {
    int c, tx, ty, rows;
    bool on;
    __device__ __forceinline__ GnPlace(int V, int D, int txn, int rows_) : rows(rows_) {
        ty = threadIdx.x / txn;
        tx = threadIdx.x - ty * txn;
        c = (blockIdx.y * txn + tx) * V;
        on = c < D;
    }
};

// Channel parameters of a group norm call for V channels.
template <typename T, int V>
__device__ __forceinline__ void channel_param(const void* from, int c, float none, float (&v)[V]) {
    if (from) {
        seq_ldv<V>(static_cast<const T*>(from) + c, v);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = none;
    }
}

// Rows a thread has on their way at once.
template <bool BWD>
constexpr int GN_AHEAD = BWD ? 2 : 4;

// The sums of a slab: forward a channel's mean and sum of squared differences over the slab's tokens, backward the
// sums of dz and dz xhat.  Empty slabs write zeros.
template <typename T, int V, bool BWD, int ACT>
__global__ void __launch_bounds__(2 * GN_BLOCK) gn_sums_kernel(const __grid_constant__ SeqGnormParams p, int txn, int tyn) {
    constexpr int AHEAD = GN_AHEAD<BWD>;
    __shared__ float2 part[2 * GN_BLOCK][V + (V > 1)];
    const CutPiece cut = cut_piece(p.ax, blockIdx.x, p.slab);
    const GnPlace at(V, p.D, txn, tyn);
    const T* x = static_cast<const T*>(p.x) + (long long)cut.t0 * p.x_ld + at.c;
    const T* dy = BWD ? static_cast<const T*>(p.dy) + (long long)cut.t0 * p.dy_ld + at.c : nullptr;
    float a[V], b[V], shift[V];
    float mean[V], rstd[V], w[V], bias[V];
#pragma unroll
    for (int i = 0; i < V; ++i) a[i] = b[i] = shift[i] = 0.f;
    if (BWD && at.on && cut.n > 0) {
        channel_param<T, V>(p.w, at.c, 1.f, w);
        channel_param<T, V>(p.b, at.c, 0.f, bias);
        const int cpg = p.D / p.G;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float2 st = reinterpret_cast<const float2*>(p.coef)[(long long)cut.s * p.G + (at.c + i) / cpg];
            mean[i] = st.x;
            rstd[i] = st.y;
        }
    }
    int n = 0;
    if (at.on && cut.n > 0) {
        if (!BWD && at.ty < cut.n) seq_ldv<V>(x + at.ty * p.x_ld, shift);
        for (int t = at.ty; t < cut.n; t += AHEAD * tyn) {
            float v[AHEAD][V], d[BWD ? AHEAD : 1][V];
#pragma unroll
            for (int u = 0; u < AHEAD; ++u)
                if (t + u * tyn < cut.n) {
                    seq_ldv<V>(x + (t + u * tyn) * p.x_ld, v[u]);
                    if (BWD) seq_ldv<V>(dy + (t + u * tyn) * p.dy_ld, d[BWD ? u : 0]);
                }
#pragma unroll
            for (int u = 0; u < AHEAD; ++u)
                if (t + u * tyn < cut.n) {
                    ++n;
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        if (BWD) {
                            const float xh = (v[u][i] - mean[i]) * rstd[i];
                            const float dz = d[BWD ? u : 0][i] * slope_of<ACT>(fmaf(xh, w[i], bias[i]));
                            a[i] += dz;
                            b[i] = fmaf(dz, xh, b[i]);
                        } else {
                            const float e = v[u][i] - shift[i];
                            a[i] += e;
                            b[i] = fmaf(e, e, b[i]);
                        }
                    }
                }
        }
        if (!BWD && n > 0) {
#pragma unroll
            for (int i = 0; i < V; ++i) {           // mean and squared differences from it
                const float m = a[i] / (float)n;
                b[i] = fmaxf(fmaf(-a[i], m, b[i]), 0.f) + (b[i] - b[i]);      // (a NaN or infinity stays one)
                a[i] = shift[i] + m;
            }
        }
    }
    launch_next();
    if (at.ty < tyn) {
#pragma unroll
        for (int i = 0; i < V; ++i) part[threadIdx.x][i] = make_float2(a[i], b[i]);
    }
    __syncthreads();
    // the rows of threads in order; forward: row r has the tokens r, r + tyn, ... of the slab
    for (int j = threadIdx.x; j < txn * V; j += blockDim.x) {
        const int tx = j / V, i = j - tx * V, c = blockIdx.y * txn * V + j;
        if (c >= p.D) continue;
        float2 s = part[tx][i];
        float sn = (float)((cut.n + tyn - 1) / tyn);
        for (int r = 1; r < tyn && (BWD || r < cut.n); ++r) {
            const float2 o = part[r * txn + tx][i];
            if (BWD) {
                s.x += o.x;
                s.y += o.y;
            } else {
                const float on = (float)((cut.n - r + tyn - 1) / tyn), all = sn + on, d = o.x - s.x;
                s.x = fmaf(d, on / all, s.x);
                s.y += o.y + d * d * (sn * on / all);
                sn = all;
            }
        }
        reinterpret_cast<float2*>(p.part)[(long long)blockIdx.x * p.D + c] = cut.n > 0 ? s : make_float2(0.f, 0.f);
    }
}

// Sum over the threads of a group: the lanes of a warp, or all of a block of GN_BLOCK.
template <bool BLOCK>
__device__ __forceinline__ float group_sum(float v, float* buf) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    if (!BLOCK) return v;
    __syncthreads();
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < GN_BLOCK / 32; ++i) s += buf[i];
    return s;
}

// Statistics of a sequence and group from its slabs' and channels': a warp (BLOCK: a block) each.
template <bool BLOCK>
__global__ void __launch_bounds__(GN_BLOCK) gn_stats_kernel(const __grid_constant__ SeqGnormParams p) {
    __shared__ float buf[GN_BLOCK / 32];
    launch_next();
    wait_before();
    const long long at = BLOCK ? blockIdx.x : (long long)blockIdx.x * (GN_BLOCK / 32) + (threadIdx.x >> 5);
    if (at >= (long long)p.ax.S * p.G) return;          // (whole warps)
    const int s = (int)(at / p.G), gi = (int)(at - (long long)s * p.G), cpg = p.D / p.G;
    const int t0 = p.ax.L > 0 ? s * p.ax.L : seq_start(p.ax, s, 0), t1 = p.ax.L > 0 ? t0 + p.ax.L : seq_start(p.ax, s + 1, t0);
    const int len = t1 - t0, slabs = (len + p.slab - 1) / p.slab;
    const float2* from = reinterpret_cast<const float2*>(p.part) + (long long)cut_base(p.ax, s, p.slab) * p.D + gi * cpg;
    const int step = BLOCK ? GN_BLOCK : 32, first = BLOCK ? threadIdx.x : threadIdx.x & 31;
    const long long all = (long long)slabs * cpg;
    const float tokens = (float)p.slab, rest = (float)(len - (slabs - 1) * p.slab);
    float sum = 0.f, m2 = 0.f;
    // about the first slab's and channel's mean, so that small differences of large means survive
    const float about = len > 0 ? from[0].x : 0.f;
    for (long long i = first; i < all; i += step) {
        const int k = (int)(i / cpg);
        sum = fmaf((from[(long long)k * p.D + (i - (long long)k * cpg)].x - about), k == slabs - 1 ? rest : tokens, sum);
    }
    const float count = (float)len * (float)cpg;
    sum = group_sum<BLOCK>(sum, buf);
    const float shift = len > 0 ? sum / count : 0.f, mean = about + shift;
    for (long long i = first; i < all; i += step) {
        const int k = (int)(i / cpg);
        const float2 v = from[(long long)k * p.D + (i - (long long)k * cpg)];
        const float d = (v.x - about) - shift;
        m2 += fmaf(d * d, k == slabs - 1 ? rest : tokens, v.y);
    }
    m2 = group_sum<BLOCK>(m2, buf);
    if (first == 0) {
        const float2 st = len > 0 ? make_float2(mean, 1.f / sqrtf(m2 / count + p.eps)) : make_float2(0.f, 0.f);
        reinterpret_cast<float2*>(p.coef)[at] = st;
        if (p.stats) reinterpret_cast<float2*>(p.stats)[at] = st;
    }
}

// Backward: the group's means of dz w and dz w xhat.
template <typename T, bool BLOCK>
__global__ void __launch_bounds__(GN_BLOCK) gn_means_kernel(const __grid_constant__ SeqGnormParams p) {
    __shared__ float buf[GN_BLOCK / 32];
    launch_next();
    wait_before();
    const long long at = BLOCK ? blockIdx.x : (long long)blockIdx.x * (GN_BLOCK / 32) + (threadIdx.x >> 5);
    if (at >= (long long)p.ax.S * p.G) return;
    const int s = (int)(at / p.G), gi = (int)(at - (long long)s * p.G), cpg = p.D / p.G;
    const int t0 = p.ax.L > 0 ? s * p.ax.L : seq_start(p.ax, s, 0), t1 = p.ax.L > 0 ? t0 + p.ax.L : seq_start(p.ax, s + 1, t0);
    const int len = t1 - t0, slabs = (len + p.slab - 1) / p.slab;
    const float2* from = reinterpret_cast<const float2*>(p.part) + (long long)cut_base(p.ax, s, p.slab) * p.D + gi * cpg;
    const int step = BLOCK ? GN_BLOCK : 32, first = BLOCK ? threadIdx.x : threadIdx.x & 31;
    const T* w = static_cast<const T*>(p.w);
    float m1 = 0.f, m2 = 0.f;
    for (long long i = first; i < (long long)slabs * cpg; i += step) {
        const int k = (int)(i / cpg), c = (int)(i - (long long)k * cpg);
        const float2 v = from[(long long)k * p.D + c];
        const float wc = w ? seq_ld(w + gi * cpg + c) : 1.f;
        m1 = fmaf(wc, v.x, m1);
        m2 = fmaf(wc, v.y, m2);
    }
    m1 = group_sum<BLOCK>(m1, buf);
    m2 = group_sum<BLOCK>(m2, buf);
    if (first == 0) {
        const float count = (float)len * (float)cpg;
        reinterpret_cast<float2*>(p.coef)[at] = len > 0 ? make_float2(m1 / count, m2 / count) : make_float2(0.f, 0.f);
    }
}

// dw and db: the slabs' sums of all sequences in order.
__global__ void __launch_bounds__(COLUMN_THREADS, 2) gn_param_kernel(const __grid_constant__ SeqGnormParams p) {
    wait_before();
    const long long col = (long long)blockIdx.x * 32 + (threadIdx.x & 31);      // db and dw of a channel side by side
    const bool on = col < 2LL * p.D;
    const float v = column_sum(p.part + col, 2LL * p.D, p.slots, on);
    if (threadIdx.x < 32 && on) {
        float* to = col & 1 ? p.dw : p.db;
        if (to) to[col >> 1] = v;
    }
}

// y, or dx, of a slab.
template <typename T, int V, bool BWD, int ACT>
__global__ void __launch_bounds__(2 * GN_BLOCK) gn_apply_kernel(const __grid_constant__ SeqGnormParams p, int txn, int tyn) {
    constexpr int AHEAD = GN_AHEAD<BWD>;
    const CutPiece cut = cut_piece(p.ax, gridDim.x - 1 - blockIdx.x, p.slab);
    const GnPlace at(V, p.D, txn, tyn);
    float w[V], bias[V], mean[V], rstd[V];
    const bool on = at.on && at.ty < tyn && cut.n > 0;
    if (on) {
        channel_param<T, V>(p.w, at.c, 1.f, w);
        channel_param<T, V>(p.b, at.c, 0.f, bias);
    }
    wait_before();
    if (!on) return;
    const int cpg = p.D / p.G;
    const float2* stats = reinterpret_cast<const float2*>(BWD ? p.stats : p.coef) + (long long)cut.s * p.G;
    float m1[BWD ? V : 1], m2[BWD ? V : 1];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int gi = (at.c + i) / cpg;
        if (BWD) {
            const float2 m = reinterpret_cast<const float2*>(p.coef)[(long long)cut.s * p.G + gi];
            m1[BWD ? i : 0] = m.x;
            m2[BWD ? i : 0] = m.y;
        }
        const float2 st = stats[gi];
        mean[i] = st.x;
        rstd[i] = st.y;
    }
    const T* x = static_cast<const T*>(p.x) + (long long)cut.t0 * p.x_ld + at.c;
    const T* dy = BWD ? static_cast<const T*>(p.dy) + (long long)cut.t0 * p.dy_ld + at.c : nullptr;
    T* to = static_cast<T*>(BWD ? p.dx : p.y) + (long long)cut.t0 * (BWD ? p.dx_ld : p.y_ld) + at.c;
    const long long to_ld = BWD ? p.dx_ld : p.y_ld;
    for (int t = at.ty; t < cut.n; t += AHEAD * tyn) {
        float v[AHEAD][V], d[BWD ? AHEAD : 1][V];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
            if (t + u * tyn < cut.n) {
                seq_ldv<V>(x + (t + u * tyn) * p.x_ld, v[u]);
                if (BWD) seq_ldv<V>(dy + (t + u * tyn) * p.dy_ld, d[BWD ? u : 0]);
            }
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
            if (t + u * tyn < cut.n) {
                float out[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float xh = (v[u][i] - mean[i]) * rstd[i];
                    const float z = fmaf(xh, w[i], bias[i]);
                    if (BWD) {
                        const float dn = d[BWD ? u : 0][i] * slope_of<ACT>(z) * w[i];
                        out[i] = rstd[i] * ((dn - m1[BWD ? i : 0]) - xh * m2[BWD ? i : 0]);
                    } else {
                        out[i] = act_of<ACT>(z);
                    }
                }
                seq_stv<V>(to + (t + u * tyn) * to_ld, out);
            }
    }
}

template <typename T, int V, bool BWD, int ACT>
cudaError_t launch_act(const SeqGnormParams& p, cudaStream_t stream) {
    const GnShape s = gn_shape(p.D, V);
    const dim3 grid((unsigned)p.slots, (unsigned)s.cblocks), block((unsigned)(s.tx * s.ty));
    SeqGnormParams sums = p;
    if (BWD) sums.coef = p.stats;                      // (the sums need the forward call's statistics there)
    cudaError_t e = launch_kernel(gn_sums_kernel<T, V, BWD, ACT>, grid, block, 0, stream, false, 1, sums, s.tx, s.ty);
    if (e != cudaSuccess) return e;
    const long long groups = (long long)p.ax.S * p.G;
    // entries of a sequence's group: with few of them a warp each, else a block
    const long long entries = (long long)(p.ax.T / p.ax.S / p.slab + 1) * (p.D / p.G);
    const bool big = entries > 512;
    const dim3 sgrid((unsigned)(big ? groups : (groups + GN_BLOCK / 32 - 1) / (GN_BLOCK / 32)));
    if (BWD)
        e = launch_kernel(big ? gn_means_kernel<T, true> : gn_means_kernel<T, false>, sgrid, dim3(GN_BLOCK), 0, stream, true, 1, p);
    else
        e = launch_kernel(big ? gn_stats_kernel<true> : gn_stats_kernel<false>, sgrid, dim3(GN_BLOCK), 0, stream, true, 1, p);
    if (e == cudaSuccess) e = launch_kernel(gn_apply_kernel<T, V, BWD, ACT>, grid, block, 0, stream, true, 1, p, s.tx, s.ty);
    if (BWD && e == cudaSuccess && (p.dw || p.db))
        e = launch_kernel(gn_param_kernel, dim3((unsigned)((2LL * p.D + 31) / 32)), dim3(COLUMN_THREADS), 0, stream, false, 1, p);
    return e;
}

template <typename T, bool BWD>
cudaError_t launch(const SeqGnormParams& p, cudaStream_t stream) {
    if (p.slots == 0) return cudaSuccess;
    if (p.vec) {
        if (p.act == SEQ_ACT_SILU) return launch_act<T, 8, BWD, SEQ_ACT_SILU>(p, stream);
        if (p.act == SEQ_ACT_GELU) return launch_act<T, 8, BWD, SEQ_ACT_GELU>(p, stream);
        return launch_act<T, 8, BWD, 0>(p, stream);
    }
    if (p.act == SEQ_ACT_SILU) return launch_act<T, 1, BWD, SEQ_ACT_SILU>(p, stream);
    if (p.act == SEQ_ACT_GELU) return launch_act<T, 1, BWD, SEQ_ACT_GELU>(p, stream);
    return launch_act<T, 1, BWD, 0>(p, stream);
}

}  // namespace

// Tokens of a slab: about four blocks of 256 threads an SM, 8 tokens at least and 256 at most.
int seq_gnorm_slab(long long S, long long T, int D, int sms) {
    const GnShape s = gn_shape(D, 8);
    const long long L = S > 0 && T > S ? T / S : 1, want = 4LL * sms;
    long long slabs = want / ((S < 1 ? 1 : S) * s.cblocks);          // of a sequence
    if (slabs < 1) slabs = 1;
    long long len = (L + slabs - 1) / slabs;
    const long long least = 8 * (s.ty < 1 ? 1 : s.ty) > 64 ? 64 : 8;
    if (len < least) len = least;
    return (int)(len > 256 ? 256 : len);
}

cudaError_t launch_seq_gnorm_fwd(const SeqGnormParams& p, bool bf16, cudaStream_t stream) {
    return bf16 ? launch<__nv_bfloat16, false>(p, stream) : launch<float, false>(p, stream);
}
cudaError_t launch_seq_gnorm_bwd(const SeqGnormParams& p, bool bf16, cudaStream_t stream) {
    return bf16 ? launch<__nv_bfloat16, true>(p, stream) : launch<float, true>(p, stream);
}

}  // namespace convfwd

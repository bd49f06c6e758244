// Short causal depthwise convolution over packed sequences (forward, one-token step, gradients).
//
//   pre[t] = bias + sum_j w[j] x[t - W + 1 + j],  y = silu(pre) or pre
//
// A few multiply-adds a value: bound by the bytes of x and y (dy, dx).  A thread owns V consecutive channels
// (as packed pairs) and walks a run of tokens with the last W inputs in registers, so each row is read once,
// plus W - 1 rows at the start of a run.  The inputs lie in a ring of W slots; tokens are unrolled in groups of
// a multiple of W, so that every token's slots are known to the compiler and nothing moves.  The next group's
// rows are on their way while this one is computed.
//
// 8 x 2048 x 4096 bf16, 4 taps, silu: forward 46 us (268 MB: 5.8 TB/s, 87% of a plain copy's rate), backward 90 us
// (403 MB: 4.5 TB/s; a sigmoid and 12 multiply-adds a value, 0.55 instructions a clock and scheduler at the 15 warps
// an SM that the registers of its windows and sums allow).
#include <type_traits>

#include "seq_common.cuh"
#include "seq_internal.h"

namespace convfwd {
namespace {

constexpr int BWD_LANES = 32, BWD_ROWS = 8;   // backward block: channel vectors x runs
// Tokens in a group: about 8 forward, 4 backward (where x and dy are on their way).
__host__ __device__ constexpr int group_of(int W, int about) { return W == 1 || W == 2 || W == 4 ? about : W; }

// V values as loaded, and as pairs (one value: a pair with nothing in its second place).
template <typename T, int V>
struct RowVec {
    static constexpr int P = V == 1 ? 1 : V / 2;
    using Q = typename std::conditional<sizeof(T) * V == 16, uint4, typename std::conditional<sizeof(T) * V == 8, uint2, T>::type>::type;
    Q q;
    __device__ __forceinline__ void load(const T* p) { q = *reinterpret_cast<const Q*>(p); }
    __device__ __forceinline__ void get(float2 (&v)[P]) const {
        const T* e = reinterpret_cast<const T*>(&q);
        if constexpr (V == 1) {
            v[0] = make_float2(seq_ld(e), 0.f);
        } else {
#pragma unroll
            for (int i = 0; i < P; ++i) v[i] = seq_ld2(e + 2 * i);
        }
    }
};
template <typename T, int V>
__device__ __forceinline__ void row_put(T* p, const float2 (&v)[V == 1 ? 1 : V / 2]) {
    if constexpr (V == 1) {
        seq_st(p, v[0].x);
    } else {
        float w[V];
#pragma unroll
        for (int i = 0; i < V / 2; ++i) w[2 * i] = v[i].x, w[2 * i + 1] = v[i].y;
        seq_stv<V>(p, w);
    }
}

// One input before the token at position pos of sequence s, `back` positions before it: from x (`at` is the
// token's row) or, before the sequence's first token, from its state.
template <typename T, int V>
__device__ __forceinline__ void load_before(const SeqConvParams& p, long long slot, const T* at, int pos, int back, int c,
                                            float2 (&v)[V == 1 ? 1 : V / 2]) {
    RowVec<T, V> r;
    if (pos >= back) {
        r.load(at - back * p.x_ld);
        r.get(v);
    } else if (slot >= 0) {
        r.load(static_cast<const T*>(p.state_in) + (slot * (p.W - 1) + pos + p.W - 1 - back) * p.D + c);
        r.get(v);
    } else {
#pragma unroll
        for (int i = 0; i < (V == 1 ? 1 : V / 2); ++i) v[i] = make_float2(0.f, 0.f);
    }
}
__device__ __forceinline__ long long state_slot(const SeqConvParams& p, int s) { return p.state_in ? seq_slot(p.sl, s) : -1; }

template <typename T, int V, int W>
__device__ __forceinline__ void load_params(const SeqConvParams& p, int c, float2 (&w)[W][V == 1 ? 1 : V / 2], float2 (&b)[V == 1 ? 1 : V / 2]) {
    constexpr int P = V == 1 ? 1 : V / 2, BYTES = V * W * (int)sizeof(T);
    auto at = [&](const void* from, long long i) { return seq_ld(static_cast<const T*>(from) + i); };
    if (BYTES % 8 == 0 && reinterpret_cast<uintptr_t>(p.w) % 8 == 0) {          // the channels' taps lie together
        uint2 q[BYTES / 8 + 1];
#pragma unroll
        for (int i = 0; i < BYTES / 8; ++i) q[i] = reinterpret_cast<const uint2*>(static_cast<const T*>(p.w) + (long long)c * W)[i];
        auto tap = [&](int i) {
            if constexpr (sizeof(T) == 2) {
                const uint32_t two = i & 2 ? q[i / 4].y : q[i / 4].x;
                return __uint_as_float(i & 1 ? two & 0xffff0000u : two << 16);
            } else {
                return __uint_as_float(i & 1 ? q[i / 2].y : q[i / 2].x);
            }
        };
#pragma unroll
        for (int i = 0; i < P; ++i)
#pragma unroll
            for (int j = 0; j < W; ++j) w[j][i] = make_float2(tap(2 * i * W + j), V == 1 ? 0.f : tap((2 * i + (V > 1)) * W + j));
    } else {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const long long c0 = c + 2 * i, c1 = V == 1 ? c0 : c0 + 1;
#pragma unroll
            for (int j = 0; j < W; ++j) w[j][i] = make_float2(at(p.w, c0 * W + j), V == 1 ? 0.f : at(p.w, c1 * W + j));
        }
    }
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const long long c0 = c + 2 * i, c1 = V == 1 ? c0 : c0 + 1;
        b[i] = p.bias ? make_float2(at(p.bias, c0), V == 1 ? 0.f : at(p.bias, c1)) : make_float2(0.f, 0.f);
    }
}

// The sequence that holds token t, and where it begins and ends.
struct Place {
    int s, begin, end;
};
__device__ __forceinline__ Place place_of(const SeqAxis& ax, int t) {
    Place q;
    // the last sequence that starts at or before t: a ragged axis is searched in eight parts a step, whose bounds
    // are read together, so that a step costs one wait for memory
    if (ax.L > 0) {
        q.s = min(t / ax.L, ax.S - 1);
    } else {
        int lo = 0, hi = ax.S;
        while (lo < hi) {
            const int step = (hi - lo + 7) >> 3;
            int less = 0;
#pragma unroll
            for (int k = 1; k <= 8; ++k) {
                const int m = lo + k * step;
                if (m <= hi && seq_start(ax, m - 1, 0) <= t) less = k;
            }
            lo += less * step;
            hi = min(hi, lo + step - 1);
        }
        q.s = lo - 1;
    }
    q.begin = q.s < 0 ? 0 : seq_start(ax, q.s, 0);
    q.end = seq_start(ax, q.s + 1, t + 1);
    return q;
}
// The next sequence that holds token t (t: the end of the current one).
__device__ __forceinline__ void next_place(const SeqAxis& ax, int t, Place& q) {
    do {
        ++q.s;
        q.end = seq_start(ax, q.s + 1, t);
    } while (q.end == t && q.s + 1 < ax.S);
    q.begin = t;
}

template <typename T, int V, int W>
__global__ void __launch_bounds__(128, 4) seq_conv_fwd_kernel(const __grid_constant__ SeqConvParams p) {
    constexpr int P = RowVec<T, V>::P, GROUP = group_of(W, 8);
    const int c = (blockIdx.y * 128 + threadIdx.x) * V;
    if (c >= p.D) return;
    const int t0 = blockIdx.x * p.run, t1 = min(t0 + p.run, p.ax.T);
    griddep_launch();
    const T* x = static_cast<const T*>(p.x) + (long long)t0 * p.x_ld + c;
    T* y = static_cast<T*>(p.y) + (long long)t0 * p.y_ld + c;
    RowVec<T, V> next[GROUP];
    const T* ahead = x;
    auto fetch = [&](int t) {
#pragma unroll
        for (int i = 0; i < GROUP; ++i) {
            if (t + i < t1) next[i].load(ahead);
            ahead += p.x_ld;
        }
    };
    fetch(t0);
    float2 w[W][P], b[P], win[W][P];          // the token with i = t - t0 mod W has its input in slot i
    load_params<T, V, W>(p, c, w, b);
    Place q = place_of(p.ax, t0);
    auto window = [&](int i, int t, const T* at) {          // the inputs before token t of slot i
        const long long slot = state_slot(p, q.s);
#pragma unroll
        for (int k = 1; k < W; ++k) load_before<T, V>(p, slot, at, t - q.begin, k, c, win[(i + W - k) % W]);
    };
    window(0, t0, x);
    for (int tb = t0; tb < t1; tb += GROUP) {
        RowVec<T, V> rows[GROUP];
#pragma unroll
        for (int i = 0; i < GROUP; ++i) rows[i] = next[i];
        if (tb + GROUP < t1) fetch(tb + GROUP);
#pragma unroll
        for (int i = 0; i < GROUP; ++i) {
            const int t = tb + i;
            if (t < t1) {
                if (t == q.end) {
                    next_place(p.ax, t, q);
                    window(i % W, t, x);
                }
                rows[i].get(win[i % W]);
                float2 o[P];
#pragma unroll
                for (int v = 0; v < P; ++v) {
                    float2 a = b[v];
#pragma unroll
                    for (int j = 0; j < W; ++j) a = __ffma2_rn(w[j][v], win[(i + 1 + j) % W][v], a);
                    o[v] = p.silu ? __fmul2_rn(a, make_float2(sigmoid(a.x), V == 1 ? 0.f : sigmoid(a.y))) : a;
                }
                row_put<T, V>(y, o);
                x += p.x_ld;
                y += p.y_ld;
            }
        }
    }
}

// The states after the last tokens.  A launch of its own behind the forward kernel: with
// state_out == state_in a thread there may still read the state that this one replaces.  It starts while that
// one runs, and waits for its end only between its loads and its stores.
template <typename T, int V, int W>
__global__ void __launch_bounds__(128) seq_conv_state_kernel(const __grid_constant__ SeqConvParams p) {
    const int c = (blockIdx.x * 128 + threadIdx.x) * V;
    bool waited = false;
    for (int s = blockIdx.y; s < p.ax.S; s += gridDim.y) {
        const long long to = seq_slot(p.sl, s);
        if (to < 0 || c >= p.D) continue;
        const int begin = seq_start(p.ax, s, 0), end = seq_start(p.ax, s + 1, begin);
        const T* x = static_cast<const T*>(p.x) + (long long)end * p.x_ld + c;
        float2 win[W][RowVec<T, V>::P];
#pragma unroll
        for (int k = 1; k < W; ++k) load_before<T, V>(p, state_slot(p, s), x, end - begin, k, c, win[W - k]);
        if (!waited) griddep_wait();
        waited = true;
#pragma unroll
        for (int k = 1; k < W; ++k) row_put<T, V>(static_cast<T*>(p.state_out) + (to * (W - 1) + W - 1 - k) * p.D + c, win[W - k]);
    }
    if (!waited) griddep_wait();
}

// One token per sequence: row s of x follows the W - 1 rows of its state.
template <typename T, int V, int W>
__global__ void __launch_bounds__(128) seq_conv_step_kernel(const __grid_constant__ SeqConvParams p) {
    constexpr int P = RowVec<T, V>::P;
    const int c = (blockIdx.x * 128 + threadIdx.x) * V;
    if (c >= p.D) return;
    float2 w[W][P], b[P];
    load_params<T, V, W>(p, c, w, b);
    for (int s = blockIdx.y; s < p.ax.S; s += gridDim.y) {
        float2 win[W][P], o[P];
        const long long slot = seq_slot(p.sl, s);
        const T* x = static_cast<const T*>(p.x) + (long long)s * p.x_ld + c;
#pragma unroll
        for (int k = 0; k < W; ++k) load_before<T, V>(p, state_slot(p, s), x, 0, k, c, win[W - 1 - k]);
#pragma unroll
        for (int v = 0; v < P; ++v) {
            float2 a = b[v];
#pragma unroll
            for (int j = 0; j < W; ++j) a = __ffma2_rn(w[j][v], win[j][v], a);
            o[v] = p.silu ? __fmul2_rn(a, make_float2(sigmoid(a.x), V == 1 ? 0.f : sigmoid(a.y))) : a;
        }
        row_put<T, V>(static_cast<T*>(p.y) + (long long)s * p.y_ld + c, o);
        if (p.state_out && slot >= 0) {
#pragma unroll
            for (int j = 0; j < W - 1; ++j) row_put<T, V>(static_cast<T*>(p.state_out) + (slot * (W - 1) + j) * p.D + c, win[j + 1]);
        }
    }
}

// Gradients.  dpre[t] = dy[t] silu'(pre[t]); dx[t] = sum_j w[j] dpre[t + W - 1 - j] over the tokens
// of t's sequence; dw[j] = sum_t dpre[t] x[t - W + 1 + j]; dbias = sum_t dpre[t].
// A thread walks its run and W - 1 tokens behind it (they see its last inputs), keeps the last
// W values of dpre in slots as its inputs, and emits dx with a delay of W - 1 tokens.  The parameter sums of
// the block's runs meet in shared memory in a fixed order and leave as one partial row per block.
// LAYERS: rows of more channel blocks than a launch's second dimension takes lie on the third as well.  Kernels of
// their own: the third index in the others costs 4 taps of bf16 8 bytes of spilled registers and 144 -> 172 us
// a training pass of 8 x 2048 x 4096.
template <typename T, int V, int W, bool LAYERS = false>
__global__ void __launch_bounds__(BWD_LANES * BWD_ROWS, W <= 4 ? 2 : 1) seq_conv_bwd_kernel(const __grid_constant__ SeqConvParams p) {
    constexpr int P = RowVec<T, V>::P, GROUP = group_of(W, 4);
    __shared__ float sums[BWD_ROWS][BWD_LANES * V + 1];
    const int lane = threadIdx.x % BWD_LANES, row = threadIdx.x / BWD_LANES;
    const int cblock = LAYERS ? blockIdx.z * gridDim.y + blockIdx.y : blockIdx.y;
    const int c = (cblock * BWD_LANES + lane) * V;
    const int t0 = (int)min(((long long)blockIdx.x * BWD_ROWS + row) * p.run, (long long)p.ax.T);
    const int t1 = min(t0 + p.run, p.ax.T);
    float2 acc[W + 1][P];
#pragma unroll
    for (int j = 0; j <= W; ++j)
#pragma unroll
        for (int v = 0; v < P; ++v) acc[j][v] = make_float2(0.f, 0.f);
    if (c < p.D && t0 < t1) {
        // the run, and behind it the tokens of the same sequence that its last inputs reach
        Place q = place_of(p.ax, t0);
        int t2 = min(t1 + W - 1, p.ax.T);
        RowVec<T, V> xn[GROUP], dn[GROUP];
        const T* x = static_cast<const T*>(p.x) + (long long)t0 * p.x_ld + c;
        const T* x_ahead = x;
        const T* dy = static_cast<const T*>(p.dy) + (long long)t0 * p.dy_ld + c;
        T* dx = static_cast<T*>(p.dx) + ((long long)t0 - (W - 1)) * p.dx_ld + c;      // of token t - W + 1
        auto fetch = [&](int t) {
#pragma unroll
            for (int i = 0; i < GROUP; ++i) {
                if (t + i < t2) {
                    xn[i].load(x_ahead);
                    dn[i].load(dy);
                }
                x_ahead += p.x_ld;
                dy += p.dy_ld;
            }
        };
        fetch(t0);
        float2 w[W][P], b[P], win[W][P], dp[W][P];
        load_params<T, V, W>(p, c, w, b);
        auto window = [&](int i, int t) {
            const long long slot = state_slot(p, q.s);
#pragma unroll
            for (int k = 1; k < W; ++k) load_before<T, V>(p, slot, x, t - q.begin, k, c, win[(i + W - k) % W]);
#pragma unroll
            for (int j = 0; j < W; ++j)
#pragma unroll
                for (int v = 0; v < P; ++v) dp[j][v] = make_float2(0.f, 0.f);
        };
        window(0, t0);
        // The sequence ends before token t, whose slot would be i: dx of its last W - 1 tokens, those before
        // the run apart, from the dpre there are.
        auto flush = [&](int i, int t) {
#pragma unroll
            for (int k = W - 1; k >= 1; --k) {                  // token t - k
                const int m = t - k;
                if (m < t0 || m < q.begin || m >= t1) continue;
                float2 o[P];
#pragma unroll
                for (int v = 0; v < P; ++v) {
                    o[v] = make_float2(0.f, 0.f);
#pragma unroll
                    for (int u = k; u >= 1; --u) o[v] = __ffma2_rn(w[W - 1 - (k - u)][v], dp[(i + W - u) % W][v], o[v]);
                }
                row_put<T, V>(static_cast<T*>(p.dx) + (long long)m * p.dx_ld + c, o);
            }
        };
        for (int tb = t0; tb < t2; tb += GROUP) {
            RowVec<T, V> xr[GROUP], dr[GROUP];
#pragma unroll
            for (int i = 0; i < GROUP; ++i) {
                xr[i] = xn[i];
                dr[i] = dn[i];
            }
            if (tb + GROUP < t2) fetch(tb + GROUP);
#pragma unroll
            for (int i = 0; i < GROUP; ++i) {
                const int t = tb + i;
                if (t < t2) {
                    if (t == q.end) {
                        flush(i % W, t);
                        if (t >= t1) {
                            t2 = t;                              // the tokens behind are of another sequence
                        } else {
                            next_place(p.ax, t, q);
                            window(i % W, t);
                        }
                    }
                }
                if (t < t2) {
                    xr[i].get(win[i % W]);
                    dr[i].get(dp[i % W]);
#pragma unroll
                    for (int v = 0; v < P; ++v) {
                        float2 d = dp[i % W][v];
                        if (p.silu) {
                            float2 a = b[v];
#pragma unroll
                            for (int j = 0; j < W; ++j) a = __ffma2_rn(w[j][v], win[(i + 1 + j) % W][v], a);
                            // silu' = s (1 + a (1 - s))
                            const float2 s = make_float2(sigmoid(a.x), V == 1 ? 0.f : sigmoid(a.y)), one = make_float2(1.f, 1.f);
                            d = __fmul2_rn(__fmul2_rn(d, s), __ffma2_rn(a, __fadd2_rn(one, make_float2(-s.x, -s.y)), one));
                            dp[i % W][v] = d;
                        }
                        if (t < t1) {
#pragma unroll
                            for (int j = 0; j < W; ++j) acc[j][v] = __ffma2_rn(d, win[(i + 1 + j) % W][v], acc[j][v]);
                            acc[W][v] = __fadd2_rn(acc[W][v], d);
                        }
                    }
                    const int m = t - (W - 1);
                    if (m >= t0 && m >= q.begin) {               // (m < t1: t < t2)
                        float2 o[P];
#pragma unroll
                        for (int v = 0; v < P; ++v) {
                            o[v] = make_float2(0.f, 0.f);
#pragma unroll
                            for (int j = 0; j < W; ++j) o[v] = __ffma2_rn(w[W - 1 - j][v], dp[(i + 1 + j) % W][v], o[v]);
                        }
                        row_put<T, V>(dx, o);
                    }
                    x += p.x_ld;
                    dx += p.dx_ld;
                }
            }
            // (the slots of the next group's tokens continue these: GROUP is a multiple of W)
            if (tb + GROUP >= t2 && q.end == t2 && t2 < t1 + W - 1) {
                // the axis ends: nothing follows to flush the last tokens
#pragma unroll
                for (int i = 0; i < GROUP; ++i)
                    if (t2 - tb == i + 1) flush((i + 1) % W, t2);
            }
        }
    }
    griddep_launch();
#pragma unroll
    for (int j = 0; j <= W; ++j) {
        __syncthreads();
#pragma unroll
        for (int v = 0; v < P; ++v) {
            sums[row][lane * V + 2 * v] = acc[j][v].x;
            if (V > 1) sums[row][lane * V + 2 * v + 1] = acc[j][v].y;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < BWD_LANES * V; i += BWD_LANES * BWD_ROWS) {
            const int d = cblock * BWD_LANES * V + i;
            if (d >= p.D) break;
            float s = 0.f;
#pragma unroll
            for (int r = 0; r < BWD_ROWS; ++r) s += sums[r][i];
            p.ws[((long long)blockIdx.x * (W + 1) + j) * p.D + d] = s;
        }
    }
}

// dw and dbias: the blocks' rows of partial sums, added up in a fixed order.
__global__ void __launch_bounds__(COLUMN_THREADS, 2) seq_conv_param_kernel(const __grid_constant__ SeqConvParams p) {
    const int d = blockIdx.x * 32 + (threadIdx.x & 31), j = blockIdx.y;
    griddep_wait();
    const float v = column_sum(p.ws + (long long)j * p.D + d, (long long)(p.W + 1) * p.D, p.tblocks, d < p.D);
    if (threadIdx.x >= 32 || d >= p.D) return;
    if (j < p.W) p.dw[(long long)d * p.W + j] = v;
    else if (p.dbias) p.dbias[d] = v;
}

enum class Pass { Fwd, Bwd, Step };

template <typename T, int V, int W>
cudaError_t launch_w(const SeqConvParams& p, Pass pass, cudaStream_t stream) {
    const unsigned cb = (unsigned)((p.D + 128 * V - 1) / (128 * V));
    const unsigned sb = (unsigned)(p.ax.S < 32768 ? p.ax.S : 32768);
    constexpr int V4 = V < 4 ? V : 4, VB = V < 4 ? V : sizeof(T) == 2 ? 4 : 2;
    cudaError_t e = cudaSuccess;
    if (pass == Pass::Step)
        return launch_kernel(seq_conv_step_kernel<T, V, W>, dim3(cb, sb), dim3(128), 0, stream, false, 1, p);
    if (pass == Pass::Fwd) {
        if (p.ax.T > 0)
            e = launch_kernel(seq_conv_fwd_kernel<T, V4, W>,
                              dim3((unsigned)((p.ax.T + p.run - 1) / p.run), (unsigned)((p.D + 128 * V4 - 1) / (128 * V4))), dim3(128), 0,
                              stream, false, 1, p);
        if (e == cudaSuccess && p.state_out && W > 1)
            e = launch_kernel(seq_conv_state_kernel<T, V, W>, dim3(cb, sb), dim3(128), 0, stream, p.ax.T > 0, 1, p);
        return e;
    }
    if (p.ax.T > 0) {
        const unsigned most = 65535, blocks = (unsigned)((p.D + BWD_LANES * VB - 1) / (BWD_LANES * VB));
        const unsigned single = (unsigned)((p.D + BWD_LANES - 1) / BWD_LANES), layers = (single + most - 1) / most;
        e = blocks <= most ? launch_kernel(seq_conv_bwd_kernel<T, VB, W>, dim3((unsigned)p.tblocks, blocks), dim3(BWD_LANES * BWD_ROWS), 0,
                                           stream, false, 1, p)
                           : launch_kernel(seq_conv_bwd_kernel<T, 1, W, true>, dim3((unsigned)p.tblocks, (single + layers - 1) / layers, layers),
                                           dim3(BWD_LANES * BWD_ROWS), 0, stream, false, 1, p);
    }
    if (e == cudaSuccess)
        e = launch_kernel(seq_conv_param_kernel, dim3((unsigned)((p.D + 31) / 32), (unsigned)(W + 1)), dim3(COLUMN_THREADS), 0,
                          stream, p.ax.T > 0, 1, p);
    return e;
}

// Over whole sequences a thread has 4 channels (8 bytes of bf16, 16 of fp32; backward 8 of fp32): with 8
// channels the windows, sums and weights of 4 taps alone are 136 registers backward, and with 4 of fp32 the
// rows on their way are 64 (1500 x 8 x 1280: 68 us, spilling).
template <typename T, int V>
cudaError_t launch_v(const SeqConvParams& p, Pass pass, cudaStream_t stream) {
    switch (p.W) {
        case 1: return launch_w<T, V, 1>(p, pass, stream);
        case 2: return launch_w<T, V, 2>(p, pass, stream);
        case 3: return launch_w<T, V, 3>(p, pass, stream);
        case 4: return launch_w<T, V, 4>(p, pass, stream);
        case 5: return launch_w<T, V, 5>(p, pass, stream);
        case 6: return launch_w<T, V, 6>(p, pass, stream);
        case 7: return launch_w<T, V, 7>(p, pass, stream);
        default: return launch_w<T, V, 8>(p, pass, stream);
    }
}

cudaError_t launch(const SeqConvParams& p, bool bf16, Pass pass, cudaStream_t stream) {
    if (bf16) return p.vec ? launch_v<__nv_bfloat16, 8>(p, pass, stream) : launch_v<__nv_bfloat16, 1>(p, pass, stream);
    return p.vec ? launch_v<float, 4>(p, pass, stream) : launch_v<float, 1>(p, pass, stream);
}

}  // namespace

// Tokens a thread walks, 8 to 256: whole rounds of resident blocks (4, 5 or 8 an SM forward, 2 or 1 backward, as the
// kernels of 4 taps fit; fewer taps leave room for more: bf16 forward 6 at 2 taps and 7 at 3), where
// a round costs its run and, for the several waits for memory before a thread's first token (its sequence, its
// window, its weights), about `start` tokens more.  (Two rounds of 512 threads an SM instead, whatever is left
// over: 6011 x 2560 ragged bf16 25.9 us, here 20.6; 8 x 2048 x 4096 bf16 forward and backward 154, here 144; 8 x 1500 x
// 1280 fp32 89, here 76.)
int seq_conv_run(long long T, int D, int W, bool bf16, bool bwd, int sms) {
    const bool vec = D * (bf16 ? 2 : 4) % 16 == 0;
    const int columns = bwd ? BWD_LANES * (!vec ? 1 : bf16 ? 4 : 2) : 128 * (vec ? 4 : 1), rows = bwd ? BWD_ROWS : 1;
    const long long cb = (D + columns - 1) / columns, slots = (bwd ? (W <= 4 ? 2ll : 1ll) : !vec ? 8ll : bf16 ? 5ll : 4ll) * sms;
    const int start = bwd ? 16 : 12;
    long long best = 0;
    int run = 8;
    for (int r = 8; r <= 256; r += 8) {
        const long long blocks = (T + (long long)r * rows - 1) / ((long long)r * rows) * cb;
        const long long cost = (blocks + slots - 1) / slots * (r + start);
        if (r == 8 || cost < best) best = cost, run = r;
    }
    return run;
}
int seq_conv_bwd_token_blocks(long long T, int run) { return (int)((T + (long long)run * BWD_ROWS - 1) / ((long long)run * BWD_ROWS)); }
cudaError_t launch_seq_conv_fwd(const SeqConvParams& p, bool bf16, cudaStream_t stream) { return launch(p, bf16, Pass::Fwd, stream); }
cudaError_t launch_seq_conv_bwd(const SeqConvParams& p, bool bf16, cudaStream_t stream) { return launch(p, bf16, Pass::Bwd, stream); }
cudaError_t launch_seq_conv_step(const SeqConvParams& p, bool bf16, cudaStream_t stream) { return launch(p, bf16, Pass::Step, stream); }

}  // namespace convfwd

// Short causal depthwise convolution over packed sequences (forward, one-token step, gradients).
//
//   pre[t] = bias + sum_j w[j] x[t - W + 1 + j],  y = silu(pre) or pre
//
// A few multiply-adds a value: every kernel here is bound by the bytes of x and y (dy, dx).
// A thread owns V consecutive channels (16 bytes of a row) and walks a run of tokens with the
// last W inputs in registers, so each row is read once, plus W - 1 rows at the start of a run.
#include "seq_common.cuh"
#include "seq_internal.h"

namespace convfwd {
namespace {

constexpr int FWD_RUN = 16;      // tokens per thread, forward
constexpr int BWD_RUN = 32;      // tokens per thread, backward
constexpr int BWD_LANES = 32, BWD_ROWS = 8;   // backward block: channel vectors x runs

// The window before the token at position pos of sequence s: positions pos - (W-1) .. pos - 1,
// oldest first, from x or (before the first token) from the sequence's state.
template <typename T, int V, int W>
__device__ __forceinline__ void load_window(const SeqConvParams& p, int s, int t, int pos, int c, float (&win)[W][V]) {
    const long long slot = p.state_in ? seq_slot(p.sl, s) : -1;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const int q = pos - (W - 1) + j;
        if (q >= 0) {
            seq_ldv<V>(static_cast<const T*>(p.x) + (long long)(t - (W - 1) + j) * p.x_ld + c, win[j]);
        } else if (slot >= 0) {
            seq_ldv<V>(static_cast<const T*>(p.state_in) + (slot * (W - 1) + pos + j) * p.D + c, win[j]);
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) win[j][v] = 0.f;
        }
    }
}

template <typename T, int V, int W>
__device__ __forceinline__ void load_params(const SeqConvParams& p, int c, float (&w)[W][V], float (&b)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][v] = seq_ld(static_cast<const T*>(p.w) + (long long)(c + v) * W + j);
        b[v] = p.bias ? seq_ld(static_cast<const T*>(p.bias) + c + v) : 0.f;
    }
}

// The sequence that holds token t, and where it begins and ends; none (s = -1 .. ) on an empty axis.
struct Place {
    int s, begin, end;
};
__device__ __forceinline__ Place place_of(const SeqAxis& ax, int t) {
    Place q;
    q.s = seq_first_at(ax, t + 1) - 1;      // the last sequence that starts at or before t
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

// The state sequence s leaves: its last W - 1 inputs, from its tokens and the state before.
template <typename T, int V, int W>
__device__ __forceinline__ void leave_state(const SeqConvParams& p, int s, int c) {
    const long long slot = seq_slot(p.sl, s);
    if (slot < 0) return;
    const int begin = seq_start(p.ax, s, 0), end = seq_start(p.ax, s + 1, begin);
    float win[W][V];
    load_window<T, V, W>(p, s, end, end - begin, c, win);
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
        seq_stv<V>(static_cast<T*>(p.state_out) + (slot * (W - 1) + j) * p.D + c, win[j]);
}

template <typename T, int V, int W>
__global__ void __launch_bounds__(128) seq_conv_fwd_kernel(const __grid_constant__ SeqConvParams p) {
    const int c = (blockIdx.y * 128 + threadIdx.x) * V;
    if (c >= p.D) return;
    const int t0 = blockIdx.x * FWD_RUN, t1 = min(t0 + FWD_RUN, p.ax.T);
    float w[W][V], b[V], win[W][V];
    load_params<T, V, W>(p, c, w, b);
    Place q = place_of(p.ax, t0);
    load_window<T, V, W>(p, q.s, t0, t0 - q.begin, c, win);
    const T* x = static_cast<const T*>(p.x) + c;
    T* y = static_cast<T*>(p.y) + c;
#pragma unroll 4
    for (int t = t0; t < t1; ++t) {
        if (t == q.end) {
            next_place(p.ax, t, q);
            load_window<T, V, W>(p, q.s, t, 0, c, win);
        }
        seq_ldv<V>(x + (long long)t * p.x_ld, win[W - 1]);
        float o[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float a = b[v];
#pragma unroll
            for (int j = 0; j < W; ++j) a = fmaf(w[j][v], win[j][v], a);
            o[v] = p.silu ? silu(a) : a;
        }
        seq_stv<V>(y + (long long)t * p.y_ld, o);
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v) win[j][v] = win[j + 1][v];
    }
}

// The states after the last tokens.  A launch of its own behind the forward kernel: with
// state_out == state_in a thread there may still read the state that this one replaces.
template <typename T, int V, int W>
__global__ void __launch_bounds__(128) seq_conv_state_kernel(const __grid_constant__ SeqConvParams p) {
    const int c = (blockIdx.x * 128 + threadIdx.x) * V;
    if (c >= p.D) return;
    for (int s = blockIdx.y; s < p.ax.S; s += gridDim.y) leave_state<T, V, W>(p, s, c);
}

// One token per sequence: row s of x follows the W - 1 rows of its state.
template <typename T, int V, int W>
__global__ void __launch_bounds__(128) seq_conv_step_kernel(const __grid_constant__ SeqConvParams p) {
    const int c = (blockIdx.x * 128 + threadIdx.x) * V;
    if (c >= p.D) return;
    float w[W][V], b[V];
    load_params<T, V, W>(p, c, w, b);
    for (int s = blockIdx.y; s < p.ax.S; s += gridDim.y) {
        float win[W][V], o[V];
        const long long slot = seq_slot(p.sl, s);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            if (p.state_in && slot >= 0) {
                seq_ldv<V>(static_cast<const T*>(p.state_in) + (slot * (W - 1) + j) * p.D + c, win[j]);
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) win[j][v] = 0.f;
            }
        }
        seq_ldv<V>(static_cast<const T*>(p.x) + (long long)s * p.x_ld + c, win[W - 1]);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float a = b[v];
#pragma unroll
            for (int j = 0; j < W; ++j) a = fmaf(w[j][v], win[j][v], a);
            o[v] = p.silu ? silu(a) : a;
        }
        seq_stv<V>(static_cast<T*>(p.y) + (long long)s * p.y_ld + c, o);
        if (p.state_out && slot >= 0) {
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
                seq_stv<V>(static_cast<T*>(p.state_out) + (slot * (W - 1) + j) * p.D + c, win[j + 1]);
        }
    }
}

// Gradients.  dpre[t] = dy[t] silu'(pre[t]); dx[t] = sum_j w[j] dpre[t + W - 1 - j] over the tokens
// of t's sequence; dw[j] = sum_t dpre[t] x[t - W + 1 + j]; dbias = sum_t dpre[t].
// A thread walks its run and W - 1 tokens behind it (they see its last inputs), keeps the last
// W values of dpre in registers and emits dx with a delay of W - 1 tokens.  The parameter sums of
// the block's runs meet in shared memory in a fixed order and leave as one partial row per block.
template <typename T, int V, int W>
__global__ void __launch_bounds__(BWD_LANES * BWD_ROWS) seq_conv_bwd_kernel(const __grid_constant__ SeqConvParams p) {
    __shared__ float sums[BWD_ROWS][BWD_LANES * V + 1];
    const int lane = threadIdx.x % BWD_LANES, row = threadIdx.x / BWD_LANES;
    const int c = (blockIdx.y * BWD_LANES + lane) * V;
    const int t0 = min(((int)blockIdx.x * BWD_ROWS + row) * BWD_RUN, p.ax.T);
    const int t1 = min(t0 + BWD_RUN, p.ax.T);
    float acc[W + 1][V];
#pragma unroll
    for (int j = 0; j <= W; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) acc[j][v] = 0.f;
    if (c < p.D && t0 < t1) {
        float w[W][V], b[V], win[W][V], dp[W][V];
        load_params<T, V, W>(p, c, w, b);
        Place q = place_of(p.ax, t0);
        load_window<T, V, W>(p, q.s, t0, t0 - q.begin, c, win);
#pragma unroll
        for (int j = 0; j < W; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v) dp[j][v] = 0.f;
        const T* x = static_cast<const T*>(p.x) + c;
        const T* dy = static_cast<const T*>(p.dy) + c;
        T* dx = static_cast<T*>(p.dx) + c;
        // dp[j] holds dpre of token t - W + 1 + j; emit(t) writes dx of token t - W + 1
        auto emit = [&](int t) {
            const int m = t - (W - 1);
            if (m < t0 || m < q.begin || m >= t1) return;
            float o[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float a = 0.f;
#pragma unroll
                for (int j = 0; j < W; ++j) a = fmaf(w[W - 1 - j][v], dp[j][v], a);
                o[v] = a;
            }
            seq_stv<V>(dx + (long long)m * p.dx_ld, o);
        };
        auto push = [&](const float (&d)[V]) {
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v) dp[j][v] = dp[j + 1][v];
#pragma unroll
            for (int v = 0; v < V; ++v) dp[W - 1][v] = d[v];
        };
        const float zero[V] = {};
        // the run, and behind it the tokens of the same sequence that its last inputs reach
        int t = t0;
        for (;; ++t) {
            if (t == q.end) {                       // the sequence ends: its last W - 1 inputs
#pragma unroll
                for (int k = 0; k < W - 1; ++k) {
                    push(zero);
                    emit(t + k);
                }
                if (t >= t1) break;
                next_place(p.ax, t, q);
                load_window<T, V, W>(p, q.s, t, 0, c, win);
#pragma unroll
                for (int j = 0; j < W; ++j)
#pragma unroll
                    for (int v = 0; v < V; ++v) dp[j][v] = 0.f;
            }
            if (t >= t1 + W - 1) break;
            seq_ldv<V>(x + (long long)t * p.x_ld, win[W - 1]);
            float d[V];
            seq_ldv<V>(dy + (long long)t * p.dy_ld, d);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (p.silu) {
                    float a = b[v];
#pragma unroll
                    for (int j = 0; j < W; ++j) a = fmaf(w[j][v], win[j][v], a);
                    d[v] *= silu_grad(a, sigmoid(a));
                }
                if (t < t1) {
#pragma unroll
                    for (int j = 0; j < W; ++j) acc[j][v] = fmaf(d[v], win[j][v], acc[j][v]);
                    acc[W][v] += d[v];
                }
            }
            push(d);
            emit(t);
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v) win[j][v] = win[j + 1][v];
        }
    }
#pragma unroll
    for (int j = 0; j <= W; ++j) {
        __syncthreads();
#pragma unroll
        for (int v = 0; v < V; ++v) sums[row][lane * V + v] = acc[j][v];
        __syncthreads();
        for (int i = threadIdx.x; i < BWD_LANES * V; i += BWD_LANES * BWD_ROWS) {
            const int d = blockIdx.y * BWD_LANES * V + i;
            if (d >= p.D) break;
            float s = 0.f;
#pragma unroll
            for (int r = 0; r < BWD_ROWS; ++r) s += sums[r][i];
            p.ws[((long long)blockIdx.x * (W + 1) + j) * p.D + d] = s;
        }
    }
}

// Sums the blocks' partial rows, in block order: one thread per channel and tap.
__global__ void __launch_bounds__(128) seq_conv_param_kernel(const __grid_constant__ SeqConvParams p) {
    const int d = blockIdx.x * 128 + threadIdx.x, j = blockIdx.y;
    if (d >= p.D) return;
    float s[4] = {};
    const float* src = p.ws + (long long)j * p.D + d;
    const long long step = (long long)(p.W + 1) * p.D;
    int b = 0;
    for (; b + 4 <= p.tblocks; b += 4)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] += src[(b + i) * step];
    for (; b < p.tblocks; ++b) s[0] += src[b * step];
    const float v = (s[0] + s[1]) + (s[2] + s[3]);
    if (j < p.W) p.dw[(long long)d * p.W + j] = v;
    else if (p.dbias) p.dbias[d] = v;
}

enum class Pass { Fwd, Bwd, Step };

template <typename T, int V, int W>
cudaError_t launch_w(const SeqConvParams& p, Pass pass, cudaStream_t stream) {
    const unsigned cb = (unsigned)((p.D + 128 * V - 1) / (128 * V));
    const unsigned sb = (unsigned)(p.ax.S < 32768 ? p.ax.S : 32768);
    cudaError_t e = cudaSuccess;
    if (pass == Pass::Step)
        return launch_kernel(seq_conv_step_kernel<T, V, W>, dim3(cb, sb), dim3(128), 0, stream, false, 1, p);
    if (pass == Pass::Fwd) {
        if (p.ax.T > 0)
            e = launch_kernel(seq_conv_fwd_kernel<T, V, W>, dim3((unsigned)((p.ax.T + FWD_RUN - 1) / FWD_RUN), cb),
                              dim3(128), 0, stream, false, 1, p);
        if (e == cudaSuccess && p.state_out && W > 1)
            e = launch_kernel(seq_conv_state_kernel<T, V, W>, dim3(cb, sb), dim3(128), 0, stream, false, 1, p);
        return e;
    }
    if (p.ax.T > 0)
        e = launch_kernel(seq_conv_bwd_kernel<T, V, W>,
                          dim3((unsigned)p.tblocks, (unsigned)((p.D + BWD_LANES * V - 1) / (BWD_LANES * V))),
                          dim3(BWD_LANES * BWD_ROWS), 0, stream, false, 1, p);
    if (e == cudaSuccess)
        e = launch_kernel(seq_conv_param_kernel, dim3((unsigned)((p.D + 127) / 128), (unsigned)(W + 1)), dim3(128), 0,
                          stream, false, 1, p);
    return e;
}

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

int seq_conv_bwd_token_blocks(long long T) { return (int)((T + BWD_RUN * BWD_ROWS - 1) / (BWD_RUN * BWD_ROWS)); }
cudaError_t launch_seq_conv_fwd(const SeqConvParams& p, bool bf16, cudaStream_t stream) { return launch(p, bf16, Pass::Fwd, stream); }
cudaError_t launch_seq_conv_bwd(const SeqConvParams& p, bool bf16, cudaStream_t stream) { return launch(p, bf16, Pass::Bwd, stream); }
cudaError_t launch_seq_conv_step(const SeqConvParams& p, bool bf16, cudaStream_t stream) { return launch(p, bf16, Pass::Step, stream); }

}  // namespace convfwd

// Selective state space scan, forward and one-token step: see seq.h for the formulas.
//
// Per token, channel and state: one exponential (exp(delta A) as 2^(delta A log2 e)) and four
// multiply-adds, so the forward pass is bound by the special-function and FMA pipes, and the step by
// the bytes of the states.  A thread holds NPT states of one channel in registers and walks the
// tokens of a piece; LN neighbouring lanes share a channel when it has more states.
#include "seq_scan.cuh"

namespace convfwd {
namespace {

constexpr int THREADS = 128;

template <typename T, int NPT, int LN, bool SUMMARY>
__global__ void __launch_bounds__(THREADS) seq_scan_kernel(const __grid_constant__ SeqScanParams p) {
    constexpr int CB = THREADS / LN, NP = NPT * LN;
    __shared__ __align__(16) float sB[SCAN_TILE][NP], sC[SUMMARY ? 1 : SCAN_TILE][NP];
    __shared__ ScanBounds sb;
    const int piece = blockIdx.x;
    int t0, t1;
    scan_piece_range(p.ax, p.pc, piece, t0, t1);
    if (SUMMARY) {                  // the last piece of a sequence (of the axis) hands nothing on
        if (p.pc.pps > 0 ? piece % p.pc.pps == p.pc.pps - 1 : piece == p.pc.count - 1) return;
    }
    const int per = p.D / p.G, bpg = (per + CB - 1) / CB;
    const int g = blockIdx.y / bpg;
    const int cl = (blockIdx.y - g * bpg) * CB + threadIdx.x / LN;      // channel in its group
    const bool on = cl < per;
    const int d = g * per + (on ? cl : per - 1);
    const int ln = threadIdx.x % LN, n0 = ln * NPT;
    float A2[NPT], h[NPT];
#pragma unroll
    for (int k = 0; k < NPT; ++k) {
        A2[k] = n0 + k < p.N ? p.A[(long long)d * p.N + n0 + k] * LOG2E : 0.f;
        h[k] = 0.f;
    }
    const float Dd = p.Dskip ? p.Dskip[d] : 0.f, bias = p.dt_bias ? p.dt_bias[d] : 0.f;
    float total = 0.f;
    // the state before the piece: what the sequence's earlier pieces leave, one after another
    if (!SUMMARY && t0 < t1) {
        const int s = seq_first_at(p.ax, t0 + 1) - 1;
        const int begin = s < 0 ? t0 : seq_start(p.ax, s, 0);
        if (begin < t0) {
            const int q0 = p.pc.pps > 0 ? piece - piece % p.pc.pps : begin / p.pc.len;
            for (int q = q0; q < piece; ++q) {
                const float sum = p.piece_delta[(long long)q * p.D + d];
#pragma unroll
                for (int k = 0; k < NPT; ++k) {
                    const float e = n0 + k < ((p.N + 3) & ~3) ? p.piece_state[scan_state_at(p, q, (n0 + k) >> 2, d) + (k & 3)] : 0.f;
                    h[k] = fmaf(ex2_approx(sum * A2[k]), h[k], e);
                }
            }
        }
    }
    const T* x = static_cast<const T*>(p.x) + d;
    const T* dt = static_cast<const T*>(p.dt) + d;
    const T* z = static_cast<const T*>(p.z) + d;
    T* y = static_cast<T*>(p.y) + d;
    for (int tb = t0; tb < t1; tb += SCAN_TILE) {
        const int n = min(SCAN_TILE, t1 - tb);
        __syncthreads();
        for (int i = threadIdx.x; i < n * NP; i += THREADS) {
            const int t = i / NP, k = i - t * NP;
            sB[t][k] = k < p.N ? seq_ld(static_cast<const T*>(p.B) + (long long)(tb + t) * p.B_ld + g * p.N + k) : 0.f;
            if (!SUMMARY)
                sC[t][k] = k < p.N ? seq_ld(static_cast<const T*>(p.C) + (long long)(tb + t) * p.C_ld + g * p.N + k) : 0.f;
        }
        if (threadIdx.x < 32) scan_bounds(p.ax, tb, n, &sb);
        __syncthreads();
        const unsigned first = sb.first, last = sb.last;
        for (int i = 0; i < n; ++i) {
            const long long t = tb + i;
            if (first >> i & 1) {
                const int s = sb.seq[i];
                // a sequence that runs on behind the piece: its starting state was put aside by the
                // pass before, since the block that ends it may already have written h_out
                if (!SUMMARY && p.h_in && p.pc.pps != 1 && p.pc.count > 1 && seq_start(p.ax, s + 1, 0) > t1) {
#pragma unroll
                    for (int k = 0; k < NPT; ++k)
                        h[k] = n0 + k < p.N ? p.piece_init[scan_state_at(p, piece, (n0 + k) >> 2, d) + (k & 3)] : 0.f;
                } else {
                    scan_h_load<NPT>(p, p.h_in, seq_slot(p.sl, s), d, n0, h);
                }
                if (SUMMARY && on && p.h_in) {
#pragma unroll
                    for (int k = 0; k < NPT; ++k)
                        if (n0 + k < p.N) p.piece_init[scan_state_at(p, piece, (n0 + k) >> 2, d) + (k & 3)] = h[k];
                }
                total = 0.f;
            }
            if (!SUMMARY && i == 0 && p.saved && on) {
                const long long row = scan_tile_row(p.ax, tb);
#pragma unroll
                for (int k = 0; k < NPT; ++k)
                    if (n0 + k < ((p.N + 3) & ~3)) p.saved[scan_state_at(p, row, (n0 + k) >> 2, d) + (k & 3)] = h[k];
            }
            const float xv = seq_ld(x + t * p.x_ld);
            float delta = seq_ld(dt + t * p.dt_ld) + bias;
            if (p.softplus) delta = softplus(delta);
            const float u = delta * xv;
            float acc = 0.f;
#pragma unroll
            for (int k = 0; k < NPT; ++k) {
                h[k] = fmaf(ex2_approx(delta * A2[k]), h[k], u * sB[i][n0 + k]);
                if (!SUMMARY) acc = fmaf(sC[i][n0 + k], h[k], acc);
            }
            total += delta;
            if (!SUMMARY) {
#pragma unroll
                for (int o = LN / 2; o > 0; o >>= 1) acc += __shfl_xor_sync(~0u, acc, o);
                if (ln == 0 && on) {
                    float v = fmaf(Dd, xv, acc);
                    if (p.z) v *= silu(seq_ld(z + t * p.z_ld));
                    seq_st(y + t * p.y_ld, v);
                }
                if ((last >> i & 1) && on) scan_h_store<NPT>(p, p.h_out, seq_slot(p.sl, sb.seq[i]), d, n0, h);
            }
        }
    }
    if (SUMMARY && on) {
#pragma unroll
        for (int k = 0; k < NPT; ++k)
            if (n0 + k < ((p.N + 3) & ~3)) p.piece_state[scan_state_at(p, piece, (n0 + k) >> 2, d) + (k & 3)] = h[k];
        if (ln == 0) p.piece_delta[(long long)piece * p.D + d] = total;
    }
}

// Empty sequences hand their state on.
__global__ void __launch_bounds__(128) seq_scan_empty_kernel(SeqAxis ax, SeqSlots sl, const float* from, float* to, long long DN) {
    for (int s = blockIdx.y; s < ax.S; s += gridDim.y) {
        const int b = seq_start(ax, s, 0);
        const long long slot = seq_slot(sl, s);
        if (seq_start(ax, s + 1, b) != b || slot < 0) continue;
        for (long long i = blockIdx.x * 128ll + threadIdx.x; i < DN; i += gridDim.x * 128ll)
            to[slot * DN + i] = from ? from[slot * DN + i] : 0.f;
    }
}

// One token per sequence.  A lane holds 4 states of a channel (16 bytes of its state row), LN lanes
// share the channel.
template <typename T, int LN>
__global__ void __launch_bounds__(THREADS) seq_scan_step_kernel(const __grid_constant__ SeqScanParams p) {
    const int d0 = (blockIdx.x * THREADS + threadIdx.x) / LN;
    const bool on = d0 < p.D;
    const int d = on ? d0 : p.D - 1;
    const int n0 = threadIdx.x % LN * 4, g = d / (p.D / p.G);
    float A2[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) A2[k] = n0 + k < p.N ? p.A[(long long)d * p.N + n0 + k] * LOG2E : 0.f;
    const float bias = p.dt_bias ? p.dt_bias[d] : 0.f, Dd = p.Dskip ? p.Dskip[d] : 0.f;
    for (long long s = blockIdx.y; s < p.ax.S; s += gridDim.y) {
        const long long slot = seq_slot(p.sl, (int)s);
        float h[4];
        scan_h_load<4>(p, p.h_in, slot, d, n0, h);
        const float xv = seq_ld(static_cast<const T*>(p.x) + s * p.x_ld + d);
        float delta = seq_ld(static_cast<const T*>(p.dt) + s * p.dt_ld + d) + bias;
        if (p.softplus) delta = softplus(delta);
        const float u = delta * xv;
        float acc = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float b = n0 + k < p.N ? seq_ld(static_cast<const T*>(p.B) + s * p.B_ld + g * p.N + n0 + k) : 0.f;
            const float c = n0 + k < p.N ? seq_ld(static_cast<const T*>(p.C) + s * p.C_ld + g * p.N + n0 + k) : 0.f;
            h[k] = fmaf(ex2_approx(delta * A2[k]), h[k], u * b);
            acc = fmaf(c, h[k], acc);
        }
        if (on) scan_h_store<4>(p, p.h_out, slot, d, n0, h);
#pragma unroll
        for (int o = LN / 2; o > 0; o >>= 1) acc += __shfl_xor_sync(~0u, acc, o);
        if (n0 == 0 && on) {
            float v = fmaf(Dd, xv, acc);
            if (p.z) v *= silu(seq_ld(static_cast<const T*>(p.z) + s * p.z_ld + d));
            seq_st(static_cast<T*>(p.y) + s * p.y_ld + d, v);
        }
    }
}

template <typename T, int NPT, int LN>
cudaError_t launch_fwd(const SeqScanParams& p, cudaStream_t stream) {
    constexpr int CB = THREADS / LN;
    const int per = p.D / p.G;
    const dim3 grid((unsigned)p.pc.count, (unsigned)(p.G * ((per + CB - 1) / CB)));
    cudaError_t e = cudaSuccess;
    if (p.ax.T > 0) {
        if (p.pc.pps != 1 && p.pc.count > 1)
            e = launch_kernel(seq_scan_kernel<T, NPT, LN, true>, grid, dim3(THREADS), 0, stream, false, 1, p);
        if (e == cudaSuccess)
            e = launch_kernel(seq_scan_kernel<T, NPT, LN, false>, grid, dim3(THREADS), 0, stream, false, 1, p);
    }
    if (e == cudaSuccess && p.h_out && p.h_out != p.h_in && p.ax.L == 0) e = launch_seq_scan_empty(p, p.h_in, p.h_out, stream);
    return e;
}

template <typename T>
cudaError_t launch_t(const SeqScanParams& p, cudaStream_t stream) {
    if (p.N <= 4) return launch_fwd<T, 4, 1>(p, stream);
    if (p.N <= 8) return launch_fwd<T, 8, 1>(p, stream);
    if (p.N <= 16) return launch_fwd<T, 16, 1>(p, stream);
    if (p.N <= 32) return launch_fwd<T, 16, 2>(p, stream);
    if (p.N <= 64) return launch_fwd<T, 16, 4>(p, stream);
    return launch_fwd<T, 16, 8>(p, stream);
}

template <typename T, int LN>
cudaError_t launch_step(const SeqScanParams& p, cudaStream_t stream) {
    const dim3 grid((unsigned)(((long long)p.D * LN + THREADS - 1) / THREADS), (unsigned)(p.ax.S < 32768 ? p.ax.S : 32768));
    return launch_kernel(seq_scan_step_kernel<T, LN>, grid, dim3(THREADS), 0, stream, false, 1, p);
}
template <typename T>
cudaError_t launch_step_t(const SeqScanParams& p, cudaStream_t stream) {
    if (p.N <= 4) return launch_step<T, 1>(p, stream);
    if (p.N <= 8) return launch_step<T, 2>(p, stream);
    if (p.N <= 16) return launch_step<T, 4>(p, stream);
    if (p.N <= 32) return launch_step<T, 8>(p, stream);
    if (p.N <= 64) return launch_step<T, 16>(p, stream);
    return launch_step<T, 32>(p, stream);
}

}  // namespace

cudaError_t launch_seq_scan_empty(const SeqScanParams& p, const float* from, float* to, cudaStream_t stream) {
    const long long DN = (long long)p.D * p.N, blocks = DN / 1024 + 1;
    return launch_kernel(seq_scan_empty_kernel, dim3((unsigned)(blocks < 64 ? blocks : 64), (unsigned)(p.ax.S < 32768 ? p.ax.S : 32768)),
                         dim3(128), 0, stream, false, 1, p.ax, p.sl, from, to, DN);
}
cudaError_t launch_seq_scan_fwd(const SeqScanParams& p, bool bf16, cudaStream_t stream) {
    return bf16 ? launch_t<__nv_bfloat16>(p, stream) : launch_t<float>(p, stream);
}
cudaError_t launch_seq_scan_step(const SeqScanParams& p, bool bf16, cudaStream_t stream) {
    return bf16 ? launch_step_t<__nv_bfloat16>(p, stream) : launch_step_t<float>(p, stream);
}

}  // namespace convfwd

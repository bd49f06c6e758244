// Selective state space scan, one token of each of several sequences: see seq.h for the formulas.
//
// Bound by the bytes of the states: 256 x 4096 x 16 reads 67 MB of them and writes as many in 29 us (143 MB with x,
// dt, z, y: 4.9 TB/s, 73% of a plain copy's rate).
#include "seq_scan.cuh"

namespace convfwd {
namespace {

constexpr int STEP_THREADS = 128;

// One token per sequence: bound by the bytes of the states.  A lane holds 4 states of a channel (16 bytes of
// its state row), LN lanes share the channel; a thread keeps its row of A and takes ROWS sequences at a
// time, all of their loads on their way before the first is used.  VEC: states, A, B and C in whole aligned
// groups of 4.
template <typename T, int LN, int ROWS, int CH, bool VEC>
__global__ void __launch_bounds__(STEP_THREADS, ROWS > 1 && VEC ? 7 : 1) seq_scan_step_kernel(const __grid_constant__ SeqScanParams p) {
    const int d0 = (int)((blockIdx.x * (long long)STEP_THREADS + threadIdx.x) / LN) * CH;
    const bool on = d0 < p.D;
    const int d = on ? d0 : p.D - CH;
    const int n0 = threadIdx.x % LN * 4, bc = d / (p.D / p.G) * p.N + n0;
    const bool any = n0 < p.N;                       // (lanes behind the states only take part in the sum)
    const float2 zero = make_float2(0.f, 0.f);
    auto four = [&](const float* from, float2 (&v)[2]) {
        v[0] = v[1] = zero;
        if (VEC) {
            if (any) ld2(from, v[0], v[1]);
        } else {
            if (n0 < p.N) v[0].x = from[0];
            if (n0 + 1 < p.N) v[0].y = from[1];
            if (n0 + 2 < p.N) v[1].x = from[2];
            if (n0 + 3 < p.N) v[1].y = from[3];
        }
    };
    auto four_t = [&](const T* from, float2 (&v)[2]) {
        v[0] = v[1] = zero;
        if (VEC) {
            if (any) {
                v[0] = seq_ld2(from);
                v[1] = seq_ld2(from + 2);
            }
        } else {
            if (n0 < p.N) v[0].x = seq_ld(from);
            if (n0 + 1 < p.N) v[0].y = seq_ld(from + 1);
            if (n0 + 2 < p.N) v[1].x = seq_ld(from + 2);
            if (n0 + 3 < p.N) v[1].y = seq_ld(from + 3);
        }
    };
    // the thread's channels as a pair (the second is nothing where there is one)
    auto channels = [&](auto* from) { return CH == 2 ? seq_ld2(from) : make_float2(seq_ld(from), 0.f); };
    float2 A2[CH][2];
    const int at = d * p.N + n0, DN = p.D * p.N;     // (D N < 2^31: see the plan)
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        four(p.A + at + c * p.N, A2[c]);
        A2[c][0] = mul2(A2[c][0], dup2(LOG2E));
        A2[c][1] = mul2(A2[c][1], dup2(LOG2E));
    }
    auto of_channels = [&](const float* v) { return v ? make_float2(v[d], CH == 2 ? v[d + CH - 1] : 0.f) : zero; };
    const float2 bias = of_channels(p.dt_bias), Dd = of_channels(p.Dskip);
    // row s of a tensor (rows are less than 2^31 elements apart)
    auto row = [](const void* base, int s, long long ld) { return static_cast<const T*>(base) + (long long)s * (int)ld; };
    for (int s0 = blockIdx.y * ROWS; s0 < p.ax.S; s0 += gridDim.y * ROWS) {
        float2 h[ROWS][CH][2], B[ROWS][2], C[ROWS][2];
        float2 x[ROWS], raw[ROWS], z[ROWS];
        int slot[ROWS];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) slot[r] = s0 + r < p.ax.S ? (int)seq_slot(p.sl, s0 + r) : -1;
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            const int s = min(s0 + r, p.ax.S - 1);
#pragma unroll
            for (int c = 0; c < CH; ++c) h[r][c][0] = h[r][c][1] = zero;
            if (p.h_in && slot[r] >= 0) {
                const float* from = p.h_in + (long long)slot[r] * DN + at;
#pragma unroll
                for (int c = 0; c < CH; ++c) four(from + c * p.N, h[r][c]);
            }
            x[r] = channels(row(p.x, s, p.x_ld) + d);
            raw[r] = sum2(channels(row(p.dt, s, p.dt_ld) + d), bias);
            z[r] = p.z ? channels(row(p.z, s, p.z_ld) + d) : zero;
            four_t(row(p.B, s, p.B_ld) + bc, B[r]);
            four_t(row(p.C, s, p.C_ld) + bc, C[r]);
        }
        float2 delta[ROWS];
        if (CH == 1 && ROWS % 2 == 0) {              // two sequences' steps at once
#pragma unroll
            for (int r = 0; r + 1 < ROWS; r += 2) {
                const float2 v = make_float2(raw[r].x, raw[r + 1].x), w = p.softplus ? softplus2(v, nullptr) : v;
                delta[r] = dup2(w.x);
                delta[r + 1] = dup2(w.y);
            }
        } else {
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                delta[r] = raw[r];
                if (p.softplus) delta[r] = CH == 2 ? softplus2(raw[r], nullptr) : dup2(softplus(raw[r].x));
            }
        }
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            const float2 u = mul2(delta[r], x[r]);
            float sum[CH];
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const float2 dl = dup2(c ? delta[r].y : delta[r].x), uu = dup2(c ? u.y : u.x);
                float2 acc = zero;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    h[r][c][k] = fma2(decay2(dl, A2[c][k]), h[r][c][k], mul2(uu, B[r][k]));
                    acc = fma2(C[r][k], h[r][c][k], acc);
                }
                sum[c] = acc.x + acc.y;
            }
            if (on && p.h_out && slot[r] >= 0) {
                float* to = p.h_out + (long long)slot[r] * DN + at;
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    if (VEC) {
                        if (any) st2(to + c * p.N, h[r][c][0], h[r][c][1]);
                    } else {
                        if (n0 < p.N) to[c * p.N] = h[r][c][0].x;
                        if (n0 + 1 < p.N) to[c * p.N + 1] = h[r][c][0].y;
                        if (n0 + 2 < p.N) to[c * p.N + 2] = h[r][c][1].x;
                        if (n0 + 3 < p.N) to[c * p.N + 3] = h[r][c][1].y;
                    }
                }
            }
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int o = LN / 2; o > 0; o >>= 1) sum[c] += __shfl_xor_sync(~0u, sum[c], o);
            if (n0 == 0 && on && s0 + r < p.ax.S) {
                float2 v = fma2(Dd, x[r], make_float2(sum[0], CH == 2 ? sum[CH - 1] : 0.f));
                if (p.z) v = mul2(v, make_float2(silu(z[r].x), CH == 2 ? silu(z[r].y) : 0.f));
                seq_st2(const_cast<T*>(row(p.y, s0 + r, p.y_ld)) + d, v, CH == 2, true);
            }
        }
    }
}

template <typename T, int LN, int ROWS, int CH>
cudaError_t launch_step_of(const SeqScanParams& p, cudaStream_t stream) {
    const long long lanes = (long long)(p.D / CH) * LN;
    const int rows = (p.ax.S + ROWS - 1) / ROWS;
    const dim3 grid((unsigned)((lanes + STEP_THREADS - 1) / STEP_THREADS), (unsigned)(rows < 32768 ? rows : 32768));
    if (p.quads) return launch_kernel(seq_scan_step_kernel<T, LN, ROWS, CH, true>, grid, dim3(STEP_THREADS), 0, stream, false, 1, p);
    if constexpr (CH == 1) return launch_kernel(seq_scan_step_kernel<T, LN, ROWS, CH, false>, grid, dim3(STEP_THREADS), 0, stream, false, 1, p);
    else return cudaErrorInvalidValue;
}
template <typename T, int LN>
cudaError_t launch_step(const SeqScanParams& p, cudaStream_t stream) {
    const long long blocks = ((long long)p.D * LN + STEP_THREADS - 1) / STEP_THREADS;
    // Several sequences a thread once that still leaves the GPU several blocks an SM.  256 x 4096 x 16 bf16: one
    // sequence and channel 54 us; 4 sequences 32.5; 2 sequences of 2 channels, which share the rows' addresses,
    // 29.4; 4 of 2 (half the warps) 37.
    if (blocks * p.ax.S < 16ll * p.sms * 4) return launch_step_of<T, LN, 1, 1>(p, stream);
    const bool pairs = p.quads && p.wide >= 2 * (int)sizeof(T);        // whole aligned pairs of channels
    return pairs ? launch_step_of<T, LN, 2, 2>(p, stream) : launch_step_of<T, LN, 4, 1>(p, stream);
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

cudaError_t launch_seq_scan_step(const SeqScanParams& p, bool bf16, cudaStream_t stream) {
    return bf16 ? launch_step_t<__nv_bfloat16>(p, stream) : launch_step_t<float>(p, stream);
}

}  // namespace convfwd

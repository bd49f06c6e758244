// Gated delta rule, one token of each of several sequences: see delta.h for the recurrence.
//
// Bound by the bytes of the states, each read and written once.  With a = h^T k and c = h^T q of the old state,
//   u = beta (v - exp(g) a),  h <- exp(g) h + k u^T,  y = scale (exp(g) c + (q.k) u),
// so that one pass over the state in registers does both sums, and one meeting of the block's warps joins them.  The states pass
// L2 as what is used once, and three blocks are on an SM, so that some load while others store: 256 sequences of 32 heads of 128 x 128 take 178 to 187 us,
// 5.8 to 6.0 TB/s, with plain accesses and two blocks 210 us (with blocks of 512 threads 338).
#include "seq_delta.cuh"

namespace convfwd {
namespace {

constexpr int STEP_T = 256, STEP_W = STEP_T / 32;

// A block: a sequence, a value head and 32 V columns of its state; a lane V columns, a warp the rows w, w + 8, ...
template <typename T, int ROWS, int V>
__global__ void __launch_bounds__(STEP_T, 3) delta_step_kernel(const __grid_constant__ SeqDeltaParams p, int dvbs) {
    __shared__ float qs[128], ks[128];
    __shared__ float part[2][STEP_W][32 * V];
    __shared__ float sums[3][STEP_W];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int dvb = blockIdx.x % dvbs, sh = blockIdx.x / dvbs, h = sh % p.Hv, seq = sh / p.Hv, kh = h / (p.Hv / p.Hk);
    const int c = dvb * 32 * V + lane * V;
    const long long row = seq_slot(p.sl, seq), state = (row * p.Hv + h) * (long long)p.Dk * p.Dv + c;
    float st[ROWS][V];
    const bool have = p.h_in && row >= 0;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const int i = warp + r * STEP_W;
        const bool on = have && i < p.Dk;
        const float* from = p.h_in + state + (long long)i * p.Dv;
        if (V == 4) {
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (on && c < p.Dv) v = __ldcs(reinterpret_cast<const float4*>(from));
            st[r][0] = v.x; st[r][V > 1 ? 1 : 0] = v.y; st[r][V > 2 ? 2 : 0] = v.z; st[r][V > 3 ? 3 : 0] = v.w;
        } else {
            st[r][0] = on && c < p.Dv ? *from : 0.f;
        }
    }
    // q and k of the head, their lengths and product
    {
        const int i = threadIdx.x;
        float q = 0.f, k = 0.f;
        if (i < p.Dk) {
            q = seq_ld(static_cast<const T*>(p.q) + seq * p.q_ld + kh * p.Dk + i);
            k = seq_ld(static_cast<const T*>(p.k) + seq * p.k_ld + kh * p.Dk + i);
        }
        float qq = q * q, kk = k * k, qk = q * k;
        if (i < 128) {
            qs[i] = q;
            ks[i] = k;
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            qq += __shfl_xor_sync(0xffffffffu, qq, d);
            kk += __shfl_xor_sync(0xffffffffu, kk, d);
            qk += __shfl_xor_sync(0xffffffffu, qk, d);
        }
        if (lane == 0) {
            sums[0][warp] = qq;
            sums[1][warp] = kk;
            sums[2][warp] = qk;
        }
    }
    const float decay = expf(p.g[seq * p.g_ld + h]), beta = p.beta[seq * p.beta_ld + h];
    __syncthreads();
    float a[V], o[V];
#pragma unroll
    for (int e = 0; e < V; ++e) a[e] = o[e] = 0.f;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const int i = warp + r * STEP_W;
        const float k = ks[i], q = qs[i];
#pragma unroll
        for (int e = 0; e < V; ++e) {
            a[e] = fmaf(k, st[r][e], a[e]);
            o[e] = fmaf(q, st[r][e], o[e]);
        }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
        part[0][warp][lane * V + e] = a[e];
        part[1][warp][lane * V + e] = o[e];
    }
    __syncthreads();
    float qq = 0.f, kk = 0.f, qk = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {                // (128 values: the first four warps')
        qq += sums[0][w];
        kk += sums[1][w];
        qk += sums[2][w];
    }
    const float rq = p.norm ? 1.f / sqrtf(qq + QK_EPS) : 1.f, rk = p.norm ? 1.f / sqrtf(kk + QK_EPS) : 1.f;
    float u[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        float sa = 0.f;
#pragma unroll
        for (int w = 0; w < STEP_W; ++w) sa += part[0][w][lane * V + e];
        const float v = c + e < p.Dv ? seq_ld(static_cast<const T*>(p.v) + seq * p.v_ld + h * p.Dv + c + e) : 0.f;
        u[e] = beta * (v - decay * (rk * sa));
    }
    if (warp == 0) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            float so = 0.f;
#pragma unroll
            for (int w = 0; w < STEP_W; ++w) so += part[1][w][lane * V + e];
            if (c + e < p.Dv)
                seq_st(static_cast<T*>(p.y) + seq * p.y_ld + h * p.Dv + c + e, p.scale * rq * fmaf(decay, so, rk * qk * u[e]));
        }
    }
    if (!p.h_out || row < 0) return;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const int i = warp + r * STEP_W;
        if (i < p.Dk && c < p.Dv) {
            const float k = ks[i] * rk;
            float* to = p.h_out + state + (long long)i * p.Dv;
            if (V == 4) {
                __stcs(reinterpret_cast<float4*>(to),
                       make_float4(fmaf(decay, st[r][0], k * u[0]), fmaf(decay, st[r][V > 1 ? 1 : 0], k * u[V > 1 ? 1 : 0]),
                                   fmaf(decay, st[r][V > 2 ? 2 : 0], k * u[V > 2 ? 2 : 0]), fmaf(decay, st[r][V > 3 ? 3 : 0], k * u[V > 3 ? 3 : 0])));
            } else {
                *to = fmaf(decay, st[r][0], k * u[0]);
            }
        }
    }
}

template <typename T, int ROWS, int V>
cudaError_t launch_step(const SeqDeltaParams& p, cudaStream_t stream) {
    const int dvbs = (p.Dv + 32 * V - 1) / (32 * V);
    return launch_kernel(delta_step_kernel<T, ROWS, V>, dim3((unsigned)(p.ax.S * (long long)p.Hv * dvbs)), dim3(STEP_T), 0, stream, false, 1, p, dvbs);
}

template <typename T>
cudaError_t launch(const SeqDeltaParams& p, cudaStream_t stream) {
    if (p.quads) return p.Dk <= 64 ? launch_step<T, 8, 4>(p, stream) : launch_step<T, 16, 4>(p, stream);
    return p.Dk <= 64 ? launch_step<T, 8, 1>(p, stream) : launch_step<T, 16, 1>(p, stream);
}

}  // namespace

cudaError_t launch_seq_delta_step(const SeqDeltaParams& p, bool bf16, cudaStream_t stream) {
    if (p.ax.T == 0) return cudaSuccess;
    return bf16 ? launch<__nv_bfloat16>(p, stream) : launch<float>(p, stream);
}

}  // namespace convfwd

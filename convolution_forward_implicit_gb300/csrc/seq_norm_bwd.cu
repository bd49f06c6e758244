// Norm, gate and residual around a block, gradients.  With hat = norm(v), r = 1 / sqrt(...) and d the
// gradient at w hat + b:  dw = sum_rows d hat, db = sum_rows d, and at v, with e = d w,
//   dv = r (e - hat mean(e hat))           (RMS; layer: also less mean(e)).
// Bound by bytes.  A block keeps its share of the rows' parameter sums in registers (its threads stay
// on their columns), writes them once, and a second kernel adds the blocks up in their order.
#include "seq_norm.cuh"

namespace convfwd {
namespace {

constexpr int SUMS = 5;      // w_post, b_post, scale, w_pre, b_pre

// e (the gradient behind w) -> the gradient at v, in place
template <int UPT>
__device__ __forceinline__ void norm_back(float (&d)[UPT][8], const float (&hat)[UPT][8], float r, int D, bool layer,
                                          float (*buf)[32][2], int& turn) {
    float s[2] = {};
#pragma unroll
    for (int u = 0; u < UPT; ++u)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            s[0] = fmaf(d[u][e], hat[u][e], s[0]);
            s[1] += d[u][e];
        }
    row_sum(s, buf, turn);
    const float c = s[0] / (float)D, m = layer ? s[1] / (float)D : 0.f;
#pragma unroll
    for (int u = 0; u < UPT; ++u)
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if ((threadIdx.x + u * blockDim.x) * 8 + e < D) d[u][e] = r * (d[u][e] - fmaf(hat[u][e], c, m));
}

#define EACH_UE _Pragma("unroll") for (int u = 0; u < UPT; ++u) _Pragma("unroll") for (int e = 0; e < 8; ++e)

template <typename T, typename RT, bool WIDE, int UPT, bool BIAS>
__global__ void __launch_bounds__(1024) seq_norm_bwd_kernel(const __grid_constant__ SeqNormParams p) {
    __shared__ float buf[2][32][2];
    int turn = 0;
    const bool layer = p.flags & SEQ_NORM_LAYER;
    const bool post = p.flags & SEQ_NORM_POST, pre = p.flags & SEQ_NORM_PRE, residual = p.flags & SEQ_NORM_RESIDUAL;
    const bool gate = p.flags & (SEQ_NORM_GATE_BEFORE | SEQ_NORM_GATE_AFTER), after = p.flags & SEQ_NORM_GATE_AFTER;
    float s_wpost[UPT][8] = {}, s_bpost[UPT][8] = {}, s_scale[UPT][8] = {}, s_wpre[UPT][8] = {}, s_bpre[UPT][8] = {};
    for (long long base = (long long)blockIdx.x * blockDim.y; base < p.rows; base += (long long)gridDim.x * blockDim.y) {
        const long long row = base + threadIdx.y;
        const int D = row < p.rows ? p.D : 0;
        float x[UPT][8], g[UPT][8], hat[UPT][8], hat2[UPT][8], d[UPT][8], t[UPT][8];
        float r_post = 0.f, r_pre = 0.f;
        // the forward pass again: hat (POST), u in t, r in hat2 -> hat2 (PRE)
        row_load<T, WIDE, UPT>(p.x, row * p.x_ld, D, x);
        if (gate) row_load<T, WIDE, UPT>(p.gate, row * p.gate_ld, D, g);
        EACH_UE hat[u][e] = gate && !after ? x[u][e] * silu(g[u][e]) : x[u][e];
        if (post) r_post = row_norm(hat, p.D, layer, p.eps, buf, turn);
        EACH_UE hat2[u][e] = hat[u][e];
        if (post) {
            col_load<T, WIDE, UPT>(p.w_post, 1.f, D, t);
            EACH_UE hat2[u][e] *= t[u][e];
            if (BIAS && p.b_post) {
                col_load<T, WIDE, UPT>(p.b_post, 0.f, D, t);
                EACH_UE hat2[u][e] += t[u][e];
            }
        }
        if (after) EACH_UE hat2[u][e] *= silu(g[u][e]);
        EACH_UE t[u][e] = hat2[u][e];
        if (p.scale) {
            col_load<T, WIDE, UPT>(p.scale, 1.f, D, d);
            EACH_UE hat2[u][e] *= d[u][e];
        }
        if (residual && pre) {
            row_load<RT, WIDE, UPT>(p.res, row * p.res_ld, D, d);
            EACH_UE hat2[u][e] += d[u][e];
        }
        // d: the gradient at r
        if (pre) {
            r_pre = row_norm(hat2, p.D, layer, p.eps, buf, turn);
            row_load<T, WIDE, UPT>(p.dy, row * p.dy_ld, D, d);
            EACH_UE s_wpre[u][e] = fmaf(d[u][e], hat2[u][e], s_wpre[u][e]);
            if (BIAS) EACH_UE s_bpre[u][e] += d[u][e];
            float w[UPT][8];
            col_load<T, WIDE, UPT>(p.w_pre, 1.f, D, w);
            EACH_UE d[u][e] *= w[u][e];
            norm_back(d, hat2, r_pre, p.D, layer, buf, turn);
        } else if (!residual) {
            row_load<T, WIDE, UPT>(p.dy, row * p.dy_ld, D, d);
        } else {
            EACH_UE d[u][e] = 0.f;
        }
        if (residual) {
            if (p.dres_out) {
                row_load<RT, WIDE, UPT>(p.dres_out, row * p.dres_out_ld, D, hat2);
                EACH_UE d[u][e] += hat2[u][e];
            }
            row_store<RT, WIDE, UPT>(p.dres, row * p.dres_ld, D, d);
        }
        // back through scale, gate, POST, gate
        if (p.scale) {
            EACH_UE s_scale[u][e] = fmaf(d[u][e], t[u][e], s_scale[u][e]);
            col_load<T, WIDE, UPT>(p.scale, 1.f, D, hat2);
            EACH_UE d[u][e] *= hat2[u][e];
        }
        if (post) col_load<T, WIDE, UPT>(p.w_post, 1.f, D, hat2);     // w_post
        if (after) {
            if (BIAS && p.b_post) col_load<T, WIDE, UPT>(p.b_post, 0.f, D, t);
            EACH_UE {
                const float s = sigmoid(g[u][e]);
                const float n = post ? fmaf(hat[u][e], hat2[u][e], BIAS && p.b_post ? t[u][e] : 0.f) : x[u][e];
                const float dg = d[u][e] * n * silu_grad(g[u][e], s);
                d[u][e] *= g[u][e] * s;
                g[u][e] = dg;
            }
            row_store<T, WIDE, UPT>(p.dgate, row * p.dgate_ld, D, g);
        }
        if (post) {
            EACH_UE s_wpost[u][e] = fmaf(d[u][e], hat[u][e], s_wpost[u][e]);
            if (BIAS) EACH_UE s_bpost[u][e] += d[u][e];
            EACH_UE d[u][e] *= hat2[u][e];
            norm_back(d, hat, r_post, p.D, layer, buf, turn);
        }
        if (gate && !after) {
            EACH_UE {
                const float s = sigmoid(g[u][e]);
                const float dg = d[u][e] * x[u][e] * silu_grad(g[u][e], s);
                d[u][e] *= g[u][e] * s;
                g[u][e] = dg;
            }
            row_store<T, WIDE, UPT>(p.dgate, row * p.dgate_ld, D, g);
        }
        row_store<T, WIDE, UPT>(p.dx, row * p.dx_ld, D, d);
    }
    if (!p.ws) return;
    const long long part = ((long long)blockIdx.x * blockDim.y + threadIdx.y) * SUMS * p.D;
    if (p.dw_post) row_store<float, WIDE, UPT>(p.ws, part, p.D, s_wpost);
    if (BIAS && p.db_post) row_store<float, WIDE, UPT>(p.ws, part + p.D, p.D, s_bpost);
    if (p.dscale) row_store<float, WIDE, UPT>(p.ws, part + 2 * p.D, p.D, s_scale);
    if (p.dw_pre) row_store<float, WIDE, UPT>(p.ws, part + 3 * p.D, p.D, s_wpre);
    if (BIAS && p.db_pre) row_store<float, WIDE, UPT>(p.ws, part + 4 * p.D, p.D, s_bpre);
}

__global__ void __launch_bounds__(128) seq_norm_param_kernel(const __grid_constant__ SeqNormParams p, int parts) {
    const int c = blockIdx.x * 128 + threadIdx.x, k = blockIdx.y;
    float* out = k == 0 ? p.dw_post : k == 1 ? p.db_post : k == 2 ? p.dscale : k == 3 ? p.dw_pre : p.db_pre;
    if (!out || c >= p.D) return;
    float s[4] = {};
    const float* src = p.ws + (long long)k * p.D + c;
    const long long step = (long long)SUMS * p.D;
    int b = 0;
    for (; b + 4 <= parts; b += 4)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] += src[(b + i) * step];
    for (; b < parts; ++b) s[0] += src[b * step];
    out[c] = (s[0] + s[1]) + (s[2] + s[3]);
}

dim3 bwd_block(int D) { return norm_block(D, D > 8192 ? 2 : 1, 256); }

template <typename T, typename RT, bool WIDE, int UPT>
cudaError_t launch_u(const SeqNormParams& p, cudaStream_t stream) {
    const dim3 block = bwd_block(p.D), grid((unsigned)(p.blocks / block.y));
    const bool bias = p.b_post || p.b_pre || p.db_post || p.db_pre;
    cudaError_t e = bias ? launch_kernel(seq_norm_bwd_kernel<T, RT, WIDE, UPT, true>, grid, block, 0, stream, false, 1, p)
                         : launch_kernel(seq_norm_bwd_kernel<T, RT, WIDE, UPT, false>, grid, block, 0, stream, false, 1, p);
    if (e == cudaSuccess && p.ws)
        e = launch_kernel(seq_norm_param_kernel, dim3((unsigned)((p.D + 127) / 128), SUMS), dim3(128), 0, stream, false, 1,
                          p, p.blocks);
    return e;
}

template <typename T, typename RT>
cudaError_t launch(const SeqNormParams& p, cudaStream_t stream) {
    if (p.D > 8192) return p.vec ? launch_u<T, RT, true, 2>(p, stream) : launch_u<T, RT, false, 2>(p, stream);
    return p.vec ? launch_u<T, RT, true, 1>(p, stream) : launch_u<T, RT, false, 1>(p, stream);
}

}  // namespace

// Rows of partial sums: blocks times the rows a block holds at once.
int seq_norm_bwd_blocks(int rows, int D, int sms) {
    const dim3 block = bwd_block(D);
    const int most = (rows + (int)block.y - 1) / (int)block.y;
    const int per_sm = 1024 / (int)(block.x * block.y) < 1 ? 1 : 1024 / (int)(block.x * block.y);
    const int want = sms * per_sm;
    return (most < want ? most : want) * (int)block.y;
}

cudaError_t launch_seq_norm_bwd(const SeqNormParams& p, bool bf16, bool res_bf16, cudaStream_t stream) {
    using B = __nv_bfloat16;
    if (!bf16) return launch<float, float>(p, stream);
    return res_bf16 ? launch<B, B>(p, stream) : launch<B, float>(p, stream);
}

}  // namespace convfwd

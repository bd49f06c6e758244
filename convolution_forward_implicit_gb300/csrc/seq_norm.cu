// Norm, gate and residual around a block, forward: see seq.h for the formulas.  Bound by bytes: each
// row is read once into registers, normalised there (up to twice) and written once.
#include "seq_norm.cuh"

namespace convfwd {
namespace {

template <typename T, typename RT, bool WIDE, int UPT>
__global__ void __launch_bounds__(1024) seq_norm_fwd_kernel(const __grid_constant__ SeqNormParams p) {
    __shared__ float buf[2][32][2];
    int turn = 0;
    const int row = blockIdx.x * blockDim.y + threadIdx.y;
    const bool on = row < p.rows;
    const int D = on ? p.D : 0;            // a row behind the last one has no columns
    const bool layer = p.flags & SEQ_NORM_LAYER;
    float v[UPT][8], a[UPT][8], b[UPT][8];
    row_load<T, WIDE, UPT>(p.x, (long long)row * p.x_ld, D, v);
    if (p.flags & (SEQ_NORM_GATE_BEFORE | SEQ_NORM_GATE_AFTER)) {
        row_load<T, WIDE, UPT>(p.gate, (long long)row * p.gate_ld, D, b);
#pragma unroll
        for (int u = 0; u < UPT; ++u)
#pragma unroll
            for (int e = 0; e < 8; ++e) b[u][e] = silu(b[u][e]);
    }
    if (p.flags & SEQ_NORM_GATE_BEFORE) {
#pragma unroll
        for (int u = 0; u < UPT; ++u)
#pragma unroll
            for (int e = 0; e < 8; ++e) v[u][e] *= b[u][e];
    }
    if (p.flags & SEQ_NORM_POST) {
        row_norm(v, p.D, layer, p.eps, buf, turn);
        col_load<T, WIDE, UPT>(p.w_post, 1.f, D, a);
#pragma unroll
        for (int u = 0; u < UPT; ++u)
#pragma unroll
            for (int e = 0; e < 8; ++e) v[u][e] *= a[u][e];
        if (p.b_post) {
            col_load<T, WIDE, UPT>(p.b_post, 0.f, D, a);
#pragma unroll
            for (int u = 0; u < UPT; ++u)
#pragma unroll
                for (int e = 0; e < 8; ++e) v[u][e] += a[u][e];
        }
    }
    if (p.flags & SEQ_NORM_GATE_AFTER) {
#pragma unroll
        for (int u = 0; u < UPT; ++u)
#pragma unroll
            for (int e = 0; e < 8; ++e) v[u][e] *= b[u][e];
    }
    if (p.scale) {
        col_load<T, WIDE, UPT>(p.scale, 1.f, D, a);
#pragma unroll
        for (int u = 0; u < UPT; ++u)
#pragma unroll
            for (int e = 0; e < 8; ++e) v[u][e] *= a[u][e];
    }
    if (p.flags & SEQ_NORM_RESIDUAL) {
        row_load<RT, WIDE, UPT>(p.res, (long long)row * p.res_ld, D, a);
#pragma unroll
        for (int u = 0; u < UPT; ++u)
#pragma unroll
            for (int e = 0; e < 8; ++e) v[u][e] += a[u][e];
        row_store<RT, WIDE, UPT>(p.res_out, (long long)row * p.res_out_ld, D, v);
    }
    if (p.flags & SEQ_NORM_PRE) {
        row_norm(v, p.D, layer, p.eps, buf, turn);
        col_load<T, WIDE, UPT>(p.w_pre, 1.f, D, a);
        col_load<T, WIDE, UPT>(p.b_pre, 0.f, D, b);
#pragma unroll
        for (int u = 0; u < UPT; ++u)
#pragma unroll
            for (int e = 0; e < 8; ++e) v[u][e] = fmaf(v[u][e], a[u][e], b[u][e]);
    }
    if ((p.flags & SEQ_NORM_PRE) || !(p.flags & SEQ_NORM_RESIDUAL))
        row_store<T, WIDE, UPT>(p.y, (long long)row * p.y_ld, D, v);
}

template <typename T, typename RT, bool WIDE>
cudaError_t launch(const SeqNormParams& p, cudaStream_t stream) {
    const int upt = p.D > 8192 ? 2 : 1;
    const dim3 block = norm_block(p.D, upt, 128);
    const dim3 grid((unsigned)((p.rows + block.y - 1) / block.y));
    return upt == 2 ? launch_kernel(seq_norm_fwd_kernel<T, RT, WIDE, 2>, grid, block, 0, stream, false, 1, p)
                    : launch_kernel(seq_norm_fwd_kernel<T, RT, WIDE, 1>, grid, block, 0, stream, false, 1, p);
}

}  // namespace

cudaError_t launch_seq_norm_fwd(const SeqNormParams& p, bool bf16, bool res_bf16, cudaStream_t stream) {
    using B = __nv_bfloat16;
    if (!bf16) return p.vec ? launch<float, float, true>(p, stream) : launch<float, float, false>(p, stream);
    if (res_bf16) return p.vec ? launch<B, B, true>(p, stream) : launch<B, B, false>(p, stream);
    return p.vec ? launch<B, float, true>(p, stream) : launch<B, float, false>(p, stream);
}

}  // namespace convfwd

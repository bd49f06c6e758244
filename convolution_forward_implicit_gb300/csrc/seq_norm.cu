// Norm, gate and residual around a block, forward: see seq.h for the formulas.  Bound by bytes: each
// row is read once into registers (all of its tensors before the first sum), normalised there, up to twice,
// and written once.  A block has one row, or several narrow ones; many blocks on an SM hide the barriers of
// each other's sums.  8192 x 4096 bf16 with an fp32 residual and everything on: 75 us for 470 MB, 94% of a plain
// copy's rate; 6007 x 1280 fp32 layer norm: 24 us for 123 MB (77%).
#include "seq_norm.cuh"

namespace convfwd {
namespace {

template <typename T, typename RT, bool WIDE, int UPT, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) seq_norm_fwd_kernel(const __grid_constant__ SeqNormParams p) {
    __shared__ __align__(16) NormSums buf;
    RowSums<THREADS> sums;
    const long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y;
    const int D = row < p.rows ? p.D : 0;            // a row behind the last one has no columns
    const bool layer = p.flags & SEQ_NORM_LAYER, gate = p.flags & (SEQ_NORM_GATE_BEFORE | SEQ_NORM_GATE_AFTER);
    const bool residual = p.flags & SEQ_NORM_RESIDUAL;
    // all of the row is on its way before the first sum (a thread stores the residual's columns that it has loaded
    // itself, so that res_out may be res)
    RowIn<T, WIDE, UPT> x_in, g_in;
    RowIn<RT, WIDE, UPT> r_in;
    x_in.load(p.x, row * p.x_ld, D);
    if (gate) g_in.load(p.gate, row * p.gate_ld, D);
    if (residual) r_in.load(p.res, row * p.res_ld, D);
    sums.template init<UPT>(buf, p.D);
    float2 v[UPT][4], a[UPT][4];
    x_in.get(v);
    if (p.flags & SEQ_NORM_GATE_BEFORE) {
        g_in.get(a);
        EACH_PAIR v[u][e] = pmul(v[u][e], silu2(a[u][e]));
    }
    if (p.flags & SEQ_NORM_POST) {
        row_norm<WIDE>(v, p.D, layer, p.eps, sums, D > 0);
        col_mul<T, WIDE, UPT>(p.w_post, D, v);
        col_add<T, WIDE, UPT>(p.b_post, D, v);
    }
    if (p.flags & SEQ_NORM_GATE_AFTER) {
        g_in.get(a);
        EACH_PAIR v[u][e] = pmul(v[u][e], silu2(a[u][e]));
    }
    col_mul<T, WIDE, UPT>(p.scale, D, v);
    if (residual) {
        r_in.get(a);
        EACH_PAIR v[u][e] = padd(v[u][e], a[u][e]);
        row_store<RT, WIDE, UPT>(p.res_out, row * p.res_out_ld, D, v);
    }
    if (p.flags & SEQ_NORM_PRE) {
        row_norm<WIDE>(v, p.D, layer, p.eps, sums, D > 0);
        col_mul<T, WIDE, UPT>(p.w_pre, D, v);
        col_add<T, WIDE, UPT>(p.b_pre, D, v);
    }
    if ((p.flags & SEQ_NORM_PRE) || !residual) row_store<T, WIDE, UPT>(p.y, row * p.y_ld, D, v);
}

template <typename T, typename RT, bool WIDE, int UPT, int THREADS>
cudaError_t launch_u(const SeqNormParams& p, cudaStream_t stream) {
    const dim3 block = norm_block(p.D, UPT);
    return launch_kernel(seq_norm_fwd_kernel<T, RT, WIDE, UPT, THREADS>, dim3((unsigned)((p.rows + block.y - 1) / block.y)), block, 0, stream,
                         false, 1, p);
}

template <typename T, typename RT, bool WIDE>
cudaError_t launch(const SeqNormParams& p, cudaStream_t stream) {
    // 8 values a thread keep more rows in flight; 16 halve what the sums cost each
    if (p.D <= 2048) return launch_u<T, RT, WIDE, 1, 256>(p, stream);
    if (p.D <= 4096) return p.rows < 4 * p.sms ? launch_u<T, RT, WIDE, 1, 512>(p, stream) : launch_u<T, RT, WIDE, 2, 256>(p, stream);
    if (p.D <= 8192) return launch_u<T, RT, WIDE, 2, 512>(p, stream);
    return launch_u<T, RT, WIDE, 2, 1024>(p, stream);
}

}  // namespace

cudaError_t launch_seq_norm_fwd(const SeqNormParams& p, bool bf16, bool res_bf16, cudaStream_t stream) {
    using B = __nv_bfloat16;
    if (!bf16) return p.vec ? launch<float, float, true>(p, stream) : launch<float, float, false>(p, stream);
    if (res_bf16) return p.vec ? launch<B, B, true>(p, stream) : launch<B, B, false>(p, stream);
    return p.vec ? launch<B, float, true>(p, stream) : launch<B, float, false>(p, stream);
}

}  // namespace convfwd

// Norm, gate and residual around a block, gradients.  With hat = norm(v), r = 1 / sqrt(...) and d the
// gradient at w hat + b:  dw = sum_rows d hat, db = sum_rows d, and at v, with e = d w,
//   dv = r (e - hat mean(e hat))           (RMS; layer: also less mean(e)).
// The sums S1 = sum_rows d' hat and S0 = sum_rows d' over the rows of POST, with d' the gradient at r (times
// silu(gate) where it comes after), serve three parameters: r = res + scale (w_post hat + b_post) gives
//   dw_post = scale S1,   db_post = scale S0,   dscale = w_post S1 + b_post S0.
// Bound by bytes.  A block keeps its share of the rows' parameter sums in registers (its threads stay
// on their columns), writes them once, and a second kernel adds the blocks up in their order.
//
// 8192 x 4096 bf16 with an fp32 residual and everything on: 180 us for 738 MB (4.1 TB/s, 61% of a plain copy's
// rate); 6007 x 1280 fp32 layer norm: 48 us for 185 MB (58%).  With the sums' registers, 15 or 16 warps an SM: each
// row is a chain of loads, special functions, sums and barriers that few other rows overlap.  Above 4096 columns a thread has
// 16 and spills (bytes stored without and with biases: up to 372 and 828 where rows pass through shared memory, 984 and
// 1264 in blocks of 1024 threads): 4096 x 5120 bf16 with everything on 179 us, 4096 x 8192 253 (cold; 39 and 44%).
#include "seq_norm.cuh"

namespace convfwd {
namespace {

constexpr int SUMS = 4;      // S1, S0, and those of w_pre and b_pre

// d (the gradient behind w) -> the gradient at v, in place, with hat, its r, c = mean(d hat), m = mean(d)
template <bool WIDE, int UPT>
__device__ __forceinline__ void norm_back(float2 (&d)[UPT][4], const float2 (&hat)[UPT][4], float r, float c, float m, int D, bool layer) {
    if (layer) row_shift<WIDE>(d, D, m);
    EACH_PAIR d[u][e] = pmul(pdup(r), pfma(hat[u][e], pdup(-c), d[u][e]));
}

// A block walks its rows.  RING: the next row is on its way to shared memory while this one is computed,
// and what a row needs twice (x, gate) is taken from there twice.
template <typename T, typename RT, bool WIDE, bool RING, int UPT, bool BIAS, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS <= 512 ? 512 / THREADS : 1) seq_norm_bwd_kernel(const __grid_constant__ SeqNormParams p) {
    extern __shared__ __align__(16) unsigned char ring[];
    __shared__ __align__(16) NormSums buf;
    constexpr bool ONE = THREADS > 128 && RING;      // one row at a time
    const int ty = ONE ? 0 : threadIdx.y, rows_at_once = ONE ? 1 : blockDim.y;
    const bool layer = p.flags & SEQ_NORM_LAYER;
    const bool post = p.flags & SEQ_NORM_POST, pre = p.flags & SEQ_NORM_PRE, residual = p.flags & SEQ_NORM_RESIDUAL;
    const bool gate = p.flags & (SEQ_NORM_GATE_BEFORE | SEQ_NORM_GATE_AFTER), after = p.flags & SEQ_NORM_GATE_AFTER;
    const bool has_dy = pre || !residual, has_dro = residual && p.dres_out, use_res = residual && pre;
    constexpr int tb = row_bytes<T, UPT, THREADS>(), rb = row_bytes<RT, UPT, THREADS>();
    // places in a stage: x, gate, dy, res, dres_out
    const int at_g = tb, at_dy = at_g + (gate ? tb : 0), at_res = at_dy + (has_dy ? tb : 0), at_dro = at_res + (use_res ? rb : 0);
    const int stage_bytes = at_dro + (has_dro ? rb : 0);
    uint32_t mine = (uint32_t)__cvta_generic_to_shared(ring) + (ty * blockDim.x + threadIdx.x) * 16;
    asm volatile("" : "+r"(mine));             // (not to be worked out again at every use)
    const float inv_D = 1.0f / (float)p.D;
    const long long step = (long long)gridDim.x * rows_at_once;
    auto fetch = [&](long long row, int stage) {
        if (!RING) return;
        if (row < p.rows) {
            const uint32_t at = mine + stage * stage_bytes;
            row_copy<T, UPT, THREADS>(at, p.x, row * p.x_ld, p.D);
            if (gate) row_copy<T, UPT, THREADS>(at + at_g, p.gate, row * p.gate_ld, p.D);
            if (has_dy) row_copy<T, UPT, THREADS>(at + at_dy, p.dy, row * p.dy_ld, p.D);
            if (use_res) row_copy<RT, UPT, THREADS>(at + at_res, p.res, row * p.res_ld, p.D);
            if (has_dro) row_copy<RT, UPT, THREADS>(at + at_dro, p.dres_out, row * p.dres_out_ld, p.D);
        }
        copies_commit();
    };
    float2 s_1[UPT][4], s_0[UPT][4], s_wpre[UPT][4], s_bpre[UPT][4];
    EACH_PAIR s_1[u][e] = s_0[u][e] = s_wpre[u][e] = s_bpre[u][e] = make_float2(0.f, 0.f);
    long long row = (long long)blockIdx.x * rows_at_once + ty;
#pragma unroll
    for (int i = 0; i < NORM_RING - 1; ++i) fetch(row + i * step, i);
    int stage = 0;
    Column<T, WIDE, UPT, THREADS <= 512, true> w_post, scale, w_pre;
    Column<T, WIDE, UPT, THREADS <= 512, false> b_post;
    w_post.open(p.w_post, p.D);
    b_post.open(BIAS ? p.b_post : nullptr, p.D);
    scale.open(p.scale, p.D);
    w_pre.open(p.w_pre, p.D);
    RowSums<THREADS> sums;
    sums.template init<UPT>(buf, p.D);
    for (long long base = (long long)blockIdx.x * rows_at_once; base < p.rows; base += step, row += step, stage = stage == NORM_RING - 1 ? 0 : stage + 1) {
        fetch(row + (NORM_RING - 1) * step, stage == 0 ? NORM_RING - 1 : stage - 1);
        const int D = ONE || row < p.rows ? p.D : 0;
        const uint32_t at = mine + stage * stage_bytes;
        if (RING) copies_wait<NORM_RING - 1>();
        auto take = [&](auto type, const void* from, long long ld, int place, float2 (&v)[UPT][4]) {
            using E = decltype(type);
            if (RING) {
                row_take<E, UPT, THREADS>(at + place, v);
                if (!ONE && D == 0) EACH_PAIR v[u][e] = make_float2(0.f, 0.f);
            } else {
                row_load<E, WIDE, UPT>(from, row * ld, D, v);
            }
        };
        // behind POST: u from its hat, times silu(gate) if it comes after
        auto behind_post = [&](float2 (&v)[UPT][4], bool gated) {
            if (post) {
                w_post.mul(D, v);
                if (BIAS) b_post.add(D, v);
            }
            if (after && gated) {
                float2 g[UPT][4];
                take(T(), p.gate, p.gate_ld, at_g, g);
                EACH_PAIR v[u][e] = pmul(v[u][e], silu2(g[u][e]));
            }
        };
        float2 hat[UPT][4], d[UPT][4];
        float r_post = 0.f;
        take(T(), p.x, p.x_ld, 0, hat);
        if (gate && !after) {
            float2 g[UPT][4];
            take(T(), p.gate, p.gate_ld, at_g, g);
            EACH_PAIR hat[u][e] = pmul(hat[u][e], silu2(g[u][e]));
        }
        if (post) r_post = row_norm<WIDE>(hat, p.D, layer, p.eps, sums, D > 0);
        // d: the gradient at r
        if (has_dy) take(T(), p.dy, p.dy_ld, at_dy, d);
        else EACH_PAIR d[u][e] = make_float2(0.f, 0.f);
        if (pre) {
            float2 hat2[UPT][4];
            EACH_PAIR hat2[u][e] = hat[u][e];
            behind_post(hat2, true);
            scale.mul(D, hat2);
            if (use_res) {
                float2 r[UPT][4];
                take(RT(), p.res, p.res_ld, at_res, r);
                EACH_PAIR hat2[u][e] = padd(hat2[u][e], r[u][e]);
            }
            // hat2 is still v.  Its norm and the sums behind the gradient through it need one barrier together:
            // mean(e hat) = r mean(e (v - mean)), e = d w.
            float q, c, m = 0.f;
            {
                float2 e_[UPT][4];
                EACH_PAIR e_[u][e] = d[u][e];
                w_pre.mul(D, e_);
                if (layer) {
                    const float first = sums.warp(lane_total(hat2), lane_total(e_));
                    const float mine_m = __shfl_sync(~0u, first, 0) * sums.inv_n;
                    row_shift<WIDE>(hat2, p.D, mine_m);
                    sums.store(sums.half, threadIdx.x & 16 ? first : mine_m);
                    sums.store(sums.half + 2 * 64 * 4, sums.warp(lane_dot(hat2, hat2), lane_dot(e_, hat2)));
                    sums.barrier();
                    float mean;
                    row_moments<true>(sums, inv_D, mean, q, c, m);
                    sums.next();
                    row_shift<WIDE>(hat2, p.D, mean - mine_m);
                } else {
                    q = lane_dot(hat2, hat2);
                    c = lane_dot(e_, hat2);
                    sums.sum(q, c);
                }
            }
            const float r_pre = norm_factor(fmaf(q, inv_D, p.eps), D > 0);
            EACH_PAIR hat2[u][e] = pmul(hat2[u][e], pdup(r_pre));
            EACH_PAIR s_wpre[u][e] = pfma(d[u][e], hat2[u][e], s_wpre[u][e]);
            if (BIAS) EACH_PAIR s_bpre[u][e] = padd(d[u][e], s_bpre[u][e]);
            w_pre.mul(D, d);
            norm_back<WIDE>(d, hat2, r_pre, c * r_pre * inv_D, m * inv_D, p.D, layer);
        }
        if (residual) {
            if (has_dro) {
                float2 r[UPT][4];
                take(RT(), p.dres_out, p.dres_out_ld, at_dro, r);
                EACH_PAIR d[u][e] = padd(d[u][e], r[u][e]);
            }
            row_store<RT, WIDE, UPT>(p.dres, row * p.dres_ld, D, d);
        }
        // back through scale, gate, POST, gate
        // through u * silu(g): dg = d u silu'(g), d *= silu(g)
        auto back_gate = [&](float2 (&n)[UPT][4]) {
            float2 g[UPT][4];
            take(T(), p.gate, p.gate_ld, at_g, g);
            EACH_PAIR {
                const float2 s = make_float2(sigmoid(g[u][e].x), sigmoid(g[u][e].y)), v = g[u][e], dv = pmul(d[u][e], s);
                // silu' = s (1 + v (1 - s))
                n[u][e] = pmul(pmul(dv, n[u][e]), pfma(v, padd(pdup(1.f), make_float2(-s.x, -s.y)), pdup(1.f)));
                d[u][e] = pmul(dv, v);
            }
            row_store<T, WIDE, UPT>(p.dgate, row * p.dgate_ld, D, n);
        };
        if (after) {
            float2 n[UPT][4];
            EACH_PAIR n[u][e] = hat[u][e];
            behind_post(n, false);
            scale.mul(D, n);                   // (d has not been through scale yet)
            back_gate(n);
        }
        EACH_PAIR s_1[u][e] = pfma(d[u][e], hat[u][e], s_1[u][e]);
        if (BIAS) EACH_PAIR s_0[u][e] = padd(d[u][e], s_0[u][e]);
        scale.mul(D, d);
        if (post) {
            w_post.mul(D, d);
            float c = lane_dot(d, hat), m = 0.f;
            if (layer) {
                m = lane_total(d);
                sums.sum(c, m);
            } else {
                c = sums.sum(c);
            }
            norm_back<WIDE>(d, hat, r_post, c * inv_D, m * inv_D, p.D, layer);
        }
        if (gate && !after) {
            float2 n[UPT][4];
            take(T(), p.x, p.x_ld, 0, n);
            back_gate(n);
        }
        row_store<T, WIDE, UPT>(p.dx, row * p.dx_ld, D, d);
    }
    griddep_launch();
    if (!p.ws) return;
    const long long part = ((long long)blockIdx.x * rows_at_once + ty) * SUMS * p.D;
    row_store<float, WIDE, UPT>(p.ws, part, p.D, s_1);
    if (BIAS) row_store<float, WIDE, UPT>(p.ws, part + p.D, p.D, s_0);
    if (p.dw_pre) row_store<float, WIDE, UPT>(p.ws, part + 2 * p.D, p.D, s_wpre);
    if (BIAS && p.db_pre) row_store<float, WIDE, UPT>(p.ws, part + 3 * p.D, p.D, s_bpre);
}

// The parameters' gradients: the blocks' rows of partial sums, added up in a fixed order.
template <typename T>
__global__ void __launch_bounds__(COLUMN_THREADS, 2) seq_norm_param_kernel(const __grid_constant__ SeqNormParams p, int parts, bool bias) {
    griddep_wait();
    const int c = blockIdx.x * 32 + (threadIdx.x & 31);
    const bool on = c < p.D, first = threadIdx.x < 32 && on;
    auto total = [&](int k) { return column_sum(p.ws + (long long)k * p.D + c, (long long)SUMS * p.D, parts, on); };
    auto param = [&](const void* v, float none) { return v && on ? seq_ld(static_cast<const T*>(v) + c) : none; };
    // y 0: S1 alone; 1 (with biases): S1 and S0; 2, 3: those of w_pre and b_pre
    if (blockIdx.y == 0) {
        if (!p.dw_post && (bias || !p.dscale)) return;
        const float s1 = total(0);
        if (first && p.dw_post) p.dw_post[c] = param(p.scale, 1.f) * s1;
        if (first && !bias && p.dscale) p.dscale[c] = param(p.w_post, 1.f) * s1;
    } else if (blockIdx.y == 1) {
        if (!bias || (!p.db_post && !p.dscale)) return;
        const float s0 = total(1);
        if (first && p.db_post) p.db_post[c] = param(p.scale, 1.f) * s0;
        if (!p.dscale) return;
        __syncthreads();
        const float s1 = total(0);
        if (first) p.dscale[c] = fmaf(param(p.w_post, 1.f), s1, param(p.b_post, 0.f) * s0);
    } else {
        float* out = blockIdx.y == 2 ? p.dw_pre : p.db_pre;
        if (!out) return;
        const float v = total(blockIdx.y);
        if (first) out[c] = v;
    }
}

// How rows are spread: upt groups of 8 columns to a thread, `threads` (128, 256, 512 or 1024) at most in a
// block, rows through shared memory or not.
struct Shape {
    int upt, threads;
    bool ring;
    dim3 block;
    int smem, blocks;
};
// `wide`: rows of aligned groups.  8 columns a thread up to 4096 (8192 x 4096 bf16 with everything on, measured before
// the sums shared their barriers: 204 us with one block of 512 threads an SM; 212 with two of 256 and 16 columns
// each, which spills; 237 with two of 512 and 64 registers).
Shape shape_of(int rows, int D, unsigned flags, bool wide, int esize, int rsize, int sms) {
    const bool gate = flags & (SEQ_NORM_GATE_BEFORE | SEQ_NORM_GATE_AFTER), residual = flags & SEQ_NORM_RESIDUAL;
    const bool pre = flags & SEQ_NORM_PRE;
    const int row = esize * (1 + gate + (pre || !residual)) + rsize * ((residual && pre) + residual);
    Shape s;
    s.upt = D > 4096 ? 2 : 1;
    s.block = norm_block(D, s.upt);
    const int threads = (int)(s.block.x * s.block.y);
    s.threads = threads <= 128 ? 128 : threads <= 256 ? 256 : 512;
    s.smem = NORM_RING * s.threads * s.upt * 8 * row;
    s.ring = wide && D <= 8192 && s.smem <= NORM_RING_MAX;
    if (!s.ring) {
        s.smem = 0;
        s.threads = s.upt == 1 ? 512 : 1024;
    }
    int fit = 65536 / ((s.threads == 1024 ? 64 : 128) * threads);
    if (s.smem > 0 && 228 * 1024 / (s.smem + 3584) < fit) fit = 228 * 1024 / (s.smem + 3584);
    const int most = (rows + (int)s.block.y - 1) / (int)s.block.y, want = (fit < 1 ? 1 : fit) * sms;
    s.blocks = most < want ? most : want;
    return s;
}

template <typename T, typename RT, bool WIDE, bool RING, int UPT, int THREADS>
cudaError_t launch_u(const SeqNormParams& p, const Shape& s, bool bias, cudaStream_t stream) {
    const auto kernel = bias ? seq_norm_bwd_kernel<T, RT, WIDE, RING, UPT, true, THREADS> : seq_norm_bwd_kernel<T, RT, WIDE, RING, UPT, false, THREADS>;
    // always the same limit, not this call's bytes: host threads may call at the same time, and what one sets must
    // do for the other's launch
    cudaError_t e = RING ? cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, NORM_RING_MAX) : cudaSuccess;
    if (e == cudaSuccess) e = launch_kernel(kernel, dim3((unsigned)s.blocks), s.block, (size_t)s.smem, stream, false, 1, p);
    if (e == cudaSuccess && p.ws)
        e = launch_kernel(seq_norm_param_kernel<T>, dim3((unsigned)((p.D + 31) / 32), SUMS), dim3(COLUMN_THREADS), 0, stream, true, 1, p,
                          s.blocks * (int)s.block.y, bias);
    return e;
}

template <typename T, typename RT>
cudaError_t launch(const SeqNormParams& p, cudaStream_t stream) {
    const bool bias = p.b_post || p.b_pre;
    const Shape s = shape_of(p.rows, p.D, p.flags, p.vec, (int)sizeof(T), (int)sizeof(RT), p.sms);
    if (s.ring) {
        if (s.upt == 2) return launch_u<T, RT, true, true, 2, 512>(p, s, bias, stream);
        return s.threads == 128   ? launch_u<T, RT, true, true, 1, 128>(p, s, bias, stream)
               : s.threads == 256 ? launch_u<T, RT, true, true, 1, 256>(p, s, bias, stream)
                                  : launch_u<T, RT, true, true, 1, 512>(p, s, bias, stream);
    }
    if (s.threads == 1024) return p.vec ? launch_u<T, RT, true, false, 2, 1024>(p, s, bias, stream) : launch_u<T, RT, false, false, 2, 1024>(p, s, bias, stream);
    return p.vec ? launch_u<T, RT, true, false, 1, 512>(p, s, bias, stream) : launch_u<T, RT, false, false, 1, 512>(p, s, bias, stream);
}

}  // namespace

// Rows of partial sums at most, with and without wide rows.
int seq_norm_bwd_blocks(int rows, int D, unsigned flags, int esize, int rsize, int sms) {
    int most = 1;
    for (int wide = 0; wide < 2; ++wide) {
        const Shape s = shape_of(rows, D, flags, wide, esize, rsize, sms);
        const int parts = s.blocks * (int)s.block.y;
        if (parts > most) most = parts;
    }
    return most;
}

cudaError_t launch_seq_norm_bwd(const SeqNormParams& p, bool bf16, bool res_bf16, cudaStream_t stream) {
    using B = __nv_bfloat16;
    if (!bf16) return launch<float, float>(p, stream);
    return res_bf16 ? launch<B, B>(p, stream) : launch<B, float>(p, stream);
}

}  // namespace convfwd

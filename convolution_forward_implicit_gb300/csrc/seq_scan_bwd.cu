// Selective state space scan, gradients.  With dyc_t = dy_t silu(z_t), a_t = exp(delta_t A) and
// g_t the gradient at h_t,
//   g_t = C_t dyc_t + a_{t+1} g_{t+1},          q_t = g_t a_t h_{t-1}   (the gradient at delta_t A)
//   dx_t = delta_t (sum_n g_t B_t) + D dyc_t,   ddelta_t = sum_n q_t A + x_t sum_n g_t B_t
//   dA = sum_t q_t delta_t,  dB_t = sum_d g_t delta_t x_t,  dC_t = sum_d h_t dyc_t
//   dz_t = dy_t (C_t . h_t + D x_t) silu'(z_t),  dD = sum_t dyc_t x_t,  ddt_bias = sum_t ddt_t
//
// A block walks a piece backwards, a tile of SCAN_TILE tokens at a time: from the state saved at the
// tile's first token it runs the recurrence forward again, keeping the state before every token in
// shared memory, and then backward.  A thread holds 4 channels x 4 states; LN lanes share a channel's
// states and the 32 / LN groups of lanes hold different channels, so the sums over states (dx, ddelta,
// dz) and those over channels (dB, dC) both are sums over lanes of a warp: each lane gives away half of
// its values a step (4 or 8 values over as many lanes cost 3 or 7 shuffles, not 12 or 24).  dB and dC
// of a block's channels leave as partial rows, which a second kernel adds up in block order.
#include "seq_scan.cuh"

namespace convfwd {
namespace {

constexpr int THREADS = 128, WARPS = THREADS / 32;

// Sums K values over R lanes whose numbers differ by multiples of STRIDE (R, K powers of two).  Lane
// bits from the highest down choose halves: on return v[0 .. max(K / R, 1) - 1] are the sums of the
// values from `return` on.
template <int K, int R, int STRIDE>
__device__ __forceinline__ int lane_sum(float* v) {
    if constexpr (R == 1) {
        return 0;
    } else {
        constexpr int O = STRIDE * R / 2;
        if constexpr (K > 1) {
            const bool up = threadIdx.x & O;
#pragma unroll
            for (int i = 0; i < K / 2; ++i) {
                const float give = up ? v[i] : v[i + K / 2];
                const float keep = up ? v[i + K / 2] : v[i];
                v[i] = keep + __shfl_xor_sync(~0u, give, O);
            }
            return (up ? K / 2 : 0) + lane_sum<K / 2, R / 2, STRIDE>(v);
        } else {
            v[0] += __shfl_xor_sync(~0u, v[0], O);
            return lane_sum<1, R / 2, STRIDE>(v);
        }
    }
}

template <int LN>
struct BwdShape {
    static constexpr int CPW = 32 / LN * 4;       // channels per warp
    static constexpr int CB = CPW * WARPS;        // channels per block
    static constexpr int NP = LN * 4;             // states, padded
    static constexpr int CPL = CB > THREADS ? CB / THREADS : 1;   // channels per thread outside the recurrence
};
template <int LN>
struct BwdSmem {
    using S = BwdShape<LN>;
    float4 h[SCAN_TILE][4][THREADS];              // the states before each token
    float delta[SCAN_TILE][S::CB], u[SCAN_TILE][S::CB], dyc[SCAN_TILE][S::CB];
    float gB[SCAN_TILE][S::CB], qA[SCAN_TILE][S::CB], Ch[SCAN_TILE][S::CB];
    float B[SCAN_TILE][S::NP], C[SCAN_TILE][S::NP];
    float bc[WARPS][SCAN_TILE][2][S::NP];
    ScanBounds sb;
};

template <typename T, int LN>
__global__ void __launch_bounds__(THREADS) seq_scan_bwd_kernel(const __grid_constant__ SeqScanParams p) {
    using S = BwdShape<LN>;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    BwdSmem<LN>& sm = *reinterpret_cast<BwdSmem<LN>*>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int piece = blockIdx.x;
    int t0, t1;
    scan_piece_range(p.ax, p.pc, piece, t0, t1);
    const int per = p.D / p.G, bpg = (per + S::CB - 1) / S::CB;
    const int g = blockIdx.y / bpg;
    const int cb0 = (blockIdx.y - g * bpg) * S::CB;              // the block's first channel in its group
    const int n0 = lane % LN * 4;
    const int cw = warp * S::CPW + lane / LN * 4;                // the thread's first channel in the block
    float A2[4][4], gam[4][4], dA[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int cl = cb0 + cw + i;
            A2[i][k] = cl < per && n0 + k < p.N ? p.A[(long long)(g * per + cl) * p.N + n0 + k] * LOG2E : 0.f;
            gam[i][k] = dA[i][k] = 0.f;
        }
    float sumD[S::CPL] = {}, sumdt[S::CPL] = {};
    const int quads = (p.N + 3) >> 2;

    const int tiles = (t1 - t0 + SCAN_TILE - 1) / SCAN_TILE;
    for (int tile = tiles - 1; tile >= 0; --tile) {
        const int tb = t0 + tile * SCAN_TILE, n = min(SCAN_TILE, t1 - tb);
        __syncthreads();
        for (int i = tid; i < n * S::NP; i += THREADS) {
            const int t = i / S::NP, k = i - t * S::NP;
            sm.B[t][k] = k < p.N ? seq_ld(static_cast<const T*>(p.B) + (long long)(tb + t) * p.B_ld + g * p.N + k) : 0.f;
            sm.C[t][k] = k < p.N ? seq_ld(static_cast<const T*>(p.C) + (long long)(tb + t) * p.C_ld + g * p.N + k) : 0.f;
        }
        for (int i = tid; i < n * S::CB; i += THREADS) {
            const int t = i / S::CB, c = i - t * S::CB;
            float delta = 0.f, u = 0.f, dyc = 0.f;
            if (cb0 + c < per) {
                const int d = g * per + cb0 + c;
                const long long tt = tb + t;
                delta = seq_ld(static_cast<const T*>(p.dt) + tt * p.dt_ld + d) + (p.dt_bias ? p.dt_bias[d] : 0.f);
                if (p.softplus) delta = softplus(delta);
                u = delta * seq_ld(static_cast<const T*>(p.x) + tt * p.x_ld + d);
                dyc = seq_ld(static_cast<const T*>(p.dy) + tt * p.dy_ld + d);
                if (p.z) dyc *= silu(seq_ld(static_cast<const T*>(p.z) + tt * p.z_ld + d));
            }
            sm.delta[t][c] = delta;
            sm.u[t][c] = u;
            sm.dyc[t][c] = dyc;
        }
        if (warp == 0) scan_bounds(p.ax, tb, n, &sm.sb);
        __syncthreads();
        const unsigned first = sm.sb.first, last = sm.sb.last;
        // forward again
        {
            float h[4][4];
            const long long row = scan_tile_row(p.ax, tb);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                if (cb0 + cw + i < per && n0 < quads * 4)
                    v = *reinterpret_cast<const float4*>(p.saved + scan_state_at(p, row, n0 >> 2, g * per + cb0 + cw + i));
                h[i][0] = v.x; h[i][1] = v.y; h[i][2] = v.z; h[i][3] = v.w;
            }
            for (int t = 0; t < n; ++t) {
                if (t > 0 && (first >> t & 1)) {
                    const long long slot = seq_slot(p.sl, sm.sb.seq[t]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (cb0 + cw + i < per) {
                            scan_h_load<4>(p, p.h_in, slot, g * per + cb0 + cw + i, n0, h[i]);
                        } else {
#pragma unroll
                            for (int k = 0; k < 4; ++k) h[i][k] = 0.f;
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    sm.h[t][i][tid] = make_float4(h[i][0], h[i][1], h[i][2], h[i][3]);
                    const float delta = sm.delta[t][cw + i], u = sm.u[t][cw + i];
#pragma unroll
                    for (int k = 0; k < 4; ++k) h[i][k] = fmaf(ex2_approx(delta * A2[i][k]), h[i][k], u * sm.B[t][n0 + k]);
                }
            }
        }
        // backward
        for (int t = n - 1; t >= 0; --t) {
            if (last >> t & 1) {
                const long long slot = seq_slot(p.sl, sm.sb.seq[t]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (cb0 + cw + i < per) {
                        scan_h_load<4>(p, p.dh_out, slot, g * per + cb0 + cw + i, n0, gam[i]);
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k) gam[i][k] = 0.f;
                    }
                }
            }
            float bc[8] = {}, gB[4] = {}, qA[4] = {}, Ch[4] = {};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float delta = sm.delta[t][cw + i], u = sm.u[t][cw + i], dyc = sm.dyc[t][cw + i];
                const float4 hv = sm.h[t][i][tid];
                const float hp[4] = {hv.x, hv.y, hv.z, hv.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float b = sm.B[t][n0 + k], c = sm.C[t][n0 + k];
                    const float a = ex2_approx(delta * A2[i][k]);
                    const float ah = a * hp[k];
                    const float h = fmaf(u, b, ah);
                    const float gr = fmaf(c, dyc, gam[i][k]);
                    Ch[i] = fmaf(c, h, Ch[i]);
                    bc[4 + k] = fmaf(dyc, h, bc[4 + k]);
                    bc[k] = fmaf(gr, u, bc[k]);
                    gB[i] = fmaf(gr, b, gB[i]);
                    const float q = gr * ah;
                    qA[i] = fmaf(q, A2[i][k], qA[i]);
                    dA[i][k] = fmaf(q, delta, dA[i][k]);
                    gam[i][k] = gr * a;
                }
            }
            if ((first >> t & 1) && p.dh_in) {
                const long long slot = seq_slot(p.sl, sm.sb.seq[t]);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (cb0 + cw + i < per) scan_h_store<4>(p, p.dh_in, slot, g * per + cb0 + cw + i, n0, gam[i]);
            }
            const int bi = lane_sum<8, 32 / LN, LN>(bc);
            constexpr int BK = 8 * LN / 32 > 1 ? 8 * LN / 32 : 1;
            constexpr int BD = LN < 4 ? 4 / LN : 1;        // lanes that hold the same sums
            if (lane / LN % BD == 0) {
#pragma unroll
                for (int j = 0; j < BK; ++j) sm.bc[warp][t][(bi + j) >> 2][n0 + ((bi + j) & 3)] = bc[j];
            }
            const int ci = lane_sum<4, LN, 1>(gB);
            lane_sum<4, LN, 1>(qA);
            lane_sum<4, LN, 1>(Ch);
            constexpr int CK = LN < 4 ? 4 / LN : 1;
            constexpr int CD = LN > 4 ? LN / 4 : 1;
            if (lane % CD == 0) {
#pragma unroll
                for (int j = 0; j < CK; ++j) {
                    sm.gB[t][cw + ci + j] = gB[j];
                    sm.qA[t][cw + ci + j] = qA[j];
                    sm.Ch[t][cw + ci + j] = Ch[j];
                }
            }
        }
        __syncthreads();
        // per channel and token: dx, ddt, dz; a thread keeps its channel (or channels)
#pragma unroll
        for (int m = 0; m < S::CPL; ++m) {
            const int c = S::CB >= THREADS ? tid + m * THREADS : tid % S::CB;
            if (cb0 + c >= per) continue;
            const int d = g * per + cb0 + c;
            const float Dd = p.Dskip ? p.Dskip[d] : 0.f, bias = p.dt_bias ? p.dt_bias[d] : 0.f;
            for (int t = S::CB >= THREADS ? 0 : tid / S::CB; t < n; t += S::CB >= THREADS ? 1 : THREADS / S::CB) {
                const long long tt = tb + t;
                const float xv = seq_ld(static_cast<const T*>(p.x) + tt * p.x_ld + d);
                const float dyv = seq_ld(static_cast<const T*>(p.dy) + tt * p.dy_ld + d);
                const float dyc = sm.dyc[t][c], gB = sm.gB[t][c];
                seq_st(static_cast<T*>(p.dx) + tt * p.dx_ld + d, fmaf(sm.delta[t][c], gB, Dd * dyc));
                float dd = fmaf(xv, gB, sm.qA[t][c] * 0.6931471805599453f);       // A2 = A / ln 2
                if (p.softplus) dd *= sigmoid(seq_ld(static_cast<const T*>(p.dt) + tt * p.dt_ld + d) + bias);
                seq_st(static_cast<T*>(p.ddt) + tt * p.ddt_ld + d, dd);
                if (p.dz) {
                    const float zv = seq_ld(static_cast<const T*>(p.z) + tt * p.z_ld + d);
                    seq_st(static_cast<T*>(p.dz) + tt * p.dz_ld + d,
                           dyv * fmaf(Dd, xv, sm.Ch[t][c]) * silu_grad(zv, sigmoid(zv)));
                }
                sumD[m] = fmaf(dyc, xv, sumD[m]);
                sumdt[m] += dd;
            }
        }
        for (int i = tid; i < n * 2 * p.N; i += THREADS) {
            const int t = i / (2 * p.N), r = i - t * 2 * p.N, w = r >= p.N, k = r - w * p.N;
            float s = 0.f;
#pragma unroll
            for (int j = 0; j < WARPS; ++j) s += sm.bc[j][t][w][k];
            p.part_bc[((long long)blockIdx.y * p.ax.T + tb + t) * 2 * p.N + r] = s;
        }
    }
    float* par = p.part_par + (long long)piece * (p.N + 2) * p.D;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (cb0 + cw + i < per) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (n0 + k < p.N) par[(long long)(n0 + k) * p.D + g * per + cb0 + cw + i] = dA[i][k];
        }
    if (S::CB >= THREADS) {
#pragma unroll
        for (int m = 0; m < S::CPL; ++m) {
            const int c = tid + m * THREADS;
            if (cb0 + c < per) {
                par[(long long)p.N * p.D + g * per + cb0 + c] = sumD[m];
                par[(long long)(p.N + 1) * p.D + g * per + cb0 + c] = sumdt[m];
            }
        }
    } else {
        __syncthreads();
        float* red = &sm.bc[0][0][0][0];          // 2 x THREADS values: fewer than bc holds
        red[tid] = sumD[0];
        red[THREADS + tid] = sumdt[0];
        __syncthreads();
        if (tid < S::CB && cb0 + tid < per) {
            float a = 0.f, b = 0.f;
            for (int j = tid; j < THREADS; j += S::CB) {
                a += red[j];
                b += red[THREADS + j];
            }
            par[(long long)p.N * p.D + g * per + cb0 + tid] = a;
            par[(long long)(p.N + 1) * p.D + g * per + cb0 + tid] = b;
        }
    }
}

// dB and dC: the partial rows of a group's channel blocks, added in block order.
template <typename T>
__global__ void __launch_bounds__(128) seq_scan_bc_kernel(const __grid_constant__ SeqScanParams p) {
    const int bpg = p.cblocks / p.G;
    const long long all = (long long)p.ax.T * p.G * 2 * p.N;
    for (long long i = blockIdx.x * 128ll + threadIdx.x; i < all; i += gridDim.x * 128ll) {
        const int r = (int)(i % (2 * p.N));
        const long long tg = i / (2 * p.N);
        const int g = (int)(tg % p.G);
        const long long t = tg / p.G;
        float s = 0.f;
        for (int b = 0; b < bpg; ++b) s += p.part_bc[((long long)(g * bpg + b) * p.ax.T + t) * 2 * p.N + r];
        if (r < p.N) seq_st(static_cast<T*>(p.dB) + t * p.dB_ld + g * p.N + r, s);
        else seq_st(static_cast<T*>(p.dC) + t * p.dC_ld + g * p.N + r - p.N, s);
    }
}

// dA, dD, ddt_bias: the pieces' partial sums, added in piece order.
__global__ void __launch_bounds__(128) seq_scan_par_kernel(const __grid_constant__ SeqScanParams p) {
    const int d = blockIdx.x * 128 + threadIdx.x, k = blockIdx.y;
    if (d >= p.D) return;
    float s[4] = {};
    const float* src = p.part_par + (long long)k * p.D + d;
    const long long step = (long long)(p.N + 2) * p.D;
    const int count = p.ax.T > 0 ? p.pc.count : 0;
    int b = 0;
    for (; b + 4 <= count; b += 4)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] += src[(b + i) * step];
    for (; b < count; ++b) s[0] += src[b * step];
    const float v = (s[0] + s[1]) + (s[2] + s[3]);
    if (k < p.N) p.dA[(long long)d * p.N + k] = v;
    else if (k == p.N) { if (p.dD) p.dD[d] = v; }
    else if (p.ddt_bias) p.ddt_bias[d] = v;
}

template <typename T, int LN>
cudaError_t launch_ln(const SeqScanParams& p, cudaStream_t stream) {
    cudaError_t e = cudaSuccess;
    if (p.ax.T > 0) {
        e = cudaFuncSetAttribute(seq_scan_bwd_kernel<T, LN>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(BwdSmem<LN>));
        if (e == cudaSuccess)
            e = launch_kernel(seq_scan_bwd_kernel<T, LN>, dim3((unsigned)p.pc.count, (unsigned)p.cblocks), dim3(THREADS),
                              sizeof(BwdSmem<LN>), stream, false, 1, p);
        const long long all = ((long long)p.ax.T * p.G * 2 * p.N + 127) / 128;
        if (e == cudaSuccess)
            e = launch_kernel(seq_scan_bc_kernel<T>, dim3((unsigned)(all < 65536 ? all : 65536)), dim3(128), 0, stream, false, 1, p);
    }
    if (e == cudaSuccess && p.dh_in && p.ax.L == 0) e = launch_seq_scan_empty(p, p.dh_out, p.dh_in, stream);
    if (e == cudaSuccess)
        e = launch_kernel(seq_scan_par_kernel, dim3((unsigned)((p.D + 127) / 128), (unsigned)(p.N + 2)), dim3(128), 0, stream,
                          false, 1, p);
    return e;
}

template <typename T>
cudaError_t launch_t(const SeqScanParams& p, cudaStream_t stream) {
    if (p.N <= 8) return launch_ln<T, 2>(p, stream);
    if (p.N <= 16) return launch_ln<T, 4>(p, stream);
    if (p.N <= 32) return launch_ln<T, 8>(p, stream);
    if (p.N <= 64) return launch_ln<T, 16>(p, stream);
    return launch_ln<T, 32>(p, stream);
}

}  // namespace

int seq_scan_bwd_channel_blocks(int D, int N, int G) {
    const int ln = N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : N <= 64 ? 16 : 32;
    const int cb = 32 / ln * 4 * WARPS, per = D / G;
    return G * ((per + cb - 1) / cb);
}

cudaError_t launch_seq_scan_bwd(const SeqScanParams& p, bool bf16, cudaStream_t stream) {
    return bf16 ? launch_t<__nv_bfloat16>(p, stream) : launch_t<float>(p, stream);
}

}  // namespace convfwd

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
//
// 4 x 2048 x 4096 x 16 bf16: 713 us (and 119 for what the pieces send back, see there).  About 490 instructions a
// warp and token of 32 channels x 16 states, where the mathematics needs 120 packed multiply-adds, 41 special
// functions and 16 shuffles; 0.59 a clock and scheduler with three blocks an SM.  Tried, in times of half the case
// (this form: 387): two tokens at a time (380, but spills), the next tile's inputs in registers at two blocks an SM
// (386), loops unrolled 4 and 8 times (457, 648: instruction cache misses), every state in shared memory (392).
#include "seq_scan.cuh"

namespace convfwd {
namespace {

constexpr int THREADS = 128, WARPS = THREADS / 32;

// Sums K values over R lanes whose numbers differ by multiples of STRIDE (R, K powers of two): at each
// step a lane gives away half of its values and adds its partner's to the other half.  Lane bits from the
// highest down choose halves: on return v[0 .. max(K / R, 1) - 1] are the sums of the values from `return`
// on.  SWAPPED: lanes with the highest bit set hold their halves in opposite order (their first half is the
// one they keep), and so their returned place counts in that order.
template <int K, int R, int STRIDE, bool SWAPPED = false>
__device__ __forceinline__ int lane_sum(float* v) {
    if constexpr (R == 1) {
        return 0;
    } else {
        constexpr int O = STRIDE * R / 2;
        if constexpr (K > 1) {
            const bool up = !SWAPPED && (threadIdx.x & O);
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

// The place that lane_sum returns.
template <int K, int R, int STRIDE, bool SWAPPED = false>
__device__ __forceinline__ int lane_place() {
    if constexpr (R == 1 || K == 1) return 0;
    else return (!SWAPPED && (threadIdx.x & (STRIDE * R / 2)) ? K / 2 : 0) + lane_place<K / 2, R / 2, STRIDE>();
}

template <int LN>
struct BwdShape {
    static constexpr int CPW = 32 / LN * 4;       // channels per warp
    static constexpr int CB = CPW * WARPS;        // channels per block
    static constexpr int NP = LN * 4;             // states, padded
    // Outside the recurrence a thread has the items (token, pair of channels) with its pair p = tid % PAIRS
    // and the tokens tid / PAIRS + j STEP.
    static constexpr int PAIRS = CB / 2, STEP = THREADS / PAIRS, J = SCAN_TILE > STEP ? SCAN_TILE / STEP : 1;
};
// What a token has in shared memory: one record a token, so that a thread's places in all of them are at
// constant distances from one address a token.
template <int LN>
struct BwdToken {
    using S = BwdShape<LN>;
    float delta[S::CB], dyc[S::CB];
    float u[S::CB];                               // delta x; then the sum over the states of C h
    float gB[S::CB], qA[S::CB];                   // sums over the states: g B, q A
    float2 B[S::NP], C[S::NP];                    // both lanes of a packed operand
    float bc[WARPS][2][S::NP];                    // dB, dC over a warp's channels
};
template <typename T, int LN>
struct BwdSmem {
    using S = BwdShape<LN>;
    float4 h[SCAN_TILE / 2][4][THREADS];          // the states before every other token
    BwdToken<LN> tok[SCAN_TILE];
    // the next tile's inputs, on their way while this one is computed
    float saved[LN][S::CB][4];
    T x[SCAN_TILE][S::CB], dt[SCAN_TILE][S::CB], dy[SCAN_TILE][S::CB], z[SCAN_TILE][S::CB];
};

template <typename T, int LN, bool GATED, bool WIDE>
__global__ void __launch_bounds__(THREADS, 3) seq_scan_bwd_kernel(const __grid_constant__ SeqScanParams p) {
    using S = BwdShape<LN>;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    BwdSmem<T, LN>& sm = *reinterpret_cast<BwdSmem<T, LN>*>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int piece = blockIdx.x;
    int t0, t1;
    scan_piece_range(p.ax, p.pc, piece, t0, t1);
    const int per = p.D / p.G, bpg = (per + S::CB - 1) / S::CB;
    const int g = blockIdx.y / bpg;
    const int cb0 = (blockIdx.y - g * bpg) * S::CB;              // the block's first channel in its group
    const int width = min(S::CB, per - cb0);                     // its channels
    const int d0 = g * per + cb0;                                // the first one in the tensors
    const int quads = (p.N + 3) >> 2;
    // The thread's channels: pair i is cw[i], cw[i] + 1; its states: n0[0], n0[0] + 1, n0[1], n0[1] + 1.  Lanes
    // that differ in the bit a sum over lanes starts with hold their pairs in opposite order, so that at
    // that step every lane keeps its first pairs and gives away its second ones: nothing to select.
    constexpr bool SWAP_C = LN >= 2, SWAP_N = LN <= 16;
    int place_c[2], place_n[2], place_h, place_bc, place_s;      // in shared memory, see `own`
    const int ch = SWAP_C ? lane % LN / (LN / 2 > 0 ? LN / 2 : 1) : 0, nh = SWAP_N ? lane >> 4 : 0;
    const int cw[2] = {warp * S::CPW + lane / LN * 4 + 2 * ch, warp * S::CPW + lane / LN * 4 + 2 - 2 * ch};
    const int nq = lane % LN * 4;
    const int n0[2] = {nq + 2 * nh, nq + 2 - 2 * nh};
    const int tiles = (t1 - t0 + SCAN_TILE - 1) / SCAN_TILE;
    // The compiler would otherwise work these out again from the thread's number at every use.
    auto own = [](int v) { asm volatile("" : "+r"(v)); return v; };
    place_c[0] = own(cw[0]);
    place_c[1] = own(cw[1]);
    place_n[0] = own(n0[0]);
    place_n[1] = own(n0[1]);
    place_h = own(tid);
    {
        // where lane_sum leaves the lane's sums; -1 for lanes that hold another lane's
        constexpr int BD = LN < 4 ? 4 / LN : 1, CD = LN > 4 ? LN / 4 : 1;
        const int bi = lane_place<8, 32 / LN, LN, SWAP_N>(), ci = lane_place<4, LN, 1, SWAP_C>();
        place_bc = own(lane / LN % BD == 0 ? (warp * 2 + (bi >> 1 & 1)) * S::NP + n0[bi >> 2] + (bi & 1) : -1);
        place_s = own(lane % CD == 0 ? cw[0] + ci : -1);
    }

    auto fetch = [&](int tb) {
        const int n = min(SCAN_TILE, t1 - tb);
        auto rows = [&](T (*to)[S::CB], const void* from, long long ld) {
            rows_to_shared<T, SCAN_TILE, S::CB, THREADS, WIDE>(to, static_cast<const T*>(from) + (long long)tb * ld + d0, ld, n, width, p.wide);
        };
        rows(sm.x, p.x, p.x_ld);
        rows(sm.dt, p.dt, p.dt_ld);
        rows(sm.dy, p.dy, p.dy_ld);
        if (GATED) rows(sm.z, p.z, p.z_ld);
        const float* from = p.saved + scan_state_at(p, scan_tile_row(p.ax, tb), 0, d0);
#pragma unroll
        for (int j = 0; j < LN * S::CB / THREADS; ++j) {
            const int i = tid + j * THREADS, q = i / S::CB, c = i % S::CB;
            const bool on = q < quads && c < width;
            copy16_async(&sm.saved[q][c][0], on ? from + ((long long)q * p.D + c) * 4 : from, on);
        }
        copies_commit();
    };
    // rows of B and C: few values, through registers
    constexpr int JR = (SCAN_TILE * S::NP + THREADS - 1) / THREADS;
    T Br[JR], Cr[JR];
    auto fetch_bc = [&](int tb) {
        const int n = min(SCAN_TILE, t1 - tb);
#pragma unroll
        for (int j = 0; j < JR; ++j) {
            const int i = tid + j * THREADS, k = g * p.N + min(i % S::NP, p.N - 1);
            const long long t = tb + min(i / S::NP, n - 1);
            Br[j] = static_cast<const T*>(p.B)[t * p.B_ld + k];
            Cr[j] = static_cast<const T*>(p.C)[t * p.C_ld + k];
        }
    };
    if (tiles > 0) {
        fetch(t0 + (tiles - 1) * SCAN_TILE);
        fetch_bc(t0 + (tiles - 1) * SCAN_TILE);
    }

    // Every packed value holds channels cw[i] and cw[i] + 1.
    float2 A2[2][4], gam[2][4], dA[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float2 v[2][2];                           // channel, pair of states in the lane's own order
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            scan_decays<4>(p, d0 + min(cw[i] + e, width - 1), nq, v[e]);
            if (cw[i] + e >= width) v[e][0] = v[e][1] = make_float2(0.f, 0.f);
            if (nh) {
                const float2 t = v[e][0];
                v[e][0] = v[e][1];
                v[e][1] = t;
            }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            A2[i][2 * k] = make_float2(v[0][k].x, v[1][k].x);
            A2[i][2 * k + 1] = make_float2(v[0][k].y, v[1][k].y);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) gam[i][k] = dA[i][k] = make_float2(0.f, 0.f);
    }
    griddep_wait();          // (as the forward kernel: above here, the call's inputs only)
    // the gradient that the sequence's later pieces send back to the state behind this piece
    if (t0 < t1 && p.pc.pps != 1 && p.pc.count > 1) {
        const int s = seq_first_at(p.ax, t1) - 1;                // the sequence of the piece's last token
        if (s >= 0 && seq_start(p.ax, s + 1, t1) > t1 && nq < quads * 4) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float2 v[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        v[e] = cw[i] + e < width ? *reinterpret_cast<const float2*>(p.piece_state + scan_state_at(p, piece, nq >> 2, d0 + cw[i] + e) + (n0[k] & 3))
                                                 : make_float2(0.f, 0.f);
                    gam[i][2 * k] = make_float2(v[0].x, v[1].x);
                    gam[i][2 * k + 1] = make_float2(v[0].y, v[1].y);
                }
        }
    }
    // the thread's pair of channels outside the recurrence
    const int pc = tid % S::PAIRS * 2, tok0 = tid / S::PAIRS;
    const bool on0 = pc < width, on1 = pc + 1 < width;
    const float2 Dd = make_float2(on0 && p.Dskip ? p.Dskip[d0 + pc] : 0.f, on1 && p.Dskip ? p.Dskip[d0 + pc + 1] : 0.f);
    const float2 bias = make_float2(on0 && p.dt_bias ? p.dt_bias[d0 + pc] : 0.f, on1 && p.dt_bias ? p.dt_bias[d0 + pc + 1] : 0.f);
    float2 sumD = make_float2(0.f, 0.f), sumdt = sumD;
    const long long top = t0 + (tiles - 1) * SCAN_TILE + tok0;
    T* dxp = static_cast<T*>(p.dx) + top * p.dx_ld + d0 + pc;
    T* ddtp = static_cast<T*>(p.ddt) + top * p.ddt_ld + d0 + pc;
    T* dzp = GATED ? static_cast<T*>(p.dz) + top * p.dz_ld + d0 + pc : nullptr;

    ScanPlace place = {-1, 0, 0};
    for (int tile = tiles - 1; tile >= 0; --tile) {
        const int tb = t0 + tile * SCAN_TILE, n = min(SCAN_TILE, t1 - tb);
        copies_wait<0>();
        __syncthreads();
        // what the items of this tile need behind the recurrence: x, the slope of softplus, dy silu'(z)
        float2 xv[S::J], slope[S::J], wz[S::J];
#pragma unroll
        for (int j = 0; j < S::J; ++j) {
            const int t = tok0 + j * S::STEP;
            if (S::STEP > SCAN_TILE && t >= SCAN_TILE) break;
            const float2 raw = sum2(seq_ld2(&sm.dt[t][pc]), bias);
            float2 dy = seq_ld2(&sm.dy[t][pc]);
            xv[j] = seq_ld2(&sm.x[t][pc]);
            float2 delta = softplus2(raw, &slope[j]);
            if (!p.softplus) {
                delta = raw;
                slope[j] = make_float2(1.f, 1.f);
            }
            if (!(t < n && on0)) delta.x = dy.x = 0.f;
            if (!(t < n && on1)) delta.y = dy.y = 0.f;
            if (GATED) {
                const float2 z = seq_ld2(&sm.z[t][pc]);
                const float sx = sigmoid(z.x), sy = sigmoid(z.y);
                wz[j] = make_float2(dy.x * silu_grad(z.x, sx), dy.y * silu_grad(z.y, sy));
                dy = mul2(dy, make_float2(z.x * sx, z.y * sy));
            }
            *reinterpret_cast<float2*>(&sm.tok[t].delta[pc]) = delta;
            *reinterpret_cast<float2*>(&sm.tok[t].u[pc]) = mul2(delta, xv[j]);
            *reinterpret_cast<float2*>(&sm.tok[t].dyc[pc]) = dy;
        }
#pragma unroll
        for (int j = 0; j < JR; ++j) {
            const int i = tid + j * THREADS, t = i / S::NP, k = i % S::NP;
            if (JR * THREADS == SCAN_TILE * S::NP || i < SCAN_TILE * S::NP) {
                const bool valid = k < p.N && t < n;
                sm.tok[t].B[k] = dup2(valid ? seq_ld(&Br[j]) : 0.f);
                sm.tok[t].C[k] = dup2(valid ? seq_ld(&Cr[j]) : 0.f);
            }
        }
        float2 h[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float2 v0 = *reinterpret_cast<const float2*>(&sm.saved[nq >> 2][cw[i]][n0[k] & 3]);
                const float2 v1 = *reinterpret_cast<const float2*>(&sm.saved[nq >> 2][cw[i] + 1][n0[k] & 3]);
                h[i][2 * k] = make_float2(v0.x, v1.x);
                h[i][2 * k + 1] = make_float2(v0.y, v1.y);
            }
        __syncthreads();
        if (tile > 0) {
            fetch(tb - SCAN_TILE);
            fetch_bc(tb - SCAN_TILE);
        }
        const ScanMarks marks = scan_marks(p.ax, tb, n, place);
        const unsigned first = marks.first, last = marks.last;
        auto load_states = [&](const float* from, int t, float2 (&v)[2][4]) {
            const long long slot = scan_slot(p.ax, p.sl, tb + t, place);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float v2[2][2][2];
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        scan_h_load<2>(p, cw[i] + e < width ? from : nullptr, slot, d0 + cw[i] + e, n0[k], v2[e][k]);
#pragma unroll
                for (int k = 0; k < 4; ++k) v[i][k] = make_float2(v2[0][k >> 1][k & 1], v2[1][k >> 1][k & 1]);
            }
        };
        // forward again (tokens behind the piece have delta = u = dyc = 0 and B = C = 0: nothing changes there)
#pragma unroll 2
        for (int t = 0; t < SCAN_TILE; ++t) {
            if (t > 0 && (first >> t & 1)) load_states(p.h_in, t, h);
            if (t % 2 == 0) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    st2(&sm.h[t / 2][2 * i][place_h].x, h[i][0], h[i][1]);
                    st2(&sm.h[t / 2][2 * i + 1][place_h].x, h[i][2], h[i][3]);
                }
                if (t == SCAN_TILE - 2) break;      // the last pair's second state is not needed
            }
            float2 b[4];
            ld2(&sm.tok[t].B[place_n[0]].x, b[0], b[1]);
            ld2(&sm.tok[t].B[place_n[1]].x, b[2], b[3]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float2 delta = *reinterpret_cast<const float2*>(&sm.tok[t].delta[place_c[i]]);
                const float2 u = *reinterpret_cast<const float2*>(&sm.tok[t].u[place_c[i]]);
#pragma unroll
                for (int k = 0; k < 4; ++k) h[i][k] = fma2(decay2(delta, A2[i][k]), h[i][k], mul2(u, b[k]));
            }
        }
        // Backward.  Shared memory holds the state before every other token; the one before an odd token is
        // one step from there (or a sequence's starting state).
#pragma unroll 1
        for (int t = SCAN_TILE - 1; t >= 0; --t) {
            if (last >> t & 1) load_states(p.dh_out, t, gam);
            float2 hp[2][4];
            if ((t & 1) && (first >> t & 1)) {
                load_states(p.h_in, t, hp);
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    ld2(&sm.h[t / 2][2 * i][place_h].x, hp[i][0], hp[i][1]);
                    ld2(&sm.h[t / 2][2 * i + 1][place_h].x, hp[i][2], hp[i][3]);
                }
                if (t & 1) {
                    float2 b[4];
                    ld2(&sm.tok[t - 1].B[place_n[0]].x, b[0], b[1]);
                    ld2(&sm.tok[t - 1].B[place_n[1]].x, b[2], b[3]);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 delta = *reinterpret_cast<const float2*>(&sm.tok[t - 1].delta[place_c[i]]);
                        const float2 u = *reinterpret_cast<const float2*>(&sm.tok[t - 1].u[place_c[i]]);
#pragma unroll
                        for (int k = 0; k < 4; ++k) hp[i][k] = fma2(decay2(delta, A2[i][k]), hp[i][k], mul2(u, b[k]));
                    }
                }
            }
            float2 sB[4], sC[4], gB[2], qA[2], Ch[2];
            float2 b[4], c[4];
            ld2(&sm.tok[t].B[place_n[0]].x, b[0], b[1]);
            ld2(&sm.tok[t].B[place_n[1]].x, b[2], b[3]);
            ld2(&sm.tok[t].C[place_n[0]].x, c[0], c[1]);
            ld2(&sm.tok[t].C[place_n[1]].x, c[2], c[3]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float2 delta = *reinterpret_cast<const float2*>(&sm.tok[t].delta[place_c[i]]);
                const float2 u = *reinterpret_cast<const float2*>(&sm.tok[t].u[place_c[i]]);
                const float2 dyc = *reinterpret_cast<const float2*>(&sm.tok[t].dyc[place_c[i]]);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 a = decay2(delta, A2[i][k]);
                    const float2 ah = mul2(a, hp[i][k]);
                    const float2 h = fma2(u, b[k], ah);
                    const float2 gr = fma2(c[k], dyc, gam[i][k]);
                    const float2 q = mul2(gr, ah);
                    if (GATED) Ch[i] = k ? fma2(c[k], h, Ch[i]) : mul2(c[k], h);
                    sC[k] = i ? fma2(dyc, h, sC[k]) : mul2(dyc, h);
                    sB[k] = i ? fma2(gr, u, sB[k]) : mul2(gr, u);
                    gB[i] = k ? fma2(gr, b[k], gB[i]) : mul2(gr, b[k]);
                    qA[i] = k ? fma2(q, A2[i][k], qA[i]) : mul2(q, A2[i][k]);
                    dA[i][k] = fma2(q, delta, dA[i][k]);
                    gam[i][k] = mul2(gr, a);
                }
            }
            if ((first >> t & 1) && p.dh_in) {
                const long long slot = scan_slot(p.ax, p.sl, tb + t, place);
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const float v[2] = {e ? gam[i][2 * k].y : gam[i][2 * k].x, e ? gam[i][2 * k + 1].y : gam[i][2 * k + 1].x};
                            if (cw[i] + e < width) scan_h_store<2>(p, p.dh_in, slot, d0 + cw[i] + e, n0[k], v);
                        }
            }
            // dB and dC: over the channels.  bc: slots 0, 1 of dB and dC, then slots 2, 3.
            float bc[8], s3[3][4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                bc[(k & 1) + (k >> 1) * 4] = sB[k].x + sB[k].y;
                bc[(k & 1) + (k >> 1) * 4 + 2] = sC[k].x + sC[k].y;
            }
            // what dx, ddelta and dz need: over the states
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                unpack(gB[i], s3[0][2 * i], s3[0][2 * i + 1]);
                unpack(qA[i], s3[1][2 * i], s3[1][2 * i + 1]);
                if (GATED) unpack(Ch[i], s3[2][2 * i], s3[2][2 * i + 1]);
            }
            const int bi = lane_sum<8, 32 / LN, LN, SWAP_N>(bc);
            const int ci = lane_sum<4, LN, 1, SWAP_C>(s3[0]);
            lane_sum<4, LN, 1, SWAP_C>(s3[1]);
            if (GATED) lane_sum<4, LN, 1, SWAP_C>(s3[2]);
            __syncwarp();                      // the sums over C h take the place of u, which every lane has read
            constexpr int BK = 8 * LN / 32 > 1 ? 8 * LN / 32 : 1, CK = LN < 4 ? 4 / LN : 1;
            constexpr int BD = LN < 4 ? 4 / LN : 1, CD = LN > 4 ? LN / 4 : 1;     // lanes that hold the same sums
            if (BD == 1 || place_bc >= 0) {
                (void)bi;
                float* to = &sm.tok[t].bc[0][0][0] + place_bc;
#pragma unroll
                for (int j = 0; j < BK; ++j) to[(j >> 1 & 1) * S::NP + (LN == 32 ? 2 * (j >> 2) : 0) + (j & 1)] = bc[j];
            }
            if (CD == 1 || place_s >= 0) {
                (void)ci;
#pragma unroll
                for (int j = 0; j < CK; ++j) {
                    sm.tok[t].gB[place_s + j] = s3[0][j];
                    sm.tok[t].qA[place_s + j] = s3[1][j];
                    if (GATED) sm.tok[t].u[place_s + j] = s3[2][j];
                }
            }
        }
        __syncthreads();
        // per token and pair of channels: dx, ddt, dz
        {
            float2 tD = make_float2(0.f, 0.f), tdt = tD;
            T *qx = dxp, *qt = ddtp, *qz = dzp;
#pragma unroll
            for (int j = 0; j < S::J; ++j) {
                const int t = tok0 + j * S::STEP;
                if (t < n) {
                    const bool both = on1 && WIDE, one = on0;
                    const float2 gB = *reinterpret_cast<const float2*>(&sm.tok[t].gB[pc]);
                    const float2 dyc = *reinterpret_cast<const float2*>(&sm.tok[t].dyc[pc]);
                    const float2 delta = *reinterpret_cast<const float2*>(&sm.tok[t].delta[pc]);
                    const float2 qA = *reinterpret_cast<const float2*>(&sm.tok[t].qA[pc]);
                    const float2 dx = fma2(delta, gB, mul2(Dd, dyc));
                    const float2 dd = mul2(fma2(xv[j], gB, mul2(qA, dup2(0.6931471805599453f))), slope[j]);   // A2 = A / ln 2
                    seq_st2(qx, dx, both, one);
                    seq_st2(qt, dd, both, one);
                    float2 dz = make_float2(0.f, 0.f);
                    if (GATED) {
                        dz = mul2(wz[j], fma2(Dd, xv[j], *reinterpret_cast<const float2*>(&sm.tok[t].u[pc])));
                        seq_st2(qz, dz, both, one);
                    }
                    if (on1 && !WIDE) {
                        seq_st(qx + 1, dx.y);
                        seq_st(qt + 1, dd.y);
                        if (GATED) seq_st(qz + 1, dz.y);
                    }
                    tD = fma2(dyc, xv[j], tD);
                    tdt = sum2(tdt, dd);
                }
                qx += p.dx_ld * S::STEP;
                qt += p.ddt_ld * S::STEP;
                if (GATED) qz += p.dz_ld * S::STEP;
            }
            dxp -= p.dx_ld * SCAN_TILE;
            ddtp -= p.ddt_ld * SCAN_TILE;
            if (GATED) dzp -= p.dz_ld * SCAN_TILE;
            sumD = sum2(sumD, tD);
            sumdt = sum2(sumdt, tdt);
        }
        float* bc = p.part_bc + ((long long)blockIdx.y * p.ax.T + tb) * 2 * S::NP;
#pragma unroll
        for (int j = 0; j < (SCAN_TILE * 2 * S::NP + THREADS - 1) / THREADS; ++j) {
            const int i = tid + j * THREADS, t = i / (2 * S::NP), r = i % (2 * S::NP);
            if (t >= n) break;
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) s += (&sm.tok[t].bc[w][0][0])[r];
            bc[i] = s;
        }
    }
    float* par = p.part_par + (long long)piece * (p.N + 2) * p.D;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int nk = n0[k >> 1] + (k & 1);
            if (nk < p.N && cw[i] < width) par[(long long)nk * p.D + d0 + cw[i]] = dA[i][k].x;
            if (nk < p.N && cw[i] + 1 < width) par[(long long)nk * p.D + d0 + cw[i] + 1] = dA[i][k].y;
        }
    // dD and ddt_bias: a pair's threads in the order of their tokens
    __syncthreads();
    float4* red = &sm.h[0][0][0];
    red[tid] = make_float4(sumD.x, sumD.y, sumdt.x, sumdt.y);
    __syncthreads();
    if (tid < S::PAIRS) {
        float4 s = red[tid];
#pragma unroll
        for (int j = 1; j < S::STEP; ++j) {
            const float4 v = red[tid + j * S::PAIRS];
            s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w);
        }
        float* to = par + (long long)p.N * p.D + d0 + pc;
        if (on0) to[0] = s.x, to[p.D] = s.z;
        if (on1) to[1] = s.y, to[p.D + 1] = s.w;
    }
}

// What a piece sends back to the state before it: its share of a_t g_t at its first token (from its
// first sequence alone, if another begins in it), and the sum of delta over it.  Threads hold channels and
// states as in the forward kernel: two channels, NPT states of each, LN lanes to a channel.
constexpr int BACK_THREADS = 64;
template <typename T, int NPT, int LN, bool GATED, bool WIDE>
__global__ void __launch_bounds__(BACK_THREADS) seq_scan_back_kernel(const __grid_constant__ SeqScanParams p) {
    constexpr int CB = 2 * BACK_THREADS / LN, NP = NPT * LN, STAGES = sizeof(T) == 2 ? 4 : 3;
    constexpr int JR = (SCAN_TILE * NP + BACK_THREADS - 1) / BACK_THREADS;
    __shared__ __align__(16) float sC[2][SCAN_TILE][NP];
    __shared__ __align__(16) T sdt[STAGES][SCAN_TILE][CB], sdy[STAGES][SCAN_TILE][CB], sz[GATED ? STAGES : 1][GATED ? SCAN_TILE : 1][CB];
    const int piece = blockIdx.x;
    if (p.pc.pps > 0 ? piece % p.pc.pps == 0 : piece == 0) return;      // nothing comes before it
    int t0, t1;
    scan_piece_range(p.ax, p.pc, piece, t0, t1);
    const int per = p.D / p.G, bpg = (per + CB - 1) / CB;
    const int g = blockIdx.y / bpg;
    const int cb0 = (blockIdx.y - g * bpg) * CB;
    const int width = min(CB, per - cb0), d0 = g * per + cb0;
    const int c = threadIdx.x / LN * 2;
    const bool on[2] = {c < width, c + 1 < width};
    const int d[2] = {d0 + min(c, width - 1), d0 + min(c + 1, width - 1)};
    const int ln = threadIdx.x % LN, n0 = ln * NPT;
    // a sequence that begins in the piece sends nothing behind its first token: only the tokens
    // before it count
    const int s1 = seq_first_at(p.ax, t0 + 1);
    t1 = min(t1, seq_start(p.ax, s1, t0 + 1));
    const int tiles = (t1 - t0 + SCAN_TILE - 1) / SCAN_TILE;
    auto fetch = [&](int tile) {
        if (tile >= 0) {
            const int tb = t0 + tile * SCAN_TILE, n = min(SCAN_TILE, t1 - tb), stage = tile % STAGES;
            auto rows = [&](T (*to)[CB], const void* from, long long ld) {
                rows_to_shared<T, SCAN_TILE, CB, BACK_THREADS, WIDE>(to, static_cast<const T*>(from) + (long long)tb * ld + d0, ld, n, width, p.wide);
            };
            rows(sdt[stage], p.dt, p.dt_ld);
            rows(sdy[stage], p.dy, p.dy_ld);
            if (GATED) rows(sz[stage], p.z, p.z_ld);
        }
        copies_commit();
    };
    T Cr[JR];
    auto fetch_c = [&](int tb) {
        const int n = min(SCAN_TILE, t1 - tb);
#pragma unroll
        for (int j = 0; j < JR; ++j) {
            const int i = threadIdx.x + j * BACK_THREADS;
            Cr[j] = static_cast<const T*>(p.C)[(long long)(tb + min(i / NP, n - 1)) * p.C_ld + g * p.N + min(i % NP, p.N - 1)];
        }
    };
#pragma unroll
    for (int i = 1; i < STAGES; ++i) fetch(tiles - i);
    if (tiles > 0) fetch_c(t0 + (tiles - 1) * SCAN_TILE);

    float2 A2[2][NPT / 2], gam[2][NPT / 2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        scan_decays<NPT>(p, d[e], n0, A2[e]);
#pragma unroll
        for (int k = 0; k < NPT / 2; ++k) gam[e][k] = make_float2(0.f, 0.f);
    }
    const float2 bias = p.dt_bias ? make_float2(p.dt_bias[d[0]], p.dt_bias[d[1]]) : make_float2(0.f, 0.f);
    float2 total = make_float2(0.f, 0.f);
    // the only end of a sequence here is at t1, and the only beginning at t0
    if (tiles > 0 && p.dh_out) {
        const ScanPlace q = scan_place(p.ax, t1 - 1);
        if (q.end == t1) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float v[NPT];
                scan_h_load<NPT>(p, p.dh_out, seq_slot(p.sl, q.s), d[e], n0, v);
#pragma unroll
                for (int k = 0; k < NPT / 2; ++k) gam[e][k] = make_float2(v[2 * k], v[2 * k + 1]);
            }
        }
    }
    griddep_launch();
    for (int tile = tiles - 1; tile >= 0; --tile) {
        const int tb = t0 + tile * SCAN_TILE, n = min(SCAN_TILE, t1 - tb), buf = tile & 1, stage = tile % STAGES;
#pragma unroll
        for (int j = 0; j < JR; ++j) {
            const int i = threadIdx.x + j * BACK_THREADS;
            if (JR * BACK_THREADS == SCAN_TILE * NP || i < SCAN_TILE * NP) sC[buf][i / NP][i % NP] = i % NP < p.N ? seq_ld(&Cr[j]) : 0.f;
        }
        copies_wait<STAGES - 2>();
        __syncthreads();
        fetch(tile - (STAGES - 1));          // into the stage of the tile before this one (tile + 1)
        if (tile > 0) fetch_c(tb - SCAN_TILE);
#pragma unroll
        for (int i = SCAN_TILE - 1; i >= 0; --i) {
            if (i >= n) continue;
            const float2 raw = sum2(seq_ld2(&sdt[stage][i][c]), bias);
            float2 delta = softplus2(raw, nullptr), dyc = seq_ld2(&sdy[stage][i][c]);
            if (!p.softplus) delta = raw;
            if (GATED) {
                const float2 z = seq_ld2(&sz[GATED ? stage : 0][GATED ? i : 0][c]);
                dyc = mul2(dyc, make_float2(silu(z.x), silu(z.y)));
            }
            const float2 dl[2] = {dup2(delta.x), dup2(delta.y)}, dc[2] = {dup2(dyc.x), dup2(dyc.y)};
#pragma unroll
            for (int k = 0; k < NPT / 2; k += 2) {
                float2 ck[2];
                ld2(&sC[buf][i][n0 + 2 * k], ck[0], ck[1]);
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        gam[e][k + j] = mul2(decay2(dl[e], A2[e][k + j]), fma2(ck[j], dc[e], gam[e][k + j]));
            }
            total = sum2(total, delta);
        }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        if (!on[e]) continue;
#pragma unroll
        for (int k = 0; k < NPT / 2; k += 2)
            if (n0 + 2 * k < ((p.N + 3) & ~3)) st2(p.piece_state + scan_state_at(p, piece, (n0 + 2 * k) >> 2, d[e]), gam[e][k], gam[e][k + 1]);
        if (ln == 0) p.piece_delta[(long long)piece * p.D + d[e]] = e ? total.y : total.x;
    }
}

// dB and dC: the partial rows of a group's channel blocks, added in block order.
template <typename T, int NP>
__global__ void __launch_bounds__(128) seq_scan_bc_kernel(const __grid_constant__ SeqScanParams p) {
    griddep_wait();
    const int bpg = p.cblocks / p.G;
    const long long all = (long long)p.ax.T * p.G * 2 * NP;
    for (long long i = blockIdx.x * 128ll + threadIdx.x; i < all; i += gridDim.x * 128ll) {
        const int r = (int)(i % (2 * NP)), k = r % NP;
        const long long tg = i / (2 * NP);
        const int g = p.G == 1 ? 0 : (int)(tg % p.G);
        const long long t = p.G == 1 ? tg : tg / p.G;
        if (k >= p.N) continue;
        const float* src = p.part_bc + ((long long)g * bpg * p.ax.T + t) * 2 * NP + r;
        const long long step = (long long)p.ax.T * 2 * NP;
        float s[4] = {};
        int b = 0;
        for (; b + 4 <= bpg; b += 4)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[j] += src[(b + j) * step];
        for (; b < bpg; ++b) s[0] += src[b * step];
        const float v = (s[0] + s[1]) + (s[2] + s[3]);
        if (r < NP) seq_st(static_cast<T*>(p.dB) + t * p.dB_ld + g * p.N + k, v);
        else seq_st(static_cast<T*>(p.dC) + t * p.dC_ld + g * p.N + k, v);
    }
}

// dA, dD, ddt_bias: the pieces' partial sums, added in piece order.
__global__ void __launch_bounds__(128) seq_scan_par_kernel(const __grid_constant__ SeqScanParams p) {
    griddep_wait();
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

// The kernel for the call's rows: gated or not, in whole 16-byte groups or not.
inline auto of_rows(const SeqScanParams& p, void (*gated_wide)(const SeqScanParams), void (*wide)(const SeqScanParams),
             void (*gated)(const SeqScanParams), void (*other)(const SeqScanParams)) {
    return p.wide == 16 ? (p.z ? gated_wide : wide) : (p.z ? gated : other);
}

// LN: lanes of the main kernel; NPT, LB: states and lanes of the pieces' kernel
template <typename T, int LN, int NPT, int LB>
cudaError_t launch_ln(const SeqScanParams& p, cudaStream_t stream) {
    cudaError_t e = cudaSuccess;
    if (p.ax.T > 0) {
        if (p.pc.pps != 1 && p.pc.count > 1) {
            constexpr int CB = 2 * BACK_THREADS / LB;
            const int per = p.D / p.G;
            const dim3 grid((unsigned)p.pc.count, (unsigned)(p.G * ((per + CB - 1) / CB)));
            e = launch_kernel(of_rows(p, seq_scan_back_kernel<T, NPT, LB, true, true>, seq_scan_back_kernel<T, NPT, LB, false, true>,
                                         seq_scan_back_kernel<T, NPT, LB, true, false>, seq_scan_back_kernel<T, NPT, LB, false, false>),
                              grid, dim3(BACK_THREADS), 0, stream, false, 1, p);
        }
        if (e == cudaSuccess && p.pc.pps != 1 && p.pc.count > 1) e = launch_seq_scan_join(p, true, stream);
        const auto main = of_rows(p, seq_scan_bwd_kernel<T, LN, true, true>, seq_scan_bwd_kernel<T, LN, false, true>,
                                     seq_scan_bwd_kernel<T, LN, true, false>, seq_scan_bwd_kernel<T, LN, false, false>);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(main, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(BwdSmem<T, LN>));
        if (e == cudaSuccess)
            e = launch_kernel(main, dim3((unsigned)p.pc.count, (unsigned)p.cblocks), dim3(THREADS), sizeof(BwdSmem<T, LN>), stream,
                              p.pc.pps != 1 && p.pc.count > 1, 1, p);
        const long long all = ((long long)p.ax.T * p.G * 8 * LN + 127) / 128;
        if (e == cudaSuccess)
            e = launch_kernel(seq_scan_bc_kernel<T, 4 * LN>, dim3((unsigned)(all < 65536 ? all : 65536)), dim3(128), 0, stream, true, 1, p);
    }
    if (e == cudaSuccess && p.dh_in && p.ax.L == 0) e = launch_seq_scan_empty(p, p.dh_out, p.dh_in, stream);
    if (e == cudaSuccess)
        e = launch_kernel(seq_scan_par_kernel, dim3((unsigned)((p.D + 127) / 128), (unsigned)(p.N + 2)), dim3(128), 0, stream,
                          p.ax.T > 0 && !p.dh_in, 1, p);
    return e;
}

template <typename T>
cudaError_t launch_t(const SeqScanParams& p, cudaStream_t stream) {
    if (p.N <= 8) return launch_ln<T, 2, 8, 1>(p, stream);
    if (p.N <= 16) return launch_ln<T, 4, 16, 1>(p, stream);
    if (p.N <= 32) return launch_ln<T, 8, 16, 2>(p, stream);
    if (p.N <= 64) return launch_ln<T, 16, 16, 4>(p, stream);
    return launch_ln<T, 32, 16, 8>(p, stream);
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

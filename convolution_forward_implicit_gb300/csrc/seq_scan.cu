// Selective state space scan, forward: see seq.h for the formulas.
//
// Per token, channel and state: one exponential (exp(delta A) as 2^(delta A log2 e)) and four
// multiply-adds, so the pass is bound by the special-function and FMA pipes.  A thread holds NPT states of one channel in registers and walks the
// tokens of a piece; LN neighbouring lanes share a channel when it has more states.
//
// 4 x 2048 x 4096 x 16 bf16 in 7 pieces a sequence: 157 us, and 106 for the pieces' contributions before it (the
// exponentials alone are 58 us of each; uncut, the 4 x 4096 channels fill a third of the GPU's warps: 710 us at an
// earlier state, cut 410).  0.58 instructions a clock and scheduler: what is left is dependent latency.
#include "seq_scan.cuh"

namespace convfwd {
namespace {

constexpr int THREADS = 64;         // of the scan; a thread has two channels

// Rows of B or C of a tile, on their way through registers to shared memory as fp32.
template <typename T, int NP>
struct TileRows {
    static constexpr int J = (SCAN_TILE * NP + THREADS - 1) / THREADS;
    T v[J];
    __device__ __forceinline__ void load(const void* base, long long ld, int col, int N, int tb, int n) {
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int i = threadIdx.x + j * THREADS, t = min(i / NP, n - 1), k = min(i % NP, N - 1);
            v[j] = static_cast<const T*>(base)[(long long)(tb + t) * ld + col + k];
        }
    }
    __device__ __forceinline__ void store(float (*to)[NP], int N) const {
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int i = threadIdx.x + j * THREADS;
            if (J * THREADS == SCAN_TILE * NP || i < SCAN_TILE * NP) to[i / NP][i % NP] = i % NP < N ? seq_ld(&v[j]) : 0.f;
        }
    }
};

// A block walks a piece, a tile of SCAN_TILE tokens at a time.  x, dt and z of the next tiles are copied
// to shared memory while this one is computed (STAGES tiles in flight or in use); B and C pass through
// registers into two buffers of fp32.  One barrier a tile.  A thread has two neighbouring channels: what
// a token costs besides its states (conversions, softplus, silu, addresses, the rows of B and C) is shared
// by the two.  SUMMARY: only the state behind the piece and the sum of delta.
template <typename T, int NPT, int LN, bool SUMMARY, bool GATED, bool WIDE>
__global__ void __launch_bounds__(THREADS, 6) seq_scan_kernel(const __grid_constant__ SeqScanParams p) {
    constexpr int CB = 2 * THREADS / LN, NP = NPT * LN, STAGES = sizeof(T) == 2 ? 4 : 3;
    __shared__ __align__(16) float sB[2][SCAN_TILE][NP], sC[2][SUMMARY ? 1 : SCAN_TILE][NP];
    __shared__ __align__(16) T sx[STAGES][SCAN_TILE][CB], sdt[STAGES][SCAN_TILE][CB], sz[GATED ? STAGES : 1][GATED ? SCAN_TILE : 1][CB];
    const int piece = blockIdx.x;
    int t0, t1;
    scan_piece_range(p.ax, p.pc, piece, t0, t1);
    if (SUMMARY) {                  // the last piece of a sequence (of the axis) hands nothing on
        if (p.pc.pps > 0 ? piece % p.pc.pps == p.pc.pps - 1 : piece == p.pc.count - 1) return;
    }
    if (t0 >= t1) return;
    const int per = p.D / p.G, bpg = (per + CB - 1) / CB;
    const int g = blockIdx.y / bpg;
    const int cb0 = (blockIdx.y - g * bpg) * CB;                        // the block's first channel in its group
    const int width = min(CB, per - cb0), d0 = g * per + cb0;
    const int c = threadIdx.x / LN * 2;                                 // the thread's first channel in the block
    const bool on[2] = {c < width, c + 1 < width};
    const int d[2] = {d0 + min(c, width - 1), d0 + min(c + 1, width - 1)};
    const int ln = threadIdx.x % LN, n0 = ln * NPT;
    const int padded = (p.N + 3) & ~3;
    T* yp = SUMMARY ? nullptr : static_cast<T*>(p.y) + (long long)t0 * p.y_ld + d[0];

    auto fetch = [&](int tb, int stage) {
        if (tb < t1) {
            const int n = min(SCAN_TILE, t1 - tb);
            auto rows = [&](T (*to)[CB], const void* from, long long ld) {
                rows_to_shared<T, SCAN_TILE, CB, THREADS, WIDE>(to, static_cast<const T*>(from) + (long long)tb * ld + d0, ld, n, width, p.wide);
            };
            rows(sx[stage], p.x, p.x_ld);
            rows(sdt[stage], p.dt, p.dt_ld);
            if (GATED) rows(sz[stage], p.z, p.z_ld);
        }
        copies_commit();
    };
    TileRows<T, NP> Br, Cr;
    auto fetch_bc = [&](int tb) {
        const int n = min(SCAN_TILE, t1 - tb);
        Br.load(p.B, p.B_ld, g * p.N, p.N, tb, n);
        if (!SUMMARY) Cr.load(p.C, p.C_ld, g * p.N, p.N, tb, n);
    };
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) fetch(t0 + i * SCAN_TILE, i);
    fetch_bc(t0);

    // packed values hold states 2 k and 2 k + 1 of the thread's, or its two channels
    float2 A2[2][NPT / 2], h[2][NPT / 2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        scan_decays<NPT>(p, d[e], n0, A2[e]);
#pragma unroll
        for (int k = 0; k < NPT / 2; ++k) h[e][k] = make_float2(0.f, 0.f);
    }
    const float2 Dd = p.Dskip ? make_float2(p.Dskip[d[0]], p.Dskip[d[1]]) : make_float2(0.f, 0.f);
    const float2 bias = p.dt_bias ? make_float2(p.dt_bias[d[0]], p.dt_bias[d[1]]) : make_float2(0.f, 0.f);
    float2 total = make_float2(0.f, 0.f);
    ScanPlace q = scan_place(p.ax, t0);
    // states at the workspace's layout and at the caller's
    auto get = [&](const float* from, long long row) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int k = 0; k < NPT / 2; k += 2) {
                h[e][k] = h[e][k + 1] = make_float2(0.f, 0.f);
                if (n0 + 2 * k < padded) ld2(from + scan_state_at(p, row, (n0 + 2 * k) >> 2, d[e]), h[e][k], h[e][k + 1]);
            }
    };
    auto put = [&](float* to, long long row) {
#pragma unroll
        for (int k = 0; k < NPT / 2; k += 2)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (on[e] && n0 + 2 * k < padded) st2(to + scan_state_at(p, row, (n0 + 2 * k) >> 2, d[e]), h[e][k], h[e][k + 1]);
    };
    auto begin_sequence = [&](int t) {
        const ScanPlace r = t >= q.begin && t < q.end ? q : scan_place(p.ax, t);
        // a sequence that runs on behind the piece: its starting state was put aside by the pass
        // before, since the block that ends it may already have written h_out
        if (!SUMMARY && p.h_in && p.pc.pps != 1 && p.pc.count > 1 && r.end > t1) {
            get(p.piece_init, piece);
        } else {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float v[NPT];
                scan_h_load<NPT>(p, p.h_in, seq_slot(p.sl, r.s), d[e], n0, v);
#pragma unroll
                for (int k = 0; k < NPT / 2; ++k) h[e][k] = make_float2(v[2 * k], v[2 * k + 1]);
            }
        }
        if (SUMMARY && p.h_in) put(p.piece_init, piece);
        total = make_float2(0.f, 0.f);
    };
    auto end_sequence = [&](int t) {
        if (SUMMARY || !p.h_out) return;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float v[NPT];
#pragma unroll
            for (int k = 0; k < NPT / 2; ++k) unpack(h[e][k], v[2 * k], v[2 * k + 1]);
            if (on[e]) scan_h_store<NPT>(p, p.h_out, scan_slot(p.ax, p.sl, t, q), d[e], n0, v);
        }
    };
    // one token from its row in the stage and its rows of B and C in shared memory
    auto token = [&](const T* xs, const T* dts, const T* zs, const float* b, const float* cc) {
        const float2 x = seq_ld2(xs + c), raw = sum2(seq_ld2(dts + c), bias);
        float2 delta = softplus2(raw, nullptr);
        if (!p.softplus) delta = raw;
        const float2 u = mul2(delta, x);
        const float2 dl[2] = {dup2(delta.x), dup2(delta.y)}, uu[2] = {dup2(u.x), dup2(u.y)};
        float2 acc[2][2];
#pragma unroll
        for (int k = 0; k < NPT / 2; k += 2) {
            float2 bk[2], ck[2];
            ld2(b + n0 + 2 * k, bk[0], bk[1]);
            if (!SUMMARY) ld2(cc + n0 + 2 * k, ck[0], ck[1]);
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    h[e][k + j] = fma2(decay2(dl[e], A2[e][k + j]), h[e][k + j], mul2(uu[e], bk[j]));
                    if (!SUMMARY) acc[e][j] = k ? fma2(ck[j], h[e][k + j], acc[e][j]) : mul2(ck[j], h[e][k + j]);
                }
        }
        total = sum2(total, delta);
        if (!SUMMARY) {
            const float2 s0 = sum2(acc[0][0], acc[0][1]), s1 = sum2(acc[1][0], acc[1][1]);
            float2 y = make_float2(s0.x + s0.y, s1.x + s1.y);
#pragma unroll
            for (int o = LN / 2; o > 0; o >>= 1)
                y = sum2(y, make_float2(__shfl_xor_sync(~0u, y.x, o), __shfl_xor_sync(~0u, y.y, o)));
            y = fma2(Dd, x, y);
            if (GATED) {
                const float2 z = seq_ld2(zs + c);
                y = mul2(y, make_float2(silu(z.x), silu(z.y)));
            }
            if (ln == 0) {
                seq_st2(yp, y, on[1] && WIDE, on[0]);
                if (on[1] && !WIDE) seq_st(yp + 1, y.y);
            }
            yp += p.y_ld;
        }
    };
    // Launched behind the joining kernel, this one may have started before it ended: what is above here reads the
    // call's inputs only, which were there before its first kernel began.
    if (SUMMARY) griddep_launch();
    else griddep_wait();
    if (!SUMMARY && q.begin < t0) get(p.piece_state, piece);      // the state that the pieces before leave
    int buf = 0, stage = 0;
    for (int tb = t0; tb < t1; tb += SCAN_TILE, buf ^= 1) {
        const int n = min(SCAN_TILE, t1 - tb);
        Br.store(sB[buf], p.N);
        if (!SUMMARY) Cr.store(sC[buf], p.N);
        copies_wait<STAGES - 2>();
        __syncthreads();
        // into the stage that the tile before this one used: every thread is past it
        fetch(tb + (STAGES - 1) * SCAN_TILE, stage == 0 ? STAGES - 1 : stage - 1);
        if (tb + SCAN_TILE < t1) fetch_bc(tb + SCAN_TILE);
        const ScanMarks m = scan_marks(p.ax, tb, n, q);
        if (m.first & 1) begin_sequence(tb);
        if (!SUMMARY && p.saved) put(p.saved, scan_tile_row(p.ax, tb));
        const T(*xs)[CB] = sx[stage], (*dts)[CB] = sdt[stage], (*zs)[CB] = sz[GATED ? stage : 0];
        if (n == SCAN_TILE && !(m.first >> 1)) {
#pragma unroll
            for (int i = 0; i < SCAN_TILE; ++i) token(xs[i], dts[i], zs[GATED ? i : 0], sB[buf][i], sC[buf][SUMMARY ? 0 : i]);
            if (m.last) end_sequence(tb + n - 1);
        } else {                                        // a short tile, or one that sequences begin in
#pragma unroll 1
            for (int i = 0; i < n; ++i) {
                if (i > 0 && (m.first >> i & 1)) begin_sequence(tb + i);
                token(xs[i], dts[i], zs[GATED ? i : 0], sB[buf][i], sC[buf][SUMMARY ? 0 : i]);
                if (m.last >> i & 1) end_sequence(tb + i);
            }
        }
        stage = stage == STAGES - 1 ? 0 : stage + 1;
    }
    if (SUMMARY) {
        put(p.piece_state, piece);
        if (ln == 0) {
            if (on[0]) p.piece_delta[(long long)piece * p.D + d[0]] = total.x;
            if (on[1]) p.piece_delta[(long long)piece * p.D + d[1]] = total.y;
        }
    }
}

// Joins the pieces of a sequence (of a ragged axis): with e_r what piece r adds to the state behind it and
// sum_r its sum of delta, the state before piece r + 1 is c_{r+1} = e_r + exp(sum_r A) c_r, or e_r alone where
// a sequence begins in piece r (backward: the same from the last piece down).  A thread replaces e_r by c_r for
// 4 states of a channel in one part of the pieces, 16 at most, whose loads are all on their way at once.  It first
// joins its own part from a zero state, keeping the sum of delta over it; the parts' results pass through shared
// memory; then it walks its part again from the state before it.  (2048 x 2048 x 16 in 52 pieces: one part, in
// batches of loads, 8.3 us; 4 parts 4.)  Up to 16 pieces one part is enough, and faster: 4 us against 15 with 4 parts
// for 4 x 2048 x 4096 x 16 in 7 pieces a sequence.
constexpr int JOIN_MOST = 16;
__host__ __device__ constexpr int join_threads(int parts) { return parts == 8 ? 256 : 128; }       // several parts: a warp has one of them
template <bool REVERSE, int JOIN_PARTS>
__global__ void __launch_bounds__(join_threads(JOIN_PARTS)) seq_scan_join_kernel(const __grid_constant__ SeqScanParams p) {
    constexpr int JOIN_LANES = join_threads(JOIN_PARTS) / JOIN_PARTS;
    __shared__ float4 sh_e[JOIN_PARTS][JOIN_LANES];
    __shared__ float sh_sum[JOIN_PARTS][JOIN_LANES];
    __shared__ bool sh_cut[JOIN_PARTS];
    const int pieces = p.pc.pps > 0 ? p.pc.pps : p.pc.count, first = blockIdx.y * pieces;
    const int lane = threadIdx.x % JOIN_LANES, part = threadIdx.x / JOIN_LANES;
    const int len = (pieces + JOIN_PARTS - 1) / JOIN_PARTS, r0 = part * len, r1 = min(r0 + len, pieces);
    // which of the part's pieces cut the chain, in the order of the walk: lane l looks at the l-th
    bool stop = false;
    const int look = r0 + (threadIdx.x & 31);
    if (look < r1) {
        int t0, t1;
        scan_piece_range(p.ax, p.pc, first + (REVERSE ? pieces - 1 - look : look), t0, t1);
        const int s = seq_first_at(p.ax, REVERSE ? t0 + 1 : t0);      // the first sequence that begins in the piece (behind its first token)
        const int begin = seq_start(p.ax, s, t0);
        stop = REVERSE ? begin <= t1 : begin < t1;
    }
    const unsigned cut = __ballot_sync(~0u, stop);
    const int quads = (p.N + 3) >> 2;
    const long long i = blockIdx.x * (long long)JOIN_LANES + lane;
    const bool on = i < (long long)quads * p.D;
    const int quad = on ? (int)(i / p.D) : 0, d = on ? (int)(i - (long long)quad * p.D) : 0;
    float A2[4];                     // A log2(e) / 2
#pragma unroll
    for (int k = 0; k < 4; ++k) A2[k] = on && 4 * quad + k < p.N ? p.A[(long long)d * p.N + 4 * quad + k] * (0.5f * LOG2E) : 0.f;
    griddep_wait();                  // from here on: what the pass before wrote
    griddep_launch();
    float4 e[JOIN_MOST];
    float sum[JOIN_MOST];
#pragma unroll
    for (int j = 0; j < JOIN_MOST; ++j) {
        const int r = r0 + j, at = first + (REVERSE ? pieces - 1 - r : r);
        e[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        sum[j] = 0.f;
        if (on && r < r1 && r < pieces - 1) {                        // (the last piece hands nothing on)
            e[j] = *reinterpret_cast<const float4*>(p.piece_state + scan_state_at(p, at, quad, d));
            sum[j] = p.piece_delta[(long long)at * p.D + d];
        }
    }
    float4 c = make_float4(0.f, 0.f, 0.f, 0.f);
    float total = 0.f;
    // exp(sum A) c + e, the factor in two halves: one beyond fp32's range (states that grow: A > 0) is then not infinity
    // where there is nothing to grow, or little.
    auto carry = [](float half_v, float c, float e) {
        const float half = fminf(ex2_approx(half_v), 3.4e38f);
        return fmaf(half * c, half, e);
    };
    auto step = [&](float4 c, float4 e, float sum, bool stop) {
        if (stop) return e;
        return make_float4(carry(sum * A2[0], c.x, e.x), carry(sum * A2[1], c.y, e.y), carry(sum * A2[2], c.z, e.z), carry(sum * A2[3], c.w, e.w));
    };
#pragma unroll
    for (int j = 0; j < JOIN_MOST; ++j)
        if (r0 + j < r1) {
            c = step(c, e[j], sum[j], cut >> j & 1);
            total = cut >> j & 1 ? 0.f : total + sum[j];
        }
    sh_e[part][lane] = c;
    sh_sum[part][lane] = total;
    if (lane == 0) sh_cut[part] = cut != 0;
    __syncthreads();
    c = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int q = 0; q < part; ++q) c = step(c, sh_e[q][lane], sh_sum[q][lane], sh_cut[q]);
    if (!on) return;
#pragma unroll
    for (int j = 0; j < JOIN_MOST; ++j)
        if (r0 + j < r1) {
            const int r = r0 + j, at = first + (REVERSE ? pieces - 1 - r : r);
            *reinterpret_cast<float4*>(p.piece_state + scan_state_at(p, at, quad, d)) = c;
            c = step(c, e[j], sum[j], cut >> j & 1);
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

template <typename T, int NPT, int LN, bool WIDE>
cudaError_t launch_fwd_of(const SeqScanParams& p, cudaStream_t stream) {
    constexpr int CB = 2 * THREADS / LN;
    const int per = p.D / p.G;
    const dim3 grid((unsigned)p.pc.count, (unsigned)(p.G * ((per + CB - 1) / CB)));
    cudaError_t e = cudaSuccess;
    if (p.ax.T > 0) {
        const bool cut = p.pc.pps != 1 && p.pc.count > 1;
        if (cut)
            e = launch_kernel(seq_scan_kernel<T, NPT, LN, true, false, WIDE>, grid, dim3(THREADS), 0, stream, false, 1, p);
        if (e == cudaSuccess && cut) e = launch_seq_scan_join(p, false, stream);
        if (e == cudaSuccess)
            e = p.z ? launch_kernel(seq_scan_kernel<T, NPT, LN, false, true, WIDE>, grid, dim3(THREADS), 0, stream, cut, 1, p)
                    : launch_kernel(seq_scan_kernel<T, NPT, LN, false, false, WIDE>, grid, dim3(THREADS), 0, stream, cut, 1, p);
    }
    if (e == cudaSuccess && p.h_out && p.h_out != p.h_in && p.ax.L == 0) e = launch_seq_scan_empty(p, p.h_in, p.h_out, stream);
    return e;
}

// (Rows that are not whole 16-byte groups have kernels of their own: their copies beside the others in one kernel, even
// out of line, cost the others registers.)
template <typename T, int NPT, int LN>
cudaError_t launch_fwd(const SeqScanParams& p, cudaStream_t stream) {
    return p.wide == 16 ? launch_fwd_of<T, NPT, LN, true>(p, stream) : launch_fwd_of<T, NPT, LN, false>(p, stream);
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

}  // namespace

cudaError_t launch_seq_scan_join(const SeqScanParams& p, bool reverse, cudaStream_t stream) {
    const long long all = (long long)((p.N + 3) / 4) * p.D;
    const int pieces = p.pc.pps > 0 ? p.pc.pps : p.pc.count;
    const int parts = pieces <= JOIN_MOST ? 1 : pieces <= 4 * JOIN_MOST ? 4 : 8, lanes = join_threads(parts) / parts;
    if (pieces > 8 * JOIN_MOST) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)((all + lanes - 1) / lanes), (unsigned)(p.pc.pps > 0 ? p.ax.S : 1));
    auto kernel = parts == 1   ? (reverse ? seq_scan_join_kernel<true, 1> : seq_scan_join_kernel<false, 1>)
                  : parts == 4 ? (reverse ? seq_scan_join_kernel<true, 4> : seq_scan_join_kernel<false, 4>)
                               : (reverse ? seq_scan_join_kernel<true, 8> : seq_scan_join_kernel<false, 8>);
    return launch_kernel(kernel, grid, dim3(join_threads(parts)), 0, stream, true, 1, p);
}
cudaError_t launch_seq_scan_empty(const SeqScanParams& p, const float* from, float* to, cudaStream_t stream) {
    const long long DN = (long long)p.D * p.N, blocks = DN / 1024 + 1;
    return launch_kernel(seq_scan_empty_kernel, dim3((unsigned)(blocks < 64 ? blocks : 64), (unsigned)(p.ax.S < 32768 ? p.ax.S : 32768)),
                         dim3(128), 0, stream, false, 1, p.ax, p.sl, from, to, DN);
}
cudaError_t launch_seq_scan_fwd(const SeqScanParams& p, bool bf16, cudaStream_t stream) {
    return bf16 ? launch_t<__nv_bfloat16>(p, stream) : launch_t<float>(p, stream);
}

}  // namespace convfwd

// Gated delta rule, whole sequences forward: see delta.h for the recurrence and seq_delta.cuh for its form in chunks.
//
// Two kernels.  The first takes every chunk and key head by itself: products of its rows, the triangular inverse T and
// the matrix A of each value head, and the factors of the rows, all to the workspace.  The second walks the
// chunks of a sequence and value head in order, for a block of the state's columns, which do not depend on one another:
// the state stays in registers and shared memory.
//
// What bounds them: the first, latency between its stages (inversion, products of 64 rows, factors by one warp a head): 8192 tokens, 32 value heads on
// 16 key heads of 128 x 128 in bf16 take 117 us, 220 MB of traffic (28% of copy rate).  The walk, the order of its chunks: 3802 tokens of a head of
// 48 x 80 in fp32 (60 chunks) take 244 us, 4 us a chunk, about as many in any number of CTAs an SM holds at once; in pieces of the axis 54 + 11 + 77.  Operands on their way
// a chunk ahead made no difference (257 us against 255): the products of 16 or 32 columns and their splits are one chain.
#include "seq_delta.cuh"

namespace convfwd {
namespace {

constexpr int LSQ = 72;              // row of a 64 x 64 matrix in shared memory: conflict-free pairs along rows

// (I + L)^-1 for the strictly lower triangular L in shared memory (rows of LSQ; the rest of it zero), to `inv` (all of it).
// Diagonal blocks of 8 by forward substitution, a thread a column; then [[P, 0], [B, Q]]^-1 = [[P', 0], [-Q' B P', Q']]
// for blocks of 8, 16 and 32.  No powers of L: they cancel badly where keys are alike.
__device__ __forceinline__ void invert(const float* L, float* inv, float* tmp) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t2 = (lane & 3) * 2;
    for (int i = threadIdx.x; i < DC * DC / 4; i += DT) {
        const int r = i / (DC / 4), c = i % (DC / 4) * 4;
        if (r / 8 != c / 8) *reinterpret_cast<float4*>(inv + r * LSQ + c) = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (threadIdx.x < DC) {
        const int o = threadIdx.x / 8 * 8, c = threadIdx.x % 8;
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float4 l0 = *reinterpret_cast<const float4*>(L + (o + i) * LSQ + o), l1 = *reinterpret_cast<const float4*>(L + (o + i) * LSQ + o + 4);
            const float l[8] = {l0.x, l0.y, l0.z, l0.w, l1.x, l1.y, l1.z, l1.w};
            float s0 = i == c ? 1.f : 0.f, s1 = 0.f;
#pragma unroll
            for (int j = 0; j < i; ++j) {
                if (j & 1) s1 = fmaf(-l[j], x[j], s1);
                else s0 = fmaf(-l[j], x[j], s0);
            }
            x[i] = s0 + s1;
            inv[(o + i) * LSQ + o + c] = x[i];
        }
    }
    __syncthreads();
    {                                // blocks of 8: rows o + 8, columns o; a thread an element
        const int o = threadIdx.x / 64 * 16, r = o + 8 + threadIdx.x % 64 / 8, c = o + threadIdx.x % 8;
        float v = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) v = fmaf(L[r * LSQ + o + k], inv[(o + k) * LSQ + c], v);
        tmp[r * LSQ + c] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) v = fmaf(inv[r * LSQ + o + 8 + k], tmp[(o + 8 + k) * LSQ + c], v);
        inv[r * LSQ + c] = -v;
    }
    __syncthreads();
    if (warp < 4) {                  // blocks of 16: rows o + 16, columns o; a warp 8 columns
        const int o = warp / 2 * 32, n0 = o + warp % 2 * 8;
        float acc[1][4];
        zero(acc);
        warp_mma<1>(acc, Along<float>{L, LSQ}, Across<float>{inv, LSQ}, o + 16, n0, o, o + 16);
        float* to = tmp + (o + 16 + g) * LSQ + n0 + t2;
        *reinterpret_cast<float2*>(to) = make_float2(acc[0][0], acc[0][1]);
        *reinterpret_cast<float2*>(to + 8 * LSQ) = make_float2(acc[0][2], acc[0][3]);
        __syncwarp();
        zero(acc);
        warp_mma<1>(acc, Along<float>{inv, LSQ}, Across<float>{tmp, LSQ}, o + 16, n0, o + 16, o + 32);
        to = inv + (o + 16 + g) * LSQ + n0 + t2;
        *reinterpret_cast<float2*>(to) = make_float2(-acc[0][0], -acc[0][1]);
        *reinterpret_cast<float2*>(to + 8 * LSQ) = make_float2(-acc[0][2], -acc[0][3]);
    }
    __syncthreads();
    {                                // blocks of 32: rows 32.., columns 0..31; a warp 16 rows and 8 columns
        const int m0 = 32 + warp / 4 * 16, n0 = warp % 4 * 8;
        float acc[1][4];
        zero(acc);
        warp_mma<1>(acc, Along<float>{L, LSQ}, Across<float>{inv, LSQ}, m0, n0, 0, 32);
        float* to = tmp + (m0 + g) * LSQ + n0 + t2;
        *reinterpret_cast<float2*>(to) = make_float2(acc[0][0], acc[0][1]);
        *reinterpret_cast<float2*>(to + 8 * LSQ) = make_float2(acc[0][2], acc[0][3]);
        __syncthreads();
        zero(acc);
        warp_mma<1>(acc, Along<float>{inv, LSQ}, Across<float>{tmp, LSQ}, m0, n0, 32, 64);
        to = inv + (m0 + g) * LSQ + n0 + t2;
        *reinterpret_cast<float2*>(to) = make_float2(-acc[0][0], -acc[0][1]);
        *reinterpret_cast<float2*>(to + 8 * LSQ) = make_float2(-acc[0][2], -acc[0][3]);
    }
    __syncthreads();
}

constexpr int CHUNK_HEADS = 4;       // value heads whose decay is prepared at once

template <typename T, int KP>
struct ChunkSmem {
    static constexpr int LD = KP + 8;
    T q[DC * LD], k[DC * LD];
    float L[DC * LSQ], inv[DC * LSQ], tmp[DC * LSQ], a[DC * LSQ];
    float2 b[CHUNK_HEADS][DC];
    float rq[DC], rk[DC], beta[CHUNK_HEADS][DC];
    float before[4][DC];             // exp(b_16r - b_j), j < 16 r: decay from a token to the first row of a tile
};

template <typename T, int KP>
__global__ void __launch_bounds__(DT) delta_chunk_kernel(const __grid_constant__ SeqDeltaParams p) {
    extern __shared__ __align__(16) unsigned char raw[];
    using Smem = ChunkSmem<T, KP>;
    Smem& s = *reinterpret_cast<Smem*>(raw);
    constexpr int LD = Smem::LD;
    const CutPiece cut = cut_piece(p.ax, blockIdx.x, DC);
    dep_launch();
    if (cut.n <= 0) return;
    const int kh = blockIdx.y, rep = p.Hv / p.Hk;
    load_rows<KP, LD>(s.q, static_cast<const T*>(p.q) + cut.t0 * p.q_ld + kh * p.Dk, p.q_ld, cut.n, p.Dk, p.wide);
    load_rows<KP, LD>(s.k, static_cast<const T*>(p.k) + cut.t0 * p.k_ld + kh * p.Dk, p.k_ld, cut.n, p.Dk, p.wide);
    copies_commit();
    copies_wait<0>();
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t2 = (lane & 3) * 2;
    {
        const float r = p.norm ? row_length<KP, LD>(threadIdx.x < 128 ? s.q : s.k) : 1.f;
        if ((threadIdx.x & 1) == 0) (threadIdx.x < 128 ? s.rq : s.rk)[(threadIdx.x & 127) >> 1] = r;
    }
    // rows of K K^T (warps 0..3) and Q K^T (4..7), 16 a warp, for all of the key head's value heads
    float acc[8][4];
    zero(acc);
    const int m0 = (warp & 3) * 16;
    warp_mma<8>(acc, Along<T>{warp < 4 ? s.k : s.q, LD}, Along<T>{s.k, LD}, m0, 0, 0, KP);
    for (int h = kh * rep; h < (kh + 1) * rep; ++h) {
        __syncthreads();             // (the lengths are there; the last head's matrices are read)
        float* tri = p.tri + ((long long)blockIdx.x * p.Hv + h) * (p.planes ? DELTA_PLANES / 4 : 2 * DC * DC);
        const int hs = (h - kh * rep) % CHUNK_HEADS;
        if (hs == 0) {               // the next heads' decay, a warp each
            const int hw = h + warp;
            if (warp < CHUNK_HEADS && hw < (kh + 1) * rep) {
                float2 b[2];
                chunk_decay(p.g + cut.t0 * p.g_ld + hw, p.g_ld, cut.n, b);
                float* rows = p.rows + ((long long)blockIdx.x * p.Hv + hw) * DELTA_ROWS;
                const float2 end = make_float2(__shfl_sync(0xffffffffu, b[1].x, 31), __shfl_sync(0xffffffffu, b[1].y, 31));
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int r = 2 * lane + i;
                    const float beta = r < cut.n ? p.beta[(cut.t0 + r) * p.beta_ld + hw] : 0.f;
                    const float e = expf(b[i].x) * (1.f + b[i].y);
                    s.b[warp][r] = b[i];
                    s.beta[warp][r] = beta;
                    rows[RF_IN + r] = beta * e * s.rk[r];
                    rows[RF_OUT + r] = p.scale * e * s.rq[r];
                    rows[RF_END + r] = decay_between(end, b[i]) * s.rk[r];
                    rows[RF_BETA + r] = beta;
                    rows[RF_RQ + r] = s.rq[r];
                    rows[RF_RK + r] = s.rk[r];
                    *reinterpret_cast<float2*>(rows + RF_B + 2 * r) = b[i];
                }
                if (lane == 0) rows[RF_DECAY] = expf(end.x) * (1.f + end.y);
            }
            __syncthreads();
        }
        {                            // (with the column's length: every use has both)
            const int r = threadIdx.x >> 6, j = threadIdx.x & 63;
            s.before[r][j] = j < 16 * r ? decay_between(s.b[hs][16 * r], s.b[hs][j]) * s.rk[j] : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int i = m0 + g + 8 * half;
            const float2 bi = s.b[hs][i];
            const float f = warp < 4 ? s.beta[hs][i] * s.rk[i] : p.scale * s.rq[i];
            const float lead = f * decay_between(bi, s.b[hs][m0]);       // from the tile's first row
            const float* before = s.before[m0 >> 4];
#pragma unroll
            for (int n = 0; n < 8; ++n) {
                float v[2] = {0.f, 0.f};
                if (8 * n < m0) {    // to the left of the diagonal tile: both factors are at most 1
                    const float2 e = *reinterpret_cast<const float2*>(before + 8 * n + t2);
                    v[0] = acc[n][2 * half] * lead * e.x;
                    v[1] = acc[n][2 * half + 1] * lead * e.y;
                } else if (8 * n < m0 + 16) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int j = 8 * n + t2 + e;
                        if (j < i || (j == i && warp >= 4)) v[e] = acc[n][2 * half + e] * f * s.rk[j] * decay_between(bi, s.b[hs][j]);
                    }
                }
                float* to = warp < 4 ? s.L + i * LSQ : p.planes ? s.a + i * LSQ : tri + DC * DC + i * DC;
                *reinterpret_cast<float2*>(to + 8 * n + t2) = make_float2(v[0], v[1]);
            }
        }
        __syncthreads();
        invert(s.L, s.inv, s.tmp);
        if (p.planes) {
            const float* below = s.a;
            if (p.planes == 1) {     // A T: y is then of R, like U
                const int n0 = (warp >> 2) * 32;
                float at[4][4];
                zero(at);
                warp_mma<4>(at, Along<float>{s.a, LSQ}, Across<float>{s.inv, LSQ}, m0, n0, 0, m0 + 16);
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    float* to = s.tmp + (m0 + g) * LSQ + n0 + 8 * n + t2;
                    *reinterpret_cast<float2*>(to) = make_float2(at[n][0], at[n][1]);
                    *reinterpret_cast<float2*>(to + 8 * LSQ) = make_float2(at[n][2], at[n][3]);
                }
                below = s.tmp;
                __syncthreads();
            }
            for (int i = threadIdx.x; i < 2 * DC * 8; i += DT) {
                const int r = i >> 3, c = i & 7;
                const float* from = (r < DC ? s.inv + r * LSQ : below + (r - DC) * LSQ) + c * 8;
                float x[8];
                *reinterpret_cast<float4*>(x) = *reinterpret_cast<const float4*>(from);
                *reinterpret_cast<float4*>(x + 4) = *reinterpret_cast<const float4*>(from + 4);
#pragma unroll
                for (int k = 0; k < 3; ++k) {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        w[e] = bf2_pack(x[2 * e], x[2 * e + 1]);
                        float a, b;
                        bf2_unpack(w[e], a, b);
                        x[2 * e] -= a;
                        x[2 * e + 1] -= b;
                    }
                    reinterpret_cast<uint4*>(tri)[(k * 2 * DC + r) * 8 + (c ^ (r & 7))] = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            continue;
        }
        for (int i = threadIdx.x; i < DC * DC / 4; i += DT) {
            const int r = i / (DC / 4), c = i % (DC / 4) * 4;
            *reinterpret_cast<float4*>(tri + r * DC + c) = *reinterpret_cast<const float4*>(s.inv + r * LSQ + c);
        }
    }
}

// ---- the walk ----
// DVB columns of the state of a sequence and value head.  Warps 0..3 hold the state (16 MT rows each) and K's rows of the first
// product; warps 4..7 Q's, and the rows of y.
template <typename T, int KP, int DVB>
struct WalkSmem {
    static constexpr int LD = KP + 8, LV = DVB + 4;      // LV: conflict-free where k runs across rows
    T k[DC * LD], q[DC * LD];
    float inv[DC * LSQ], a[DC * LSQ];
    float h[KP * LV], r[DC * LV], u[DC * LV];
    float rows[DELTA_FACTORS];
};

template <typename T, int KP, int DVB, int MODE>
__global__ void __launch_bounds__(DT) delta_walk_kernel(const __grid_constant__ SeqDeltaParams p, int dvbs, int dkbs) {
    extern __shared__ __align__(16) unsigned char raw[];
    using Smem = WalkSmem<T, KP, DVB>;
    Smem& s = *reinterpret_cast<Smem*>(raw);
    constexpr int LD = Smem::LD, LV = Smem::LV, NT = DVB / 8, MT = KP / 64;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t2 = (lane & 3) * 2;
    const WalkPlace w = walk_place<MODE>(p, dvbs, dkbs);
    if (MODE != DELTA_WHOLE) dep_wait();
    if (w.none) return;
    const int h = w.h, c0 = w.dvb * DVB, kh = h / (p.Hv / p.Hk), t0 = w.t0, t1 = w.t1, chunks = w.chunks, slot0 = w.slot0;
    const long long row = seq_slot(p.sl, w.seq), state = (row * p.Hv + h) * (long long)p.Dk * p.Dv;
    const long long kept = ((long long)w.mark * p.Hv + h) * p.Dk;             // rows of what is kept by piece
    const float* from = MODE == DELTA_JOINED && !(w.first && w.last) ? (w.first ? p.added : p.left) + kept * p.Dvp : nullptr;
    float* saved = MODE == DELTA_PIECES ? nullptr : p.saved;
    const int Dv = w.unit ? 0 : p.Dv;
    // the state in the layout of a product's sums: rows 16 (warp MT + m) + g and + 8, columns c0 + 8 n + t2 and + 1
    float st[MT][NT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = (warp * MT + m) * 16 + g + (e >> 1) * 8, c = c0 + 8 * n + t2 + (e & 1);
                st[m][n][e] = 0.f;
                if (warp < 4 && r < p.Dk) {
                    if (w.unit) st[m][n][e] = r == c ? 1.f : 0.f;
                    else if (from) st[m][n][e] = c < p.Dvp ? from[(long long)r * p.Dvp + c] : 0.f;
                    else if ((MODE != DELTA_PIECES || w.first) && p.h_in && row >= 0 && c < p.Dv) st[m][n][e] = p.h_in[state + (long long)r * p.Dv + c];
                }
            }
    auto put_state = [&]() {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float* to = s.h + ((warp * MT + m) * 16 + g) * LV + 8 * n + t2;
                *reinterpret_cast<float2*>(to) = make_float2(st[m][n][0], st[m][n][1]);
                *reinterpret_cast<float2*>(to + 8 * LV) = make_float2(st[m][n][2], st[m][n][3]);
            }
    };
    if (warp < 4) put_state();
    if (MODE == DELTA_WHOLE) dep_wait();
    for (int c = 0; c < chunks; ++c) {
        const int t = t0 + c * DC, n = min(DC, t1 - t);
        const long long at = (long long)(slot0 + c) * p.Hv + h;
        load_rows<KP, LD>(s.k, static_cast<const T*>(p.k) + t * p.k_ld + kh * p.Dk, p.k_ld, n, p.Dk, p.wide);
        load_rows<KP, LD>(s.q, static_cast<const T*>(p.q) + t * p.q_ld + kh * p.Dk, p.q_ld, n, p.Dk, p.wide);
        load_square<LSQ>(s.inv, p.tri + at * (2 * DC * DC));
        load_square<LSQ>(s.a, p.tri + at * (2 * DC * DC) + DC * DC);
        if (threadIdx.x < DELTA_FACTORS / 4) copy16_async(s.rows + threadIdx.x * 4, p.rows + at * DELTA_ROWS + threadIdx.x * 4, true);
        copies_commit();
        const int i0 = (warp & 3) * 16 + g;
        float2 v[2][NT];             // the rows of v that R needs, as the product's sums lie
        if (warp < 4) {
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const int i = i0 + 8 * half, col = c0 + 8 * j + t2;
                    v[half][j] = i < n ? load_pair(static_cast<const T*>(p.v) + (t + i) * p.v_ld + h * p.Dv + col, col, Dv, p.pairs) : make_float2(0.f, 0.f);
                }
            if (saved) {             // the state before the chunk
                float* to = saved + at * p.Dk * p.Dvp;
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        const int r = (warp * MT + m) * 16 + g, col = c0 + 8 * j + t2;
                        if (col < p.Dvp) {
                            if (r < p.Dk) *reinterpret_cast<float2*>(to + (long long)r * p.Dvp + col) = make_float2(st[m][j][0], st[m][j][1]);
                            if (r + 8 < p.Dk) *reinterpret_cast<float2*>(to + (long long)(r + 8) * p.Dvp + col) = make_float2(st[m][j][2], st[m][j][3]);
                        }
                    }
            }
        }
        copies_wait<0>();
        __syncthreads();
        float acc[NT][4];            // K h0 (warps 0..3), Q h0 (4..7)
        zero(acc);
        if (MODE != DELTA_PIECES || warp < 4)
            warp_mma<NT>(acc, Along<T>{warp < 4 ? s.k : s.q, LD}, Across<float>{s.h, LV}, (warp & 3) * 16, 0, 0, KP);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int i = i0 + 8 * half;
            if (warp < 4) {
                const float beta = s.rows[RF_BETA + i], f = s.rows[RF_IN + i];
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    *reinterpret_cast<float2*>(s.r + i * LV + 8 * j + t2) =
                        make_float2(beta * v[half][j].x - f * acc[j][2 * half], beta * v[half][j].y - f * acc[j][2 * half + 1]);
            } else {
                const float f = s.rows[RF_OUT + i];
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    acc[j][2 * half] *= f;
                    acc[j][2 * half + 1] *= f;
                }
            }
        }
        __syncthreads();
        {                            // U = T R: a warp 16 rows and half of the columns; T's columns end with its rows
            float u[NT / 2][4];
            zero(u);
            const int m0 = (warp & 3) * 16, n0 = (warp >> 2) * (DVB / 2);
            warp_mma<NT / 2>(u, Along<float>{s.inv, LSQ}, Across<float>{s.r, LV}, m0, n0, 0, m0 + 16);
#pragma unroll
            for (int j = 0; j < NT / 2; ++j) {
                float* to = s.u + (m0 + g) * LV + n0 + 8 * j + t2;
                *reinterpret_cast<float2*>(to) = make_float2(u[j][0], u[j][1]);
                *reinterpret_cast<float2*>(to + 8 * LV) = make_float2(u[j][2], u[j][3]);
            }
            if (saved) {
                float* keep = saved + p.saved_u + at * DC * p.Dvp;
#pragma unroll
                for (int j = 0; j < NT / 2; ++j) {
                    const int col = c0 + n0 + 8 * j + t2;
                    if (col < p.Dvp) {
                        *reinterpret_cast<float2*>(keep + (long long)(m0 + g) * p.Dvp + col) = make_float2(u[j][0], u[j][1]);
                        *reinterpret_cast<float2*>(keep + (long long)(m0 + g + 8) * p.Dvp + col) = make_float2(u[j][2], u[j][3]);
                    }
                }
            }
        }
        __syncthreads();
        if (warp < 4) {              // h = exp(b_C) h0 + (exp(b_C - b) K)^T U
            const float decay = s.rows[RF_DECAY];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                float d[NT][4];
                zero(d);
                warp_mma<NT>(d, Across<T>{s.k, LD}, AcrossScaled{s.u, LV, s.rows + RF_END}, (warp * MT + m) * 16, 0, 0, DC);
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) st[m][j][e] = fmaf(decay, st[m][j][e], d[j][e]);
            }
            put_state();
        } else if (MODE != DELTA_PIECES) {       // Y = scale exp(b) Q h0 + A U
            const int m0 = (warp & 3) * 16;
            float d[NT][4];
            zero(d);
            warp_mma<NT>(d, Along<float>{s.a, LSQ}, Across<float>{s.u, LV}, m0, 0, 0, m0 + 16);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int i = i0 + 8 * half;
                if (i < n) {
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        const int col = c0 + 8 * j + t2;
                        store_pair(static_cast<T*>(p.y) + (t + i) * p.y_ld + h * p.Dv + col, col, p.Dv, p.pairs,
                                   make_float2(acc[j][2 * half] + d[j][2 * half], acc[j][2 * half + 1] + d[j][2 * half + 1]));
                    }
                }
            }
        }
        __syncthreads();
    }
    if (MODE == DELTA_PIECES) {
        float* to = w.unit ? p.through : p.added;
        const int width = w.unit ? p.Dkp : p.Dvp;
        if (warp < 4)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int r = (warp * MT + m) * 16 + g + (e >> 1) * 8, c = c0 + 8 * n + t2 + (e & 1);
                        if (r < p.Dk && c < width) to[(kept + r) * width + c] = st[m][n][e];
                    }
        return;
    }
    if (warp < 4 && p.h_out && row >= 0 && w.last) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int r = (warp * MT + m) * 16 + g + (e >> 1) * 8, c = c0 + 8 * n + t2 + (e & 1);
                    if (r < p.Dk && c < p.Dv) p.h_out[state + (long long)r * p.Dv + c] = st[m][n][e];
                }
    }
}

template <typename T, int KP>
cudaError_t launch_chunks(const SeqDeltaParams& p, cudaStream_t stream) {
    constexpr int smem = (int)sizeof(ChunkSmem<T, KP>);
    cudaError_t e = cudaFuncSetAttribute(delta_chunk_kernel<T, KP>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_kernel(delta_chunk_kernel<T, KP>, dim3((unsigned)p.slots, (unsigned)p.Hk), dim3(DT), smem, stream, false, 1, p);
}

// The states that the pieces of a sequence leave, but for the last, 16 columns of a value head a block: h <- through h + added from piece to piece, the
// next piece's matrix and this one's sums on their way during the products.  A matrix of a piece over which states grow (keys longer than 1, g above
// 0) may hold what is beyond fp32's range; where the state is zero nothing of it passes on, as in a walk: results that are not finite are taken
// again, without the products of zeros.
template <int KP>
struct JoinSmem {
    static constexpr int LP = KP + 8, LV = 20;
    float m[2][KP * LP], h[2][KP * LV];
};
template <int KP>
__global__ void __launch_bounds__(DT) delta_join_kernel(const __grid_constant__ SeqDeltaParams p, int cols) {
    extern __shared__ __align__(16) unsigned char raw[];
    using Smem = JoinSmem<KP>;
    Smem& s = *reinterpret_cast<Smem*>(raw);
    constexpr int LP = Smem::LP, LV = Smem::LV, NT = KP / 64;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t2 = (lane & 3) * 2;
    const int c0 = blockIdx.x % cols * 16, sh = blockIdx.x / cols, h = sh % p.Hv, at = sh / p.Hv, len = p.run * DC;
    int seq = at;
    bool first = true;
    if (p.ax.S > p.marks) {              // by the marks of first pieces, where those are fewer
        const MarkPiece c = mark_piece(p.ax, at, len);
        first = c.index == 0;
        seq = c.s;
    }
    const int t0 = p.ax.L > 0 ? seq * p.ax.L : seq_start(p.ax, seq, 0), t1 = p.ax.L > 0 ? t0 + p.ax.L : seq_start(p.ax, seq + 1, t0);
    const int n = (t1 - t0 + len - 1) / len;
    dep_wait();
    if (n < 2 || !first) return;
    const int base = first_mark(t0, len);
    const long long row = seq_slot(p.sl, seq), state = (row * p.Hv + h) * (long long)p.Dk * p.Dv;
    auto rows_of = [&](int i) { return ((long long)(base + i) * p.Hv + h) * p.Dk; };
    auto load = [&](int i) {             // the matrix of piece i
        for (int e = threadIdx.x; e < KP * (KP / 4); e += DT) {
            const int r = e / (KP / 4), c = e % (KP / 4) * 4;
            const bool on = i < n - 1 && r < p.Dk && c < p.Dkp;
            copy16_async(s.m[i & 1] + r * LP + c, on ? p.through + (rows_of(i) + r) * p.Dkp + c : p.through, on);
        }
        copies_commit();
    };
    load(1);
    for (int e = threadIdx.x; e < KP * 16; e += DT) {
        const int r = e / 16, c = c0 + e % 16;
        const bool on = r < p.Dk && c < p.Dvp;
        const float v = on ? p.added[(rows_of(0) + r) * p.Dvp + c] : 0.f;
        s.h[0][r * LV + e % 16] = v;
        if (on) {
            p.left[(rows_of(0) + r) * p.Dvp + c] = v;
            p.added[(rows_of(0) + r) * p.Dvp + c] = p.h_in && row >= 0 && c < p.Dv ? p.h_in[state + (long long)r * p.Dv + c] : 0.f;
        }
    }
    const int m0 = warp % (KP / 16) * 16, n0 = warp / (KP / 16) * 8;
    for (int i = 1; i < n - 1; ++i) {
        copies_wait<0>();
        __syncthreads();                 // (the last one's matrix and state have been read)
        load(i + 1);
        float acc[NT][4], more[NT][4];
        zero(acc);
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = m0 + g + (e >> 1) * 8, c = c0 + n0 + 8 * j + t2 + (e & 1);
                more[j][e] = r < p.Dk && c < p.Dvp ? p.added[(rows_of(i) + r) * p.Dvp + c] : 0.f;
            }
        warp_mma<NT>(acc, Along<float>{s.m[i & 1], LP}, Across<float>{s.h[(i - 1) & 1], LV}, m0, n0, 0, KP);
        bool finite = true;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) finite = finite && isfinite(acc[j][e]);
        if (!finite) {
            for (int j = 0; j < NT; ++j)
                for (int e = 0; e < 4; ++e) {
                    const float* m = s.m[i & 1] + (m0 + g + (e >> 1) * 8) * LP;
                    const float* h = s.h[(i - 1) & 1] + n0 + 8 * j + t2 + (e & 1);
                    float v = 0.f;
                    for (int k = 0; k < KP; ++k)
                        if (h[k * LV] != 0.f) v = fmaf(m[k], h[k * LV], v);
                    acc[j][e] = v;
                }
        }
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = m0 + g + (e >> 1) * 8, cl = n0 + 8 * j + t2 + (e & 1), c = c0 + cl;
                const bool on = r < p.Dk && c < p.Dvp;
                const float v = on ? acc[j][e] + more[j][e] : 0.f;
                s.h[i & 1][r * LV + cl] = v;
                if (on) p.left[(rows_of(i) + r) * p.Dvp + c] = v;
            }
    }
    copies_wait<0>();
}
template <int KP>
cudaError_t launch_join(const SeqDeltaParams& p, cudaStream_t stream) {
    constexpr int smem = (int)sizeof(JoinSmem<KP>);
    cudaError_t e = cudaFuncSetAttribute(delta_join_kernel<KP>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int cols = (p.Dv + 15) / 16;
    return launch_kernel(delta_join_kernel<KP>, dim3((unsigned)(delta_joined(p.ax.S, p.marks) * p.Hv * cols)), dim3(DT), smem, stream, true, 1, p, cols);
}

template <typename T, int KP, int DVB, int MODE>
cudaError_t launch_mode(const SeqDeltaParams& p, cudaStream_t stream) {
    constexpr int smem = (int)sizeof(WalkSmem<T, KP, DVB>);
    cudaError_t e = cudaFuncSetAttribute(delta_walk_kernel<T, KP, DVB, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int dvbs = (p.Dv + DVB - 1) / DVB, dkbs = (p.Dk + DVB - 1) / DVB;
    const long long blocks = (MODE == DELTA_WHOLE ? p.ax.S : MODE == DELTA_PIECES ? p.marks : p.pieces) * (long long)p.Hv * (MODE == DELTA_PIECES ? dvbs + dkbs : dvbs);
    return launch_kernel(delta_walk_kernel<T, KP, DVB, MODE>, dim3((unsigned)blocks), dim3(DT), smem, stream, p.slots > 0, 1, p, dvbs, dkbs);
}
template <typename T, int KP, int DVB>
cudaError_t launch_walk(const SeqDeltaParams& p, cudaStream_t stream) {
    if (!p.run) return launch_mode<T, KP, DVB, DELTA_WHOLE>(p, stream);
    cudaError_t e = launch_mode<T, KP, DVB, DELTA_PIECES>(p, stream);
    if (e == cudaSuccess) e = launch_join<KP>(p, stream);
    return e == cudaSuccess ? launch_mode<T, KP, DVB, DELTA_JOINED>(p, stream) : e;
}

template <typename T>
cudaError_t launch(const SeqDeltaParams& p, cudaStream_t stream) {
    // 32 columns a block, or 16 where that leaves SMs without one, or where the axis is cut (5003 tokens of 6 heads of
    // 48 x 80 in pieces: the last walk takes 76 us with 16, 103 with 32)
    const bool narrow = p.Dv <= 16 || p.run || p.ax.S * (long long)p.Hv * ((p.Dv + 31) / 32) < p.sms;
    if (p.Dk <= 64) return narrow ? launch_walk<T, 64, 16>(p, stream) : launch_walk<T, 64, 32>(p, stream);
    return narrow ? launch_walk<T, 128, 16>(p, stream) : launch_walk<T, 128, 32>(p, stream);
}

}  // namespace

cudaError_t launch_seq_delta_chunks(const SeqDeltaParams& p, bool bf16, cudaStream_t stream) {
    if (p.slots == 0) return cudaSuccess;
    if (bf16) return p.Dk <= 64 ? launch_chunks<__nv_bfloat16, 64>(p, stream) : launch_chunks<__nv_bfloat16, 128>(p, stream);
    return p.Dk <= 64 ? launch_chunks<float, 64>(p, stream) : launch_chunks<float, 128>(p, stream);
}

cudaError_t launch_seq_delta_fwd(const SeqDeltaParams& args, bool bf16, cudaStream_t stream) {
    SeqDeltaParams p = args;
    p.planes = bf16 && p.wide && p.compact && p.Dv > 16 ? 1 : 0;
    const cudaError_t e = launch_seq_delta_chunks(p, bf16, stream);
    if (e != cudaSuccess) return e;
    if (p.planes) {
        if (!p.run) return launch_seq_delta_walk_tc(p, DELTA_WHOLE, stream);
        cudaError_t f = launch_seq_delta_walk_tc(p, DELTA_PIECES, stream);
        if (f == cudaSuccess) f = p.Dk <= 64 ? launch_join<64>(p, stream) : launch_join<128>(p, stream);
        return f == cudaSuccess ? launch_seq_delta_walk_tc(p, DELTA_JOINED, stream) : f;
    }
    return bf16 ? launch<__nv_bfloat16>(p, stream) : launch<float>(p, stream);
}

}  // namespace convfwd

// Gated delta rule, whole sequences backward: see delta.h for the recurrence and seq_delta.cuh for its form in chunks.
// With dh the gradient at the state a chunk leaves and dY at its outputs:
//   dU = A^T dY + (exp(b_C - b) K) dh        dR = T^T dU        dV = beta dR
//   dh0 = exp(b_C) dh + scale (exp(b) Q)^T dY - (beta exp(b) K)^T dR
//   dQ = scale (E . dY U^T) K + scale exp(b) dY h0^T
//   X  = -(E . dR U^T) K - exp(b) dR h0^T                      (what beta K takes part in)
//   Z  = scale (E . dY U^T)^T Q - (beta E . dR U^T)^T K + (exp(b_C - b) U) dh^T
//   dK = beta X + Z,   dbeta_i = V_i.dR_i + k_i.X_i
//   db_i = q_i.dQ_i + beta_i k_i.X_i - k_i.Z_i, and at the chunk's last token exp(b_C) <h0, dh> + sum_j k_j.(exp(b_C - b) U dh^T)_j;
//   dg is the sum of db from its token on.
// Two terms of db stand in it twice, with either sign, and are as large as the outputs' gradients, while dg is as small as its factor exp(g):
// q_i k_i scale dY_i.U_i, in q_i.dQ_i and k_i.Z_i, and the last token's k.(U dh^T), in k.Z and in the sum over j.  They are left out on both sides: with
// them dg was off by 4e-3 of its terms at g = -12 for all tokens, now by 1e-6 at any.  (What tokens behind a strong decay do among themselves still cancels in
// that token's dg: it is off by 1e-7 or so of theirs.)
//
// Three kernels: the forward pass's first again (T, A, factors of the rows); a walk over the chunks from the last to the
// first for a block of columns (dV, the gradients of the states); and every chunk by itself for the rest.  In fp32 2 sequences of 1500
// tokens, 6 heads of 64 x 64 take 17, 135 and 50 us: the walk's 24 chunks in order are what bounds them (see seq_delta.cu).
#include "seq_delta.cuh"

namespace convfwd {
namespace {

// element (i, k) of a matrix of the plan's type at p[k ld + i], times f[k]
template <typename T>
struct AcrossRows {
    const T* p;
    int ld;
    const float* f;
    static constexpr bool EXACT = false;
    __device__ __forceinline__ float2 get(int i, int k) const {
        const float2 s = *reinterpret_cast<const float2*>(f + k);
        return make_float2(seq_ld(p + k * ld + i) * s.x, seq_ld(p + (k + 1) * ld + i) * s.y);
    }
};

// 64 rows of W columns, from column c0 of `width`, of a tensor of tokens to shared memory rows of LD; zero behind
// the rows and columns.  Done on return.
template <int W, int LD, typename T>
__device__ __forceinline__ void load_block(T* to, const T* from, long long ld, int n, int c0, int width, bool pairs) {
#pragma unroll
    for (int j = 0; j < DC * W / 2 / DT; ++j) {
        const int i = threadIdx.x + j * DT, r = i / (W / 2), c = i % (W / 2) * 2;
        const float2 v = r < n ? load_pair(from + r * ld + c, c0 + c, width, pairs) : make_float2(0.f, 0.f);
        seq_st2(to + r * LD + c, v, true, true);
    }
}

constexpr int LT = 68;               // row of T and A: conflict-free where k runs across rows

template <typename T, int KP, int DVB>
struct BackSmem {
    static constexpr int LD = KP + 8, LV = DVB + 4, LY = DVB + (sizeof(T) == 2 ? 8 : 4);
    T k[DC * LD], q[DC * LD];
    float inv[DC * LT], a[DC * LT];
    float dh[KP * LV], du[DC * LV], ndr[DC * LV];
    T dy[DC * LY];
    float rows[DELTA_FACTORS];
};

template <typename T, int KP, int DVB>
__global__ void __launch_bounds__(DT) delta_back_kernel(const __grid_constant__ SeqDeltaParams p, int dvbs) {
    extern __shared__ __align__(16) unsigned char raw[];
    using Smem = BackSmem<T, KP, DVB>;
    Smem& s = *reinterpret_cast<Smem*>(raw);
    constexpr int LD = Smem::LD, LV = Smem::LV, LY = Smem::LY;
    constexpr int WPM = 8 / (KP / 16), NS = DVB / 8 / WPM;       // warps that share 16 rows of the state; 8-column tiles of each
    constexpr int NH = DVB / 16;                                 // the same for products of tokens: two warps share 16 rows
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t2 = (lane & 3) * 2;
    const int dvb = blockIdx.x % dvbs, sh = blockIdx.x / dvbs, h = sh % p.Hv, seq = sh / p.Hv;
    const int c0 = dvb * DVB, kh = h / (p.Hv / p.Hk);
    const int t0 = p.ax.L > 0 ? seq * p.ax.L : seq_start(p.ax, seq, 0), t1 = p.ax.L > 0 ? t0 + p.ax.L : seq_start(p.ax, seq + 1, t0);
    const int chunks = (t1 - t0 + DC - 1) / DC, slot0 = cut_base(p.ax, seq, DC);
    const long long row = seq_slot(p.sl, seq), state = (row * p.Hv + h) * (long long)p.Dk * p.Dv;
    const int sr = warp / WPM * 16 + g, sc = warp % WPM * (NS * 8) + t2;      // the thread's part of the state: rows sr, sr + 8
    float st[NS][4];
#pragma unroll
    for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int r = sr + (e >> 1) * 8, c = c0 + sc + 8 * n + (e & 1);
            st[n][e] = p.dh_out && row >= 0 && r < p.Dk && c < p.Dv ? p.dh_out[state + (long long)r * p.Dv + c] : 0.f;
        }
    dep_launch();
    dep_wait();
    for (int c = chunks - 1; c >= 0; --c) {
        const int t = t0 + c * DC, n = min(DC, t1 - t);
        const long long at = (long long)(slot0 + c) * p.Hv + h;
        load_rows<KP, LD>(s.k, static_cast<const T*>(p.k) + t * p.k_ld + kh * p.Dk, p.k_ld, n, p.Dk, p.wide);
        load_rows<KP, LD>(s.q, static_cast<const T*>(p.q) + t * p.q_ld + kh * p.Dk, p.q_ld, n, p.Dk, p.wide);
        load_square<LT>(s.inv, p.tri + at * (2 * DC * DC));
        load_square<LT>(s.a, p.tri + at * (2 * DC * DC) + DC * DC);
        if (threadIdx.x < DELTA_FACTORS / 4) copy16_async(s.rows + threadIdx.x * 4, p.rows + at * DELTA_ROWS + threadIdx.x * 4, true);
        copies_commit();
        load_block<DVB, LY>(s.dy, static_cast<const T*>(p.dy) + t * p.dy_ld + h * p.Dv + c0, p.dy_ld, n, c0, p.Dv, p.pairs);
        float* keep = p.dstate + at * p.Dk * p.Dvp;
#pragma unroll
        for (int j = 0; j < NS; ++j) {
            *reinterpret_cast<float2*>(s.dh + sr * LV + sc + 8 * j) = make_float2(st[j][0], st[j][1]);
            *reinterpret_cast<float2*>(s.dh + (sr + 8) * LV + sc + 8 * j) = make_float2(st[j][2], st[j][3]);
            const int col = c0 + sc + 8 * j;
            if (col < p.Dvp) {
                if (sr < p.Dk) *reinterpret_cast<float2*>(keep + (long long)sr * p.Dvp + col) = make_float2(st[j][0], st[j][1]);
                if (sr + 8 < p.Dk) *reinterpret_cast<float2*>(keep + (long long)(sr + 8) * p.Dvp + col) = make_float2(st[j][2], st[j][3]);
            }
        }
        copies_wait<0>();
        __syncthreads();
        const int m0 = (warp & 3) * 16, n0 = (warp >> 2) * (DVB / 2);
        {
            float kd[NH][4], ay[NH][4];
            zero(kd);
            zero(ay);
            warp_mma<NH>(kd, Along<T>{s.k, LD}, Across<float>{s.dh, LV}, m0, n0, 0, KP);
            warp_mma<NH>(ay, Across<float>{s.a, LT}, Across<T>{s.dy, LY}, m0, n0, m0, DC);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const float f = s.rows[RF_END + m0 + g + 8 * half];
#pragma unroll
                for (int j = 0; j < NH; ++j)
                    *reinterpret_cast<float2*>(s.du + (m0 + g + 8 * half) * LV + n0 + 8 * j + t2) =
                        make_float2(fmaf(f, kd[j][2 * half], ay[j][2 * half]), fmaf(f, kd[j][2 * half + 1], ay[j][2 * half + 1]));
            }
        }
        __syncthreads();
        {
            float dr[NH][4];
            zero(dr);
            warp_mma<NH>(dr, Across<float>{s.inv, LT}, Across<float>{s.du, LV}, m0, n0, m0, DC);
            float* to = p.dr + at * DC * p.Dvp;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int i = m0 + g + 8 * half;
                const float beta = s.rows[RF_BETA + i];
#pragma unroll
                for (int j = 0; j < NH; ++j) {
                    const float2 v = make_float2(dr[j][2 * half], dr[j][2 * half + 1]);
                    const int col = c0 + n0 + 8 * j + t2;
                    *reinterpret_cast<float2*>(s.ndr + i * LV + n0 + 8 * j + t2) = make_float2(-v.x, -v.y);
                    if (col < p.Dvp) *reinterpret_cast<float2*>(to + (long long)i * p.Dvp + col) = v;
                    if (i < n)
                        store_pair(static_cast<T*>(p.dv) + (t + i) * p.dv_ld + h * p.Dv + col, col, p.Dv, p.pairs, make_float2(beta * v.x, beta * v.y));
                }
            }
        }
        __syncthreads();
        {
            const float decay = s.rows[RF_DECAY];
            float d[NS][4];
            zero(d);
            warp_mma<NS>(d, Across<T>{s.q, LD}, AcrossRows<T>{s.dy, LY, s.rows + RF_OUT}, warp / WPM * 16, warp % WPM * (NS * 8), 0, DC);
            warp_mma<NS>(d, Across<T>{s.k, LD}, AcrossScaled{s.ndr, LV, s.rows + RF_IN}, warp / WPM * 16, warp % WPM * (NS * 8), 0, DC);
#pragma unroll
            for (int j = 0; j < NS; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) st[j][e] = fmaf(decay, st[j][e], d[j][e]);
        }
        __syncthreads();
    }
    if (p.dh_in && row >= 0) {
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = sr + (e >> 1) * 8, c = c0 + sc + 8 * n + (e & 1);
                if (r < p.Dk && c < p.Dv) p.dh_in[state + (long long)r * p.Dv + c] = st[n][e];
            }
    }
}

// ---- every chunk by itself ----
constexpr int GB = 32;               // columns of the states, u, dR and dY at a time
constexpr int LB = GB + 8;           // their rows in shared memory: conflict-free pairs
constexpr int LP = 72;               // rows of the 64 x 64 matrices

template <typename T, int KP>
struct GradSmem {
    static constexpr int LD = KP + 8;
    T k[DC * LD], q[DC * LD];
    union {
        struct {
            float h0[KP * LB], dh[KP * LB], u[DC * LB], dr[DC * LB];
            T dy[DC * LB];
        };
        float m[4][DC * LP];         // scale E dYU^T by key and by query lengths, -E dRU^T the same
    };
    float2 b[DC];
    float rq[DC], rk[DC], beta[DC], vdr[DC];
    float qk[DC], own[DC];           // q.k and scale dY.U of a token
    float dots[4][2][DC];            // q.dQ, k.X, k.Z, k.(exp(b_C - b) U dh^T): by the two warps of a row
    float dotq[DC], dotk[DC];        // sums over the value heads
    float hh[DT / 32];
    int zero[DT / 32];
};

// Rows of W floats, `width` of them there (a multiple of 4), to rows of LB; `rows` of R rows.  Part of the copy group at hand.
template <int R>
__device__ __forceinline__ void load_floats(float* to, const float* from, long long ld, int rows, int c0, int width) {
#pragma unroll
    for (int j = 0; j < R * GB / 4 / DT; ++j) {
        const int i = threadIdx.x + j * DT, r = i / (GB / 4), c = i % (GB / 4) * 4;
        const bool on = r < rows && c0 + c < width;
        copy16_async(to + r * LB + c, on ? from + r * ld + c0 + c : from, on);
    }
}

template <typename T, int KP, bool SHARED>
__global__ void __launch_bounds__(DT, 1) delta_grad_kernel(const __grid_constant__ SeqDeltaParams p) {
    extern __shared__ __align__(16) unsigned char raw[];
    using Smem = GradSmem<T, KP>;
    Smem& s = *reinterpret_cast<Smem*>(raw);
    constexpr int LD = Smem::LD, NT = KP / 16;
    const CutPiece cut = cut_piece(p.ax, blockIdx.x, DC);
    if (cut.n <= 0) {
        dep_wait();                  // (what follows in the stream then follows the walk before it, too)
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t2 = (lane & 3) * 2;
    const int kh = blockIdx.y, rep = SHARED ? p.Hv / p.Hk : 1;
    const int m0 = (warp & 3) * 16, n0 = (warp >> 2) * (KP / 2), j0 = (warp >> 2) * 32;
    load_rows<KP, LD>(s.q, static_cast<const T*>(p.q) + cut.t0 * p.q_ld + kh * p.Dk, p.q_ld, cut.n, p.Dk, p.wide);
    load_rows<KP, LD>(s.k, static_cast<const T*>(p.k) + cut.t0 * p.k_ld + kh * p.Dk, p.k_ld, cut.n, p.Dk, p.wide);
    copies_commit();
    copies_wait<0>();
    __syncthreads();
    {
        const float r = p.norm ? row_length<KP, LD>(threadIdx.x < 128 ? s.q : s.k) : 1.f;
        if ((threadIdx.x & 1) == 0) (threadIdx.x < 128 ? s.rq : s.rk)[(threadIdx.x & 127) >> 1] = r;
    }
    {
        const int r = threadIdx.x >> 2;
        float d = 0.f;
#pragma unroll 4
        for (int c = (threadIdx.x & 3) * 2; c < KP; c += 8) {
            const float2 a = seq_ld2(s.q + r * LD + c), b = seq_ld2(s.k + r * LD + c);
            d = fmaf(a.x, b.x, fmaf(a.y, b.y, d));
        }
        d += __shfl_xor_sync(0xffffffffu, d, 1);
        d += __shfl_xor_sync(0xffffffffu, d, 2);
        if ((threadIdx.x & 3) == 0) s.qk[r] = d;
    }
    if (threadIdx.x < DC) s.dotq[threadIdx.x] = s.dotk[threadIdx.x] = 0.f;
    float tq[SHARED ? NT : 1][4], tk[SHARED ? NT : 1][4];
    zero(tq);
    zero(tk);
    dep_wait();
    for (int h = kh * rep; h < (kh + 1) * rep; ++h) {
        const long long at = (long long)blockIdx.x * p.Hv + h;
        float dq[NT][4], x[NT][4], z[NT][4], da[4][4], dl[4][4];
        zero(dq);
        zero(x);
        zero(z);
        zero(da);
        zero(dl);
        float vdr = 0.f, hh = 0.f;
        bool from_zero = true;       // the state before the chunk is zero
        for (int c0 = 0; c0 < p.Dv; c0 += GB) {
            __syncthreads();         // what was read of the block before (or of the last head's matrices)
            load_floats<KP>(s.h0, p.saved + at * p.Dk * p.Dvp, p.Dvp, p.Dk, c0, p.Dvp);
            load_floats<KP>(s.dh, p.dstate + at * p.Dk * p.Dvp, p.Dvp, p.Dk, c0, p.Dvp);
            load_floats<DC>(s.u, p.saved + p.saved_u + at * DC * p.Dvp, p.Dvp, DC, c0, p.Dvp);
            load_floats<DC>(s.dr, p.dr + at * DC * p.Dvp, p.Dvp, DC, c0, p.Dvp);
            copies_commit();
            load_block<GB, LB>(s.dy, static_cast<const T*>(p.dy) + cut.t0 * p.dy_ld + h * p.Dv + c0, p.dy_ld, cut.n, c0, p.Dv, p.pairs);
            const int vr = threadIdx.x >> 2, vc = (threadIdx.x & 3) * 8;      // a row of v.dR: four threads, 8 columns each
            float2 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = vr < cut.n ? load_pair(static_cast<const T*>(p.v) + (cut.t0 + vr) * p.v_ld + h * p.Dv + c0 + vc + 2 * i, c0 + vc + 2 * i, p.Dv, p.pairs)
                                  : make_float2(0.f, 0.f);
            copies_wait<0>();
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 d = *reinterpret_cast<const float2*>(s.dr + vr * LB + vc + 2 * i);
                vdr = fmaf(v[i].x, d.x, fmaf(v[i].y, d.y, vdr));
            }
#pragma unroll
            for (int j = 0; j < KP * GB / DT; ++j) {
                const int i = threadIdx.x + j * DT, o = i / GB * LB + i % GB;
                hh = fmaf(s.h0[o], s.dh[o], hh);
                from_zero = from_zero && s.h0[o] == 0.f;
            }
            warp_mma<NT>(dq, Along<T>{s.dy, LB}, Along<float>{s.h0, LB}, m0, n0, 0, GB);
            warp_mma<NT>(x, Along<float>{s.dr, LB}, Along<float>{s.h0, LB}, m0, n0, 0, GB);
            warp_mma<NT>(z, Along<float>{s.u, LB}, Along<float>{s.dh, LB}, m0, n0, 0, GB);
            if (j0 <= m0) {          // (below the diagonal)
                warp_mma<4>(da, Along<T>{s.dy, LB}, Along<float>{s.u, LB}, m0, j0, 0, GB);
                warp_mma<4>(dl, Along<float>{s.dr, LB}, Along<float>{s.u, LB}, m0, j0, 0, GB);
            }
        }
        vdr += __shfl_xor_sync(0xffffffffu, vdr, 1);
        vdr += __shfl_xor_sync(0xffffffffu, vdr, 2);
        if ((threadIdx.x & 3) == 0) s.vdr[threadIdx.x >> 2] = vdr;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) hh += __shfl_xor_sync(0xffffffffu, hh, d);
        from_zero = __all_sync(0xffffffffu, from_zero);
        if (lane == 0) {
            s.hh[warp] = hh;
            s.zero[warp] = from_zero;
        }
        float2 end = make_float2(0.f, 0.f);
        if (warp == 0) {
            float2 b[2];
            chunk_decay(p.g + cut.t0 * p.g_ld + h, p.g_ld, cut.n, b);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = 2 * lane + i;
                s.b[r] = b[i];
                s.beta[r] = r < cut.n ? p.beta[(cut.t0 + r) * p.beta_ld + h] : 0.f;
            }
        }
        __syncthreads();
        end = s.b[DC - 1];
        // the two triangles with their factors; rows of the sums scaled
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int i = m0 + g + 8 * half;
            const float2 bi = s.b[i];
            const float eb = expf(bi.x) * (1.f + bi.y), rqi = s.rq[i], rki = s.rk[i], bki = s.beta[i] * rki;
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int j = j0 + 8 * n + t2 + e, o = i * LP + j;
                    const float E = j < i ? decay_between(bi, s.b[j]) : 0.f, rkj = s.rk[j];
                    const float a = j < i ? p.scale * da[n][2 * half + e] * E : 0.f, l = j < i ? -dl[n][2 * half + e] * E : 0.f;
                    if (j == i) s.own[i] = p.scale * da[n][2 * half + e];
                    s.m[0][o] = a * rkj;
                    s.m[1][o] = a * rqi;
                    s.m[2][o] = l * rkj;
                    s.m[3][o] = l * bki;
                }
            const float fq = p.scale * eb, fz = decay_between(end, bi);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    dq[n][2 * half + e] *= fq;
                    x[n][2 * half + e] *= -eb;
                    z[n][2 * half + e] *= fz;
                }
        }
        // k.(exp(b_C - b) U dh^T) before the rest joins it; then all row products
        float dot[4][2];
        auto row_dot = [&](const float (&v)[NT][4], const T* with, float (&to)[2]) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float d = 0.f;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const float2 w = seq_ld2(with + (m0 + g + 8 * half) * LD + n0 + 8 * n + t2);
                    d = fmaf(w.x, v[n][2 * half], fmaf(w.y, v[n][2 * half + 1], d));
                }
                to[half] = d;
            }
        };
        row_dot(z, s.k, dot[3]);
        __syncthreads();
        warp_mma<NT>(dq, Along<float>{s.m[0], LP}, Across<T>{s.k, LD}, m0, n0, 0, m0 + 16);
        warp_mma<NT>(x, Along<float>{s.m[2], LP}, Across<T>{s.k, LD}, m0, n0, 0, m0 + 16);
        warp_mma<NT>(z, Across<float>{s.m[1], LP}, Across<T>{s.q, LD}, m0, n0, m0, DC);
        warp_mma<NT>(z, Across<float>{s.m[3], LP}, Across<T>{s.k, LD}, m0, n0, m0, DC);
        row_dot(dq, s.q, dot[0]);
        row_dot(x, s.k, dot[1]);
        row_dot(z, s.k, dot[2]);
        // a token's own term (see above), behind the products for db
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int i = m0 + g + 8 * half;
            const float own = s.own[i], oq = own * s.rk[i], ok = own * s.rq[i];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float2 kv = seq_ld2(s.k + i * LD + n0 + 8 * n + t2), qv = seq_ld2(s.q + i * LD + n0 + 8 * n + t2);
                dq[n][2 * half] = fmaf(oq, kv.x, dq[n][2 * half]);
                dq[n][2 * half + 1] = fmaf(oq, kv.y, dq[n][2 * half + 1]);
                z[n][2 * half] = fmaf(ok, qv.x, z[n][2 * half]);
                z[n][2 * half + 1] = fmaf(ok, qv.y, z[n][2 * half + 1]);
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float d = dot[k][half];
                d += __shfl_xor_sync(0xffffffffu, d, 1);
                d += __shfl_xor_sync(0xffffffffu, d, 2);
                if ((lane & 3) == 0) s.dots[k][warp >> 2][m0 + g + 8 * half] = d;
            }
        __syncthreads();
        if (warp == 0) {             // dbeta and dg, two tokens a lane
            float total = 0.f;
            double db[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = 2 * lane + i;
                const float rq = s.rq[r], rk = s.rk[r], beta = s.beta[r];
                const float qq = rq * (s.dots[0][0][r] + s.dots[0][1][r]), kx = rk * (s.dots[1][0][r] + s.dots[1][1][r]);
                const float kz = rk * (s.dots[2][0][r] + s.dots[2][1][r]);
                const float own = s.own[r] * s.qk[r] * rq * rk;
                const bool end = r == cut.n - 1;             // (no token behind it has a part in its k.Z)
                total += end ? 0.f : rk * (s.dots[3][0][r] + s.dots[3][1][r]);
                db[i] = (double)(end ? qq : qq - kz) + (double)(beta * kx);
                if (r < cut.n) p.dbeta[(cut.t0 + r) * p.dbeta_ld + h] = s.vdr[r] + kx;
                s.dotq[r] += qq + own;
                s.dotk[r] += fmaf(beta, kx, kz + own);
            }
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
            float all = 0.f;
#pragma unroll
            for (int w = 0; w < DT / 32; ++w) all += s.hh[w];
            if (lane == 31) db[1] += (double)fmaf(expf(end.x) * (1.f + end.y), all, total);
            double sum = db[0] + db[1];                     // from the lane's first token on
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const double o = __shfl_down_sync(0xffffffffu, sum, d);
                if (lane + d < 32) sum += o;
            }
            const double next = __shfl_down_sync(0xffffffffu, sum, 1);
            double dg[2] = {sum, db[1] + (lane < 31 ? next : 0.0)};
            int zero = 1;
#pragma unroll
            for (int w = 0; w < DT / 32; ++w) zero = zero && s.zero[w];
            // All of db together is <h0, gradient at h0>: nothing where h0 is.  The first half of the tokens then has dg from
            // the sums before it, the very first none.
            const double whole = __shfl_sync(0xffffffffu, sum, 0);
            if (zero && lane < 16) {
                dg[0] -= whole;
                dg[1] -= whole;
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = 2 * lane + i;
                if (r < cut.n)       // (nothing passes a factor of zero)
                    p.dg[(cut.t0 + r) * p.dg_ld + h] = expf(p.g[(cut.t0 + r) * p.g_ld + h]) == 0.f ? 0.f : (float)dg[i];
            }
        }
        const float beta0 = s.beta[m0 + g], beta1 = s.beta[m0 + g + 8];
        if (SHARED) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    tq[SHARED ? n : 0][e] += dq[n][e];
                    tk[SHARED ? n : 0][e] += fmaf(e < 2 ? beta0 : beta1, x[n][e], z[n][e]);
                }
        }
        if (!SHARED || h == (kh + 1) * rep - 1) {
            __syncthreads();
            // through the lengths: d(k / |k|) = (d - k^ (k^.d)) / |k|
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int i = m0 + g + 8 * half;
                if (i >= cut.n) continue;
                const float rq = s.rq[i], rk = s.rk[i], beta = half ? beta1 : beta0;
                const float cq = p.norm ? s.dotq[i] * rq : 0.f, ck = p.norm ? s.dotk[i] * rk : 0.f;
                T* to_q = static_cast<T*>(p.dq) + (cut.t0 + i) * p.dq_ld + kh * p.Dk;
                T* to_k = static_cast<T*>(p.dk) + (cut.t0 + i) * p.dk_ld + kh * p.Dk;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const int c = n0 + 8 * n + t2;
                    const float2 qv = seq_ld2(s.q + i * LD + c), kv = seq_ld2(s.k + i * LD + c);
                    float2 a, b;
                    if (SHARED) {
                        a = make_float2(tq[SHARED ? n : 0][2 * half], tq[SHARED ? n : 0][2 * half + 1]);
                        b = make_float2(tk[SHARED ? n : 0][2 * half], tk[SHARED ? n : 0][2 * half + 1]);
                    } else {
                        a = make_float2(dq[n][2 * half], dq[n][2 * half + 1]);
                        b = make_float2(fmaf(beta, x[n][2 * half], z[n][2 * half]), fmaf(beta, x[n][2 * half + 1], z[n][2 * half + 1]));
                    }
                    store_pair(to_q + c, c, p.Dk, p.key_pairs, make_float2(rq * (a.x - qv.x * cq), rq * (a.y - qv.y * cq)));
                    store_pair(to_k + c, c, p.Dk, p.key_pairs, make_float2(rk * (b.x - kv.x * ck), rk * (b.y - kv.y * ck)));
                }
            }
        }
    }
}

template <typename T, int KP, int DVB>
cudaError_t launch_back(const SeqDeltaParams& p, cudaStream_t stream) {
    constexpr int smem = (int)sizeof(BackSmem<T, KP, DVB>);
    cudaError_t e = cudaFuncSetAttribute(delta_back_kernel<T, KP, DVB>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int dvbs = (p.Dv + DVB - 1) / DVB;
    return launch_kernel(delta_back_kernel<T, KP, DVB>, dim3((unsigned)(p.ax.S * (long long)p.Hv * dvbs)), dim3(DT), smem, stream, p.slots > 0, 1, p, dvbs);
}

template <typename T, int KP, bool SHARED>
cudaError_t launch_grad_of(const SeqDeltaParams& p, cudaStream_t stream) {
    constexpr int smem = (int)sizeof(GradSmem<T, KP>);
    cudaError_t e = cudaFuncSetAttribute(delta_grad_kernel<T, KP, SHARED>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_kernel(delta_grad_kernel<T, KP, SHARED>, dim3((unsigned)p.slots, (unsigned)p.Hk), dim3(DT), smem, stream, true, 1, p);
}
template <typename T, int KP>
cudaError_t launch_grad(const SeqDeltaParams& p, cudaStream_t stream) {
    return p.Hv > p.Hk ? launch_grad_of<T, KP, true>(p, stream) : launch_grad_of<T, KP, false>(p, stream);
}

template <typename T>
cudaError_t launch(const SeqDeltaParams& p, cudaStream_t stream) {
    const bool narrow = p.Dv <= 16 || p.ax.S * (long long)p.Hv * ((p.Dv + 31) / 32) < p.sms;
    cudaError_t e;
    if (p.planes) e = launch_seq_delta_back_tc(p, stream);
    else if (p.Dk <= 64) e = narrow ? launch_back<T, 64, 16>(p, stream) : launch_back<T, 64, 32>(p, stream);
    else e = narrow ? launch_back<T, 128, 16>(p, stream) : launch_back<T, 128, 32>(p, stream);
    if (e != cudaSuccess || p.slots == 0) return e;
    if (p.planes) return launch_seq_delta_grad_tc(p, stream);
    return p.Dk <= 64 ? launch_grad<T, 64>(p, stream) : launch_grad<T, 128>(p, stream);
}

}  // namespace

cudaError_t launch_seq_delta_bwd(const SeqDeltaParams& args, bool bf16, cudaStream_t stream) {
    SeqDeltaParams p = args;
    p.planes = bf16 && p.wide && p.compact && p.Dv > 16 ? 2 : 0;
    const cudaError_t e = launch_seq_delta_chunks(p, bf16, stream);
    if (e != cudaSuccess) return e;
    return bf16 ? launch<__nv_bfloat16>(p, stream) : launch<float>(p, stream);
}

}  // namespace convfwd

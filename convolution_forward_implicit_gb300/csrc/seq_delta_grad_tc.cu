// Gated delta rule in bf16 backward, every chunk by itself, on tcgen05 tensor cores: see seq_delta_bwd.cu for the
// formulas.  A CTA takes a chunk and a key head, its value heads in turn, and 64 columns of their states at a time.  Rows of
// the chunk are TMEM lanes, those of dY (and dQ) the first 64, those of dR, U (and X, Z) the others:
//   D1 = [dY; dR] h0^T     D2 = [dY; dR] U^T     D3 = [.; U] dh^T            over all columns, then with
//   P = E . dY U^T, S = -E . dR U^T (from D2), both below the diagonal:
//   D4 = [P |k|^-1; S |k|^-1] K                  D5 = [.; (P |q|^-1)^T Q + (S beta |k|^-1)^T K]
// and dQ = scale exp(b) D1 + scale D4, X = D4 - exp(b) D1, Z = exp(b_C - b) D3 + D5 in the rows of a lane, to which P's diagonal adds
// its multiples of k and q once the products for the decay's gradient are taken.  Operands that
// are not exact in bf16 are three bf16 parts each (24 bits), written by the threads; products of two such take the six
// large ones of the parts' nine.
//
// What bounds it: one CTA is on an SM (210 KB of shared memory and all of TMEM), and its stages follow one another.  8192 tokens, 32 value
// heads on 16 key heads of 128 x 128 take about 550 us (578 by itself): 13.5 CTAs an SM of two value heads each, at 78000 cycles, of which the
// products take 21000, and the bytes (580 KB) would take 25000; the rest are splits, factors and row sums by 16 warps that wait for
// one another.  A 17th warp that issues leaves 96 registers a thread instead of 128: the whole call took 1246 us with what spilled,
// 1194 without it; products issued by three different warps made it 1187.
#include "seq_delta.cuh"
#include "seq_delta_tc.cuh"

namespace convfwd {
namespace {

constexpr int GT_WARPS = 16, GW = 32 * GT_WARPS;      // four warps a quarter of the lanes; the first also issues

template <int KP>
struct GradTc {
    static constexpr uint32_t KQ = KP / 64 * ATOM;                    // [K; Q], 64 columns an atom
    static constexpr uint32_t A = KQ, U = A + 3 * ATOM, H = U + 3 * 8192, DH = H + 3 * ATOM;
    static constexpr uint32_t M0 = H, M1 = DH, M3 = DH + 3 * 8192;    // the chunk's matrices, where the states were
    static constexpr uint32_t REST = DH + 3 * ATOM;
    static constexpr uint32_t BYTES = REST + 8192 + 1024;
    static constexpr uint32_t D1 = 0, D3 = 128, D4 = 256, D5 = 384, D2 = 384;      // TMEM columns
};
struct GradRest {
    float2 b[DC];
    float rq[DC], rk[DC], beta[DC], g[DC], vdr[DC], own[DC];
    float dots[5][4][DC];            // q.dQ, k.X, k.Z, k.(exp(b_C - b) U dh^T), q.k: by the four warps of a row
    float hh[GT_WARPS];
    int zero[GT_WARPS];
    alignas(8) uint64_t bars[4];
    uint32_t slot;
    int abort;
};

// 8 values to three parts of 16 bytes at `to`, `plane` bytes apart.
__device__ __forceinline__ void split8(uint8_t* to, uint32_t plane, const float (&x)[8]) {
    float r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = x[i];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = bf2_pack(r[2 * i], r[2 * i + 1]);
            if (k < 2) {
                float a, b;
                bf2_unpack(w[i], a, b);
                r[2 * i] -= a;
                r[2 * i + 1] -= b;
            }
        }
        *reinterpret_cast<uint4*>(to + k * plane) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}
__device__ __forceinline__ void floats8(const float* from, bool first, bool second, float (&x)[8]) {
    const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
    const float4 a = first ? *reinterpret_cast<const float4*>(from) : z, b = second ? *reinterpret_cast<const float4*>(from + 4) : z;
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
// 8 bf16 of a row from column c of `width` on; wide: whole aligned groups
__device__ __forceinline__ uint4 row8(const __nv_bfloat16* from, int c, int width, bool there, bool wide) {
    uint32_t w[4] = {0, 0, 0, 0};
    if (there) {
        if (wide) {
            if (c < width) return *reinterpret_cast<const uint4*>(from);
        } else {
            const uint16_t* h = reinterpret_cast<const uint16_t*>(from);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c + i < width) w[i / 2] |= (uint32_t)h[i] << (i % 2 * 16);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void meet() { asm volatile("bar.sync 1, %0;" ::"n"(GW) : "memory"); }      // all warps

// A from shared memory too
__device__ __forceinline__ void mma_ss_k4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate, uint32_t astep, uint32_t bstep) {
#pragma unroll
    for (int k = 0; k < 4; ++k) mma_bf16(d, a + k * (astep >> 4), b + k * (bstep >> 4), idesc, accumulate || k > 0 ? 1u : 0u);
}
template <int N>
__device__ __forceinline__ void lanes_of(uint32_t at, uint32_t (&v)[N]) {       // N columns of the warp's lanes
    if constexpr (N == 16)
        tmem_ld16(at, v);
    else
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                     : "r"(at));
}
// the products of parts that carry 24 bits: (2, 0), (0, 2), (1, 1), (1, 0), (0, 1), (0, 0)
__device__ __forceinline__ int part_a(int q) { return 0x052 >> 2 * q & 3; }
__device__ __forceinline__ int part_b(int q) { return 0x118 >> 2 * q & 3; }

template <int KP, bool SHARED>
__global__ void __launch_bounds__(GW, 1) delta_grad_tc_kernel(const __grid_constant__ SeqDeltaParams p, unsigned* err) {
    extern __shared__ uint8_t smem_raw[];
    using G = GradTc<KP>;
    using T = __nv_bfloat16;
    constexpr int HC = KP / 4;                   // columns of a row that a thread holds of a result
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t* sm = smem_raw + (base - smem_u32(smem_raw));
    GradRest& s = *reinterpret_cast<GradRest*>(sm + G::REST);
    const CutPiece cut = cut_piece(p.ax, blockIdx.x, DC);
    if (cut.n <= 0) {
        dep_wait();                              // (what follows in the stream then follows the walk before it, too)
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, wq = warp & 3, cq = warp >> 2;
    const int kh = blockIdx.y, rep = SHARED ? p.Hv / p.Hk : 1, blocks = (p.Dv + 63) / 64;
    // Two barriers say what is ready, the states' D3 by its own: a warp goes on from one telling to the other without a wait between,
    // and would else be counted in place of one that has not told the first yet.
    const uint32_t ready = smem_u32(&s.bars[0]), ready_dh = smem_u32(&s.bars[3]), bar_h = smem_u32(&s.bars[1]), bar_e = smem_u32(&s.bars[2]);
    volatile int* abort_flag = &s.abort;
    if (threadIdx.x == 0) {
        mbar_init(ready, GT_WARPS);
        mbar_init(ready_dh, GT_WARPS);
        mbar_init(bar_h, 1);
        mbar_init(bar_e, 1);
        s.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) {
        tmem_alloc(smem_u32(&s.slot), 512);
        tmem_relinquish();
    }
    {
        load_kq<KP, GW>(base, static_cast<const T*>(p.k) + cut.t0 * p.k_ld + kh * p.Dk, static_cast<const T*>(p.q) + cut.t0 * p.q_ld + kh * p.Dk, p.k_ld,
                        p.q_ld, cut.n, p.Dk, threadIdx.x);
        cp_async_commit();                       // (waited for where the first head's matrices are)
        for (int i = threadIdx.x; i < 2 * 8192 / 16; i += GW)      // dY is one part: its others are zero
            *reinterpret_cast<uint4*>(sm + G::A + (1 + i / 512) * ATOM + i % 512 * 16) = make_uint4(0, 0, 0, 0);
    }
    dep_wait();
    // A thread's pieces of 8 columns: row r8 of the tokens, rows r8 and r8 + 64 of the states.  What a block needs
    // is on its way while the one before is worked on, in registers: with loads where they are used the call took 1470 us instead of 1391 (8192 tokens, 32 heads).
    const int r8 = threadIdx.x >> 3, c8 = threadIdx.x & 7;
    const uint32_t place = (uint32_t)(r8 * 128 + (c8 ^ (r8 & 7)) * 16);
    float h0[KP / 64][8], u[8], dr[8];
    uint4 dy, vv;
    auto states = [&](const float* from, int h, int v, float (&x)[KP / 64][8]) {
        const long long at = (long long)blockIdx.x * p.Hv + h;
        const int col = v * 64 + c8 * 8;
#pragma unroll
        for (int j = 0; j < KP / 64; ++j) {
            const int r = r8 + 64 * j;
            floats8(from + (at * p.Dk + r) * p.Dvp + col, col < p.Dvp && r < p.Dk, col + 4 < p.Dvp && r < p.Dk, x[j]);
        }
    };
    auto tokens = [&](int h, int v) {
        const long long at = (long long)blockIdx.x * p.Hv + h;
        const int col = v * 64 + c8 * 8;
        const bool first = col < p.Dvp, second = col + 4 < p.Dvp;
        floats8(p.saved + p.saved_u + (at * DC + r8) * p.Dvp + col, first, second, u);
        floats8(p.dr + (at * DC + r8) * p.Dvp + col, first, second, dr);
        dy = row8(static_cast<const T*>(p.dy) + (cut.t0 + r8) * p.dy_ld + h * p.Dv + col, col, p.Dv, r8 < cut.n, p.val_wide);
        vv = row8(static_cast<const T*>(p.v) + (cut.t0 + r8) * p.v_ld + h * p.Dv + col, col, p.Dv, r8 < cut.n, p.val_wide);
    };
    states(p.saved, kh * rep, 0, h0);
    tokens(kh * rep, 0);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s.slot, lanes = tmem + ((uint32_t)(wq * 32) << 16);
    constexpr uint32_t B_ACROSS = 1u << 16, A_ACROSS = 1u << 15, ID_KP = idesc_f32acc(128, KP, 1u), ID_64 = idesc_f32acc(128, 64, 1u);
    // After a wait has run out every later one ends at once (see wait_turn); the warps go on together to the end.
    {
        // what the first warp issues once all have told: D2 and D1 of a block, its D3, or D4 and D5
        enum Part { ROWS, STATES, MATRICES };
        uint32_t turn = 0, turn_dh = 0;
        auto issue = [&](Part part, bool first) {
            if (warp != 0) return;
            const bool ok = part == STATES ? wait_turn(ready_dh, turn_dh, abort_flag, err) : wait_turn(ready, turn, abort_flag, err);
            (part == STATES ? turn_dh : turn) ^= 1;
            tc_fence_after();
            if (ok && lane == 0 && !(p.test_stall && part == MATRICES)) {      // (test hook: the wait for them runs out)
                if (part == ROWS) {
#pragma unroll 1
                    for (int q = 0; q < 6; ++q)
                        mma_ss_k4(tmem + G::D2, sw128_desc(base + G::A + part_a(q) * ATOM), sw128_desc(base + G::U + part_b(q) * 8192), ID_64, !first || q > 0, 32, 32);
#pragma unroll 1
                    for (int q = 0; q < 6; ++q)
                        mma_ss_k4(tmem + G::D1, sw128_desc(base + G::A + part_a(q) * ATOM), sw128_desc(base + G::H + part_b(q) * ATOM), ID_KP, !first || q > 0, 32, 32);
                    mma_commit(bar_h);
                } else if (part == STATES) {
#pragma unroll 1
                    for (int q = 0; q < 6; ++q)      // (U's rows are the second 64: the first are whatever lies before it)
                        mma_ss_k4(tmem + G::D3, sw128_desc(base + G::U + part_a(q) * 8192 - 8192), sw128_desc(base + G::DH + part_b(q) * ATOM), ID_KP,
                                  !first || q > 0, 32, 32);
                    mma_commit(bar_e);
                } else {
#pragma unroll 1
                    for (int pl = 2; pl >= 0; --pl)
                        mma_ss_k4(tmem + G::D4, sw128_desc(base + G::M0 + pl * ATOM), mn_desc(base, ATOM), ID_KP | B_ACROSS, pl < 2, 32, 2048);
#pragma unroll 1
                    for (int pl = 2; pl >= 0; --pl) {    // (blocks of rows 8 KB apart, the matrix the second)
                        mma_ss_k4(tmem + G::D5, mn_desc(base + G::M1 + pl * 8192 - 8192, 8192), mn_desc(base + 8192, ATOM), ID_KP | A_ACROSS | B_ACROSS, pl < 2, 2048, 2048);
                        mma_ss_k4(tmem + G::D5, mn_desc(base + G::M3 + pl * 8192 - 8192, 8192), mn_desc(base, ATOM), ID_KP | A_ACROSS | B_ACROSS, true, 2048, 2048);
                    }
                    mma_commit(bar_e);
                }
            }
            __syncwarp();
        };
        uint32_t turn_h = 0, turn_e = 0;
        auto wait_h = [&]() {
            wait_turn(bar_h, turn_h, abort_flag, err);
            turn_h ^= 1;
            tc_fence_after();
        };
        auto wait_e = [&]() {
            wait_turn(bar_e, turn_e, abort_flag, err);
            turn_e ^= 1;
            tc_fence_after();
        };
        auto tell = [&](uint32_t bar) {
            fence_proxy_async();
            tc_fence_before();
            __syncwarp();
            arrive_once(bar);
        };
        // the row of K (second 64 lanes) or Q that the lane holds: 16-byte pieces of the swizzled atoms
        const int i = (wq & 1) * 32 + lane, isk = wq >> 1;
        auto piece = [&](int row, int c) {       // columns 8 c .. of row (K: 0 .. 63, Q: 64 .. 127)
            return *reinterpret_cast<const uint4*>(sm + (c >> 3) * ATOM + row * 128 + ((c & 7) ^ (row & 7)) * 16);
        };
        float along = 0.f;                       // <row of q or k, its gradient>
        float total[SHARED ? HC : 1];
#pragma unroll
        for (int c = 0; c < (SHARED ? HC : 1); ++c) total[c] = 0.f;
        for (int h = kh * rep; h < (kh + 1) * rep; ++h) {
            if (threadIdx.x >= GW - DC) {        // (read behind the meeting below)
                const int r = threadIdx.x - (GW - DC);
                const float* rows = p.rows + ((long long)blockIdx.x * p.Hv + h) * DELTA_ROWS;
                s.b[r] = *reinterpret_cast<const float2*>(rows + RF_B + 2 * r);
                s.rq[r] = rows[RF_RQ + r];
                s.rk[r] = rows[RF_RK + r];
                s.beta[r] = rows[RF_BETA + r];
                s.g[r] = r < cut.n ? p.g[(cut.t0 + r) * p.g_ld + h] : 0.f;
            }
            float vdr = 0.f, hh = 0.f;
            bool from_zero = true;               // the state before the chunk is zero
            for (int v = 0; v < blocks; ++v) {
                const bool more = v + 1 < blocks || h + 1 < (kh + 1) * rep;
                const int h_next = v + 1 < blocks ? h : h + 1, v_next = v + 1 < blocks ? v + 1 : 0;
                if (v > 0) wait_h();                 // the block before has read its h0
#pragma unroll
                for (int j = 0; j < KP / 64; ++j) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) from_zero = from_zero && h0[j][e] == 0.f;
                    split8(sm + G::H + place + j * 8192, ATOM, h0[j]);
                }
                float dh[KP / 64][8];
                states(p.dstate, h, v, dh);
                if (v > 0) wait_e();                 // and all else
                split8(sm + G::U + place, 8192, u);
                split8(sm + G::A + 8192 + place, ATOM, dr);
                *reinterpret_cast<uint4*>(sm + G::A + place) = dy;
                const uint32_t w[4] = {vv.x, vv.y, vv.z, vv.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float a, b;
                    bf2_unpack(w[e], a, b);
                    vdr = fmaf(a, dr[2 * e], fmaf(b, dr[2 * e + 1], vdr));
                }
                tell(ready);
                if (more) tokens(h_next, v_next);
                issue(ROWS, v == 0);
#pragma unroll
                for (int j = 0; j < KP / 64; ++j) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) hh = fmaf(h0[j][e], dh[j][e], hh);
                    split8(sm + G::DH + place + j * 8192, ATOM, dh[j]);
                }
                tell(ready_dh);
                if (more) states(p.saved, h_next, v_next, h0);
                issue(STATES, v == 0);
            }
#pragma unroll
            for (int d = 1; d < 8; d <<= 1) vdr += __shfl_xor_sync(0xffffffffu, vdr, d);
            if (c8 == 0) s.vdr[r8] = vdr;
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) hh += __shfl_xor_sync(0xffffffffu, hh, d);
            from_zero = __all_sync(0xffffffffu, from_zero);
            if (lane == 0) {
                s.hh[warp] = hh;
                s.zero[warp] = from_zero;
            }
            cp_async_wait<0>();                  // K and Q: told with the matrices
            meet();
            const float2 bi = s.b[i], end = s.b[DC - 1];
            const float rqi = s.rq[i], rki = s.rk[i], beta = s.beta[i];
            wait_h();
            wait_e();
            // ---- the chunk's matrices from D2: 16 columns of the lane's row
            {
                uint32_t d[16];
                tmem_ld16(lanes + G::D2 + cq * 16, d);
                tmem_ld_wait();
                const float f = isk ? -1.f : p.scale, own = isk ? beta * rki : rqi;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    float by_key[8], by_row[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int j = cq * 16 + half * 8 + e;
                        const float x = j < i ? f * __uint_as_float(d[half * 8 + e]) * decay_between(bi, s.b[j]) : 0.f;
                        if (j == i && !isk) s.own[i] = f * __uint_as_float(d[half * 8 + e]);
                        by_key[e] = x * s.rk[j];
                        by_row[e] = x * own;
                    }
                    const int chunk = cq * 2 + half;
                    split8(sm + G::M0 + (isk * 64 + i) * 128 + ((chunk ^ (i & 7)) * 16), ATOM, by_key);
                    split8(sm + (isk ? G::M3 : G::M1) + i * 128 + ((chunk ^ (i & 7)) * 16), 8192, by_row);
                }
            }
            tell(ready);
            issue(MATRICES, true);
            meet();                              // (P's diagonal is there)
            const float eb = expf(bi.x) * (1.f + bi.y), fq = p.scale * eb, fz = decay_between(end, bi);
            wait_e();
            const float own_f = s.own[i] * (isk ? rqi : rki);
            // ---- rows: dQ (first 64 lanes), X and Z (the others), in pieces of columns (with 16 and the sums of heads registers spill)
            constexpr int PIECE = SHARED ? 8 : 16;
            float dot[3][4] = {};                // (four sums each: their differences make dg)
            float out[SHARED ? 1 : HC];
#pragma unroll
            for (int c = 0; c < HC; c += PIECE) {
                const int col = cq * HC + c;
                uint32_t d1[PIECE], d4[PIECE], d3[PIECE], d5[PIECE];
                lanes_of(lanes + G::D1 + col, d1);
                lanes_of(lanes + G::D4 + col, d4);
                lanes_of(lanes + G::D3 + col, d3);
                lanes_of(lanes + G::D5 + col, d5);
                const int row = isk ? i : 64 + i;
                uint32_t w[PIECE / 2], o[PIECE / 2];        // the token's k (or q), and its q (or k)
#pragma unroll
                for (int e = 0; e < PIECE; e += 8) {
                    const uint4 k = piece(row, (col + e) / 8), q = piece(row ^ 64, (col + e) / 8);
                    w[e / 2] = k.x; w[e / 2 + 1] = k.y; w[e / 2 + 2] = k.z; w[e / 2 + 3] = k.w;
                    o[e / 2] = q.x; o[e / 2 + 1] = q.y; o[e / 2 + 2] = q.z; o[e / 2 + 3] = q.w;
                }
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < PIECE; ++e) {
                    float lo, hi;
                    bf2_unpack(w[e / 2], lo, hi);
                    const float own = e & 1 ? hi : lo;
                    bf2_unpack(o[e / 2], lo, hi);
                    const float other = e & 1 ? hi : lo;
                    float r;
                    if (!isk) {
                        r = fmaf(fq, __uint_as_float(d1[e]), __uint_as_float(d4[e]));
                        dot[0][e & 3] = fmaf(own, r, dot[0][e & 3]);
                        dot[1][e & 3] = fmaf(own, other, dot[1][e & 3]);
                    } else {
                        const float x = fmaf(-eb, __uint_as_float(d1[e]), __uint_as_float(d4[e])), zu = fz * __uint_as_float(d3[e]);
                        const float z = zu + __uint_as_float(d5[e]);
                        dot[0][e & 3] = fmaf(own, x, dot[0][e & 3]);
                        dot[1][e & 3] = fmaf(own, z, dot[1][e & 3]);
                        dot[2][e & 3] = fmaf(own, zu, dot[2][e & 3]);
                        r = fmaf(beta, x, z);
                    }
                    r = fmaf(own_f, other, r);
                    if (SHARED) total[SHARED ? c + e : 0] += r;
                    else out[SHARED ? 0 : c + e] = r;
                }
            }
            if (!isk) {
                s.dots[0][cq][i] = (dot[0][0] + dot[0][1]) + (dot[0][2] + dot[0][3]);
                s.dots[4][cq][i] = (dot[1][0] + dot[1][1]) + (dot[1][2] + dot[1][3]);
            } else {
#pragma unroll
                for (int k = 0; k < 3; ++k) s.dots[1 + k][cq][i] = (dot[k][0] + dot[k][1]) + (dot[k][2] + dot[k][3]);
            }
            meet();
            auto of = [&](int k, int r) { return (s.dots[k][0][r] + s.dots[k][1][r]) + (s.dots[k][2][r] + s.dots[k][3][r]); };
            along += s.own[i] * rqi * rki * of(4, i) + (isk ? fmaf(beta, rki * of(1, i), rki * of(2, i)) : rqi * of(0, i));
            if (!SHARED || h == (kh + 1) * rep - 1) {
                // through the lengths: d(k / |k|) = (d - k^ (k^.d)) / |k|; through shared memory, for whole rows: written by
                // the lanes that hold them, 4 KB apart, they took 180 us of the call's 1390 (8192 tokens, 32 heads)
                {
                    const float r = isk ? rki : rqi, f = p.norm ? along * r : 0.f;
                    const int row = isk ? i : 64 + i;
#pragma unroll
                    for (int c = 0; c < HC; c += 8) {
                        const int col = cq * HC + c;
                        const uint4 q = piece(row, col / 8);
                        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
                        uint32_t o[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float lo, hi;
                            bf2_unpack(w[e], lo, hi);
                            const float v0 = SHARED ? total[SHARED ? c + 2 * e : 0] : out[SHARED ? 0 : c + 2 * e];
                            const float v1 = SHARED ? total[SHARED ? c + 2 * e + 1 : 0] : out[SHARED ? 0 : c + 2 * e + 1];
                            o[e] = bf2_pack(r * (v0 - lo * f), r * (v1 - hi * f));
                        }
                        // (16-byte pieces of a row turned by its number, so that neither side's accesses meet in a bank)
                        *reinterpret_cast<uint4*>(sm + G::H + (row * (KP / 8) + ((col / 8) ^ (row & 7))) * 16) = make_uint4(o[0], o[1], o[2], o[3]);
                    }
                }
                meet();
                for (int j = threadIdx.x; j < 128 * (KP / 8); j += GW) {
                    const int row = j / (KP / 8), c = j % (KP / 8) * 8, t = row & 63;
                    if (t >= cut.n || c >= p.Dk) continue;
                    const uint4 q = *reinterpret_cast<const uint4*>(sm + G::H + (row * (KP / 8) + ((c / 8) ^ (row & 7))) * 16);
                    T* to = (row < 64 ? static_cast<T*>(p.dk) + (cut.t0 + t) * p.dk_ld : static_cast<T*>(p.dq) + (cut.t0 + t) * p.dq_ld) + kh * p.Dk + c;
                    if (p.key_wide) {
                        *reinterpret_cast<uint4*>(to) = q;
                    } else {
                        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (c + e < p.Dk) reinterpret_cast<uint16_t*>(to)[e] = (uint16_t)(w[e / 2] >> (e % 2 * 16));
                    }
                }
            }
            if (warp == GT_WARPS - 1) {                  // dbeta and dg, two tokens a lane
                float all = 0.f, sum3 = 0.f;
                double db[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = 2 * lane + e;
                    const float rq = s.rq[r], rk = s.rk[r], be = s.beta[r];
                    const float qq = rq * (of(0, r)), kx = rk * (of(1, r));
                    const bool last = r == cut.n - 1;        // (see seq_delta_bwd.cu: without what stands in both sums)
                    const float kz = last ? 0.f : rk * (of(2, r));
                    sum3 += last ? 0.f : rk * (of(3, r));
                    db[e] = (double)(qq - kz) + (double)(be * kx);
                    if (r < cut.n) p.dbeta[(cut.t0 + r) * p.dbeta_ld + h] = s.vdr[r] + kx;
                }
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) sum3 += __shfl_xor_sync(0xffffffffu, sum3, d);
#pragma unroll
                for (int w = 0; w < GT_WARPS; ++w) all += s.hh[w];
                if (lane == 31) db[1] += (double)fmaf(expf(end.x) * (1.f + end.y), all, sum3);
                double sum = db[0] + db[1];      // from the lane's first token on
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const double o = __shfl_down_sync(0xffffffffu, sum, d);
                    if (lane + d < 32) sum += o;
                }
                const double after = __shfl_down_sync(0xffffffffu, sum, 1);
                double dg[2] = {sum, db[1] + (lane < 31 ? after : 0.0)};
                int zero = 1;
#pragma unroll
                for (int w = 0; w < GT_WARPS; ++w) zero = zero && s.zero[w];
                // All of db together is <h0, gradient at h0>: nothing where h0 is.  The first half of the tokens then has dg from
                // the sums before it, the very first none.
                const double whole = __shfl_sync(0xffffffffu, sum, 0);
                if (zero && lane < 16) {
                    dg[0] -= whole;
                    dg[1] -= whole;
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = 2 * lane + e;
                    if (r < cut.n)               // (nothing passes a factor of zero)
                        p.dg[(cut.t0 + r) * p.dg_ld + h] = expf(s.g[r]) == 0.f ? 0.f : (float)dg[e];
                }
            }
            meet();                              // (the next head's sums go where these were read)
        }
    }
    if (s.abort && threadIdx.x == 0) {           // products that may still run: bounded, before TMEM goes
        const long long since = clock64();
        while (clock64() - since < WAIT_CYCLES / 8) {
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int KP, bool SHARED>
cudaError_t launch_of(const SeqDeltaParams& p, unsigned* err, cudaStream_t stream) {
    const auto kernel = delta_grad_tc_kernel<KP, SHARED>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)GradTc<KP>::BYTES);
    if (e != cudaSuccess) return e;
    return launch_kernel(kernel, dim3((unsigned)p.slots, (unsigned)p.Hk), dim3(GW), GradTc<KP>::BYTES, stream, true, 1, p, err);
}

}  // namespace

cudaError_t launch_seq_delta_grad_tc(const SeqDeltaParams& p, cudaStream_t stream) {
    static_assert(sizeof(GradRest) <= 8192, "room behind the operands");
    unsigned* err = device_error_word();
    if (!err) return cudaErrorUnknown;
    const bool shared = p.Hv > p.Hk;
    if (p.Dk <= 64) return shared ? launch_of<64, true>(p, err, stream) : launch_of<64, false>(p, err, stream);
    return shared ? launch_of<128, true>(p, err, stream) : launch_of<128, false>(p, err, stream);
}

}  // namespace convfwd

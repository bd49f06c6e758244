// Gated delta rule in bf16, the walks over the chunks of a sequence on tcgen05 tensor cores: see seq_delta.cuh for the
// formulas.  A CTA has 128 columns of the state of a sequence and value head, and works on everything transposed, so that
// the state's columns are the 128 rows (TMEM lanes) of every product:
//   forward   [h0^T K^T | h0^T Q^T], [R^T T^T | R^T (A T)^T], U'^T K
// The left operands lie in TMEM, written there by the threads that hold a lane: they hold the state in fp32 registers,
// split what the next product needs into three bf16 parts (24 bits of an fp32 value) and write those.  K and Q are exact
// in bf16, so three products take part with them, six with T (its parts come from the chunk kernel): fp32 accuracy
// at a third or a sixth of the bf16 rate.  The right operands lie in shared memory, for two chunks: while one is worked
// on, the next one's are on their way.
//
// What bounds a walk: the products and the threads' work between them follow one another, three times a chunk.  2048 tokens of 16 heads
// of 128 x 128 (16 CTAs, 32 chunks in order) take 143 us: 4.5 us a chunk, of which the products are 2 (60 of 64 cycles);
// in five pieces of the axis 37, 22 to join them and 42.
// 8192 tokens, 32 heads, 4 sequences (128 CTAs) take 194 us, backward 201, where the kernel moves 760 MB, most of it what is saved
// (57% of copy rate); with mma.sync they took 814 and 776.
#include "seq_delta.cuh"
#include "seq_delta_tc.cuh"

namespace convfwd {
namespace {

constexpr int WT = 512;                       // threads that hold lanes: four warps a quarter of the lanes, a quarter of the columns each
constexpr int TPT = 64 * 128 / WT;            // tokens of a chunk a thread holds of its lane
constexpr int LOADERS = 3;                    // warps behind the first, issuing, one that fetch
constexpr int WALK_THREADS = WT + 32 * (1 + LOADERS);
constexpr uint32_t PLANES = 3 * ATOM;         // [T; A T] (backward: [T; A]) in three parts

// D += A B for 64 of k, A in TMEM (a lane's 16 bf16 of a step in 8 columns), issued by the calling thread: four steps in one
// block, B's address BSTEP bytes further each (4 steps one by one took about 100 cycles each to issue).
template <int BSTEP>
__device__ __forceinline__ void mma_ts_k4(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, t;\n\t.reg .b64 b1, b2, b3;\n\t.reg .b32 a1, a2, a3;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
        "add.s64 b1, %2, %5;\n\tadd.s64 b2, %2, %6;\n\tadd.s64 b3, %2, %7;\n\t"
        "add.s32 a1, %1, 8;\n\tadd.s32 a2, %1, 16;\n\tadd.s32 a3, %1, 24;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, t;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, t;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, t;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate), "n"(BSTEP >> 4), "n"(2 * BSTEP >> 4), "n"(3 * BSTEP >> 4)
        : "memory");
}
// N steps of 16 along k: A's columns follow one another; B's lie side by side (64 of them, 128 bytes, an atom) or, ACROSS, in rows.
template <int N, bool ACROSS_ROWS>
__device__ __forceinline__ void steps(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate) {
#pragma unroll
    for (int k = 0; k < N; k += 4) mma_ts_k4<ACROSS_ROWS ? 2048 : 32>(d, a + k * 8, b + (ACROSS_ROWS ? k * (2048 >> 4) : k / 4 * (ATOM >> 4)), idesc, accumulate || k > 0);
}
__device__ __forceinline__ void tmem_st8(uint32_t at, const uint32_t (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 16 values in three bf16 parts to 8 columns each of three planes `stride` columns apart.
__device__ __forceinline__ void put_parts(uint32_t at, uint32_t stride, const float (&x)[16]) {
    uint32_t part[3][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float a = x[2 * i], b = x[2 * i + 1];
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            part[k][i] = pack_bf16x2(a, b);
            if (k < 2) {
                float ha, hb;
                bf2_unpack(part[k][i], ha, hb);
                a -= ha;
                b -= hb;
            }
        }
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) tmem_st8(at + k * stride, part[k]);
}

// 16 row factors from shared memory.
__device__ __forceinline__ void read16(const float* from, float (&v)[16]) {
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
        const float4 q = *reinterpret_cast<const float4*>(from + i);
        v[i] = q.x; v[i + 1] = q.y; v[i + 2] = q.z; v[i + 3] = q.w;
    }
}

template <int KP>
struct WalkTc {
    static constexpr uint32_t KQ = KP / 64 * ATOM;                       // [K; Q], 64 columns an atom
    static constexpr uint32_t STAGE = KQ + PLANES + 2048;                // and the row factors
    static constexpr uint32_t BYTES = 2 * STAGE + 1024 + 128;
    static constexpr uint32_t H = 0, P = 3 * KP / 2, ACC = P + 96;       // TMEM columns
};

// The barriers of a walk's CTA, every wait bounded.  The threads that hold lanes (16 warps) tell the issuing warp when its
// operands are ready, and learn from `mma` when its products are done; `full`: a stage's operands have arrived, `empty`:
// it may be written again.
struct Turns {
    uint32_t mma, ready, full, empty;         // shared addresses (full, empty: two)
    uint32_t phase;                   // of mma (the issuing warp: of ready)
    volatile int* abort_flag;
    unsigned* err;
    __device__ __forceinline__ bool next(uint32_t bar) {
        const bool ok = wait_turn(bar, phase, abort_flag, err);
        phase ^= 1;
        tc_fence_after();
        return ok;
    }
    // what this warp wrote to TMEM (and shared memory) is there
    __device__ __forceinline__ void tell() {
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        arrive_once(ready);
    }
    __device__ __forceinline__ void release(int n) const {       // this warp has read the stage for the last time
        __syncwarp();
        arrive_once(empty + 8 * (n & 1));
    }
    __device__ __forceinline__ bool free(int n) { return n < 2 || wait_turn(empty + 8 * (n & 1), ((n >> 1) & 1) ^ 1, abort_flag, err); }
    __device__ __forceinline__ bool arrived(int n) { return wait_turn(full + 8 * (n & 1), (n >> 1) & 1, abort_flag, err); }
    // The issuing threads' last: the copies of the `sent` stages begun (the last two of them), the products committed so far.
    __device__ __forceinline__ void settle_copies(int sent) const {
        for (int n = sent > 2 ? sent - 2 : 0; n < sent; ++n) settle(full + 8 * (n & 1), (n >> 1) & 1);
    }
    __device__ __forceinline__ void settle_products(int committed) const {
        if (committed > 0) settle(mma, (committed - 1) & 1);
    }
};

// The start of a walk's CTA: its place, barriers, TMEM.
template <int KP>
struct Walk {
    uint32_t base, tmem, lanes;
    uint8_t* smem;
    int warp, lane, cq, tok, h, seq, kh, dv, t0, t1, chunks, slot0;
    bool on;
    long long row, state;
    Turns turn;
    __device__ __forceinline__ Walk(const SeqDeltaParams& p, const WalkPlace& place, unsigned* err, uint8_t* raw) {
        using W = WalkTc<KP>;
        base = (smem_u32(raw) + 1023u) & ~1023u;
        smem = raw + (base - smem_u32(raw));
        const uint32_t bars = base + 2 * W::STAGE;
        uint32_t* slot = reinterpret_cast<uint32_t*>(smem + 2 * W::STAGE + 64);
        turn = {bars, bars + 24, bars + 8, bars + 32, 0, reinterpret_cast<volatile int*>(smem + 2 * W::STAGE + 72), err};
        warp = threadIdx.x >> 5;
        lane = threadIdx.x & 31;
        cq = (warp >> 2) - 1;                     // (the first four warps hold no lanes)
        tok = cq * TPT;                           // the thread's tokens of a chunk: tok .. tok + TPT - 1
        h = place.h;
        seq = place.seq;
        kh = h / (p.Hv / p.Hk);
        dv = place.dvb * 128 + (warp & 3) * 32 + lane;
        on = dv < p.Dv && warp > LOADERS && !place.unit;
        t0 = place.t0;
        t1 = place.t1;
        chunks = place.chunks;
        slot0 = place.slot0;
        row = seq_slot(p.sl, seq);
        state = (row * p.Hv + h) * (long long)p.Dk * p.Dv + dv;
        if (threadIdx.x == 0) {
            mbar_init(turn.mma, 1);
            for (int i = 0; i < 2; ++i) {
                mbar_init(turn.full + 8 * i, 1 + LOADERS);
                mbar_init(turn.empty + 8 * i, WT / 32);
            }
            mbar_init(turn.ready, WT / 32);
            *turn.abort_flag = 0;
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
        if (warp == 0) {
            tmem_alloc(smem_u32(slot), 512);
            tmem_relinquish();
        }
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        tmem = *slot;
        lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    }
    __device__ __forceinline__ long long at(const SeqDeltaParams& p, int c) const { return (long long)(slot0 + c) * p.Hv + h; }
    __device__ __forceinline__ uint32_t stage(int n) const { return base + (n & 1) * WalkTc<KP>::STAGE; }
    __device__ __forceinline__ const float* rows(int n) const {
        return reinterpret_cast<const float*>(smem + (n & 1) * WalkTc<KP>::STAGE + WalkTc<KP>::KQ + PLANES);
    }
    // The loaders' part: the operands of every chunk in order (backward: from the last), copies of whole matrices, and K and Q
    // in copies of 16 bytes.
    __device__ __forceinline__ void load(const SeqDeltaParams& p, bool backward) {
        const int thread = threadIdx.x - 32;
        int sent = 0;
        for (int i = 0; i < chunks; ++i) {
            const int c = backward ? chunks - 1 - i : i, t = t0 + c * DC;
            const uint32_t to = stage(i), bar = turn.full + 8 * (i & 1);
            if (!turn.free(i)) break;
            if (thread == 0) {
                mbar_arrive_expect_tx(bar, PLANES + DELTA_FACTORS * 4);
                bulk_g2s(to + WalkTc<KP>::KQ, reinterpret_cast<const uint8_t*>(p.tri) + at(p, c) * PLANES, PLANES, bar);
                bulk_g2s(to + WalkTc<KP>::KQ + PLANES, p.rows + at(p, c) * DELTA_ROWS, DELTA_FACTORS * 4, bar);
                sent = i + 1;
            }
            load_kq<KP, 32 * LOADERS>(to, static_cast<const __nv_bfloat16*>(p.k) + t * p.k_ld + kh * p.Dk, static_cast<const __nv_bfloat16*>(p.q) + t * p.q_ld + kh * p.Dk,
                        p.k_ld, p.q_ld, min(DC, t1 - t), p.Dk, thread);
            cp_async_commit();
            cp_async_wait<0>();
            fence_proxy_async();
            __syncwarp();
            arrive_once(bar);
        }
        if (thread == 0) turn.settle_copies(sent);
    }
    // The thread's values of a chunk's rows of v or dY, as pairs of tokens.  Where rows lie in aligned pairs (`pairs`), an even lane
    // reads its own and its neighbour's column of the first token of each two, an odd one those of the second, and they exchange.
    __device__ __forceinline__ void values(const void* from, long long ld, const SeqDeltaParams& p, int c, uint32_t (&v)[TPT / 2]) const {
        const int t = t0 + c * DC + tok, n = on ? min(DC, t1 - t0 - c * DC) - tok : 0;
        const uint16_t* at = static_cast<const uint16_t*>(from) + t * ld + h * p.Dv + dv;
        const uint32_t step = (uint32_t)ld;       // (64 rows lie within 2^31 bytes: see the caller)
        if (__all_sync(0xffffffffu, p.pairs && n >= TPT)) {
            const uint32_t odd = lane & 1;
            const uint16_t* row = at + odd * step - odd;
            uint32_t w[TPT / 2];
#pragma unroll
            for (int i = 0; i < TPT / 2; ++i) w[i] = *reinterpret_cast<const uint32_t*>(row + 2 * i * step);
#pragma unroll
            for (int i = 0; i < TPT / 2; ++i) {
                const uint32_t o = __shfl_xor_sync(0xffffffffu, w[i], 1);
                // even: the low halves (own column) of token 2i (own) and 2i + 1 (the neighbour's); odd: the high ones
                v[i] = odd ? __byte_perm(o, w[i], 0x7632) : __byte_perm(w[i], o, 0x5410);
            }
        } else {
#pragma unroll
            for (int i = 0; i < TPT / 2; ++i) {
                const uint32_t a = 2 * i < n ? at[2 * i * step] : 0, b = 2 * i + 1 < n ? at[(2 * i + 1) * step] : 0;
                v[i] = a | b << 16;
            }
        }
    }
    // 16 of the thread's values to rows first .. of a tensor whose chunk has n tokens; the same exchange.
    __device__ __forceinline__ void store(void* to, long long ld, const SeqDeltaParams& p, int t, int n, int first, const float (&x)[16]) const {
        __nv_bfloat16* at = static_cast<__nv_bfloat16*>(to) + (long long)(t + first) * ld + h * p.Dv + dv;
        const uint32_t step = (uint32_t)ld;
        if (__all_sync(0xffffffffu, p.pairs && on && n - first >= 16)) {
            const uint32_t odd = lane & 1;
            __nv_bfloat16* row = at + odd * step - odd;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t own = pack_bf16x2(x[2 * i], x[2 * i + 1]), o = __shfl_xor_sync(0xffffffffu, own, 1);
                *reinterpret_cast<uint32_t*>(row + 2 * i * step) = odd ? __byte_perm(o, own, 0x7632) : __byte_perm(own, o, 0x5410);
            }
        } else if (on) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (first + i < n) at[i * step] = __float2bfloat16_rn(x[i]);
        }
    }
    // The thread's part of a state to rows of `width` floats.
    __device__ __forceinline__ void keep(float* to, const SeqDeltaParams& p, int width, const float (&st)[KP * 128 / WT]) const {
        if (dv >= width) return;
        float* at = to + cq * (KP * 128 / WT) * width + dv;
        if (p.Dk == KP) {
#pragma unroll
            for (int i = 0; i < KP * 128 / WT; ++i) at[i * width] = st[i];
        } else {
#pragma unroll
            for (int i = 0; i < KP * 128 / WT; ++i)
                if (cq * (KP * 128 / WT) + i < p.Dk) at[i * width] = st[i];
        }
    }
    __device__ __forceinline__ void close() {
        tc_fence_before();
        __syncthreads();
        if (warp == 0) {
            tc_fence_after();
            tmem_dealloc(tmem, 512);
        }
    }
};

// The thread's rows of the state in three parts to `to`, planes KP/2 columns apart.
template <int KP>
__device__ __forceinline__ void put_state(uint32_t to, const float (&st)[KP * 128 / WT]) {
#pragma unroll
    for (int i = 0; i < KP * 128 / WT; i += 16) {
        float x[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = st[i + e];
        put_parts(to + i / 2, KP / 2, x);
    }
}
// st <- decay st + the products' sums
template <int KP>
__device__ __forceinline__ void next_state(uint32_t from, float decay, float (&st)[KP * 128 / WT]) {
#pragma unroll
    for (int i = 0; i < KP * 128 / WT; i += 16) {
        uint32_t a[16];
        tmem_ld16(from + i, a);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 16; ++e) st[i + e] = fmaf(decay, st[i + e], __uint_as_float(a[e]));
    }
}

template <int KP, int MODE>
__global__ void __launch_bounds__(WALK_THREADS, 1) delta_walk_tc_kernel(const __grid_constant__ SeqDeltaParams p, int dvbs, int dkbs, unsigned* err) {
    extern __shared__ uint8_t smem_raw[];
    using W = WalkTc<KP>;
    using T = __nv_bfloat16;
    constexpr int HK = KP * 128 / WT;                  // the thread's rows of the state: cq HK ..
    constexpr bool Y = MODE != DELTA_PIECES;           // outputs too
    constexpr uint32_t ID_ROWS = idesc_f32acc(128, Y ? 128 : 64, 1u), ID_KP = idesc_f32acc(128, KP, 1u) | (1u << 16);
    const WalkPlace place = walk_place<MODE>(p, dvbs, dkbs);
    if (MODE != DELTA_WHOLE) dep_wait();
    if (place.none) return;
    Walk<KP> w(p, place, err, smem_raw);
    const long long kept = ((long long)place.mark * p.Hv + place.h) * p.Dk;        // rows of what is kept by piece
    const float* from = MODE == DELTA_JOINED && !(place.first && place.last) ? (place.first ? p.added : p.left) + kept * p.Dvp : nullptr;
    if (w.warp > 0 && w.warp <= LOADERS) {
        dep_wait();
        w.load(p, false);
    } else if (w.warp == 0) {                   // the issuing warp (the first: the oldest is served first)
        bool ok = true;
        int committed = 0;
        for (int c = 0; c < w.chunks && ok; ++c) {
            if (p.test_stall && c == 1) break;       // (test hook: the other warps' wait runs out)
            const uint32_t kq = w.stage(c), tp = kq + W::KQ, acc = w.tmem + W::ACC;
            ok = w.turn.arrived(c) && w.turn.next(w.turn.ready);
            if (!ok) break;
            if (w.lane == 0) {
#pragma unroll 1
                for (int pl = 2; pl >= 0; --pl) steps<KP / 16, false>(acc, w.tmem + W::H + pl * (KP / 2), sw128_desc(kq), ID_ROWS, pl < 2);
                mma_commit(w.turn.mma);
            }
            ++committed;
            __syncwarp();
            if (!(ok = w.turn.next(w.turn.ready))) break;
            if (w.lane == 0) {
                // the six products of parts, small ones first: (2, 0), (0, 2), (1, 1), (1, 0), (0, 1), (0, 0)
#pragma unroll 1
                for (int q = 0; q < 6; ++q)
                    steps<4, false>(acc, w.tmem + W::P + (0x052 >> 2 * q & 3) * 32, sw128_desc(tp + (0x118 >> 2 * q & 3) * ATOM), ID_ROWS, q > 0);
                mma_commit(w.turn.mma);
            }
            ++committed;
            __syncwarp();
            if (!(ok = w.turn.next(w.turn.ready))) break;
            if (w.lane == 0) {
#pragma unroll 1
                for (int pl = 2; pl >= 0; --pl) steps<4, true>(acc, w.tmem + W::P + pl * 32, mn_desc(kq, ATOM), ID_KP, pl < 2);
                mma_commit(w.turn.mma);
            }
            ++committed;
            __syncwarp();
        }
        if (w.lane == 0) w.turn.settle_products(committed);
        __syncwarp();
    } else {
        float st[HK];                           // of column dv
#pragma unroll
        for (int i = 0; i < HK; ++i) {
            const int r = w.cq * HK + i;
            st[i] = 0.f;
            if (place.unit) st[i] = r == w.dv && r < p.Dk ? 1.f : 0.f;
            else if (from) st[i] = w.dv < p.Dvp && r < p.Dk ? from[(long long)r * p.Dvp + w.dv] : 0.f;
            else if ((Y || place.first) && p.h_in && w.row >= 0 && w.on && r < p.Dk) st[i] = p.h_in[w.state + (long long)r * p.Dv];
        }
        uint32_t v[TPT / 2];
        dep_wait();
        if (w.chunks > 0) {
            w.values(p.v, p.v_ld, p, 0, v);
            put_state<KP>(w.lanes + W::H + w.cq * (HK / 2), st);
        }
        const int tok = w.tok;
        for (int c = 0; c < w.chunks; ++c) {
            const int t = w.t0 + c * DC, n = min(DC, w.t1 - t);
            w.turn.tell();                        // h0's parts are in TMEM
            const float* rows = w.rows(c);
            if (Y && p.saved) w.keep(p.saved + w.at(p, c) * p.Dk * p.Dvp, p, p.Dvp, st);
            if (!w.turn.next(w.turn.mma) || !w.turn.arrived(c)) break;
            float y[TPT];
#pragma unroll
            for (int j = 0; j < TPT; j += 16) {
                uint32_t a[16];
                tmem_ld16(w.lanes + W::ACC + tok + j, a);
                float r[16], f[16];
                read16(rows + RF_BETA + tok + j, r);
                read16(rows + RF_IN + tok + j, f);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float v0, v1;
                    bf2_unpack(v[j / 2 + i], v0, v1);
                    r[2 * i] = r[2 * i] * v0 - f[2 * i] * __uint_as_float(a[2 * i]);
                    r[2 * i + 1] = r[2 * i + 1] * v1 - f[2 * i + 1] * __uint_as_float(a[2 * i + 1]);
                }
                put_parts(w.lanes + W::P + (tok + j) / 2, 32, r);
            }
            if constexpr (Y) {
#pragma unroll
                for (int j = 0; j < TPT; j += 16) {       // (before the products with R overwrite it)
                    uint32_t a[16];
                    tmem_ld16(w.lanes + W::ACC + 64 + tok + j, a);
                    float f[16];
                    read16(rows + RF_OUT + tok + j, f);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 16; ++i) y[j + i] = f[i] * __uint_as_float(a[i]);
                }
            }
            w.turn.tell();
            if (c + 1 < w.chunks) w.values(p.v, p.v_ld, p, c + 1, v);
            if (!w.turn.next(w.turn.mma)) break;
#pragma unroll
            for (int j = 0; j < TPT; j += 16) {
                uint32_t a[16];
                tmem_ld16(w.lanes + W::ACC + tok + j, a);
                float f[16];
                read16(rows + RF_END + tok + j, f);
                tmem_ld_wait();
                if (Y && p.saved && w.dv < p.Dvp) {
                    float* to = p.saved + p.saved_u + (w.at(p, c) * DC + tok + j) * p.Dvp + w.dv;
#pragma unroll
                    for (int i = 0; i < 16; ++i) to[i * p.Dvp] = __uint_as_float(a[i]);
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) f[i] *= __uint_as_float(a[i]);
                put_parts(w.lanes + W::P + (tok + j) / 2, 32, f);
            }
            if constexpr (Y) {
#pragma unroll
                for (int j = 0; j < TPT; j += 16) {
                    uint32_t a[16];
                    tmem_ld16(w.lanes + W::ACC + 64 + tok + j, a);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 16; ++i) y[j + i] += __uint_as_float(a[i]);
                }
            }
            const float decay = rows[RF_DECAY];
            w.turn.tell();
            if constexpr (Y) {
#pragma unroll
                for (int j = 0; j < TPT; j += 16) {
                    float x[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[i] = y[j + i];
                    w.store(p.y, p.y_ld, p, t, n, tok + j, x);
                }
            }
            if (!w.turn.next(w.turn.mma)) break;
            w.turn.release(c);
            next_state<KP>(w.lanes + W::ACC + w.cq * HK, decay, st);
            if (c + 1 < w.chunks) put_state<KP>(w.lanes + W::H + w.cq * (HK / 2), st);
        }
        if (MODE == DELTA_PIECES) {
            if (place.unit) w.keep(p.through + kept * p.Dkp, p, p.Dkp, st);
            else w.keep(p.added + kept * p.Dvp, p, p.Dvp, st);
        } else if (p.h_out && w.row >= 0 && w.on && place.last) {
#pragma unroll
            for (int i = 0; i < HK; ++i)
                if (w.cq * HK + i < p.Dk) p.h_out[w.state + (long long)(w.cq * HK + i) * p.Dv] = st[i];
        }
    }
    w.close();
}

template <int KP, int MODE>
cudaError_t launch_walk_tc(const SeqDeltaParams& p, unsigned* err, cudaStream_t stream) {
    const auto kernel = delta_walk_tc_kernel<KP, MODE>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)WalkTc<KP>::BYTES);
    if (e != cudaSuccess) return e;
    const int dvbs = (p.Dv + 127) / 128, dkbs = 1;
    const long long blocks = (MODE == DELTA_WHOLE ? p.ax.S : MODE == DELTA_PIECES ? p.marks : p.pieces) * (long long)p.Hv * (MODE == DELTA_PIECES ? dvbs + dkbs : dvbs);
    return launch_kernel(kernel, dim3((unsigned)blocks), dim3(WALK_THREADS), WalkTc<KP>::BYTES, stream, p.slots > 0, 1, p, dvbs, dkbs, err);
}
template <int KP>
cudaError_t launch_walk_tc(const SeqDeltaParams& p, DeltaWalk mode, unsigned* err, cudaStream_t stream) {
    return mode == DELTA_WHOLE    ? launch_walk_tc<KP, DELTA_WHOLE>(p, err, stream)
           : mode == DELTA_PIECES ? launch_walk_tc<KP, DELTA_PIECES>(p, err, stream)
                                  : launch_walk_tc<KP, DELTA_JOINED>(p, err, stream);
}

// ---- backward ----
// The walk from the last chunk to the first (see seq_delta_bwd.cu):
//   [dh^T K^T | dY^T A], dU^T T, Y1^T Q + X1^T K,   dU = exp(b_C - b) |k|^-1 (K dh) + A^T dY, dR = T^T dU,
// Y1 = scale exp(b) |q|^-1 dY, X1 = -beta exp(b) |k|^-1 dR.  The same shared memory and threads; T, A, K and Q are
// read across their rows (K-major for the first product with K).
template <int KP>
struct BackTc {
    static constexpr uint32_t H = 0, P = 3 * KP / 2, Y = P + 96, ACC = Y + 96;       // TMEM columns: dh, dY or dU or X1, Y1
};

template <int KP>
__global__ void __launch_bounds__(WALK_THREADS, 1) delta_back_tc_kernel(const __grid_constant__ SeqDeltaParams p, int dvbs, unsigned* err) {
    extern __shared__ uint8_t smem_raw[];
    using W = WalkTc<KP>;
    using B = BackTc<KP>;
    using T = __nv_bfloat16;
    constexpr int HK = KP * 128 / WT;
    constexpr uint32_t ACROSS = 1u << 16, ID_64 = idesc_f32acc(128, 64, 1u), ID_KP = idesc_f32acc(128, KP, 1u) | ACROSS;
    Walk<KP> w(p, walk_place<DELTA_WHOLE>(p, dvbs, 0), err, smem_raw);
    dep_launch();
    if (w.warp > 0 && w.warp <= LOADERS) {
        dep_wait();
        w.load(p, true);
    } else if (w.warp == 0) {                   // the issuing warp (the first: the oldest is served first)
        bool ok = true;
        int committed = 0;
        for (int s = 0; s < w.chunks && ok; ++s) {
            if (p.test_stall && s == 1) break;       // (test hook: the other warps' wait runs out)
            const uint32_t kq = w.stage(s), tp = kq + W::KQ, acc = w.tmem + B::ACC;
            ok = w.turn.arrived(s) && w.turn.next(w.turn.ready);
            if (!ok) break;
            if (w.lane == 0) {
#pragma unroll 1
                for (int pl = 2; pl >= 0; --pl) steps<KP / 16, false>(acc, w.tmem + B::H + pl * (KP / 2), sw128_desc(kq), ID_64, pl < 2);
#pragma unroll 1
                for (int pl = 2; pl >= 0; --pl)       // A's rows are behind T's 64 (8 KB)
                    steps<4, true>(acc + 64, w.tmem + B::P, mn_desc(tp + pl * ATOM + 8192, ATOM), ID_64 | ACROSS, pl < 2);
                mma_commit(w.turn.mma);
            }
            ++committed;
            __syncwarp();
            if (!(ok = w.turn.next(w.turn.ready))) break;
            if (w.lane == 0) {
                // the six products of parts, small ones first: (2, 0), (0, 2), (1, 1), (1, 0), (0, 1), (0, 0)
#pragma unroll 1
                for (int q = 0; q < 6; ++q)
                    steps<4, true>(acc, w.tmem + B::P + (0x052 >> 2 * q & 3) * 32, mn_desc(tp + (0x118 >> 2 * q & 3) * ATOM, ATOM), ID_64 | ACROSS, q > 0);
                mma_commit(w.turn.mma);
            }
            ++committed;
            __syncwarp();
            if (!(ok = w.turn.next(w.turn.ready))) break;
            if (w.lane == 0) {
#pragma unroll 1
                for (int pl = 2; pl >= 0; --pl) {     // K's rows are the first 64 of an atom, Q's the others
                    steps<4, true>(acc, w.tmem + B::P + pl * 32, mn_desc(kq, ATOM), ID_KP, pl < 2);
                    steps<4, true>(acc, w.tmem + B::Y + pl * 32, mn_desc(kq + 8192, ATOM), ID_KP, true);
                }
                mma_commit(w.turn.mma);
            }
            ++committed;
            __syncwarp();
        }
        if (w.lane == 0) w.turn.settle_products(committed);
        __syncwarp();
    } else {
        float st[HK];                           // of column dv: the gradient at the state the chunk leaves
#pragma unroll
        for (int i = 0; i < HK; ++i) {
            const int r = w.cq * HK + i;
            st[i] = p.dh_out && w.row >= 0 && w.on && r < p.Dk ? p.dh_out[w.state + (long long)r * p.Dv] : 0.f;
        }
        uint32_t dy[TPT / 2];
        auto put_dy = [&]() {                   // dY is exact in one part
#pragma unroll
            for (int j = 0; j < TPT; j += 16) {
                uint32_t x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = dy[j / 2 + i];
                tmem_st8(w.lanes + B::P + (w.tok + j) / 2, x);
            }
        };
        dep_wait();
        if (w.chunks > 0) {
            w.values(p.dy, p.dy_ld, p, w.chunks - 1, dy);
            put_state<KP>(w.lanes + B::H + w.cq * (HK / 2), st);
            put_dy();
        }
        const int tok = w.tok;
        for (int s = 0; s < w.chunks; ++s) {
            const int c = w.chunks - 1 - s, t = w.t0 + c * DC, n = min(DC, w.t1 - t);
            w.turn.tell();
            const float* rows = w.rows(s);
            w.keep(p.dstate + w.at(p, c) * p.Dk * p.Dvp, p, p.Dvp, st);
            if (!w.turn.next(w.turn.mma) || !w.turn.arrived(s)) break;
#pragma unroll
            for (int j = 0; j < TPT; j += 16) {
                uint32_t a[16], b[16];
                tmem_ld16(w.lanes + B::ACC + tok + j, a);
                tmem_ld16(w.lanes + B::ACC + 64 + tok + j, b);
                float f[16];
                read16(rows + RF_END + tok + j, f);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) f[i] = fmaf(f[i], __uint_as_float(a[i]), __uint_as_float(b[i]));
                put_parts(w.lanes + B::P + (tok + j) / 2, 32, f);
            }
            w.turn.tell();
#pragma unroll
            for (int j = 0; j < TPT; j += 16) {     // Y1, and the next chunk's dY, while the products run
                float f[16];
                read16(rows + RF_OUT + tok + j, f);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float a, b;
                    bf2_unpack(dy[j / 2 + i], a, b);
                    f[2 * i] *= a;
                    f[2 * i + 1] *= b;
                }
                put_parts(w.lanes + B::Y + (tok + j) / 2, 32, f);
            }
            if (s + 1 < w.chunks) w.values(p.dy, p.dy_ld, p, c - 1, dy);
            if (!w.turn.next(w.turn.mma)) break;
            const float decay = rows[RF_DECAY];
            float dr[TPT];
#pragma unroll
            for (int j = 0; j < TPT; j += 16) {
                uint32_t a[16];
                tmem_ld16(w.lanes + B::ACC + tok + j, a);
                float f[16];
                read16(rows + RF_IN + tok + j, f);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    dr[j + i] = __uint_as_float(a[i]);
                    f[i] *= -dr[j + i];
                }
                put_parts(w.lanes + B::P + (tok + j) / 2, 32, f);
            }
            w.turn.tell();
#pragma unroll
            for (int j = 0; j < TPT; j += 16) {
                if (w.dv < p.Dvp) {
                    float* to = p.dr + (w.at(p, c) * DC + tok + j) * p.Dvp + w.dv;
#pragma unroll
                    for (int i = 0; i < 16; ++i) to[i * p.Dvp] = dr[j + i];
                }
                float beta[16];
                read16(rows + RF_BETA + tok + j, beta);
#pragma unroll
                for (int i = 0; i < 16; ++i) beta[i] *= dr[j + i];
                w.store(p.dv, p.dv_ld, p, t, n, tok + j, beta);
            }
            if (!w.turn.next(w.turn.mma)) break;
            w.turn.release(s);
            next_state<KP>(w.lanes + B::ACC + w.cq * HK, decay, st);
            if (s + 1 < w.chunks) {
                put_state<KP>(w.lanes + B::H + w.cq * (HK / 2), st);
                put_dy();
            }
        }
        if (p.dh_in && w.row >= 0 && w.on) {
#pragma unroll
            for (int i = 0; i < HK; ++i)
                if (w.cq * HK + i < p.Dk) p.dh_in[w.state + (long long)(w.cq * HK + i) * p.Dv] = st[i];
        }
    }
    w.close();
}

template <int KP>
cudaError_t launch_back_tc(const SeqDeltaParams& p, unsigned* err, cudaStream_t stream) {
    cudaError_t e = cudaFuncSetAttribute(delta_back_tc_kernel<KP>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)WalkTc<KP>::BYTES);
    if (e != cudaSuccess) return e;
    const int dvbs = (p.Dv + 127) / 128;
    return launch_kernel(delta_back_tc_kernel<KP>, dim3((unsigned)(p.ax.S * (long long)p.Hv * dvbs)), dim3(WALK_THREADS), WalkTc<KP>::BYTES, stream, p.slots > 0, 1, p,
                         dvbs, err);
}

}  // namespace

cudaError_t launch_seq_delta_walk_tc(const SeqDeltaParams& p, DeltaWalk mode, cudaStream_t stream) {
    unsigned* err = device_error_word();
    if (!err) return cudaErrorUnknown;
    return p.Dk <= 64 ? launch_walk_tc<64>(p, mode, err, stream) : launch_walk_tc<128>(p, mode, err, stream);
}

cudaError_t launch_seq_delta_back_tc(const SeqDeltaParams& p, cudaStream_t stream) {
    unsigned* err = device_error_word();
    if (!err) return cudaErrorUnknown;
    return p.Dk <= 64 ? launch_back_tc<64>(p, err, stream) : launch_back_tc<128>(p, err, stream);
}

}  // namespace convfwd

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
// What bounds a walk: the products and the threads' work between them follow one another, three times a chunk.
#include "seq_delta.cuh"
#include "tc_common.cuh"

namespace convfwd {
namespace {

constexpr int WT = 512;                       // threads: four warps a quarter of the lanes, a quarter of the columns each
constexpr uint32_t ATOM = 128 * 128;          // 128 rows of 64 bf16
constexpr uint32_t PLANES = 3 * ATOM;         // [T; A T] (backward: [T; A]) in three parts

__device__ __forceinline__ uint64_t mn_desc(uint32_t saddr, uint32_t stride) {     // N side by side, blocks of 64 `stride` bytes apart
    uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)((stride >> 4) & 0x3FFFu) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}
// D += A B with A in TMEM (a lane's 16 bf16 of a step in 8 columns)
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
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

// What a walk's CTA needs to wait: barriers of the products and of the two stages' copies, all bounded.
struct Waits {
    uint32_t mma, full;               // shared addresses (full: two)
    uint32_t mma_phase;
    volatile int* abort_flag;
    unsigned* err;
    __device__ __forceinline__ bool products() {
        const bool ok = wait_bar(mma, mma_phase, abort_flag, err);
        mma_phase ^= 1;
        return ok;
    }
    // After a wait ran out: the last fetched chunk's copies and products that were issued, before shared memory and TMEM go
    // (bounded as well).
    __device__ __forceinline__ void drain(int fetched) {
        const unsigned long long since = globaltimer();
        for (int c = fetched > 1 ? fetched - 2 : 0; c < fetched; ++c)
            while (!mbar_try_wait(full + 8 * (c & 1), (c >> 1) & 1) && globaltimer() - since < WAIT_LIMIT_NS) {
            }
        while (!mbar_try_wait(mma, mma_phase) && !mbar_try_wait(mma, mma_phase ^ 1) && globaltimer() - since < WAIT_LIMIT_NS) {
        }
    }
};

// K and Q rows of a chunk to [K; Q] atoms in the 128-byte swizzle; rows at and behind n and columns behind the width are zero.
template <int KP>
__device__ __forceinline__ void load_kq(uint32_t to, const __nv_bfloat16* k, const __nv_bfloat16* q, long long k_ld, long long q_ld, int n, int width) {
    constexpr int CPR = KP / 8;
#pragma unroll
    for (int j = 0; j < 128 * CPR / WT; ++j) {
        const int i = threadIdx.x + j * WT, row = i / CPR, c = i % CPR, r = row & 63;
        const bool on = r < n && c * 8 < width;
        const __nv_bfloat16* from = row < 64 ? k : q;
        cp_async_16(to + (uint32_t)(c / 8) * ATOM + row * 128 + ((c % 8) ^ (row & 7)) * 16,
                    on ? from + r * (row < 64 ? k_ld : q_ld) + c * 8 : from, on ? 16 : 0);
    }
}

template <int KP>
__global__ void __launch_bounds__(WT, 1) delta_walk_tc_kernel(const __grid_constant__ SeqDeltaParams p, int dvbs, unsigned* err) {
    extern __shared__ uint8_t smem_raw[];
    using W = WalkTc<KP>;
    using T = __nv_bfloat16;
    constexpr int HK = KP / 4;                  // the thread's rows of the state: cq HK ..; its tokens: 16 cq ..
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - smem_u32(smem_raw));
    const uint32_t bars = base + 2 * W::STAGE;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + 2 * W::STAGE + 64);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + 2 * W::STAGE + 72);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, wq = warp & 3, cq = warp >> 2;
    const int dvb = blockIdx.x % dvbs, sh = blockIdx.x / dvbs, h = sh % p.Hv, seq = sh / p.Hv, kh = h / (p.Hv / p.Hk);
    const int dv = dvb * 128 + wq * 32 + lane;
    const bool on = dv < p.Dv;
    const int t0 = p.ax.L > 0 ? seq * p.ax.L : seq_start(p.ax, seq, 0), t1 = p.ax.L > 0 ? t0 + p.ax.L : seq_start(p.ax, seq + 1, t0);
    const int chunks = (t1 - t0 + DC - 1) / DC, slot0 = cut_base(p.ax, seq, DC);
    if (threadIdx.x == 0) {
        mbar_init(bars, 1);
        mbar_init(bars + 8, 1);
        mbar_init(bars + 16, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot, lanes = tmem + ((uint32_t)(wq * 32) << 16);
    Waits wait = {bars, bars + 8, 0, abort_flag, err};

    const long long row = seq_slot(p.sl, seq), state = (row * p.Hv + h) * (long long)p.Dk * p.Dv + dv;
    float st[HK];                               // of column dv
#pragma unroll
    for (int i = 0; i < HK; ++i) {
        const int r = cq * HK + i;
        st[i] = p.h_in && row >= 0 && on && r < p.Dk ? p.h_in[state + (long long)r * p.Dv] : 0.f;
    }
    auto put_state = [&]() {
#pragma unroll
        for (int i = 0; i < HK; i += 16) {
            float x[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = st[i + e];
            put_parts(lanes + W::H + cq * (HK / 2) + i / 2, KP / 2, x);
        }
    };
    int fetched = 0;
    auto fetch = [&](int c) {                   // a chunk's operands to its stage
        fetched = c + 1;
        const uint32_t to = base + (c & 1) * W::STAGE, bar = wait.full + 8 * (c & 1);
        const int t = t0 + c * DC;
        const long long at = (long long)(slot0 + c) * p.Hv + h;
        if (threadIdx.x == 0) {
            mbar_arrive_expect_tx(bar, PLANES + DELTA_ROWS * 4);
            bulk_g2s(to + W::KQ, reinterpret_cast<const uint8_t*>(p.tri) + at * PLANES, PLANES, bar);
            bulk_g2s(to + W::KQ + PLANES, p.rows + at * DELTA_ROWS, DELTA_ROWS * 4, bar);
        }
        load_kq<KP>(to, static_cast<const T*>(p.k) + t * p.k_ld + kh * p.Dk, static_cast<const T*>(p.q) + t * p.q_ld + kh * p.Dk, p.k_ld, p.q_ld,
                    min(DC, t1 - t), p.Dk);
        cp_async_commit();
    };
    dep_wait();
    if (chunks > 0) {
        put_state();
        fetch(0);
        tmem_st_wait();
    }
    bool ok = true;
    constexpr uint32_t ID_64 = idesc_f32acc(128, 64, 1u), ID_128 = idesc_f32acc(128, 128, 1u), ID3 = idesc_f32acc(128, KP, 1u) | (1u << 16);
    for (int c = 0; c < chunks; ++c) {
        const uint32_t kq = base + (c & 1) * W::STAGE, tp = kq + W::KQ;
        const float* rows = reinterpret_cast<const float*>(smem + (c & 1) * W::STAGE + W::KQ + PLANES);
        const int t = t0 + c * DC, n = min(DC, t1 - t);
        const long long at = (long long)(slot0 + c) * p.Hv + h;
        // this chunk's K and Q are there, the state's parts are in TMEM
        cp_async_wait<0>();
        fence_proxy_async();
        ok = wait_bar(wait.full + 8 * (c & 1), (c >> 1) & 1, abort_flag, err) && ok;
        tc_fence_before();
        if (__syncthreads_or(!ok)) break;
        if (threadIdx.x == 0) {      // y needs two parts of h only: the last one goes with K alone
            tc_fence_after();
#pragma unroll
            for (int q = 0; q < 3; ++q) {
                const int pl = q == 0 ? 1 : q == 1 ? 0 : 2;
#pragma unroll
                for (int k = 0; k < KP / 16; ++k)
                    mma_ts(tmem + W::ACC, tmem + W::H + pl * (KP / 2) + k * 8, sw128_desc(kq + (k / 4) * ATOM) + (uint64_t)((k % 4) * 2),
                           pl == 2 ? ID_64 : ID_128, q > 0 || k > 0);
            }
            mma_commit(wait.mma);
        }
        if (c + 1 < chunks) fetch(c + 1);
        const int tok = cq * 16;                 // the thread's tokens of the chunk
        T v[16];
        {
            const T* from = static_cast<const T*>(p.v) + (long long)(t + tok) * p.v_ld + h * p.Dv + dv;
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = on && tok + i < n ? from[i * p.v_ld] : T(0.f);
        }
        if (p.saved && dv < p.Dvp) {
            float* to = p.saved + at * p.Dk * p.Dvp + dv;
#pragma unroll
            for (int i = 0; i < HK; ++i)
                if (cq * HK + i < p.Dk) to[(cq * HK + i) * p.Dvp] = st[i];
        }
        ok = wait.products() && ok;
        tc_fence_after();
        float y[16];
        {
            uint32_t a[16], q[16];
            tmem_ld16(lanes + W::ACC + tok, a);
            tmem_ld16(lanes + W::ACC + 64 + tok, q);
            float beta[16], in[16];
            read16(rows + RF_BETA + tok, beta);
            read16(rows + RF_IN + tok, in);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) beta[i] = beta[i] * __bfloat162float(v[i]) - in[i] * __uint_as_float(a[i]);
            put_parts(lanes + W::P + cq * 8, 32, beta);
            read16(rows + RF_OUT + tok, in);
#pragma unroll
            for (int i = 0; i < 16; ++i) y[i] = in[i] * __uint_as_float(q[i]);
        }
        tmem_st_wait();
        tc_fence_before();
        if (__syncthreads_or(!ok)) break;
        if (threadIdx.x == 0) {
            tc_fence_after();
            // U needs six products of parts, y the three large ones
            constexpr int PA[6] = {1, 0, 0, 2, 0, 1}, PB[6] = {0, 1, 0, 0, 2, 1};
#pragma unroll
            for (int q = 0; q < 6; ++q)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mma_ts(tmem + W::ACC, tmem + W::P + PA[q] * 32 + k * 8, sw128_desc(tp + PB[q] * ATOM) + (uint64_t)(k * 2), q < 3 ? ID_128 : ID_64,
                           q > 0 || k > 0);
            mma_commit(wait.mma);
        }
        ok = wait.products() && ok;
        tc_fence_after();
        {
            uint32_t a[16], q[16];
            tmem_ld16(lanes + W::ACC + tok, a);
            tmem_ld16(lanes + W::ACC + 64 + tok, q);
            float end[16];
            read16(rows + RF_END + tok, end);
            tmem_ld_wait();
            if (p.saved && dv < p.Dvp) {
                float* to = p.saved + p.saved_u + (at * DC + tok) * p.Dvp + dv;
#pragma unroll
                for (int i = 0; i < 16; ++i) to[i * p.Dvp] = __uint_as_float(a[i]);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) end[i] *= __uint_as_float(a[i]);
            put_parts(lanes + W::P + cq * 8, 32, end);
#pragma unroll
            for (int i = 0; i < 16; ++i) y[i] += __uint_as_float(q[i]);
        }
        tmem_st_wait();
        tc_fence_before();
        if (__syncthreads_or(!ok)) break;
        if (threadIdx.x == 0) {
            tc_fence_after();
#pragma unroll
            for (int pl = 2; pl >= 0; --pl)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mma_ts(tmem + W::ACC, tmem + W::P + pl * 32 + k * 8, mn_desc(kq + k * 2048, ATOM), ID3, pl < 2 || k > 0);
            mma_commit(wait.mma);
        }
        if (on) {
            T* to = static_cast<T*>(p.y) + (long long)(t + tok) * p.y_ld + h * p.Dv + dv;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (tok + i < n) to[i * p.y_ld] = __float2bfloat16_rn(y[i]);
        }
        const float decay = rows[RF_DECAY];
        ok = wait.products() && ok;
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < HK; i += 16) {
            uint32_t a[16];
            tmem_ld16(lanes + W::ACC + cq * HK + i, a);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) st[i + e] = fmaf(decay, st[i + e], __uint_as_float(a[e]));
        }
        if (c + 1 < chunks) {
            put_state();
            tmem_st_wait();
        }
    }
    if (p.h_out && row >= 0 && on) {
#pragma unroll
        for (int i = 0; i < HK; ++i)
            if (cq * HK + i < p.Dk) p.h_out[state + (long long)(cq * HK + i) * p.Dv] = st[i];
    }
    cp_async_wait<0>();
    if (threadIdx.x == 0 && *abort_flag) wait.drain(fetched);
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int KP>
cudaError_t launch_walk_tc(const SeqDeltaParams& p, unsigned* err, cudaStream_t stream) {
    cudaError_t e = cudaFuncSetAttribute(delta_walk_tc_kernel<KP>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)WalkTc<KP>::BYTES);
    if (e != cudaSuccess) return e;
    const int dvbs = (p.Dv + 127) / 128;
    return launch_kernel(delta_walk_tc_kernel<KP>, dim3((unsigned)(p.ax.S * (long long)p.Hv * dvbs)), dim3(WT), WalkTc<KP>::BYTES, stream, p.slots > 0, 1, p,
                         dvbs, err);
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
__global__ void __launch_bounds__(WT, 1) delta_back_tc_kernel(const __grid_constant__ SeqDeltaParams p, int dvbs, unsigned* err) {
    extern __shared__ uint8_t smem_raw[];
    using W = WalkTc<KP>;
    using B = BackTc<KP>;
    using T = __nv_bfloat16;
    constexpr int HK = KP / 4;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - smem_u32(smem_raw));
    const uint32_t bars = base + 2 * W::STAGE;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + 2 * W::STAGE + 64);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + 2 * W::STAGE + 72);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, wq = warp & 3, cq = warp >> 2;
    const int dvb = blockIdx.x % dvbs, sh = blockIdx.x / dvbs, h = sh % p.Hv, seq = sh / p.Hv, kh = h / (p.Hv / p.Hk);
    const int dv = dvb * 128 + wq * 32 + lane;
    const bool on = dv < p.Dv;
    const int t0 = p.ax.L > 0 ? seq * p.ax.L : seq_start(p.ax, seq, 0), t1 = p.ax.L > 0 ? t0 + p.ax.L : seq_start(p.ax, seq + 1, t0);
    const int chunks = (t1 - t0 + DC - 1) / DC, slot0 = cut_base(p.ax, seq, DC);
    if (threadIdx.x == 0) {
        mbar_init(bars, 1);
        mbar_init(bars + 8, 1);
        mbar_init(bars + 16, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot, lanes = tmem + ((uint32_t)(wq * 32) << 16);
    Waits wait = {bars, bars + 8, 0, abort_flag, err};

    const long long row = seq_slot(p.sl, seq), state = (row * p.Hv + h) * (long long)p.Dk * p.Dv + dv;
    float st[HK];                               // of column dv: the gradient at the state the chunk leaves
#pragma unroll
    for (int i = 0; i < HK; ++i) {
        const int r = cq * HK + i;
        st[i] = p.dh_out && row >= 0 && on && r < p.Dk ? p.dh_out[state + (long long)r * p.Dv] : 0.f;
    }
    int fetched = 0;
    const int tok = cq * 16;                    // the thread's tokens of a chunk
    uint32_t dy[8];                             // and dY of those of the next one: pairs of tokens
    auto fetch = [&](int s) {                   // the operands of the s-th chunk from the end
        fetched = s + 1;
        const uint32_t to = base + (s & 1) * W::STAGE, bar = wait.full + 8 * (s & 1);
        const int c = chunks - 1 - s, t = t0 + c * DC, n = min(DC, t1 - t);
        const long long at = (long long)(slot0 + c) * p.Hv + h;
        if (threadIdx.x == 0) {
            mbar_arrive_expect_tx(bar, PLANES + DELTA_ROWS * 4);
            bulk_g2s(to + W::KQ, reinterpret_cast<const uint8_t*>(p.tri) + at * PLANES, PLANES, bar);
            bulk_g2s(to + W::KQ + PLANES, p.rows + at * DELTA_ROWS, DELTA_ROWS * 4, bar);
        }
        load_kq<KP>(to, static_cast<const T*>(p.k) + t * p.k_ld + kh * p.Dk, static_cast<const T*>(p.q) + t * p.q_ld + kh * p.Dk, p.k_ld, p.q_ld, n, p.Dk);
        cp_async_commit();
        const uint16_t* from = static_cast<const uint16_t*>(p.dy) + (long long)(t + tok) * p.dy_ld + h * p.Dv + dv;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t a = on && tok + 2 * i < n ? from[2 * i * p.dy_ld] : 0, b = on && tok + 2 * i + 1 < n ? from[(2 * i + 1) * p.dy_ld] : 0;
            dy[i] = a | b << 16;
        }
    };
    auto put_state = [&]() {
#pragma unroll
        for (int i = 0; i < HK; i += 16) {
            float x[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = st[i + e];
            put_parts(lanes + B::H + cq * (HK / 2) + i / 2, KP / 2, x);
        }
        tmem_st8(lanes + B::P + cq * 8, dy);    // dY is exact in one part
    };
    dep_launch();
    dep_wait();
    if (chunks > 0) {
        fetch(0);
        put_state();
        tmem_st_wait();
    }
    bool ok = true;
    constexpr uint32_t ID_64 = idesc_f32acc(128, 64, 1u), ACROSS = 1u << 16, ID_KP = idesc_f32acc(128, KP, 1u) | ACROSS;
    for (int s = 0; s < chunks; ++s) {
        const uint32_t kq = base + (s & 1) * W::STAGE, tp = kq + W::KQ;
        const float* rows = reinterpret_cast<const float*>(smem + (s & 1) * W::STAGE + W::KQ + PLANES);
        const int c = chunks - 1 - s, t = t0 + c * DC, n = min(DC, t1 - t);
        const long long at = (long long)(slot0 + c) * p.Hv + h;
        cp_async_wait<0>();
        fence_proxy_async();
        ok = wait_bar(wait.full + 8 * (s & 1), (s >> 1) & 1, abort_flag, err) && ok;
        tc_fence_before();
        if (__syncthreads_or(!ok)) break;
        if (threadIdx.x == 0) {
            tc_fence_after();
#pragma unroll
            for (int pl = 2; pl >= 0; --pl)
#pragma unroll
                for (int k = 0; k < KP / 16; ++k)
                    mma_ts(tmem + B::ACC, tmem + B::H + pl * (KP / 2) + k * 8, sw128_desc(kq + (k / 4) * ATOM) + (uint64_t)((k % 4) * 2), ID_64, pl < 2 || k > 0);
#pragma unroll
            for (int pl = 2; pl >= 0; --pl)
#pragma unroll
                for (int k = 0; k < 4; ++k)      // A's rows are behind T's 64 (8 KB)
                    mma_ts(tmem + B::ACC + 64, tmem + B::P + k * 8, mn_desc(tp + pl * ATOM + 8192 + k * 2048, ATOM), ID_64 | ACROSS, pl < 2 || k > 0);
            mma_commit(wait.mma);
        }
        // Y1 while the products run
        {
            float f[16];
            read16(rows + RF_OUT + tok, f);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float a, b;
                bf2_unpack(dy[i], a, b);
                f[2 * i] *= a;
                f[2 * i + 1] *= b;
            }
            put_parts(lanes + B::Y + cq * 8, 32, f);
        }
        if (s + 1 < chunks) fetch(s + 1);
        if (dv < p.Dvp) {
            float* to = p.dstate + at * p.Dk * p.Dvp + dv;
#pragma unroll
            for (int i = 0; i < HK; ++i)
                if (cq * HK + i < p.Dk) to[(cq * HK + i) * p.Dvp] = st[i];
        }
        ok = wait.products() && ok;
        tc_fence_after();
        {
            uint32_t a[16], b[16];
            tmem_ld16(lanes + B::ACC + tok, a);
            tmem_ld16(lanes + B::ACC + 64 + tok, b);
            float f[16];
            read16(rows + RF_END + tok, f);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) f[i] = fmaf(f[i], __uint_as_float(a[i]), __uint_as_float(b[i]));
            put_parts(lanes + B::P + cq * 8, 32, f);
        }
        tmem_st_wait();
        tc_fence_before();
        if (__syncthreads_or(!ok)) break;
        if (threadIdx.x == 0) {
            tc_fence_after();
            constexpr int PA[6] = {2, 0, 1, 1, 0, 0}, PB[6] = {0, 2, 1, 0, 1, 0};
#pragma unroll
            for (int q = 0; q < 6; ++q)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mma_ts(tmem + B::ACC, tmem + B::P + PA[q] * 32 + k * 8, mn_desc(tp + PB[q] * ATOM + k * 2048, ATOM), ID_64 | ACROSS, q > 0 || k > 0);
            mma_commit(wait.mma);
        }
        ok = wait.products() && ok;
        tc_fence_after();
        {
            uint32_t a[16];
            tmem_ld16(lanes + B::ACC + tok, a);
            float f[16], beta[16];
            read16(rows + RF_IN + tok, f);
            read16(rows + RF_BETA + tok, beta);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) f[i] *= -__uint_as_float(a[i]);
            put_parts(lanes + B::P + cq * 8, 32, f);
            if (dv < p.Dvp) {
                float* to = p.dr + (at * DC + tok) * p.Dvp + dv;
#pragma unroll
                for (int i = 0; i < 16; ++i) to[i * p.Dvp] = __uint_as_float(a[i]);
            }
            if (on) {
                T* to = static_cast<T*>(p.dv) + (long long)(t + tok) * p.dv_ld + h * p.Dv + dv;
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (tok + i < n) to[i * p.dv_ld] = __float2bfloat16_rn(beta[i] * __uint_as_float(a[i]));
            }
        }
        tmem_st_wait();
        tc_fence_before();
        if (__syncthreads_or(!ok)) break;
        if (threadIdx.x == 0) {
            tc_fence_after();
#pragma unroll
            for (int pl = 2; pl >= 0; --pl)
#pragma unroll
                for (int k = 0; k < 4; ++k) {    // K's rows are the first 64 of an atom, Q's the others
                    mma_ts(tmem + B::ACC, tmem + B::P + pl * 32 + k * 8, mn_desc(kq + k * 2048, ATOM), ID_KP, pl < 2 || k > 0);
                    mma_ts(tmem + B::ACC, tmem + B::Y + pl * 32 + k * 8, mn_desc(kq + 8192 + k * 2048, ATOM), ID_KP, true);
                }
            mma_commit(wait.mma);
        }
        const float decay = rows[RF_DECAY];
        ok = wait.products() && ok;
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < HK; i += 16) {
            uint32_t a[16];
            tmem_ld16(lanes + B::ACC + cq * HK + i, a);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) st[i + e] = fmaf(decay, st[i + e], __uint_as_float(a[e]));
        }
        if (s + 1 < chunks) {
            put_state();
            tmem_st_wait();
        }
    }
    if (p.dh_in && row >= 0 && on) {
#pragma unroll
        for (int i = 0; i < HK; ++i)
            if (cq * HK + i < p.Dk) p.dh_in[state + (long long)(cq * HK + i) * p.Dv] = st[i];
    }
    cp_async_wait<0>();
    if (threadIdx.x == 0 && *abort_flag) wait.drain(fetched);
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int KP>
cudaError_t launch_back_tc(const SeqDeltaParams& p, unsigned* err, cudaStream_t stream) {
    cudaError_t e = cudaFuncSetAttribute(delta_back_tc_kernel<KP>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)WalkTc<KP>::BYTES);
    if (e != cudaSuccess) return e;
    const int dvbs = (p.Dv + 127) / 128;
    return launch_kernel(delta_back_tc_kernel<KP>, dim3((unsigned)(p.ax.S * (long long)p.Hv * dvbs)), dim3(WT), WalkTc<KP>::BYTES, stream, p.slots > 0, 1, p,
                         dvbs, err);
}

}  // namespace

cudaError_t launch_seq_delta_walk_tc(const SeqDeltaParams& p, cudaStream_t stream) {
    unsigned* err = device_error_word();
    if (!err) return cudaErrorUnknown;
    return p.Dk <= 64 ? launch_walk_tc<64>(p, err, stream) : launch_walk_tc<128>(p, err, stream);
}

cudaError_t launch_seq_delta_back_tc(const SeqDeltaParams& p, cudaStream_t stream) {
    unsigned* err = device_error_word();
    if (!err) return cudaErrorUnknown;
    return p.Dk <= 64 ? launch_back_tc<64>(p, err, stream) : launch_back_tc<128>(p, err, stream);
}

}  // namespace convfwd

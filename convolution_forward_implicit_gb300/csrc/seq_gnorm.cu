// Group norm with an activation, channels last: see gnorm.h for the formulas.  Bound by bytes.  Statistics
// cross the whole sequence, so a call reads its rows twice: a pass for the sums of every slab of tokens, a
// small one that joins them to the groups' statistics (a warp or a block a sequence and group), and one that
// applies them, last slabs first, so that it finds in L2 what the first pass read last.  32 x 56 x 56 x 512 in bf16 (103 MB) takes 31 and 40 us
// forward, 47 and 55 backward, 750 MB from and to memory, 4.3 TB/s: a block's chain of loads, sums and stores at 8 to 32
// warps an SM.  16 of them (51 MB, both passes within L2) take 41 us (21 and 22 cold), of which the bytes alone would take 15.
//
// A slab's statistics are means and sums of squared differences, joined by terms that are all positive (see Joined).  A thread
// sums over differences from the first value it meets in a channel; that value is one of the data, so the
// variance it takes part in is at least (its distance from the mean)^2 / n, and the rounding of the sums stays below
// about n 2^-24 of the result for n tokens a thread, wherever the mean lies.
//
// One kernel that keeps a sequence's rows in the shared memory of a cluster and reads global memory once was measured
// too, and is not kept: its CTAs load, compute and store in step (16 x 56 x 56 x 512 bf16: 63 us).
//
// gelu and its slope go by a polynomial of erfc (below) and an approximate reciprocal, as elsewhere in the library: y of fp32 calls is off by 1.9e-7 of its
// norm, 0.8e-7 with erff; with silu's reciprocals and the sums' order the gradients by 3.4e-7 (1.8e-7).
#include "gnorm.h"
#include "seq_common.cuh"
#include "seq_internal.h"

namespace convfwd {
namespace {

constexpr int GT = 256;              // threads a block at most

// How the channels lie on a block's threads: tx threads of V channels in a row, ty rows; cblocks blocks for all
// channels.  grouped: no group lies in two blocks, so that a block's sums can be those of groups.
struct GnShape {
    int tx, ty, cblocks, grouped;
};
GnShape gn_shape(int D, int cpg, int V) {
    int a = cpg, b = V;
    while (b) {
        const int r = a % b;
        a = b;
        b = r;
    }
    const long long unit = cpg / a;                   // threads whose channels are whole groups: lcm(cpg, V) / V
    const int n = (D + V - 1) / V;
    GnShape s;
    if (n <= GT) {
        s.tx = n;
        s.cblocks = s.grouped = 1;
    } else if (unit <= GT) {
        const int most = (int)(GT / unit * unit);
        const int blocks = (n + most - 1) / most;
        s.tx = (int)(((n + blocks - 1) / blocks + unit - 1) / unit * unit);
        s.cblocks = (n + s.tx - 1) / s.tx;
        s.grouped = 1;
    } else {
        s.cblocks = (n + GT - 1) / GT;
        s.tx = (n + s.cblocks - 1) / s.cblocks;
        s.grouped = 0;
    }
    s.ty = GT / s.tx;
    return s;
}

__device__ __forceinline__ void wait_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void launch_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 neg2(float2 a) { return make_float2(-a.x, -a.y); }
__device__ __forceinline__ float2 dup(float a) { return make_float2(a, a); }

// V channels of a thread, as loaded; as pairs (one channel: the second of its pair is nothing).
template <typename T, int V>
struct Raw {
    static constexpr int P = V > 1 ? V / 2 : 1, W = V * sizeof(T) >= 4 ? V * sizeof(T) / 4 : 1;
    uint32_t w[W];
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (W == 4) {
            const uint4 q = *reinterpret_cast<const uint4*>(p);
            w[0] = q.x; w[1] = q.y; w[2] = q.z; w[3] = q.w;
        } else if constexpr (W == 2) {
            const uint2 q = *reinterpret_cast<const uint2*>(p);
            w[0] = q.x; w[1] = q.y;
        } else if constexpr (V * sizeof(T) == 4) {
            w[0] = *reinterpret_cast<const uint32_t*>(p);
        } else {
            w[0] = (uint32_t)*reinterpret_cast<const uint16_t*>(p);
        }
    }
    __device__ __forceinline__ void get(float2 (&v)[P]) const {
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int i = 0; i < P; ++i) bf2_unpack(w[i], v[i].x, v[i].y);
        } else if constexpr (V == 1) {
            v[0] = make_float2(__uint_as_float(w[0]), 0.f);
        } else {
#pragma unroll
            for (int i = 0; i < P; ++i) v[i] = make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
        }
    }
};
template <typename T, int V>
__device__ __forceinline__ void put(T* p, const float2 (&v)[Raw<T, V>::P]) {
    if constexpr (V == 1) {
        seq_st(p, v[0].x);
    } else if constexpr (V == 2) {
        seq_st2(p, v[0], true, true);
    } else {
        float f[V];
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            f[2 * i] = v[i].x;
            f[2 * i + 1] = v[i].y;
        }
        seq_stv<V>(p, f);
    }
}
template <typename T, int V>
__device__ __forceinline__ void channel_param(const void* from, int c, float none, float2 (&v)[Raw<T, V>::P]) {
#pragma unroll
    for (int i = 0; i < Raw<T, V>::P; ++i) v[i] = dup(none);
    if (from) {
        Raw<T, V> r;
        r.load(static_cast<const T*>(from) + c);
        r.get(v);
    }
}

// act(z) of a pair, and its slope
template <int ACT>
__device__ __forceinline__ float2 act_of(float2 z) {
    if (ACT == SEQ_ACT_SILU) {
        const float2 e = mul2(z, dup(-LOG2E)), d = add2(make_float2(ex2_approx(e.x), ex2_approx(e.y)), dup(1.f));
        return mul2(z, make_float2(rcp_approx(d.x), rcp_approx(d.y)));
    }
    if (ACT == SEQ_ACT_GELU) return make_float2(gelu(z.x), gelu(z.y));
    return z;
}
// d gelu = Phi(z) + z phi(z).  Phi from A&S 7.1.28 as in gelu (y^-16 = erfc(|z| / sqrt 2)).
__device__ __forceinline__ float gelu_slope(float z) {
    const float u = fabsf(z) * 0.70710678118654752f;
    float y = fmaf(u, 0.0000430638f, 0.0002765672f);
    y = fmaf(u, y, 0.0001520143f);
    y = fmaf(u, y, 0.0092705272f);
    y = fmaf(u, y, 0.0422820123f);
    y = fmaf(u, y, 0.0705230784f);
    y = fmaf(u, y, 1.0f);
    y = y * y; y = y * y; y = y * y; y = y * y;
    const float tail = 0.5f * rcp_approx(y);
    const float phi = 0.39894228040143268f * ex2_approx(-0.5f * LOG2E * z * z);
    return fmaf(z, phi, z < 0.f ? tail : 1.f - tail);
}
template <int ACT>
__device__ __forceinline__ float2 slope_of(float2 z) {
    if (ACT == SEQ_ACT_SILU) {           // s (1 + z (1 - s))
        const float2 e = mul2(z, dup(-LOG2E)), d = add2(make_float2(ex2_approx(e.x), ex2_approx(e.y)), dup(1.f));
        const float2 s = make_float2(rcp_approx(d.x), rcp_approx(d.y));
        return mul2(s, fma2(z, add2(dup(1.f), neg2(s)), dup(1.f)));
    }
    if (ACT == SEQ_ACT_GELU) return make_float2(gelu_slope(z.x), gelu_slope(z.y));
    return dup(1.f);
}

// A thread's place: its channels c .. c + V - 1 and row of threads.
struct GnPlace {
    int c, tx, ty;
    bool on;
    __device__ __forceinline__ GnPlace(int V, int D, int txn) {
        ty = threadIdx.x / txn;
        tx = threadIdx.x - ty * txn;
        c = (blockIdx.y * txn + tx) * V;
        on = c < D;
    }
};

// mean, rstd w and b of V channels of a sequence: z = (x - mean) (rstd w) + b; `stats`: of the sequence's groups
template <typename T, int V>
struct Affine {
    static constexpr int P = Raw<T, V>::P;
    float2 mean[P], a[P], b[P];
    __device__ __forceinline__ void params(const SeqGnormParams& p, int c) {
        channel_param<T, V>(p.w, c, 1.f, a);
        channel_param<T, V>(p.b, c, 0.f, b);
    }
    // rstd: kept where it is wanted by itself
    __device__ __forceinline__ void stats(const float2* stats, int c, int cpg, float2* rstd = nullptr) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const float2 s0 = stats[(c + 2 * i) / cpg], s1 = V > 1 ? stats[(c + 2 * i + 1) / cpg] : s0;
            mean[i] = make_float2(s0.x, V > 1 ? s1.x : 0.f);
            const float2 r = make_float2(s0.y, s1.y);
            a[i] = mul2(a[i], r);
            if (rstd) rstd[i] = r;
        }
    }
};

// Rows a thread works on at once; as many more are on their way meanwhile.
constexpr int AHEAD = 2, AHEAD_BWD = 2;
// Blocks of 256 threads an SM: what the registers of the rows on their way leave room for (backward in bf16, 8 channels a
// thread, three blocks spill: 32 x 56 x 56 x 512 253 us against 191).
constexpr int gn_blocks(bool bwd, int esize) { return bwd ? (esize == 2 ? 2 : 3) : 4; }

// Calls f(row, x, dy) for the rows first, first + step, ... below n.
template <typename T, int V, int N, bool TWO, typename F>
__device__ __forceinline__ void each_row(const T* x, long long x_ld, const T* dy, long long dy_ld, int first, int step, int n, F f) {
    Raw<T, V> xr[2][N], dr[2][TWO ? N : 1];
    auto fetch = [&](int b, int t) {
#pragma unroll
        for (int u = 0; u < N; ++u)
            if (t + u * step < n) {
                xr[b][u].load(x + (t + u * step) * x_ld);
                if (TWO) dr[b][TWO ? u : 0].load(dy + (t + u * step) * dy_ld);
            }
    };
    fetch(0, first);
    for (int t = first; t < n; t += 2 * N * step) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int at = t + b * N * step;
            if (at >= n) break;
            fetch(b ^ 1, at + N * step);
#pragma unroll
            for (int u = 0; u < N; ++u)
                if (at + u * step < n) {
                    float2 v[Raw<T, V>::P], d[Raw<T, V>::P];
                    xr[b][u].get(v);
                    if (TWO) dr[b][TWO ? u : 0].get(d);
                    f(at + u * step, v, d);
                }
        }
    }
}

// The sums of a slab: forward a group's (or channel's) mean and sum of squared differences, backward every
// channel's sums of dz and dz xhat and the groups' of those times w.  Empty slabs write zeros for the channels.
template <typename T, int V, bool BWD, int ACT>
__global__ void __launch_bounds__(GT, gn_blocks(BWD, sizeof(T))) gn_sums_kernel(const __grid_constant__ SeqGnormParams p, int txn, int tyn, int grouped) {
    constexpr int P = Raw<T, V>::P, N = BWD ? AHEAD_BWD : AHEAD;
    extern __shared__ float2 part[];                  // [tyn][txn V]
    const CutPiece cut = cut_piece(p.ax, blockIdx.x, p.slab);
    const GnPlace at(V, p.D, txn);
    const int cpg = p.D / p.G;
    float2 a[P], b[P], shift[P];
#pragma unroll
    for (int i = 0; i < P; ++i) a[i] = b[i] = shift[i] = dup(0.f);
    launch_next();
    if (at.on && at.ty < cut.n) {
        const T* x = static_cast<const T*>(p.x) + (long long)cut.t0 * p.x_ld + at.c;
        const T* dy = BWD ? static_cast<const T*>(p.dy) + (long long)cut.t0 * p.dy_ld + at.c : nullptr;
        Affine<T, V> f;
        float2 rstd[BWD ? P : 1];
        if (BWD) {
            f.params(p, at.c);
            f.stats(reinterpret_cast<const float2*>(p.stats) + (long long)cut.s * p.G, at.c, cpg, rstd);
        } else {
            Raw<T, V> r;
            r.load(x + at.ty * p.x_ld);
            r.get(shift);
        }
        int n = 0;
        each_row<T, V, N, BWD>(x, p.x_ld, dy, p.dy_ld, at.ty, tyn, cut.n, [&](int, float2 (&v)[P], float2 (&d)[P]) {
            ++n;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                if (BWD) {
                    const float2 e = add2(v[i], neg2(f.mean[i])), dz = mul2(d[i], slope_of<ACT>(fma2(e, f.a[i], f.b[i])));
                    a[i] = add2(a[i], dz);
                    b[i] = fma2(dz, e, b[i]);
                } else {
                    const float2 e = add2(v[i], neg2(shift[i]));
                    a[i] = add2(a[i], e);
                    b[i] = fma2(e, e, b[i]);
                }
            }
        });
        if (BWD) {
#pragma unroll
            for (int i = 0; i < P; ++i) b[i] = mul2(b[i], rstd[BWD ? i : 0]);
        } else {                                      // mean and squared differences from it
            const float r = 1.f / (float)n;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const float2 m = mul2(a[i], dup(r)), q = fma2(neg2(a[i]), m, b[i]);
                b[i] = make_float2(q.x < 0.f ? 0.f : q.x, q.y < 0.f ? 0.f : q.y);
                a[i] = add2(shift[i], m);
            }
        }
    }
    const int width = txn * V, c0 = blockIdx.y * width, wide = min(width, p.D - c0);
#pragma unroll
    for (int i = 0; i < P; ++i) {
        float2* to = part + at.ty * width + at.tx * V + 2 * i;
        if (at.ty < tyn) {
            to[0] = make_float2(a[i].x, b[i].x);
            if (V > 1) to[1] = make_float2(a[i].y, b[i].y);
        }
    }
    __syncthreads();
    // the rows of threads in order; forward: row r has the tokens r, r + tyn, ... of the slab
    for (int j = threadIdx.x; j < wide; j += blockDim.x) {
        float2 s = part[j];
        float sn = (float)((cut.n + tyn - 1) / tyn);
        for (int r = 1; r < tyn && (BWD || r < cut.n); ++r) {
            const float2 o = part[r * width + j];
            if (BWD) {
                s = add2(s, o);
            } else {
                const float on = (float)((cut.n - r + tyn - 1) / tyn), all = sn + on, d = o.x - s.x;
                s.x = fmaf(d, on / all, s.x);
                s.y += o.y + d * d * (sn * on / all);
                sn = all;
            }
        }
        if (BWD || !grouped) reinterpret_cast<float2*>(p.part)[(long long)blockIdx.x * p.D + c0 + j] = cut.n > 0 ? s : dup(0.f);
        if (BWD && grouped && p.w) {
            const float w = seq_ld(static_cast<const T*>(p.w) + c0 + j);
            s = make_float2(s.x * w, s.y * w);
        }
        part[j] = s;
    }
    if (!grouped) return;
    __syncthreads();
    // channels of equal counts to groups: a warp a group, or a thread
    float2* to = reinterpret_cast<float2*>(p.gpart) + (long long)blockIdx.x * p.G + c0 / cpg;
    const int groups = wide / cpg;
    if (cpg <= 4) {
        for (int gi = threadIdx.x; gi < groups; gi += blockDim.x) {
            float2 s = part[gi * cpg];
            for (int c = 1; c < cpg; ++c) {
                const float2 o = part[gi * cpg + c];
                if (BWD) {
                    s = add2(s, o);
                } else {
                    const float d = o.x - s.x, share = 1.f / (float)(c + 1);
                    s.x = fmaf(d, share, s.x);
                    s.y += o.y + d * d * ((float)cut.n * (float)c * share);
                }
            }
            to[gi] = s;
        }
        return;
    }
    const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;      // (a last part of a warp takes none)
    if (threadIdx.x >> 5 >= warps) return;
    for (int gi = threadIdx.x >> 5; gi < groups; gi += warps) {
        float2 s = dup(0.f);
        const float about = BWD ? 0.f : part[gi * cpg].x;
        for (int c = lane; c < cpg; c += 32) {
            const float2 o = part[gi * cpg + c];
            s = add2(s, make_float2(o.x - about, o.y));
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) s = add2(s, make_float2(__shfl_xor_sync(0xffffffffu, s.x, d), __shfl_xor_sync(0xffffffffu, s.y, d)));
        if (!BWD) {
            const float off = s.x / (float)cpg;
            float q = 0.f;
            for (int c = lane; c < cpg; c += 32) {
                const float d = (part[gi * cpg + c].x - about) - off;
                q = fmaf(d, d, q);
            }
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) q += __shfl_xor_sync(0xffffffffu, q, d);
            s = make_float2(about + off, fmaf((float)cut.n, q, s.y));
        }
        if (lane == 0) to[gi] = s;
    }
}

// A sequence's groups from its slabs' entries: forward mean and rstd, backward the means of dz w and dz w xhat.
template <bool BWD>
__device__ __forceinline__ void join_store(const SeqGnormParams& p, long long at, float2 st) {
    reinterpret_cast<float2*>(p.coef)[at] = st;
    if (!BWD && p.stats) reinterpret_cast<float2*>(p.stats)[at] = st;
}
// Parts joined.  Forward: number, mean (less the first entry's, `about`) and sum of squared differences of the values in them; of several parts first
// the mean of all, then M2 = sum (M2k + nk (mean k - mean)^2), whose terms are positive: it keeps its relative accuracy wherever the parts' means
// lie (sums of d and d^2 about one entry, subtracted at the end, were off by 4e-3 with one channel of 4096 far from the others).  Backward: two sums.
template <bool BWD>
struct Joined {
    float n, a, b;
    __device__ __forceinline__ float2 finish(const SeqGnormParams& p, float about, float count) const {
        if (BWD) return make_float2(a / count, b / count);
        return make_float2(about + a, 1.f / sqrtf(b / count + p.eps));
    }
};
// `each` calls its argument with (n, a, b) of every part; forward twice.
template <bool BWD, typename Each>
__device__ __forceinline__ Joined<BWD> joined_of(Each each) {
    Joined<BWD> s = {};
    if (BWD) {
        each([&](float, float a, float b) {
            s.a += a;
            s.b += b;
        });
        return s;
    }
    each([&](float n, float a, float) {
        s.n += n;
        s.a = fmaf(n, a, s.a);
    });
    s.a = s.n > 0.f ? s.a / s.n : 0.f;
    each([&](float n, float a, float b) {
        const float d = a - s.a;
        s.b += fmaf(n * d, d, b);
    });
    return s;
}
// Entries of groups: a block 32 neighbouring groups of a sequence, a warp every eighth slab.
template <bool BWD>
__global__ void __launch_bounds__(GT) gn_join_groups_kernel(const __grid_constant__ SeqGnormParams p, int blocks) {
    __shared__ Joined<BWD> buf[GT];
    const int s = blockIdx.x / blocks, gi = (blockIdx.x - s * blocks) * 32 + (threadIdx.x & 31), cpg = p.D / p.G;
    const int t0 = p.ax.L > 0 ? s * p.ax.L : seq_start(p.ax, s, 0), t1 = p.ax.L > 0 ? t0 + p.ax.L : seq_start(p.ax, s + 1, t0);
    const int len = t1 - t0, slabs = (len + p.slab - 1) / p.slab;
    const float2* from = reinterpret_cast<const float2*>(p.gpart) + (long long)cut_base(p.ax, s, p.slab) * p.G + gi;
    const float tokens = (float)p.slab * (float)cpg, rest = (float)(len - (slabs - 1) * p.slab) * (float)cpg, count = (float)len * (float)cpg;
    launch_next();
    wait_before();
    const float about = !BWD && gi < p.G && len > 0 ? from[0].x : 0.f;
    buf[threadIdx.x] = joined_of<BWD>([&](auto part) {
        if (gi < p.G)
#pragma unroll 4
            for (int k = threadIdx.x >> 5; k < slabs; k += GT / 32) {
                const float2 v = from[(long long)k * p.G];
                part(k == slabs - 1 ? rest : tokens, v.x - about, v.y);
            }
    });
    __syncthreads();
    if (threadIdx.x < 32 && gi < p.G) {
        const Joined<BWD> st = joined_of<BWD>([&](auto part) {
#pragma unroll
            for (int w = 0; w < GT / 32; ++w) part(buf[w * 32 + threadIdx.x].n, buf[w * 32 + threadIdx.x].a, buf[w * 32 + threadIdx.x].b);
        });
        join_store<BWD>(p, (long long)s * p.G + gi, len > 0 ? st.finish(p, about, count) : dup(0.f));
    }
}
// Entries of channels (groups so wide that they lie in several blocks of the sums): a block a sequence and group.
template <typename T, bool BWD>
__global__ void __launch_bounds__(GT) gn_join_channels_kernel(const __grid_constant__ SeqGnormParams p) {
    __shared__ Joined<BWD> buf[GT];
    const long long at = blockIdx.x;
    const int s = (int)(at / p.G), gi = (int)(at - (long long)s * p.G), cpg = p.D / p.G;
    const int t0 = p.ax.L > 0 ? s * p.ax.L : seq_start(p.ax, s, 0), t1 = p.ax.L > 0 ? t0 + p.ax.L : seq_start(p.ax, s + 1, t0);
    const int len = t1 - t0, slabs = (len + p.slab - 1) / p.slab;
    const float2* from = reinterpret_cast<const float2*>(p.part) + (long long)cut_base(p.ax, s, p.slab) * p.D + gi * cpg;
    const T* w = BWD ? static_cast<const T*>(p.w) : nullptr;
    const float tokens = (float)p.slab, rest = (float)(len - (slabs - 1) * p.slab), count = (float)len * (float)cpg;
    launch_next();
    wait_before();
    const float about = !BWD && len > 0 ? from[0].x : 0.f;
    buf[threadIdx.x] = joined_of<BWD>([&](auto part) {
        for (int c = threadIdx.x; c < cpg; c += GT) {
            const float wc = w ? seq_ld(w + gi * cpg + c) : 1.f;
#pragma unroll 4
            for (int k = 0; k < slabs; ++k) {
                const float2 v = from[(long long)k * p.D + c];
                part(k == slabs - 1 ? rest : tokens, BWD ? wc * v.x : v.x - about, BWD ? wc * v.y : v.y);
            }
        }
    });
    __syncthreads();
    // 256 parts to 32, to one
    auto fold = [&](int parts, int step) {
        return joined_of<BWD>([&](auto part) {
            for (int i = threadIdx.x; i < parts; i += step) part(buf[i].n, buf[i].a, buf[i].b);
        });
    };
    if (threadIdx.x >= 32) return;
    const Joined<BWD> st = fold(GT, 32);
    __syncwarp();
    buf[threadIdx.x] = st;
    __syncwarp();
    if (threadIdx.x == 0) join_store<BWD>(p, at, len > 0 ? fold(32, 1).finish(p, about, count) : dup(0.f));
}

// dw and db: the slabs' sums of all sequences in order.  It runs beside the kernel before it in the stream, which lets it go
// once those sums are complete.
__global__ void __launch_bounds__(COLUMN_THREADS, 2) gn_param_kernel(const __grid_constant__ SeqGnormParams p) {
    const long long col = (long long)blockIdx.x * 32 + (threadIdx.x & 31);      // db and dw of a channel side by side
    const bool on = col < 2LL * p.D;
    const float v = column_sum(p.part + col, 2LL * p.D, p.slots, on);
    if (threadIdx.x < 32 && on) {
        float* to = col & 1 ? p.dw : p.db;
        if (to) to[col >> 1] = v;
    }
    wait_before();                  // (so that what follows in the stream follows the kernel before, too)
}

// The same by every block for its own channels: `groups` of a sequence from g0 on, to `to` (shared memory; `buf`: an entry a thread).
template <bool BWD>
__device__ __forceinline__ void join_groups(const SeqGnormParams& p, const CutPiece& cut, int g0, int groups, float2* to, Joined<BWD>* buf) {
    const int parts = blockDim.x / groups, gi = threadIdx.x % groups, k0 = threadIdx.x / groups, cpg = p.D / p.G;
    const int t0 = cut.t0 - cut.index * p.slab, t1 = p.ax.L > 0 ? t0 + p.ax.L : seq_start(p.ax, cut.s + 1, t0);
    const int len = t1 - t0, slabs = (len + p.slab - 1) / p.slab;
    const float2* from = reinterpret_cast<const float2*>(p.gpart) + (long long)cut_base(p.ax, cut.s, p.slab) * p.G + g0 + gi;
    const float tokens = (float)p.slab * (float)cpg, rest = (float)(len - (slabs - 1) * p.slab) * (float)cpg, count = (float)len * (float)cpg;
    // A thread's 16 or so in one pass, as differences from its first: what subtracting their mean loses goes with their number.
    float about = 0.f;
    if (k0 < parts) {
        if (!BWD) about = from[0].x;
        const float first = !BWD && k0 < slabs ? from[(long long)k0 * p.G].x : 0.f;
        Joined<BWD> st = {};
#pragma unroll 4
        for (int k = k0; k < slabs; k += parts) {
            const float2 v = from[(long long)k * p.G];
            if (BWD) {
                st.a += v.x;
                st.b += v.y;
            } else {
                const float d = v.x - first, n = k == slabs - 1 ? rest : tokens;
                st.n += n;
                st.a = fmaf(n, d, st.a);
                st.b += fmaf(n * d, d, v.y);
            }
        }
        if (!BWD && st.n > 0.f) {
            const float mean = st.a / st.n, m2 = fmaf(-st.a, mean, st.b);
            st.b = m2 < 0.f ? 0.f : m2;
            st.a = (first - about) + mean;
        }
        buf[threadIdx.x] = st;
    }
    __syncthreads();
    if (threadIdx.x < groups) {
        const Joined<BWD> st = joined_of<BWD>([&](auto part) {
#pragma unroll 4
            for (int k = 0; k < parts; ++k) part(buf[k * groups + threadIdx.x].n, buf[k * groups + threadIdx.x].a, buf[k * groups + threadIdx.x].b);
        });
        const float2 all = st.finish(p, about, count);
        if (!BWD && p.stats && cut.index == 0) reinterpret_cast<float2*>(p.stats)[(long long)cut.s * p.G + g0 + threadIdx.x] = all;
        to[threadIdx.x] = all;
    }
    __syncthreads();
}

// y, or dx, of a slab.  SELF: the block joins its groups' entries itself.
template <typename T, int V, bool BWD, int ACT, bool SELF>
__global__ void __launch_bounds__(GT, gn_blocks(BWD, sizeof(T))) gn_apply_kernel(const __grid_constant__ SeqGnormParams p, int txn, int tyn) {
    constexpr int P = Raw<T, V>::P, N = BWD ? AHEAD_BWD : AHEAD;
    __shared__ float2 joined[SELF ? GT : 1];
    __shared__ Joined<BWD> buf[SELF ? GT : 1];
    const CutPiece cut = cut_piece(p.ax, gridDim.x - 1 - blockIdx.x, p.slab);
    const GnPlace at(V, p.D, txn);
    const bool on = at.on && at.ty < tyn && at.ty < cut.n;
    const int cpg = p.D / p.G;
    Affine<T, V> f;
    if (on) f.params(p, at.c);
    wait_before();
    if (BWD) launch_next();         // the parameters' sums: see gn_param_kernel
    if (SELF) {
        const int g0 = blockIdx.y * txn * V / cpg, groups = min(txn * V, p.D - blockIdx.y * txn * V) / cpg;
        if (cut.n <= 0) {           // (a first piece without tokens: an empty sequence; each has a slot of its own)
            if (!BWD && p.stats && cut.index == 0)
                for (int gi = threadIdx.x; gi < groups; gi += blockDim.x) reinterpret_cast<float2*>(p.stats)[(long long)cut.s * p.G + g0 + gi] = dup(0.f);
            return;
        }
        join_groups<BWD>(p, cut, g0, groups, joined, buf);
    }
    if (!on) return;
    float2 c1[BWD ? P : 1], c2[BWD ? P : 1], rstd[BWD ? P : 1];
    const long long first = (long long)cut.s * p.G;
    const float2* join = SELF ? joined - blockIdx.y * txn * V / cpg : reinterpret_cast<const float2*>(p.coef) + first;
    f.stats(BWD ? reinterpret_cast<const float2*>(p.stats) + first : join, at.c, cpg, BWD ? rstd : nullptr);
    if (BWD) {                                        // dx = rstd w dz - rstd m1 - (x - mean) rstd^2 m2
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const float2 m0 = join[(at.c + 2 * i) / cpg], m1 = V > 1 ? join[(at.c + 2 * i + 1) / cpg] : m0;
            const float2 r = rstd[BWD ? i : 0];
            c1[BWD ? i : 0] = mul2(make_float2(-m0.x, -m1.x), r);
            c2[BWD ? i : 0] = mul2(make_float2(-m0.y, -m1.y), mul2(r, r));
        }
        // a group of one value is its mean, whatever it is: no gradient, and not what is left of terms that cancel
        const int from = p.ax.L > 0 ? 0 : seq_start(p.ax, cut.s, 0);
        if (cpg == 1 && (p.ax.L > 0 ? p.ax.L : seq_start(p.ax, cut.s + 1, from) - from) == 1) {
#pragma unroll
            for (int i = 0; i < P; ++i) f.a[i] = c1[BWD ? i : 0] = c2[BWD ? i : 0] = dup(0.f);
        }
    }
    const T* x = static_cast<const T*>(p.x) + (long long)cut.t0 * p.x_ld + at.c;
    const T* dy = BWD ? static_cast<const T*>(p.dy) + (long long)cut.t0 * p.dy_ld + at.c : nullptr;
    T* to = static_cast<T*>(BWD ? p.dx : p.y) + (long long)cut.t0 * (BWD ? p.dx_ld : p.y_ld) + at.c;
    const long long to_ld = BWD ? p.dx_ld : p.y_ld;
    each_row<T, V, N, BWD>(x, p.x_ld, dy, p.dy_ld, at.ty, tyn, cut.n, [&](int t, float2 (&v)[P], float2 (&d)[P]) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const float2 e = add2(v[i], neg2(f.mean[i])), z = fma2(e, f.a[i], f.b[i]);
            if (BWD) {
                const float2 r = fma2(e, c2[BWD ? i : 0], c1[BWD ? i : 0]);
                v[i] = fma2(f.a[i], mul2(d[i], slope_of<ACT>(z)), r);
            } else {
                v[i] = act_of<ACT>(z);
            }
        }
        put<T, V>(to + t * to_ld, v);
    });
}

// Few entries: every block of the apply pass joins its groups' itself, one launch less.  By the slabs that a sequence may have, all of them where
// lengths are not known: by their mean, the blocks of one long sequence among many short ones each joined all of its slabs (2,000,000 tokens
// behind 20,000 of one, 32 channels fp32: 1502 us, 1135 this way; no more than a launch lost elsewhere: 27 against 29).
bool gn_self(const SeqGnormParams& p, const GnShape& s, int V) {
    const long long own = s.tx * V / (p.D / p.G), slabs = (p.ax.L > 0 ? p.ax.L : p.ax.T) / p.slab + 1;       // groups of a block
    return s.grouped && own <= s.tx * s.ty && own * slabs <= 16 * GT;
}
template <typename T, int V, bool BWD, int ACT>
cudaError_t launch_act(const SeqGnormParams& p, cudaStream_t stream) {
    const GnShape s = gn_shape(p.D, p.D / p.G, V);
    const dim3 grid((unsigned)p.slots, (unsigned)s.cblocks), block((unsigned)(s.tx * s.ty));
    cudaError_t e = launch_kernel(gn_sums_kernel<T, V, BWD, ACT>, grid, block, (size_t)s.tx * s.ty * V * sizeof(float2), stream, false, 1, p, s.tx, s.ty, s.grouped);
    if (e != cudaSuccess) return e;
    const long long groups = (long long)p.ax.S * p.G;
    const bool self = gn_self(p, s, V);
    if (!self) {
        const int each = (p.G + 31) / 32;
        if (s.grouped) e = launch_kernel(gn_join_groups_kernel<BWD>, dim3((unsigned)(p.ax.S * (long long)each)), dim3(GT), 0, stream, true, 1, p, each);
        else e = launch_kernel(gn_join_channels_kernel<T, BWD>, dim3((unsigned)groups), dim3(GT), 0, stream, true, 1, p);
    }
    if (e == cudaSuccess)
        e = launch_kernel(self ? gn_apply_kernel<T, V, BWD, ACT, true> : gn_apply_kernel<T, V, BWD, ACT, false>, grid, block, 0, stream, true, 1, p, s.tx, s.ty);
    if (BWD && e == cudaSuccess && (p.dw || p.db))
        e = launch_kernel(gn_param_kernel, dim3((unsigned)((2LL * p.D + 31) / 32)), dim3(COLUMN_THREADS), 0, stream, true, 1, p);
    return e;
}
template <typename T, int V, bool BWD>
cudaError_t launch_v(const SeqGnormParams& p, cudaStream_t stream) {
    if (p.act == SEQ_ACT_SILU) return launch_act<T, V, BWD, SEQ_ACT_SILU>(p, stream);
    if (p.act == SEQ_ACT_GELU) return launch_act<T, V, BWD, SEQ_ACT_GELU>(p, stream);
    return launch_act<T, V, BWD, SEQ_ACT_NONE>(p, stream);
}
template <typename T, bool BWD>
cudaError_t launch(const SeqGnormParams& p, cudaStream_t stream) {
    if (p.slots == 0) return cudaSuccess;
    if (p.grain == 16) return launch_v<T, 16 / sizeof(T), BWD>(p, stream);
    return p.grain ? launch_v<T, 2, BWD>(p, stream) : launch_v<T, 1, BWD>(p, stream);
}

}  // namespace

// Tokens of a slab: those of one round of blocks, but 16 rows a thread while every SM has a block (a block's first loads and
// its part of the joining cost about as much as ten), 4 rows at least and 128 at most.
int seq_gnorm_slab(long long S, long long T, int D, int G, int esize, bool bwd, int sms) {
    const GnShape s = gn_shape(D, D / G, 16 / esize);
    const long long L = S > 0 && T > S ? T / S : 1, rows = (S < 1 ? 1 : S) * s.cblocks;
    const long long round = (long long)(esize == 4 ? 4 : gn_blocks(bwd, esize)) * GT * sms / (s.tx * s.ty);
    auto tokens = [&](long long blocks) { return (L + (blocks < rows ? 1 : blocks / rows) - 1) / (blocks < rows ? 1 : blocks / rows); };
    long long len = tokens(round);
    const long long enough = 16 * s.ty < tokens(sms) ? 16 * s.ty : tokens(sms);
    if (len < enough) len = enough;
    if (len < 4 * s.ty) len = 4 * s.ty;
    if (len > 128 * s.ty) len = 128 * s.ty;
    return (int)len;
}

cudaError_t launch_seq_gnorm_fwd(const SeqGnormParams& p, bool bf16, cudaStream_t stream) {
    return bf16 ? launch<__nv_bfloat16, false>(p, stream) : launch<float, false>(p, stream);
}
cudaError_t launch_seq_gnorm_bwd(const SeqGnormParams& p, bool bf16, cudaStream_t stream) {
    return bf16 ? launch<__nv_bfloat16, true>(p, stream) : launch<float, true>(p, stream);
}

}  // namespace convfwd

// C-ABI of the sequence-mixing operators: plans, argument checks, workspace layout.  Declarations
// and the contract of every entry point are in include/seq.h.
#include <stdio.h>

#include <new>

#include "seq_internal.h"

using namespace convfwd;

namespace {

enum class Op { Conv, Scan, Norm };

constexpr int64_t MAX_EXTENT = (int64_t)1 << 30;     // tokens: sums of two token indices stay in 32 bits
constexpr int64_t MAX_CHANNELS = (int64_t)1 << 22;   // channel blocks are a launch's second dimension

int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        (void)cudaGetLastError();
        return 152;
    }
    return n;
}

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace

struct seq_plan {
    Op op;
    seq_direction dir;
    conv_dtype dtype, res_dtype;
    unsigned flags;
    int S, T, D, L;        // L: tokens per sequence, 0 when ragged (or T = 0)
    int W, N, G;
    int run;               // conv: tokens a thread walks
    int sms;
    ScanPieces pc;
    int blocks;            // conv backward: token blocks; scan backward: channel blocks; norm backward: partial rows
    size_t ws_bytes;
    void* ws;
    float eps;
    char desc[256];

    bool ragged() const { return flags & SEQ_RAGGED; }
    size_t esize() const { return dtype == CONV_BF16 ? 2 : 4; }
    size_t rsize() const { return res_dtype == CONV_BF16 ? 2 : 4; }
    SeqAxis axis(const int32_t* starts) const { return SeqAxis{S, T, L, starts}; }
};

namespace {

bool bad_dtype(conv_dtype d) { return d != CONV_F32 && d != CONV_BF16; }
bool bad_dir(seq_direction d) { return d != SEQ_FWD && d != SEQ_BWD && d != SEQ_STEP; }
const char* dir_name(seq_direction d) { return d == SEQ_FWD ? "fwd" : d == SEQ_BWD ? "bwd" : "step"; }
const char* type_name(conv_dtype d) { return d == CONV_BF16 ? "bf16" : "f32"; }

conv_status check_axis(int64_t S, int64_t T, int64_t D, seq_direction dir, bool ragged) {
    if (S < 1 || T < 0 || D < 1) return CONV_ERR_INVALID_ARG;
    if (S > MAX_EXTENT || T > MAX_EXTENT || D > MAX_CHANNELS) return CONV_ERR_UNSUPPORTED;
    if (!ragged && T % S != 0) return CONV_ERR_INVALID_ARG;
    if (dir == SEQ_STEP && (T != S || ragged)) return CONV_ERR_INVALID_ARG;
    return CONV_OK;
}

seq_plan* new_plan(Op op, int64_t S, int64_t T, int64_t D, conv_dtype dtype, seq_direction dir, unsigned flags) {
    seq_plan* p = new (std::nothrow) seq_plan();
    if (!p) return nullptr;
    p->op = op; p->dir = dir; p->dtype = p->res_dtype = dtype; p->flags = flags;
    p->S = (int)S; p->T = (int)T; p->D = (int)D;
    p->L = p->ragged() ? 0 : (int)(T / S);
    p->sms = sm_count();
    return p;
}

// A tensor argument: present, aligned to its element, rows wide enough.  `wide` stays true while
// every tensor that the kernels read or write in groups of elements lies in 16-byte aligned rows; what they read
// one element at a time (`Elements`: bounds, slots, parameter gradients, the scan's B and C, ...) has no part in it.
struct Checker {
    enum Access { Groups, Elements };
    conv_status st = CONV_OK;
    bool wide = true, words = true;      // words: 4-byte aligned rows
    void fail(conv_status s) { if (st == CONV_OK) st = s; }
    void ptr(const void* v, size_t esize, bool needed, Access access = Elements, size_t align = 0) {
        if (!v) {
            if (needed) fail(CONV_ERR_INVALID_ARG);
            return;
        }
        const uintptr_t a = reinterpret_cast<uintptr_t>(v);
        if (a % (align ? align : esize)) fail(CONV_ERR_ALIGNMENT);
        if (access == Elements) return;
        if (a % 16) wide = false;
        if (a % 4) words = false;
    }
    void rows(const void* v, int64_t ld, int64_t width, size_t esize, bool needed = true, Access access = Groups) {
        ptr(v, esize, needed, access);
        if (!v) return;
        if (ld < width) fail(CONV_ERR_INVALID_ARG);
        if (ld > INT32_MAX) fail(CONV_ERR_UNSUPPORTED);      // the kernels multiply it in 32 bits by 32
        if (access == Elements) return;
        if (((uint64_t)ld * esize) % 16) wide = false;
        if (((uint64_t)ld * esize) % 4) words = false;
    }
};

conv_status finish(cudaError_t e) { return e == cudaSuccess ? CONV_OK : CONV_ERR_CUDA; }

conv_status check_call(seq_plan_t p, const void* args, Op op, seq_direction dir) {
    if (!p || !args || p->op != op || p->dir != dir) return CONV_ERR_INVALID_ARG;
    return CONV_OK;
}

// starts goes with the plan's kind of axis; the state buffers with their slots.
void check_states(const seq_plan* p, Checker& c, const int32_t* starts, const int32_t* slots, int64_t slot_count,
                  const void* in, const void* out, size_t esize, Checker::Access access) {
    if (p->ragged() ? !starts : starts != nullptr) c.fail(CONV_ERR_INVALID_ARG);
    c.ptr(starts, 4, false);
    c.ptr(slots, 4, false);
    c.ptr(in, esize, false, access);
    c.ptr(out, esize, false, access);
    if (slot_count > MAX_EXTENT) c.fail(CONV_ERR_UNSUPPORTED);
    if ((in || out) && (slot_count < 0 || (!slots && slot_count < p->S))) c.fail(CONV_ERR_INVALID_ARG);
}

// How many pieces the scan cuts a sequence (a ragged axis) of `axis` tokens into.  `base` thread
// blocks walk one piece of every sequence and all channels; `slots` of them keep the GPU busy.  Uncut,
// a block walks all tokens in order; cut, `again` of the work is done twice, for the states between the
// pieces, and joining the pieces costs about as much as `join` tokens a piece.  The estimate: waves of blocks, times
// the work of a block.  (5003 x 770 x 12 ragged fp32: 79 us in 105 pieces of 48 tokens, 97 in 63 of 80.)
ScanPieces scan_pieces(const seq_plan* p, int blocks, int slots, float again, float join) {
    const int shortest = 32, most_pieces = 128;      // (128: what the joining kernel can take)
    const long long axis = p->L > 0 ? p->L : p->T;
    const long long base = p->L > 0 ? (long long)p->S * blocks : blocks;
    long long best_len = 0;
    float best = 0.f;
    for (int n = 1; n <= most_pieces; ++n) {
        long long len = ((axis + n - 1) / n + SCAN_TILE - 1) / SCAN_TILE * SCAN_TILE;
        if (len < SCAN_TILE) len = SCAN_TILE;
        if (n > 1 && len < shortest) break;
        const long long count = (axis + len - 1) / len;
        const long long waves = (base * (count < 1 ? 1 : count) + slots - 1) / slots;
        const float cost = (float)waves * ((float)len * (count > 1 ? 1.f + again : 1.f) + join * (float)count);
        if (!best_len || cost < best) {
            best = cost;
            best_len = len;
        }
    }
    ScanPieces pc = {1, (int)best_len, 0};
    const long long n = (axis + best_len - 1) / best_len < 1 ? 1 : (axis + best_len - 1) / best_len;
    if (p->L > 0) {
        pc.pps = (int)n;
        pc.count = (int)(n * p->S);
    } else {
        pc.count = (int)n;
    }
    return pc;
}

int scan_fwd_blocks(int D, int N, int G) {
    const int ln = N <= 16 ? 1 : N <= 32 ? 2 : N <= 64 ? 4 : 8, cb = 128 / ln, per = D / G;
    return G * ((per + cb - 1) / cb);
}

// Floats of a token's partial dB and dC in the backward workspace: states padded as the kernel's lanes hold them.
size_t scan_bc_row(const seq_plan* p) { return 2 * (size_t)(p->N <= 8 ? 8 : p->N <= 16 ? 16 : p->N <= 32 ? 32 : p->N <= 64 ? 64 : 128); }

size_t scan_state_row(const seq_plan* p) { return (size_t)((p->N + 3) / 4) * 4 * p->D; }   // floats

}  // namespace

extern "C" {

const char* seq_plan_describe(seq_plan_t plan) { return plan ? plan->desc : ""; }
size_t seq_workspace_bytes(seq_plan_t plan) { return plan ? plan->ws_bytes : 0; }

conv_status seq_plan_set_workspace(seq_plan_t plan, void* workspace, size_t bytes) {
    if (!plan) return CONV_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(workspace) % 16) return CONV_ERR_ALIGNMENT;
    if (plan->ws_bytes && (!workspace || bytes < plan->ws_bytes)) return CONV_ERR_WORKSPACE;
    plan->ws = workspace;
    return CONV_OK;
}

conv_status seq_plan_destroy(seq_plan_t plan) {
    delete plan;
    return CONV_OK;
}

// ------------------------------------------------------------------------------- convolution
conv_status seq_conv_plan_create(seq_plan_t* out, int64_t S, int64_t T, int64_t D, int64_t W, conv_dtype dtype,
                                 seq_direction direction, unsigned flags) {
    if (!out || bad_dtype(dtype) || bad_dir(direction) || W < 1 || (flags & ~(unsigned)(SEQ_RAGGED | SEQ_CONV_SILU)))
        return CONV_ERR_INVALID_ARG;
    const conv_status st = check_axis(S, T, D, direction, flags & SEQ_RAGGED);
    if (st != CONV_OK) return st;
    if (W > 8) return CONV_ERR_UNSUPPORTED;
    seq_plan* p = new_plan(Op::Conv, S, T, D, dtype, direction, flags);
    if (!p) return CONV_ERR_INVALID_ARG;
    p->W = (int)W;
    p->run = seq_conv_run(T, p->D, p->W, dtype == CONV_BF16, direction == SEQ_BWD, p->sms);
    if (direction == SEQ_BWD) {
        p->blocks = seq_conv_bwd_token_blocks(T, p->run);
        p->ws_bytes = align256((size_t)(p->blocks > 0 ? p->blocks : 1) * (W + 1) * D * sizeof(float));
    }
    snprintf(p->desc, sizeof p->desc, "op=conv direction=%s dtype=%s sequences=%d tokens=%d ragged=%d width=%d taps=%d silu=%d run=%d blocks=%d",
             dir_name(direction), type_name(dtype), p->S, p->T, p->ragged(), p->D, p->W, !!(flags & SEQ_CONV_SILU), p->run, p->blocks);
    *out = p;
    return CONV_OK;
}

static conv_status conv_call(seq_plan_t p, const seq_conv_args* a, seq_direction dir, void* stream) {
    conv_status st = check_call(p, a, Op::Conv, dir);
    if (st != CONV_OK) return st;
    Checker c;
    const size_t e = p->esize();
    const bool bwd = dir == SEQ_BWD, any = p->T > 0;
    c.rows(a->x, a->x_ld, p->D, e, any);
    c.ptr(a->w, e, true);
    c.ptr(a->bias, e, false);
    check_states(p, c, a->starts, a->slots, a->slot_count, a->state_in, bwd ? nullptr : a->state_out, e, Checker::Groups);
    if (p->W == 1 && !bwd && a->state_out) c.fail(CONV_ERR_INVALID_ARG);
    if (!bwd) {
        c.rows(a->y, a->y_ld, p->D, e, any);
    } else {
        c.rows(a->dy, a->dy_ld, p->D, e, any);
        c.rows(a->dx, a->dx_ld, p->D, e, any);
        c.ptr(a->dw, 4, true);
        c.ptr(a->dbias, 4, false);
        if (a->dbias && !a->bias) c.fail(CONV_ERR_INVALID_ARG);
    }
    if (c.st != CONV_OK) return c.st;
    if (bwd && !p->ws) return CONV_ERR_WORKSPACE;
    SeqConvParams q = {};
    q.ax = p->axis(a->starts);
    q.sl = SeqSlots{a->slots, a->slot_count};
    q.D = p->D; q.W = p->W; q.silu = !!(p->flags & SEQ_CONV_SILU);
    q.x = a->x; q.w = a->w; q.bias = a->bias; q.state_in = a->state_in; q.state_out = a->state_out; q.y = a->y;
    q.dy = a->dy; q.dx = a->dx; q.dw = a->dw; q.dbias = a->dbias;
    q.x_ld = a->x_ld; q.y_ld = a->y_ld; q.dy_ld = a->dy_ld; q.dx_ld = a->dx_ld;
    q.ws = static_cast<float*>(p->ws);
    q.run = p->run;
    q.tblocks = p->blocks;
    q.vec = c.wide && (p->D * e) % 16 == 0;
    const bool bf16 = p->dtype == CONV_BF16;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return finish(dir == SEQ_FWD ? launch_seq_conv_fwd(q, bf16, s) : bwd ? launch_seq_conv_bwd(q, bf16, s)
                                                                        : launch_seq_conv_step(q, bf16, s));
}
conv_status seq_conv_fwd(seq_plan_t plan, const seq_conv_args* args, void* stream) { return conv_call(plan, args, SEQ_FWD, stream); }
conv_status seq_conv_bwd(seq_plan_t plan, const seq_conv_args* args, void* stream) { return conv_call(plan, args, SEQ_BWD, stream); }
conv_status seq_conv_step(seq_plan_t plan, const seq_conv_args* args, void* stream) { return conv_call(plan, args, SEQ_STEP, stream); }

// ------------------------------------------------------------------------------------- scan
conv_status seq_scan_plan_create(seq_plan_t* out, int64_t S, int64_t T, int64_t D, int64_t N, int64_t G, conv_dtype dtype,
                                 seq_direction direction, unsigned flags) {
    if (!out || bad_dtype(dtype) || bad_dir(direction) || N < 1 || G < 1 || (flags & ~(unsigned)(SEQ_RAGGED | SEQ_SCAN_SOFTPLUS)))
        return CONV_ERR_INVALID_ARG;
    conv_status st = check_axis(S, T, D, direction, flags & SEQ_RAGGED);
    if (st != CONV_OK) return st;
    if (D % G != 0) return CONV_ERR_INVALID_ARG;
    if (N > 128 || G > 32768 || D * N > INT32_MAX) return CONV_ERR_UNSUPPORTED;
    seq_plan* p = new_plan(Op::Scan, S, T, D, dtype, direction, flags);
    if (!p) return CONV_ERR_INVALID_ARG;
    p->N = (int)N; p->G = (int)G;
    p->pc = ScanPieces{1, SCAN_TILE, 0};
    if (direction == SEQ_FWD) {
        const int blocks = scan_fwd_blocks(p->D, p->N, p->G);
        if (blocks > 65535) st = CONV_ERR_UNSUPPORTED;
        p->pc = scan_pieces(p, blocks, 6 * p->sms, 0.75f, 0.5f);
        if (p->pc.pps != 1 && p->pc.count > 1)
            p->ws_bytes = 2 * align256(scan_state_row(p) * p->pc.count * sizeof(float)) +
                          align256((size_t)p->pc.count * D * sizeof(float));
    } else if (direction == SEQ_BWD) {
        p->blocks = seq_scan_bwd_channel_blocks(p->D, p->N, p->G);
        if (p->blocks > 65535) st = CONV_ERR_UNSUPPORTED;
        p->pc = scan_pieces(p, p->blocks, 3 * p->sms, 0.25f, 0.5f);
        p->ws_bytes = align256((size_t)p->blocks * p->T * scan_bc_row(p) * sizeof(float)) +
                      align256((size_t)p->pc.count * (N + 2) * D * sizeof(float));
        if (p->pc.pps != 1 && p->pc.count > 1)
            p->ws_bytes += align256(scan_state_row(p) * p->pc.count * sizeof(float)) + align256((size_t)p->pc.count * D * sizeof(float));
    }
    if (st != CONV_OK) {
        delete p;
        return st;
    }
    snprintf(p->desc, sizeof p->desc,
             "op=scan direction=%s dtype=%s sequences=%d tokens=%d ragged=%d width=%d states=%d groups=%d softplus=%d pieces=%d piece_tokens=%d",
             dir_name(direction), type_name(dtype), p->S, p->T, p->ragged(), p->D, p->N, p->G, !!(flags & SEQ_SCAN_SOFTPLUS),
             p->pc.count, p->pc.len);
    *out = p;
    return CONV_OK;
}

size_t seq_scan_saved_bytes(seq_plan_t p) {
    if (!p || p->op != Op::Scan || p->dir == SEQ_STEP) return 0;
    const size_t rows = p->L > 0 ? (size_t)p->S * ((p->L + SCAN_TILE - 1) / SCAN_TILE) : ((size_t)p->T + SCAN_TILE - 1) / SCAN_TILE;
    return rows * scan_state_row(p) * sizeof(float);
}

static conv_status scan_call(seq_plan_t p, const seq_scan_args* a, seq_direction dir, void* stream) {
    conv_status st = check_call(p, a, Op::Scan, dir);
    if (st != CONV_OK) return st;
    Checker c;
    const size_t e = p->esize();
    const bool bwd = dir == SEQ_BWD, any = p->T > 0;
    const int64_t GN = (int64_t)p->G * p->N;
    c.rows(a->x, a->x_ld, p->D, e, any);
    c.rows(a->dt, a->dt_ld, p->D, e, any);
    c.rows(a->B, a->B_ld, GN, e, any, Checker::Elements);
    c.rows(a->C, a->C_ld, GN, e, any, Checker::Elements);
    c.rows(a->z, a->z_ld, p->D, e, false);
    c.ptr(a->A, 4, true);
    c.ptr(a->D, 4, false);
    c.ptr(a->dt_bias, 4, false);
    check_states(p, c, a->starts, a->slots, a->slot_count, bwd && !a->h_in ? a->dh_in : a->h_in, bwd ? a->dh_out : a->h_out, 4, Checker::Elements);
    if (dir != SEQ_STEP) c.ptr(a->saved, 4, bwd && any, Checker::Elements, 16);
    if (!bwd) {
        c.rows(a->y, a->y_ld, p->D, e, any);
    } else {
        c.rows(a->dy, a->dy_ld, p->D, e, any);
        c.rows(a->dx, a->dx_ld, p->D, e, any);
        c.rows(a->ddt, a->ddt_ld, p->D, e, any);
        c.rows(a->dB, a->dB_ld, GN, e, any, Checker::Elements);
        c.rows(a->dC, a->dC_ld, GN, e, any, Checker::Elements);
        c.rows(a->dz, a->dz_ld, p->D, e, a->z && any);
        c.ptr(a->dA, 4, true);
        c.ptr(a->dD, 4, a->D != nullptr);
        c.ptr(a->ddt_bias, 4, a->dt_bias != nullptr);
        c.ptr(a->dh_in, 4, false);
        if ((a->dz && !a->z) || (a->dD && !a->D) || (a->ddt_bias && !a->dt_bias)) c.fail(CONV_ERR_INVALID_ARG);
    }
    if (c.st != CONV_OK) return c.st;
    if (p->ws_bytes && !p->ws) return CONV_ERR_WORKSPACE;
    SeqScanParams q = {};
    q.ax = p->axis(a->starts);
    q.sl = SeqSlots{a->slots, a->slot_count};
    q.pc = p->pc;
    q.D = p->D; q.N = p->N; q.G = p->G; q.softplus = !!(p->flags & SEQ_SCAN_SOFTPLUS);
    q.x = a->x; q.dt = a->dt; q.B = a->B; q.C = a->C; q.z = a->z; q.dy = a->dy;
    q.A = a->A; q.Dskip = a->D; q.dt_bias = a->dt_bias; q.h_in = a->h_in; q.dh_out = a->dh_out;
    q.y = a->y; q.dx = a->dx; q.ddt = a->ddt; q.dB = a->dB; q.dC = a->dC; q.dz = a->dz;
    q.h_out = a->h_out; q.saved = a->saved; q.dA = a->dA; q.dD = a->dD; q.ddt_bias = a->ddt_bias; q.dh_in = a->dh_in;
    q.x_ld = a->x_ld; q.dt_ld = a->dt_ld; q.B_ld = a->B_ld; q.C_ld = a->C_ld; q.z_ld = a->z_ld; q.y_ld = a->y_ld;
    q.dy_ld = a->dy_ld; q.dx_ld = a->dx_ld; q.ddt_ld = a->ddt_ld; q.dB_ld = a->dB_ld; q.dC_ld = a->dC_ld; q.dz_ld = a->dz_ld;
    q.cblocks = p->blocks;
    q.sms = p->sms;
    auto aligned = [](const void* v, size_t n) { return reinterpret_cast<uintptr_t>(v) % n == 0; };
    q.quads = p->N % 4 == 0 && aligned(a->A, 16);
    if (dir == SEQ_STEP)
        q.quads = q.quads && aligned(a->h_in, 16) && aligned(a->h_out, 16) && aligned(a->B, 4 * e) && aligned(a->C, 4 * e) &&
                  a->B_ld % 4 == 0 && a->C_ld % 4 == 0;
    q.wide = c.wide && (p->D / p->G * e) % 16 == 0 ? 16 : c.words && (p->D / p->G * e) % 4 == 0 ? 4 : 0;
    unsigned char* w = static_cast<unsigned char*>(p->ws);
    if (dir == SEQ_FWD && p->ws_bytes) {
        const size_t row = align256(scan_state_row(p) * p->pc.count * sizeof(float));
        q.piece_state = reinterpret_cast<float*>(w);
        q.piece_init = reinterpret_cast<float*>(w + row);
        q.piece_delta = reinterpret_cast<float*>(w + 2 * row);
    } else if (bwd) {
        q.part_bc = reinterpret_cast<float*>(w);
        w += align256((size_t)p->blocks * p->T * scan_bc_row(p) * sizeof(float));
        q.part_par = reinterpret_cast<float*>(w);
        w += align256((size_t)p->pc.count * (p->N + 2) * p->D * sizeof(float));
        q.piece_state = reinterpret_cast<float*>(w);
        q.piece_delta = reinterpret_cast<float*>(w + align256(scan_state_row(p) * p->pc.count * sizeof(float)));
    }
    const bool bf16 = p->dtype == CONV_BF16;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return finish(dir == SEQ_FWD ? launch_seq_scan_fwd(q, bf16, s) : bwd ? launch_seq_scan_bwd(q, bf16, s)
                                                                        : launch_seq_scan_step(q, bf16, s));
}
conv_status seq_scan_fwd(seq_plan_t plan, const seq_scan_args* args, void* stream) { return scan_call(plan, args, SEQ_FWD, stream); }
conv_status seq_scan_bwd(seq_plan_t plan, const seq_scan_args* args, void* stream) { return scan_call(plan, args, SEQ_BWD, stream); }
conv_status seq_scan_step(seq_plan_t plan, const seq_scan_args* args, void* stream) { return scan_call(plan, args, SEQ_STEP, stream); }

// ------------------------------------------------------------------------------------- norm
conv_status seq_norm_plan_create(seq_plan_t* out, int64_t rows, int64_t D, conv_dtype dtype, conv_dtype res_dtype,
                                 seq_direction direction, unsigned flags, float eps) {
    const unsigned gates = flags & (SEQ_NORM_GATE_BEFORE | SEQ_NORM_GATE_AFTER);
    if (!out || bad_dtype(dtype) || bad_dtype(res_dtype) || (direction != SEQ_FWD && direction != SEQ_BWD) || rows < 1 || D < 1 ||
        !(flags & (SEQ_NORM_POST | SEQ_NORM_PRE)) || gates == (SEQ_NORM_GATE_BEFORE | SEQ_NORM_GATE_AFTER) ||
        (flags & ~(unsigned)(SEQ_NORM_LAYER | SEQ_NORM_POST | SEQ_NORM_PRE | SEQ_NORM_GATE_BEFORE | SEQ_NORM_GATE_AFTER | SEQ_NORM_RESIDUAL)) ||
        !(eps >= 0.f) || !(eps < 1e30f))
        return CONV_ERR_INVALID_ARG;
    if (rows > MAX_EXTENT || D > 16384 || (res_dtype != dtype && res_dtype != CONV_F32)) return CONV_ERR_UNSUPPORTED;
    seq_plan* p = new_plan(Op::Norm, 1, rows, D, dtype, direction, flags & ~(unsigned)SEQ_RAGGED);
    if (!p) return CONV_ERR_INVALID_ARG;
    p->res_dtype = res_dtype;
    p->eps = eps;
    if (direction == SEQ_BWD) {
        p->blocks = seq_norm_bwd_blocks(p->T, p->D, flags, (int)p->esize(), (int)p->rsize(), p->sms);
        p->ws_bytes = align256((size_t)p->blocks * 4 * D * sizeof(float));
    }
    snprintf(p->desc, sizeof p->desc, "op=norm direction=%s dtype=%s residual=%s rows=%d width=%d kind=%s post=%d pre=%d gate=%s partial_rows=%d",
             dir_name(direction), type_name(dtype), flags & SEQ_NORM_RESIDUAL ? type_name(res_dtype) : "none", p->T, p->D,
             flags & SEQ_NORM_LAYER ? "layer" : "rms", !!(flags & SEQ_NORM_POST), !!(flags & SEQ_NORM_PRE),
             flags & SEQ_NORM_GATE_BEFORE ? "before" : flags & SEQ_NORM_GATE_AFTER ? "after" : "none", p->blocks);
    *out = p;
    return CONV_OK;
}

static conv_status norm_call(seq_plan_t p, const seq_norm_args* a, seq_direction dir, void* stream) {
    const conv_status st = check_call(p, a, Op::Norm, dir);
    if (st != CONV_OK) return st;
    Checker c;
    const size_t e = p->esize(), r = p->rsize();
    const unsigned f = p->flags;
    const bool bwd = dir == SEQ_BWD, gate = f & (SEQ_NORM_GATE_BEFORE | SEQ_NORM_GATE_AFTER);
    const bool residual = f & SEQ_NORM_RESIDUAL, has_y = (f & SEQ_NORM_PRE) || !residual;
    auto unwanted = [&](const void* v, bool wanted) { if (v && !wanted) c.fail(CONV_ERR_INVALID_ARG); };
    c.rows(a->x, a->x_ld, p->D, e);
    c.rows(a->gate, a->gate_ld, p->D, e, gate);
    c.rows(a->res, a->res_ld, p->D, r, residual);
    for (const void* v : {a->w_post, a->b_post, a->scale, a->w_pre, a->b_pre}) c.ptr(v, e, false, Checker::Groups);
    unwanted(a->gate, gate);
    unwanted(a->res, residual);
    unwanted(a->w_post, f & SEQ_NORM_POST);
    unwanted(a->b_post, f & SEQ_NORM_POST);
    unwanted(a->w_pre, f & SEQ_NORM_PRE);
    unwanted(a->b_pre, f & SEQ_NORM_PRE);
    bool sums = false;
    if (!bwd) {
        c.rows(a->y, a->y_ld, p->D, e, has_y);
        c.rows(a->res_out, a->res_out_ld, p->D, r, residual);
        unwanted(a->y, has_y);
        unwanted(a->res_out, residual);
    } else {
        c.rows(a->dy, a->dy_ld, p->D, e, has_y);
        c.rows(a->dres_out, a->dres_out_ld, p->D, r, false);
        c.rows(a->dx, a->dx_ld, p->D, e);
        c.rows(a->dgate, a->dgate_ld, p->D, e, gate);
        c.rows(a->dres, a->dres_ld, p->D, r, residual);
        unwanted(a->dy, has_y);
        unwanted(a->dres_out, residual);
        unwanted(a->dgate, gate);
        unwanted(a->dres, residual);
        const void* par[5] = {a->w_post, a->b_post, a->scale, a->w_pre, a->b_pre};
        const float* grad[5] = {a->dw_post, a->db_post, a->dscale, a->dw_pre, a->db_pre};
        for (int i = 0; i < 5; ++i) {
            c.ptr(grad[i], 4, false);
            unwanted(grad[i], par[i] != nullptr);
            sums = sums || grad[i];
        }
    }
    if (c.st != CONV_OK) return c.st;
    if (sums && !p->ws) return CONV_ERR_WORKSPACE;
    SeqNormParams q = {};
    q.rows = p->T; q.D = p->D; q.flags = f; q.eps = p->eps;
    q.x = a->x; q.gate = a->gate; q.w_post = a->w_post; q.b_post = a->b_post; q.scale = a->scale; q.res = a->res;
    q.w_pre = a->w_pre; q.b_pre = a->b_pre; q.dy = a->dy; q.dres_out = a->dres_out;
    q.y = a->y; q.res_out = a->res_out; q.dx = a->dx; q.dgate = a->dgate; q.dres = a->dres;
    q.dw_post = a->dw_post; q.db_post = a->db_post; q.dscale = a->dscale; q.dw_pre = a->dw_pre; q.db_pre = a->db_pre;
    q.x_ld = a->x_ld; q.gate_ld = a->gate_ld; q.res_ld = a->res_ld; q.y_ld = a->y_ld; q.res_out_ld = a->res_out_ld;
    q.dy_ld = a->dy_ld; q.dres_out_ld = a->dres_out_ld; q.dx_ld = a->dx_ld; q.dgate_ld = a->dgate_ld; q.dres_ld = a->dres_ld;
    q.ws = sums ? static_cast<float*>(p->ws) : nullptr;
    q.vec = c.wide && p->D % 8 == 0;
    q.sms = p->sms;
    const bool bf16 = p->dtype == CONV_BF16, rbf16 = p->res_dtype == CONV_BF16;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return finish(bwd ? launch_seq_norm_bwd(q, bf16, rbf16, s) : launch_seq_norm_fwd(q, bf16, rbf16, s));
}
conv_status seq_norm_fwd(seq_plan_t plan, const seq_norm_args* args, void* stream) { return norm_call(plan, args, SEQ_FWD, stream); }
conv_status seq_norm_bwd(seq_plan_t plan, const seq_norm_args* args, void* stream) { return norm_call(plan, args, SEQ_BWD, stream); }

}  // extern "C"

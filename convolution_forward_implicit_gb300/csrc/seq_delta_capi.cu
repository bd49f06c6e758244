// C-ABI of the gated delta rule: plan, argument checks, workspace layout.  Declarations and the contract of
// every entry point are in include/delta.h.
#include <math.h>
#include <stdlib.h>

#include "delta.h"
#include "seq_plan.h"

using namespace convfwd;

namespace {

int padded(const seq_plan* p) { return (p->W + 3) / 4 * 4; }        // a state's row, in floats
size_t tri_bytes(const seq_plan* p) {
    const size_t each = p->dtype == CONV_BF16 ? DELTA_PLANES : 2 * DELTA_CHUNK * DELTA_CHUNK * sizeof(float);
    return align256((size_t)p->slots * p->Hv * each);
}
size_t row_bytes(const seq_plan* p) { return align256((size_t)p->slots * p->Hv * DELTA_ROWS * sizeof(float)); }
size_t state_bytes(const seq_plan* p) { return align256((size_t)p->slots * p->Hv * p->N * padded(p) * sizeof(float)); }
size_t token_bytes(const seq_plan* p) { return align256((size_t)p->slots * p->Hv * DELTA_CHUNK * padded(p) * sizeof(float)); }

int padded_keys(const seq_plan* p) { return (p->N + 3) / 4 * 4; }
size_t marks(const seq_plan* p) { return p->run ? (size_t)delta_marks(p->T, p->run) : 0; }
size_t piece_bytes(const seq_plan* p) { return align256(marks(p) * p->Hv * p->N * padded(p) * sizeof(float)); }
size_t through_bytes(const seq_plan* p) { return align256(marks(p) * p->Hv * p->N * padded_keys(p) * sizeof(float)); }

// Chunks of a piece of the axis (0: it is not cut), by times in chunks (4 to 5 us): a walk takes 2 more to begin; pieces walk at once, but
// twice, the first time also with the columns of a unit matrix (without outputs: 0.8 of it); their states are joined in order (0.7
// a piece); launches 3.  It has to promise a fifth.  Of lengths that the plan does not know the longest is taken to be four times the mean, three
// quarters of all tokens at most; beside it the others' blocks (2 chunks to begin, half a chunk at the end) fill the SMs.
// 2048 tokens, 16 heads of 128 x 128 bf16: 119 us cut, 187 not; 13 sequences, 6011 tokens, 32 heads: 385 us not cut, a third more in pieces of 16;
// 64 and 256 sequences of 64 tokens by their bounds, 8 heads: 125 and 471 when only their tokens counted and the plan cut, 77 and 295 now.
int choose_run(const seq_plan* p) {
    const bool wide = p->dtype == CONV_BF16 && p->W > 16, known = p->L > 0 || p->S == 1;
    const int64_t width = wide ? 128 : 16, cap = wide ? p->sms : 2 * (int64_t)p->sms, S = p->S, T = p->T;
    const int64_t dv = (p->W + width - 1) / width, dk = (p->N + width - 1) / width, cols = (p->W + 15) / 16;
    const int64_t longest = known ? T / S : 4 * T / S < 3 * T / 4 ? 4 * T / S : 3 * T / 4, alike = known ? S : 1;
    const int64_t n = (longest + DELTA_CHUNK - 1) / DELTA_CHUNK;
    auto rounds = [&](int64_t blocks) { return (double)((blocks + cap - 1) / cap); };
    // the longest sequences' blocks, and those of all (unknown lengths) with `more` that begin, in chunks
    auto walk = [&](double time, int64_t blocks, int64_t more) {
        const double own = time * rounds(blocks * p->Hv * dv), all = known ? 0 : ((double)T / DELTA_CHUNK + 2.5 * (S + more)) * p->Hv * dv / cap;
        return own > all ? own : all;
    };
    double best = 0.8 * walk(n + 2, alike, 0);
    int run = 0;
    for (int64_t r = 2; r <= n / 2; r += 1 + r / 16) {
        const int64_t m = (n + r - 1) / r, marks = delta_marks(T, (int)r);
        const double t = 0.8 * (r + 2) * rounds((known ? S * (m - 1) : marks - 1) * p->Hv * (dv + dk)) + walk(r + 2, alike * m, marks) +
                         0.7 * (m - 2) * rounds(alike * p->Hv * cols) + (known ? 0 : 0.2 * rounds(delta_joined(S, marks) * p->Hv * cols)) + 3;
        if (t < best && cut_slots(S, T, p->L, (int)(r * DELTA_CHUNK)) * p->Hv * (dv + dk) < (1 << 24)) {
            best = t;
            run = (int)r;
        }
    }
    return run;
}

}  // namespace

extern "C" {

conv_status seq_delta_plan_create(seq_plan_t* out, int64_t S, int64_t T, int64_t Hk, int64_t Hv, int64_t Dk, int64_t Dv,
                                  conv_dtype dtype, seq_direction direction, unsigned flags, float scale) {
    if (!out || bad_dtype(dtype) || bad_dir(direction) || Hk < 1 || Hv < 1 || Dk < 1 || Dv < 1 || !isfinite(scale) ||
        (flags & ~(unsigned)(SEQ_RAGGED | SEQ_DELTA_QK_NORM)))
        return CONV_ERR_INVALID_ARG;
    if (Dk > 128 || Dv > 1024 || Hv > 4096 || Hk > Hv) return Hk > Hv ? CONV_ERR_INVALID_ARG : CONV_ERR_UNSUPPORTED;
    if (Hv % Hk != 0) return CONV_ERR_INVALID_ARG;
    const conv_status st = check_axis(S, T, Hv * Dv, direction, flags & SEQ_RAGGED);
    if (st != CONV_OK) return st;
    seq_plan* p = new_plan(Op::Delta, S, T, Hv * Dv, dtype, direction, flags);
    if (!p) return CONV_ERR_INVALID_ARG;
    p->Hk = (int)Hk; p->Hv = (int)Hv; p->N = (int)Dk; p->W = (int)Dv;
    p->scale = scale != 0.f ? scale : 1.f / sqrtf((float)Dk);
    // blocks a kernel launches at most: 16 columns of a state each (a step: 32 or 128)
    const int64_t slots = direction == SEQ_STEP ? 0 : cut_slots(S, T, p->L, DELTA_CHUNK);
    if (slots > INT32_MAX || S * Hv * ((Dv + 15) / 16) > INT32_MAX) {
        delete p;
        return CONV_ERR_UNSUPPORTED;
    }
    p->slots = (int)slots;
    const char* stall = getenv("CONV_TEST_STALL");
    p->test_stall = stall && atoi(stall) ? 1 : 0;
    if (direction != SEQ_STEP) p->ws_bytes = tri_bytes(p) + row_bytes(p);
    if (direction == SEQ_FWD) {
        p->run = choose_run(p);
        p->pieces = p->run ? (int)cut_slots(S, T, p->L, p->run * DELTA_CHUNK) : 0;
        p->ws_bytes += 2 * piece_bytes(p) + through_bytes(p);
    }
    if (direction == SEQ_BWD) p->ws_bytes += state_bytes(p) + token_bytes(p);
    snprintf(p->desc, sizeof p->desc,
             "op=delta direction=%s dtype=%s sequences=%d tokens=%d ragged=%d key_heads=%d value_heads=%d key_width=%d value_width=%d qk_norm=%d chunks=%d piece_chunks=%d",
             dir_name(direction), type_name(dtype), p->S, p->T, p->ragged(), p->Hk, p->Hv, p->N, p->W, !!(flags & SEQ_DELTA_QK_NORM), p->slots, p->run);
    *out = p;
    return CONV_OK;
}

size_t seq_delta_saved_bytes(seq_plan_t p) {
    return p && p->op == Op::Delta && p->dir != SEQ_STEP ? state_bytes(p) + token_bytes(p) : 0;
}

static conv_status delta_call(seq_plan_t p, const seq_delta_args* a, seq_direction dir, void* stream) {
    const conv_status st = check_call(p, a, Op::Delta, dir);
    if (st != CONV_OK) return st;
    const size_t e = p->esize();
    const bool bwd = dir == SEQ_BWD, any = p->T > 0;
    const int64_t K = (int64_t)p->Hk * p->N, V = (int64_t)p->Hv * p->W;
    Checker keys, vals, c;               // q and k are read in groups of 16 bytes, v, y and their gradients in pairs
    keys.rows(a->q, a->q_ld, K, e, any);
    keys.rows(a->k, a->k_ld, K, e, any);
    vals.rows(a->v, a->v_ld, V, e, any);
    c.rows(a->g, a->g_ld, p->Hv, 4, any, Checker::Elements);
    c.rows(a->beta, a->beta_ld, p->Hv, 4, any, Checker::Elements);
    check_states(p, c, a->starts, a->slots, a->slot_count, bwd ? a->dh_in : a->h_in, bwd ? a->dh_out : a->h_out, 4, Checker::Elements);
    if (dir != SEQ_STEP) c.ptr(a->saved, 4, bwd && any, Checker::Elements, 16);
    if (!bwd) {
        vals.rows(a->y, a->y_ld, V, e, any);
    } else {
        vals.rows(a->dy, a->dy_ld, V, e, any);
        vals.rows(a->dv, a->dv_ld, V, e, any);
        c.rows(a->dq, a->dq_ld, K, e, any, Checker::Elements);
        c.rows(a->dk, a->dk_ld, K, e, any, Checker::Elements);
        c.rows(a->dg, a->dg_ld, p->Hv, 4, any, Checker::Elements);
        c.rows(a->dbeta, a->dbeta_ld, p->Hv, 4, any, Checker::Elements);
    }
    for (const Checker* k : {&keys, &vals, &c})
        if (k->st != CONV_OK) return k->st;
    if (p->ws_bytes && !p->ws) return CONV_ERR_WORKSPACE;
    SeqDeltaParams q = {};
    q.ax = p->axis(a->starts);
    q.sl = SeqSlots{a->slots, a->slot_count};
    q.Hk = p->Hk; q.Hv = p->Hv; q.Dk = p->N; q.Dv = p->W; q.Dvp = padded(p);
    q.norm = !!(p->flags & SEQ_DELTA_QK_NORM);
    q.scale = p->scale;
    q.q = a->q; q.k = a->k; q.v = a->v; q.g = a->g; q.beta = a->beta; q.h_in = a->h_in; q.h_out = a->h_out; q.y = a->y;
    q.saved = a->saved; q.dy = a->dy; q.dh_out = a->dh_out; q.dq = a->dq; q.dk = a->dk; q.dv = a->dv; q.dg = a->dg;
    q.dbeta = a->dbeta; q.dh_in = a->dh_in;
    q.q_ld = a->q_ld; q.k_ld = a->k_ld; q.v_ld = a->v_ld; q.g_ld = a->g_ld; q.beta_ld = a->beta_ld; q.y_ld = a->y_ld;
    q.dy_ld = a->dy_ld; q.dq_ld = a->dq_ld; q.dk_ld = a->dk_ld; q.dv_ld = a->dv_ld; q.dg_ld = a->dg_ld; q.dbeta_ld = a->dbeta_ld;
    q.slots = p->slots;
    q.saved_u = (long long)(state_bytes(p) / sizeof(float));
    unsigned char* w = static_cast<unsigned char*>(p->ws);
    if (dir != SEQ_STEP) {
        q.tri = reinterpret_cast<float*>(w);
        q.rows = reinterpret_cast<float*>(w + tri_bytes(p));
        if (dir == SEQ_FWD) {
            q.run = p->run; q.pieces = p->pieces; q.marks = (int)marks(p); q.Dkp = padded_keys(p);
            q.added = reinterpret_cast<float*>(w + tri_bytes(p) + row_bytes(p));
            q.left = q.added + piece_bytes(p) / sizeof(float);
            q.through = q.left + piece_bytes(p) / sizeof(float);
        }
        q.dstate = reinterpret_cast<float*>(w + tri_bytes(p) + row_bytes(p));
        q.dr = reinterpret_cast<float*>(w + tri_bytes(p) + row_bytes(p) + state_bytes(p));
    }
    q.wide = keys.wide && (p->N * e) % 16 == 0;
    q.compact = 1;
    for (int64_t ld : {a->q_ld, a->k_ld, a->v_ld, a->y_ld, a->dy_ld, a->dv_ld}) q.compact = q.compact && ld < (INT64_C(1) << 24);
    // pairs of elements: 4 bytes of bf16, 8 of fp32
    auto paired = [&](const void* v, int64_t ld) { return !v || (reinterpret_cast<uintptr_t>(v) % (2 * e) == 0 && ld % 2 == 0); };
    q.pairs = p->W % 2 == 0 && paired(a->v, a->v_ld) && paired(a->y, a->y_ld) && paired(a->dy, a->dy_ld) && paired(a->dv, a->dv_ld);
    q.key_pairs = p->N % 2 == 0 && paired(a->dq, a->dq_ld) && paired(a->dk, a->dk_ld);
    auto grouped = [&](const void* v, int64_t ld) { return !v || (reinterpret_cast<uintptr_t>(v) % 16 == 0 && (uint64_t)ld * e % 16 == 0); };
    q.val_wide = (p->W * e) % 16 == 0 && grouped(a->v, a->v_ld) && grouped(a->dy, a->dy_ld);
    q.key_wide = (p->N * e) % 16 == 0 && grouped(a->dq, a->dq_ld) && grouped(a->dk, a->dk_ld);
    auto aligned = [](const void* v) { return reinterpret_cast<uintptr_t>(v) % 16 == 0; };
    q.quads = p->W % 4 == 0 && aligned(a->h_in) && aligned(a->h_out);
    q.sms = p->sms;
    q.test_stall = p->test_stall;
    const bool bf16 = p->dtype == CONV_BF16;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return finish(dir == SEQ_FWD ? launch_seq_delta_fwd(q, bf16, s) : bwd ? launch_seq_delta_bwd(q, bf16, s)
                                                                         : launch_seq_delta_step(q, bf16, s));
}
conv_status seq_delta_fwd(seq_plan_t plan, const seq_delta_args* args, void* stream) { return delta_call(plan, args, SEQ_FWD, stream); }
conv_status seq_delta_bwd(seq_plan_t plan, const seq_delta_args* args, void* stream) { return delta_call(plan, args, SEQ_BWD, stream); }
conv_status seq_delta_check(seq_plan_t plan, void* stream) {
    return plan && plan->op == Op::Delta ? check_error_word(static_cast<cudaStream_t>(stream)) : CONV_ERR_INVALID_ARG;
}
conv_status seq_delta_step(seq_plan_t plan, const seq_delta_args* args, void* stream) { return delta_call(plan, args, SEQ_STEP, stream); }

}  // extern "C"

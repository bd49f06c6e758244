// C-ABI of the group norm with an activation: plan, argument checks, workspace layout.  Declarations and
// the contract of every entry point are in include/gnorm.h.
#include "gnorm.h"
#include "seq_plan.h"

using namespace convfwd;

namespace {

size_t part_bytes(const seq_plan* p) { return align256((size_t)p->slots * p->D * 2 * sizeof(float)); }
size_t gpart_bytes(const seq_plan* p) { return align256((size_t)p->slots * p->G * 2 * sizeof(float)); }

}  // namespace

extern "C" {

conv_status seq_gnorm_plan_create(seq_plan_t* out, int64_t S, int64_t T, int64_t D, int64_t G, conv_dtype dtype,
                                  seq_direction direction, unsigned flags, seq_act act, float eps) {
    if (!out || bad_dtype(dtype) || (direction != SEQ_FWD && direction != SEQ_BWD) || G < 1 || (flags & ~(unsigned)SEQ_RAGGED) ||
        (act != SEQ_ACT_NONE && act != SEQ_ACT_SILU && act != SEQ_ACT_GELU) || !(eps >= 0.f) || !(eps < 1e30f))
        return CONV_ERR_INVALID_ARG;
    const conv_status st = check_axis(S, T, D, direction, flags & SEQ_RAGGED);
    if (st != CONV_OK) return st;
    if (D % G != 0) return CONV_ERR_INVALID_ARG;
    if (D > ((int64_t)1 << 20) || S * G > INT32_MAX) return CONV_ERR_UNSUPPORTED;
    seq_plan* p = new_plan(Op::GroupNorm, S, T, D, dtype, direction, flags);
    if (!p) return CONV_ERR_INVALID_ARG;
    p->G = (int)G;
    p->act = (int)act;
    p->eps = eps;
    p->run = seq_gnorm_slab(S, T, p->D, p->G, (int)p->esize(), direction == SEQ_BWD, p->sms);
    const int64_t slots = cut_slots(S, T, p->L, p->run);
    if (slots > INT32_MAX) {
        delete p;
        return CONV_ERR_UNSUPPORTED;
    }
    p->slots = (int)slots;
    p->ws_bytes = part_bytes(p) + gpart_bytes(p) + align256((size_t)S * G * 2 * sizeof(float));
    snprintf(p->desc, sizeof p->desc,
             "op=gnorm direction=%s dtype=%s sequences=%d tokens=%d ragged=%d width=%d groups=%d act=%s slabs=%d slab_tokens=%d",
             dir_name(direction), type_name(dtype), p->S, p->T, p->ragged(), p->D, p->G,
             act == SEQ_ACT_SILU ? "silu" : act == SEQ_ACT_GELU ? "gelu" : "none", p->slots, p->run);
    *out = p;
    return CONV_OK;
}

static conv_status gnorm_call(seq_plan_t p, const seq_gnorm_args* a, seq_direction dir, void* stream) {
    const conv_status st = check_call(p, a, Op::GroupNorm, dir);
    if (st != CONV_OK) return st;
    Checker c;
    const size_t e = p->esize();
    const bool bwd = dir == SEQ_BWD, any = p->T > 0;
    c.rows(a->x, a->x_ld, p->D, e, any);
    c.ptr(a->w, e, false, Checker::Groups);
    c.ptr(a->b, e, false, Checker::Groups);
    if (p->ragged() ? !a->starts : a->starts != nullptr) c.fail(CONV_ERR_INVALID_ARG);
    c.ptr(a->starts, 4, false);
    c.ptr(a->stats, 4, bwd, Checker::Elements, 8);
    if (!bwd) {
        c.rows(a->y, a->y_ld, p->D, e, any);
    } else {
        c.rows(a->dy, a->dy_ld, p->D, e, any);
        c.rows(a->dx, a->dx_ld, p->D, e, any);
        c.ptr(a->dw, 4, false);
        c.ptr(a->db, 4, false);
        if ((a->dw && !a->w) || (a->db && !a->b)) c.fail(CONV_ERR_INVALID_ARG);
    }
    if (c.st != CONV_OK) return c.st;
    if (!p->ws) return CONV_ERR_WORKSPACE;
    bool paired = true;                  // rows of aligned pairs of elements: 4 bytes of bf16, 8 of fp32
    auto pairs = [&](const void* v, int64_t ld) { paired = paired && reinterpret_cast<uintptr_t>(v) % (2 * e) == 0 && ld % 2 == 0; };
    pairs(a->x, a->x_ld);
    pairs(a->w, 0);
    pairs(a->b, 0);
    pairs(bwd ? a->dy : a->y, bwd ? a->dy_ld : a->y_ld);
    if (bwd) pairs(a->dx, a->dx_ld);
    SeqGnormParams q = {};
    q.ax = p->axis(a->starts);
    q.D = p->D; q.G = p->G; q.act = p->act; q.eps = p->eps;
    q.slab = p->run; q.slots = p->slots;
    q.x = a->x; q.w = a->w; q.b = a->b; q.dy = a->dy; q.y = a->y; q.dx = a->dx;
    q.stats = a->stats; q.dw = a->dw; q.db = a->db;
    q.x_ld = a->x_ld; q.y_ld = a->y_ld; q.dy_ld = a->dy_ld; q.dx_ld = a->dx_ld;
    q.part = static_cast<float*>(p->ws);
    q.gpart = q.part + part_bytes(p) / sizeof(float);
    q.coef = q.gpart + gpart_bytes(p) / sizeof(float);
    q.grain = c.wide && (p->D * e) % 16 == 0 ? 16 : p->D % 2 == 0 && paired ? 2 : 0;
    q.sms = p->sms;
    const bool bf16 = p->dtype == CONV_BF16;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return finish(bwd ? launch_seq_gnorm_bwd(q, bf16, s) : launch_seq_gnorm_fwd(q, bf16, s));
}
conv_status seq_gnorm_fwd(seq_plan_t plan, const seq_gnorm_args* args, void* stream) { return gnorm_call(plan, args, SEQ_FWD, stream); }
conv_status seq_gnorm_bwd(seq_plan_t plan, const seq_gnorm_args* args, void* stream) { return gnorm_call(plan, args, SEQ_BWD, stream); }

}  // extern "C"

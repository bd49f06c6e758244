/*
 * delta.h -- C ABI of the gated delta rule of libconvfwd.so: a linear recurrence with a matrix
 * state, which stands in a block where the selective scan of seq.h does (short convolution before
 * it, gated norm behind it).  Statuses, types, token axis, states, slots, plans, streams and errors
 * are those of seq.h.
 *
 * For each value head, with the state h (Dk x Dv, fp32) from its slot, or zero:
 *   h'  = exp(g_t) h_{t-1}
 *   u   = beta_t (v_t - h'^T k_t)
 *   h_t = h' + k_t u^T
 *   y_t = scale h_t^T q_t
 * Hk key heads hold q and k, Hv value heads v, g, beta and y; value head i goes with key head
 * i / (Hv / Hk) (Hk divides Hv).  With SEQ_DELTA_QK_NORM q and k of a head are first divided by
 * sqrt(their sum of squares + 1e-6).  Without it they are taken as they are: keys of length above
 * 1 let the state grow where beta is near 1.
 *
 * Whole sequences are worked on in chunks of 64 tokens: an infinity or NaN in a token may reach
 * every token of its chunk and all later ones of its sequence, in its value head (q, k: in the
 * heads that share them), and nothing else; of gradients any token of its sequence.  g may be minus infinity (a finite state is dropped).
 * Where g is above 0 and its sum between two tokens of a chunk passes 80, or a state grows beyond fp32's range over the
 * tokens of a piece (below) from however small values, the results may overflow; across pieces a state of zero stays zero.
 * dg of a token whose factor is much smaller than those behind it in its chunk is off by 1e-7 or so of what these have.
 * Where few heads have long sequences the plan of a forward call cuts the axis (the description
 * has the chunks of a piece): sums are then taken in another order than by a plan of other sizes.
 */
#ifndef CONVFWD_DELTA_H
#define CONVFWD_DELTA_H

#include "seq.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { SEQ_DELTA_QK_NORM = 512 };      /* with SEQ_RAGGED: the flags of the plan_create call */

/* scale: of y; 0 stands for 1 / sqrt(Dk).  CONV_ERR_INVALID_ARG for sizes out of range, Hk that does not divide Hv,
 * or a scale that is not finite; CONV_ERR_UNSUPPORTED for Dk > 128, Dv > 1024, more than 2^30 tokens, 4096
 * value heads, 2^22 values a token (Hv Dv) or 2^31 - 1 sixteenths of states (S Hv Dv / 16). */
conv_status seq_delta_plan_create(seq_plan_t* out, int64_t S, int64_t T, int64_t Hk, int64_t Hv, int64_t Dk, int64_t Dv,
                                  conv_dtype dtype, seq_direction direction, unsigned flags, float scale);

/* Bytes of what a forward call saves for the backward call of the same problem: the state at every
 * chunk's first token and every token's u, fp32; the same for a forward and a backward plan.  0 on NULL. */
size_t seq_delta_saved_bytes(seq_plan_t plan);

typedef struct {
    const void* q;  int64_t q_ld;          /* T x Hk*Dk, dtype      */
    const void* k;  int64_t k_ld;          /* T x Hk*Dk, dtype      */
    const void* v;  int64_t v_ld;          /* T x Hv*Dv, dtype      */
    const float* g; int64_t g_ld;          /* T x Hv, fp32: logarithm of the decay factor */
    const float* beta; int64_t beta_ld;    /* T x Hv, fp32          */
    const int32_t* starts;                 /* S + 1, with SEQ_RAGGED (else NULL) */
    const int32_t* slots;                  /* S, or NULL            */
    int64_t slot_count;                    /* rows of the state buffers */
    const float* h_in;                     /* slot_count x Hv x Dk x Dv, or NULL */
    float* h_out;                          /* the same, or NULL; may be h_in */
    void* y;        int64_t y_ld;          /* T x Hv*Dv, dtype (forward, step) */
    float* saved;                          /* seq_delta_saved_bytes, 16-byte aligned; forward: written
                                              unless NULL; backward: read */
    /* backward: the forward call's q, k, v, g, beta, starts and slots, and */
    const void* dy; int64_t dy_ld;         /* T x Hv*Dv, dtype      */
    const float* dh_out;                   /* as h_out: the gradient at the states left, or NULL */
    void* dq;       int64_t dq_ld;         /* T x Hk*Dk, dtype      */
    void* dk;       int64_t dk_ld;         /* T x Hk*Dk, dtype      */
    void* dv;       int64_t dv_ld;         /* T x Hv*Dv, dtype      */
    float* dg;      int64_t dg_ld;         /* T x Hv                */
    float* dbeta;   int64_t dbeta_ld;      /* T x Hv                */
    float* dh_in;                          /* as h_in: the gradient at the starting states, or NULL */
} seq_delta_args;

conv_status seq_delta_fwd(seq_plan_t plan, const seq_delta_args* args, void* stream);
conv_status seq_delta_bwd(seq_plan_t plan, const seq_delta_args* args, void* stream);
/* The bf16 kernels wait for the tensor cores and for copies, for one second at most.  Waits for the stream (not while it
 * is captured) and returns CONV_ERR_TIMEOUT if a wait ran out since the last check (of any plan, conv_plan_check's among
 * them): the results of the calls between are not to be used. */
conv_status seq_delta_check(seq_plan_t plan, void* stream);
/* One token per sequence: q and k are S x Hk*Dk, v and y S x Hv*Dv, g and beta S x Hv. */
conv_status seq_delta_step(seq_plan_t plan, const seq_delta_args* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* CONVFWD_DELTA_H */

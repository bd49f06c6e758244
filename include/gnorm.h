/*
 * gnorm.h -- C ABI of the group norm with an activation, channels last, of libconvfwd.so: what
 * stands between two convolutions.  Statuses, types, token axis, plans, streams and errors are
 * those of seq.h: the N L C output of a convolution (conv.h) is S = N sequences of T/S = L tokens,
 * an N D H W C one S = N sequences of D H W tokens, C channels each.
 *
 *   mean, var     over the tokens of a sequence and the D/G channels of a group
 *   rstd        = 1 / sqrt(var + eps)
 *   z[t, c]     = (x[t, c] - mean) rstd w[c] + b[c],   y = act(z)
 *
 * gelu is the erf form.  G = D gives every channel statistics of its own, G = 1 all channels
 * together.  var is the mean of the squared differences from the mean (not less one).
 */
#ifndef CONVFWD_GNORM_H
#define CONVFWD_GNORM_H

#include "seq.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { SEQ_ACT_NONE = 0, SEQ_ACT_SILU = 1, SEQ_ACT_GELU = 2 } seq_act;

/* flags: SEQ_RAGGED or 0; direction SEQ_FWD or SEQ_BWD.  CONV_ERR_INVALID_ARG for sizes out of range
 * or G that does not divide D, CONV_ERR_UNSUPPORTED for more than 2^30 tokens, 2^20 channels or a
 * number of sequences times groups beyond 2^31 - 1.  Both directions need the plan's workspace. */
conv_status seq_gnorm_plan_create(seq_plan_t* out, int64_t S, int64_t T, int64_t D, int64_t G, conv_dtype dtype,
                                  seq_direction direction, unsigned flags, seq_act act, float eps);

typedef struct {
    const void* x;  int64_t x_ld;      /* T x D, dtype                                       */
    const void* w;                     /* D, dtype, or NULL (ones)                           */
    const void* b;                     /* D, dtype, or NULL (zeros)                          */
    const int32_t* starts;             /* S + 1, with SEQ_RAGGED (else NULL)                 */
    float* stats;                      /* S x G x 2, 8-byte aligned: mean and rstd (both 0 for an
                                          empty sequence); forward: written unless NULL; backward: read */
    void* y;        int64_t y_ld;      /* T x D, dtype (forward); may be x, with the same ld */
    /* backward: x, w, b, starts and stats as the forward call had and left them */
    const void* dy; int64_t dy_ld;     /* T x D, dtype                                       */
    void* dx;       int64_t dx_ld;     /* T x D, dtype; may be dy, with the same ld          */
    float* dw;                         /* D; NULL: not wanted, or w is                       */
    float* db;                         /* D; NULL: not wanted, or b is                       */
} seq_gnorm_args;

conv_status seq_gnorm_fwd(seq_plan_t plan, const seq_gnorm_args* args, void* stream);
conv_status seq_gnorm_bwd(seq_plan_t plan, const seq_gnorm_args* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* CONVFWD_GNORM_H */

/*
 * seq.h -- C ABI of the sequence-mixing operators of libconvfwd.so: a short causal
 * depthwise convolution, the selective state space scan it feeds, and the norm, gate and
 * residual step around such a block.  Statuses, data types and conv_status_string are
 * those of conv.h; dense projections around these operators are its 1x1 convolutions.
 *
 * The token axis.  Tokens of S sequences lie one after another on one axis of T tokens,
 * channels last.  Without SEQ_RAGGED the sequences have T/S tokens each (S divides T; the
 * N L C layout of conv.h).  With SEQ_RAGGED their bounds are `starts`, S+1 int32 values on
 * the device, starts[0] = 0, non-decreasing, starts[S] = T; a sequence may be empty.  No
 * token sees a token of another sequence.  (Values outside that contract are clamped into
 * range: they give other results, never an access outside the T tokens.)
 *
 * Layout of a tensor of T tokens: element (t, c) at t * ld + c, c contiguous; `ld` (in
 * elements, at least the row's width, at most 2^31 - 1) lets a call read a slice of a wider
 * projection.  Offsets are 64-bit.  Pointers need the alignment of their element only; rows that are
 * 16-byte aligned (pointer and ld) are read with wide loads.  Inputs and outputs do not
 * overlap, except that the state a call leaves may be the buffer it starts from, and that
 * seq_norm_fwd may update the residual stream in place (res_out = res, with the same ld).
 *
 * States.  Sequence s starts from row slots[s] of the state buffers, or row s when slots is
 * NULL; a slot outside 0 .. slot_count-1 names no state: that sequence starts from zero and
 * leaves nothing.  Two sequences never share a slot.  A NULL state input means zero states;
 * a NULL state output means that no states are kept.  An empty sequence hands its state on.
 *
 * Types: "dtype" is the plan's conv_dtype.  All arithmetic, states of the scan, sums and
 * statistics are fp32; an output of the plan's type is rounded once, to nearest even.
 * Parameter gradients are fp32 whatever the plan's type (an optimizer adds them up).  Sums
 * have a fixed order: a call on the same inputs gives the same bits.
 *
 * Conventions (ownership, streams, errors, threads): as conv.h.  Calls only enqueue kernels
 * on `stream` (a cudaStream_t; NULL: the legacy default stream), allocate nothing and may be
 * captured in a CUDA graph.  No kernel here waits on another, so there is no check call.  A
 * plan owns host memory only; calls that use a workspace concurrently need one each.
 * Argument structs are read during the call and not kept.
 */
#ifndef CONVFWD_SEQ_H
#define CONVFWD_SEQ_H

#include "conv.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct seq_plan* seq_plan_t;

typedef enum {
    SEQ_FWD = 0,     /* whole sequences, forward        */
    SEQ_BWD = 1,     /* whole sequences, gradients      */
    SEQ_STEP = 2     /* one new token per sequence (T = S) */
} seq_direction;

enum {               /* flags of the plan_create calls, added up */
    SEQ_RAGGED = 1,          /* conv, scan: sequence bounds come from `starts`          */
    SEQ_CONV_SILU = 2,       /* conv: y = silu(pre); without it y = pre                  */
    SEQ_SCAN_SOFTPLUS = 4,   /* scan: delta = softplus(dt + dt_bias); without it dt + dt_bias */
    SEQ_NORM_LAYER = 8,      /* norm: layer norm; without it RMS norm                    */
    SEQ_NORM_POST = 16,      /* norm: normalise the block's output x                     */
    SEQ_NORM_PRE = 32,       /* norm: normalise the (new) residual for the next block    */
    SEQ_NORM_GATE_BEFORE = 64,   /* norm: x is multiplied by silu(gate) before POST      */
    SEQ_NORM_GATE_AFTER = 128,   /* norm: ... after POST                                 */
    SEQ_NORM_RESIDUAL = 256      /* norm: a residual stream is added to and returned     */
};

/* Static string of what the plan chose (variant, split, grid).  Valid while the plan lives. */
const char* seq_plan_describe(seq_plan_t plan);

/* Bytes of device workspace the plan's call needs (0: none; 0 on a NULL plan), and its
 * attachment: caller-owned, 16-byte aligned, CONV_ERR_WORKSPACE if too small. */
size_t seq_workspace_bytes(seq_plan_t plan);
conv_status seq_plan_set_workspace(seq_plan_t plan, void* workspace, size_t bytes);

/* Free the plan's host memory.  NULL is accepted. */
conv_status seq_plan_destroy(seq_plan_t plan);

/* ------------------------------------------------------------------ short causal convolution
 *   pre[t, d] = bias[d] + sum_{j < W} w[d, j] * x[t - W + 1 + j, d],   y = silu(pre) or pre
 * depthwise, over the tokens of one sequence; positions before its first token are the rows
 * of its state, the W-1 inputs that came before it (oldest first), or zero.
 * 1 <= W <= 8.  CONV_ERR_INVALID_ARG for sizes out of range, CONV_ERR_UNSUPPORTED for W > 8,
 * more than 2^30 tokens or 2^22 channels.
 */
conv_status seq_conv_plan_create(seq_plan_t* out, int64_t S, int64_t T, int64_t D, int64_t W, conv_dtype dtype,
                                 seq_direction direction, unsigned flags);

typedef struct {
    const void* x;  int64_t x_ld;      /* T x D, dtype                                         */
    const void* w;                     /* D x W, dtype (the G K X C weight layout at C = K = 1) */
    const void* bias;                  /* D, dtype, or NULL                                     */
    const int32_t* starts;             /* S + 1, with SEQ_RAGGED (else NULL)                    */
    const int32_t* slots;              /* S, or NULL                                            */
    int64_t slot_count;                /* rows of the state buffers                             */
    const void* state_in;              /* slot_count x (W-1) x D, dtype, or NULL                */
    void* state_out;                   /* the same, or NULL; may be state_in                    */
    void* y;        int64_t y_ld;      /* T x D, dtype (forward, step)                          */
    /* backward: x, w, bias, starts, slots and state_in as in the forward call */
    const void* dy; int64_t dy_ld;     /* T x D, dtype: the loss's gradient at y                */
    void* dx;       int64_t dx_ld;     /* T x D, dtype                                          */
    float* dw;                         /* D x W                                                 */
    float* dbias;                      /* D; NULL when bias is                                  */
} seq_conv_args;

/* Forward over whole sequences; leaves the states after the last tokens in state_out. */
conv_status seq_conv_fwd(seq_plan_t plan, const seq_conv_args* args, void* stream);
/* Gradients with respect to x, w and bias (the states are constants of it).  Needs the plan's
 * workspace. */
conv_status seq_conv_bwd(seq_plan_t plan, const seq_conv_args* args, void* stream);
/* One token per sequence: x and y are S x D; the states move on by one token. */
conv_status seq_conv_step(seq_plan_t plan, const seq_conv_args* args, void* stream);

/* ------------------------------------------------------------------ selective state space scan
 *   delta = softplus(dt + dt_bias)   (or dt + dt_bias)
 *   h_t[d, n] = exp(delta_t[d] A[d, n]) h_{t-1}[d, n] + delta_t[d] x_t[d] B_t[g(d), n]
 *   y_t[d]    = (sum_n C_t[g(d), n] h_t[d, n] + D[d] x_t[d]) * silu(z_t[d])
 * with g(d) = d / (D/G): the D channels share B and C in G groups (G divides D).  h starts
 * from the sequence's state (fp32), or zero.  1 <= N <= 128 states per channel.
 * CONV_ERR_INVALID_ARG for sizes out of range, CONV_ERR_UNSUPPORTED for N > 128, more
 * than 2^30 tokens or 2^22 channels, or D N beyond 2^31 - 1.
 */
conv_status seq_scan_plan_create(seq_plan_t* out, int64_t S, int64_t T, int64_t D, int64_t N, int64_t G,
                                 conv_dtype dtype, seq_direction direction, unsigned flags);

/* Bytes of the states a forward call saves for the backward call of the same problem: fp32
 * states at every 8th token, the same for a forward and a backward plan.  0 on NULL. */
size_t seq_scan_saved_bytes(seq_plan_t plan);

typedef struct {
    const void* x;  int64_t x_ld;      /* T x D, dtype          */
    const void* dt; int64_t dt_ld;     /* T x D, dtype          */
    const float* A;                    /* D x N, fp32           */
    const void* B;  int64_t B_ld;      /* T x G*N, dtype        */
    const void* C;  int64_t C_ld;      /* T x G*N, dtype        */
    const float* D;                    /* D, fp32, or NULL      */
    const void* z;  int64_t z_ld;      /* T x D, dtype, or NULL: no gate */
    const float* dt_bias;              /* D, fp32, or NULL      */
    const int32_t* starts;             /* S + 1, with SEQ_RAGGED (else NULL) */
    const int32_t* slots;              /* S, or NULL            */
    int64_t slot_count;                /* rows of the state buffers */
    const float* h_in;                 /* slot_count x D x N, or NULL */
    float* h_out;                      /* the same, or NULL; may be h_in */
    void* y;        int64_t y_ld;      /* T x D, dtype (forward, step) */
    float* saved;                      /* seq_scan_saved_bytes, 16-byte aligned; forward: written
                                          unless NULL; backward: read */
    /* backward: the forward call's inputs, and */
    const void* dy; int64_t dy_ld;     /* T x D, dtype          */
    const float* dh_out;               /* as h_out: the gradient at the states left, or NULL */
    void* dx;       int64_t dx_ld;     /* T x D, dtype          */
    void* ddt;      int64_t ddt_ld;    /* T x D, dtype: the gradient at dt */
    void* dB;       int64_t dB_ld;     /* T x G*N, dtype        */
    void* dC;       int64_t dC_ld;     /* T x G*N, dtype        */
    void* dz;       int64_t dz_ld;     /* T x D, dtype; NULL when z is */
    float* dA;                         /* D x N                 */
    float* dD;                         /* D; NULL when D is     */
    float* ddt_bias;                   /* D; NULL when dt_bias is */
    float* dh_in;                      /* as h_in: the gradient at the starting states, or NULL */
} seq_scan_args;

conv_status seq_scan_fwd(seq_plan_t plan, const seq_scan_args* args, void* stream);
conv_status seq_scan_bwd(seq_plan_t plan, const seq_scan_args* args, void* stream);
/* One token per sequence: x, dt, z, y are S x D, B and C are S x G*N. */
conv_status seq_scan_step(seq_plan_t plan, const seq_scan_args* args, void* stream);

/* ------------------------------------------------------------------ norm, gate and residual
 * Around a block whose output is x (rows x D):
 *   u = x * silu(gate)                      SEQ_NORM_GATE_BEFORE
 *   u = norm(u) * w_post + b_post           SEQ_NORM_POST
 *   u = u * silu(gate)                      SEQ_NORM_GATE_AFTER
 *   r = res + scale * u                     SEQ_NORM_RESIDUAL (else r = scale * u); r -> res_out
 *   y = norm(r) * w_pre + b_pre             SEQ_NORM_PRE (else y = r, without a residual)
 * norm(v) = v / sqrt(mean(v^2) + eps), with SEQ_NORM_LAYER of v less its mean.  At least one of
 * POST and PRE; at most one GATE.  y is computed from r before r is rounded to res_dtype.
 * 1 <= D <= 16384.  res_dtype is the residual stream's type (CONV_F32, or the plan's type).
 */
conv_status seq_norm_plan_create(seq_plan_t* out, int64_t rows, int64_t D, conv_dtype dtype, conv_dtype res_dtype,
                                 seq_direction direction, unsigned flags, float eps);

typedef struct {
    const void* x;    int64_t x_ld;        /* rows x D, dtype                             */
    const void* gate; int64_t gate_ld;     /* rows x D, dtype (with a GATE flag)          */
    const void* w_post;                    /* D, dtype, or NULL (ones)                    */
    const void* b_post;                    /* D, dtype, or NULL (zeros)                   */
    const void* scale;                     /* D, dtype, or NULL (ones)                    */
    const void* res;  int64_t res_ld;      /* rows x D, res_dtype (with RESIDUAL)         */
    const void* w_pre;                     /* D, dtype, or NULL (ones)                    */
    const void* b_pre;                     /* D, dtype, or NULL (zeros)                   */
    void* y;          int64_t y_ld;        /* rows x D, dtype: with PRE, or without RESIDUAL */
    void* res_out;    int64_t res_out_ld;  /* rows x D, res_dtype: with RESIDUAL          */
    /* backward: the forward call's inputs, and */
    const void* dy;   int64_t dy_ld;       /* as y                                        */
    const void* dres_out; int64_t dres_out_ld;   /* as res_out, or NULL (zeros)           */
    void* dx;         int64_t dx_ld;       /* rows x D, dtype                             */
    void* dgate;      int64_t dgate_ld;    /* rows x D, dtype (with a GATE flag)          */
    void* dres;       int64_t dres_ld;     /* rows x D, res_dtype (with RESIDUAL)         */
    float* dw_post;                        /* D each; NULL when the parameter is          */
    float* db_post;
    float* dscale;
    float* dw_pre;
    float* db_pre;
} seq_norm_args;

conv_status seq_norm_fwd(seq_plan_t plan, const seq_norm_args* args, void* stream);
/* Gradients of both outputs' losses with respect to every input.  Needs the plan's workspace
 * when any parameter's gradient is asked for. */
conv_status seq_norm_bwd(seq_plan_t plan, const seq_norm_args* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* CONVFWD_SEQ_H */

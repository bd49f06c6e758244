// Internal definitions of the sequence-mixing operators (not installed): the token axis as the
// kernels see it, the kernels' parameters and their launchers.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.h"
#include "seq.h"

namespace convfwd {

// The token axis: S sequences on T tokens; L > 0: L tokens each, L = 0: bounds in starts.
struct SeqAxis {
    int S, T, L;
    const int* starts;
};

// States: row of sequence s in the state buffers, or -1.
struct SeqSlots {
    const int* slots;
    long long count;
};

#ifdef __CUDACC__
// First token of sequence s, clamped into [lo, T] (s = S: the end of the axis), so that a
// bound outside its contract never leads outside the tensors.
__device__ __forceinline__ int seq_start(const SeqAxis& a, int s, int lo) {
    if (s >= a.S) return a.T;
    const int v = a.L > 0 ? s * a.L : (a.starts ? a.starts[s] : 0);
    return min(max(v, lo), a.T);
}
// The first sequence whose first token is at or behind t (S if none is).
__device__ __forceinline__ int seq_first_at(const SeqAxis& a, int t) {
    if (a.L > 0) return min((t + a.L - 1) / a.L, a.S);
    int lo = 0, hi = a.S;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (seq_start(a, mid, 0) < t) lo = mid + 1; else hi = mid;
    }
    return lo;
}
__device__ __forceinline__ long long seq_slot(const SeqSlots& s, int seq) {
    if (seq < 0) return -1;
    const long long v = s.slots ? (long long)s.slots[seq] : (long long)seq;
    return v >= 0 && v < s.count ? v : -1;
}
#endif

// A piece of the token axis that does not cross sequences: `len` tokens at most.  Sequence s has the slots from
// cut_base(s) on, ceil(length / len) of them.  Equal lengths: s ceil(L / len).  Unequal ones: floor(start / len) + s,
// which needs no sums over the sequences before it and leaves room, since ceil((b - a) / len) <= floor(b / len) -
// floor(a / len) + 1; slots between are empty.  T / len + S slots are enough, for bounds outside their contract too
// (they are clamped, so that a <= b <= T).
struct CutPiece {
    int s, index, t0, n;            // sequence, piece of it, first token, tokens (0: none)
};
__host__ __device__ inline long long cut_slots(long long S, long long T, long long L, int len) {
    return L > 0 ? S * ((L + len - 1) / len) : T / len + S;
}
#ifdef __CUDACC__
__device__ __forceinline__ int cut_base(const SeqAxis& a, int s, int len) {
    return a.L > 0 ? s * ((a.L + len - 1) / len) : seq_start(a, s, 0) / len + s;
}
__device__ __forceinline__ CutPiece cut_piece(const SeqAxis& a, int slot, int len) {
    CutPiece c;
    if (a.L > 0) {
        const int per = (a.L + len - 1) / len;
        c.s = slot / per;
        c.index = slot - c.s * per;
        c.t0 = c.s * a.L + c.index * len;
        c.n = min(len, a.L - c.index * len);
        return c;
    }
    int lo = 0, hi = a.S - 1;       // the last sequence whose first slot is at or before this one
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cut_base(a, mid, len) <= slot) lo = mid; else hi = mid - 1;
    }
    const int t0 = seq_start(a, lo, 0), t1 = seq_start(a, lo + 1, t0);
    c.s = lo;
    c.index = max(slot - cut_base(a, lo, len), 0);
    const long long at = t0 + (long long)c.index * len;
    c.t0 = (int)min(at, (long long)t1);
    c.n = min(len, t1 - c.t0);
    return c;
}
#endif

// ---- short causal convolution ----
struct SeqConvParams {
    SeqAxis ax;
    SeqSlots sl;
    int D, W, silu;
    const void *x, *w, *bias, *state_in, *dy;
    void *y, *state_out, *dx;
    float *dw, *dbias;
    float* ws;                      // backward: partial sums [token blocks][W + 1][D]
    long long x_ld, y_ld, dy_ld, dx_ld;
    int run;                        // tokens a thread walks (whole sequences)
    int tblocks;                    // backward: token blocks
    int vec;                        // 1: 16-byte rows
};
cudaError_t launch_seq_conv_fwd(const SeqConvParams& p, bool bf16, cudaStream_t stream);
cudaError_t launch_seq_conv_bwd(const SeqConvParams& p, bool bf16, cudaStream_t stream);
cudaError_t launch_seq_conv_step(const SeqConvParams& p, bool bf16, cudaStream_t stream);
int seq_conv_run(long long T, int D, int W, bool bf16, bool bwd, int sms);
int seq_conv_bwd_token_blocks(long long T, int run);

// ---- selective scan ----
constexpr int SCAN_TILE = 8;        // tokens between two saved states
// Pieces of the token axis: each is walked by one thread block per channel block.  Without
// ragged bounds pieces do not cross sequences (pps pieces of each); else piece p is the tokens
// p * len .. of the axis.  len is a multiple of SCAN_TILE.
struct ScanPieces {
    int count, len, pps;
};
struct SeqScanParams {
    SeqAxis ax;
    SeqSlots sl;
    ScanPieces pc;
    int D, N, G, softplus;
    const void *x, *dt, *B, *C, *z, *dy;
    const float *A, *Dskip, *dt_bias, *h_in, *dh_out;
    void *y, *dx, *ddt, *dB, *dC, *dz;
    float *h_out, *saved, *dA, *dD, *ddt_bias, *dh_in;
    long long x_ld, dt_ld, B_ld, C_ld, z_ld, y_ld, dy_ld, dx_ld, ddt_ld, dB_ld, dC_ld, dz_ld;
    // workspace; states lie as [row][quad of states][channel][4] (scan_state_at), as the saved ones do
    float* piece_state;             // a row a piece: what it adds to the state behind it (backward: to the gradient
                                    // before it); then the state before it (the gradient behind it)
    float* piece_init;              // a row a piece: starting state of the last sequence that starts in it
    float* piece_delta;             // [pieces][D]: sum of delta over a piece
    float* part_bc;                 // backward: [channel blocks][T][2][P] partial dB, dC; P: N padded to 8, 16, 32, 64 or 128
    float* part_par;                // backward: [pieces][N + 2][D] partial dA, dD, ddt_bias
    int cblocks;                    // backward: channel blocks (over all groups)
    int quads;                      // 1 when A (step: states, B and C too) lies in whole aligned groups of 4
    int wide;                       // rows and groups consist of whole aligned pieces of so many bytes: 16, 4 or 0 (of single elements)
    int sms;
};

#ifdef __CUDACC__
__device__ __forceinline__ void scan_piece_range(const SeqAxis& a, const ScanPieces& pc, int p, int& t0, int& t1) {
    if (pc.pps > 0) {
        const int s = p / pc.pps, k = p - s * pc.pps;
        t0 = s * a.L + k * pc.len;
        t1 = min(t0 + pc.len, (s + 1) * a.L);
    } else {
        t0 = p * pc.len;
        t1 = min(t0 + pc.len, a.T);
    }
}
// Row of the saved states that token t's tile starts with (t: a tile's first token).
__device__ __forceinline__ long long scan_tile_row(const SeqAxis& a, int t) {
    if (a.L > 0) {
        const int s = t / a.L;
        return (long long)s * ((a.L + SCAN_TILE - 1) / SCAN_TILE) + (t - s * a.L) / SCAN_TILE;
    }
    return t / SCAN_TILE;
}
#endif
cudaError_t launch_seq_scan_fwd(const SeqScanParams& p, bool bf16, cudaStream_t stream);
cudaError_t launch_seq_scan_bwd(const SeqScanParams& p, bool bf16, cudaStream_t stream);
cudaError_t launch_seq_scan_step(const SeqScanParams& p, bool bf16, cudaStream_t stream);
// From what every piece adds to what reaches every piece: piece_state in place, piece after piece.
cudaError_t launch_seq_scan_join(const SeqScanParams& p, bool reverse, cudaStream_t stream);
// States of empty sequences: from -> to (zero where from is NULL).
cudaError_t launch_seq_scan_empty(const SeqScanParams& p, const float* from, float* to, cudaStream_t stream);
int seq_scan_bwd_channel_blocks(int D, int N, int G);

// ---- norm, gate, residual ----
struct SeqNormParams {
    int rows, D;
    unsigned flags;                 // SEQ_NORM_*
    float eps;
    const void *x, *gate, *w_post, *b_post, *scale, *res, *w_pre, *b_pre, *dy, *dres_out;
    void *y, *res_out, *dx, *dgate, *dres;
    float *dw_post, *db_post, *dscale, *dw_pre, *db_pre;
    long long x_ld, gate_ld, res_ld, y_ld, res_out_ld, dy_ld, dres_out_ld, dx_ld, dgate_ld, dres_ld;
    float* ws;                      // backward: [rows of partial sums][4][D]
    int vec;                        // 1: rows of whole 16-byte aligned groups of 8
    int sms;
};
cudaError_t launch_seq_norm_fwd(const SeqNormParams& p, bool bf16, bool res_bf16, cudaStream_t stream);
cudaError_t launch_seq_norm_bwd(const SeqNormParams& p, bool bf16, bool res_bf16, cudaStream_t stream);
int seq_norm_bwd_blocks(int rows, int D, unsigned flags, int esize, int rsize, int sms);

// ---- group norm with an activation ----
// The token axis is cut into slabs of `slab` tokens that do not cross sequences (CutPiece).
struct SeqGnormParams {
    SeqAxis ax;
    int D, G, act;
    float eps;
    int slab, slots;
    const void *x, *w, *b, *dy;
    void *y, *dx;
    float *stats, *dw, *db;
    long long x_ld, y_ld, dy_ld, dx_ld;
    float* part;                    // [slots][D][2]: a slab's mean and sum of squared differences; backward: sums
    float* gpart;                   // [slots][G][2]: the same of groups
    float* coef;                    // [S][G][2]: mean and rstd; backward: the group's two means
    int grain;                      // rows in whole aligned groups of 16 bytes: 16, of pairs of elements: 2, else 0
    int sms;
};
cudaError_t launch_seq_gnorm_fwd(const SeqGnormParams& p, bool bf16, cudaStream_t stream);
cudaError_t launch_seq_gnorm_bwd(const SeqGnormParams& p, bool bf16, cudaStream_t stream);
int seq_gnorm_slab(long long S, long long T, int D, int G, int esize, bool bwd, int sms);

// ---- gated delta rule ----
constexpr int DELTA_CHUNK = 64;     // tokens worked on at once; saved states lie at every chunk's first token
constexpr int DELTA_PLANES = 3 * 128 * 128;      // bytes of a chunk's matrices in parts
constexpr int DELTA_FACTORS = 264, DELTA_ROWS = 520;      // floats of a chunk's row factors, and with what they come from (see seq_delta.cuh)
// Pieces of `run` chunks that another piece of their sequence follows are whole: each holds exactly one token whose index is a multiple of
// their length, its mark, whatever the lengths of the sequences, and the pieces of a sequence follow one another by marks.  So there are
// T / length marks and no more, and blocks and memory go by them, not by the number of sequences.
__host__ __device__ inline long long delta_marks(long long T, int run) {
    const long long len = (long long)run * DELTA_CHUNK;
    return (T + len - 1) / len;
}
__host__ __device__ inline long long delta_joined(long long S, long long marks) { return S < marks ? S : marks; }
struct SeqDeltaParams {
    SeqAxis ax;
    SeqSlots sl;
    int Hk, Hv, Dk, Dv, norm;
    float scale;
    const void *q, *k, *v, *dy;
    const float *g, *beta, *h_in, *dh_out;
    void *y, *dq, *dk, *dv;
    float *h_out, *saved, *dg, *dbeta, *dh_in;
    long long q_ld, k_ld, v_ld, g_ld, beta_ld, y_ld, dy_ld, dq_ld, dk_ld, dv_ld, dg_ld, dbeta_ld;
    int slots;                      // chunks of the token axis at most
    // workspace, by chunk and value head
    float* tri;                     // [slots][Hv]: T and A, [2][64][64] fp32; or (planes) [3][128][64] bf16: the three
                                    // parts of [T; A T] (1) or [T; A] (2), rows of 128 bytes in the 128-byte swizzle
    int planes;
    int compact;                    // 64 rows of q, k, v, y, dy, dv lie within 2^31 bytes each
    float* rows;                    // [slots][Hv][DELTA_ROWS]
    float* dstate;                  // backward: [slots][Hv][Dk][Dvp] gradient at the state a chunk leaves
    float* dr;                      // backward: [slots][Hv][64][Dvp]
    int Dvp;                        // Dv rounded up to 4
    long long saved_u;              // where the saved u begin, in floats: [slots][Hv][64][Dvp] behind [slots][Hv][Dk][Dvp]
    int wide;                       // q and k in whole aligned 16-byte groups
    int pairs, key_pairs;           // v, y, dy, dv; dq, dk in aligned pairs of elements
    int val_wide, key_wide;         // v and dy; dq and dk in whole aligned 16-byte groups
    int quads;                      // step: states in whole aligned groups of 4
    // forward, where the axis is cut for the walk (run > 0): chunks of a piece, pieces at most, the marks of those that another follows
    // (see delta_marks), and by mark and value head what a piece adds to a state [Dk][Dvp] (of a sequence's first, once joined: the state it
    // starts from), the matrix it passes one through [Dk][Dkp], and the state it leaves [Dk][Dvp]
    int run, pieces, marks, Dkp;
    float *added, *through, *left;
    int sms;
    int test_stall;                 // test hook: products that others wait for are never issued (bf16 kernels)
};
cudaError_t launch_seq_delta_fwd(const SeqDeltaParams& p, bool bf16, cudaStream_t stream);
cudaError_t launch_seq_delta_bwd(const SeqDeltaParams& p, bool bf16, cudaStream_t stream);
enum DeltaWalk { DELTA_WHOLE = 0, DELTA_PIECES = 1, DELTA_JOINED = 2 };     // see seq_delta.cuh
cudaError_t launch_seq_delta_walk_tc(const SeqDeltaParams& p, DeltaWalk mode, cudaStream_t stream);
cudaError_t launch_seq_delta_grad_tc(const SeqDeltaParams& p, cudaStream_t stream);
cudaError_t launch_seq_delta_back_tc(const SeqDeltaParams& p, cudaStream_t stream);
cudaError_t launch_seq_delta_step(const SeqDeltaParams& p, bool bf16, cudaStream_t stream);

}  // namespace convfwd

// What the C-ABI files of the sequence operators share: the plan, argument checks, and the rules for the
// token axis and the states.  Host code only.
#pragma once
#include <stdio.h>

#include <new>

#include "conv.h"
#include "seq_internal.h"

namespace convfwd {

enum class Op { Conv, Scan, Norm, Delta, GroupNorm };

constexpr int64_t MAX_EXTENT = (int64_t)1 << 30;     // tokens: sums of two token indices stay in 32 bits
constexpr int64_t MAX_CHANNELS = (int64_t)1 << 22;   // channel blocks are a launch's second dimension

inline int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        (void)cudaGetLastError();
        return 152;
    }
    return n;
}

inline size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

conv_status check_error_word(cudaStream_t stream);       // capi.cu

}  // namespace convfwd

struct seq_plan {
    convfwd::Op op;
    seq_direction dir;
    conv_dtype dtype, res_dtype;
    unsigned flags;
    int S, T, D, L;        // L: tokens per sequence, 0 when ragged (or T = 0)
    int W, N, G;
    int run;               // conv: tokens a thread walks; group norm: of a slab; delta rule: chunks of a piece (0: none)
    int sms;
    convfwd::ScanPieces pc;
    int blocks;            // conv backward: token blocks; scan backward: channel blocks; norm backward: partial rows
    size_t ws_bytes;
    void* ws;
    float eps;
    int Hk, Hv;            // delta rule: key and value heads (N, W: their widths); group norm: N channels a group
    float scale;           // delta rule
    int act;               // group norm
    int slots;             // delta rule, group norm: chunks or slabs of the token axis
    int pieces;            // delta rule: of `run` chunks each (0: the axis is not cut for the walk)
    int test_stall;        // delta rule, CONV_TEST_STALL: see SeqDeltaParams
    char desc[256];

    bool ragged() const { return flags & SEQ_RAGGED; }
    size_t esize() const { return dtype == CONV_BF16 ? 2 : 4; }
    size_t rsize() const { return res_dtype == CONV_BF16 ? 2 : 4; }
    convfwd::SeqAxis axis(const int32_t* starts) const { return convfwd::SeqAxis{S, T, L, starts}; }
};

namespace convfwd {

inline bool bad_dtype(conv_dtype d) { return d != CONV_F32 && d != CONV_BF16; }
inline bool bad_dir(seq_direction d) { return d != SEQ_FWD && d != SEQ_BWD && d != SEQ_STEP; }
inline const char* dir_name(seq_direction d) { return d == SEQ_FWD ? "fwd" : d == SEQ_BWD ? "bwd" : "step"; }
inline const char* type_name(conv_dtype d) { return d == CONV_BF16 ? "bf16" : "f32"; }

inline conv_status check_axis(int64_t S, int64_t T, int64_t D, seq_direction dir, bool ragged) {
    if (S < 1 || T < 0 || D < 1) return CONV_ERR_INVALID_ARG;
    if (S > MAX_EXTENT || T > MAX_EXTENT || D > MAX_CHANNELS) return CONV_ERR_UNSUPPORTED;
    if (!ragged && T % S != 0) return CONV_ERR_INVALID_ARG;
    if (dir == SEQ_STEP && (T != S || ragged)) return CONV_ERR_INVALID_ARG;
    return CONV_OK;
}

inline seq_plan* new_plan(Op op, int64_t S, int64_t T, int64_t D, conv_dtype dtype, seq_direction dir, unsigned flags) {
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

inline conv_status finish(cudaError_t e) { return e == cudaSuccess ? CONV_OK : CONV_ERR_CUDA; }

inline conv_status check_call(seq_plan_t p, const void* args, Op op, seq_direction dir) {
    if (!p || !args || p->op != op || p->dir != dir) return CONV_ERR_INVALID_ARG;
    return CONV_OK;
}

// starts goes with the plan's kind of axis; the state buffers with their slots.
inline void check_states(const seq_plan* p, Checker& c, const int32_t* starts, const int32_t* slots, int64_t slot_count,
                  const void* in, const void* out, size_t esize, Checker::Access access) {
    if (p->ragged() ? !starts : starts != nullptr) c.fail(CONV_ERR_INVALID_ARG);
    c.ptr(starts, 4, false);
    c.ptr(slots, 4, false);
    c.ptr(in, esize, false, access);
    c.ptr(out, esize, false, access);
    if (slot_count > MAX_EXTENT) c.fail(CONV_ERR_UNSUPPORTED);
    if ((in || out) && (slot_count < 0 || (!slots && slot_count < p->S))) c.fail(CONV_ERR_INVALID_ARG);
}

}  // namespace convfwd

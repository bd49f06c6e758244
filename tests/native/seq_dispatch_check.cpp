// Which arguments of the sequence operators' calls choose between the kernels for rows of aligned groups and those
// for any rows: the library's own argument checks (csrc/seq_capi.cu) with launchers that note what they were given.
// Prints, for each call, the arguments whose misplacement by one element (pointers) or by one (strides) changes that.
#include <stdio.h>
#include <string.h>

#include <string>
#include <vector>

#include "seq_capi.cu"

extern "C" cudaError_t cudaGetDevice(int* d) { *d = 0; return cudaSuccess; }
extern "C" cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int) { *v = 152; return cudaSuccess; }
extern "C" cudaError_t cudaGetLastError() { return cudaSuccess; }

static int rows, quads;       // what the launcher was given
namespace convfwd {
static cudaError_t note(const SeqConvParams& p) { rows = p.vec; return cudaSuccess; }
static cudaError_t note(const SeqScanParams& p) { rows = p.wide; quads = p.quads; return cudaSuccess; }
static cudaError_t note(const SeqNormParams& p) { rows = p.vec; return cudaSuccess; }
cudaError_t launch_seq_conv_fwd(const SeqConvParams& p, bool, cudaStream_t) { return note(p); }
cudaError_t launch_seq_conv_bwd(const SeqConvParams& p, bool, cudaStream_t) { return note(p); }
cudaError_t launch_seq_conv_step(const SeqConvParams& p, bool, cudaStream_t) { return note(p); }
cudaError_t launch_seq_scan_fwd(const SeqScanParams& p, bool, cudaStream_t) { return note(p); }
cudaError_t launch_seq_scan_bwd(const SeqScanParams& p, bool, cudaStream_t) { return note(p); }
cudaError_t launch_seq_scan_step(const SeqScanParams& p, bool, cudaStream_t) { return note(p); }
cudaError_t launch_seq_norm_fwd(const SeqNormParams& p, bool, bool, cudaStream_t) { return note(p); }
cudaError_t launch_seq_norm_bwd(const SeqNormParams& p, bool, bool, cudaStream_t) { return note(p); }
int seq_conv_run(long long, int, int, bool, bool, int) { return 8; }
int seq_conv_bwd_token_blocks(long long, int) { return 1; }
int seq_scan_bwd_channel_blocks(int, int, int) { return 1; }
int seq_norm_bwd_blocks(int, int, unsigned, int, int, int) { return 1; }
}  // namespace convfwd

struct Field {
    const char* name;
    size_t at;          // in the argument struct
    int bytes;          // of an element; 0: a stride
};
#define P(type, f, bytes) {#f, offsetof(type, f), bytes}
#define ROWS(type, f, bytes) {#f, offsetof(type, f), bytes}, {#f "_ld", offsetof(type, f##_ld), 0}

template <typename Args>
static void show(const char* name, seq_plan_t plan, conv_status (*call)(seq_plan_t, const Args*, void*), Args good,
                 const std::vector<Field>& fields) {
    alignas(16) static unsigned char ws[1 << 24];
    if (seq_plan_set_workspace(plan, ws, sizeof ws) != CONV_OK) printf("%s: workspace\n", name);
    if (call(plan, &good, nullptr) != CONV_OK) printf("%s: refused\n", name);
    const int rows0 = rows, quads0 = quads;
    std::string in_rows, in_quads;
    for (const Field& f : fields) {
        Args a = good;
        int64_t v;
        memcpy(&v, (char*)&a + f.at, 8);
        v += f.bytes ? f.bytes : 1;
        memcpy((char*)&a + f.at, &v, 8);
        if (call(plan, &a, nullptr) != CONV_OK) printf("%s: refused with another %s\n", name, f.name);
        if (rows != rows0) in_rows += std::string(" ") + f.name;
        if (quads != quads0) in_quads += std::string(" ") + f.name;
    }
    printf("%s %d:%s\n", name, rows0, in_rows.c_str());
    if (!in_quads.empty()) printf("%s quads %d:%s\n", name, quads0, in_quads.c_str());
    seq_plan_destroy(plan);
}

template <typename T>
static T* at() {
    return reinterpret_cast<T*>(1 << 20);      // never read
}

int main() {
    const int e = 2, D = 64, N = 16;
    seq_plan_t p = nullptr;
    {
        using A = seq_conv_args;
        A a = {};
        a.x = a.w = a.bias = a.state_in = a.dy = at<void>();
        a.starts = a.slots = at<int32_t>();
        a.y = a.dx = a.state_out = at<void>();
        a.x_ld = a.y_ld = a.dy_ld = a.dx_ld = 2 * D;
        a.slot_count = 2;
        a.dw = a.dbias = at<float>();
        const std::vector<Field> f = {ROWS(A, x, e), P(A, w, e), P(A, bias, e), P(A, starts, 4), P(A, slots, 4), P(A, state_in, e)};
        auto all = [&](std::vector<Field> more) { more.insert(more.begin(), f.begin(), f.end()); return more; };
        seq_conv_plan_create(&p, 2, 8, D, 4, CONV_BF16, SEQ_FWD, SEQ_RAGGED);
        show("conv_fwd", p, seq_conv_fwd, a, all({P(A, state_out, e), ROWS(A, y, e)}));
        seq_conv_plan_create(&p, 2, 8, D, 4, CONV_BF16, SEQ_BWD, SEQ_RAGGED);
        show("conv_bwd", p, seq_conv_bwd, a, all({ROWS(A, dy, e), ROWS(A, dx, e), P(A, dw, 4), P(A, dbias, 4)}));
        seq_conv_plan_create(&p, 2, 2, D, 4, CONV_BF16, SEQ_STEP, 0);
        a.starts = nullptr;
        show("conv_step", p, seq_conv_step, a,
             {ROWS(A, x, e), P(A, w, e), P(A, bias, e), P(A, slots, 4), P(A, state_in, e), P(A, state_out, e), ROWS(A, y, e)});
    }
    {
        using A = seq_scan_args;
        A a = {};
        a.x = a.dt = a.B = a.C = a.z = a.dy = at<void>();
        a.A = a.D = a.dt_bias = a.h_in = a.dh_out = at<float>();
        a.starts = a.slots = at<int32_t>();
        a.h_out = a.saved = a.dA = a.dD = a.ddt_bias = a.dh_in = at<float>();
        a.y = a.dx = a.ddt = a.dB = a.dC = a.dz = at<void>();
        a.x_ld = a.dt_ld = a.B_ld = a.C_ld = a.z_ld = a.y_ld = a.dy_ld = a.dx_ld = a.ddt_ld = a.dB_ld = a.dC_ld = a.dz_ld = 2 * D;
        a.slot_count = 2;
        const std::vector<Field> f = {ROWS(A, x, e), ROWS(A, dt, e), P(A, A, 4), ROWS(A, B, e), ROWS(A, C, e), P(A, D, 4), ROWS(A, z, e), P(A, dt_bias, 4),
                                      P(A, slots, 4), P(A, h_in, 4)};
        auto all = [&](std::vector<Field> more) { more.insert(more.begin(), f.begin(), f.end()); return more; };
        seq_scan_plan_create(&p, 2, 8, D, N, 1, CONV_BF16, SEQ_FWD, SEQ_RAGGED);
        show("scan_fwd", p, seq_scan_fwd, a, all({P(A, starts, 4), P(A, h_out, 4), ROWS(A, y, e)}));
        seq_scan_plan_create(&p, 2, 8, D, N, 1, CONV_BF16, SEQ_BWD, SEQ_RAGGED);
        show("scan_bwd", p, seq_scan_bwd, a,
             all({P(A, starts, 4), ROWS(A, dy, e), P(A, dh_out, 4), ROWS(A, dx, e), ROWS(A, ddt, e), ROWS(A, dB, e), ROWS(A, dC, e), ROWS(A, dz, e),
                  P(A, dA, 4), P(A, dD, 4), P(A, ddt_bias, 4), P(A, dh_in, 4)}));
        a.starts = nullptr;
        seq_scan_plan_create(&p, 2, 2, D, N, 1, CONV_BF16, SEQ_STEP, 0);
        show("scan_step", p, seq_scan_step, a, all({P(A, h_out, 4), ROWS(A, y, e)}));
    }
    {
        using A = seq_norm_args;
        A a = {};
        a.x = a.gate = a.w_post = a.b_post = a.scale = a.res = a.w_pre = a.b_pre = a.dy = a.dres_out = at<void>();
        a.y = a.res_out = a.dx = a.dgate = a.dres = at<void>();
        a.dw_post = a.db_post = a.dscale = a.dw_pre = a.db_pre = at<float>();
        a.x_ld = a.gate_ld = a.res_ld = a.y_ld = a.res_out_ld = a.dy_ld = a.dres_out_ld = a.dx_ld = a.dgate_ld = a.dres_ld = 2 * D;
        const std::vector<Field> f = {ROWS(A, x, e), ROWS(A, gate, e), P(A, w_post, e), P(A, b_post, e), P(A, scale, e), ROWS(A, res, 4), P(A, w_pre, e),
                                      P(A, b_pre, e)};
        auto all = [&](std::vector<Field> more) { more.insert(more.begin(), f.begin(), f.end()); return more; };
        const unsigned flags = SEQ_NORM_POST | SEQ_NORM_PRE | SEQ_NORM_GATE_BEFORE | SEQ_NORM_RESIDUAL;
        seq_norm_plan_create(&p, 8, D, CONV_BF16, CONV_F32, SEQ_FWD, flags, 1e-5f);
        show("norm_fwd", p, seq_norm_fwd, a, all({ROWS(A, y, e), ROWS(A, res_out, 4)}));
        seq_norm_plan_create(&p, 8, D, CONV_BF16, CONV_F32, SEQ_BWD, flags, 1e-5f);
        show("norm_bwd", p, seq_norm_bwd, a,
             all({ROWS(A, dy, e), ROWS(A, dres_out, 4), ROWS(A, dx, e), ROWS(A, dgate, e), ROWS(A, dres, 4), P(A, dw_post, 4), P(A, db_post, 4),
                  P(A, dscale, 4), P(A, dw_pre, 4), P(A, db_pre, 4)}));
    }
    return 0;
}

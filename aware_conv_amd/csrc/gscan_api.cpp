// C-ABI front end of the gated linear recurrence: argument checks (before
// anything is enqueued), then the kernels of the layout.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "call_buffers.h"
#include "gscan.h"
#include "gscan_internal.h"

namespace {

// Rows (sequences x channels) of a call: a wavefront each, and a launch holds
// fewer than 2^32 threads.
constexpr long long kMaxRows = 1LL << 25;

using calls::hip_status;
using calls::put;

gsc::Plan plan_of(const gscan_shape& s) {
    return s.layout == GSCAN_BCT ? gsc::planes_plan(s) : gsc::tokens_plan(s);
}

int check_form(const gscan_shape* s) {
    if (!s) return WTCONV_ERR_NULL;
    if (s->B < 0 || s->C < 0 || s->T < 0 || s->T > (1 << 30)) return WTCONV_ERR_SHAPE;
    if (s->dtype != GSCAN_F32 && s->dtype != GSCAN_F16 && s->dtype != GSCAN_BF16)
        return WTCONV_ERR_DTYPE;
    if (s->layout != GSCAN_BCT && s->layout != GSCAN_BTC) return WTCONV_ERR_LAYOUT;
    if (!(s->decay > 0.f) || !isfinite(s->decay)) return WTCONV_ERR_VALUE;
    return (long long)s->B * s->C > kMaxRows ? WTCONV_ERR_SHAPE : WTCONV_OK;
}
int check_shape(const gscan_shape* s) {
    const int rc = check_form(s);
    if (rc) return rc;
    return plan_of(*s).fits ? WTCONV_OK : WTCONV_ERR_UNSUPPORTED;
}

// A call's buffers; its activations have the call's layout.
class Bufs : public calls::Bufs {
  public:
    explicit Bufs(const gscan_shape& s) : s_(s) {}
    void view(const gscan_view* v, bool out) {
        const long long R = s_.layout == GSCAN_BCT ? s_.C : s_.T;
        const long long run = s_.layout == GSCAN_BCT ? s_.T : s_.C;
        calls::Bufs::view(v, s_.B, R, run, calls::elem_size(s_.dtype), out);
    }

  private:
    const gscan_shape& s_;
};

int check_ws(const gsc::Plan& p, const void* ws, size_t bytes) {
    return calls::check_ws(p.scratch, ws, bytes);
}

}  // namespace

extern "C" {

int gscan_states_size(const gscan_shape* s, size_t* bytes) {
    const int rc = check_shape(s);
    if (rc) return rc;
    if (!bytes) return WTCONV_ERR_NULL;
    *bytes = plan_of(*s).states;
    return WTCONV_OK;
}

int gscan_workspace_size(const gscan_shape* s, size_t* bytes) {
    const int rc = check_shape(s);
    if (rc) return rc;
    if (!bytes) return WTCONV_ERR_NULL;
    *bytes = plan_of(*s).scratch;
    return WTCONV_OK;
}

int gscan_fwd(const gscan_shape* s, const gscan_view* x, const gscan_view* r,
              const gscan_view* i, const float* lam, const float* h0, const int* lengths,
              const gscan_view* h, float* h_last, float* states, void* workspace,
              size_t ws_bytes, void* stream) {
    int rc = check_shape(s);
    if (rc) return rc;
    const long long rows = (long long)s->B * s->C;
    const gsc::Plan p = plan_of(*s);
    Bufs q(*s);
    q.view(x, false);
    q.view(r, false);
    q.view(i, false);
    q.flat(lam, s->C, false, false);
    q.flat(h0, rows, false, true);
    q.flat(lengths, s->B, false, true);
    q.view(h, true);
    q.flat(h_last, rows, true, true);
    q.flat(states, (long long)(p.states / 4), true, true);
    if (workspace && ws_bytes >= p.scratch) q.flat(workspace, (long long)p.scratch, true, true, 1);
    if ((rc = q.done())) return rc;
    if (rows == 0) return WTCONV_OK;
    if ((rc = check_ws(p, workspace, ws_bytes))) return rc;
    gsc::Args a{};
    put(x, a.x, a.x_sb, a.x_sr);
    put(r, a.r, a.r_sb, a.r_sr);
    put(i, a.i, a.i_sb, a.i_sr);
    put(h, a.h, a.h_sb, a.h_sr);
    a.lam = lam;
    a.h0 = h0;
    a.lengths = lengths;
    a.h_last = h_last;
    a.states = states;
    a.B = s->B;
    a.C = s->C;
    a.T = s->T;
    a.decay = s->decay;
    hipStream_t st = static_cast<hipStream_t>(stream);
    return hip_status(s->layout == GSCAN_BCT ? gsc::planes_fwd(*s, a, workspace, st)
                                             : gsc::tokens_fwd(*s, a, workspace, st));
}

int gscan_bwd(const gscan_shape* s, const gscan_view* x, const gscan_view* r,
              const gscan_view* i, const float* lam, const float* states, const int* lengths,
              const gscan_view* dh, const float* dh_last, const gscan_view* dx,
              const gscan_view* dr, const gscan_view* di, float* dlam, float* dh0,
              void* workspace, size_t ws_bytes, void* stream) {
    int rc = check_shape(s);
    if (rc) return rc;
    const long long rows = (long long)s->B * s->C;
    const gsc::Plan p = plan_of(*s);
    Bufs q(*s);
    q.view(x, false);
    q.view(r, false);
    q.view(i, false);
    q.flat(lam, s->C, false, false);
    q.flat(states, (long long)(p.states / 4), false, false);
    q.flat(lengths, s->B, false, true);
    q.view(dh, false);
    q.flat(dh_last, rows, false, true);
    q.view(dx, true);
    q.view(dr, true);
    q.view(di, true);
    q.flat(dlam, s->C, true, false);
    q.flat(dh0, rows, true, true);
    if (workspace && ws_bytes >= p.scratch) q.flat(workspace, (long long)p.scratch, true, true, 1);
    if ((rc = q.done())) return rc;
    if (s->C == 0) return WTCONV_OK;
    gsc::Args a{};
    a.lam = lam;
    a.dlam = dlam;
    a.B = s->B;
    a.C = s->C;
    a.T = s->T;
    a.decay = s->decay;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (s->B == 0) return hip_status(gsc::close_dlam(a, 0, st));
    if ((rc = check_ws(p, workspace, ws_bytes))) return rc;
    put(x, a.x, a.x_sb, a.x_sr);
    put(r, a.r, a.r_sb, a.r_sr);
    put(i, a.i, a.i_sb, a.i_sr);
    put(dh, a.dh, a.dh_sb, a.dh_sr);
    put(dx, a.dx, a.dx_sb, a.dx_sr);
    put(dr, a.dr, a.dr_sb, a.dr_sr);
    put(di, a.di, a.di_sb, a.di_sr);
    a.states = const_cast<float*>(states);
    a.lengths = lengths;
    a.dh_last = dh_last;
    a.dh0 = dh0;
    return hip_status(s->layout == GSCAN_BCT ? gsc::planes_bwd(*s, a, workspace, st)
                                             : gsc::tokens_bwd(*s, a, workspace, st));
}

int gscan_step(int B, int C, int S, int dtype, float decay, const gscan_view* x,
               const gscan_view* r, const gscan_view* i, const float* lam, float* state,
               const int* slots, const gscan_view* h, void* stream) {
    const gscan_shape s{B, C, 1, GSCAN_BTC, dtype, 0, decay};
    int rc = check_form(&s);  // any number of rows fits its launch
    if (rc) return rc;
    if (S < 0 || (long long)S * C > (1LL << 40)) return WTCONV_ERR_SHAPE;
    if (!slots && S < B) return WTCONV_ERR_SHAPE;
    Bufs q(s);
    q.view(x, false);
    q.view(r, false);
    q.view(i, false);
    q.flat(lam, C, false, false);
    q.flat(state, (long long)S * C, true, false);
    q.flat(slots, B, false, true);
    q.view(h, true);
    if ((rc = q.done())) return rc;
    if (B == 0 || C == 0) return WTCONV_OK;
    return hip_status(gsc::step(B, C, S, dtype, decay, *x, *r, *i, lam, state, slots, *h,
                                static_cast<hipStream_t>(stream)));
}

}  // extern "C"

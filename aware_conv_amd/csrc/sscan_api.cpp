// C-ABI front end of the selective scan: argument checks (before anything is
// enqueued), then the kernels.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "call_buffers.h"
#include "sscan.h"
#include "sscan_internal.h"

namespace {

using calls::elem_size;
using calls::hip_status;
using calls::put;

int check_form(const sscan_shape* s) {
    if (!s) return WTCONV_ERR_NULL;
    if (s->B < 0 || s->T < 0 || s->D < 0 || s->T > (1 << 30)) return WTCONV_ERR_SHAPE;
    if (s->N < 1 || s->N > SSCAN_MAX_STATES || s->G < 1 || s->D % s->G) return WTCONV_ERR_SHAPE;
    if (s->dtype != GSCAN_F32 && s->dtype != GSCAN_F16 && s->dtype != GSCAN_BF16)
        return WTCONV_ERR_DTYPE;
    const long long rows = (long long)s->B * s->D;
    if (rows > (1LL << 25) || (long long)s->D * s->N > (1LL << 25)) return WTCONV_ERR_SHAPE;
    if (rows * s->N > (1LL << 31) || (long long)s->G * s->N > (1LL << 20)) return WTCONV_ERR_SHAPE;
    return WTCONV_OK;
}
int check_shape(const sscan_shape* s) {
    const int rc = check_form(s);
    if (rc) return rc;
    return ssc::plan(*s, false).fits ? WTCONV_OK : WTCONV_ERR_UNSUPPORTED;
}

// A call's buffers.
class Bufs : public calls::Bufs {
  public:
    Bufs(const sscan_shape& s, long long T) : s_(s), T_(T), e_(elem_size(s.dtype)) {}
    void wide(const gscan_view* v, bool out) { act(v, s_.D, out); }
    void low(const gscan_view* v, bool out) { act(v, (long long)s_.G * s_.N, out); }
    // what is wrong, stride too far last
    int done() const {
        const int rc = calls::Bufs::done();
        return rc ? rc : far_ ? WTCONV_ERR_UNSUPPORTED : WTCONV_OK;
    }

  private:
    void act(const gscan_view* v, long long run, bool out) {
        view(v, s_.B, T_, run, e_, out);
        if (v && T_ > 1 && v->sr > kMaxStride) far_ = true;
    }
    // 15 rows are within 32 bits of bytes
    static constexpr long long kMaxStride = 1LL << 26;
    bool far_ = false;
    const sscan_shape& s_;
    long long T_;
    size_t e_;
};

ssc::Args args_of(const sscan_shape& s) {
    ssc::Args a{};
    a.B = s.B;
    a.T = s.T;
    a.D = s.D;
    a.N = s.N;
    a.G = s.G;
    a.Dg = s.D / s.G;
    return a;
}

}  // namespace

extern "C" {

int sscan_states_size(const sscan_shape* s, size_t* bytes) {
    const int rc = check_shape(s);
    if (rc) return rc;
    if (!bytes) return WTCONV_ERR_NULL;
    *bytes = ssc::plan(*s, false).states;
    return WTCONV_OK;
}

int sscan_workspace_size(const sscan_shape* s, int backward, size_t* bytes) {
    const int rc = check_shape(s);
    if (rc) return rc;
    if (!bytes) return WTCONV_ERR_NULL;
    *bytes = ssc::plan(*s, backward != 0).scratch;
    return WTCONV_OK;
}

int sscan_fwd(const sscan_shape* s, const gscan_view* x, const gscan_view* dt, const float* a_log,
              const gscan_view* b, const gscan_view* c, const float* d, const gscan_view* z,
              const float* dt_bias, const float* h0, const int* lengths, const gscan_view* y,
              float* h_last, float* states, void* workspace, size_t ws_bytes, void* stream) {
    int rc = check_shape(s);
    if (rc) return rc;
    const long long rows = (long long)s->B * s->D, all = rows * s->N;
    const ssc::Plan p = ssc::plan(*s, false);
    Bufs q(*s, s->T);
    q.wide(x, false);
    q.wide(dt, false);
    q.low(b, false);
    q.low(c, false);
    if (z) q.wide(z, false);
    q.flat(a_log, (long long)s->D * s->N, false, false);
    q.flat(d, s->D, false, true);
    q.flat(dt_bias, s->D, false, true);
    q.flat(h0, all, false, true);
    q.flat(lengths, s->B, false, true);
    q.wide(y, true);
    q.flat(h_last, all, true, true);
    q.flat(states, (long long)(p.states / 4), true, true);
    if (workspace && ws_bytes >= p.scratch) q.flat(workspace, (long long)p.scratch, true, true, 1);
    if ((rc = q.done())) return rc;
    if (rows == 0) return WTCONV_OK;
    if ((rc = calls::check_ws(p.scratch, workspace, ws_bytes))) return rc;
    ssc::Args a = args_of(*s);
    put(x, a.x, a.x_sb, a.x_sr);
    put(dt, a.dt, a.dt_sb, a.dt_sr);
    put(b, a.b, a.b_sb, a.b_sr);
    put(c, a.c, a.c_sb, a.c_sr);
    if (z) put(z, a.z, a.z_sb, a.z_sr);
    put(y, a.y, a.y_sb, a.y_sr);
    a.a_log = a_log;
    a.d = d;
    a.dt_bias = dt_bias;
    a.h0 = h0;
    a.lengths = lengths;
    a.h_last = h_last;
    a.states = states;
    return hip_status(ssc::fwd(*s, a, workspace, static_cast<hipStream_t>(stream)));
}

int sscan_bwd(const sscan_shape* s, const gscan_view* x, const gscan_view* dt, const float* a_log,
              const gscan_view* b, const gscan_view* c, const float* d, const gscan_view* z,
              const float* dt_bias, const float* states, const int* lengths, const gscan_view* dy,
              const float* dh_last, const gscan_view* dx, const gscan_view* ddt, float* da_log,
              const gscan_view* db, const gscan_view* dc, float* dd, const gscan_view* dz,
              float* ddt_bias, float* dh0, void* workspace, size_t ws_bytes, void* stream) {
    int rc = check_shape(s);
    if (rc) return rc;
    const long long rows = (long long)s->B * s->D, all = rows * s->N, na = (long long)s->D * s->N;
    const ssc::Plan p = ssc::plan(*s, true);
    // a term's gradient comes with the term
    if (!z != !dz || !d != !dd || !dt_bias != !ddt_bias) return WTCONV_ERR_NULL;
    Bufs q(*s, s->T);
    q.wide(x, false);
    q.wide(dt, false);
    q.low(b, false);
    q.low(c, false);
    if (z) q.wide(z, false);
    q.wide(dy, false);
    q.flat(a_log, na, false, false);
    q.flat(d, s->D, false, true);
    q.flat(dt_bias, s->D, false, true);
    q.flat(states, (long long)(p.states / 4), false, false);
    q.flat(lengths, s->B, false, true);
    q.flat(dh_last, all, false, true);
    q.wide(dx, true);
    q.wide(ddt, true);
    q.low(db, true);
    q.low(dc, true);
    if (dz) q.wide(dz, true);
    q.flat(da_log, na, true, false);
    q.flat(dd, s->D, true, true);
    q.flat(ddt_bias, s->D, true, true);
    q.flat(dh0, all, true, true);
    if (workspace && ws_bytes >= p.scratch) q.flat(workspace, (long long)p.scratch, true, true, 1);
    if ((rc = q.done())) return rc;
    ssc::Args a = args_of(*s);
    a.a_log = a_log;
    a.d = d;
    a.dt_bias = dt_bias;
    a.da_log = da_log;
    a.dd = dd;
    a.ddt_bias = ddt_bias;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (s->B == 0) return hip_status(ssc::bwd_empty(*s, a, st));
    if ((rc = calls::check_ws(p.scratch, workspace, ws_bytes))) return rc;
    put(x, a.x, a.x_sb, a.x_sr);
    put(dt, a.dt, a.dt_sb, a.dt_sr);
    put(b, a.b, a.b_sb, a.b_sr);
    put(c, a.c, a.c_sb, a.c_sr);
    put(dy, a.dy, a.dy_sb, a.dy_sr);
    put(dx, a.dx, a.dx_sb, a.dx_sr);
    put(ddt, a.ddt, a.ddt_sb, a.ddt_sr);
    put(db, a.db, a.db_sb, a.db_sr);
    put(dc, a.dc, a.dc_sb, a.dc_sr);
    if (z) {
        put(z, a.z, a.z_sb, a.z_sr);
        put(dz, a.dz, a.dz_sb, a.dz_sr);
    }
    a.states = const_cast<float*>(states);
    a.lengths = lengths;
    a.dh_last = dh_last;
    a.dh0 = dh0;
    return hip_status(ssc::bwd(*s, a, workspace, st));
}

int sscan_step(const sscan_shape* s, int S, const gscan_view* x, const gscan_view* dt,
               const float* a_log, const gscan_view* b, const gscan_view* c, const float* d,
               const gscan_view* z, const float* dt_bias, float* state, const int* slots,
               const gscan_view* y, void* stream) {
    int rc = check_form(s);  // any number of rows fits its launch
    if (rc) return rc;
    if (S < 0 || (long long)S * s->D > (1LL << 40)) return WTCONV_ERR_SHAPE;
    if (!slots && S < s->B) return WTCONV_ERR_SHAPE;
    Bufs q(*s, 1);
    q.wide(x, false);
    q.wide(dt, false);
    q.low(b, false);
    q.low(c, false);
    if (z) q.wide(z, false);
    q.flat(a_log, (long long)s->D * s->N, false, false);
    q.flat(d, s->D, false, true);
    q.flat(dt_bias, s->D, false, true);
    q.flat(state, (long long)S * s->D * s->N, true, false);
    q.flat(slots, s->B, false, true);
    q.wide(y, true);
    if ((rc = q.done())) return rc;
    if (s->B == 0 || s->D == 0) return WTCONV_OK;
    ssc::StepArgs a{};
    a.x = x->p;
    a.x_sb = x->sb;
    a.dt = dt->p;
    a.dt_sb = dt->sb;
    a.b = b->p;
    a.b_sb = b->sb;
    a.c = c->p;
    a.c_sb = c->sb;
    if (z) {
        a.z = z->p;
        a.z_sb = z->sb;
    }
    a.y = y->p;
    a.y_sb = y->sb;
    a.a_log = a_log;
    a.d = d;
    a.dt_bias = dt_bias;
    a.state = state;
    a.slots = slots;
    a.B = s->B;
    a.D = s->D;
    a.N = s->N;
    a.G = s->G;
    a.Dg = s->D / s->G;
    a.S = S;
    return hip_status(ssc::step(s->dtype, a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

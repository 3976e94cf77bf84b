// C-ABI front end of the root-mean-square norm: argument checks (before anything
// is enqueued), then the kernels.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "call_buffers.h"
#include "rmsnorm.h"
#include "rmsnorm_internal.h"

namespace {

using calls::elem_size;
using calls::hip_status;
using calls::put;

int check_shape(const rmsnorm_shape* s) {
    if (!s) return WTCONV_ERR_NULL;
    if (s->B < 0 || s->T < 0 || s->C < 0 || s->C > (1 << 20)) return WTCONV_ERR_SHAPE;
    if ((long long)s->B * s->T > 0x7fffffffLL) return WTCONV_ERR_SHAPE;
    if (s->dtype != GSCAN_F32 && s->dtype != GSCAN_F16 && s->dtype != GSCAN_BF16)
        return WTCONV_ERR_DTYPE;
    if (s->rdtype != s->dtype && s->rdtype != GSCAN_F32) return WTCONV_ERR_DTYPE;
    return s->eps >= 0.f && isfinite(s->eps) ? WTCONV_OK : WTCONV_ERR_VALUE;
}

// A call's buffers.
class Bufs : public calls::Bufs {
  public:
    explicit Bufs(const rmsnorm_shape& s) : s_(s) {}
    void rows(const gscan_view* v, size_t e, bool out) { view(v, s_.B, s_.T, s_.C, e, out); }

  private:
    const rmsnorm_shape& s_;
};

rmn::Args args_of(const rmsnorm_shape& s) {
    rmn::Args a{};
    a.T = s.T;
    a.C = s.C;
    a.rows = (long long)s.B * s.T;
    a.eps = s.eps;
    return a;
}

bool same(const gscan_view* a, const gscan_view* b) {
    return a->p == b->p && a->sb == b->sb && a->sr == b->sr;
}

int forward(const rmsnorm_shape* s, const gscan_view* x, const gscan_view* residual, const float* w,
            const gscan_view* y, float* scale, const gscan_view* total, float* rstd, bool e4m3,
            void* stream) {
    int rc = check_shape(s);
    if (rc) return rc;
    if (!residual != !total) return WTCONV_ERR_NULL;
    const long long n = (long long)s->B * s->T;
    const size_t e = elem_size(s->dtype), r = elem_size(s->rdtype);
    Bufs q(*s);
    q.rows(x, e, false);
    q.flat(w, s->C, false, false);
    // written in place of the residual, the sum is its only buffer
    if (residual && !same(residual, total)) q.rows(residual, r, false);
    if (total) q.rows(total, r, true);
    q.rows(y, e4m3 ? 1 : e, true);
    if (e4m3) q.flat(scale, n, true, false);
    q.flat(rstd, n, true, true);
    if ((rc = q.done())) return rc;
    if (n == 0) return WTCONV_OK;  // rows of no elements have an rstd and a scale too
    rmn::Args a = args_of(*s);
    put(x, a.x, a.x_sb, a.x_sr);
    if (residual) {
        put(residual, a.res, a.res_sb, a.res_sr);
        put(total, a.total, a.total_sb, a.total_sr);
    }
    put(y, a.y, a.y_sb, a.y_sr);
    a.w = w;
    a.rstd = rstd;
    a.scale = scale;
    rmsnorm_shape form = *s;
    if (!residual) form.rdtype = form.dtype;  // nothing is of the other type
    return hip_status(rmn::fwd(form, a, e4m3, static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

int rmsnorm_workspace_size(const rmsnorm_shape* s, size_t* bytes) {
    const int rc = check_shape(s);
    if (rc) return rc;
    if (!bytes) return WTCONV_ERR_NULL;
    *bytes = rmn::plan(*s).scratch;
    return WTCONV_OK;
}

int rmsnorm_fwd(const rmsnorm_shape* s, const gscan_view* x, const gscan_view* residual,
                const float* w, const gscan_view* y, const gscan_view* total, float* rstd,
                void* stream) {
    return forward(s, x, residual, w, y, nullptr, total, rstd, false, stream);
}

int rmsnorm_fwd_e4m3(const rmsnorm_shape* s, const gscan_view* x, const gscan_view* residual,
                     const float* w, const gscan_view* codes, float* scale,
                     const gscan_view* total, float* rstd, void* stream) {
    return forward(s, x, residual, w, codes, scale, total, rstd, true, stream);
}

int rmsnorm_bwd(const rmsnorm_shape* s, const gscan_view* kept, const float* w, const float* rstd,
                const gscan_view* dy, const gscan_view* dtotal, const gscan_view* dx,
                const gscan_view* dresidual, float* dw, void* workspace, size_t ws_bytes,
                void* stream) {
    int rc = check_shape(s);
    if (rc) return rc;
    const long long n = (long long)s->B * s->T;
    const size_t e = elem_size(s->dtype), r = elem_size(s->rdtype);
    const rmn::Plan p = rmn::plan(*s);
    Bufs q(*s);
    q.rows(kept, r, false);
    q.flat(w, s->C, false, false);
    q.flat(rstd, n, false, false);
    q.rows(dy, e, false);
    if (dtotal) q.rows(dtotal, r, false);
    if (dx) q.rows(dx, e, true);
    if (dresidual) q.rows(dresidual, r, true);
    q.flat(dw, s->C, true, true);
    if (workspace && ws_bytes >= p.scratch) q.flat(workspace, (long long)p.scratch, true, true, 1);
    if ((rc = q.done())) return rc;
    if (s->C == 0) return WTCONV_OK;
    if ((rc = calls::check_ws(p.scratch, workspace, ws_bytes))) return rc;
    rmn::Args a = args_of(*s);
    put(kept, a.kept, a.kept_sb, a.kept_sr);
    put(dy, a.dy, a.dy_sb, a.dy_sr);
    if (dtotal) put(dtotal, a.dtotal, a.dtotal_sb, a.dtotal_sr);
    if (dx) put(dx, a.dx, a.dx_sb, a.dx_sr);
    if (dresidual) put(dresidual, a.dres, a.dres_sb, a.dres_sr);
    a.w = w;
    a.rstd_in = rstd;
    a.dw = dw;
    return hip_status(rmn::bwd(*s, a, workspace, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

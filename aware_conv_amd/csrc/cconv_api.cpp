// C-ABI front end of the causal convolution: argument checks (before anything is
// enqueued), then the kernels.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "call_buffers.h"
#include "cconv.h"
#include "cconv_internal.h"
#include "close_sums.h"

namespace {

using calls::elem_size;
using calls::hip_status;
using calls::put;

int check_form(const cconv_shape* s) {
    if (!s) return WTCONV_ERR_NULL;
    if (s->B < 0 || s->T < 0 || s->C < 0 || s->T > (1 << 30)) return WTCONV_ERR_SHAPE;
    if (s->K < 1 || s->K > CCONV_MAX_TAPS) return WTCONV_ERR_SHAPE;
    if (s->dtype != GSCAN_F32 && s->dtype != GSCAN_F16 && s->dtype != GSCAN_BF16)
        return WTCONV_ERR_DTYPE;
    if ((long long)s->C * s->K > (1LL << 27)) return WTCONV_ERR_SHAPE;
    return (long long)s->B * s->C > (1LL << 31) ? WTCONV_ERR_SHAPE : WTCONV_OK;
}
int check_shape(const cconv_shape* s) {
    const int rc = check_form(s);
    if (rc) return rc;
    return ccv::plan(*s).fits ? WTCONV_OK : WTCONV_ERR_UNSUPPORTED;
}

ccv::Args args_of(const cconv_shape& s) {
    ccv::Args a{};
    a.B = s.B;
    a.T = s.T;
    a.C = s.C;
    a.K = s.K;
    a.silu = s.silu != 0;
    return a;
}

}  // namespace

extern "C" {

int cconv_workspace_size(const cconv_shape* s, size_t* bytes) {
    const int rc = check_shape(s);
    if (rc) return rc;
    if (!bytes) return WTCONV_ERR_NULL;
    *bytes = ccv::plan(*s).scratch;
    return WTCONV_OK;
}

int cconv_fwd(const cconv_shape* s, const gscan_view* x, const float* w, const float* bias,
              const void* h0, const int* lengths, const gscan_view* y, void* last, void* stream) {
    int rc = check_shape(s);
    if (rc) return rc;
    const size_t e = elem_size(s->dtype);
    const long long kept = (long long)s->B * (s->K - 1) * s->C;
    calls::Bufs q;
    q.view(x, s->B, s->T, s->C, e, false);
    q.flat(w, (long long)s->C * s->K, false, false);
    q.flat(bias, s->C, false, true);
    q.flat(h0, kept, false, true, e);
    q.flat(lengths, s->B, false, true);
    q.view(y, s->B, s->T, s->C, e, true);
    q.flat(last, kept, true, true, e);
    if ((rc = q.done())) return rc;
    if (s->B == 0 || s->C == 0) return WTCONV_OK;
    ccv::Args a = args_of(*s);
    put(x, a.x, a.x_sb, a.x_sr);
    put(y, a.y, a.y_sb, a.y_sr);
    a.w = w;
    a.bias = bias;
    a.h0 = h0;
    a.lengths = lengths;
    a.last = last;
    return hip_status(ccv::fwd(s->dtype, a, static_cast<hipStream_t>(stream)));
}

int cconv_bwd(const cconv_shape* s, const gscan_view* x, const float* w, const float* bias,
              const void* h0, const int* lengths, const gscan_view* dy, const void* dlast,
              const gscan_view* dx, float* dw, float* dbias, void* dh0, void* workspace,
              size_t ws_bytes, void* stream) {
    int rc = check_shape(s);
    if (rc) return rc;
    if (!bias != !dbias) return WTCONV_ERR_NULL;  // a term's gradient comes with the term
    if (!calls::close_fits((long long)s->C * s->K, bias ? s->C : 0)) return WTCONV_ERR_UNSUPPORTED;
    const ccv::Plan p = ccv::plan(*s);
    const size_t e = elem_size(s->dtype);
    const long long kept = (long long)s->B * (s->K - 1) * s->C;
    calls::Bufs q;
    q.view(x, s->B, s->T, s->C, e, false);
    q.flat(w, (long long)s->C * s->K, false, false);
    q.flat(bias, s->C, false, true);
    q.flat(h0, kept, false, true, e);
    q.flat(lengths, s->B, false, true);
    q.view(dy, s->B, s->T, s->C, e, false);
    q.flat(dlast, kept, false, true, e);
    q.view(dx, s->B, s->T, s->C, e, true);
    q.flat(dw, (long long)s->C * s->K, true, false);
    q.flat(dbias, s->C, true, true);
    q.flat(dh0, kept, true, true, e);
    if (workspace && ws_bytes >= p.scratch) q.flat(workspace, (long long)p.scratch, true, true, 1);
    if ((rc = q.done())) return rc;
    if (s->C == 0) return WTCONV_OK;
    if ((rc = calls::check_ws(p.scratch, workspace, ws_bytes))) return rc;
    ccv::Args a = args_of(*s);
    put(x, a.x, a.x_sb, a.x_sr);
    put(dy, a.dy, a.dy_sb, a.dy_sr);
    put(dx, a.dx, a.dx_sb, a.dx_sr);
    a.w = w;
    a.bias = bias;
    a.h0 = h0;
    a.lengths = lengths;
    a.dlast = dlast;
    a.dw = dw;
    a.dbias = dbias;
    a.dh0 = dh0;
    return hip_status(ccv::bwd(*s, a, workspace, static_cast<hipStream_t>(stream)));
}

int cconv_step(const cconv_shape* s, int S, const gscan_view* x, const float* w, const float* bias,
               void* cache, const int* slots, const gscan_view* y, void* stream) {
    int rc = check_form(s);  // any number of rows fits its launch
    if (rc) return rc;
    if (S < 0 || (long long)S * s->C > (1LL << 40)) return WTCONV_ERR_SHAPE;
    if (!slots && S < s->B) return WTCONV_ERR_SHAPE;
    const size_t e = elem_size(s->dtype);
    calls::Bufs q;
    q.view(x, s->B, 1, s->C, e, false);
    q.flat(w, (long long)s->C * s->K, false, false);
    q.flat(bias, s->C, false, true);
    q.flat(cache, (long long)S * (s->K - 1) * s->C, true, false, e);
    q.flat(slots, s->B, false, true);
    q.view(y, s->B, 1, s->C, e, true);
    if ((rc = q.done())) return rc;
    if (s->B == 0 || s->C == 0) return WTCONV_OK;
    ccv::StepArgs a{};
    a.x = x->p;
    a.x_sb = x->sb;
    a.y = y->p;
    a.y_sb = y->sb;
    a.w = w;
    a.bias = bias;
    a.cache = cache;
    a.slots = slots;
    a.B = s->B;
    a.C = s->C;
    a.K = s->K;
    a.S = S;
    a.silu = s->silu != 0;
    return hip_status(ccv::step(s->dtype, a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

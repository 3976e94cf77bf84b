// C-ABI front end of the gated linear recurrence: argument checks (before
// anything is enqueued), then the kernels of the layout.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "gscan.h"
#include "gscan_internal.h"

namespace {

// Rows (sequences x channels) of a call: a wavefront each, and a launch holds
// fewer than 2^32 threads.
constexpr long long kMaxRows = 1LL << 25;

size_t elem_size(int dtype) { return dtype == GSCAN_F32 ? 4 : 2; }
bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

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

// A buffer of the call: `rows` runs of `run` adjacent elements per sequence.
struct Buf {
    uintptr_t p;
    long long B, sb, R, sr, run;  // R rows of stride sr in each of B sequences
    size_t e;
    bool out;
};

// Elements from the first to one past the last; -1 where that is absurd.
long long span(const Buf& q) {
    if (q.B == 0 || q.R == 0 || q.run == 0) return 0;
    const double far = double(q.B - 1) * double(q.sb) + double(q.R - 1) * double(q.sr) + double(q.run);
    if (far > 1e15) return -1;
    return (q.B - 1) * q.sb + (q.R - 1) * q.sr + q.run;
}

// Whether no element of the buffer lies on another of it.
bool own_apart(const Buf& q) {
    if (span(q) == 0) return true;
    const long long rows = q.R > 1 ? (q.R - 1) * q.sr + q.run : q.run;
    if (q.R <= 1 || q.sr >= q.run) {
        if (q.B <= 1 || q.sb >= rows) return true;
        // sequences inside rows
        if (q.sb >= q.run && (q.R <= 1 || q.sr >= (q.B - 1) * q.sb + q.run)) return true;
    }
    return false;
}

// Whether buffers of the same strides that share a span are known to have no
// element in common: their runs lie side by side at every row or sequence.
bool side_by_side(const Buf& a, const Buf& b) {
    if (a.B != b.B || a.sb != b.sb || a.R != b.R || a.sr != b.sr || a.run != b.run || a.e != b.e)
        return false;
    const long long bytes = (long long)(b.p - a.p);
    if (bytes % (long long)a.e) return false;
    long long d = bytes / (long long)a.e;
    if (d < 0) d = -d;
    // from the outer stride inwards: at each, either what the other holds lies
    // in the gap that the stride leaves, or only the remainder matters
    long long outer = a.sb, on = a.B, inner = a.sr, in = a.R;
    if (a.sr > a.sb) {
        outer = a.sr;
        on = a.R;
        inner = a.sb;
        in = a.B;
    }
    const long long block = in > 1 ? (in - 1) * inner + a.run : a.run;
    if (on > 1) {
        if (outer < block) return false;
        const long long z = d % outer;
        if (z >= block && outer - z >= block) return true;
        // within one block of rows; a remainder that reaches around leaves it open
        if (z >= block) return false;
        d = z;
    }
    if (in > 1) {
        if (inner < a.run) return false;
        const long long z = d % inner;
        // a remainder that reaches into the next block of rows meets the same
        // remainder there only if the outer stride is a whole number of rows
        if (on > 1 && outer % inner) return false;
        return z >= a.run && inner - z >= a.run;
    }
    return d >= a.run;
}

bool clash(const Buf& a, const Buf& b) {
    const long long na = span(a), nb = span(b);
    if (na == 0 || nb == 0) return false;
    if (a.p >= b.p + size_t(nb) * b.e || b.p >= a.p + size_t(na) * a.e) return false;
    return !side_by_side(a, b);
}

// The buffers of a call, checked as they are added.
class Bufs {
  public:
    explicit Bufs(const gscan_shape& s) : s_(s) {}
    // an activation
    void view(const gscan_view* v, bool out) {
        if (rc_) return;
        if (!v) return fail(WTCONV_ERR_NULL);
        const long long R = s_.layout == GSCAN_BCT ? s_.C : s_.T;
        const long long run = s_.layout == GSCAN_BCT ? s_.T : s_.C;
        if (s_.B == 0 || R == 0 || run == 0) return;
        if (!v->p) return fail(WTCONV_ERR_NULL);
        if (v->sb < 0 || v->sr < 0) return fail(WTCONV_ERR_LAYOUT);
        add(Buf{reinterpret_cast<uintptr_t>(v->p), s_.B, v->sb, R, v->sr, run, elem_size(s_.dtype), out});
    }
    // `n` contiguous elements of `e` bytes; NULL only where `optional`
    void flat(const void* p, long long n, bool out, bool optional, size_t e = 4) {
        if (rc_ || n == 0) return;
        if (!p) {
            if (!optional) fail(WTCONV_ERR_NULL);
            return;
        }
        add(Buf{reinterpret_cast<uintptr_t>(p), 1, n, 1, n, n, e, out});
    }
    int done() const {
        if (rc_) return rc_;
        for (int i = 0; i < n_; ++i)
            for (int j = i + 1; j < n_; ++j)
                if ((b_[i].out || b_[j].out) && clash(b_[i], b_[j])) return WTCONV_ERR_ALIAS;
        return WTCONV_OK;
    }

  private:
    void fail(int rc) { rc_ = rc; }
    void add(const Buf& q) {
        if (q.p % q.e) return fail(WTCONV_ERR_ALIGN);
        if (span(q) < 0) return fail(WTCONV_ERR_SHAPE);
        if (q.out && !own_apart(q)) return fail(WTCONV_ERR_LAYOUT);
        b_[n_++] = q;
    }
    const gscan_shape& s_;
    Buf b_[20];
    int n_ = 0, rc_ = WTCONV_OK;
};

int check_ws(const gsc::Plan& p, const void* ws, size_t bytes) {
    if (bytes < p.scratch) return WTCONV_ERR_WORKSPACE;
    if (p.scratch && !ws) return WTCONV_ERR_NULL;
    if (p.scratch && !aligned(ws, 16)) return WTCONV_ERR_ALIGN;
    return WTCONV_OK;
}

void put(const gscan_view* v, const void*& p, long long& sb, long long& sr) {
    p = v->p;
    sb = v->sb;
    sr = v->sr;
}
void put(const gscan_view* v, void*& p, long long& sb, long long& sr) {
    p = v->p;
    sb = v->sb;
    sr = v->sr;
}

int hip_status(hipError_t e) { return e == hipSuccess ? WTCONV_OK : WTCONV_ERR_HIP; }

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

// Checks of the buffers that a call of a sequence operator is given: strided
// activations and contiguous tensors, none of whose outputs may lie on another
// buffer or on itself.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gscan.h"

namespace calls {

inline size_t elem_size(int dtype) { return dtype == GSCAN_F32 ? 4 : 2; }
inline bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// A buffer of the call: rows of adjacent elements per sequence.
struct Buf {
    uintptr_t p;
    long long B, sb, R, sr, run;  // R rows of stride sr in each of B sequences
    size_t e;
    bool out;
};

// Elements from the first to one past the last; -1 where that is absurd.
inline long long span(const Buf& q) {
    if (q.B == 0 || q.R == 0 || q.run == 0) return 0;
    const double far = double(q.B - 1) * double(q.sb) + double(q.R - 1) * double(q.sr) + double(q.run);
    if (far > 1e15) return -1;
    return (q.B - 1) * q.sb + (q.R - 1) * q.sr + q.run;
}

// Whether no element of the buffer lies on another of it.
inline bool own_apart(const Buf& q) {
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
inline bool side_by_side(const Buf& a, const Buf& b) {
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

inline bool clash(const Buf& a, const Buf& b) {
    const long long na = span(a), nb = span(b);
    if (na == 0 || nb == 0) return false;
    if (a.p >= b.p + size_t(nb) * b.e || b.p >= a.p + size_t(na) * a.e) return false;
    return !side_by_side(a, b);
}

// The buffers of a call, checked as they are added; the first fault stays.
class Bufs {
  public:
    // `rows` rows of `run` adjacent elements in each of B sequences
    void view(const gscan_view* v, long long B, long long rows, long long run, size_t e, bool out) {
        if (rc_) return;
        if (!v) return fail(WTCONV_ERR_NULL);
        if (B == 0 || rows == 0 || run == 0) return;
        if (!v->p) return fail(WTCONV_ERR_NULL);
        if (v->sb < 0 || v->sr < 0) return fail(WTCONV_ERR_LAYOUT);
        add(Buf{reinterpret_cast<uintptr_t>(v->p), B, v->sb, rows, v->sr, run, e, out});
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
        if (n_ == kMost) return fail(WTCONV_ERR_UNSUPPORTED);
        b_[n_++] = q;
    }
    static constexpr int kMost = 32;
    Buf b_[kMost];
    int n_ = 0, rc_ = WTCONV_OK;
};

inline int check_ws(size_t need, const void* ws, size_t bytes) {
    if (bytes < need) return WTCONV_ERR_WORKSPACE;
    if (need && !ws) return WTCONV_ERR_NULL;
    if (need && !aligned(ws, 16)) return WTCONV_ERR_ALIGN;
    return WTCONV_OK;
}

// The handed-over view as pointer and strides.
inline void put(const gscan_view* v, const void*& p, long long& sb, long long& sr) {
    p = v->p;
    sb = v->sb;
    sr = v->sr;
}
inline void put(const gscan_view* v, void*& p, long long& sb, long long& sr) {
    p = v->p;
    sb = v->sb;
    sr = v->sr;
}

inline int hip_status(hipError_t e) { return e == hipSuccess ? WTCONV_OK : WTCONV_ERR_HIP; }

}  // namespace calls

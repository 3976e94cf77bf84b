// Gated linear recurrence over planes ([B][C][T], time contiguous).
//
// A row (b, c) is scanned by LW neighbouring lanes of a wavefront.  A tile is
// LW * V positions: each lane takes V consecutive ones, composes their maps
// h -> a h + b in registers, the lanes' compositions are scanned with DPP
// moves (no LDS), and each lane runs its V steps again from the state that it
// then knows.  The state passes from tile to tile in a register.  Everything
// is read once and written once.
//
// Backwards the same tile gives h (from the state the forward kept for it)
// and, for the sequence u_t = a_t g_t that passes from position to position,
// the maps u -> a (dh + u), scanned in the other direction.
#include <hip/hip_runtime.h>

#include "gscan_math.h"

namespace gsc {
namespace {

constexpr int kThreads = 256;

// Value of `v` at the lane CTRL names, `idle` where there is none.
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ float dpp(float v, float idle) {
    return __builtin_bit_cast(
        float, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, idle), __builtin_bit_cast(int, v),
                                           CTRL, ROWS, 0xf, false));
}

// (a, h) becomes the composition of the maps of this lane and the one CTRL
// names, which comes earlier.
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ void compose(float& a, float& h) {
    const float pa = dpp<CTRL, ROWS>(a, 1.f), ph = dpp<CTRL, ROWS>(h, 0.f);
    h = fmaf(a, ph, h);
    a *= pa;
}

// Inclusive scan over each group of LW lanes (64, 16 or 1).
template <int LW>
__device__ __forceinline__ void lane_scan(float& a, float& h) {
    if constexpr (LW >= 16) {
        compose<0x111>(a, h);  // row_shr:1, 2, 4, 8 within rows of 16
        compose<0x112>(a, h);
        compose<0x114>(a, h);
        compose<0x118>(a, h);
    }
    if constexpr (LW == 64) {
        compose<0x142, 0xa>(a, h);  // row_bcast:15 into rows 1 and 3
        compose<0x143, 0xc>(a, h);  // row_bcast:31 into rows 2 and 3
    }
}

// The value of the lane before (idle in the first lane of a group).
template <int LW>
__device__ __forceinline__ float lane_before(float v, float idle) {
    if constexpr (LW == 64) return dpp<0x138>(v, idle);       // wave_shr:1
    else if constexpr (LW == 16) return dpp<0x111>(v, idle);  // row_shr:1
    else return idle;
}
// The value of the last lane of the group.
template <int LW>
__device__ __forceinline__ float lane_last(float v) {
    if constexpr (LW == 64)
        return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
    else if constexpr (LW == 16) return __shfl(v, int(threadIdx.x & 63) | 15);
    else return v;
}
// The value of the mirrored lane of the group.
template <int LW>
__device__ __forceinline__ float lane_mirror(float v) {
    if constexpr (LW == 1) return v;
    else return __shfl_xor(v, LW - 1);
}
template <int LW>
__device__ __forceinline__ float lane_sum(float v) {
#pragma unroll
    for (int d = LW / 2; d > 0; d /= 2) v += __shfl_xor(v, d);
    return v;
}

// Positions p0 .. p0 + V - 1 of a row in scan order, `len` of them valid.
// REV: position p lies at len - 1 - p.
template <class D, int V, bool REV>
__device__ __forceinline__ void fetch(Raw<D, V>& out, const typename D::S* row, int p0, int len) {
    if (p0 + V <= len) {
        load_vec<D, V>(out, row + (REV ? len - V - p0 : p0));
    } else {
#pragma unroll
        for (int k = 0; k < Raw<D, V>::kWords; ++k) out.w[k] = 0;
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (p0 + j < len) out.set(REV ? V - 1 - j : j, load_one<D>(row + (REV ? len - 1 - p0 - j : p0 + j)));
    }
}
// The same positions written; those in len .. T - 1 (which lie at their own
// index in both directions) become zero.
template <class D, int V, bool REV>
__device__ __forceinline__ void put(typename D::S* row, const float (&v)[V], int p0, int len,
                                    int T) {
    if (p0 + V <= len) {
        Raw<D, V> q;
#pragma unroll
        for (int k = 0; k < Raw<D, V>::kWords; ++k) q.w[k] = 0;
#pragma unroll
        for (int j = 0; j < V; ++j) q.set(REV ? V - 1 - j : j, v[j]);
        store_vec<D, V>(row + (REV ? len - V - p0 : p0), q);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int p = p0 + j;
            if (p < len) store_one<D>(row + (REV ? len - 1 - p : p), v[j]);
            else if (p < T) store_one<D>(row + p, 0.f);
        }
    }
}
template <class D, int V, bool REV>
__device__ __forceinline__ float at(const Raw<D, V>& q, int j) {
    return q.get(REV ? V - 1 - j : j);
}

template <class S>
__device__ __forceinline__ S* row_of(const void* p, long long sb, long long sr, int b, int c) {
    return const_cast<S*>(static_cast<const S*>(p)) + b * sb + c * sr;
}

struct Row {
    int b, c, len;
    long long id;  // b * C + c
    bool live;
};
template <int LW>
__device__ __forceinline__ Row my_row(const Args& g) {
    Row w;
    const long long rows = (long long)g.B * g.C;
    w.id = (long long)blockIdx.x * (kThreads / LW) + threadIdx.x / LW;
    w.live = w.id < rows;
    const long long id = w.live ? w.id : rows - 1;
    w.b = int(id / g.C);
    w.c = int(id - (long long)w.b * g.C);
    w.len = g.T;
    if (g.lengths) w.len = min(max(g.lengths[w.b], 0), g.T);
    return w;
}

template <class D, int V, int LW, bool REV>
__global__ __launch_bounds__(kThreads) void k_planes_fwd(Args g) {
    using S = typename D::S;
    const Row w = my_row<LW>(g);
    if (!w.live) return;  // whole groups of lanes
    const long long rows = (long long)g.B * g.C;
    const int lane = threadIdx.x % LW;
    const S* x = row_of<const S>(g.x, g.x_sb, g.x_sr, w.b, w.c);
    const S* r = row_of<const S>(g.r, g.r_sb, g.r_sr, w.b, w.c);
    const S* i = row_of<const S>(g.i, g.i_sb, g.i_sr, w.b, w.c);
    S* h = row_of<S>(g.h, g.h_sb, g.h_sr, w.b, w.c);
    const float rate = g.decay * softplus(g.lam[w.c]) * kLog2e;
    float carry = g.h0 ? g.h0[w.id] : 0.f;
    for (int n = 0; n < g.tiles; ++n) {
        const int p0 = (n * LW + lane) * V;
        if (g.states && lane == 0) g.states[n * rows + w.id] = carry;
        Raw<D, V> qx, qr, qi;
        fetch<D, V, REV>(qx, x, p0, w.len);
        fetch<D, V, REV>(qr, r, p0, w.len);
        fetch<D, V, REV>(qi, i, p0, w.len);
        float a[V], b[V];
        float A = 1.f, H = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            gate_fwd(at<D, V, REV>(qx, j), at<D, V, REV>(qr, j), at<D, V, REV>(qi, j), rate, a[j],
                     b[j]);
            if (p0 + j >= w.len) {
                a[j] = 1.f;
                b[j] = 0.f;
            }
            H = fmaf(a[j], H, b[j]);
            A *= a[j];
        }
        lane_scan<LW>(A, H);
        float s = fmaf(lane_before<LW>(A, 1.f), carry, lane_before<LW>(H, 0.f));
        carry = fmaf(lane_last<LW>(A), carry, lane_last<LW>(H));
#pragma unroll
        for (int j = 0; j < V; ++j) {
            s = fmaf(a[j], s, b[j]);
            b[j] = s;
        }
        put<D, V, REV>(h, b, p0, w.len, g.T);
    }
    if (g.h_last && lane == 0) g.h_last[w.id] = carry;
}

template <class D, int V, int LW, bool REV>
__global__ __launch_bounds__(kThreads) void k_planes_bwd(Args g) {
    using S = typename D::S;
    const Row w = my_row<LW>(g);
    if (!w.live) return;
    const long long rows = (long long)g.B * g.C;
    const int lane = threadIdx.x % LW;
    const S* x = row_of<const S>(g.x, g.x_sb, g.x_sr, w.b, w.c);
    const S* r = row_of<const S>(g.r, g.r_sb, g.r_sr, w.b, w.c);
    const S* i = row_of<const S>(g.i, g.i_sb, g.i_sr, w.b, w.c);
    const S* dh = row_of<const S>(g.dh, g.dh_sb, g.dh_sr, w.b, w.c);
    S* dx = row_of<S>(g.dx, g.dx_sb, g.dx_sr, w.b, w.c);
    S* dr = row_of<S>(g.dr, g.dr_sb, g.dr_sr, w.b, w.c);
    S* di = row_of<S>(g.di, g.di_sb, g.di_sr, w.b, w.c);
    const float rate = g.decay * softplus(g.lam[w.c]) * kLog2e;
    float after = g.dh_last ? g.dh_last[w.id] : 0.f;  // u of the position after the tile
    float sum = 0.f;
    for (int n = g.tiles - 1; n >= 0; --n) {
        const int p0 = (n * LW + lane) * V;
        Raw<D, V> qx, qr, qi, qd;
        fetch<D, V, REV>(qx, x, p0, w.len);
        fetch<D, V, REV>(qr, r, p0, w.len);
        fetch<D, V, REV>(qi, i, p0, w.len);
        fetch<D, V, REV>(qd, dh, p0, w.len);
        const float carry = g.states[n * rows + w.id];
        float a[V], hp[V], d[V];
        float A = 1.f, H = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            gate_fwd(at<D, V, REV>(qx, j), at<D, V, REV>(qr, j), at<D, V, REV>(qi, j), rate, a[j],
                     hp[j]);
            if (p0 + j >= w.len) {
                a[j] = 1.f;
                hp[j] = 0.f;
            }
            d[j] = at<D, V, REV>(qd, j);
            H = fmaf(a[j], H, hp[j]);
            A *= a[j];
        }
        float B = A, U = 0.f;
#pragma unroll
        for (int j = V - 1; j >= 0; --j) U = a[j] * (d[j] + U);
        lane_scan<LW>(A, H);
        float s = fmaf(lane_before<LW>(A, 1.f), carry, lane_before<LW>(H, 0.f));
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float b = hp[j];
            hp[j] = s;
            s = fmaf(a[j], s, b);
        }
        B = lane_mirror<LW>(B);
        U = lane_mirror<LW>(U);
        lane_scan<LW>(B, U);
        const float Bb = lane_mirror<LW>(lane_before<LW>(B, 1.f));
        const float Ub = lane_mirror<LW>(lane_before<LW>(U, 0.f));
        float u = fmaf(Bb, after, Ub);
        after = fmaf(lane_last<LW>(B), after, lane_last<LW>(U));
        float ox[V], orr[V], oi[V];
#pragma unroll
        for (int j = V - 1; j >= 0; --j) {
            const float gt = d[j] + u;
            float e;
            gate_bwd(at<D, V, REV>(qx, j), at<D, V, REV>(qr, j), at<D, V, REV>(qi, j), rate, a[j],
                     hp[j], gt, ox[j], orr[j], oi[j], e);
            sum += p0 + j < w.len ? e : 0.f;
            u = a[j] * gt;
        }
        put<D, V, REV>(dx, ox, p0, w.len, g.T);
        put<D, V, REV>(dr, orr, p0, w.len, g.T);
        put<D, V, REV>(di, oi, p0, w.len, g.T);
    }
    sum = lane_sum<LW>(sum);
    if (lane == 0) {
        g.part[w.id] = sum;
        if (g.dh0) g.dh0[w.id] = after;
    }
}

// Lanes per row and positions per lane, by the row's length alone, so that
// the states of a forward call fit the backward one: the narrowest group that
// holds the row in one tile, else whole wavefronts of 8 positions per lane.
struct Form {
    int V, LW;
};
Form form_of(int T) {
    if (T <= 4) return {4, 1};
    if (T <= 64) return {4, 16};
    if (T <= 256) return {4, 64};
    return {8, 64};
}

template <class D, int V, int LW>
void launch(bool bwd, bool rev, const Args& a, hipStream_t st) {
    const long long rows = (long long)a.B * a.C;
    const int per = kThreads / LW;
    const dim3 grid((unsigned)((rows + per - 1) / per));
    if (bwd) {
        if (rev) k_planes_bwd<D, V, LW, true><<<grid, kThreads, 0, st>>>(a);
        else k_planes_bwd<D, V, LW, false><<<grid, kThreads, 0, st>>>(a);
    } else {
        if (rev) k_planes_fwd<D, V, LW, true><<<grid, kThreads, 0, st>>>(a);
        else k_planes_fwd<D, V, LW, false><<<grid, kThreads, 0, st>>>(a);
    }
}
template <class D>
void launch_form(bool bwd, bool rev, const Args& a, hipStream_t st) {
    const Form f = form_of(a.T);
    if (f.LW == 1) launch<D, 4, 1>(bwd, rev, a, st);
    else if (f.LW == 16) launch<D, 4, 16>(bwd, rev, a, st);
    else if (f.V == 4) launch<D, 4, 64>(bwd, rev, a, st);
    else launch<D, 8, 64>(bwd, rev, a, st);
}
void launch_type(int dtype, bool bwd, bool rev, const Args& a, hipStream_t st) {
    if (dtype == GSCAN_F32) launch_form<F32>(bwd, rev, a, st);
    else if (dtype == GSCAN_F16) launch_form<F16>(bwd, rev, a, st);
    else launch_form<BF16>(bwd, rev, a, st);
}

}  // namespace

Plan planes_plan(const gscan_shape& s) {
    const Form f = form_of(s.T);
    const int tile = f.V * f.LW;
    Plan p;
    p.tiles = s.T > 0 ? (s.T - 1) / tile + 1 : 1;
    p.parts = s.B;
    p.states = sizeof(float) * size_t(p.tiles) * s.B * s.C;
    p.scratch = sizeof(float) * size_t(p.parts) * s.C;
    return p;
}

hipError_t planes_fwd(const gscan_shape& s, Args a, void*, hipStream_t st) {
    a.tiles = planes_plan(s).tiles;
    launch_type(s.dtype, false, s.reverse != 0, a, st);
    return hipGetLastError();
}

hipError_t planes_bwd(const gscan_shape& s, Args a, void* ws, hipStream_t st) {
    const Plan p = planes_plan(s);
    a.tiles = p.tiles;
    a.part = static_cast<float*>(ws);
    launch_type(s.dtype, true, s.reverse != 0, a, st);
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? close_dlam(a, p.parts, st) : e;
}

}  // namespace gsc

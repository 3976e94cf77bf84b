// Gated linear recurrence over tokens ([B][T][C], channels contiguous), and
// its form for one position.
//
// A workgroup takes 64 channels of one sequence and walks tiles of kSub * kLen
// positions.  A thread takes two neighbouring channels and kLen consecutive
// positions: it composes their maps h -> a h + b in registers, the kSub
// compositions of a channel meet in LDS, and each thread runs its positions
// again from the state that it then knows.  Everything is read once and
// written once.
#include <hip/hip_runtime.h>

#include "gscan_math.h"

namespace gsc {
namespace {

constexpr int kLanes = 32;             // threads across the channels of a tile
constexpr int kChan = 2 * kLanes;      // channels of a tile
constexpr int kSub = 16;               // threads along time
constexpr int kLen = 8;                // positions of a thread
constexpr int kTile = kSub * kLen;     // positions of a tile
constexpr int kThreads = kLanes * kSub;

// Two channels at one position; `n` of them exist (0, 1 or 2).
template <class D>
__device__ __forceinline__ Raw<D, 2> fetch2(const typename D::S* p, int n) {
    Raw<D, 2> q;
#pragma unroll
    for (int k = 0; k < Raw<D, 2>::kWords; ++k) q.w[k] = 0;
    if (n == 2) load_vec<D, 2>(q, p);
    else if (n == 1) q.set(0, load_one<D>(p));
    return q;
}
template <class D>
__device__ __forceinline__ void put2(typename D::S* p, float v0, float v1, int n) {
    if (n == 2) {
        Raw<D, 2> q;
#pragma unroll
        for (int k = 0; k < Raw<D, 2>::kWords; ++k) q.w[k] = 0;
        q.set(0, v0);
        q.set(1, v1);
        store_vec<D, 2>(p, q);
    } else if (n == 1) {
        store_one<D>(p, v0);
    }
}

// What a thread works on.
struct Me {
    int b, c, n;  // sequence, first channel, channels that exist
    int cl, sub;  // place in the tile
    int len;
};
__device__ __forceinline__ Me me_of(const Args& g) {
    Me m;
    const unsigned wide = (g.C + kChan - 1) / kChan;
    m.b = blockIdx.x / wide;
    m.cl = threadIdx.x % kLanes;
    m.sub = threadIdx.x / kLanes;
    m.c = (blockIdx.x % wide) * kChan + 2 * m.cl;
    m.n = min(max(g.C - m.c, 0), 2);
    m.len = g.T;
    if (g.lengths) m.len = min(max(g.lengths[m.b], 0), g.T);
    return m;
}

// First element of the thread's channels at scan position p (< len), or at
// its own index beyond.
template <class S>
__device__ __forceinline__ S* place(const void* base, long long sb, long long sr, const Me& m,
                                    int p, bool rev) {
    const int t = rev && p < m.len ? m.len - 1 - p : p;
    return const_cast<S*>(static_cast<const S*>(base)) + m.b * sb + t * sr + m.c;
}

struct Two {
    float a0, h0, a1, h1;
};

__device__ __forceinline__ void rates(const Args& g, const Me& m, float (&rate)[2]) {
    rate[0] = m.n > 0 ? g.decay * softplus(g.lam[m.c]) * kLog2e : 0.f;
    rate[1] = m.n > 1 ? g.decay * softplus(g.lam[m.c + 1]) * kLog2e : 0.f;
}

template <class D>
__global__ __launch_bounds__(kThreads) void k_tokens_fwd(Args g, bool rev) {
    using S = typename D::S;
    __shared__ Two part[2][kSub][kLanes];
    __shared__ float2 state[2][kLanes];
    const Me m = me_of(g);
    const size_t at = size_t(m.b) * g.C + m.c;
    float rate[2];
    rates(g, m, rate);
    if (m.sub == 0) {
        float2 s{0.f, 0.f};
        if (g.h0 && m.n > 0) s.x = g.h0[at];
        if (g.h0 && m.n > 1) s.y = g.h0[at + 1];
        state[0][m.cl] = s;
    }
    for (int n = 0; n < g.tiles; ++n) {
        const int p0 = n * kTile + m.sub * kLen;
        Raw<D, 2> qx[kLen], qr[kLen], qi[kLen];
#pragma unroll
        for (int j = 0; j < kLen; ++j) {
            const int k = p0 + j < m.len ? m.n : 0;
            qx[j] = fetch2<D>(place<const S>(g.x, g.x_sb, g.x_sr, m, p0 + j, rev), k);
            qr[j] = fetch2<D>(place<const S>(g.r, g.r_sb, g.r_sr, m, p0 + j, rev), k);
            qi[j] = fetch2<D>(place<const S>(g.i, g.i_sb, g.i_sr, m, p0 + j, rev), k);
        }
        float a[2][kLen], b[2][kLen], A[2], H[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            A[e] = 1.f;
            H[e] = 0.f;
#pragma unroll
            for (int j = 0; j < kLen; ++j) {
                gate_fwd(qx[j].get(e), qr[j].get(e), qi[j].get(e), rate[e], a[e][j], b[e][j]);
                if (p0 + j >= m.len) {
                    a[e][j] = 1.f;
                    b[e][j] = 0.f;
                }
                H[e] = fmaf(a[e][j], H[e], b[e][j]);
                A[e] *= a[e][j];
            }
        }
        // two buffers, by turns: what the next tile writes, nobody still reads
        part[n & 1][m.sub][m.cl] = Two{A[0], H[0], A[1], H[1]};
        __syncthreads();
        float2 s = state[n & 1][m.cl];
        if (m.sub == 0 && g.states) {
            float* q = g.states + size_t(n) * g.B * g.C + at;
            if (m.n > 0) q[0] = s.x;
            if (m.n > 1) q[1] = s.y;
        }
        for (int k = 0; k < m.sub; ++k) {
            const Two t = part[n & 1][k][m.cl];
            s.x = fmaf(t.a0, s.x, t.h0);
            s.y = fmaf(t.a1, s.y, t.h1);
        }
#pragma unroll
        for (int j = 0; j < kLen; ++j) {
            s.x = fmaf(a[0][j], s.x, b[0][j]);
            s.y = fmaf(a[1][j], s.y, b[1][j]);
            const bool in = p0 + j < m.len;
            put2<D>(place<S>(g.h, g.h_sb, g.h_sr, m, p0 + j, rev), in ? s.x : 0.f, in ? s.y : 0.f,
                    p0 + j < g.T ? m.n : 0);
        }
        if (m.sub == kSub - 1) state[(n + 1) & 1][m.cl] = s;
    }
    if (m.sub == kSub - 1 && g.h_last) {
        const float2 s = state[g.tiles & 1][m.cl];  // this thread's own store
        if (m.n > 0) g.h_last[at] = s.x;
        if (m.n > 1) g.h_last[at + 1] = s.y;
    }
}

template <class D>
__global__ __launch_bounds__(kThreads) void k_tokens_bwd(Args g, bool rev) {
    using S = typename D::S;
    __shared__ Two part[2][kSub][kLanes];   // maps of h
    __shared__ float2 upart[2][kSub][kLanes];  // and of u (the factors are the same)
    __shared__ float2 ustate[2][kLanes];
    const Me m = me_of(g);
    const size_t at = size_t(m.b) * g.C + m.c;
    float rate[2], sum[2] = {0.f, 0.f};
    rates(g, m, rate);
    if (m.sub == 0) {
        float2 s{0.f, 0.f};
        if (g.dh_last && m.n > 0) s.x = g.dh_last[at];
        if (g.dh_last && m.n > 1) s.y = g.dh_last[at + 1];
        ustate[0][m.cl] = s;
    }
    for (int turn = 0; turn < g.tiles; ++turn) {
        const int n = g.tiles - 1 - turn, side = turn & 1;
        const int p0 = n * kTile + m.sub * kLen;
        Raw<D, 2> qx[kLen], qr[kLen], qi[kLen], qd[kLen];
#pragma unroll
        for (int j = 0; j < kLen; ++j) {
            const int k = p0 + j < m.len ? m.n : 0;
            qx[j] = fetch2<D>(place<const S>(g.x, g.x_sb, g.x_sr, m, p0 + j, rev), k);
            qr[j] = fetch2<D>(place<const S>(g.r, g.r_sb, g.r_sr, m, p0 + j, rev), k);
            qi[j] = fetch2<D>(place<const S>(g.i, g.i_sb, g.i_sr, m, p0 + j, rev), k);
            qd[j] = fetch2<D>(place<const S>(g.dh, g.dh_sb, g.dh_sr, m, p0 + j, rev), k);
        }
        float2 s{0.f, 0.f};
        {
            const float* q = g.states + size_t(n) * g.B * g.C + at;
            if (m.n > 0) s.x = q[0];
            if (m.n > 1) s.y = q[1];
        }
        float a[2][kLen], hp[2][kLen], A[2], H[2], U[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            A[e] = 1.f;
            H[e] = U[e] = 0.f;
#pragma unroll
            for (int j = 0; j < kLen; ++j) {
                gate_fwd(qx[j].get(e), qr[j].get(e), qi[j].get(e), rate[e], a[e][j], hp[e][j]);
                if (p0 + j >= m.len) {
                    a[e][j] = 1.f;
                    hp[e][j] = 0.f;
                }
                H[e] = fmaf(a[e][j], H[e], hp[e][j]);
                A[e] *= a[e][j];
            }
#pragma unroll
            for (int j = kLen - 1; j >= 0; --j) U[e] = a[e][j] * (qd[j].get(e) + U[e]);
        }
        part[side][m.sub][m.cl] = Two{A[0], H[0], A[1], H[1]};
        upart[side][m.sub][m.cl] = float2{U[0], U[1]};
        __syncthreads();
        for (int k = 0; k < m.sub; ++k) {
            const Two t = part[side][k][m.cl];
            s.x = fmaf(t.a0, s.x, t.h0);
            s.y = fmaf(t.a1, s.y, t.h1);
        }
        float2 u = ustate[side][m.cl];
        for (int k = kSub - 1; k > m.sub; --k) {
            const Two t = part[side][k][m.cl];
            const float2 v = upart[side][k][m.cl];
            u.x = fmaf(t.a0, u.x, v.x);
            u.y = fmaf(t.a1, u.y, v.y);
        }
#pragma unroll
        for (int j = 0; j < kLen; ++j) {
            float v = hp[0][j];
            hp[0][j] = s.x;
            s.x = fmaf(a[0][j], s.x, v);
            v = hp[1][j];
            hp[1][j] = s.y;
            s.y = fmaf(a[1][j], s.y, v);
        }
#pragma unroll
        for (int j = kLen - 1; j >= 0; --j) {
            float ox[2], orr[2], oi[2], e;
            const bool in = p0 + j < m.len;
            float gt = qd[j].get(0) + u.x;
            gate_bwd(qx[j].get(0), qr[j].get(0), qi[j].get(0), rate[0], a[0][j], hp[0][j], gt, ox[0],
                     orr[0], oi[0], e);
            sum[0] += in ? e : 0.f;
            u.x = a[0][j] * gt;
            gt = qd[j].get(1) + u.y;
            gate_bwd(qx[j].get(1), qr[j].get(1), qi[j].get(1), rate[1], a[1][j], hp[1][j], gt, ox[1],
                     orr[1], oi[1], e);
            sum[1] += in ? e : 0.f;
            u.y = a[1][j] * gt;
            const int k = p0 + j < g.T ? m.n : 0;
            put2<D>(place<S>(g.dx, g.dx_sb, g.dx_sr, m, p0 + j, rev), in ? ox[0] : 0.f, in ? ox[1] : 0.f, k);
            put2<D>(place<S>(g.dr, g.dr_sb, g.dr_sr, m, p0 + j, rev), in ? orr[0] : 0.f, in ? orr[1] : 0.f, k);
            put2<D>(place<S>(g.di, g.di_sb, g.di_sr, m, p0 + j, rev), in ? oi[0] : 0.f, in ? oi[1] : 0.f, k);
        }
        if (m.sub == 0) ustate[side ^ 1][m.cl] = u;
    }
    if (m.sub == 0 && g.dh0) {
        const float2 u = ustate[g.tiles & 1][m.cl];  // this thread's own store
        if (m.n > 0) g.dh0[at] = u.x;
        if (m.n > 1) g.dh0[at + 1] = u.y;
    }
    // the sub-tiles' sums in order
    __syncthreads();
    upart[0][m.sub][m.cl] = float2{sum[0], sum[1]};
    __syncthreads();
    if (m.sub == 0) {
        float2 t = upart[0][0][m.cl];
        for (int k = 1; k < kSub; ++k) {
            t.x += upart[0][k][m.cl].x;
            t.y += upart[0][k][m.cl].y;
        }
        if (m.n > 0) g.part[at] = t.x;
        if (m.n > 1) g.part[at + 1] = t.y;
    }
}

// 16 channels by 32 threads along the rows of partial sums; the threads' sums
// are added in order.
constexpr int kCloseChan = 16, kCloseRows = 32;
__global__ __launch_bounds__(kCloseChan* kCloseRows) void k_close_dlam(Args g, int parts) {
    __shared__ double acc[kCloseRows][kCloseChan];
    const int cl = threadIdx.x % kCloseChan, k = threadIdx.x / kCloseChan;
    const int c = blockIdx.x * kCloseChan + cl;
    double t = 0;
    if (c < g.C)
        for (int p = k; p < parts; p += kCloseRows) t += double(g.part[size_t(p) * g.C + c]);
    acc[k][cl] = t;
    __syncthreads();
    if (k == 0 && c < g.C) {
        for (int j = 1; j < kCloseRows; ++j) t += acc[j][cl];
        // d softplus = sig
        const double l = double(g.lam[c]);
        g.dlam[c] = float(t * -double(g.decay) / (1.0 + exp(-l)));
    }
}

template <class D>
__global__ __launch_bounds__(256) void k_step(int C, int S, const typename D::S* x, long long xs,
                                              const typename D::S* r, long long rs,
                                              const typename D::S* i, long long is,
                                              const float* lam, float decay, float* state,
                                              const int* slots, typename D::S* h, long long hs) {
    const unsigned wide = (C + 511) / 512;
    const long long b = blockIdx.x / wide;
    const int c = ((blockIdx.x % wide) * 256 + threadIdx.x) * 2;
    const int n = min(C - c, 2);
    if (n <= 0) return;
    const int slot = slots ? slots[b] : int(b);
    const bool on = slot >= 0 && slot < S;
    const Raw<D, 2> qx = fetch2<D>(x + b * xs + c, on ? n : 0);
    const Raw<D, 2> qr = fetch2<D>(r + b * rs + c, on ? n : 0);
    const Raw<D, 2> qi = fetch2<D>(i + b * is + c, on ? n : 0);
    float out[2] = {0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        if (!on || e >= n) continue;
        float a, v;
        gate_fwd(qx.get(e), qr.get(e), qi.get(e), decay * softplus(lam[c + e]) * kLog2e, a, v);
        float* s = state + (long long)slot * C + c + e;
        out[e] = fmaf(a, *s, v);
        *s = out[e];
    }
    put2<D>(h + b * hs + c, out[0], out[1], n);
}

template <class D>
void launch(bool bwd, bool rev, const Args& a, hipStream_t st) {
    const dim3 grid((a.C + kChan - 1) / kChan * unsigned(a.B));
    if (bwd) k_tokens_bwd<D><<<grid, kThreads, 0, st>>>(a, rev);
    else k_tokens_fwd<D><<<grid, kThreads, 0, st>>>(a, rev);
}
void launch_type(int dtype, bool bwd, bool rev, const Args& a, hipStream_t st) {
    if (dtype == GSCAN_F32) launch<F32>(bwd, rev, a, st);
    else if (dtype == GSCAN_F16) launch<F16>(bwd, rev, a, st);
    else launch<BF16>(bwd, rev, a, st);
}

}  // namespace

Plan tokens_plan(const gscan_shape& s) {
    Plan p;
    p.tiles = s.T > 0 ? (s.T - 1) / kTile + 1 : 1;
    p.parts = s.B;
    p.states = sizeof(float) * size_t(p.tiles) * s.B * s.C;
    p.scratch = sizeof(float) * size_t(p.parts) * s.C;
    return p;
}

hipError_t tokens_fwd(const gscan_shape& s, Args a, void*, hipStream_t st) {
    a.tiles = tokens_plan(s).tiles;
    launch_type(s.dtype, false, s.reverse != 0, a, st);
    return hipGetLastError();
}

hipError_t tokens_bwd(const gscan_shape& s, Args a, void* ws, hipStream_t st) {
    const Plan p = tokens_plan(s);
    a.tiles = p.tiles;
    a.part = static_cast<float*>(ws);
    launch_type(s.dtype, true, s.reverse != 0, a, st);
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? close_dlam(a, p.parts, st) : e;
}

hipError_t close_dlam(const Args& a, int parts, hipStream_t st) {
    k_close_dlam<<<dim3((a.C + kCloseChan - 1) / kCloseChan), kCloseChan * kCloseRows, 0, st>>>(
        a, parts);
    return hipGetLastError();
}

template <class D>
static void launch_step(int B, int C, int S, float decay, const gscan_view& x, const gscan_view& r,
                        const gscan_view& i, const float* lam, float* state, const int* slots,
                        const gscan_view& h, hipStream_t st) {
    using E = typename D::S;
    k_step<D><<<dim3((C + 511) / 512 * unsigned(B)), 256, 0, st>>>(
        C, S, static_cast<const E*>(x.p), x.sb, static_cast<const E*>(r.p), r.sb,
        static_cast<const E*>(i.p), i.sb, lam, decay, state, slots, static_cast<E*>(h.p), h.sb);
}

hipError_t step(int B, int C, int S, int dtype, float decay, const gscan_view& x,
                const gscan_view& r, const gscan_view& i, const float* lam, float* state,
                const int* slots, const gscan_view& h, hipStream_t st) {
    if (dtype == GSCAN_F32) launch_step<F32>(B, C, S, decay, x, r, i, lam, state, slots, h, st);
    else if (dtype == GSCAN_F16) launch_step<F16>(B, C, S, decay, x, r, i, lam, state, slots, h, st);
    else launch_step<BF16>(B, C, S, decay, x, r, i, lam, state, slots, h, st);
    return hipGetLastError();
}

}  // namespace gsc

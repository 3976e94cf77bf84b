// Gated linear recurrence over tokens ([B][T][C], channels contiguous), and
// its form for one position.
//
// A workgroup takes a tile of `sub` * `len` positions of 64 channels of one
// sequence.  A thread takes two neighbouring channels and `len` consecutive
// positions: it composes their maps h -> a h + b in registers, the sub
// compositions of a channel meet in LDS, and each thread runs its positions
// again from the state that it then knows.  The state passes from tile to tile
// between workgroups (gscan_carry.h).  Everything is read once and written
// once.
//
// What bounds it (8x4096x2048, against a large copy's 4.94 TB/s): in fp32 HBM
// (213 us forwards, 5.0 TB/s; 396 us backwards, 4.7 TB/s); in bf16, with half
// the bytes for the same arithmetic, the vector ALU is busy for 59% of the
// forward (130 to 145 us, 3.7 to 4.1 TB/s) and 52% of the backward (236 to 255
// us, 3.7 to 4.0 TB/s) and the rest is the tile's latency chain: counter, loads,
// LDS, the wait for the tiles before.  16 positions per thread amortise the
// address and LDS work (8: 145 and 304 us where 16 took 132 and 245); 8 threads
// along time backwards hold 32 elements in up to 256 registers, two workgroups
// to a unit, which beats more threads of fewer registers (512 threads of 16
// elements: 304 us).  Wider tiles (128 channels) and workgroups that stay and
// fetch their next unit early were slower (267 and 293 us backwards).  Channels
// past a multiple of 64 cost a whole tile: 8x65536 positions of 64, 65 and 128
// channels take 323, 501 and 490 us fwd + bwd.
#include <hip/hip_runtime.h>

#include "gscan_math.h"

namespace gsc {
namespace {

constexpr int kLanes = 32;             // threads across the channels of a tile
constexpr int kChan = 2 * kLanes;      // channels of a tile
constexpr int kFwdSub = 16;            // threads along time, forwards
constexpr int kBwdSub = 8;             // and backwards
constexpr int kLen = 16;               // positions of a thread where tiles are spread
constexpr int kStateTile = kBwdSub * kLen;  // positions from one kept state to the next

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
        const float v[2] = {v0, v1};
        store_vec<D, 2>(p, pack<D, false>(v));
    } else if (n == 1) {
        store_one<D>(p, v0);
    }
}

// What a thread works on.  `SPREAD`: the tiles of a sequence are spread over
// workgroups (gscan_carry.h), units in the order of the tiles.
struct Me {
    int b, c, n;   // sequence, first channel, channels that exist
    int cl, sub;   // place in the tile
    int len;       // valid positions of the sequence
    int valid;     // its tiles that hold any
    int m;         // place of the tile in the order of the scan
};
template <int TILE>
__device__ __forceinline__ Me me_of(const Args& g, unsigned unit) {
    Me me;
    const unsigned wide = (g.C + kChan - 1) / kChan;
    const unsigned side = unit / wide;
    me.m = side / unsigned(g.B);
    me.b = side - me.m * unsigned(g.B);
    me.cl = threadIdx.x % kLanes;
    me.sub = threadIdx.x / kLanes;
    me.c = (unit - side * wide) * kChan + 2 * me.cl;
    me.n = min(max(g.C - me.c, 0), 2);
    me.len = g.T;
    if (g.lengths) me.len = min(max(g.lengths[me.b], 0), g.T);
    me.valid = (me.len + TILE - 1) / TILE;
    return me;
}

// The thread's channels at its positions: `p` points at the first, `step`
// (the same for all threads) leads from one to the next.
template <class S>
struct Run {
    S* p;
    long long step;
    __device__ __forceinline__ S* at(int j) const { return p + j * step; }
};
template <class S>
__device__ __forceinline__ Run<S> run_of(const void* base, long long sb, long long sr, const Me& m,
                                         int p0, bool rev) {
    const int t = rev ? m.len - 1 - p0 : p0;
    return Run<S>{const_cast<S*>(static_cast<const S*>(base)) + m.b * sb + t * sr + m.c,
                  rev ? -sr : sr};
}

// A thread's positions.  FULL: all of the tile are valid, all its channels
// exist.  Otherwise every thread still loads two channels of every position,
// without a branch between the loads, from the nearest place that has them:
// positions past the end read the last one, channels past the end the last
// two.  What that gives in excess is not used.  (With a branch around each
// load, 24 x 1024 x 1022 fp16 took 75 us forwards and 158 backwards; 1024
// channels take 53 and 105.)
template <class D, int LEN, bool FULL>
__device__ __forceinline__ void fetch_run(Raw<D, 2> (&q)[LEN], const Run<const typename D::S>& r,
                                          const Me& m, int p0, int C) {
    if (FULL) {
#pragma unroll
        for (int j = 0; j < LEN; ++j) load_vec<D, 2>(q[j], r.at(j));
        return;
    }
    const int last = m.len - 1 - p0;  // of the thread's positions; may be negative
    if (C == 1) {
#pragma unroll
        for (int j = 0; j < LEN; ++j) {
            q[j] = fetch2<D>(r.at(min(j, last)), min(m.n, 1));
        }
        return;
    }
    const int back = min(C - 2 - m.c, 0);
#pragma unroll
    for (int j = 0; j < LEN; ++j) load_vec<D, 2>(q[j], r.at(min(j, last)) + back);
    if (back == -1) {  // only the first of the thread's channels exists: it came second
#pragma unroll
        for (int j = 0; j < LEN; ++j) q[j].w[0] = D::kBytes == 4 ? q[j].w[Raw<D, 2>::kWords - 1] : q[j].w[0] >> 16;
    }
}
template <int TILE>
__device__ __forceinline__ bool full_tile(const Args& g, const Me& m, int tile) {
    return m.c - 2 * m.cl + kChan <= g.C && (tile + 1) * TILE <= m.len;
}

struct Two {
    float a0, h0, a1, h1;
};

__device__ __forceinline__ void rates(const Args& g, const Me& m, float (&rate)[2]) {
    rate[0] = m.n > 0 ? rate_of(g.decay, g.lam[m.c]) : 0.f;
    rate[1] = m.n > 1 ? rate_of(g.decay, g.lam[m.c + 1]) : 0.f;
}

__device__ __forceinline__ float2 load_row(const float* p, const Me& m) {
    float2 s{0.f, 0.f};
    if (p && m.n > 0) s.x = p[0];
    if (p && m.n > 1) s.y = p[1];
    return s;
}
__device__ __forceinline__ void store_row(float* p, const Me& m, float2 s) {
    if (m.n > 0) p[0] = s.x;
    if (m.n > 1) p[1] = s.y;
}

// Zeros at the padding among the thread's positions from p0 on (at its own
// index in both directions).
template <class D, int LEN>
__device__ __forceinline__ void pad(const Args& g, void* out, long long sb, long long sr,
                                    const Me& m, int p0) {
    using S = typename D::S;
    const Run<S> q = run_of<S>(out, sb, sr, m, p0, false);
    for (int j = max(m.len - p0, 0); j < LEN; ++j)
        if (p0 + j < g.T) put2<D>(q.at(j), 0.f, 0.f, m.n);
}

// Word `w` of what a tile needs of the tiles before it, as the threads along
// time wait for one or two each: the map of the w-th tile of the group, or for
// the last w the state at the group's start.
__device__ __forceinline__ Two await(const Args& g, const Me& m, int w) {
    const int grp = m.m / kGroup, k = m.m % kGroup;
    Two t{1.f, 0.f, 1.f, 0.f};
    if (m.n == 0) return t;
    if (w < k) {
        const unsigned long long* p =
            g.carry.maps + (size_t(grp * kGroup + w) * g.B + m.b) * g.C + m.c;
        unsigned long long w0, w1;
        for (;;) {
            w0 = peek_map(p);
            w1 = m.n > 1 ? peek_map(p + 1) : 0;
            if (w0 != ~0ull && w1 != ~0ull) break;
            __builtin_amdgcn_s_sleep(1);
        }
        t = Two{map_a(w0), map_h(w0), map_a(w1), map_h(w1)};
    } else if (w == kGroup - 1 && grp > 0) {
        const unsigned* p = g.carry.starts + (size_t(grp) * g.B + m.b) * g.C + m.c;
        unsigned w0, w1;
        for (;;) {
            w0 = peek_start(p);
            w1 = m.n > 1 ? peek_start(p + 1) : 0;
            if (w0 != ~0u && w1 != ~0u) break;
            __builtin_amdgcn_s_sleep(1);
        }
        t.h0 = __uint_as_float(w0);
        t.h1 = __uint_as_float(w1);
    }
    return t;
}

// Shared by both directions: the state before the tile for the thread's
// channels, from `first`, that before the whole scan.  Call after the threads'
// maps were stored; their composition, `map_of`, is published by row `last`.
template <int SUB, bool SPREAD, class Map>
__device__ __forceinline__ float2 before_tile(const Args& g, const Me& m, const float* first,
                                              Two (*look)[kLanes], int last, Map map_of) {
    const size_t at = size_t(m.b) * g.C + m.c;
    __syncthreads();
    if (SPREAD && m.sub == last && m.m + 1 < m.valid && m.m % kGroup != kGroup - 1) {
        const Two t = map_of();
        unsigned long long* p = g.carry.maps + (size_t(m.m) * g.B + m.b) * g.C + m.c;
        if (m.n > 0) publish_map(p, t.a0, t.h0);
        if (m.n > 1) publish_map(p + 1, t.a1, t.h1);
    }
    float2 s = load_row(first && (!SPREAD || m.m < kGroup) ? first + at : nullptr, m);
    if constexpr (SPREAD) {
        if (m.m > 0) {
            for (int w = m.sub; w < kGroup; w += SUB) look[w][m.cl] = await(g, m, w);
            __syncthreads();
            if (m.m >= kGroup) s = float2{look[kGroup - 1][m.cl].h0, look[kGroup - 1][m.cl].h1};
            for (int k = 0; k < m.m % kGroup; ++k) {
                const Two t = look[k][m.cl];
                s.x = fmaf(t.a0, s.x, t.h0);
                s.y = fmaf(t.a1, s.y, t.h1);
            }
        }
    }
    return s;
}

// After the last position of the scan's order in this tile, at state s.
template <bool SPREAD>
__device__ __forceinline__ void after_tile(const Args& g, const Me& m, float* last, float2 s) {
    if (SPREAD && m.m + 1 < m.valid) {
        if (m.m % kGroup == kGroup - 1) {
            unsigned* p = g.carry.starts + (size_t(m.m / kGroup + 1) * g.B + m.b) * g.C + m.c;
            if (m.n > 0) publish_start(p, s.x);
            if (m.n > 1) publish_start(p + 1, s.y);
        }
    } else if (last) {
        store_row(last + size_t(m.b) * g.C + m.c, m, s);
    }
}

struct FwdShared {
    Two part[kFwdSub][kLanes], look[kGroup][kLanes];
    unsigned unit;
};

// FULL: all positions of the tile are valid and all its channels exist.
template <class D, int LEN, bool SPREAD, bool FULL>
__device__ __forceinline__ void tile_fwd(const Args& g, const Me& m, bool rev, FwdShared& sh) {
    using S = typename D::S;
    auto& part = sh.part;
    const size_t at = size_t(m.b) * g.C + m.c;
    const int p0 = m.m * kFwdSub * LEN + m.sub * LEN;
    Raw<D, 2> qx[LEN], qr[LEN], qi[LEN];
    fetch_run<D, LEN, FULL>(qx, run_of<const S>(g.x, g.x_sb, g.x_sr, m, p0, rev), m, p0, g.C);
    fetch_run<D, LEN, FULL>(qr, run_of<const S>(g.r, g.r_sb, g.r_sr, m, p0, rev), m, p0, g.C);
    fetch_run<D, LEN, FULL>(qi, run_of<const S>(g.i, g.i_sb, g.i_sr, m, p0, rev), m, p0, g.C);
    float rate[2];
    rates(g, m, rate);
    float a[2][LEN], b[2][LEN], A[2], H[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        A[e] = 1.f;
        H[e] = 0.f;
#pragma unroll
        for (int j = 0; j < LEN; ++j) {
            float sr, si;
            gate_fwd(qx[j].get(e), qr[j].get(e), qi[j].get(e), rate[e], a[e][j], b[e][j], sr, si);
            if (!FULL && p0 + j >= m.len) {
                a[e][j] = 1.f;
                b[e][j] = 0.f;
            }
            H[e] = fmaf(a[e][j], H[e], b[e][j]);
            A[e] *= a[e][j];
        }
    }
    part[m.sub][m.cl] = Two{A[0], H[0], A[1], H[1]};
    float2 s = before_tile<kFwdSub, SPREAD>(g, m, g.h0, sh.look, kFwdSub - 1, [&] {
        Two t = part[0][m.cl];
#pragma unroll 3
        for (int k = 1; k < kFwdSub; ++k) {
            const Two q = part[k][m.cl];
            t = Two{q.a0 * t.a0, fmaf(q.a0, t.h0, q.h0), q.a1 * t.a1, fmaf(q.a1, t.h1, q.h1)};
        }
        return t;
    });
    for (int k = 0; k < m.sub; ++k) {
        const Two t = part[k][m.cl];
        s.x = fmaf(t.a0, s.x, t.h0);
        s.y = fmaf(t.a1, s.y, t.h1);
    }
    if (g.states && p0 % kStateTile == 0 && p0 < m.len)
        store_row(g.states + size_t(p0 / kStateTile) * g.B * g.C + at, m, s);
    const Run<S> out = run_of<S>(g.h, g.h_sb, g.h_sr, m, p0, rev);
#pragma unroll
    for (int j = 0; j < LEN; ++j) {
        s.x = fmaf(a[0][j], s.x, b[0][j]);
        s.y = fmaf(a[1][j], s.y, b[1][j]);
        if (FULL || p0 + j < m.len) put2<D>(out.at(j), s.x, s.y, FULL ? 2 : m.n);
    }
    if (!FULL) pad<D, LEN>(g, g.h, g.h_sb, g.h_sr, m, p0);
    if (m.sub == kFwdSub - 1) after_tile<SPREAD>(g, m, g.h_last, s);
}

template <class D, int LEN, bool SPREAD>
__global__ __launch_bounds__(kLanes* kFwdSub, 4) void k_tokens_fwd(Args g, bool rev) {
    __shared__ FwdShared sh;
    const Me m = me_of<kFwdSub * LEN>(g, SPREAD ? take_share(g.carry, &sh.unit) : blockIdx.x);
    if (m.m >= m.valid) {  // padding only
        const size_t at = size_t(m.b) * g.C + m.c;
        if (m.m == 0 && m.sub == 0 && g.h_last)
            store_row(g.h_last + at, m, load_row(g.h0 ? g.h0 + at : nullptr, m));
        pad<D, LEN>(g, g.h, g.h_sb, g.h_sr, m, m.m * kFwdSub * LEN + m.sub * LEN);
    } else if (full_tile<kFwdSub * LEN>(g, m, m.m)) {
        tile_fwd<D, LEN, SPREAD, true>(g, m, rev, sh);
    } else {
        tile_fwd<D, LEN, SPREAD, false>(g, m, rev, sh);
    }
}

struct BwdShared {
    Two part[kBwdSub][kLanes];      // maps of h
    float2 upart[kBwdSub][kLanes];  // and of u (the factors are the same)
    Two look[kGroup][kLanes];
    unsigned unit;
};

template <class D, int LEN, bool SPREAD, bool FULL>
__device__ __forceinline__ void tile_bwd(const Args& g, const Me& m, bool rev, BwdShared& sh) {
    using S = typename D::S;
    auto& part = sh.part;
    auto& upart = sh.upart;
    const size_t at = size_t(m.b) * g.C + m.c;
    const int n = m.valid - 1 - m.m;  // the tile
    const int p0 = n * kBwdSub * LEN + m.sub * LEN;
    Raw<D, 2> qx[LEN], qr[LEN], qi[LEN], qd[LEN];
    fetch_run<D, LEN, FULL>(qx, run_of<const S>(g.x, g.x_sb, g.x_sr, m, p0, rev), m, p0, g.C);
    fetch_run<D, LEN, FULL>(qr, run_of<const S>(g.r, g.r_sb, g.r_sr, m, p0, rev), m, p0, g.C);
    fetch_run<D, LEN, FULL>(qi, run_of<const S>(g.i, g.i_sb, g.i_sr, m, p0, rev), m, p0, g.C);
    fetch_run<D, LEN, FULL>(qd, run_of<const S>(g.dh, g.dh_sb, g.dh_sr, m, p0, rev), m, p0, g.C);
    float2 s = load_row(g.states + size_t(n) * g.B * g.C + at, m);
    float rate[2], sum[2] = {0.f, 0.f};
    rates(g, m, rate);
    float a[2][LEN], hp[2][LEN], sr[2][LEN], si[2][LEN], A[2], H[2], U[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        A[e] = 1.f;
        H[e] = U[e] = 0.f;
#pragma unroll
        for (int j = 0; j < LEN; ++j) {
            gate_fwd(qx[j].get(e), qr[j].get(e), qi[j].get(e), rate[e], a[e][j], hp[e][j], sr[e][j],
                     si[e][j]);
            if (!FULL && p0 + j >= m.len) {
                a[e][j] = 1.f;
                hp[e][j] = 0.f;
            }
            H[e] = fmaf(a[e][j], H[e], hp[e][j]);
            A[e] *= a[e][j];
        }
#pragma unroll
        for (int j = LEN - 1; j >= 0; --j)
            U[e] = FULL || p0 + j < m.len ? a[e][j] * (qd[j].get(e) + U[e]) : 0.f;
    }
    part[m.sub][m.cl] = Two{A[0], H[0], A[1], H[1]};
    upart[m.sub][m.cl] = float2{U[0], U[1]};
    float2 u = before_tile<kBwdSub, SPREAD>(g, m, g.dh_last, sh.look, 0, [&] {
        Two t = part[kBwdSub - 1][m.cl];
        t.h0 = upart[kBwdSub - 1][m.cl].x;
        t.h1 = upart[kBwdSub - 1][m.cl].y;
#pragma unroll 3
        for (int k = kBwdSub - 2; k >= 0; --k) {
            const Two q = part[k][m.cl];
            const float2 v = upart[k][m.cl];
            t = Two{q.a0 * t.a0, fmaf(q.a0, t.h0, v.x), q.a1 * t.a1, fmaf(q.a1, t.h1, v.y)};
        }
        return t;
    });
    for (int k = 0; k < m.sub; ++k) {
        const Two t = part[k][m.cl];
        s.x = fmaf(t.a0, s.x, t.h0);
        s.y = fmaf(t.a1, s.y, t.h1);
    }
    for (int k = kBwdSub - 1; k > m.sub; --k) {
        const Two t = part[k][m.cl];
        const float2 v = upart[k][m.cl];
        u.x = fmaf(t.a0, u.x, v.x);
        u.y = fmaf(t.a1, u.y, v.y);
    }
#pragma unroll
    for (int j = 0; j < LEN; ++j) {
        float v = hp[0][j];
        hp[0][j] = s.x;
        s.x = fmaf(a[0][j], s.x, v);
        v = hp[1][j];
        hp[1][j] = s.y;
        s.y = fmaf(a[1][j], s.y, v);
    }
    const Run<S> px = run_of<S>(g.dx, g.dx_sb, g.dx_sr, m, p0, rev);
    const Run<S> pr = run_of<S>(g.dr, g.dr_sb, g.dr_sr, m, p0, rev);
    const Run<S> pi = run_of<S>(g.di, g.di_sb, g.di_sr, m, p0, rev);
#pragma unroll
    for (int j = LEN - 1; j >= 0; --j) {
        float ox[2], orr[2], oi[2], e;
        const bool in = FULL || p0 + j < m.len;
        float gt = (in ? qd[j].get(0) : 0.f) + u.x;
        gate_bwd(qx[j].get(0), sr[0][j], si[0][j], rate[0], a[0][j], hp[0][j], gt, ox[0], orr[0],
                 oi[0], e);
        sum[0] += in ? e : 0.f;
        u.x = a[0][j] * gt;
        gt = (in ? qd[j].get(1) : 0.f) + u.y;
        gate_bwd(qx[j].get(1), sr[1][j], si[1][j], rate[1], a[1][j], hp[1][j], gt, ox[1], orr[1],
                 oi[1], e);
        sum[1] += in ? e : 0.f;
        u.y = a[1][j] * gt;
        const int k = FULL ? 2 : in ? m.n : 0;
        put2<D>(px.at(j), ox[0], ox[1], k);
        put2<D>(pr.at(j), orr[0], orr[1], k);
        put2<D>(pi.at(j), oi[0], oi[1], k);
    }
    if (!FULL) {
        pad<D, LEN>(g, g.dx, g.dx_sb, g.dx_sr, m, p0);
        pad<D, LEN>(g, g.dr, g.dr_sb, g.dr_sr, m, p0);
        pad<D, LEN>(g, g.di, g.di_sb, g.di_sr, m, p0);
    }
    if (m.sub == 0) after_tile<SPREAD>(g, m, g.dh0, u);
    // the threads' sums in order
    __syncthreads();
    upart[m.sub][m.cl] = float2{sum[0], sum[1]};
    __syncthreads();
    if (m.sub == 0) {
        float2 t = upart[0][m.cl];
        for (int k = 1; k < kBwdSub; ++k) {
            t.x += upart[k][m.cl].x;
            t.y += upart[k][m.cl].y;
        }
        store_row(g.part + size_t(m.m) * g.B * g.C + at, m, t);
    }
}

template <class D, int LEN, bool SPREAD>
__global__ __launch_bounds__(kLanes* kBwdSub, 2) void k_tokens_bwd(Args g, bool rev) {
    __shared__ BwdShared sh;
    const Me m = me_of<kBwdSub * LEN>(g, SPREAD ? take_share(g.carry, &sh.unit) : blockIdx.x);
    if (m.m >= m.valid) {
        const size_t at = size_t(m.b) * g.C + m.c;
        if (m.sub == 0) {
            if (m.m == 0 && g.dh0)
                store_row(g.dh0 + at, m, load_row(g.dh_last ? g.dh_last + at : nullptr, m));
            store_row(g.part + size_t(m.m) * g.B * g.C + at, m, float2{0.f, 0.f});
        }
        const int p0 = m.m * kBwdSub * LEN + m.sub * LEN;
        pad<D, LEN>(g, g.dx, g.dx_sb, g.dx_sr, m, p0);
        pad<D, LEN>(g, g.dr, g.dr_sb, g.dr_sr, m, p0);
        pad<D, LEN>(g, g.di, g.di_sb, g.di_sr, m, p0);
    } else if (full_tile<kBwdSub * LEN>(g, m, m.valid - 1 - m.m)) {
        tile_bwd<D, LEN, SPREAD, true>(g, m, rev, sh);
    } else {
        tile_bwd<D, LEN, SPREAD, false>(g, m, rev, sh);
    }
}

// 16 channels by 32 threads along the rows of partial sums; the threads' sums
// are added in order.
constexpr int kCloseChan = 16, kCloseRows = 32;
__global__ __launch_bounds__(kCloseChan* kCloseRows) void k_close_dlam(Args g, long long parts) {
    __shared__ double acc[kCloseRows][kCloseChan];
    const int cl = threadIdx.x % kCloseChan, k = threadIdx.x / kCloseChan;
    const int c = blockIdx.x * kCloseChan + cl;
    double t = 0;
    if (c < g.C)
        for (long long p = k; p < parts; p += kCloseRows) t += double(g.part[size_t(p) * g.C + c]);
    acc[k][cl] = t;
    __syncthreads();
    if (k == 0 && c < g.C) {
        for (int j = 1; j < kCloseRows; ++j) t += acc[j][cl];
        // d softplus = sig
        const double l = double(g.lam[c]);
        g.dlam[c] = float(t * -double(g.decay) / (1.0 + exp(-l)));
    }
}

// One position: a thread takes two channels of R sequences, whose loads are
// under way together and which share the channels' rates.  512 x 4096 bf16: 9
// us, 3.7 TB/s, as long as the call's host side; a single sequence of 384
// channels 2.2 us, a launch's latency.
template <class D, int R>
__global__ __launch_bounds__(256) void k_step(int B, int C, int S, const typename D::S* x,
                                              long long xs, const typename D::S* r, long long rs,
                                              const typename D::S* i, long long is,
                                              const float* lam, float decay, float* state,
                                              const int* slots, typename D::S* h, long long hs) {
    const unsigned wide = (C + 511) / 512;
    const int b0 = int(blockIdx.x / wide) * R;
    const int c = ((blockIdx.x % wide) * 256 + threadIdx.x) * 2;
    const int n = min(C - c, 2);
    if (n <= 0) return;
    int slot[R];
    Raw<D, 2> qx[R], qr[R], qi[R];
    Raw<F32, 2> qs[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
        const int b = b0 + k;
        slot[k] = b < B ? (slots ? slots[b] : b) : -1;
        const int m = slot[k] >= 0 && slot[k] < S ? n : 0;
        qx[k] = fetch2<D>(x + b * xs + c, m);
        qr[k] = fetch2<D>(r + b * rs + c, m);
        qi[k] = fetch2<D>(i + b * is + c, m);
        qs[k] = fetch2<F32>(state + (long long)slot[k] * C + c, m);
    }
    const float rate[2] = {rate_of(decay, lam[c]), n > 1 ? rate_of(decay, lam[c + 1]) : 0.f};
#pragma unroll
    for (int k = 0; k < R; ++k) {
        float out[2] = {0.f, 0.f};
        if (slot[k] >= 0 && slot[k] < S) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float a, v, sr, si;
                gate_fwd(qx[k].get(e), qr[k].get(e), qi[k].get(e), rate[e], a, v, sr, si);
                out[e] = fmaf(a, qs[k].get(e), v);
            }
            put2<F32>(state + (long long)slot[k] * C + c, out[0], out[1], n);
        }
        if (b0 + k < B) put2<D>(h + (b0 + k) * hs + c, out[0], out[1], n);
    }
}

// Sequences of one tile take a tile as long as they need; else tiles of kLen
// positions per thread are spread.  (64 x 512 x 2048 bf16 forward: 119 us with
// 16 positions per thread, 133 with 8, 220 with 4; backward 218, 279, 301.)
int len_of(int T, bool bwd) {
    const int sub = bwd ? kBwdSub : kFwdSub;
    return T <= sub ? 1 : T <= 4 * sub ? 4 : T <= 8 * sub ? 8 : kLen;
}
int tiles_of(int T, int tile) { return T > 0 ? (T - 1) / tile + 1 : 1; }

unsigned units_of(const Args& a) {
    return (a.C + kChan - 1) / kChan * unsigned(a.B) * unsigned(a.tiles);
}

template <class D, int LEN, bool SPREAD>
void launch(bool bwd, bool rev, const Args& a, hipStream_t st) {
    const dim3 grid(units_of(a));
    if (bwd) k_tokens_bwd<D, LEN, SPREAD><<<grid, kLanes * kBwdSub, 0, st>>>(a, rev);
    else k_tokens_fwd<D, LEN, SPREAD><<<grid, kLanes * kFwdSub, 0, st>>>(a, rev);
}
template <class D>
void launch_len(bool bwd, bool rev, const Args& a, hipStream_t st) {
    const int len = len_of(a.T, bwd);
    if (a.tiles > 1) launch<D, kLen, true>(bwd, rev, a, st);
    else if (len == 1) launch<D, 1, false>(bwd, rev, a, st);
    else if (len == 4) launch<D, 4, false>(bwd, rev, a, st);
    else if (len == 8) launch<D, 8, false>(bwd, rev, a, st);
    else launch<D, kLen, false>(bwd, rev, a, st);
}
void launch_type(int dtype, bool bwd, bool rev, const Args& a, hipStream_t st) {
    if (dtype == GSCAN_F32) launch_len<F32>(bwd, rev, a, st);
    else if (dtype == GSCAN_F16) launch_len<F16>(bwd, rev, a, st);
    else launch_len<BF16>(bwd, rev, a, st);
}

__global__ __launch_bounds__(256) void k_clear(uint4* p, size_t n) {
    const size_t k = size_t(blockIdx.x) * 256 + threadIdx.x;
    const unsigned v = k < 4 ? 0u : ~0u;  // the counter's 64 bytes
    if (k < n) p[k] = uint4{v, v, v, v};
}

size_t tokens_carry(const gscan_shape& s, int tiles) {
    return tiles > 1 ? carry_bytes(size_t(s.B) * s.C, tiles) : 0;
}

}  // namespace

hipError_t clear_carry(void* ws, size_t bytes, hipStream_t st) {
    const size_t n = bytes / sizeof(uint4);
    k_clear<<<dim3((n + 255) / 256), 256, 0, st>>>(static_cast<uint4*>(ws), n);
    return hipGetLastError();
}

Plan tokens_plan(const gscan_shape& s) {
    Plan p;
    p.tiles = tiles_of(s.T, kStateTile);  // of the backward pass, the shorter ones
    p.parts = (long long)p.tiles * s.B;
    p.states = sizeof(float) * size_t(p.tiles) * s.B * s.C;
    p.scratch = tokens_carry(s, p.tiles) + sizeof(float) * size_t(p.parts) * s.C;
    // forwards a tile has twice the positions and twice the threads; rounded up
    // to whole tiles, it needs as many threads or more
    static_assert(kFwdSub == 2 * kBwdSub, "the forward's launch is the larger");
    const long long units = (long long)((s.C + kChan - 1) / kChan) * s.B;
    p.fits = units * tiles_of(s.T, kFwdSub * kLen) < kMaxThreads / (kLanes * kFwdSub);
    return p;
}

namespace {

// The words between tiles come first in the workspace, then the partial sums.
hipError_t tokens_run(const gscan_shape& s, bool bwd, Args& a, void* ws, hipStream_t st) {
    a.tiles = tiles_of(s.T, kLen * (bwd ? kBwdSub : kFwdSub));
    const size_t words = tokens_carry(s, a.tiles);
    a.part = reinterpret_cast<float*>(static_cast<char*>(ws) + words);
    if (words) {
        a.carry = carry_at(ws, size_t(s.B) * s.C, a.tiles, units_of(a), 1);
        const hipError_t e = clear_carry(ws, words, st);
        if (e != hipSuccess) return e;
    }
    launch_type(s.dtype, bwd, s.reverse != 0, a, st);
    return hipGetLastError();
}

}  // namespace

hipError_t tokens_fwd(const gscan_shape& s, Args a, void* ws, hipStream_t st) {
    return tokens_run(s, false, a, ws, st);
}

hipError_t tokens_bwd(const gscan_shape& s, Args a, void* ws, hipStream_t st) {
    const hipError_t e = tokens_run(s, true, a, ws, st);
    return e == hipSuccess ? close_dlam(a, tokens_plan(s).parts, st) : e;
}

hipError_t close_dlam(const Args& a, long long parts, hipStream_t st) {
    k_close_dlam<<<dim3((a.C + kCloseChan - 1) / kCloseChan), kCloseChan * kCloseRows, 0, st>>>(
        a, parts);
    return hipGetLastError();
}

// Sequences of a thread: one while the threads are too few to fill the device
// (latency), else four (one and four, on inputs that change from call to call:
// 256 x 2048 bf16 4.3 and 5.0 us, 512 x 4096 9.4 and 8.9, 2048 x 4096 28.0 and
// 26.8).
template <class D>
static void launch_step(int B, int C, int S, float decay, const gscan_view& x, const gscan_view& r,
                        const gscan_view& i, const float* lam, float* state, const int* slots,
                        const gscan_view& h, hipStream_t st) {
    using E = typename D::S;
    const bool many = (long long)B * C >= 1 << 21;
    const unsigned rows = many ? (B + 3) / 4 : B;
    auto* kernel = many ? k_step<D, 4> : k_step<D, 1>;
    kernel<<<dim3((C + 511) / 512 * rows), 256, 0, st>>>(
        B, C, S, static_cast<const E*>(x.p), x.sb, static_cast<const E*>(r.p), r.sb,
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

// Gated linear recurrence over planes ([B][C][T], time contiguous).
//
// A row (b, c) is scanned by LW neighbouring lanes of a wavefront.  A tile is
// LW * V positions: each lane takes V consecutive ones, composes their maps
// h -> a h + b in registers, the lanes' compositions are scanned with DPP
// moves (no LDS), and each lane runs its V steps again from the state that it
// then knows.  Everything is read once and written once.
//
// Where there are rows enough to fill the device, lanes walk the tiles of
// their row and the state passes in a register.  Where there are few and they
// are long, a tile is kWide positions of a workgroup, its wavefronts' maps
// meet in LDS, and the state passes between workgroups (gscan_carry.h).
//
// Backwards the same tile gives h (from the state the forward kept for it)
// and, for the sequence u_t = a_t g_t that passes from position to position,
// the maps u -> a (dh + u), scanned in the other direction.
//
// What bounds it, at the rate a large copy reaches on the same card (4.94
// TB/s): HBM for whole wavefronts per row -- 128x96x56x56 fp16 79 us forwards
// (3.9 TB/s), 107 to 118 us backwards (4.6 to 5.0 TB/s); 8x64x512x512 fp32,
// spread, 451 us (4.8 TB/s) and 756 us (5.0 TB/s).  Rows that fill part of a
// wavefront cost the rest of it: 64x384x14x14 fp32 (49 of 64 lanes) 21 us (3.7
// TB/s) and 33 us (4.1 TB/s).  8 positions per lane make two 16-byte accesses per tensor in
// fp32 and one in 16 bits, and amortise the 12 DPP moves of a scan; prefetching
// the next tile shortened a lone row by a tenth but cost the occupancy that
// many rows need (fp16 above: the backward call 119 -> 144 us), so it is not done.
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
// REV: position p lies at len - 1 - p.  FULL: all V are valid.  Where a row
// ends within a lane's positions, the wavefront loads elements one by one, but
// without a branch between the loads: those past the end read the last one,
// which is not used.
template <class D, int V, bool REV, bool FULL>
__device__ __forceinline__ void fetch(Raw<D, V>& out, const typename D::S* row, int p0, int len) {
    if (FULL) {
        load_vec<D, V>(out, row + (REV ? len - V - p0 : p0));
        return;
    }
#pragma unroll
    for (int k = 0; k < Raw<D, V>::kWords; ++k) out.w[k] = 0;
    if (!__any(p0 < len && len < p0 + V)) {
        if (p0 + V <= len) load_vec<D, V>(out, row + (REV ? len - V - p0 : p0));
    } else if (len > 0) {
        float v[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int p = min(p0 + j, len - 1);
            v[REV ? V - 1 - j : j] = load_one<D>(row + (REV ? len - 1 - p : p));
        }
        out = pack<D, false>(v);  // exact: the values are of the type
    }
}
// The same positions written; those in len .. T - 1 (which lie at their own
// index in both directions) become zero.
template <class D, int V, bool REV, bool FULL>
__device__ __forceinline__ void put(typename D::S* row, const float (&v)[V], int p0, int len,
                                    int T) {
    if (FULL || p0 + V <= len) {
        store_vec<D, V>(row + (REV ? len - V - p0 : p0), pack<D, REV>(v));
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
};
__device__ __forceinline__ Row row_at(const Args& g, long long id) {
    Row w;
    w.id = id;
    w.b = int(unsigned(id) / unsigned(g.C));  // fewer than 2^25 rows
    w.c = int(id) - w.b * g.C;
    w.len = g.T;
    if (g.lengths) w.len = min(max(g.lengths[w.b], 0), g.T);
    return w;
}

// A lane's part of a tile forwards: its elements' maps and their composition
// (A, H), then its outputs from the state s before its first position.
template <class D, int V, bool REV, bool FULL>
struct Fwd {
    using S = typename D::S;
    float a[V], b[V], A, H;
    __device__ __forceinline__ void open(const Args& g, const Row& w, int p0, float rate) {
        Raw<D, V> qx, qr, qi;
        fetch<D, V, REV, FULL>(qx, row_of<const S>(g.x, g.x_sb, g.x_sr, w.b, w.c), p0, w.len);
        fetch<D, V, REV, FULL>(qr, row_of<const S>(g.r, g.r_sb, g.r_sr, w.b, w.c), p0, w.len);
        fetch<D, V, REV, FULL>(qi, row_of<const S>(g.i, g.i_sb, g.i_sr, w.b, w.c), p0, w.len);
        A = 1.f;
        H = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float sr, si;
            gate_fwd(at<D, V, REV>(qx, j), at<D, V, REV>(qr, j), at<D, V, REV>(qi, j), rate, a[j],
                     b[j], sr, si);
            if (!FULL && p0 + j >= w.len) {
                a[j] = 1.f;
                b[j] = 0.f;
            }
            H = fmaf(a[j], H, b[j]);
            A *= a[j];
        }
    }
    __device__ __forceinline__ void close(const Args& g, const Row& w, int p0, float s) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            s = fmaf(a[j], s, b[j]);
            b[j] = s;
        }
        put<D, V, REV, FULL>(row_of<S>(g.h, g.h_sb, g.h_sr, w.b, w.c), b, p0, w.len, g.T);
    }
};

// Backwards: the maps of h (A, H) and of u (A, U) of its elements, then its
// outputs from the state s before its first position and u after its last.
template <class D, int V, bool REV, bool FULL>
struct Bwd {
    using S = typename D::S;
    Raw<D, V> qx, qd;
    float sr[V], si[V], a[V], b[V], A, H, U;
    __device__ __forceinline__ void open(const Args& g, const Row& w, int p0, float rate) {
        Raw<D, V> qr, qi;
        fetch<D, V, REV, FULL>(qx, row_of<const S>(g.x, g.x_sb, g.x_sr, w.b, w.c), p0, w.len);
        fetch<D, V, REV, FULL>(qr, row_of<const S>(g.r, g.r_sb, g.r_sr, w.b, w.c), p0, w.len);
        fetch<D, V, REV, FULL>(qi, row_of<const S>(g.i, g.i_sb, g.i_sr, w.b, w.c), p0, w.len);
        fetch<D, V, REV, FULL>(qd, row_of<const S>(g.dh, g.dh_sb, g.dh_sr, w.b, w.c), p0, w.len);
        A = 1.f;
        H = U = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            gate_fwd(at<D, V, REV>(qx, j), at<D, V, REV>(qr, j), at<D, V, REV>(qi, j), rate, a[j],
                     b[j], sr[j], si[j]);
            if (!FULL && p0 + j >= w.len) {
                a[j] = 1.f;
                b[j] = 0.f;
            }
            H = fmaf(a[j], H, b[j]);
            A *= a[j];
        }
#pragma unroll
        for (int j = V - 1; j >= 0; --j)
            U = FULL || p0 + j < w.len ? a[j] * (at<D, V, REV>(qd, j) + U) : 0.f;
    }
    // returns the lane's part of the sum for dlam
    __device__ __forceinline__ float close(const Args& g, const Row& w, int p0, float rate, float s,
                                           float u) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float v = b[j];
            b[j] = s;
            s = fmaf(a[j], s, v);
        }
        float ox[V], orr[V], oi[V], sum = 0.f;
#pragma unroll
        for (int j = V - 1; j >= 0; --j) {
            const bool in = FULL || p0 + j < w.len;
            const float gt = (in ? at<D, V, REV>(qd, j) : 0.f) + u;
            float e;
            gate_bwd(at<D, V, REV>(qx, j), sr[j], si[j], rate, a[j], b[j], gt, ox[j], orr[j], oi[j], e);
            sum += in ? e : 0.f;
            u = a[j] * gt;
        }
        put<D, V, REV, FULL>(row_of<S>(g.dx, g.dx_sb, g.dx_sr, w.b, w.c), ox, p0, w.len, g.T);
        put<D, V, REV, FULL>(row_of<S>(g.dr, g.dr_sb, g.dr_sr, w.b, w.c), orr, p0, w.len, g.T);
        put<D, V, REV, FULL>(row_of<S>(g.di, g.di_sb, g.di_sr, w.b, w.c), oi, p0, w.len, g.T);
        return sum;
    }
};

// ---------------------------------------------------------------------------
// a group of lanes walks its row
// ---------------------------------------------------------------------------

template <int LW>
__device__ __forceinline__ bool my_row(const Args& g, Row& w) {
    const long long id = (long long)blockIdx.x * (kThreads / LW) + threadIdx.x / LW;
    if (id >= (long long)g.B * g.C) return false;  // whole groups of lanes
    w = row_at(g, id);
    return true;
}

template <class D, int V, int LW, bool REV, bool FULL>
__device__ __forceinline__ void step_fwd(const Args& g, const Row& w, int p0, float rate,
                                         float& carry) {
    Fwd<D, V, REV, FULL> t;
    t.open(g, w, p0, rate);
    lane_scan<LW>(t.A, t.H);
    const float s = fmaf(lane_before<LW>(t.A, 1.f), carry, lane_before<LW>(t.H, 0.f));
    carry = fmaf(lane_last<LW>(t.A), carry, lane_last<LW>(t.H));
    t.close(g, w, p0, s);
}

template <class D, int V, int LW, bool REV>
__global__ __launch_bounds__(kThreads) void k_planes_fwd(Args g) {
    Row w;
    if (!my_row<LW>(g, w)) return;
    const long long rows = (long long)g.B * g.C;
    const int lane = threadIdx.x % LW;
    const float rate = rate_of(g.decay, g.lam[w.c]);
    float carry = g.h0 ? g.h0[w.id] : 0.f;
    for (int n = 0; n < g.tiles; ++n) {
        const int p0 = (n * LW + lane) * V;
        if (g.states && lane == 0) g.states[n * rows + w.id] = carry;
        if (LW == 64 && (n + 1) * LW * V <= w.len) step_fwd<D, V, LW, REV, true>(g, w, p0, rate, carry);
        else step_fwd<D, V, LW, REV, false>(g, w, p0, rate, carry);
    }
    if (g.h_last && lane == 0) g.h_last[w.id] = carry;
}

template <class D, int V, int LW, bool REV, bool FULL>
__device__ __forceinline__ float step_bwd(const Args& g, const Row& w, int p0, float rate,
                                          float state, float& after) {
    Bwd<D, V, REV, FULL> t;
    t.open(g, w, p0, rate);
    float B = lane_mirror<LW>(t.A), U = lane_mirror<LW>(t.U);
    lane_scan<LW>(t.A, t.H);
    const float s = fmaf(lane_before<LW>(t.A, 1.f), state, lane_before<LW>(t.H, 0.f));
    lane_scan<LW>(B, U);
    const float u = fmaf(lane_mirror<LW>(lane_before<LW>(B, 1.f)), after,
                         lane_mirror<LW>(lane_before<LW>(U, 0.f)));
    after = fmaf(lane_last<LW>(B), after, lane_last<LW>(U));
    return t.close(g, w, p0, rate, s, u);
}

template <class D, int V, int LW, bool REV>
__global__ __launch_bounds__(kThreads) void k_planes_bwd(Args g) {
    Row w;
    if (!my_row<LW>(g, w)) return;
    const long long rows = (long long)g.B * g.C;
    const int lane = threadIdx.x % LW;
    const float rate = rate_of(g.decay, g.lam[w.c]);
    float after = g.dh_last ? g.dh_last[w.id] : 0.f;  // u of the position after the tile
    float sum = 0.f;
    for (int n = g.tiles - 1; n >= 0; --n) {
        const int p0 = (n * LW + lane) * V;
        const float state = g.states[n * rows + w.id];
        if (LW == 64 && (n + 1) * LW * V <= w.len)
            sum += step_bwd<D, V, LW, REV, true>(g, w, p0, rate, state, after);
        else sum += step_bwd<D, V, LW, REV, false>(g, w, p0, rate, state, after);
    }
    sum = lane_sum<LW>(sum);
    if (lane == 0) {
        g.part[w.id] = sum;
        if (g.dh0) g.dh0[w.id] = after;
    }
}

// ---------------------------------------------------------------------------
// the tiles of a row spread over workgroups
// ---------------------------------------------------------------------------

constexpr int kSpread = 512;  // threads of a tile
constexpr int kWaves = kSpread / 64;
constexpr int kWideV = 8;
constexpr int kWide = kSpread * kWideV;  // positions of a tile
// Units of a share at the most: 8x64x512x512 fp32 forward 799 us with tiles of
// 2048 positions taken one by one (the counter's pace), 467 with shares of 8
// of them, 443 with shares of 8 tiles of 4096.
constexpr unsigned kShare = 8;

struct Spread {
    float A[kWaves], H[kWaves], U[kWaves];  // maps of the wavefronts
    float carry;
    unsigned unit;
};

// What a workgroup works on: tile m of its row in the order of the scan.
struct Unit {
    Row w;
    int m, valid;
};
__device__ __forceinline__ Unit unit_at(const Args& g, unsigned unit) {
    const unsigned rows = unsigned(g.B) * unsigned(g.C);
    Unit u;
    u.m = unit / rows;
    u.w = row_at(g, unit - unsigned(u.m) * rows);
    u.valid = (u.w.len + kWide - 1) / kWide;
    return u;
}

// The state before the unit's tile, from `first`, that before the whole scan:
// a lane waits for each map since the group's start and they are composed
// across lanes, always in the same order.  By one wavefront.
__device__ __forceinline__ float await(const Args& g, const Unit& u, const float* first) {
    const int lane = threadIdx.x & 63, grp = u.m / kGroup, k = u.m % kGroup;
    float a = 1.f, h = 0.f;
    if (lane < k) {
        const unsigned long long* p = g.carry.maps + u.w.id * g.tiles + (grp * kGroup + lane);
        unsigned long long v;
        while ((v = peek_map(p)) == ~0ull) __builtin_amdgcn_s_sleep(1);
        a = map_a(v);
        h = map_h(v);
    }
    float s;
    if (grp > 0) {
        const unsigned* p = g.carry.starts + u.w.id * ((g.tiles + kGroup - 1) / kGroup) + grp;
        unsigned v;
        while ((v = peek_start(p)) == ~0u) __builtin_amdgcn_s_sleep(1);
        s = __uint_as_float(v);
    } else {
        s = first ? first[u.w.id] : 0.f;
    }
    static_assert(kGroup == 16, "a group's maps lie in one row of lanes");
    lane_scan<16>(a, h);
    a = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, a), 15));
    h = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, h), 15));
    return fmaf(a, s, h);
}
__device__ __forceinline__ void give_map(const Args& g, const Unit& u, float a, float h) {
    if (u.m + 1 < u.valid && u.m % kGroup != kGroup - 1)
        publish_map(g.carry.maps + u.w.id * g.tiles + u.m, a, h);
}
// After the tile: the next group's start, or the end of the scan.
__device__ __forceinline__ void give_state(const Args& g, const Unit& u, float* last, float s) {
    if (u.m + 1 < u.valid) {
        if (u.m % kGroup == kGroup - 1)
            publish_start(g.carry.starts + u.w.id * ((g.tiles + kGroup - 1) / kGroup) +
                              u.m / kGroup + 1, s);
    } else if (last) {
        last[u.w.id] = s;
    }
}

// Zeros over the unit's tile, which is padding.
template <class D>
__device__ __forceinline__ void pad(const Args& g, const Unit& u, void* out, long long sb, long long sr) {
    using S = typename D::S;
    S* row = row_of<S>(out, sb, sr, u.w.b, u.w.c);
    for (int p = u.m * kWide + threadIdx.x; p < min(g.T, (u.m + 1) * kWide); p += kSpread)
        store_one<D>(row + p, 0.f);
}

template <class D, bool REV, bool FULL>
__device__ __forceinline__ void spread_fwd(const Args& g, const Unit& u, Spread& sh) {
    const int wave = threadIdx.x / 64, p0 = (u.m * kSpread + threadIdx.x) * kWideV;
    Fwd<D, kWideV, REV, FULL> t;
    t.open(g, u.w, p0, rate_of(g.decay, g.lam[u.w.c]));
    lane_scan<64>(t.A, t.H);
    if ((threadIdx.x & 63) == 63) {
        sh.A[wave] = t.A;
        sh.H[wave] = t.H;
    }
    __syncthreads();
    if (threadIdx.x == kSpread - 1) {
        float a = sh.A[0], h = sh.H[0];
        for (int k = 1; k < kWaves; ++k) {
            h = fmaf(sh.A[k], h, sh.H[k]);
            a *= sh.A[k];
        }
        give_map(g, u, a, h);
    }
    if (wave == 0) {
        const float s = await(g, u, g.h0);
        if (threadIdx.x == 0) {
            sh.carry = s;
            if (g.states) g.states[(long long)u.m * g.B * g.C + u.w.id] = s;
        }
    }
    __syncthreads();
    float s = sh.carry;
    for (int k = 0; k < wave; ++k) s = fmaf(sh.A[k], s, sh.H[k]);
    if (threadIdx.x == kSpread - 1) give_state(g, u, g.h_last, fmaf(t.A, s, t.H));
    s = fmaf(lane_before<64>(t.A, 1.f), s, lane_before<64>(t.H, 0.f));
    t.close(g, u.w, p0, s);
}

template <class D, bool REV>
__global__ __launch_bounds__(kSpread) void k_spread_fwd(Args g) {
    __shared__ Spread sh;
    const unsigned from = take_share(g.carry, &sh.unit);
    for (unsigned k = from; k < min(from + g.carry.share, g.carry.units); ++k) {
        const Unit u = unit_at(g, k);
        if (u.m >= u.valid) {
            if (u.m == 0 && threadIdx.x == 0 && g.h_last) g.h_last[u.w.id] = g.h0 ? g.h0[u.w.id] : 0.f;
            pad<D>(g, u, g.h, g.h_sb, g.h_sr);
        } else if ((u.m + 1) * kWide <= u.w.len) {
            spread_fwd<D, REV, true>(g, u, sh);
        } else {
            spread_fwd<D, REV, false>(g, u, sh);
        }
        __syncthreads();
    }
}

template <class D, bool REV, bool FULL>
__device__ __forceinline__ void spread_bwd(const Args& g, const Unit& u, Spread& sh) {
    const int wave = threadIdx.x / 64, n = u.valid - 1 - u.m;
    const int p0 = (n * kSpread + threadIdx.x) * kWideV;
    const long long rows = (long long)g.B * g.C;
    const float rate = rate_of(g.decay, g.lam[u.w.c]);
    float s = g.states[n * rows + u.w.id];
    Bwd<D, kWideV, REV, FULL> t;
    t.open(g, u.w, p0, rate);
    float B = lane_mirror<64>(t.A), U = lane_mirror<64>(t.U);
    lane_scan<64>(t.A, t.H);
    lane_scan<64>(B, U);
    if ((threadIdx.x & 63) == 63) {
        sh.A[wave] = t.A;
        sh.H[wave] = t.H;
        sh.U[wave] = U;
    }
    __syncthreads();
    if (threadIdx.x == kSpread - 1) {
        float a = sh.A[kWaves - 1], h = sh.U[kWaves - 1];
        for (int k = kWaves - 2; k >= 0; --k) {
            h = fmaf(sh.A[k], h, sh.U[k]);
            a *= sh.A[k];
        }
        give_map(g, u, a, h);
    }
    if (wave == 0) {
        const float v = await(g, u, g.dh_last);
        if (threadIdx.x == 0) sh.carry = v;
    }
    __syncthreads();
    for (int k = 0; k < wave; ++k) s = fmaf(sh.A[k], s, sh.H[k]);
    s = fmaf(lane_before<64>(t.A, 1.f), s, lane_before<64>(t.H, 0.f));
    float v = sh.carry;
    for (int k = kWaves - 1; k > wave; --k) v = fmaf(sh.A[k], v, sh.U[k]);
    if (threadIdx.x == 63) give_state(g, u, g.dh0, fmaf(B, v, U));
    v = fmaf(lane_mirror<64>(lane_before<64>(B, 1.f)), v, lane_mirror<64>(lane_before<64>(U, 0.f)));
    const float sum = lane_sum<64>(t.close(g, u.w, p0, rate, s, v));
    __syncthreads();
    if ((threadIdx.x & 63) == 0) sh.U[wave] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        float q = sh.U[0];
        for (int k = 1; k < kWaves; ++k) q += sh.U[k];
        g.part[u.m * rows + u.w.id] = q;
    }
}

template <class D, bool REV>
__global__ __launch_bounds__(kSpread) void k_spread_bwd(Args g) {
    __shared__ Spread sh;
    const unsigned from = take_share(g.carry, &sh.unit);
    for (unsigned k = from; k < min(from + g.carry.share, g.carry.units); ++k) {
        const Unit u = unit_at(g, k);
        if (u.m >= u.valid) {
            if (threadIdx.x == 0) {
                if (u.m == 0 && g.dh0) g.dh0[u.w.id] = g.dh_last ? g.dh_last[u.w.id] : 0.f;
                g.part[(long long)u.m * g.B * g.C + u.w.id] = 0.f;
            }
            pad<D>(g, u, g.dx, g.dx_sb, g.dx_sr);
            pad<D>(g, u, g.dr, g.dr_sb, g.dr_sr);
            pad<D>(g, u, g.di, g.di_sb, g.di_sr);
        } else if ((u.valid - u.m) * kWide <= u.w.len) {
            spread_bwd<D, REV, true>(g, u, sh);
        } else {
            spread_bwd<D, REV, false>(g, u, sh);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------

// Lanes per row and positions per lane, or LW = 0: tiles spread over
// workgroups.  By the shape alone, so that the states of a forward call fit
// the backward one: the narrowest group that holds the row in one tile, else
// whole wavefronts of 8 positions per lane.
//
// A wavefront that walks a row takes about 0.85 us per tile of 512, whatever
// else runs; spreading costs about 15 us and the counter's 13 ns per tile of
// 4096.  Forward + backward, walked and spread, fp32: 16 rows of 12544
// positions 62 and 42 us, 256 of 12544 71 and 56, 256 of 50176 297 and 149,
// 768 of 12544 96 and 125, 768 of 50176 398 and 385, 1536 of 50176 763 and 728
// (bf16 there 410 and 460).
bool spread(const gscan_shape& s) {
    const long long rows = (long long)s.B * s.C;
    return rows <= 1024 && s.T > 32 * (rows < 256 ? 256 : rows);
}
struct Form {
    int V, LW;
};
Form form_of(const gscan_shape& s) {
    if (s.T <= 4) return {4, 1};
    if (s.T <= 64) return {4, 16};
    if (s.T <= 256) return {4, 64};
    if (spread(s)) return {kWideV, 0};
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
void launch_spread(bool bwd, bool rev, const Args& a, hipStream_t st) {
    const dim3 grid(shares(a.carry));
    if (bwd) {
        if (rev) k_spread_bwd<D, true><<<grid, kSpread, 0, st>>>(a);
        else k_spread_bwd<D, false><<<grid, kSpread, 0, st>>>(a);
    } else {
        if (rev) k_spread_fwd<D, true><<<grid, kSpread, 0, st>>>(a);
        else k_spread_fwd<D, false><<<grid, kSpread, 0, st>>>(a);
    }
}
template <class D>
void launch_form(const Form& f, bool bwd, bool rev, const Args& a, hipStream_t st) {
    if (f.LW == 0) launch_spread<D>(bwd, rev, a, st);
    else if (f.LW == 1) launch<D, 4, 1>(bwd, rev, a, st);
    else if (f.LW == 16) launch<D, 4, 16>(bwd, rev, a, st);
    else if (f.V == 4) launch<D, 4, 64>(bwd, rev, a, st);
    else launch<D, 8, 64>(bwd, rev, a, st);
}

size_t words_of(const gscan_shape& s, const Form& f, int tiles) {
    return f.LW == 0 ? carry_bytes(size_t(s.B) * s.C, tiles) : 0;
}

// The words between tiles come first in the workspace, then the partial sums.
hipError_t run(const gscan_shape& s, bool bwd, Args& a, void* ws, hipStream_t st) {
    const Form f = form_of(s);
    const Plan p = planes_plan(s);
    const size_t words = words_of(s, f, p.tiles);
    a.tiles = p.tiles;
    a.part = reinterpret_cast<float*>(static_cast<char*>(ws) + words);
    if (words) {
        a.carry = carry_at(ws, size_t(s.B) * s.C, p.tiles, unsigned(s.B) * s.C * p.tiles, kShare);
        const hipError_t e = clear_carry(ws, words, st);
        if (e != hipSuccess) return e;
    }
    const bool rev = s.reverse != 0;
    if (s.dtype == GSCAN_F32) launch_form<F32>(f, bwd, rev, a, st);
    else if (s.dtype == GSCAN_F16) launch_form<F16>(f, bwd, rev, a, st);
    else launch_form<BF16>(f, bwd, rev, a, st);
    return hipGetLastError();
}

}  // namespace

Plan planes_plan(const gscan_shape& s) {
    const Form f = form_of(s);
    const int tile = f.LW == 0 ? kWide : f.V * f.LW;
    Plan p;
    p.tiles = s.T > 0 ? (s.T - 1) / tile + 1 : 1;
    p.parts = f.LW == 0 ? (long long)p.tiles * s.B : s.B;
    p.states = sizeof(float) * size_t(p.tiles) * s.B * s.C;
    p.scratch = words_of(s, f, p.tiles) + sizeof(float) * size_t(p.parts) * s.C;
    // a row that is walked takes a wavefront at the most, of rows fewer than 2^26
    p.fits = f.LW != 0 || (long long)s.B * s.C * p.tiles < kMaxThreads / kSpread;
    return p;
}

hipError_t planes_fwd(const gscan_shape& s, Args a, void* ws, hipStream_t st) {
    return run(s, false, a, ws, st);
}

hipError_t planes_bwd(const gscan_shape& s, Args a, void* ws, hipStream_t st) {
    const hipError_t e = run(s, true, a, ws, st);
    return e == hipSuccess ? close_dlam(a, planes_plan(s).parts, st) : e;
}

}  // namespace gsc

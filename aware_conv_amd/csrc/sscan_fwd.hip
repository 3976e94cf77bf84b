// Forward pass and single positions of the selective scan (include/sscan.h).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "sscan_math.h"

namespace ssc {
namespace {

constexpr int kTile = 16;   // positions whose b and c a wavefront holds
constexpr int kWaves = 4;   // of a workgroup: 64 channels, a cache line of 16-bit elements
constexpr int kPad = 18;    // floats2 between two channels' rows in LDS: no bank conflicts

// What a wavefront reads of a tile: each lane the elements of its channel at
// every fourth position, and its row's states of one position.
template <class D, int NP, bool GATE, bool SUMS>
struct Tile {
    float x[4], dt[4], z[4], b[NP], c[NP];
    __device__ __forceinline__ void load(const Args& a, const typename D::S* x_, const typename D::S* dt_,
                                         const typename D::S* z_, const typename D::S* b_,
                                         const typename D::S* c_, int t0, int n, int row, int i,
                                         bool whole) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const long long t = min(t0 + 4 * k + row, n - 1);
            x[k] = gsc::load_one<D>(x_ + t * a.x_sr);
            dt[k] = gsc::load_one<D>(dt_ + t * a.dt_sr);
            if constexpr (GATE && SUMS) z[k] = gsc::load_one<D>(z_ + t * a.z_sr);
        }
        const bool valid = t0 + i < n;
        const long long t = min(t0 + i, n - 1);
        load_states<D, NP>(b, b_ + t * a.b_sr, row * NP, a.N, whole, valid);
        if constexpr (SUMS) load_states<D, NP>(c, c_ + t * a.c_sr, row * NP, a.N, whole, valid);
    }
};

// SUMS: the pass that gives y.  Otherwise: what a segment does to a state that
// starts from zero, and its sum of delta (with which the state it starts from decays).
template <class D, int NP, bool GATE, bool SUMS>
__global__ __launch_bounds__(64 * kWaves) void k_fwd(Args a) {
    using S = typename D::S;
    __shared__ float2 lds[kWaves][16 * kPad];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int row = lane >> 4, i = lane & 15;
    const int tiles = a.G * a.tiles;
    const int tile = blockIdx.x % tiles, rest = blockIdx.x / tiles;
    const int seq = rest / a.S, s = rest % a.S;
    const int group = tile / a.tiles, c0 = (tile % a.tiles) * 64 + wave * 16;
    if (c0 >= a.Dg) return;
    const bool live = c0 + i < a.Dg;
    const int d = group * a.Dg + min(c0 + i, a.Dg - 1);
    const int n = a.lengths ? min(max(a.lengths[seq], 0), a.T) : a.T;
    const int t_lo = s * a.seg, t_end = min(a.T - t_lo, a.seg) + t_lo, t_hi = min(t_end, n);
    S* const y_ = SUMS ? (S*)a.y + seq * a.y_sb + d : nullptr;
    const long long states_at = ((long long)seq * a.D + d) * a.N;  // of a [B][D][N]
    const long long all = (long long)a.B * a.D * a.N;

    if constexpr (SUMS) {
        if (live)
            for (int t = max(n, t_lo) + row; t < t_end; t += 4)
                gsc::store_one<D>(y_ + t * a.y_sr, 0.f);
    }
    if (t_lo >= t_hi && !(SUMS && s == 0)) return;
    if (!SUMS && s == a.S - 1) return;  // nothing starts from the last one's

    float a2[NP], h[NP];
    bool there[NP];
#pragma unroll
    for (int j = 0; j < NP; ++j) {
        const int m = row * NP + j;
        there[j] = m < a.N;
        const int at = min(m, a.N - 1);
        a2[j] = there[j] ? -kLog2e * expf(a.a_log[(long long)d * a.N + at]) : 0.f;
        h[j] = SUMS && a.h0 && there[j] ? a.h0[states_at + at] : 0.f;
    }
    if constexpr (SUMS) {
        // the segments before, one after the other
        for (int k = 0; k < s; ++k) {
            const float sum = a.seg_sum[((long long)k * a.B + seq) * a.D + d];
#pragma unroll
            for (int j = 0; j < NP; ++j) {
                const float own = a.seg_state[k * all + states_at + min(row * NP + j, a.N - 1)];
                h[j] = there[j] ? fmaf(exp2_hw(sum * a2[j]), h[j], own) : 0.f;
            }
        }
        if (n == 0) {
            if (live && a.h_last)
#pragma unroll
                for (int j = 0; j < NP; ++j)
                    if (there[j]) a.h_last[states_at + row * NP + j] = h[j];
            return;
        }
    }
    const float bias = a.dt_bias ? a.dt_bias[d] : 0.f;
    const float skip = SUMS && a.d ? a.d[d] : 0.f;
    const S* const x_ = (const S*)a.x + seq * a.x_sb + d;
    const S* const dt_ = (const S*)a.dt + seq * a.dt_sb + d;
    const S* const z_ = GATE && SUMS ? (const S*)a.z + seq * a.z_sb + d : nullptr;
    const S* const b_ = (const S*)a.b + seq * a.b_sb + group * a.N;
    const S* const c_ = SUMS ? (const S*)a.c + seq * a.c_sb + group * a.N : nullptr;
    const bool whole = a.N == 4 * NP;
    constexpr int kChunk = NP == 16 ? 16 : 32;
    float2* const mine = lds[wave] + i * kPad;
    float sum = 0.f;

    Tile<D, NP, GATE, SUMS> now, next;
    now.load(a, x_, dt_, z_, b_, c_, t_lo, n, row, i, whole);
    for (int t0 = t_lo; t0 < t_hi; t0 += kTile) {
        if (SUMS && a.states && t0 % kChunk == 0 && live) {
            float* to = a.states + (t0 / kChunk) * all + states_at;
#pragma unroll
            for (int j = 0; j < NP; ++j)
                if (there[j]) to[row * NP + j] = h[j];
        }
        float xs[4], zs[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const bool valid = t0 + 4 * k + row < t_hi && live;
            xs[k] = now.x[k];
            if constexpr (GATE && SUMS) zs[k] = now.z[k];
            const float delta = valid ? softplus(now.dt[k] + bias).delta : 0.f;
            if constexpr (!SUMS) sum += delta;
            mine[4 * k + row] = make_float2(delta, valid ? delta * xs[k] : 0.f);
        }
        wave_sync();
        if (t0 + kTile < t_hi) next.load(a, x_, dt_, z_, b_, c_, t0 + kTile, n, row, i, whole);
        float own[4];
        unroll<4>([&](auto K) {
            float part[4] = {0.f, 0.f, 0.f, 0.f};
            unroll<4>([&](auto L) {
                constexpr int k = 4 * K + L;
                const float2 q = mine[k];
#pragma unroll
                for (int j = 0; j < NP; ++j) {
                    h[j] = fmaf(decay(q.x, a2[j]), h[j], bcast<k>(now.b[j]) * q.y);
                    if constexpr (SUMS) part[L] = fmaf(bcast<k>(now.c[j]), h[j], part[L]);
                }
            });
            if constexpr (SUMS) own[K] = sum_rows(part[0], part[1], part[2], part[3]);
        });
        if constexpr (SUMS) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int t = t0 + 4 * k + row;
                float v = fmaf(skip, xs[k], own[k]);
                if constexpr (GATE) v *= zs[k] * sig(zs[k]);
                if (t < t_hi && live) gsc::store_one<D>(y_ + t * a.y_sr, v);
            }
        }
        wave_sync();
        now = next;
    }
    if (!live) return;
    if constexpr (SUMS) {
        if (a.h_last && t_hi == n)
#pragma unroll
            for (int j = 0; j < NP; ++j)
                if (there[j]) a.h_last[states_at + row * NP + j] = h[j];
    } else {
#pragma unroll
        for (int j = 0; j < NP; ++j)
            if (there[j]) a.seg_state[s * all + states_at + row * NP + j] = h[j];
        const float total = sum_rows(sum, sum, sum, sum);
        if (row == 0) a.seg_sum[((long long)s * a.B + seq) * a.D + d] = total;
    }
}

template <class D, int NP>
hipError_t run_fwd(const Args& a, hipStream_t st) {
    const dim3 block(64 * kWaves);
    const unsigned units = unsigned(a.G) * a.tiles * a.B * a.S;
    if (a.S > 1) k_fwd<D, NP, false, false><<<units, block, 0, st>>>(a);
    if (a.z) k_fwd<D, NP, true, true><<<units, block, 0, st>>>(a);
    else k_fwd<D, NP, false, true><<<units, block, 0, st>>>(a);
    return hipGetLastError();
}
template <class D>
hipError_t run_fwd(const Args& a, int per_lane, hipStream_t st) {
    switch (per_lane) {
        case 1: return run_fwd<D, 1>(a, st);
        case 2: return run_fwd<D, 2>(a, st);
        case 4: return run_fwd<D, 4>(a, st);
        case 8: return run_fwd<D, 8>(a, st);
        default: return run_fwd<D, 16>(a, st);
    }
}

// One position: four lanes per channel, each with every fourth group of V states.
template <class D, int V>
__global__ __launch_bounds__(256) void k_step(StepArgs a) {
    using S = typename D::S;
    const long long at = (long long)blockIdx.x * 64 + threadIdx.x / 4;
    const int q = threadIdx.x & 3;
    if (at >= (long long)a.B * a.D) return;
    const int seq = int(at / a.D), d = int(at % a.D), group = d / a.Dg;
    const int slot = a.slots ? a.slots[seq] : seq;
    S* const y = (S*)a.y + seq * a.y_sb + d;
    if (slot < 0 || slot >= a.S) {
        if (q == 0) gsc::store_one<D>(y, 0.f);
        return;
    }
    const float x = gsc::load_one<D>((const S*)a.x + seq * a.x_sb + d);
    const float pre = gsc::load_one<D>((const S*)a.dt + seq * a.dt_sb + d) + (a.dt_bias ? a.dt_bias[d] : 0.f);
    const float delta = softplus(pre).delta, u = delta * x;
    float* const h_ = a.state + ((long long)slot * a.D + d) * a.N;
    const float* const a_ = a.a_log + (long long)d * a.N;
    const S* const b_ = (const S*)a.b + seq * a.b_sb + group * a.N;
    const S* const c_ = (const S*)a.c + seq * a.c_sb + group * a.N;
    float sum = 0.f;
    for (int m = q * V; m < a.N; m += 4 * V) {
        float h[V], al[V];
        gsc::Raw<F32, V> r;
        gsc::load_vec<F32, V>(r, h_ + m);
#pragma unroll
        for (int j = 0; j < V; ++j) h[j] = r.get(j);
        gsc::load_vec<F32, V>(r, a_ + m);
#pragma unroll
        for (int j = 0; j < V; ++j) al[j] = r.get(j);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            h[j] = fmaf(decay(delta, -kLog2e * expf(al[j])), h[j], u * gsc::load_one<D>(b_ + m + j));
            sum = fmaf(gsc::load_one<D>(c_ + m + j), h[j], sum);
        }
        gsc::store_vec<F32, V>(h_ + m, gsc::pack<F32, false>(h));
    }
    sum += __shfl_xor(sum, 1);
    sum += __shfl_xor(sum, 2);
    if (q) return;
    if (a.d) sum = fmaf(a.d[d], x, sum);
    if (a.z) {
        const float z = gsc::load_one<D>((const S*)a.z + seq * a.z_sb + d);
        sum *= z * sig(z);
    }
    gsc::store_one<D>(y, sum);
}

template <class D>
hipError_t run_step(const StepArgs& a, hipStream_t st) {
    const unsigned blocks = unsigned(((long long)a.B * a.D + 63) / 64);
    if (a.N % 4 == 0) k_step<D, 4><<<blocks, 256, 0, st>>>(a);
    else k_step<D, 1><<<blocks, 256, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace

Plan plan(const sscan_shape& s, bool backward) {
    Plan p{};
    const int q = (s.N + 3) / 4;
    p.per_lane = q <= 1 ? 1 : q <= 2 ? 2 : q <= 4 ? 4 : q <= 8 ? 8 : 16;
    p.chunk = p.per_lane == 16 ? 16 : 32;
    const long long tiles = s.G ? (s.D / s.G + 63) / 64 : 0;
    const long long units = s.G * tiles * s.B;
    const long long chunks = (s.T + p.chunk - 1LL) / p.chunk;
    p.fits = units < (1LL << 20) && s.B * ((s.T + 15LL) / 16) < (1LL << 31);
    // workgroups enough for two on each compute unit, segments of 4 chunks at least
    long long S = 1;
    if (units && units < 256) S = std::max(1LL, std::min({512 / units, chunks / 4, 64LL}));
    const long long per = S ? (chunks + S - 1) / S : 0;
    p.seg = int(std::max(1LL, per) * p.chunk);
    p.S = int(std::max(1LL, per ? (chunks + per - 1) / per : 1));
    const size_t rows = size_t(s.B) * s.D, all = rows * s.N;
    p.states = 4 * size_t(chunks) * all;
    if (p.S > 1) p.scratch += 4 * size_t(p.S) * (all + rows);
    if (backward) {
        p.scratch += 4 * size_t(tiles) * s.B * s.T * s.G * 2 * s.N;
        p.scratch += 4 * size_t(p.S) * (all + 2 * rows);
    }
    return p;
}

hipError_t fwd(const sscan_shape& s, Args a, void* ws, hipStream_t st) {
    const Plan p = plan(s, false);
    a.S = p.S;
    a.seg = p.seg;
    a.seg_state = static_cast<float*>(ws);
    a.seg_sum = a.seg_state + size_t(p.S) * s.B * s.D * s.N;
    switch (s.dtype) {
        case GSCAN_F32: return run_fwd<F32>(a, p.per_lane, st);
        case GSCAN_F16: return run_fwd<F16>(a, p.per_lane, st);
        default: return run_fwd<BF16>(a, p.per_lane, st);
    }
}

hipError_t step(int dtype, const StepArgs& a, hipStream_t st) {
    switch (dtype) {
        case GSCAN_F32: return run_step<F32>(a, st);
        case GSCAN_F16: return run_step<F16>(a, st);
        default: return run_step<BF16>(a, st);
    }
}

}  // namespace ssc

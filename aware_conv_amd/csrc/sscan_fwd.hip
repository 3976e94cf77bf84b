// Forward pass and single positions of the selective scan (include/sscan.h).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "sscan_math.h"

namespace ssc {
namespace {

constexpr int kPad = 18;  // float2s between two channels' rows in LDS: no bank conflicts

// SUMS: the pass that gives y.  Otherwise: what a segment does to a state that
// starts from zero, and its sum of delta (with which the state it starts from decays).
//
// The vector ALU bounds it: of a tile's turn 167 plain instructions, 64 with a DPP
// modifier, 40 transcendental and 12 lane exchanges, 1140 cycles of a SIMD by what
// each takes at four wavefronts and 1240 at two (694 of them are the states' own steps,
// sscan_math.h); 720 in the pass over segments.  16 states, bf16: 8 sequences of 4096
// positions of 2048 channels 435 us (362 where no states are saved), of which two
// wavefronts' instructions are 264 and HBM would take 110; one of 65521 of 2560
// channels, whose 40 workgroups become 480 by cutting it into segments, 520 us for
// what the segments do (350 by instructions) and 840 for y (610).
//
// In a tile's turn the wavefronts compute from the delta and u in one half of LDS,
// then put those of the next tile into the other half, and, past the barrier,
// add up each other's sums over states and write y.
template <class D, class F, bool GATE, bool SUMS>
__global__ __launch_bounds__(F::kThreads) __attribute__((amdgpu_waves_per_eu(2, 4))) void k_fwd(Args a) {
    using S = typename D::S;
    constexpr int NP = F::NP, NB = F::NB, kSlots = F::kSlots;
    __shared__ float2 staged[2][F::kChannels * kPad];
    __shared__ float parts[2][SUMS ? NB : 1][SUMS ? 16 * F::kChannels : 1];
    const Lane<F> l(a);
    const int first_t = l.io_base + l.io_row;  // the thread's first position of a tile
    const bool last_slot = l.last_slot;

    if constexpr (SUMS) {
        if (max(l.n, l.t_lo) < l.t_end) {  // zeros behind the sequence
            S* const y0 = (S*)a.y + l.seq * a.y_sb + l.io_d;
            for (int t = max(l.n, l.t_lo) + first_t; t < l.t_end; t += F::kStep) gsc::store_one<D>(y0 + t * a.y_sr, 0.f);
        }
    }
    if (l.t_lo >= l.t_hi && !(SUMS && l.s == 0)) return;
    if (!SUMS && l.s == a.S - 1) return;  // nothing starts from the last one's

    float h[NP];
#pragma unroll
    for (int j = 0; j < NP; ++j) h[j] = SUMS && a.h0 ? a.h0[l.states_at + l.at[j]] : 0.f;
    auto keep = [&](float* to) {
#pragma unroll
        for (int j = 0; j < NP; ++j) to[l.states_at + l.at[j]] = h[j];
    };
    if constexpr (SUMS) {
        // the segments before, one after the other
        for (int k = 0; k < l.s; ++k) {
            const float sum = a.seg_sum[((long long)k * a.B + l.seq) * a.D + l.d];
#pragma unroll
            for (int j = 0; j < NP; ++j)
                h[j] = fmaf(exp2_hw(sum * l.a2[j]), h[j], a.seg_state[k * l.all + l.states_at + l.at[j]]);
        }
        if (l.n == 0) {
            if (a.h_last) keep(a.h_last);
            return;
        }
    }
    const float skip = SUMS && a.d ? a.d[l.io_d] : 0.f;
    auto wide = [&](const void* p, long long sb, long long sr) {
        return Rows<S>(p, sb, sr, l.seq, l.t_lo + l.io_base, l.d0, l.io_row, l.io_ch);
    };
    Rows<S> x_ = wide(a.x, a.x_sb, a.x_sr), dt_ = wide(a.dt, a.dt_sb, a.dt_sr), z_ = wide(a.z, a.z_sb, a.z_sr);
    Rows<S> y_ = wide(a.y, a.y_sb, a.y_sr);
    const int low0 = l.group * a.N;
    Rows<S> b_(a.b, a.b_sb, a.b_sr, l.seq, l.t_lo, low0, l.i, 0), c_(a.c, a.c_sb, a.c_sr, l.seq, l.t_lo, low0, l.i, 0);
    float* states_ = SUMS && a.states ? a.states + saved_at(a, l, l.t_lo / kChunk) : nullptr;
    const long long states_step = saved_at(a, l, 1) - saved_at(a, l, 0);
    float sum = 0.f;

    // What is read of a tile, `left` positions of which there are (`full`: all).
    // Behind the sequence nothing is read.
    Column<D, F> x, dt, z;
    States<D, NP> b, c;
    auto load = [&](auto full, int left) {
        if constexpr (full) {
            x.load(x_, last_slot);
            dt.load(dt_, last_slot);
            if constexpr (GATE && SUMS) z.load(z_, last_slot);
            b.load(b_.at(0), l);
            if constexpr (SUMS) c.load(c_.at(0), l);
        } else {
            x.load_some(x_, last_slot, left - first_t);
            dt.load_some(dt_, last_slot, left - first_t);
            if constexpr (GATE && SUMS) z.load_some(z_, last_slot, left - first_t);
            b.clear();
            c.clear();
            if (l.i < left) {
                b.load(b_.at(0), l);
                if constexpr (SUMS) c.load(c_.at(0), l);
            }
        }
        x_.move(kChunk);
        dt_.move(kChunk);
        b_.move(kChunk);
        if constexpr (GATE && SUMS) z_.move(kChunk);
        if constexpr (SUMS) c_.move(kChunk);
    };
    float xs[kSlots], zs[kSlots], bs[NP], cs[NP];
    auto stage = [&](auto full, float2* to, int left) {
#pragma unroll
        for (int j = 0; j < NP; ++j) {
            bs[j] = b[j];
            now(bs[j]);
            if constexpr (SUMS) {
                cs[j] = l.there[j] ? c[j] : 0.f;
                now(cs[j]);
            }
        }
#pragma unroll
        for (int q = 0; q < kSlots; ++q) {
            if ((q + 1) * F::kStep > 16 && !last_slot) continue;
            const int t = first_t + F::kStep * q;
            const bool valid = full || t < left;
            xs[q] = x[q];
            now(xs[q]);
            if constexpr (GATE && SUMS) {
                zs[q] = z[q];
                now(zs[q]);
            }
            const float delta = valid ? softplus(dt[q] + l.bias).delta : 0.f;
            if constexpr (!SUMS) sum += delta;
            to[l.io_at * kPad + t] = make_float2(delta, valid ? delta * xs[q] : 0.f);
        }
    };
    int half = 0;
    // One tile's turn.  full: it and the two that follow are whole, so that what is in flight
    // at each point is known, and nothing is waited for before it is used.
    auto turn = [&](auto full, int left) {
        if (states_) {
#pragma unroll
            for (int j = 0; j < NP; ++j) __builtin_nontemporal_store(h[j], states_ + 64 * j);
            states_ += states_step;
        }
        // Four positions at a time: while the states pass them, what the next four need is
        // formed (their decays and inputs do not wait for the states), and those after
        // that are on their way from LDS.
        const float2* const mine = staged[half] + (l.ct * 16 + l.i) * kPad;
        float2 m[2][4];
        float e[2][4][NP], in[2][4][NP];
        auto fetch = [&](auto K) {
            constexpr int k = K;
#pragma unroll
            for (int q = 0; q < 4; ++q) m[k & 1][q] = mine[4 * k + q];
        };
        auto form = [&](auto K) {
            constexpr int k = K;
            unroll<4>([&](auto L) {
                constexpr int q = L;
#pragma unroll
                for (int j = 0; j < NP; ++j) {
                    e[k & 1][q][j] = decay(m[k & 1][q].x, l.a2[j]);
                    in[k & 1][q][j] = bcast<4 * k + q>(bs[j]) * m[k & 1][q].y;
                }
            });
        };
        fetch(std::integral_constant<int, 0>{});
        fetch(std::integral_constant<int, 1>{});
        form(std::integral_constant<int, 0>{});
        unroll<4>([&](auto K) {
            constexpr int k = K;
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (k < 2) fetch(std::integral_constant<int, k + 2>{});
            float part[4];
            unroll<4>([&](auto L) {
                constexpr int q = L;
#pragma unroll
                for (int j = 0; j < NP; ++j) h[j] = fmaf(e[k & 1][q][j], h[j], in[k & 1][q][j]);
                if constexpr (SUMS) part[q] = sum_bcast<4 * k + q>(cs, h);
            });
            if constexpr (k < 3) form(std::integral_constant<int, k + 1>{});
            if constexpr (SUMS) parts[half][l.nb][(4 * k + l.row) * F::kChannels + l.ct * 16 + l.i] = sum_rows(part[0], part[1], part[2], part[3]);
        });
        float xe[kSlots], ze[kSlots];
#pragma unroll
        for (int q = 0; q < kSlots; ++q) {
            xe[q] = xs[q];
            if constexpr (GATE && SUMS) ze[q] = zs[q];
        }
        if (full || left > kChunk) stage(full, staged[half ^ 1], left - kChunk);
        if (full || left > 2 * kChunk) load(full, left - 2 * kChunk);
        lds_barrier();
        if constexpr (SUMS) {
#pragma unroll
            for (int q = 0; q < kSlots; ++q) {
                if ((q + 1) * F::kStep > 16 && !last_slot) continue;
                const int t = first_t + F::kStep * q;
                float v = parts[half][0][t * F::kChannels + l.io_at];
#pragma unroll
                for (int k = 1; k < NB; ++k) v += parts[half][k][t * F::kChannels + l.io_at];
                v = fmaf(skip, xe[q], v);
                if constexpr (GATE) v *= ze[q] * sig(ze[q]);
                if (full || t < left) gsc::store_one<D>(y_.to(F::kStep * q), v);
            }
            y_.move(kChunk);
        }
        half ^= 1;
    };
    constexpr std::true_type whole{};
    constexpr std::false_type some{};
    int left = l.t_hi - l.t_lo;
    load(some, left);
    stage(some, staged[0], left);
    if (left > kChunk) load(some, left - kChunk);
    lds_barrier();
    loads_done();
    for (; left >= 3 * kChunk; left -= kChunk) turn(whole, left);
    for (; left > 0; left -= kChunk) turn(some, left);
    if constexpr (SUMS) {
        if (a.h_last && l.t_hi == l.n) keep(a.h_last);
    } else {
        keep(a.seg_state + l.s * l.all);
        const float total = over_channel<F>(sum, reinterpret_cast<float*>(staged));
        if (threadIdx.x < F::kChannels) a.seg_sum[((long long)l.s * a.B + l.seq) * a.D + l.io_d] = total;
    }
}

template <class D, class F>
hipError_t run_fwd(const Args& a, hipStream_t st) {
    const unsigned units = unsigned(a.G) * a.tiles * a.B * a.S;
    if (a.S > 1) k_fwd<D, F, false, false><<<units, F::kThreads, 0, st>>>(a);
    if (a.z) k_fwd<D, F, true, true><<<units, F::kThreads, 0, st>>>(a);
    else k_fwd<D, F, false, true><<<units, F::kThreads, 0, st>>>(a);
    return hipGetLastError();
}

// One position.  HBM bounds it: the states are most of what is read and written.  Four
// lanes take a channel, V of its states at a time, of Q sequences, so that Q vectors of
// states are under way in each thread and a channel's rates are formed once for all of
// them; the states are asked for before anything is waited for.  512 sequences of 4096
// channels, 16 states, bf16: 286 MB in 74 us (3.9 TB/s); one of 384 channels 3.7 us.
template <class D, int V, int Q>
__global__ __launch_bounds__(256) void k_step(StepArgs a) {
    using S = typename D::S;
    const int per = (a.D + 63) / 64, seq0 = a.first + blockIdx.x / per * Q;
    const int d = blockIdx.x % per * 64 + threadIdx.x / 4, lane = threadIdx.x & 3, group = d / a.Dg;
    if (d >= a.D) return;  // whole groups of four
    float x[Q], delta[Q], sum[Q];
    float* h_[Q];
    const S *b_[Q], *c_[Q];
    const float bias = a.dt_bias ? a.dt_bias[d] : 0.f;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const int seq = min(seq0 + q, a.B - 1);
        const int slot = a.slots ? a.slots[seq] : seq;
        const bool on = seq0 + q < a.B && slot >= 0 && slot < a.S;
        h_[q] = on ? a.state + ((long long)slot * a.D + d) * a.N : nullptr;
        b_[q] = (const S*)a.b + seq * a.b_sb + group * a.N;
        c_[q] = (const S*)a.c + seq * a.c_sb + group * a.N;
        x[q] = gsc::load_one<D>((const S*)a.x + seq * a.x_sb + d);
        delta[q] = gsc::load_one<D>((const S*)a.dt + seq * a.dt_sb + d);
        sum[q] = 0.f;
    }
    const float* const a_ = a.a_log + (long long)d * a.N;
    bool first = true;  // delta is still dt
    for (int m = lane * V; m < a.N; m += 4 * V) {
        gsc::Raw<F32, V> h[Q], al;
        gsc::load_vec<F32, V>(al, a_ + m);
#pragma unroll
        for (int q = 0; q < Q; ++q)
            if (h_[q]) gsc::load_vec<F32, V>(h[q], h_[q] + m);
        gsc::Raw<D, V> b[Q], c[Q];
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            if constexpr (V > 1) {
                gsc::load_vec<D, V>(b[q], b_[q] + m);
                gsc::load_vec<D, V>(c[q], c_[q] + m);
            } else {
                b[q].w[0] = c[q].w[0] = 0;
                b[q].set(0, gsc::load_one<D>(b_[q] + m));
                c[q].set(0, gsc::load_one<D>(c_[q] + m));
            }
        }
        if (first) {
#pragma unroll
            for (int q = 0; q < Q; ++q) delta[q] = softplus(delta[q] + bias).delta;
            first = false;
        }
        float a2[V];
#pragma unroll
        for (int j = 0; j < V; ++j) a2[j] = rate_of(al.get(j));
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            if (!h_[q]) continue;
            float v[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                v[j] = fmaf(decay(delta[q], a2[j]), h[q].get(j), delta[q] * x[q] * b[q].get(j));
                sum[q] = fmaf(c[q].get(j), v[j], sum[q]);
            }
            gsc::store_vec<F32, V>(h_[q] + m, gsc::pack<F32, false>(v));
        }
    }
    const float skip = a.d ? a.d[d] : 0.f;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        sum[q] += __shfl_xor(sum[q], 1);
        sum[q] += __shfl_xor(sum[q], 2);
        if (lane || seq0 + q >= a.B) continue;
        float v = fmaf(skip, x[q], sum[q]);
        if (a.z) {
            const float z = gsc::load_one<D>((const S*)a.z + (seq0 + q) * a.z_sb + d);
            v *= z * sig(z);
        }
        gsc::store_one<D>((S*)a.y + (seq0 + q) * a.y_sb + d, h_[q] ? v : 0.f);
    }
}

template <class D, int V>
hipError_t run_step(StepArgs a, hipStream_t st) {
    const long long per = (a.D + 63) / 64;
    // Two sequences to a thread from 16384 workgroups of one on: 4096 channels of 16 states, bf16,
    // 512 sequences 74 us by two, 83 by one, 84 by four; 256: 34 by two, 37 by one; 128 (8192
    // workgroups) 21 either way; 8: 4.2 by two, 3.8 by one.
    if (a.B * per < 16384) {
        k_step<D, V, 1><<<unsigned(a.B * per), 256, 0, st>>>(a);
        return hipGetLastError();
    }
    // a launch has fewer than 2^32 threads
    const long long pairs = (a.B + 1LL) / 2, most = (1LL << 23) / per;
    for (long long first = 0; first < pairs; first += most) {
        a.first = int(2 * first);
        k_step<D, V, 2><<<unsigned(std::min(most, pairs - first) * per), 256, 0, st>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}
template <class D>
hipError_t run_step(const StepArgs& a, hipStream_t st) {
    return a.N % 4 == 0 ? run_step<D, 4>(a, st) : run_step<D, 1>(a, st);
}

}  // namespace

Plan plan(const sscan_shape& s, bool backward) {
    Plan p{};
    const int q = (s.N + 3) / 4;
    // Two states to a lane wherever there are that many, divided among up to four wavefronts.
    // 16 states, 8 sequences of 4096 positions of 2048 channels, forwards and backwards: two to a
    // lane 450 and 1090 us; one to a lane, in four wavefronts, 450 and 1200; four, in one, 3660 backwards.
    // Measured at 16 states alone.  As divided here, other numbers of states, the same otherwise:
    // 4: 274 and 681; 8 (one wavefront): 325 and 853; 24: 677 and 1949; 32: 618 and 2002; 48: 1405 and
    // 6332; 64: 1279 and 3980.
    p.per_lane = q <= 1 ? 1 : q <= 8 ? 2 : 4;
    p.waves = (q + p.per_lane - 1) / p.per_lane;
    p.width = p.waves <= 2 ? 64 : 32;
    p.tiles = s.G ? (s.D / s.G + p.width - 1) / p.width : 0;
    const long long units = (long long)s.G * p.tiles * s.B;
    const long long chunks = (s.T + kChunk - 1LL) / kChunk;
    p.fits = units < (1LL << 20) && s.B * chunks < (1LL << 31);
    // One workgroup on a compute unit takes 88 ns a position forwards and 246 backwards (16 states),
    // however many others there are up to 256; a second one on it costs 30% more for both.
    // Segments cost a pass over all but the last more, so a sequence is cut where that leaves at
    // least three, of two workgroups on a compute unit in all.  Microseconds whole and cut, bf16,
    // one sequence of 4096 positions (24 and 64 states: 2048), forwards with states kept / backwards:
    //   workgroups          96          128         170         171 to 191
    //   segments            5           4           3           2
    //    8 states  whole    305 / 846   305 / 852   306 / 862   310 / 863
    //              cut      159 / 351   193 / 425   251 / 557   325 / 779
    //   16         whole    365 / 1008  371 / 1013  426 / 1026  427 / 1032
    //              cut      221 / 535   273 / 658   370 / 874   461 / 1199
    //   24         whole    196 / 489   196 / 492   195 / 498   202 / 500
    //              cut      120 / 277   145 / 331   187 / 433   225 / 596
    //   64         whole    295 / 940   296 / 962   298 / 991   297 / 998
    //              cut      216 / 495   261 / 615   338 / 813   398 / 1110
    // and 32 workgroups of 16 states forwards 361 whole, 87 in 8 or 16 segments, 110 in 32.
    // Two pay backwards only, where a wavefront has all the states (up to 8).  Three may cost a
    // forward pass more than they give: 16 states, 1024 positions 103 cut, 96 whole.
    const long long fill = units ? 512 / units : 0, least = backward && p.waves == 1 ? 2 : 3;
    long long S = 1;
    if (units < 192 && fill >= least) S = std::max(1LL, std::min({fill, chunks / 8, 64LL}));
    const long long per = (chunks + S - 1) / S;
    p.seg = int(std::max(1LL, per) * kChunk);
    p.S = int(std::max(1LL, per ? (chunks + per - 1) / per : 1));
    const size_t rows = size_t(s.B) * s.D, all = rows * s.N;
    p.states = 4 * size_t(chunks) * units * p.width * (4 * p.per_lane * p.waves);
    if (p.S > 1) p.scratch += 4 * size_t(p.S) * (all + rows);
    if (backward) {
        p.scratch += 4 * size_t(p.tiles) * s.B * s.T * s.G * 2 * (4 * p.per_lane * p.waves);
        p.scratch += 4 * size_t(p.S) * (all + 2 * rows);
    }
    return p;
}

hipError_t fwd(const sscan_shape& s, Args a, void* ws, hipStream_t st) {
    const Plan p = plan(s, false);
    a.S = p.S;
    a.seg = p.seg;
    a.tiles = p.tiles;
    a.seg_state = static_cast<float*>(ws);
    a.seg_sum = a.seg_state + size_t(p.S) * s.B * s.D * s.N;
    return with_form(s.dtype, p, [&](auto D, auto F) { return run_fwd<decltype(D), decltype(F)>(a, st); });
}

hipError_t step(int dtype, const StepArgs& a, hipStream_t st) {
    switch (dtype) {
        case GSCAN_F32: return run_step<F32>(a, st);
        case GSCAN_F16: return run_step<F16>(a, st);
        default: return run_step<BF16>(a, st);
    }
}

}  // namespace ssc

// Backward pass of the selective scan (include/sscan.h).
//
// A workgroup takes its channels of a sequence (or of a segment of it) from the last
// chunk of positions to the first.  In a chunk it forms the states again from the
// saved one, keeps those of 16 positions (8 where a lane has 4 states) in
// registers, and runs the gradient back over them.
//
// The vector ALU bounds it, at two wavefronts on a SIMD: 499 plain instructions, 248
// with a DPP modifier, 42 transcendental and 36 lane exchanges for a chunk of 128
// states to a wavefront, 3290 cycles by what each takes (sscan_math.h).
// 16 states, 8 sequences of 4096 positions of 2048 channels, bf16: 1.02 ms, of which
// that is 0.70, and 26 us for the sums of db and dc over workgroups; one workgroup of
// eight wavefronts to a compute unit is all there is in this case.  21 states in 3
// groups, 24 x 1000 x 999, fp16, ragged: 515 and 25 us; its workgroups of six
// wavefronts take 202 registers a lane, of which two do not fit a compute unit.  Three
// wavefronts, with registers in memory: 890 for 520 there; states of 8 positions at a
// time: 1189 for 1084 in the other case; 4 states to a lane: 1198.  With 33 to 64
// states, 4 to a lane, 16 to 77 registers are spilled: 48 states 6.3 ms, 64 4.0 ms for
// the 2.0 of 32.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "close_sums.h"
#include "sscan_math.h"

namespace ssc {
namespace {

constexpr std::true_type whole{};   // of tiles that have all their positions
constexpr std::false_type some{};
constexpr int kPad2 = 18;          // float2s between two channels in LDS: no bank conflicts
constexpr int kPad4 = kChunk + 1;  // and float4s

__device__ __forceinline__ float dsilu(float z, float k) { return k * fmaf(z, 1.f - k, 1.f); }

// What a segment makes of a gradient that comes from behind it, r = exp(delta A) g
// of its first position, from zero; and its sum of delta.
template <class D, class F, bool GATE>
__global__ __launch_bounds__(F::kThreads) void k_back(Args a) {
    using S = typename D::S;
    constexpr int NP = F::NP, NB = F::NB, kSlots = F::kSlots;
    __shared__ float2 staged[2][F::kChannels * kPad2];
    const Lane<F> l(a);
    if (l.t_lo >= l.t_hi || l.s == 0) return;  // nothing comes before the first segment
    const int first_t = l.io_base + l.io_row;
    const bool last_slot = l.last_slot;
    const int t_last = l.t_lo + (l.t_hi - 1 - l.t_lo) / kChunk * kChunk;
    auto wide = [&](const void* p, long long sb, long long sr) {
        return Rows<S>(p, sb, sr, l.seq, t_last + l.io_base, l.d0, l.io_row, l.io_ch);
    };
    Rows<S> dt_ = wide(a.dt, a.dt_sb, a.dt_sr), z_ = wide(a.z, a.z_sb, a.z_sr), dy_ = wide(a.dy, a.dy_sb, a.dy_sr);
    Rows<S> c_(a.c, a.c_sb, a.c_sr, l.seq, t_last, l.group * a.N, l.i, 0);
    float r[NP] = {}, sum = 0.f, cs[NP];
    Column<D, F> dt, dy, z;
    States<D, NP> c;
    auto load = [&](auto full, int n) {
        if constexpr (full) {
            dt.load(dt_, last_slot);
            dy.load(dy_, last_slot);
            if constexpr (GATE) z.load(z_, last_slot);
            c.load(c_.at(0), l);
        } else {
            dt.load_some(dt_, last_slot, n - first_t);
            dy.load_some(dy_, last_slot, n - first_t);
            if constexpr (GATE) z.load_some(z_, last_slot, n - first_t);
            c.clear();
            if (l.i < n) c.load(c_.at(0), l);
        }
        dt_.move(-kChunk);
        dy_.move(-kChunk);
        if constexpr (GATE) z_.move(-kChunk);
        c_.move(-kChunk);
    };
    auto stage = [&](auto full, float2* to, int n) {
#pragma unroll
        for (int j = 0; j < NP; ++j) {
            cs[j] = c[j];
            now(cs[j]);
        }
#pragma unroll
        for (int q = 0; q < kSlots; ++q) {
            if ((q + 1) * F::kStep > 16 && !last_slot) continue;
            const int t = first_t + F::kStep * q;
            const bool valid = full || t < n;
            const float delta = valid ? softplus(dt[q] + l.bias).delta : 0.f;
            float ds = dy[q];
            if constexpr (GATE) ds *= z[q] * sig(z[q]);
            sum += delta;
            to[l.io_at * kPad2 + t] = make_float2(delta, valid ? ds : 0.f);
        }
    };
    int half = 0;
    // full: two more chunks come before this one
    auto turn = [&](auto full, int t0) {
        const float2* const mine = staged[half] + (l.ct * 16 + l.i) * kPad2;
        float2 m[16];
        unroll<4>([&](auto K) {
            constexpr int k = 3 - K;
            float e[4][NP];
            unroll<4>([&](auto L) {
                constexpr int q = 4 * k + L;
                m[q] = mine[q];
#pragma unroll
                for (int j = 0; j < NP; ++j) e[L][j] = decay(m[q].x, l.a2[j]);
            });
            unroll<4>([&](auto L) {
                constexpr int q = 3 - L;
                add_bcast<4 * k + q>(r, cs, m[4 * k + q].y);
#pragma unroll
                for (int j = 0; j < NP; ++j) r[j] *= e[q][j];
            });
        });
        if (full || t0 > l.t_lo) stage(whole, staged[half ^ 1], kChunk);
        if (full || t0 > l.t_lo + kChunk) load(whole, kChunk);
        lds_barrier();
        half ^= 1;
    };
    load(some, l.t_hi - t_last);
    stage(some, staged[0], l.t_hi - t_last);
    if (t_last > l.t_lo) load(whole, kChunk);
    lds_barrier();
    loads_done();
    int t0 = t_last;
    for (; t0 > l.t_lo + kChunk; t0 -= kChunk) turn(whole, t0);
    for (; t0 >= l.t_lo; t0 -= kChunk) turn(some, t0);
#pragma unroll
    for (int j = 0; j < NP; ++j) a.seg_state[l.s * l.all + l.states_at + l.at[j]] = r[j];
    const float total = over_channel<F>(sum, reinterpret_cast<float*>(staged));
    if (threadIdx.x < F::kChannels) a.seg_sum[((long long)l.s * a.B + l.seq) * a.D + l.io_d] = total;
}

template <class D, class F, bool GATE>
__global__ __launch_bounds__(F::kThreads) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_bwd(Args a) {
    using S = typename D::S;
    constexpr int NP = F::NP, NB = F::NB, kSlots = F::kSlots;
    // positions whose states are in registers
    constexpr int kSub = NP <= 2 ? 16 : 8, kSubs = 16 / kSub;
    constexpr int kWidth = F::kStates + 1;
    __shared__ float4 staged[F::kChannels * kPad4];         // delta, u, ds
    __shared__ float parts[3][NB][16 * F::kChannels];       // sums over states: of g b, A q and c h
    __shared__ float2 bc[F::CT][kChunk * kWidth];           // sums over 16 channels: of db and dc
    const Lane<F> l(a);
    const int first_t = l.io_base + l.io_row;  // the thread's first position of a chunk
    const bool last_slot = l.last_slot;
    if (max(l.n, l.t_lo) < l.t_end) {  // zeros behind the sequence
        S* const x0 = (S*)a.dx + l.seq * a.dx_sb + l.io_d;
        S* const t0 = (S*)a.ddt + l.seq * a.ddt_sb + l.io_d;
        S* const z0 = (S*)a.dz + l.seq * a.dz_sb + l.io_d;
        for (int t = max(l.n, l.t_lo) + first_t; t < l.t_end; t += F::kStep) {
            gsc::store_one<D>(x0 + t * a.dx_sr, 0.f);
            gsc::store_one<D>(t0 + t * a.ddt_sr, 0.f);
            if constexpr (GATE) gsc::store_one<D>(z0 + t * a.dz_sr, 0.f);
        }
    }

    const bool io_there = l.io_ch == l.io_at;
    float r[NP];  // exp(delta A) g of the position behind
    // the sum over positions of delta q, of a chunk and, with what its additions lost, of all
    float da[NP], da_all[NP] = {}, da_lost[NP] = {};
    const bool any = l.t_lo < l.t_hi;
#pragma unroll
    for (int j = 0; j < NP; ++j)
        r[j] = a.dh_last && l.there[j] && l.live && (any || l.s == 0) ? a.dh_last[l.states_at + l.at[j]] : 0.f;
    if (any) {
        // the segments behind, from the last one that has positions
        for (int k = (l.n - 1) / a.seg; k > l.s; --k) {
            const float sum = a.seg_sum[((long long)k * a.B + l.seq) * a.D + l.d];
#pragma unroll
            for (int j = 0; j < NP; ++j) {
                const float own = a.seg_state[k * l.all + l.states_at + l.at[j]];
                r[j] = l.there[j] && l.live ? fmaf(exp2_hw(sum * l.a2[j]), r[j], own) : 0.f;
            }
        }
    }
    const float skip = a.d ? a.d[l.io_d] : 0.f;
    float dd = 0.f, dbias = 0.f;
    const float4* const mine = staged + (l.ct * 16 + l.i) * kPad4;
    const int quad = l.i & 3;
    const int last = any ? (l.t_hi - 1) / kChunk : -1, first = l.t_lo / kChunk, t_last = max(last, 0) * kChunk;
    auto wide = [&](const void* p, long long sb, long long sr) {
        return Rows<S>(p, sb, sr, l.seq, t_last + l.io_base, l.d0, l.io_row, l.io_ch);
    };
    Rows<S> x_ = wide(a.x, a.x_sb, a.x_sr), dt_ = wide(a.dt, a.dt_sb, a.dt_sr), dy_ = wide(a.dy, a.dy_sb, a.dy_sr);
    Rows<S> z_ = wide(a.z, a.z_sb, a.z_sr), dx_ = wide(a.dx, a.dx_sb, a.dx_sr), ddt_ = wide(a.ddt, a.ddt_sb, a.ddt_sr);
    Rows<S> dz_ = wide(a.dz, a.dz_sb, a.dz_sr);
    Rows<S> b_(a.b, a.b_sb, a.b_sr, l.seq, t_last, l.group * a.N, l.i, 0), c_(a.c, a.c_sb, a.c_sr, l.seq, t_last, l.group * a.N, l.i, 0);
    const float* states_ = a.states + saved_at(a, l, max(last, 0));
    const long long states_step = saved_at(a, l, 1) - saved_at(a, l, 0);
    const long long width = 2LL * a.G * F::kStates;
    float* part_ = a.part_bc + (((long long)l.tile * a.B + l.seq) * a.T + t_last) * width + 2LL * l.group * F::kStates;

    // What is read of a chunk, of n positions (`full`: all 16).
    Column<D, F> x, dt, dy, z;
    float saved[NP];
    States<D, NP> raw_b, raw_c;
    auto load = [&](auto full, int n) {
        if constexpr (full) {
            x.load(x_, last_slot);
            dt.load(dt_, last_slot);
            dy.load(dy_, last_slot);
            if constexpr (GATE) z.load(z_, last_slot);
            raw_b.load(b_.at(0), l);
            raw_c.load(c_.at(0), l);
        } else {
            x.load_some(x_, last_slot, n - first_t);
            dt.load_some(dt_, last_slot, n - first_t);
            dy.load_some(dy_, last_slot, n - first_t);
            if constexpr (GATE) z.load_some(z_, last_slot, n - first_t);
            raw_b.clear();
            raw_c.clear();
            if (l.i < n) {
                raw_b.load(b_.at(0), l);
                raw_c.load(c_.at(0), l);
            }
        }
#pragma unroll
        for (int j = 0; j < NP; ++j) saved[j] = __builtin_nontemporal_load(states_ + 64 * j);
        x_.move(-kChunk);
        dt_.move(-kChunk);
        dy_.move(-kChunk);
        if constexpr (GATE) z_.move(-kChunk);
        b_.move(-kChunk);
        c_.move(-kChunk);
        states_ -= states_step;
    };
    // One chunk's turn.  full: it is whole and another comes before it, so that what is in flight
    // at each point is known, and nothing is waited for before it is used.
    auto turn = [&](auto full, int n, bool more) {
        float start[kSubs][NP], b[NP], c[NP];
#pragma unroll
        for (int j = 0; j < NP; ++j) {
            da[j] = 0.f;
            start[0][j] = saved[j];
            b[j] = raw_b[j];
            c[j] = l.there[j] ? raw_c[j] : 0.f;
            now(start[0][j]);
            now(b[j]);
            now(c[j]);
        }
        // the lane's own elements; the others' part of them goes to LDS
        float xs[kSlots], slope[kSlots], delta[kSlots], ds[kSlots], dzf[kSlots];
#pragma unroll
        for (int q = 0; q < kSlots; ++q) {
            if ((q + 1) * F::kStep > 16 && !last_slot) continue;
            const int t = first_t + F::kStep * q;
            const bool valid = full || t < n;
            const Step v = softplus(dt[q] + l.bias);
            xs[q] = x[q];
            now(xs[q]);
            slope[q] = v.slope;
            delta[q] = valid ? v.delta : 0.f;
            ds[q] = dy[q];
            if constexpr (GATE) {
                const float way = sig(z[q]);
                ds[q] = dy[q] * (z[q] * way);
                dzf[q] = dy[q] * dsilu(z[q], way);
                now(dzf[q]);
            }
            ds[q] = valid ? ds[q] : 0.f;
            now(ds[q]);
            // a channel that is not there counts for nothing in sums over channels
            staged[l.io_at * kPad4 + t] = make_float4(delta[q], valid && io_there ? delta[q] * xs[q] : 0.f, io_there ? ds[q] : 0.f, 0.f);
        }
        __builtin_amdgcn_sched_barrier(0);
        if (full || more) load(whole, kChunk);
        __builtin_amdgcn_sched_barrier(0);
        lds_barrier();
        // the states that the pieces start from
        unroll<kSubs - 1>([&](auto Q) {
            constexpr int q = Q;
#pragma unroll
            for (int j = 0; j < NP; ++j) start[q + 1][j] = start[q][j];
            unroll<kSub>([&](auto K) {
                constexpr int t = q * kSub + K;
                const float4 m = mine[t];
#pragma unroll
                for (int j = 0; j < NP; ++j)
                    start[q + 1][j] = fmaf(decay(m.x, l.a2[j]), start[q + 1][j], bcast<t>(b[j]) * m.y);
            });
        });
        unroll<kSubs>([&](auto Q) {
            constexpr int q = kSubs - 1 - Q;
            float e[kSub][NP], before[kSub + 1][NP];
#pragma unroll
            for (int j = 0; j < NP; ++j) before[0][j] = start[q][j];
            unroll<kSub / 4>([&](auto V) {
                constexpr int four = V;
                float part[4];
                unroll<4>([&](auto L) {
                    constexpr int k = 4 * four + L, t = q * kSub + k;
                    const float4 m = mine[t];
#pragma unroll
                    for (int j = 0; j < NP; ++j) {
                        e[k][j] = decay(m.x, l.a2[j]);
                        before[k + 1][j] = fmaf(e[k][j], before[k][j], bcast<t>(b[j]) * m.y);
                    }
                    if constexpr (GATE) part[L] = sum_bcast<t>(c, before[k + 1]);
                });
                if constexpr (GATE)
                    parts[2][l.nb][(q * kSub + 4 * four + l.row) * F::kChannels + l.ct * 16 + l.i] = sum_rows(part[0], part[1], part[2], part[3]);
                __builtin_amdgcn_sched_barrier(0);  // keeps registers few
            });
            unroll<kSub / 4>([&](auto V) {
                constexpr int four = kSub / 4 - 1 - V, t4 = q * kSub + 4 * four;
                asm volatile("" ::: "memory");  // the positions' values are read again, not kept in registers
                float gb[4], qa[4] = {}, pb[4][NP], pc[4][NP];
                unroll<4>([&](auto L) {
                    constexpr int w = 3 - L, k = 4 * four + w, t = q * kSub + k;
                    const float4 m = mine[t];
                    add_bcast<t>(r, c, m.z);  // r is g now
                    gb[w] = sum_bcast<t>(b, r);
#pragma unroll
                    for (int j = 0; j < NP; ++j) {
                        pb[w][j] = r[j] * m.y;
                        pc[w][j] = before[k + 1][j] * m.z;
                        r[j] *= e[k][j];
                        const float v = r[j] * before[k][j];
                        da[j] = fmaf(v, m.x, da[j]);
                        qa[w] = fmaf(v, l.a2[j], qa[w]);
                    }
                });
                const int at = (t4 + l.row) * F::kChannels + l.ct * 16 + l.i;
                parts[0][l.nb][at] = sum_rows(gb[0], gb[1], gb[2], gb[3]);
                parts[1][l.nb][at] = sum_rows(qa[0], qa[1], qa[2], qa[3]);
                // lane 4 k + q has position k's sums, the same as its three neighbours, of which
                // it writes the q-th
#pragma unroll
                for (int j = 0; j < NP; ++j)
                    sum_lanes(pb[0][j], pb[1][j], pb[2][j], pb[3][j], pc[0][j], pc[1][j], pc[2][j], pc[3][j]);
                float2 v = make_float2(pb[0][0], pc[0][0]);
#pragma unroll
                for (int k = 1; k < NP; ++k)
                    if (quad == k) v = make_float2(pb[0][k], pc[0][k]);
                if (quad < NP) bc[l.ct][(t4 + (l.i >> 2)) * kWidth + (l.nb * 4 + l.row) * NP + quad] = v;
                __builtin_amdgcn_sched_barrier(0);
            });
        });
#pragma unroll
        for (int j = 0; j < NP; ++j) {
            const float v = da[j] - da_lost[j], sum = da_all[j] + v;
            da_lost[j] = (sum - da_all[j]) - v;
            da_all[j] = sum;
        }
        lds_barrier();
        // the workgroup's sums of b's and c's gradients
        constexpr int kSums = kChunk * F::kStates * 2;
#pragma unroll
        for (int first_k = 0; first_k < kSums; first_k += F::kThreads) {
            const int k = first_k + threadIdx.x, m = k % F::kStates, which = k / F::kStates % 2, t = k / (2 * F::kStates);
            if (kSums % F::kThreads && k >= kSums) continue;
            const float* const from = reinterpret_cast<const float*>(&bc[0][t * kWidth + m]) + which;
            float v = from[0];
#pragma unroll
            for (int w = 1; w < F::CT; ++w) v += from[w * 2 * kChunk * kWidth];
            if (full || t < n) part_[t * width + which * F::kStates + m] = v;
        }
        part_ -= kChunk * width;
#pragma unroll
        for (int q = 0; q < kSlots; ++q) {
            if ((q + 1) * F::kStep > 16 && !last_slot) continue;
            const int t = first_t + F::kStep * q, at = t * F::kChannels + l.io_ch;
            float gb = parts[0][0][at], qa = parts[1][0][at], ch = GATE ? parts[2][0][at] : 0.f;
#pragma unroll
            for (int k = 1; k < NB; ++k) {
                gb += parts[0][k][at];
                qa += parts[1][k][at];
                if constexpr (GATE) ch += parts[2][k][at];
            }
            if (full || t < n) {
                const float ddv = fmaf(xs[q], gb, kLn2 * qa) * slope[q];
                gsc::store_one<D>(dx_.to(F::kStep * q), fmaf(skip, ds[q], delta[q] * gb));
                gsc::store_one<D>(ddt_.to(F::kStep * q), ddv);
                if constexpr (GATE) gsc::store_one<D>(dz_.to(F::kStep * q), dzf[q] * fmaf(skip, xs[q], ch));
                dd = fmaf(ds[q], xs[q], dd);
                dbias += ddv;
            }
        }
        dx_.move(-kChunk);
        ddt_.move(-kChunk);
        if constexpr (GATE) dz_.move(-kChunk);
    };
    if (any) {
        load(some, l.t_hi - t_last);
        turn(some, l.t_hi - t_last, last > first);
        loads_done();
        for (int chunk = last - 1; chunk > first; --chunk) turn(whole, kChunk, true);
        if (last > first) turn(some, kChunk, false);
    }
    // sums over positions
    const long long at = ((long long)l.seq * a.S + l.s) * a.D;
    const float sd = over_channel<F>(dd, reinterpret_cast<float*>(staged));
    const float sbias = over_channel<F>(dbias, reinterpret_cast<float*>(staged));
    if (threadIdx.x < F::kChannels) {
        a.part_d[at + l.io_d] = sd;
        a.part_bias[at + l.io_d] = sbias;
    }
    if (!l.live) return;
#pragma unroll
    for (int j = 0; j < NP; ++j)
        if (l.there[j]) {
            a.part_a[(at + l.d) * a.N + l.at[j]] = da_all[j] * (kLn2 * l.a2[j]);
            if (l.s == 0 && a.dh0) a.dh0[l.states_at + l.at[j]] = r[j];
        }
}

// db and dc from the partial sums of the workgroups along the channels, in order; the
// sums have `states` places for N.
template <class D>
__global__ __launch_bounds__(256) void k_close_bc(Args a, int states) {
    using S = typename D::S;
    const int width = 2 * a.G * states;
    const long long count = (long long)a.B * a.T * width;
    for (long long k = (long long)blockIdx.x * 256 + threadIdx.x; k < count; k += 256LL * gridDim.x) {
        const long long row = k / width;
        const int at = int(k % width), seq = int(row / a.T), t = int(row % a.T);
        const int group = at / (2 * states), which = at / states % 2, m = at % states;
        if (m >= a.N) continue;
        float v[4] = {};
        if (!a.lengths || t < a.lengths[seq]) {
            const float* const from = a.part_bc + k;
            int j = 0;
            for (; j + 3 < a.tiles; j += 4)
#pragma unroll
                for (int q = 0; q < 4; ++q) v[q] += from[(j + q) * count];
            for (; j < a.tiles; ++j) v[0] += from[j * count];
        }
        S* const to = which ? (S*)a.dc + seq * a.dc_sb + t * a.dc_sr : (S*)a.db + seq * a.db_sb + t * a.db_sr;
        gsc::store_one<D>(to + group * a.N + m, (v[0] + v[1]) + (v[2] + v[3]));
    }
}

// The parameters' gradients from P partial sums each.
hipError_t close_par(const Args& a, long long P, hipStream_t st) {
    return calls::close_sums<3>(P, st, {a.part_a, (long long)a.D * a.N, a.da_log}, {a.part_d, a.D, a.dd},
                                {a.part_bias, a.D, a.ddt_bias});
}

template <class D, class F>
hipError_t run_bwd(const Args& a, hipStream_t st) {
    const unsigned units = unsigned(a.G) * a.tiles * a.B * a.S;
    if (units == 0) {  // no channels: the sums over them are zero
    } else if (a.z) {
        if (a.S > 1) k_back<D, F, true><<<units, F::kThreads, 0, st>>>(a);
        k_bwd<D, F, true><<<units, F::kThreads, 0, st>>>(a);
    } else {
        if (a.S > 1) k_back<D, F, false><<<units, F::kThreads, 0, st>>>(a);
        k_bwd<D, F, false><<<units, F::kThreads, 0, st>>>(a);
    }
    const long long count = (long long)a.B * a.T * 2 * a.G * F::kStates;
    const long long blocks = std::min((count + 255) / 256, 1LL << 16);
    if (blocks) k_close_bc<D><<<unsigned(blocks), 256, 0, st>>>(a, F::kStates);
    return close_par(a, (long long)a.B * a.S, st);
}

}  // namespace

hipError_t bwd_empty(const sscan_shape&, const Args& a, hipStream_t st) { return close_par(a, 0, st); }

hipError_t bwd(const sscan_shape& s, Args a, void* ws, hipStream_t st) {
    const Plan p = plan(s, true);
    a.S = p.S;
    a.seg = p.seg;
    a.tiles = p.tiles;
    const size_t rows = size_t(s.B) * s.D, all = rows * s.N;
    float* at = static_cast<float*>(ws);
    a.part_a = at;
    at += p.S * all;
    a.part_d = at;
    at += p.S * rows;
    a.part_bias = at;
    at += p.S * rows;
    a.part_bc = at;
    at += size_t(a.tiles) * s.B * s.T * s.G * 2 * (4 * p.per_lane * p.waves);
    a.seg_state = at;
    a.seg_sum = at + p.S * all;
    return with_form(s.dtype, p, [&](auto D, auto F) { return run_bwd<decltype(D), decltype(F)>(a, st); });
}

}  // namespace ssc

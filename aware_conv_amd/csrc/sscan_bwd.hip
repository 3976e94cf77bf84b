// Backward pass of the selective scan (include/sscan.h).
//
// A workgroup takes 64 channels of a sequence (or of a segment of it), a
// wavefront 16 of them, from the last chunk of positions to the first.  In a
// chunk it forms the states again from the saved one, keeps those of up to 64 / NP
// positions in registers, and runs the gradient back over them.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "sscan_math.h"

namespace ssc {
namespace {

constexpr int kWaves = 4;

template <int NP>
struct Form {
    static constexpr int kChunk = NP == 16 ? 16 : 32;         // positions between saved states
    static constexpr int kTiles = kChunk / 16;
    static constexpr int kSub = NP <= 4 ? 16 : 64 / NP;       // positions whose states are in registers
    static constexpr int kSubs = kChunk / kSub;
    static constexpr int kOwn = kChunk / 4;                   // positions that a lane reads and writes
    static constexpr int kRow = kChunk + 1;                   // float4s between two channels in LDS
    static constexpr int kStates = 4 * NP;
};

// The sum of v over the 16 lanes of a row, in every lane.
__device__ __forceinline__ float row_sum(float v) {
    auto dpp = [](float x, auto ctrl) {
        return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), decltype(ctrl)::value,
                                                                  0xf, 0xf, true));
    };
    v += dpp(v, std::integral_constant<int, 0x128>{});  // row_ror:8
    v += dpp(v, std::integral_constant<int, 0x124>{});  // row_ror:4
    v += dpp(v, std::integral_constant<int, 0x122>{});
    v += dpp(v, std::integral_constant<int, 0x121>{});
    return v;
}

// Addresses of one lane's channel, and the parameters of its states.
template <class D, int NP>
struct Lane {
    using S = typename D::S;
    int row, i, seq, s, group, d, n, t_lo, t_end, t_hi;
    bool live, whole;
    long long states_at, all;
    const S *x, *dt, *z, *dy, *b, *c;
    float a2[NP], bias;
    bool there[NP];
    __device__ __forceinline__ Lane(const Args& a, int lane, int wave, int unit) {
        row = lane >> 4;
        i = lane & 15;
        const int tiles = a.G * a.tiles, tile = unit % tiles, rest = unit / tiles;
        seq = rest / a.S;
        s = rest % a.S;
        group = tile / a.tiles;
        const int c0 = (tile % a.tiles) * 64 + wave * 16;
        live = c0 + i < a.Dg;
        d = group * a.Dg + min(c0 + i, a.Dg - 1);
        n = a.lengths ? min(max(a.lengths[seq], 0), a.T) : a.T;
        t_lo = s * a.seg;
        t_end = min(a.T - t_lo, a.seg) + t_lo;
        t_hi = min(t_end, n);
        whole = a.N == 4 * NP;
        states_at = ((long long)seq * a.D + d) * a.N;
        all = (long long)a.B * a.D * a.N;
        x = (const S*)a.x + seq * a.x_sb + d;
        dt = (const S*)a.dt + seq * a.dt_sb + d;
        z = (const S*)a.z + seq * a.z_sb + d;
        dy = (const S*)a.dy + seq * a.dy_sb + d;
        b = (const S*)a.b + seq * a.b_sb + group * a.N;
        c = (const S*)a.c + seq * a.c_sb + group * a.N;
        bias = a.dt_bias ? a.dt_bias[d] : 0.f;
#pragma unroll
        for (int j = 0; j < NP; ++j) {
            const int m = row * NP + j;
            there[j] = m < a.N;
            a2[j] = there[j] ? -kLog2e * expf(a.a_log[(long long)d * a.N + min(m, a.N - 1)]) : 0.f;
        }
    }
};

__device__ __forceinline__ float dsilu(float z, float k) { return k * fmaf(z, 1.f - k, 1.f); }

// What a segment makes of a gradient that comes from behind it, r = exp(delta A) g
// of its first position, from zero; and its sum of delta.
template <class D, int NP, bool GATE>
__global__ __launch_bounds__(64 * kWaves) void k_back(Args a) {
    __shared__ float2 lds[kWaves][16 * 18];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const Lane<D, NP> l(a, lane, wave, blockIdx.x);
    if (l.t_lo >= l.t_hi || l.s == 0) return;  // nothing comes before the first segment
    float2* const mine = lds[wave] + l.i * 18;
    float r[NP] = {}, sum = 0.f;
    for (int t0 = l.t_lo + (l.t_hi - 1 - l.t_lo) / 16 * 16; t0 >= l.t_lo; t0 -= 16) {
        float c[NP];
        const long long tc = min(t0 + l.i, l.n - 1);
        load_states<D, NP>(c, l.c + tc * a.c_sr, l.row * NP, a.N, l.whole, t0 + l.i < l.t_hi);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const bool valid = t0 + 4 * k + l.row < l.t_hi && l.live;
            const long long t = min(t0 + 4 * k + l.row, l.n - 1);
            const float delta = valid ? softplus(gsc::load_one<D>(l.dt + t * a.dt_sr) + l.bias).delta : 0.f;
            float ds = valid ? gsc::load_one<D>(l.dy + t * a.dy_sr) : 0.f;
            if constexpr (GATE) {
                const float z = gsc::load_one<D>(l.z + t * a.z_sr);
                ds = valid ? ds * (z * sig(z)) : 0.f;
            }
            sum += delta;
            mine[4 * k + l.row] = make_float2(delta, ds);
        }
        wave_sync();
        unroll<16>([&](auto K) {
            constexpr int k = 15 - K;
            const float2 q = mine[k];
#pragma unroll
            for (int j = 0; j < NP; ++j)
                r[j] = decay(q.x, l.a2[j]) * fmaf(bcast<k>(c[j]), q.y, r[j]);
        });
        wave_sync();
    }
    if (!l.live) return;
#pragma unroll
    for (int j = 0; j < NP; ++j)
        if (l.there[j]) a.seg_state[l.s * l.all + l.states_at + l.row * NP + j] = r[j];
    const float total = sum_rows(sum, sum, sum, sum);
    if (l.row == 0) a.seg_sum[((long long)l.s * a.B + l.seq) * a.D + l.d] = total;
}

template <class D, int NP, bool GATE>
__global__ __launch_bounds__(64 * kWaves) void k_bwd(Args a) {
    using S = typename D::S;
    using F = Form<NP>;
    __shared__ float4 lds[kWaves][16 * F::kRow];                // delta, u, ds, dy silu'(z)
    __shared__ float bc[kWaves][F::kChunk][2][F::kStates];       // sums of db and dc over 16 channels
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const Lane<D, NP> l(a, lane, wave, blockIdx.x);
    const int tile = (blockIdx.x % (a.G * a.tiles)) % a.tiles;
    S* const dx_ = (S*)a.dx + l.seq * a.dx_sb + l.d;
    S* const ddt_ = (S*)a.ddt + l.seq * a.ddt_sb + l.d;
    S* const dz_ = (S*)a.dz + l.seq * a.dz_sb + l.d;
    if (l.live)
        for (int t = max(l.n, l.t_lo) + l.row; t < l.t_end; t += 4) {
            gsc::store_one<D>(dx_ + t * a.dx_sr, 0.f);
            gsc::store_one<D>(ddt_ + t * a.ddt_sr, 0.f);
            if constexpr (GATE) gsc::store_one<D>(dz_ + t * a.dz_sr, 0.f);
        }

    float r[NP];  // exp(delta A) g of the position behind
    // the sum over positions of delta q, of a chunk and, with what its additions lost, of all
    float da[NP], da_all[NP] = {}, da_lost[NP] = {};
    const bool some = l.t_lo < l.t_hi;
#pragma unroll
    for (int j = 0; j < NP; ++j)
        r[j] = a.dh_last && l.there[j] && l.live && (some || l.s == 0)
                   ? a.dh_last[l.states_at + l.row * NP + j] : 0.f;
    if (some && l.live) {
        // the segments behind, from the last one that has positions
        for (int k = (l.n - 1) / a.seg; k > l.s; --k) {
            const float sum = a.seg_sum[((long long)k * a.B + l.seq) * a.D + l.d];
#pragma unroll
            for (int j = 0; j < NP; ++j) {
                const float own = a.seg_state[k * l.all + l.states_at + min(l.row * NP + j, a.N - 1)];
                r[j] = l.there[j] ? fmaf(exp2_hw(sum * l.a2[j]), r[j], own) : 0.f;
            }
        }
    }
    const float skip = a.d ? a.d[l.d] : 0.f;
    float dd = 0.f, dbias = 0.f;
    float4* const mine = lds[wave] + l.i * F::kRow;

    const int last = some ? (l.t_hi - 1) / F::kChunk : -1, first = l.t_lo / F::kChunk;
    for (int chunk = last; chunk >= first; --chunk) {
        const int t0 = chunk * F::kChunk;
        float h[NP];
#pragma unroll
        for (int j = 0; j < NP; ++j)
            da[j] = 0.f;
#pragma unroll
        for (int j = 0; j < NP; ++j)
            h[j] = l.there[j] ? a.states[chunk * l.all + l.states_at + min(l.row * NP + j, a.N - 1)] : 0.f;
        float b[F::kTiles][NP], c[F::kTiles][NP];
#pragma unroll
        for (int k = 0; k < F::kTiles; ++k) {
            const bool valid = t0 + 16 * k + l.i < l.t_hi;
            const long long t = min(t0 + 16 * k + l.i, l.n - 1);
            load_states<D, NP>(b[k], l.b + t * a.b_sr, l.row * NP, a.N, l.whole, valid);
            load_states<D, NP>(c[k], l.c + t * a.c_sr, l.row * NP, a.N, l.whole, valid);
        }
        float xs[F::kOwn], slope[F::kOwn];
#pragma unroll
        for (int k = 0; k < F::kOwn; ++k) {
            const bool valid = t0 + 4 * k + l.row < l.t_hi && l.live;
            const long long t = min(t0 + 4 * k + l.row, l.n - 1);
            xs[k] = gsc::load_one<D>(l.x + t * a.x_sr);
            const Step q = softplus(gsc::load_one<D>(l.dt + t * a.dt_sr) + l.bias);
            const float dy = gsc::load_one<D>(l.dy + t * a.dy_sr);
            float ds = dy, dzf = 0.f;
            if constexpr (GATE) {
                const float z = gsc::load_one<D>(l.z + t * a.z_sr), way = sig(z);
                ds = dy * (z * way);
                dzf = dy * dsilu(z, way);
            }
            slope[k] = q.slope;
            mine[4 * k + l.row] = valid ? make_float4(q.delta, q.delta * xs[k], ds, dzf)
                                        : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        wave_sync();
        // the states that the pieces start from
        float start[F::kSubs][NP];
        unroll<F::kSubs>([&](auto Q) {
            constexpr int q = Q;
#pragma unroll
            for (int j = 0; j < NP; ++j) start[q][j] = h[j];
            if constexpr (q + 1 < F::kSubs)
                unroll<F::kSub>([&](auto K) {
                    constexpr int t = q * F::kSub + K;
                    const float4 m = mine[t];
#pragma unroll
                    for (int j = 0; j < NP; ++j)
                        h[j] = fmaf(decay(m.x, l.a2[j]), h[j], bcast<t % 16>(b[t / 16][j]) * m.y);
                });
        });
        unroll<F::kSubs>([&](auto Q) {
            constexpr int q = F::kSubs - 1 - Q;
            float e[F::kSub][NP], before[F::kSub + 1][NP], part[F::kSub];
#pragma unroll
            for (int j = 0; j < NP; ++j) before[0][j] = start[q][j];
            unroll<F::kSub>([&](auto K) {
                constexpr int k = K, t = q * F::kSub + k;
                const float4 m = mine[t];
                part[k] = 0.f;
#pragma unroll
                for (int j = 0; j < NP; ++j) {
                    e[k][j] = decay(m.x, l.a2[j]);
                    before[k + 1][j] = fmaf(e[k][j], before[k][j], bcast<t % 16>(b[t / 16][j]) * m.y);
                    if constexpr (GATE) part[k] = fmaf(bcast<t % 16>(c[t / 16][j]), before[k + 1][j], part[k]);
                }
            });
            unroll<F::kSub / 4>([&](auto V) {
                constexpr int four = F::kSub / 4 - 1 - V;
                float gb[4] = {}, qa[4] = {};
                float pb[4][NP], pc[4][NP];
                unroll<4>([&](auto L) {
                    constexpr int w = 3 - L, k = 4 * four + w, t = q * F::kSub + k;
                    const float4 m = mine[t];
#pragma unroll
                    for (int j = 0; j < NP; ++j) {
                        const float g = fmaf(bcast<t % 16>(c[t / 16][j]), m.z, r[j]);
                        pb[w][j] = g * m.y;
                        pc[w][j] = before[k + 1][j] * m.z;
                        gb[w] = fmaf(bcast<t % 16>(b[t / 16][j]), g, gb[w]);
                        r[j] = g * e[k][j];
                        const float v = r[j] * before[k][j];
                        da[j] = fmaf(v, m.x, da[j]);
                        qa[w] = fmaf(v, l.a2[j], qa[w]);
                    }
                });
                constexpr int t4 = q * F::kSub + 4 * four, own = t4 / 4;
                unroll<4>([&](auto W) {
#pragma unroll
                    for (int j = 0; j < NP; ++j) {
                        const float sb = row_sum(pb[W][j]), sc = row_sum(pc[W][j]);
                        if (l.i == 0) {
                            bc[wave][t4 + W][0][l.row * NP + j] = sb;
                            bc[wave][t4 + W][1][l.row * NP + j] = sc;
                        }
                    }
                });
                const float wgb = sum_rows(gb[0], gb[1], gb[2], gb[3]);
                const float wqa = sum_rows(qa[0], qa[1], qa[2], qa[3]);
                const float4 m = mine[t4 + l.row];
                const int t = t0 + t4 + l.row;
                const float dxv = fmaf(skip, m.z, m.x * wgb);
                const float ddv = fmaf(xs[own], wgb, kLn2 * wqa) * slope[own];
                float dzv = 0.f;
                if constexpr (GATE) {
                    const float sums = sum_rows(part[4 * four], part[4 * four + 1], part[4 * four + 2], part[4 * four + 3]);
                    dzv = m.w * fmaf(skip, xs[own], sums);
                }
                if (t < l.t_hi && l.live) {
                    gsc::store_one<D>(dx_ + t * a.dx_sr, dxv);
                    gsc::store_one<D>(ddt_ + t * a.ddt_sr, ddv);
                    if constexpr (GATE) gsc::store_one<D>(dz_ + t * a.dz_sr, dzv);
                    dd = fmaf(m.z, xs[own], dd);
                    dbias += ddv;
                }
            });
        });
#pragma unroll
        for (int j = 0; j < NP; ++j) {
            const float v = da[j] - da_lost[j], sum = da_all[j] + v;
            da_lost[j] = (sum - da_all[j]) - v;
            da_all[j] = sum;
        }
        __syncthreads();
        // the four wavefronts' sums of b's and c's gradients
        const int rows = min(F::kChunk, l.t_hi - t0);
        const long long width = 2LL * a.G * a.N;
        float* const to = a.part_bc + (((long long)tile * a.B + l.seq) * a.T + t0) * width + 2LL * l.group * a.N;
        for (int k = threadIdx.x; k < F::kChunk * 2 * F::kStates; k += 64 * kWaves) {
            const int m = k % F::kStates, which = k / F::kStates % 2, t = k / F::kStates / 2;
            if (m >= a.N || t >= rows) continue;
            float v = bc[0][t][which][m];
            for (int w = 1; w < kWaves; ++w) v += bc[w][t][which][m];
            to[t * width + which * a.N + m] = v;
        }
        __syncthreads();
    }
    const long long at = ((long long)l.seq * a.S + l.s) * a.D + l.d;
    const float sd = sum_rows(dd, dd, dd, dd), sbias = sum_rows(dbias, dbias, dbias, dbias);
    if (!l.live) return;
#pragma unroll
    for (int j = 0; j < NP; ++j)
        if (l.there[j]) {
            a.part_a[at * a.N + l.row * NP + j] = da_all[j] * (kLn2 * l.a2[j]);
            if (l.s == 0 && a.dh0) a.dh0[l.states_at + l.row * NP + j] = r[j];
        }
    if (l.row == 0) {
        a.part_d[at] = sd;
        a.part_bias[at] = sbias;
    }
}

// db and dc from the partial sums of the tiles of 64 channels, in order.
template <class D>
__global__ __launch_bounds__(256) void k_close_bc(Args a) {
    using S = typename D::S;
    const int width = 2 * a.G * a.N;
    const long long count = (long long)a.B * a.T * width;
    for (long long k = (long long)blockIdx.x * 256 + threadIdx.x; k < count; k += 256LL * gridDim.x) {
        const long long row = k / width;
        const int at = int(k % width), seq = int(row / a.T), t = int(row % a.T);
        const int group = at / (2 * a.N), which = at / a.N % 2, m = at % a.N;
        float v = 0.f;
        if (!a.lengths || t < a.lengths[seq])
            for (int j = 0; j < a.tiles; ++j) v += a.part_bc[j * count + k];
        S* const to = which ? (S*)a.dc + seq * a.dc_sb + t * a.dc_sr : (S*)a.db + seq * a.db_sb + t * a.db_sr;
        gsc::store_one<D>(to + group * a.N + m, v);
    }
}

// The parameters' gradients from P partial sums each, added in order in fp64.
__global__ __launch_bounds__(256) void k_close_par(Args a, int P) {
    const long long k = (long long)blockIdx.x * 256 + threadIdx.x, na = (long long)a.D * a.N;
    if (k >= na + 2 * a.D) return;
    const bool of_a = k < na, of_d = !of_a && k - na < a.D;
    const float* const from = of_a ? a.part_a + k : of_d ? a.part_d + (k - na) : a.part_bias + (k - na - a.D);
    float* const to = of_a ? a.da_log + k : of_d ? a.dd + (k - na) : a.ddt_bias + (k - na - a.D);
    if (!of_a && !(of_d ? a.dd : a.ddt_bias)) return;
    const long long step = of_a ? na : a.D;
    double v = 0;
    for (int p = 0; p < P; ++p) v += from[p * step];
    *to = float(v);
}

hipError_t close_par(const Args& a, int P, hipStream_t st) {
    const long long n = (long long)a.D * a.N + 2LL * a.D;
    k_close_par<<<unsigned((n + 255) / 256), 256, 0, st>>>(a, P);
    return hipGetLastError();
}

template <class D, int NP>
hipError_t run_bwd(const Args& a, hipStream_t st) {
    const dim3 block(64 * kWaves);
    const unsigned units = unsigned(a.G) * a.tiles * a.B * a.S;
    if (a.z) {
        if (a.S > 1) k_back<D, NP, true><<<units, block, 0, st>>>(a);
        k_bwd<D, NP, true><<<units, block, 0, st>>>(a);
    } else {
        if (a.S > 1) k_back<D, NP, false><<<units, block, 0, st>>>(a);
        k_bwd<D, NP, false><<<units, block, 0, st>>>(a);
    }
    const long long count = (long long)a.B * a.T * 2 * a.G * a.N;
    const long long blocks = std::min((count + 255) / 256, 1LL << 16);
    if (blocks) k_close_bc<D><<<unsigned(blocks), 256, 0, st>>>(a);
    return close_par(a, a.B * a.S, st);
}
template <class D>
hipError_t run_bwd(const Args& a, int per_lane, hipStream_t st) {
    switch (per_lane) {
        case 1: return run_bwd<D, 1>(a, st);
        case 2: return run_bwd<D, 2>(a, st);
        case 4: return run_bwd<D, 4>(a, st);
        case 8: return run_bwd<D, 8>(a, st);
        default: return run_bwd<D, 16>(a, st);
    }
}

}  // namespace

hipError_t bwd_empty(const sscan_shape&, const Args& a, hipStream_t st) { return close_par(a, 0, st); }

hipError_t bwd(const sscan_shape& s, Args a, void* ws, hipStream_t st) {
    const Plan p = plan(s, true);
    a.S = p.S;
    a.seg = p.seg;
    const size_t rows = size_t(s.B) * s.D, all = rows * s.N;
    float* at = static_cast<float*>(ws);
    a.part_a = at;
    at += p.S * all;
    a.part_d = at;
    at += p.S * rows;
    a.part_bias = at;
    at += p.S * rows;
    a.part_bc = at;
    at += size_t(a.tiles) * s.B * s.T * s.G * 2 * s.N;
    a.seg_state = at;
    a.seg_sum = at + p.S * all;
    switch (s.dtype) {
        case GSCAN_F32: return run_bwd<F32>(a, p.per_lane, st);
        case GSCAN_F16: return run_bwd<F16>(a, p.per_lane, st);
        default: return run_bwd<BF16>(a, p.per_lane, st);
    }
}

}  // namespace ssc

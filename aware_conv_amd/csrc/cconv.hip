// Short causal depthwise convolution over token sequences (include/cconv.h).
//
// HBM bounds it: K multiplications per element.  A thread takes a few adjacent
// channels of a run of positions and walks along it with the last K - 1 inputs in
// registers, so that only the positions before a run are read twice, and those
// from the cache: runs that follow each other are in one workgroup.  Loads of
// several positions are under way at once, and what is written goes past the
// caches.  4 taps, 8 sequences of 4096 positions of 2048 channels, bf16: forwards
// 54 us (268 MB, 5.0 TB/s; a large copy reaches 4.9), backwards 92 us (403 MB,
// 4.4 TB/s) and 5 us for the parameters' sums; 3 taps, 24 x 1000 x 999, fp16, half
// of it padding: 36, 53 and 5 us, far from its bytes (71 MB read and written forwards,
// 104 backwards, by the memory's counters); fewer than 256 channels leave lanes
// idle: 64M elements of 128, 64, 16 channels 72, 120, 418 us forwards, 109, 171, 606
// backwards (of 1024: 54 and 95).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "cconv_internal.h"
#include "close_sums.h"
#include "gscan_math.h"

namespace ccv {
namespace {

using gsc::BF16;
using gsc::F16;
using gsc::F32;
using gsc::sig;

constexpr int kLanes = 32;  // threads along the channels
constexpr int kRuns = 8;    // runs of positions in a workgroup
constexpr int kRunF = 16;   // positions of a run, forwards
constexpr int kRunB = 32;   // and backwards

// V channels from p on, `left` of which exist; zero where not `there`.
template <class D, int V>
__device__ __forceinline__ void load(float (&out)[V], const typename D::S* p, int left, bool there) {
    gsc::Raw<D, V> q;
#pragma unroll
    for (int k = 0; k < gsc::Raw<D, V>::kWords; ++k) q.w[k] = 0;
    if (there) {
        if (left >= V) {
            gsc::load_vec<D, V>(q, p);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (j < left) q.set(j, gsc::load_one<D>(p + j));
        }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) out[j] = q.get(j);
}
template <class D, int V>
__device__ __forceinline__ void store(typename D::S* p, const float (&v)[V], int left) {
    if (left >= V) {
        gsc::store_vec_once<D, V>(p, gsc::pack<D, false>(v));
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (j < left) gsc::store_one<D>(p + j, v[j]);
    }
}

template <int V, int K>
__device__ __forceinline__ void load_taps(float (&w)[K][V], float (&bias)[V], const float* w_,
                                          const float* bias_, int c, int left) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int at = c + min(j, left - 1);
        bias[j] = bias_ ? bias_[at] : 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) w[k][j] = w_[(long long)at * K + k];
    }
}

// The inputs of a sequence, position -K + 1 on.
template <class D, int V>
struct Line {
    const typename D::S *x, *h0;
    long long sr;
    int K, C, n, left;
    __device__ __forceinline__ void get(float (&out)[V], int t) const {
        if (t >= 0) load<D, V>(out, x + t * sr, left, t < n);
        else load<D, V>(out, h0 + (long long)(t + K - 1) * C, left, h0 && t >= 1 - K);
    }
};
template <class D, int V>
__device__ __forceinline__ Line<D, V> line_of(const Args& a, int seq, int c, int n) {
    using S = typename D::S;
    return {(const S*)a.x + seq * a.x_sb + c,
            a.h0 ? (const S*)a.h0 + (long long)seq * (a.K - 1) * a.C + c : nullptr,
            a.x_sr, a.K, a.C, n, min(V, a.C - c)};
}

template <class D, int V, int K>
__global__ __launch_bounds__(kLanes * kRuns) void k_fwd(Args a) {
    using S = typename D::S;
    const int blocks_c = (a.C + kLanes * V - 1) / (kLanes * V);
    const int runs = max(1, (a.T + kRunF * kRuns - 1) / (kRunF * kRuns));
    const int cb = blockIdx.x % blocks_c, rest = blockIdx.x / blocks_c;
    const int seq = rest / runs, ty = threadIdx.x / kLanes;
    const int c = (cb * kLanes + threadIdx.x % kLanes) * V;
    if (c >= a.C) return;
    const int t0 = (rest % runs * kRuns + ty) * kRunF, t1 = min(a.T, t0 + kRunF);
    const int n = a.lengths ? min(max(a.lengths[seq], 0), a.T) : a.T;
    const Line<D, V> line = line_of<D, V>(a, seq, c, n);
    if (t0 == 0 && a.last) {
        S* const to = (S*)a.last + (long long)seq * (K - 1) * a.C + c;
        for (int j = 0; j < K - 1; ++j) {
            float v[V];
            line.get(v, n - (K - 1) + j);
            store<D, V>(to + (long long)j * a.C, v, line.left);
        }
    }
    float w[K][V], bias[V], win[K][V];
    load_taps(w, bias, a.w, a.bias, c, line.left);
#pragma unroll
    for (int k = 0; k < K - 1; ++k) line.get(win[k + 1], t0 - (K - 1) + k);
    S* const y = (S*)a.y + seq * a.y_sb + c;
    for (int t = t0; t < t1; t += 8) {
        float in[8][V];
#pragma unroll
        for (int i = 0; i < 8; ++i) load<D, V>(in[i], line.x + (long long)(t + i) * line.sr, line.left, t + i < n);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
#pragma unroll
            for (int k = 0; k < K - 1; ++k)
#pragma unroll
                for (int j = 0; j < V; ++j) win[k][j] = win[k + 1][j];
            float v[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                win[K - 1][j] = in[i][j];
                v[j] = bias[j];
#pragma unroll
                for (int k = 0; k < K; ++k) v[j] = fmaf(w[k][j], win[k][j], v[j]);
                if (a.silu) v[j] *= sig(v[j]);
                if (t + i >= n) v[j] = 0.f;
            }
            if (t + i < t1) store<D, V>(y + (long long)(t + i) * a.y_sr, v, line.left);
        }
    }
}

// Row i of [h0, x] receives d_i = sum_k w[k] dv[i - k], complete as soon as dv_i
// is known: a run walks along t, forms dv_t, and gives row t, which is position
// t - K + 1.  It goes on for K - 1 positions beyond its own.
template <class D, int V, int K>
__global__ __launch_bounds__(kLanes * kRuns) void k_bwd(Args a) {
    using S = typename D::S;
    __shared__ float lds[kRuns][kLanes * V];
    const int blocks_c = (a.C + kLanes * V - 1) / (kLanes * V);
    const int runs = max(1, (a.T + kRunB * kRuns - 1) / (kRunB * kRuns));
    const int cb = blockIdx.x % blocks_c, rest = blockIdx.x / blocks_c;
    const int seq = rest / runs, ty = threadIdx.x / kLanes, tx = threadIdx.x % kLanes;
    const int c = (cb * kLanes + tx) * V;
    const bool live = c < a.C;
    const int t0 = (rest % runs * kRuns + ty) * kRunB, t1 = min(a.T, t0 + kRunB);
    const int n = a.lengths ? min(max(a.lengths[seq], 0), a.T) : a.T;
    float dw[K][V] = {}, db[V] = {};
    if (live && (t0 < t1 || t0 == 0)) {
        const Line<D, V> line = line_of<D, V>(a, seq, c, n);
        const S* const dy = (const S*)a.dy + seq * a.dy_sb + c;
        S* const dx = (S*)a.dx + seq * a.dx_sb + c;
        const long long at0 = (long long)seq * (K - 1) * a.C + c;
        float w[K][V], bias[V], win[K][V], dv[K][V] = {};
        load_taps(w, bias, a.w, a.bias, c, line.left);
#pragma unroll
        for (int k = 0; k < K - 1; ++k) line.get(win[k + 1], t0 - (K - 1) + k);
        // positions up to here have a row to give: n - 1 is row n + K - 2
        const int end = min(t1, n) + K - 1;
        for (int t = t0; t < end; t += 4) {
            float in[4][V], g[4][V];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                load<D, V>(in[i], line.x + (long long)(t + i) * line.sr, line.left, t + i < n && t + i < end);
                load<D, V>(g[i], dy + (long long)(t + i) * a.dy_sr, line.left, t + i < n && t + i < end);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float out[V], tail[V] = {};
                const int behind = t + i - n, p = t + i - (K - 1);
                if (a.dlast && behind >= 0 && behind < K - 1)
                    load<D, V>(tail, (const S*)a.dlast + at0 + (long long)behind * a.C, line.left, true);
#pragma unroll
                for (int k = 0; k < K - 1; ++k)
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        win[k][j] = win[k + 1][j];
                        dv[k][j] = dv[k + 1][j];
                    }
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    win[K - 1][j] = in[i][j];
                    float v = bias[j];
#pragma unroll
                    for (int k = 0; k < K; ++k) v = fmaf(w[k][j], win[k][j], v);
                    const float s = sig(v);
                    dv[K - 1][j] = t + i < n ? (a.silu ? g[i][j] * (s * fmaf(v, 1.f - s, 1.f)) : g[i][j]) : 0.f;
                    if (t + i < t1) {
                        db[j] += dv[K - 1][j];
#pragma unroll
                        for (int k = 0; k < K; ++k) dw[k][j] = fmaf(dv[K - 1][j], win[k][j], dw[k][j]);
                    }
                    out[j] = tail[j];
#pragma unroll
                    for (int k = 0; k < K; ++k)
                        out[j] = fmaf(w[k][j], dv[K - 1 - k][j], out[j]);
                }
                if (t + i >= end) continue;
                if (p >= t0) store<D, V>(dx + (long long)p * a.dx_sr, out, line.left);
                else if (p < 0 && a.dh0) store<D, V>((S*)a.dh0 + at0 + (long long)(t + i) * a.C, out, line.left);
            }
        }
        const float zero[V] = {};
        for (int t = max(n, t0); t < t1; ++t) store<D, V>(dx + (long long)t * a.dx_sr, zero, line.left);
    }
    // the runs' sums of the parameters' gradients
    const long long part = rest, parts = (long long)a.B * runs;
    for (int k = 0; k <= K; ++k) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float v = db[j];
#pragma unroll
            for (int q = 0; q < K; ++q)
                if (q == k) v = dw[q][j];
            lds[ty][tx * V + j] = v;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < kLanes * V; i += kLanes * kRuns) {
            const int ch = cb * kLanes * V + i;
            if (ch >= a.C) continue;
            float v = lds[0][i];
            for (int q = 1; q < kRuns; ++q) v += lds[q][i];
            if (k < K) a.part[(part * a.C + ch) * K + k] = v;
            else a.part[parts * a.C * K + part * a.C + ch] = v;
        }
        __syncthreads();
    }
}

// One position: a thread moves a few channels of a cache row on.  The launch bounds
// it: 2.2 us for one sequence of 384 channels.
template <class D, int V, int K>
__global__ __launch_bounds__(256) void k_step(StepArgs a) {
    using S = typename D::S;
    const int per = (a.C + V - 1) / V;
    const long long at = (long long)blockIdx.x * 256 + threadIdx.x;
    if (at >= (long long)a.B * per) return;
    const int seq = int(at / per), c = int(at % per) * V, left = min(V, a.C - c);
    const int slot = a.slots ? a.slots[seq] : seq;
    S* const y = (S*)a.y + seq * a.y_sb + c;
    float v[V] = {};
    if (slot >= 0 && slot < a.S) {
        S* const row = (S*)a.cache + (long long)slot * (K - 1) * a.C + c;
        float w[K][V], in[K][V];
        load_taps(w, v, a.w, a.bias, c, left);
#pragma unroll
        for (int k = 0; k < K - 1; ++k) load<D, V>(in[k], row + (long long)k * a.C, left, true);
        load<D, V>(in[K - 1], (const S*)a.x + seq * a.x_sb + c, left, true);
#pragma unroll
        for (int j = 0; j < V; ++j) {
#pragma unroll
            for (int k = 0; k < K; ++k) v[j] = fmaf(w[k][j], in[k][j], v[j]);
            if (a.silu) v[j] *= sig(v[j]);
        }
#pragma unroll
        for (int k = 0; k < K - 1; ++k) store<D, V>(row + (long long)k * a.C, in[k + 1], left);
    }
    store<D, V>(y, v, left);
}

// f with the number of taps as a constant
template <class F>
hipError_t with_taps(int K, F&& f) {
    switch (K) {
        case 1: return f(std::integral_constant<int, 1>{});
        case 2: return f(std::integral_constant<int, 2>{});
        case 3: return f(std::integral_constant<int, 3>{});
        case 4: return f(std::integral_constant<int, 4>{});
        case 5: return f(std::integral_constant<int, 5>{});
        case 6: return f(std::integral_constant<int, 6>{});
        case 7: return f(std::integral_constant<int, 7>{});
        default: return f(std::integral_constant<int, 8>{});
    }
}
template <class F>
hipError_t with_type(int dtype, F&& f) {
    switch (dtype) {
        case GSCAN_F32: return f(F32{});
        case GSCAN_F16: return f(F16{});
        default: return f(BF16{});
    }
}

constexpr int kBack = 4;  // channels of a thread, backwards
long long parts_of(const cconv_shape& s) {
    return s.B * std::max(1LL, (s.T + kRunB * kRuns - 1LL) / (kRunB * kRuns));
}

}  // namespace

Plan plan(const cconv_shape& s) {
    Plan p{};
    p.parts = parts_of(s);
    p.scratch = 4 * size_t(p.parts) * s.C * (s.K + 1);
    p.fits = s.B * ((s.C + 127LL) / 128) * ((s.T + 127LL) / 128 + 1) < (1LL << 24);  // of 256 threads
    return p;
}

hipError_t fwd(int dtype, const Args& a, hipStream_t st) {
    return with_type(dtype, [&](auto D) {
        using T = decltype(D);
        constexpr int V = 16 / T::kBytes;
        const long long runs = std::max(1LL, (a.T + kRunF * kRuns - 1LL) / (kRunF * kRuns));
        const long long blocks = (long long)a.B * runs * ((a.C + kLanes * V - 1) / (kLanes * V));
        return with_taps(a.K, [&](auto K) {
            k_fwd<T, V, K><<<unsigned(blocks), kLanes * kRuns, 0, st>>>(a);
            return hipGetLastError();
        });
    });
}

hipError_t bwd(const cconv_shape& s, Args a, void* ws, hipStream_t st) {
    const long long parts = parts_of(s);
    a.part = static_cast<float*>(ws);
    if (parts) {
        const hipError_t e = with_type(s.dtype, [&](auto D) {
            using T = decltype(D);
            const long long blocks = parts * ((a.C + kLanes * kBack - 1) / (kLanes * kBack));
            return with_taps(a.K, [&](auto K) {
                k_bwd<T, kBack, K><<<unsigned(blocks), kLanes * kRuns, 0, st>>>(a);
                return hipGetLastError();
            });
        });
        if (e != hipSuccess) return e;
    }
    const long long nw = (long long)a.C * a.K;
    return calls::close_sums<1>(parts, st, {a.part, nw, a.dw}, {a.part + parts * nw, a.C, a.dbias});
}

hipError_t step(int dtype, const StepArgs& a, hipStream_t st) {
    return with_type(dtype, [&](auto D) {
        using T = decltype(D);
        constexpr int V = 4;
        const long long n = (long long)a.B * ((a.C + V - 1) / V);
        return with_taps(a.K, [&](auto K) {
            k_step<T, V, K><<<unsigned((n + 255) / 256), 256, 0, st>>>(a);
            return hipGetLastError();
        });
    });
}

}  // namespace ccv

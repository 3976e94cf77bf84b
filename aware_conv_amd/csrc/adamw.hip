// AdamW step over many tensors at once (include/adamw.h) and the global
// gradient norm.
//
// A launch takes a table of tensors by value in its kernel arguments (so
// nothing is copied or kept, and a captured launch keeps its own); a workgroup
// takes one chunk of one tensor.  The step is bound by HBM: it reads and
// writes each value once, 16 bytes per lane and access where the type allows.
// 94M elements in fp32: 504 to 512 us, 5.2 TB/s; 140M in bf16 with masters and
// 8-bit moments 403 to 416 us, 5.5 TB/s (a large copy reaches 4.94 TB/s).  Ninety
// tensors of 1.06M elements together take 10 us, mostly launch latency.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "adamw_internal.h"
#include "gscan_math.h"

namespace adw {
namespace {

using gsc::BF16;
using gsc::F16;
using gsc::F32;
using gsc::Raw;

constexpr int kThreads = 256;
constexpr int kVec = 4;                           // elements of a lane and access
constexpr int kUnits = 4;                         // accesses of a lane
constexpr int kChunk = kThreads * kVec * kUnits;  // elements of a workgroup

constexpr float kMax = 3.402823466e38f;  // the largest finite value

// P pointers for each of up to N tensors, and the chunks before each.
template <int P, int N>
struct Table {
    void* ptr[P][N];
    long long n[N];
    int first[N + 1];
    int count;
};
// as many tensors as 4 KiB of kernel arguments hold, less 96 bytes for the rest
template <int P>
constexpr int kFit = (4096 - 96) / (8 * P + 8 + 4);

// The tensor that holds chunk `blk`: the number of tensors after the first
// that start at it or before.  The lanes compare all starts at once; a binary
// search would wait for one kernel argument after the other (the step over 90
// tensors: 9.8 us, now 9.2).
template <int P, int N>
__device__ __forceinline__ int tensor_of(const Table<P, N>& t, int blk) {
    const int lane = threadIdx.x & 63;
    int id = 0;
#pragma unroll
    for (int k = 1; k < N; k += 64) {
        const int i = k + lane;
        id += __popcll(__ballot(i < t.count && t.first[i < N ? i : 0] <= blk));
    }
    return __builtin_amdgcn_readfirstlane(id);
}

template <class D>
__device__ __forceinline__ Raw<D, kVec> fetch(const typename D::S* p, int n) {
    Raw<D, kVec> q;
    if (n >= kVec) {
        gsc::load_vec<D, kVec>(q, p);
    } else {
#pragma unroll
        for (int k = 0; k < Raw<D, kVec>::kWords; ++k) q.w[k] = 0;
#pragma unroll
        for (int j = 0; j < kVec; ++j)
            if (j < n) q.set(j, gsc::load_one<D>(p + j));
    }
    return q;
}
template <class D>
__device__ __forceinline__ void put(typename D::S* p, const float (&v)[kVec], int n) {
    if (n >= kVec) {
        gsc::store_vec<D, kVec>(p, gsc::pack<D, false>(v));
    } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j)
            if (j < n) gsc::store_one<D>(p + j, v[j]);
    }
}

// Four codes in a word.
__device__ __forceinline__ uint32_t fetch_codes(const uint8_t* p, int n) {
    uint32_t w = 0;
    if (n >= kVec) {
        struct __attribute__((packed, aligned(1))) P { uint32_t w; };
        w = reinterpret_cast<const P*>(p)->w;
    } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j)
            if (j < n) w |= uint32_t(p[j]) << (8 * j);
    }
    return w;
}
__device__ __forceinline__ void put_codes(uint8_t* p, uint32_t w, int n) {
    if (n >= kVec) {
        struct __attribute__((packed, aligned(1))) P { uint32_t w; };
        reinterpret_cast<P*>(p)->w = w;
    } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j)
            if (j < n) p[j] = uint8_t(w >> (8 * j));
    }
}
__device__ __forceinline__ void decode(uint32_t w, float (&v)[kVec]) {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(int(w), false);
    const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(int(w), true);
    v[0] = lo[0];
    v[1] = lo[1];
    v[2] = hi[0];
    v[3] = hi[1];
}

// Largest of the wavefront's non-negative values, in every lane: DPP moves (six
// instructions; lane exchanges through LDS would wait for each other six
// times), compared as integers, whose order is the same.
template <int CTRL, int ROWS>
__device__ __forceinline__ int max_from(int v) {
    return max(v, __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xf, false));
}
__device__ __forceinline__ float wave_max(float f) {
    int v = __float_as_int(f);
    v = max_from<0x111, 0xf>(v);  // row_shr:1, 2, 4, 8
    v = max_from<0x112, 0xf>(v);
    v = max_from<0x114, 0xf>(v);
    v = max_from<0x118, 0xf>(v);
    v = max_from<0x142, 0xa>(v);  // row_bcast:15, 31
    v = max_from<0x143, 0xc>(v);
    return __int_as_float(__builtin_amdgcn_readlane(v, 63));
}

// The magnitude's code (as the value it stands for) for x >= 0 in units of the
// scale and dither d.  Codes are 8 steps per power of two down to 2^-6, and
// evenly spaced below.  x / ulp is exact (ulp is a power of two), so its sum
// with d is rounded once, as adamw.h says: it is below 16, and a decision is
// off by at most 2^-21 of a step.
__device__ __forceinline__ float code_of(float x, float d) {
    const uint32_t e = max(__float_as_uint(x) & 0x7f800000u, 0x3c800000u);  // 2^exponent, at least 2^-6
    const float ulp = __uint_as_float(e - (3u << 23));
    const float per = __uint_as_float((254u << 23) - (e - (3u << 23)));  // 1 / ulp
    const float q = fminf(floorf(fmaf(x, per, d)) * ulp, 448.f);
    return x <= kMax ? q : __uint_as_float(0x7fc00000u);
}

__device__ __forceinline__ float finite_abs(float v) {
    const float a = fabsf(v);
    return a <= kMax ? a : 0.f;
}

// Codes and scale of a block of the wavefront (four elements per lane): 256
// elements, so that the block's largest magnitude takes six lane exchanges and
// no LDS, and the scales add 1/32 of a byte to an element's 16.  Every
// operation is one that adamw.h names, rounded by itself.
template <bool ROOT>
__device__ __forceinline__ uint32_t encode(const float (&v)[kVec], uint32_t k, uint32_t turn,
                                           float& scale) {
    float top = 0.f;
#pragma unroll
    for (int j = 0; j < kVec; ++j) top = fmaxf(top, finite_abs(v[j]));
    scale = wave_max(top) * (1.f / 448.f);
    const bool live = scale >= 1.17549435e-38f;
    scale = live ? scale : 0.f;
    const float inv = live ? 1.f / scale : 0.f;
    float c[kVec];
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
        const uint32_t u = (k + j) * 2654435769u + turn + (ROOT ? 0x80000000u : 0u);
        const float d = float(u >> 8) * 0x1p-24f;
        const float x = fabsf(v[j]) * inv;
        c[j] = code_of(x, d);
        if (ROOT) c[j] = x > 0.f && c[j] == 0.f ? 0x1p-9f : c[j];
        else c[j] = copysignf(c[j], v[j]);
    }
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(c[0], c[1], 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(c[2], c[3], w, true);
    return uint32_t(w);
}

// One thread: the step's number and its coefficients.
__global__ void k_begin(int* step, const float* lr_dev, const float* scale_dev, const float* norm,
                        double lr, double beta1, double beta2, double decay, double scale,
                        double max_norm, Ctl* ctl) {
    Ctl c;
    const int t = *step + 1;
    if (lr_dev) lr = double(*lr_dev);
    if (scale_dev) scale = double(*scale_dev);
    c.on = 1;
    c.factor = float(scale);
    if (norm) {
        const float n = *norm;
        c.on = fabsf(n) <= kMax;
        if (max_norm > 0) {
            scale *= fmin(1.0, max_norm / (double(n) + 1e-6));
            c.factor *= fminf(1.f, float(max_norm) / (n + 1e-6f));
        }
    }
    c.drop = float(lr * decay);
    c.rate = float(lr / (1.0 - pow(beta1, double(t))));
    c.root = float(1.0 / sqrt(1.0 - pow(beta2, double(t))));
    c.scale = scale;
    c.turn = unsigned(t) * 3242174889u;
    if (c.on) *step = t;
    *ctl = c;
}

struct Betas {
    double b1, o1;  // o = 1 - b
    float b2, o2, eps;
    float b1f, o1f;  // b1 and o1, rounded
};

// The two terms of m may cancel, which would leave an fp32 sum with few of its
// digits for a parameter whose v is small: the m that moves the parameter is
// formed in fp64, whose few instructions hide behind the memory accesses, and
// rounded once.  What the parameter changes by is formed before it is added: 1 -
// lr * decay would keep few digits of a small decay, or none.
__device__ __forceinline__ void move(float& p, float m, float s, const Ctl& c, const Betas& h) {
    p += fmaf(-c.drop, p, -c.rate * m * gsc::rcp_hw(fmaf(s, c.root, h.eps)));
}

// New moments and parameter of one element.
__device__ __forceinline__ void advance(float& p, float& m, float& v, float g, const Ctl& c,
                                        const Betas& h) {
    const double gd = double(g) * c.scale;
    m = float(fma(h.b1, double(m), h.o1 * gd));
    g = float(gd);
    v = fmaf(h.b2, v, (h.o2 * g) * g);
    // the library's root: the hardware's instruction takes v below 2^-126 (gradients
    // below 1e-18 or so) for 0, by which the parameter would be divided where eps is
    // 0; the rest of its instructions hide behind the memory accesses, too
    move(p, m, sqrtf(v), c, h);
}

// The same with moments in 8 bits: m and s are the values of the codes, then
// what is to be encoded.  A code changes by 6 to 12 % where its value crosses a
// decision by one unit in the last place, and the next step moves the parameter
// by it, so that two evaluations whose roundings differ would part; m and s are
// therefore formed by exactly the operations that adamw.h names, each rounded
// by itself (square root included), and codes and scales come out the same
// wherever they are formed.
__device__ __forceinline__ void advance8(float& p, float& m, float ms, float& s, float vs, float g,
                                         const Ctl& c, const Betas& h) {
#pragma clang fp contract(off)
    const float precise = float(fma(h.b1, double(m) * double(ms), h.o1 * (double(g) * c.scale)));
    g = g * c.factor;
    m = h.b1f * (m * ms) + h.o1f * g;
    s = s * vs;
    s = sqrtf(h.b2 * (s * s) + (h.o2 * g) * g);
    move(p, precise, s, c, h);
}

enum { P_, G_, M_, V_, X0_ };  // then: master, and/or the two scales

template <class D, bool BITS8, bool MASTER>
constexpr int kPtrs = 4 + (MASTER ? 1 : 0) + (BITS8 ? 2 : 0);

// What a lane reads of one unit, as loaded.
template <class D, bool BITS8, bool MASTER>
struct In {
    Raw<D, kVec> g, p;
    Raw<F32, kVec> w, m, v;  // v, m: moments in 32 bits
    uint32_t cm, cv;         // codes
    float sm, sv;            // and their scales
};

// The loads of a batch of units come before its first store: a store could, for
// all the compiler knows, change what a later load reads, and the loads would
// wait for one another, unit by unit.  94M elements in fp32: 515 us unit by
// unit, 509 with all four at once; 140M with 8-bit moments and masters 413 unit
// by unit, 402 in pairs, 402 with four at once (and 18 us in place of 16.5 for
// 37 small tensors, whose registers four at once double).  The rounded operations
// that adamw.h names made the pairs 403 and 18.6 us.
template <class D, bool BITS8, bool MASTER>
__global__ __launch_bounds__(kThreads) void k_step(
    Table<kPtrs<D, BITS8, MASTER>, kFit<kPtrs<D, BITS8, MASTER>>> t, const Ctl* ctl, Betas h) {
    using S = typename D::S;
    using St = std::conditional_t<BITS8, uint8_t, float>;
    const int id = tensor_of(t, blockIdx.x);
    const long long n = t.n[id];
    const long long base = (long long)(int(blockIdx.x) - t.first[id]) * kChunk;
    S* p = static_cast<S*>(t.ptr[P_][id]);
    const S* g = static_cast<const S*>(t.ptr[G_][id]);
    St* m = static_cast<St*>(t.ptr[M_][id]);
    St* v = static_cast<St*>(t.ptr[V_][id]);
    float* w = MASTER ? static_cast<float*>(t.ptr[X0_][id]) : nullptr;
    float* ms = BITS8 ? static_cast<float*>(t.ptr[X0_ + MASTER][id]) : nullptr;
    float* vs = BITS8 ? static_cast<float*>(t.ptr[X0_ + MASTER + BITS8][id]) : nullptr;
    auto at = [&](int u) { return base + (u * kThreads + threadIdx.x) * kVec; };
    auto left = [&](int u) {
        const long long r = n - at(u);
        return int(r < kVec ? (r > 0 ? r : 0) : kVec);
    };
    // a wavefront's 256 elements are one block
    auto block = [&](int u) { return (base + (u * kThreads + threadIdx.x / 64 * 64) * kVec) / ADAMW_BLOCK; };
    constexpr int kBatch = BITS8 ? 2 : kUnits;
    const Ctl c = *ctl;
    if (!c.on) return;
#pragma unroll
    for (int u0 = 0; u0 < kUnits; u0 += kBatch) {
        In<D, BITS8, MASTER> in[kBatch];
#pragma unroll
        for (int u = u0; u < u0 + kBatch; ++u) {
            In<D, BITS8, MASTER>& q = in[u - u0];
            const long long k = at(u);
            const int l = left(u);
            q.g = fetch<D>(g + k, l);
            if constexpr (MASTER) q.w = fetch<F32>(w + k, l);
            else q.p = fetch<D>(p + k, l);
            if constexpr (BITS8) {
                const bool any = block(u) * ADAMW_BLOCK < n;
                q.cm = fetch_codes(m + k, l);
                q.cv = fetch_codes(v + k, l);
                q.sm = any ? ms[block(u)] : 0.f;
                q.sv = any ? vs[block(u)] : 0.f;
            } else {
                q.m = fetch<F32>(m + k, l);
                q.v = fetch<F32>(v + k, l);
            }
        }
#pragma unroll
        for (int u = u0; u < u0 + kBatch; ++u) {
            const In<D, BITS8, MASTER>& q = in[u - u0];
            const long long k = at(u);
            const int l = left(u);
            float pv[kVec], mv[kVec], vv[kVec];  // vv: 8 bits, sqrt(v)
            if constexpr (BITS8) {
                decode(q.cm, mv);
                decode(q.cv, vv);
            }
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                if constexpr (MASTER) pv[j] = q.w.get(j);
                else pv[j] = q.p.get(j);
                if constexpr (BITS8) {
                    advance8(pv[j], mv[j], q.sm, vv[j], q.sv, q.g.get(j), c, h);
                } else {
                    mv[j] = q.m.get(j);
                    vv[j] = q.v.get(j);
                    advance(pv[j], mv[j], vv[j], q.g.get(j), c, h);
                }
            }
            if constexpr (BITS8) {
                float a, b;
                put_codes(m + k, encode<false>(mv, uint32_t(k), c.turn, a), l);
                put_codes(v + k, encode<true>(vv, uint32_t(k), c.turn, b), l);
                if (block(u) * ADAMW_BLOCK < n && threadIdx.x % 64 == 0) {
                    ms[block(u)] = a;
                    vs[block(u)] = b;
                }
            } else {
                put<F32>(m + k, mv, l);
                put<F32>(v + k, vv, l);
            }
            if constexpr (MASTER) put<F32>(w + k, pv, l);
            put<D>(p + k, pv, l);
        }
    }
}

// Partial sums of squares: 140M bf16 elements in 63 us (4.4 TB/s) where they
// come from HBM at a stretch.
template <class D>
__global__ __launch_bounds__(kThreads) void k_squares(Table<1, kFit<1>> t, double* part) {
    using S = typename D::S;
    __shared__ double acc[kThreads / 64];
    const int id = tensor_of(t, blockIdx.x);
    const long long n = t.n[id];
    const long long base = (long long)(int(blockIdx.x) - t.first[id]) * kNormChunk;
    const S* g = static_cast<const S*>(t.ptr[0][id]);
    // fp64 from the first product: the sum of squares of fp32 values may leave
    // fp32's range, and the conversion costs less than the memory access
    double s = 0;
#pragma unroll
    for (int u = 0; u < int(kNormChunk) / (kThreads * kVec); ++u) {
        const long long k = base + (u * kThreads + threadIdx.x) * kVec;
        const int left = int(n - k < kVec ? (n - k > 0 ? n - k : 0) : kVec);
        const Raw<D, kVec> q = fetch<D>(g + k, left);
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            const double v = double(q.get(j));
            s = fma(v, v, s);
        }
    }
#pragma unroll
    for (int d = 32; d > 0; d /= 2) s += __shfl_xor(s, d);
    if (threadIdx.x % 64 == 0) acc[threadIdx.x / 64] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int k = 1; k < kThreads / 64; ++k) s += acc[k];
        part[blockIdx.x] = s;
    }
}

constexpr int kSumThreads = 1024;
__global__ __launch_bounds__(kSumThreads) void k_norm(const double* part, long long parts,
                                                      double scale, const float* scale_dev,
                                                      float* norm) {
    __shared__ double acc[kSumThreads / 64];
    double s = 0;
    for (long long k = threadIdx.x; k < parts; k += kSumThreads) s += part[k];
#pragma unroll
    for (int d = 32; d > 0; d /= 2) s += __shfl_xor(s, d);
    if (threadIdx.x % 64 == 0) acc[threadIdx.x / 64] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int k = 1; k < kSumThreads / 64; ++k) s += acc[k];
        if (scale_dev) scale = double(*scale_dev);
        *norm = float(fabs(scale) * sqrt(s));
    }
}

// Chunks of one launch (threads of a grid are below 2^32); no tensor has more.
constexpr long long kMaxChunks = 1LL << 23;

// Calls launch(table, chunks) for the tensors of a list, as many to a launch
// as a table and a grid hold.
template <int P, int N, class Ptrs, class Launch>
hipError_t in_tables(const adamw_tensor* list, int count, long long chunk, Ptrs ptrs, Launch launch) {
    Table<P, N> t;
    t.count = 0;
    t.first[0] = 0;
    auto flush = [&]() -> hipError_t {
        if (t.count == 0) return hipSuccess;
        launch(t, t.first[t.count]);
        t.count = 0;
        return hipGetLastError();
    };
    for (int i = 0; i < count; ++i) {
        if (list[i].n == 0) continue;
        const long long chunks = (list[i].n + chunk - 1) / chunk;
        if (t.count == N || t.first[t.count] + chunks > kMaxChunks) {
            const hipError_t e = flush();
            if (e != hipSuccess) return e;
        }
        void* p[P];
        ptrs(list[i], p);
        for (int k = 0; k < P; ++k) t.ptr[k][t.count] = p[k];
        t.n[t.count] = list[i].n;
        t.first[t.count + 1] = t.first[t.count] + int(chunks);
        ++t.count;
    }
    return flush();
}

template <class D, bool BITS8, bool MASTER>
hipError_t run_step(const adamw_tensor* list, int count, const Ctl* ctl, const Betas& h,
                    hipStream_t st) {
    constexpr int P = kPtrs<D, BITS8, MASTER>;
    return in_tables<P, kFit<P>>(
        list, count, kChunk,
        [](const adamw_tensor& t, void** p) {
            p[P_] = t.p;
            p[G_] = const_cast<void*>(t.g);
            p[M_] = t.m;
            p[V_] = t.v;
            if (MASTER) p[X0_] = t.w;
            if (BITS8) {
                p[X0_ + MASTER] = t.ms;
                p[X0_ + MASTER + 1] = t.vs;
            }
        },
        [&](const Table<P, kFit<P>>& t, int chunks) {
            k_step<D, BITS8, MASTER><<<dim3(chunks), kThreads, 0, st>>>(t, ctl, h);
        });
}
template <class D>
hipError_t run_type(bool bits8, bool master, const adamw_tensor* list, int count, const Ctl* ctl,
                    const Betas& h, hipStream_t st) {
    if (bits8)
        return master ? run_step<D, true, true>(list, count, ctl, h, st)
                      : run_step<D, true, false>(list, count, ctl, h, st);
    return master ? run_step<D, false, true>(list, count, ctl, h, st)
                  : run_step<D, false, false>(list, count, ctl, h, st);
}

template <class D>
hipError_t run_squares(const adamw_tensor* list, int count, double* part, long long* parts,
                       hipStream_t st) {
    long long before = 0;
    const hipError_t e = in_tables<1, kFit<1>>(
        list, count, kNormChunk,
        [](const adamw_tensor& t, void** p) { p[0] = const_cast<void*>(t.g); },
        [&](const Table<1, kFit<1>>& t, int chunks) {
            k_squares<D><<<dim3(chunks), kThreads, 0, st>>>(t, part + before);
            before += chunks;
        });
    *parts = before;
    return e;
}

}  // namespace

hipError_t grad_norm(int dtype, const adamw_tensor* t, int count, double scale,
                     const float* scale_dev, float* norm, double* part, hipStream_t st) {
    long long parts = 0;
    hipError_t e;
    if (dtype == ADAMW_F32) e = run_squares<F32>(t, count, part, &parts, st);
    else if (dtype == ADAMW_F16) e = run_squares<F16>(t, count, part, &parts, st);
    else e = run_squares<BF16>(t, count, part, &parts, st);
    if (e != hipSuccess) return e;
    k_norm<<<1, kSumThreads, 0, st>>>(part, parts, scale, scale_dev, norm);
    return hipGetLastError();
}

hipError_t step(const adamw_config& c, const adamw_tensor* t, int count, int* step, Ctl* ctl,
                hipStream_t st) {
    k_begin<<<1, 1, 0, st>>>(step, c.lr_dev, c.grad_scale_dev, c.norm, c.lr, c.beta1, c.beta2,
                             c.weight_decay, c.grad_scale, c.max_norm, ctl);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const Betas h{c.beta1, 1.0 - c.beta1, float(c.beta2), float(1.0 - c.beta2),
                  float(c.eps), float(c.beta1), float(1.0 - c.beta1)};
    bool master = false;
    for (int i = 0; i < count && !master; ++i) master = t[i].n > 0 && t[i].w;
    if (c.dtype == ADAMW_F32) return run_type<F32>(c.bits == 8, master, t, count, ctl, h, st);
    if (c.dtype == ADAMW_F16) return run_type<F16>(c.bits == 8, master, t, count, ctl, h, st);
    return run_type<BF16>(c.bits == 8, master, t, count, ctl, h, st);
}

}  // namespace adw

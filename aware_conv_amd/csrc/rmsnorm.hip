// Root-mean-square norm with the residual's addition (include/rmsnorm.h).
//
// HBM bounds it for rows of 256 elements and more.  A row is read once and kept in
// the registers of a wavefront, or of a workgroup where it is longer, and written
// from there; only rows of more than 32768 elements are read again.  Elements go 8
// at a time, whatever their alignment, and past the caches on their way out.  32768
// rows of 2048 with a residual in fp32, bf16: forwards 154 us (805 MB, 5.2 TB/s),
// backwards 198 us (the sum, dy and dtotal in, dx and the residual's gradient out,
// 1074 MB, 5.4 TB/s) and 10 us for the weight's sums; 16384 rows of 4096 with a
// residual, bf16, output in 8 bits: 95 us (470 MB, 5.0 TB/s); 23976 rows of 999,
// fp16, no two rows aligned alike: 40, 58 and 8 us (192 MB each way: 4.8 and 3.3 TB/s;
// backwards dtotal is asked for only after the row's sum is known).
//
// Narrow rows leave lanes idle, 8 elements to a lane and a wavefront to a row: 64M
// elements, bf16 with a residual, rows of 256, 128, 64, 16: forwards 111, 197, 387,
// 1589 us, backwards 170, 296, 546, 2032 (rows of 1024: 77 and 109).  Rows of 16385
// to 32768 elements have 32 a lane in 16 wavefronts, whose 128 registers do not hold
// them backwards (110 are spilled): 32768 forwards 96 us, backwards 278.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "close_sums.h"
#include "gscan_math.h"
#include "rmsnorm_internal.h"

namespace rmn {
namespace {

using gsc::BF16;
using gsc::F16;
using gsc::F32;

constexpr int kV = 8;             // elements of a vector
constexpr float kTop = 448.f;     // the largest e4m3 value
constexpr unsigned kParts = 1024;  // workgroups of the backward pass at most

constexpr long long kBlocks = 1 << 21;  // of the forward pass: a launch has fewer than 2^32 threads

// Elements c..c + 7 of a row of C, zero beyond it.
template <class D>
__device__ __forceinline__ void load(float (&v)[kV], const typename D::S* p, int c, int C) {
    if (c + kV <= C) {
        gsc::Raw<D, kV> q;
        gsc::load_vec<D, kV>(q, p + c);
#pragma unroll
        for (int j = 0; j < kV; ++j) v[j] = q.get(j);
    } else {
#pragma unroll
        for (int j = 0; j < kV; ++j) v[j] = c + j < C ? gsc::load_one<D>(p + min(c + j, C - 1)) : 0.f;
    }
}
template <class D>
__device__ __forceinline__ void store(typename D::S* p, const float (&v)[kV], int c, int C) {
    if (c + kV <= C) {
        gsc::store_vec_once<D, kV>(p + c, gsc::pack<D, false>(v));
    } else {
#pragma unroll
        for (int j = 0; j < kV; ++j)
            if (c + j < C) gsc::store_one<D>(p + c + j, v[j]);
    }
}
// v rounded to the type and widened again
template <class D>
__device__ __forceinline__ float rounded(float v) {
    if constexpr (D::kBytes == 4) return v;
    else return D::widen(D::narrow(v));
}

__device__ __forceinline__ void store_codes(uint8_t* p, const float (&v)[kV], int c, int C) {
    uint32_t w[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        int q = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * k], v[4 * k + 1], 0, false);
        w[k] = uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(v[4 * k + 2], v[4 * k + 3], q, true));
    }
    if (c + kV <= C) {
        struct __attribute__((packed, aligned(1))) P { uint32_t w[2]; };
        *reinterpret_cast<P*>(p + c) = P{{w[0], w[1]}};
    } else {
#pragma unroll
        for (int j = 0; j < kV; ++j)
            if (c + j < C) p[c + j] = uint8_t(w[j / 4] >> (8 * (j % 4)));
    }
}

// Sum (or, MAX, largest) over the threads of a row, in a fixed order; `lds` holds
// a value per wavefront and is free again after the next barrier.
template <int THREADS, bool MAX>
__device__ __forceinline__ float over_row(float v, float* lds) {
    auto op = [](float a, float b) { return MAX ? fmaxf(a, b) : a + b; };
#pragma unroll
    for (int m = 1; m < 64; m *= 2) v = op(v, __shfl_xor(v, m));
    if constexpr (THREADS > 64) {
        if (threadIdx.x % 64 == 0) lds[threadIdx.x / 64] = v;
        __syncthreads();
        v = lds[0];
#pragma unroll
        for (int k = 1; k < THREADS / 64; ++k) v = op(v, lds[k]);
        __syncthreads();
    }
    return v;
}

template <int THREADS>
constexpr int kBlock = THREADS < 256 ? 256 : THREADS;

// NV vectors per thread in registers; NV = 0: the row is read again for each of its uses.
template <class D, class R, int THREADS, int NV, bool E4M3>
__global__ __launch_bounds__(kBlock<THREADS>) void k_fwd(Args a) {
    __shared__ float lds[16];
    const int tid = threadIdx.x % THREADS;
    constexpr int kRows = kBlock<THREADS> / THREADS;
    const long long first_row = (long long)blockIdx.x * kRows + threadIdx.x / THREADS;
    // one turn, unless there are more rows than a launch has threads for; rows of more than a
    // wavefront have a workgroup of their own, whose threads take the same turns
    for (long long row = first_row; row < a.rows; row += (long long)gridDim.x * kRows) {
        const long long b = row / a.T, t = row % a.T;
        const typename D::S* const x = (const typename D::S*)a.x + b * a.x_sb + t * a.x_sr;
        const typename R::S* const res = (const typename R::S*)a.res + b * a.res_sb + t * a.res_sr;
        typename R::S* const total = (typename R::S*)a.total + b * a.total_sb + t * a.total_sr;
        const bool add = a.res != nullptr;
        const int C = a.C;
        constexpr int kStep = THREADS * kV;

        auto first = [&](float(&v)[kV], int c) {  // s, and its share of the sum of squares
            load<D>(v, x, c, C);
            if (add) {
                float r[kV];
                load<R>(r, res, c, C);
#pragma unroll
                for (int j = 0; j < kV; ++j) v[j] = rounded<R>(v[j] + r[j]);
                store<R>(total, v, c, C);
            }
            float q = 0.f;
#pragma unroll
            for (int j = 0; j < kV; ++j) q = fmaf(v[j], v[j], q);
            return q;
        };
        float s[NV ? NV : 1][kV], sum = 0.f;
        if constexpr (NV > 0) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int c = k * kStep + tid * kV;
                if (c < C) {
                    sum += first(s[k], c);
                } else {
#pragma unroll
                    for (int j = 0; j < kV; ++j) s[k][j] = 0.f;
                }
            }
        } else {
            for (int c = tid * kV; c < C; c += kStep) sum += first(s[0], c);
        }
        sum = over_row<THREADS, false>(sum, lds);
        const float rstd = 1.f / sqrtf(sum / float(C) + a.eps);
        if (a.rstd && tid == 0) a.rstd[row] = rstd;

        auto normed = [&](float(&v)[kV], int c) {
            float w[kV];
            load<F32>(w, a.w, c, C);
#pragma unroll
            for (int j = 0; j < kV; ++j) v[j] = v[j] * rstd * w[j];
        };
        auto again = [&](float(&v)[kV], int c) {
            if (add) load<R>(v, total, c, C);
            else load<D>(v, x, c, C);
            normed(v, c);
        };
        if constexpr (!E4M3) {
            typename D::S* const y = (typename D::S*)a.y + b * a.y_sb + t * a.y_sr;
            if constexpr (NV > 0) {
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    const int c = k * kStep + tid * kV;
                    if (c >= C) continue;
                    normed(s[k], c);
                    store<D>(y, s[k], c, C);
                }
            } else {
                for (int c = tid * kV; c < C; c += kStep) {
                    again(s[0], c);
                    store<D>(y, s[0], c, C);
                }
            }
        } else {
            uint8_t* const y = (uint8_t*)a.y + b * a.y_sb + t * a.y_sr;
            float top = 0.f;
            auto most = [&](const float(&v)[kV]) {
#pragma unroll
                for (int j = 0; j < kV; ++j) top = fmaxf(top, fabsf(v[j]));
            };
            if constexpr (NV > 0) {
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    const int c = k * kStep + tid * kV;
                    if (c >= C) continue;
                    normed(s[k], c);
                    most(s[k]);
                }
            } else {
                for (int c = tid * kV; c < C; c += kStep) {
                    again(s[0], c);
                    most(s[0]);
                }
            }
            top = over_row<THREADS, true>(top, lds);
            // below the normal numbers a scale has no inverse: such a row is zero
            const float scale = top / kTop >= 1.17549435e-38f ? top / kTop : 0.f, inv = scale > 0.f ? 1.f / scale : 0.f;
            if (tid == 0) a.scale[row] = scale;
            auto codes = [&](float(&v)[kV], int c) {
#pragma unroll
                for (int j = 0; j < kV; ++j) {
                    const float q = v[j] * inv;
                    v[j] = q > kTop ? kTop : q < -kTop ? -kTop : q;  // a NaN stays
                }
                store_codes(y, v, c, C);
            };
            if constexpr (NV > 0) {
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    const int c = k * kStep + tid * kV;
                    if (c < C) codes(s[k], c);
                }
            } else {
                for (int c = tid * kV; c < C; c += kStep) {
                    again(s[0], c);
                    codes(s[0], c);
                }
            }
        }
    }
}

template <class D, class R, int THREADS, int NV>
__global__ __launch_bounds__(kBlock<THREADS>) void k_bwd(Args a) {
    constexpr int kRows = kBlock<THREADS> / THREADS;
    constexpr int kStep = THREADS * kV;
    __shared__ float lds[16];
    __shared__ float sums[kRows > 1 ? kRows : 1][kRows > 1 ? kStep : 1];
    const int tid = threadIdx.x % THREADS, sub = threadIdx.x / THREADS;
    const int C = a.C;
    float dw[NV][kV] = {}, w[NV][kV];
#pragma unroll
    for (int k = 0; k < NV; ++k)
        if (k * kStep + tid * kV < C) load<F32>(w[k], a.w, k * kStep + tid * kV, C);
    for (long long row = (long long)blockIdx.x * kRows + sub; row < a.rows; row += (long long)gridDim.x * kRows) {
        const long long b = row / a.T, t = row % a.T;
        const typename R::S* const kept = (const typename R::S*)a.kept + b * a.kept_sb + t * a.kept_sr;
        const typename D::S* const dy = (const typename D::S*)a.dy + b * a.dy_sb + t * a.dy_sr;
        const float rstd = a.rstd_in[row];
        float n[NV][kV], g[NV][kV], sum = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = k * kStep + tid * kV;
            if (c >= C) continue;
            load<R>(n[k], kept, c, C);
            load<D>(g[k], dy, c, C);
#pragma unroll
            for (int j = 0; j < kV; ++j) {
                n[k][j] *= rstd;
                dw[k][j] = fmaf(g[k][j], n[k][j], dw[k][j]);
                g[k][j] *= w[k][j];
                sum = fmaf(g[k][j], n[k][j], sum);
            }
        }
        const float mean = over_row<THREADS, false>(sum, lds) / float(C);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = k * kStep + tid * kV;
            if (c >= C) continue;
            float d[kV] = {};
            if (a.dtotal) load<R>(d, (const typename R::S*)a.dtotal + b * a.dtotal_sb + t * a.dtotal_sr, c, C);
#pragma unroll
            for (int j = 0; j < kV; ++j) d[j] = fmaf(rstd, fmaf(-n[k][j], mean, g[k][j]), d[j]);
            if (a.dx) store<D>((typename D::S*)a.dx + b * a.dx_sb + t * a.dx_sr, d, c, C);
            if (a.dres) store<R>((typename R::S*)a.dres + b * a.dres_sb + t * a.dres_sr, d, c, C);
        }
    }
    if (!a.dw) return;
    float* const part = a.part + (long long)blockIdx.x * C;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = k * kStep + tid * kV;
        if constexpr (kRows > 1) {
#pragma unroll
            for (int j = 0; j < kV; ++j) sums[sub][tid * kV + j] = dw[k][j];
            __syncthreads();
            for (int i = threadIdx.x; i < kStep; i += kBlock<THREADS>) {
                float v = sums[0][i];
#pragma unroll
                for (int q = 1; q < kRows; ++q) v += sums[q][i];
                if (k * kStep + i < C) part[k * kStep + i] = v;
            }
            __syncthreads();
        } else {
            if (c < C) store<F32>(part, dw[k], c, C);
        }
    }
}

// Long rows: their sums first, then dx and, for a share of the columns, dw.
template <class D, class R>
__global__ __launch_bounds__(1024) void k_bwd_long(Args a) {
    __shared__ float lds[16];
    constexpr int kStep = 1024 * kV;
    const int C = a.C;
    bool fresh = true;
    float* const part = a.part + (long long)blockIdx.x * C;
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x, fresh = false) {
        const long long b = row / a.T, t = row % a.T;
        const typename R::S* const kept = (const typename R::S*)a.kept + b * a.kept_sb + t * a.kept_sr;
        const typename D::S* const dy = (const typename D::S*)a.dy + b * a.dy_sb + t * a.dy_sr;
        const float rstd = a.rstd_in[row];
        float n[kV], g[kV], w[kV], sum = 0.f;
        for (int c = threadIdx.x * kV; c < C; c += kStep) {
            load<R>(n, kept, c, C);
            load<D>(g, dy, c, C);
            load<F32>(w, a.w, c, C);
#pragma unroll
            for (int j = 0; j < kV; ++j) sum = fmaf(g[j] * w[j], n[j] * rstd, sum);
        }
        const float mean = over_row<1024, false>(sum, lds) / float(C);
        for (int c = threadIdx.x * kV; c < C; c += kStep) {
            float d[kV] = {}, q[kV] = {};
            load<R>(n, kept, c, C);
            load<D>(g, dy, c, C);
            load<F32>(w, a.w, c, C);
            if (a.dtotal) load<R>(d, (const typename R::S*)a.dtotal + b * a.dtotal_sb + t * a.dtotal_sr, c, C);
            if (a.dw && !fresh) load<F32>(q, part, c, C);
#pragma unroll
            for (int j = 0; j < kV; ++j) {
                n[j] *= rstd;
                q[j] = fmaf(g[j], n[j], q[j]);
                d[j] = fmaf(rstd, fmaf(-n[j], mean, g[j] * w[j]), d[j]);
            }
            if (a.dw) store<F32>(part, q, c, C);
            if (a.dx) store<D>((typename D::S*)a.dx + b * a.dx_sb + t * a.dx_sr, d, c, C);
            if (a.dres) store<R>((typename R::S*)a.dres + b * a.dres_sb + t * a.dres_sr, d, c, C);
        }
    }
}

template <class F>
hipError_t with_types(const rmsnorm_shape& s, F&& f) {
    if (s.dtype == GSCAN_F32) return f(F32{}, F32{});
    if (s.dtype == GSCAN_F16) return s.rdtype == GSCAN_F32 ? f(F16{}, F32{}) : f(F16{}, F16{});
    return s.rdtype == GSCAN_F32 ? f(BF16{}, F32{}) : f(BF16{}, BF16{});
}
template <int T, int N>
struct Width {
    static constexpr int kThreads = T, kVectors = N;
};
template <class F>
hipError_t with_width(const Plan& p, F&& f) {
    switch (p.threads * 8 + p.vectors) {
        case 64 * 8 + 1: return f(Width<64, 1>{});
        case 64 * 8 + 2: return f(Width<64, 2>{});
        case 64 * 8 + 4: return f(Width<64, 4>{});
        case 256 * 8 + 2: return f(Width<256, 2>{});
        case 256 * 8 + 4: return f(Width<256, 4>{});
        case 1024 * 8 + 2: return f(Width<1024, 2>{});
        case 1024 * 8 + 4: return f(Width<1024, 4>{});
        default: return f(Width<1024, 0>{});
    }
}

}  // namespace

Plan plan(const rmsnorm_shape& s) {
    Plan p{};
    const int C = s.C;
    p.threads = C <= 64 * 32 ? 64 : C <= 256 * 32 ? 256 : 1024;
    const int vectors = (C + p.threads * kV - 1) / (p.threads * kV);
    p.vectors = vectors <= 1 && p.threads == 64 ? 1 : vectors <= 2 ? 2 : vectors <= 4 ? 4 : 0;
    p.per_block = p.threads == 64 ? 4 : 1;
    const long long rows = (long long)s.B * s.T, blocks = (rows + p.per_block - 1) / p.per_block;
    p.parts = unsigned(std::min(blocks, (long long)kParts));
    p.scratch = 4 * size_t(p.parts) * C;
    return p;
}

hipError_t fwd(const rmsnorm_shape& s, const Args& a, bool e4m3, hipStream_t st) {
    const Plan p = plan(s);
    const unsigned blocks = unsigned(std::min((a.rows + p.per_block - 1) / p.per_block, kBlocks));
    return with_types(s, [&](auto D, auto R) {
        return with_width(p, [&](auto W) {
            using T = decltype(D);
            using U = decltype(R);
            constexpr int kT = decltype(W)::kThreads, kN = decltype(W)::kVectors;
            if (e4m3) k_fwd<T, U, kT, kN, true><<<blocks, kBlock<kT>, 0, st>>>(a);
            else k_fwd<T, U, kT, kN, false><<<blocks, kBlock<kT>, 0, st>>>(a);
            return hipGetLastError();
        });
    });
}

hipError_t bwd(const rmsnorm_shape& s, Args a, void* ws, hipStream_t st) {
    const Plan p = plan(s);
    a.part = static_cast<float*>(ws);
    if (p.parts) {
        const hipError_t e = with_types(s, [&](auto D, auto R) {
            return with_width(p, [&](auto W) {
                using T = decltype(D);
                using U = decltype(R);
                constexpr int kT = decltype(W)::kThreads, kN = decltype(W)::kVectors;
                if constexpr (kN == 0) k_bwd_long<T, U><<<p.parts, 1024, 0, st>>>(a);
                else k_bwd<T, U, kT, kN><<<p.parts, kBlock<kT>, 0, st>>>(a);
                return hipGetLastError();
            });
        });
        if (e != hipSuccess) return e;
    }
    return calls::close_sums<2>(p.parts, st, {a.part, a.C, a.dw});
}

}  // namespace rmn

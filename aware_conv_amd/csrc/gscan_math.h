// Element arithmetic of the gated linear recurrence (include/gscan.h), shared
// by its kernels for planes, tokens and single positions.
//
// One element costs 6 transcendental instructions forwards (quarter rate: 16
// cycles of a SIMD per wavefront each) and about 35 others (4 cycles each), so
// that at 16-bit storage the vector ALU and HBM bound the kernels about
// equally, and instructions are counted below.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gscan_internal.h"

namespace gsc {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// v_exp_f32, v_rcp_f32, v_sqrt_f32, v_rsq_f32: one unit in the last place,
// without the library functions' range reduction and correction steps, which
// would cost more than the rest of an element
__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float rcp_hw(float x) { return __builtin_amdgcn_rcpf(x); }
__device__ __forceinline__ float sqrt_hw(float x) { return __builtin_amdgcn_sqrtf(x); }
__device__ __forceinline__ float rsq_hw(float x) { return __builtin_amdgcn_rsqf(x); }

// Storage types.  Two 16-bit values share a 32-bit word, the first low.
struct F32 {
    using S = float;
    static constexpr int kBytes = 4;
};
struct F16 {
    using S = uint16_t;
    static constexpr int kBytes = 2;
    __device__ static float widen(uint32_t lo16) {
        return float(__builtin_bit_cast(_Float16, uint16_t(lo16)));
    }
    // to nearest even, overflow to infinity
    __device__ static uint32_t narrow(float v) {
        return __builtin_bit_cast(uint16_t, _Float16(v));
    }
};
struct BF16 {
    using S = uint16_t;
    static constexpr int kBytes = 2;
    __device__ static float widen(uint32_t lo16) { return __builtin_bit_cast(float, lo16 << 16); }
    __device__ static uint32_t narrow(float v) {
        return __builtin_bit_cast(uint16_t, __bf16(v));
    }
};

// V consecutive elements as loaded.
template <class D, int V>
struct Raw {
    static constexpr int kWords = (V * D::kBytes + 3) / 4;
    uint32_t w[kWords];
    __device__ __forceinline__ float get(int j) const {
        if constexpr (D::kBytes == 4) {
            return __builtin_bit_cast(float, w[j]);
        } else if constexpr (std::is_same<D, BF16>::value) {
            return __builtin_bit_cast(float, (j & 1) ? (w[j / 2] & 0xffff0000u) : (w[j / 2] << 16));
        } else {
            return D::widen((j & 1) ? (w[j / 2] >> 16) : (w[j / 2] & 0xffffu));
        }
    }
    __device__ __forceinline__ void set(int j, float v) {
        if constexpr (D::kBytes == 4) {
            w[j] = __builtin_bit_cast(uint32_t, v);
        } else {
            const uint32_t h = D::narrow(v);
            w[j / 2] = (j & 1) ? ((w[j / 2] & 0xffffu) | (h << 16)) : ((w[j / 2] & 0xffff0000u) | h);
        }
    }
};

// Any element alignment is taken: global accesses of gfx950 need none, so a
// packed struct keeps them one wide instruction where the address is odd too.
template <class D, int V>
__device__ __forceinline__ void load_vec(Raw<D, V>& out, const typename D::S* p) {
    static_assert(V * D::kBytes >= 4, "at least a word");
    struct __attribute__((packed, aligned(D::kBytes))) P {
        uint32_t w[Raw<D, V>::kWords];
    };
    const P q = *reinterpret_cast<const P*>(p);
#pragma unroll
    for (int k = 0; k < Raw<D, V>::kWords; ++k) out.w[k] = q.w[k];
}
template <class D, int V>
__device__ __forceinline__ void store_vec(typename D::S* p, const Raw<D, V>& v) {
    struct __attribute__((packed, aligned(D::kBytes))) P {
        uint32_t w[Raw<D, V>::kWords];
    };
    P q;
#pragma unroll
    for (int k = 0; k < Raw<D, V>::kWords; ++k) q.w[k] = v.w[k];
    *reinterpret_cast<P*>(p) = q;
}
template <class D>
__device__ __forceinline__ float load_one(const typename D::S* p) {
    if constexpr (D::kBytes == 4) return *p;
    else return D::widen(*p);
}
template <class D>
__device__ __forceinline__ void store_one(typename D::S* p, float v) {
    if constexpr (D::kBytes == 4) *p = v;
    else *p = typename D::S(D::narrow(v));
}

// softplus without overflow; once per row or channel and workgroup
__device__ __forceinline__ float softplus(float v) {
    return fmaxf(v, 0.f) + log1pf(expf(-fabsf(v)));
}

// 1 - a^2 = -expm1(y) for y = 2 L <= 0.  Near 0 the first eight terms of the
// series (the ninth is below 2^-25 of the sum there); beyond, 1 - a^2 loses
// no more than a bit.
__device__ __forceinline__ float one_minus_sq(float a, float y) {
    float s = fmaf(y, 1.f / 40320.f, 1.f / 5040.f);
    s = fmaf(y, s, 1.f / 720.f);
    s = fmaf(y, s, 1.f / 120.f);
    s = fmaf(y, s, 1.f / 24.f);
    s = fmaf(y, s, 1.f / 6.f);
    s = fmaf(y, s, 0.5f);
    s = fmaf(y, s, 1.f);
    return y > -0.5f ? -y * s : fmaf(-a, a, 1.f);
}

// What the recurrence needs of an element: h = a h + b.  `rate` is
// decay * softplus(lam) * log2(e), so that exp2 takes rate * sig(r) directly.
__device__ __forceinline__ void gate_fwd(float x, float r, float i, float rate, float& a,
                                         float& b) {
    const float sr = rcp_hw(1.f + exp2_hw(-kLog2e * r));
    const float l2 = -rate * sr;
    a = exp2_hw(l2);
    const float w = sqrt_hw(one_minus_sq(a, (2.f * kLn2) * l2));
    const float si = rcp_hw(1.f + exp2_hw(-kLog2e * i));
    b = w * (si * x);
}

// sig(v) and sig(-v), each accurate where it is small
__device__ __forceinline__ void sig_both(float v, float& s, float& n) {
    const float e = exp2_hw(-kLog2e * fabsf(v));
    const float d = rcp_hw(1.f + e);
    const float ed = e * d;
    s = v >= 0.f ? d : ed;
    n = v >= 0.f ? ed : d;
}

// Gradients of one element: g is that of h_t, hp is h_{t-1}, a as formed by
// gate_fwd.  `e` returns e_t sig(r_t), the term of dlam.
__device__ __forceinline__ void gate_bwd(float x, float r, float i, float rate, float a, float hp,
                                         float g, float& dx, float& dr, float& di, float& e) {
    float sr, nr, si, ni;
    sig_both(r, sr, nr);
    sig_both(i, si, ni);
    const float L = -kLn2 * rate * sr;
    const float q = one_minus_sq(a, 2.f * L);
    // 1 / w; 0 where w is 0 or its square below the normal range (v_rsq_f32
    // would give infinity there), NaN where q is
    const float inv = q >= 1.17549435e-38f ? rsq_hw(q) : q * 0.f;
    const float w = q * inv;
    const float gx = g * si;
    dx = gx * w;
    di = dx * (x * ni);
    const float d = g * (a * hp) - gx * x * (a * a * inv);
    dr = d * L * nr;
    e = d * sr;
}

}  // namespace gsc

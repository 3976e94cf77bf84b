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

// Storage types.  Two 16-bit values share a 32-bit word, the first low;
// narrowing is to nearest even (fp16: overflow to infinity).
typedef float Float2 __attribute__((ext_vector_type(2)));
struct F32 {
    using S = float;
    static constexpr int kBytes = 4;
};
struct F16 {
    using S = uint16_t;
    using Pair = _Float16 __attribute__((ext_vector_type(2)));
    static constexpr int kBytes = 2;
    __device__ static float widen(uint32_t lo16) {
        return float(__builtin_bit_cast(_Float16, uint16_t(lo16)));
    }
    __device__ static uint32_t narrow(float v) {
        return __builtin_bit_cast(uint16_t, _Float16(v));
    }
};
struct BF16 {
    using S = uint16_t;
    using Pair = __bf16 __attribute__((ext_vector_type(2)));
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

// The values v (V even), last first if TURNED.
template <class D, bool TURNED, int V>
__device__ __forceinline__ Raw<D, V> pack(const float (&v)[V]) {
    Raw<D, V> q;
    if constexpr (D::kBytes == 4) {
#pragma unroll
        for (int j = 0; j < V; ++j) q.w[j] = __builtin_bit_cast(uint32_t, v[TURNED ? V - 1 - j : j]);
    } else {
#pragma unroll
        for (int j = 0; j < V; j += 2) {
            const Float2 f{v[TURNED ? V - 1 - j : j], v[TURNED ? V - 2 - j : j + 1]};
            q.w[j / 2] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, typename D::Pair));
        }
    }
    return q;
}

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

// decay * softplus(lam) * log2(e): the factor of sig(r) in -log2(a).
// softplus = max(lam, 0) + log1p(e) with e = exp(-|lam|) in (0, 1], by
// log1p(e) = 2 atanh(z), z = e / (2 + e) <= 1/3, and the series of atanh to
// z^15 (the next term is below 2^-26 of the sum).  The library's log1pf takes
// 120 instructions, which a thread spreads over as few as 4 elements of 45.
__device__ __forceinline__ float rate_of(float decay, float lam) {
    const float e = exp2_hw(-kLog2e * fabsf(lam));
    const float z = e * rcp_hw(2.f + e), y = z * z;
    float s = fmaf(y, 1.f / 15.f, 1.f / 13.f);
    s = fmaf(y, s, 1.f / 11.f);
    s = fmaf(y, s, 1.f / 9.f);
    s = fmaf(y, s, 1.f / 7.f);
    s = fmaf(y, s, 1.f / 5.f);
    s = fmaf(y, s, 1.f / 3.f);
    s = fmaf(y, s, 1.f);
    return decay * kLog2e * (fmaxf(lam, 0.f) + 2.f * z * s);
}

// 1 - a for a = 2^l, l <= 0, given a as the hardware forms it.  Near l = 0, -l
// times the polynomial that interpolates (1 - 2^l) / -l at the Chebyshev nodes of
// -0.25..0 (6e-8 of itself off at most); beyond, a is below 0.85 and the
// difference is as good.
__device__ __forceinline__ float one_minus(float a, float l) {
    float s = fmaf(l, 0.0089771692f, 0.055405185f);
    s = fmaf(l, s, 0.24022159f);
    s = fmaf(l, s, 0.69314712f);
    return l > -0.25f ? -l * s : 1.f - a;
}
// 1 - a^2 from a and 1 - a: no digits are lost.
__device__ __forceinline__ float one_minus_sq(float a, float e) { return fmaf(e, a, e); }

__device__ __forceinline__ float sig(float v) { return rcp_hw(1.f + exp2_hw(-kLog2e * v)); }

// What the recurrence needs of an element: h = a h + b; and its gates.
__device__ __forceinline__ void gate_fwd(float x, float r, float i, float rate, float& a,
                                         float& b, float& sr, float& si) {
    sr = sig(r);
    si = sig(i);
    const float l = -rate * sr;
    a = exp2_hw(l);
    const float e = one_minus(a, l);
    // The hardware's power is rounded with a bias, near 1 of 6e-9 downwards, which
    // a slow decay adds up: a state that lasts was 4.5e-5 off after 9000 positions,
    // 3e-4 after 60000.  1 - e has no bias (2e-6 and 8e-6), and its two instructions
    // cost up to 2% (8x4096x2048 bf16 fwd + bwd 366 and 372 us).
    a = l > -0.25f ? 1.f - e : a;
    b = sqrt_hw(one_minus_sq(a, e)) * (si * x);
}

// Gradients of one element from its gates and a as gate_fwd formed them: g is
// that of h_t, hp is h_{t-1}.  `e` returns e_t sig(r_t), the term of dlam.
__device__ __forceinline__ void gate_bwd(float x, float sr, float si, float rate, float a, float hp,
                                         float g, float& dx, float& dr, float& di, float& e) {
    const float q = one_minus_sq(a, one_minus(a, -rate * sr));
    // 1 / w, kept finite where q is 0 or leaves the normal range: its factors
    // in the gradients are below 2^-60 there, and w = q inv is 0
    const float inv = rsq_hw(q + 1.2e-37f);
    const float gx = g * si;
    dx = gx * (q * inv);
    di = dx * (x * (1.f - si));
    e = (g * (a * hp) - gx * x * (a * a * inv)) * sr;
    dr = e * ((-kLn2 * rate) * (1.f - sr));
}

}  // namespace gsc

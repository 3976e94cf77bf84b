// Element arithmetic and lane exchanges of the selective scan (include/sscan.h).
//
// A wavefront takes 16 channels of a sequence and their up to 64 states: lane
// 16 r + i holds states r NP .. r NP + NP - 1 of channel i in registers and
// walks along the positions.  What a position gives all channels, b and c, is held
// in registers too, of tiles of 16 positions: lane 16 r + i has row r's states of
// position i, and an operand modifier of the vector instructions (DPP
// row_newbcast) hands position i's value to the whole row.  So the innermost step
// of a state, h = exp2(delta A') h + u b, s += c h, is five instructions, one of
// them transcendental (24 cycles of a SIMD a wavefront), and reads nothing from
// memory but the position's delta and u, which LDS holds.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>
#include <utility>

#include "gscan_math.h"
#include "sscan_internal.h"

namespace ssc {

using gsc::BF16;
using gsc::exp2_hw;
using gsc::F16;
using gsc::F32;
using gsc::kLn2;
using gsc::kLog2e;
using gsc::rcp_hw;
using gsc::sig;

template <int N, class F, int... I>
__device__ __forceinline__ void unroll_(F&& f, std::integer_sequence<int, I...>) {
    (f(std::integral_constant<int, I>{}), ...);
}
// f(0), ..., f(N - 1), each with a constant
template <int N, class F>
__device__ __forceinline__ void unroll(F&& f) {
    unroll_<N>(f, std::make_integer_sequence<int, N>{});
}

// Lane I's value of the own row of 16, in all its lanes.
template <int I>
__device__ __forceinline__ float bcast(float v) {
    return __builtin_bit_cast(
        float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x150 + I, 0xf, 0xf, true));
}

// From each lane's parts of four sums over the four rows: row r gets the r-th.
// The exchange of halves, then of rows, is an instruction each.
__device__ __forceinline__ float sum_rows(float v0, float v1, float v2, float v3) {
    // an element of the pair is copied before its bits are taken: they are taken from the pair's start otherwise
    auto sum = [](auto q) {
        const unsigned a = q[0], b = q[1];
        return __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b);
    };
    auto bits = [](float v) { return __builtin_bit_cast(unsigned, v); };
    const float v02 = sum(__builtin_amdgcn_permlane32_swap(bits(v0), bits(v2), false, false));
    const float v13 = sum(__builtin_amdgcn_permlane32_swap(bits(v1), bits(v3), false, false));
    return sum(__builtin_amdgcn_permlane16_swap(bits(v02), bits(v13), false, false));
}

// exp2(x A'), A' = A log2(e).  The hardware's power of a small exponent is
// rounded with a bias, 7e-9 downwards near 1, which a slow decay adds up: a
// state that lasts 14000 positions would be 1e-4 off.  The addition, which costs nothing
// (the product becomes a fused one), moves the mean back: the mean error is at
// most 3e-10 down to 0.9993, 3e-9 down to 0.994, where a state forgets it
// sooner: 1.2e-6 of a state at most.  The power of 1e-8 is 1.
constexpr float kLift = 1e-8f;
__device__ __forceinline__ float decay(float delta, float a2) {
    return exp2_hw(fmaf(delta, a2, kLift));
}

// softplus(v), and from the same exponential its derivative sig(v).
// log1p(e) = 2 atanh(z) with z = e / (2 + e) <= 1/3; atanh(z) / z by the
// polynomial in z^2 that interpolates it at the Chebyshev nodes of 0..1/9, 8e-9
// off at most.
struct Step {
    float delta, slope;
};
__device__ __forceinline__ Step softplus(float v) {
    const float e = exp2_hw(-kLog2e * fabsf(v));
    const float z = e * rcp_hw(2.f + e), y = z * z;
    float p = fmaf(y, 0.140788898f, 0.139825791f);
    p = fmaf(y, p, 0.200122982f);
    p = fmaf(y, p, 0.333331615f);
    p = fmaf(y, p, 1.f);
    return {fmaxf(v, 0.f) + 2.f * z * p, (v >= 0.f ? 1.f : e) * rcp_hw(1.f + e)};
}

// LDS traffic within a wavefront: its operations are in order; the compiler is
// told to keep them so.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// NP states of a position from row r on, zero beyond the N there are.
template <class D, int NP>
__device__ __forceinline__ void load_states(float (&out)[NP], const typename D::S* p, int first,
                                            int N, bool whole, bool valid) {
    if (whole) {
        if constexpr (NP * D::kBytes >= 4) {
            gsc::Raw<D, NP> q;
            gsc::load_vec<D, NP>(q, p + first);
#pragma unroll
            for (int j = 0; j < NP; ++j) out[j] = valid ? q.get(j) : 0.f;
            return;
        }
    }
#pragma unroll
    for (int j = 0; j < NP; ++j) {
        const float v = gsc::load_one<D>(p + min(first + j, N - 1));
        out[j] = valid && first + j < N ? v : 0.f;
    }
}

}  // namespace ssc

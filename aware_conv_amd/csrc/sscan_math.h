// Element arithmetic, lane exchanges and the division of work of the selective scan
// (include/sscan.h).
//
// A wavefront takes 16 channels of a sequence and 4 NP of their states, and walks
// along the positions in tiles of 16: lane 16 r + i holds the NP states from
// r NP on of channel i in registers.  What a position gives all channels, b and c,
// is in registers too: lane 16 r + i has row r's states of the tile's position i,
// and an operand modifier of the vector instructions (DPP row_newbcast) hands
// position i's value to the whole row.  So the innermost step of a state,
// h = exp2(delta A') h + u b, s += c h, is five instructions, and reads nothing from
// memory but the position's delta and u, which LDS holds.  On this chip it takes
// 2.4 + 8.3 + 4.3 + 2.4 + 4.3 = 22 cycles of a SIMD where four wavefronts share it, 27
// with two and 42 with one: states are therefore divided among NB wavefronts of the
// same channels.
//
// A workgroup has CT x NB wavefronts.  The elements of a tile, 16 positions of its
// 16 CT channels, are divided among all of them, channels along the lanes, so that
// what is read and written of a position is one run: a thread forms delta and u (and
// the output) of a channel at every 4 NB-th position.
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

__device__ __forceinline__ float rate_of(float a_log);

// Which wavefronts of a workgroup hold what.
template <int NP_, int NB_>
struct Form {
    static constexpr int NP = NP_;                    // states of a lane
    static constexpr int NB = NB_;                    // wavefronts that share 16 channels
    static constexpr int CT = NB_ <= 2 ? 4 : 2;       // groups of 16 channels
    static constexpr int kThreads = 64 * NB * CT;
    static constexpr int kChannels = 16 * CT;
    static constexpr int kStep = 4 * NB;              // positions from one of a thread's elements to the next
    static constexpr int kSlots = (16 + kStep - 1) / kStep;  // elements of a thread in a tile, at most
    static constexpr int kStates = 4 * NP * NB;       // at least N
};

// f with the storage type and the division that a plan names.
template <class Fn>
hipError_t with_form(int dtype, const Plan& p, Fn&& f) {
    auto typed = [&](auto D) {
        switch (p.per_lane * 8 + p.waves) {
            case 1 * 8 + 1: return f(D, Form<1, 1>{});
            case 2 * 8 + 1: return f(D, Form<2, 1>{});
            case 2 * 8 + 2: return f(D, Form<2, 2>{});
            case 2 * 8 + 3: return f(D, Form<2, 3>{});
            case 2 * 8 + 4: return f(D, Form<2, 4>{});
            case 4 * 8 + 3: return f(D, Form<4, 3>{});
            default: return f(D, Form<4, 4>{});
        }
    };
    switch (dtype) {
        case GSCAN_F32: return typed(gsc::F32{});
        case GSCAN_F16: return typed(gsc::F16{});
        default: return typed(gsc::BF16{});
    }
}

// Where a lane stands, and the parameters of its states.
template <class F>
struct Lane {
    static constexpr int NP = F::NP;
    int lane, row, i, ct, nb, tile, seq, s, group, d, n, t_lo, t_end, t_hi;
    int d0;                         // the workgroup's first channel
    // its element of a tile: channel (of the workgroup's, and of all; where it is staged), first position
    // of the wavefront's and after that the lane's
    int io_ch, io_d, io_at, io_base, io_row;
    bool last_slot;                 // whether the last slot's position is in the tile
    bool live;      // whether the lane's channel is there: otherwise it goes along on the group's last one,
                    // and writes what that one's lane writes
    int at[F::NP];  // its states; those that are not there are the last one once more, with c = 0
    long long states_at, all;
    float a2[NP], bias;             // bias: of the element's channel
    bool there[NP];
    __device__ __forceinline__ Lane(const Args& a) {
        lane = threadIdx.x & 63;
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        row = lane >> 4;
        i = lane & 15;
        ct = wave / F::NB;
        nb = wave % F::NB;
        const int tiles = a.G * a.tiles, unit = blockIdx.x % tiles, rest = blockIdx.x / tiles;
        seq = rest / a.S;
        s = rest % a.S;
        group = unit / a.tiles;
        tile = unit % a.tiles;
        const int c0 = tile * F::kChannels, most = a.Dg - 1 - c0;  // channels there are, less one
        live = ct * 16 + i <= most;
        d0 = group * a.Dg + c0;
        d = d0 + min(ct * 16 + i, most);
        const int io = threadIdx.x % F::kChannels;
        io_ch = min(io, most);
        io_d = d0 + io_ch;
        io_at = io;
        io_base = wave * 64 / F::kChannels;
        io_row = lane / F::kChannels;
        last_slot = io_base + (F::kSlots - 1) * F::kStep < 16;
        n = a.lengths ? min(max(a.lengths[seq], 0), a.T) : a.T;
        t_lo = s * a.seg;
        t_end = min(a.T - t_lo, a.seg) + t_lo;
        t_hi = min(t_end, n);
        states_at = ((long long)seq * a.D + d) * a.N;
        all = (long long)a.B * a.D * a.N;
        bias = a.dt_bias ? a.dt_bias[io_d] : 0.f;
#pragma unroll
        for (int j = 0; j < NP; ++j) {
            const int m = (nb * 4 + row) * NP + j;
            there[j] = m < a.N;
            at[j] = min(m, a.N - 1);
            a2[j] = rate_of(a.a_log[(long long)d * a.N + at[j]]);
        }
    }
};

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

// acc[j] += bcast<I>(v[j]) * f.  The compiler does not put the modifier on a
// multiply-add; a register that it reads has to be two instructions old, which the
// leading s_nop sees to.
template <int I, int NP>
__device__ __forceinline__ void add_bcast(float (&acc)[NP], const float (&v)[NP], float f) {
    if constexpr (NP == 1) {
        acc[0] = fmaf(bcast<I>(v[0]), f, acc[0]);
    } else {
#pragma unroll
        for (int j = 0; j < NP; j += 2)
            asm("s_nop 1\n\t"
                "v_fmac_f32_dpp %0, %2, %4 row_newbcast:%5 row_mask:0xf bank_mask:0xf\n\t"
                "v_fmac_f32_dpp %1, %3, %4 row_newbcast:%5 row_mask:0xf bank_mask:0xf"
                : "+v"(acc[j]), "+v"(acc[j + 1])
                : "v"(v[j]), "v"(v[j + 1]), "v"(f), "n"(I));
    }
}
// sum_j bcast<I>(v[j]) * f[j]; products and sums apart, so that the products take the modifier
template <int I, int NP>
__device__ __forceinline__ float sum_bcast(const float (&v)[NP], const float (&f)[NP]) {
#pragma clang fp contract(off)
    float p[NP];
#pragma unroll
    for (int j = 0; j < NP; ++j) p[j] = bcast<I>(v[j]) * f[j];
    if constexpr (NP == 1) return p[0];
    else if constexpr (NP == 2) return p[0] + p[1];
    else return (p[0] + p[1]) + (p[2] + p[3]);
}

// From each lane's parts of four sums over the 16 lanes of its row, twice over:
// p0 and q0 hold the k-th sums in lanes 4 k .. 4 k + 3.  An addition that is
// written in some groups of four lanes only puts two sums side by side, so that
// four take eight instructions.
__device__ __forceinline__ void sum_lanes(float& p0, float& p1, float p2, float p3, float& q0,
                                          float& q1, float q2, float q3) {
    asm("s_nop 1\n\t"
        "v_add_f32_dpp %0, %0, %0 row_ror:8 row_mask:0xf bank_mask:0xf\n\t"
        "v_add_f32_dpp %2, %2, %2 row_ror:8 row_mask:0xf bank_mask:0xf\n\t"
        "v_add_f32_dpp %1, %1, %1 row_ror:8 row_mask:0xf bank_mask:0xf\n\t"
        "v_add_f32_dpp %3, %3, %3 row_ror:8 row_mask:0xf bank_mask:0xf\n\t"
        "v_add_f32_dpp %0, %4, %4 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
        "v_add_f32_dpp %2, %6, %6 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
        "v_add_f32_dpp %1, %5, %5 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
        "v_add_f32_dpp %3, %7, %7 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
        "v_add_f32_dpp %0, %0, %0 row_half_mirror row_mask:0xf bank_mask:0xf\n\t"
        "v_add_f32_dpp %2, %2, %2 row_half_mirror row_mask:0xf bank_mask:0xf\n\t"
        "v_add_f32_dpp %0, %1, %1 row_half_mirror row_mask:0xf bank_mask:0xa\n\t"
        "v_add_f32_dpp %2, %3, %3 row_half_mirror row_mask:0xf bank_mask:0xa\n\t"
        "s_nop 0\n\t"
        "v_add_f32_dpp %0, %0, %0 quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf\n\t"
        "v_add_f32_dpp %2, %2, %2 quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf\n\t"
        "s_nop 0\n\t"
        "v_add_f32_dpp %0, %0, %0 quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf\n\t"
        "v_add_f32_dpp %2, %2, %2 quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf\n\t"
        "s_nop 1"
        : "+v"(p0), "+v"(p1), "+v"(q0), "+v"(q1)
        : "v"(p2), "v"(p3), "v"(q2), "v"(q3));
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
// A' from a_log; finite, so that a step of zero leaves a state as it is.
__device__ __forceinline__ float rate_of(float a_log) {
    const float v = -kLog2e * expf(a_log);
    return v < -3e38f ? -3e38f : v;
}
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

// A barrier for what is in LDS.  __syncthreads would also wait for the loads of the
// next tile, which are under way, and for stores: 1 to 2 us a tile.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// A wavefront's view of one activation: lanes are `off` bytes from `base`, which is
// the same for all of them and stays in scalar registers, and which moves along the
// positions.  (So addresses cost a vector register per tensor and no vector
// instruction; `off` holds 15 rows of stride up to 2^26.)
template <class S>
struct Rows {
    const char* base;
    unsigned off;
    long long row;  // bytes
    // first: the wavefront's first element of its sequence; at: the position that `base` starts at
    __device__ __forceinline__ Rows(const void* p, long long sb, long long sr, int seq, long long at,
                                    int first, int lane_row, int lane_elem)
        : base(reinterpret_cast<const char*>(p) + (seq * sb + at * sr + first) * (long long)sizeof(S)),
          off((unsigned(lane_row) * unsigned(sr) + unsigned(lane_elem)) * unsigned(sizeof(S))),
          row(sr * (long long)sizeof(S)) {}
    // `t` positions after the lane's first
    __device__ __forceinline__ const S* at(int t) const { return reinterpret_cast<const S*>(base + t * row + off); }
    __device__ __forceinline__ S* to(int t) const { return const_cast<S*>(at(t)); }
    __device__ __forceinline__ void move(int t) { base += t * row; }
};

// What a load gives, before it is widened, in a register of its own (two 16-bit values
// would be packed into one as they arrive): a load that is issued a tile ahead is not
// waited for until its value is used.
template <class D>
__device__ __forceinline__ uint32_t load_raw(const typename D::S* p) {
    if constexpr (D::kBytes == 4) return __builtin_bit_cast(uint32_t, *p);
    else return *p;
}
template <class D>
__device__ __forceinline__ float widen(uint32_t v) {
    if constexpr (D::kBytes == 4) return __builtin_bit_cast(float, v);
    else return D::widen(v);
}

// Has the value formed here, and not where it is first used: the register that it is
// formed from is loaded into again meanwhile, and would have to be copied, for which
// the load is waited for.
__device__ __forceinline__ void now(float& v) { asm volatile("" : "+v"(v)); }

// Before a loop whose turns load ahead: all loads are there.  The compiler counts what
// is in flight at the loop's start, and would otherwise wait in every turn as if it
// were the first.
__device__ __forceinline__ void loads_done() { __builtin_amdgcn_s_waitcnt(0x0f70); }

// A lane's states of one position.
template <class D, int NP>
struct States {
    uint32_t v[NP];
    template <class F>
    __device__ __forceinline__ void load(const typename D::S* p, const Lane<F>& l) {
#pragma unroll
        for (int j = 0; j < NP; ++j) v[j] = load_raw<D>(p + l.at[j]);
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int j = 0; j < NP; ++j) v[j] = 0;
    }
    __device__ __forceinline__ float operator[](int j) const { return widen<D>(v[j]); }
};

// A thread's elements of a tile; `rows` starts at its first one.
template <class D, class F>
struct Column {
    uint32_t v[F::kSlots];
    // all that there are, of a whole tile
    __device__ __forceinline__ void load(const Rows<typename D::S>& rows, bool last_slot) {
#pragma unroll
        for (int q = 0; q < F::kSlots; ++q)
            if ((q + 1) * F::kStep <= 16 || last_slot) v[q] = load_raw<D>(rows.at(F::kStep * q));
    }
    // those before position `valid`, counted from the thread's first
    __device__ __forceinline__ void load_some(const Rows<typename D::S>& rows, bool last_slot, int valid) {
#pragma unroll
        for (int q = 0; q < F::kSlots; ++q)
            v[q] = F::kStep * q < valid && ((q + 1) * F::kStep <= 16 || last_slot) ? load_raw<D>(rows.at(F::kStep * q)) : 0;
    }
    __device__ __forceinline__ float operator[](int k) const { return widen<D>(v[k]); }
};

// The saved states of a chunk: each wavefront's as it holds them, one after the other.
template <class F>
__device__ __forceinline__ long long saved_at(const Args& a, const Lane<F>& l, int chunk) {
    const long long unit = ((long long)chunk * a.B + l.seq) * (a.G * a.tiles) + l.group * a.tiles + l.tile;
    return (unit * (F::CT * F::NB) + (l.ct * F::NB + l.nb)) * (F::NP * 64) + l.lane;
}

// The sum of v over the threads that have elements of a channel, for the first
// kChannels threads; `lds` holds kThreads values.
template <class F>
__device__ __forceinline__ float over_channel(float v, float* lds) {
    lds_barrier();
    lds[threadIdx.x] = v;
    lds_barrier();
    v = 0.f;
    if (threadIdx.x < F::kChannels)
        for (int k = threadIdx.x; k < F::kThreads; k += F::kChannels) v += lds[k];
    return v;
}

}  // namespace ssc

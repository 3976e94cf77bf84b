// Internal interface between the C-ABI front end of the gated linear
// recurrence (gscan_api.cpp) and its kernels.  Not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <type_traits>

#include "gscan.h"
#include "gscan_carry.h"

namespace gsc {

// One call, as the kernels take it.
struct Args {
    const void *x, *r, *i, *dh;
    void *h, *dx, *dr, *di;
    long long x_sb, x_sr, r_sb, r_sr, i_sb, i_sr, dh_sb, dh_sr;
    long long h_sb, h_sr, dx_sb, dx_sr, dr_sb, dr_sr, di_sb, di_sr;
    const float *lam, *h0, *dh_last;
    const int* lengths;
    float *h_last, *states, *dlam, *dh0;
    float* part;  // partial sums of dlam, [parts][C]
    Carry carry;  // where tiles are spread over workgroups
    int B, C, T, tiles;
    float decay;
};

struct Plan {
    int tiles;       // tiles along time (at least 1); the states are [tiles][B][C]
    long long parts;  // rows of partial sums of dlam
    size_t states;   // bytes
    size_t scratch;  // bytes of workspace
    bool fits;       // one launch holds the call's threads
};
constexpr long long kMaxThreads = 1LL << 32;  // a launch holds fewer

Plan planes_plan(const gscan_shape& s);
hipError_t planes_fwd(const gscan_shape& s, Args a, void* ws, hipStream_t st);
hipError_t planes_bwd(const gscan_shape& s, Args a, void* ws, hipStream_t st);

Plan tokens_plan(const gscan_shape& s);
hipError_t tokens_fwd(const gscan_shape& s, Args a, void* ws, hipStream_t st);
hipError_t tokens_bwd(const gscan_shape& s, Args a, void* ws, hipStream_t st);

// dlam from `parts` rows of partial sums, added in order in fp64.
hipError_t close_dlam(const Args& a, long long parts, hipStream_t st);

hipError_t step(int B, int C, int S, int dtype, float decay, const gscan_view& x,
                const gscan_view& r, const gscan_view& i, const float* lam, float* state,
                const int* slots, const gscan_view& h, hipStream_t st);

}  // namespace gsc

// Internal interface between the C-ABI front end of the selective scan
// (sscan_api.cpp) and its kernels.  Not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "sscan.h"

namespace ssc {

constexpr int kChunk = 16;  // positions between two saved states

// One call, as the kernels take it.
struct Args {
    const void *x, *dt, *b, *c, *z, *dy;
    void *y, *dx, *ddt, *db, *dc, *dz;
    long long x_sb, x_sr, dt_sb, dt_sr, b_sb, b_sr, c_sb, c_sr, z_sb, z_sr, dy_sb, dy_sr;
    long long y_sb, y_sr, dx_sb, dx_sr, ddt_sb, ddt_sr, db_sb, db_sr, dc_sb, dc_sr, dz_sb, dz_sr;
    const float *a_log, *d, *dt_bias, *h0, *dh_last;
    const int* lengths;
    float *h_last, *states, *da_log, *dd, *ddt_bias, *dh0;
    // where a sequence is cut into S segments of `seg` positions: what each does to a state
    float *seg_state, *seg_sum;  // [S][B][D][N] from zero; [S][B][D] sums of delta
    // partial sums of the backward pass
    float* part_bc;  // [tiles of a group][B][T][G][2][waves * 4 * per_lane]
    float *part_a, *part_d, *part_bias;  // [B * S][D][N], [B * S][D] twice
    int B, T, D, N, G;
    int Dg, tiles;  // channels of a group, and workgroups for them
    int S, seg;
};

struct Plan {
    int per_lane;      // states that a lane holds: 1, 2 or 4
    int waves;         // wavefronts that the states of 16 channels are divided among
    int width, tiles;  // channels of a workgroup, and workgroups for a group's
    int S, seg;        // segments of a sequence, and their length
    size_t states;     // bytes
    size_t scratch;    // bytes of workspace
    bool fits;
};

Plan plan(const sscan_shape& s, bool backward);
hipError_t fwd(const sscan_shape& s, Args a, void* ws, hipStream_t st);
hipError_t bwd(const sscan_shape& s, Args a, void* ws, hipStream_t st);
// the parameters' gradients of no position at all
hipError_t bwd_empty(const sscan_shape& s, const Args& a, hipStream_t st);

struct StepArgs {
    const void *x, *dt, *b, *c, *z;
    void* y;
    long long x_sb, dt_sb, b_sb, c_sb, z_sb, y_sb;
    const float *a_log, *d, *dt_bias;
    float* state;
    const int* slots;
    int B, D, N, G, Dg, S;
    int first;  // sequence of the launch
};
hipError_t step(int dtype, const StepArgs& a, hipStream_t st);

}  // namespace ssc

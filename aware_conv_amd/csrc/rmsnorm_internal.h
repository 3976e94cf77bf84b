// Internal interface between the C-ABI front end of the root-mean-square norm
// (rmsnorm_api.cpp) and its kernels.  Not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>

#include "rmsnorm.h"

namespace rmn {

struct Args {
    const void *x, *res, *kept, *dy, *dtotal;
    void *y, *total, *dx, *dres;
    long long x_sb, x_sr, res_sb, res_sr, kept_sb, kept_sr, dy_sb, dy_sr, dtotal_sb, dtotal_sr;
    long long y_sb, y_sr, total_sb, total_sr, dx_sb, dx_sr, dres_sb, dres_sr;
    const float *w, *rstd_in;
    float *rstd, *scale, *dw, *part;  // part: [parts][C] partial sums of dw
    int T, C;
    long long rows;
    float eps;
};

struct Plan {
    int threads, vectors;  // of a row: threads, and vectors of 8 elements in registers of each (0: read again)
    int per_block;         // rows that a workgroup works on at a time
    unsigned parts;        // workgroups of the backward pass
    size_t scratch;        // bytes of workspace
};
Plan plan(const rmsnorm_shape& s);
hipError_t fwd(const rmsnorm_shape& s, const Args& a, bool e4m3, hipStream_t st);
hipError_t bwd(const rmsnorm_shape& s, Args a, void* ws, hipStream_t st);

}  // namespace rmn

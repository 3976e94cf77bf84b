// Internal interface between the C-ABI front end of the causal convolution
// (cconv_api.cpp) and its kernels.  Not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>

#include "cconv.h"

namespace ccv {

struct Args {
    const void *x, *dy;
    void *y, *dx;
    long long x_sb, x_sr, y_sb, y_sr, dy_sb, dy_sr, dx_sb, dx_sr;
    const float *w, *bias;
    const void *h0, *dlast;
    void *last, *dh0;
    const int* lengths;
    float *dw, *dbias;
    float* part;  // [parts][C][K] and, behind, [parts][C]
    int B, T, C, K, silu;
};

struct Plan {
    long long parts;  // of the sums over positions
    size_t scratch;   // bytes of workspace
    bool fits;
};
Plan plan(const cconv_shape& s);
hipError_t fwd(int dtype, const Args& a, hipStream_t st);
hipError_t bwd(const cconv_shape& s, Args a, void* ws, hipStream_t st);

struct StepArgs {
    const void* x;
    void* y;
    long long x_sb, y_sb;
    const float *w, *bias;
    void* cache;
    const int* slots;
    int B, C, K, S, silu;
};
hipError_t step(int dtype, const StepArgs& a, hipStream_t st);

}  // namespace ccv

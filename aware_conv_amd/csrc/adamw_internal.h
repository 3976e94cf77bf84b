// Internal interface between the C-ABI front end of the AdamW step
// (adamw_api.cpp) and its kernels.  Not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>

#include "adamw.h"

namespace adw {

// What the kernels of one step share, formed on the device by the first of them.
struct Ctl {
    double scale;  // of the gradients, clipping included
    float factor;  // the same in fp32 operations, for what is held in 8 bits
    float drop;    // lr * weight_decay
    float rate;    // lr / (1 - beta1^t)
    float root;    // 1 / sqrt(1 - beta2^t)
    unsigned turn;  // t's part of the dither
    int on;        // 0: the step is left out
};

constexpr size_t kCtlBytes = 64;
constexpr long long kNormChunk = 8192;  // elements of a partial sum of squares

hipError_t grad_norm(int dtype, const adamw_tensor* t, int count, double scale,
                     const float* scale_dev, float* norm, double* part, hipStream_t st);
hipError_t step(const adamw_config& c, const adamw_tensor* t, int count, int* step, Ctl* ctl,
                hipStream_t st);

}  // namespace adw

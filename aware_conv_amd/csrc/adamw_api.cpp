// C-ABI front end of the AdamW step: argument checks (before anything is
// enqueued), then the kernels.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "adamw.h"
#include "adamw_internal.h"

namespace {

constexpr long long kMaxElements = 1LL << 34;  // of a tensor: it fits one launch

size_t elem_size(int dtype) { return dtype == ADAMW_F32 ? 4 : 2; }
bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
int hip_status(hipError_t e) { return e == hipSuccess ? WTCONV_OK : WTCONV_ERR_HIP; }

int check_dtype(int dtype) {
    return dtype == ADAMW_F32 || dtype == ADAMW_F16 || dtype == ADAMW_BF16 ? WTCONV_OK
                                                                          : WTCONV_ERR_DTYPE;
}

int check_list(const adamw_tensor* t, int count) {
    if (count < 0) return WTCONV_ERR_SHAPE;
    if (count > 0 && !t) return WTCONV_ERR_NULL;
    for (int i = 0; i < count; ++i)
        if (t[i].n < 0 || t[i].n > kMaxElements) return WTCONV_ERR_SHAPE;
    return WTCONV_OK;
}

size_t workspace(const adamw_tensor* t, int count) {
    size_t parts = 0;
    for (int i = 0; i < count; ++i)
        parts += size_t((t[i].n + adw::kNormChunk - 1) / adw::kNormChunk);
    const size_t bytes = parts * sizeof(double);
    return bytes > adw::kCtlBytes ? bytes : adw::kCtlBytes;
}

int check_ws(const adamw_tensor* t, int count, const void* ws, size_t bytes) {
    if (bytes < workspace(t, count)) return WTCONV_ERR_WORKSPACE;
    if (!ws) return WTCONV_ERR_NULL;
    return aligned(ws, 16) ? WTCONV_OK : WTCONV_ERR_ALIGN;
}

int check_ptr(const void* p, size_t e) {
    if (!p) return WTCONV_ERR_NULL;
    return aligned(p, e) ? WTCONV_OK : WTCONV_ERR_ALIGN;
}

bool unit(double v) { return v >= 0.0 && v < 1.0; }

}  // namespace

extern "C" {

int adamw_workspace_size(const adamw_tensor* tensors, int count, size_t* bytes) {
    const int rc = check_list(tensors, count);
    if (rc) return rc;
    if (!bytes) return WTCONV_ERR_NULL;
    *bytes = workspace(tensors, count);
    return WTCONV_OK;
}

int adamw_grad_norm(int dtype, const adamw_tensor* tensors, int count, double grad_scale,
                    const float* grad_scale_dev, float* norm, void* workspace, size_t ws_bytes,
                    void* stream) {
    int rc = check_dtype(dtype);
    if (rc || (rc = check_list(tensors, count))) return rc;
    if (!isfinite(grad_scale)) return WTCONV_ERR_VALUE;
    for (int i = 0; i < count; ++i)
        if (tensors[i].n > 0 && (rc = check_ptr(tensors[i].g, elem_size(dtype)))) return rc;
    if ((rc = check_ptr(norm, 4))) return rc;
    if (!aligned(grad_scale_dev, 4)) return WTCONV_ERR_ALIGN;
    if ((rc = check_ws(tensors, count, workspace, ws_bytes))) return rc;
    return hip_status(adw::grad_norm(dtype, tensors, count, grad_scale, grad_scale_dev, norm,
                                     static_cast<double*>(workspace),
                                     static_cast<hipStream_t>(stream)));
}

int adamw_step(const adamw_config* config, const adamw_tensor* tensors, int count, int* step,
               void* workspace, size_t ws_bytes, void* stream) {
    if (!config) return WTCONV_ERR_NULL;
    const adamw_config& c = *config;
    int rc = check_dtype(c.dtype);
    if (rc || (rc = check_list(tensors, count))) return rc;
    if (c.bits != 8 && c.bits != 32) return WTCONV_ERR_DTYPE;
    if (!unit(c.beta1) || !unit(c.beta2) || !(c.eps >= 0.0) || !isfinite(c.eps) ||
        !isfinite(c.lr) || !isfinite(c.weight_decay) || !isfinite(c.grad_scale) ||
        !(c.max_norm >= 0.0) || !isfinite(c.max_norm))
        return WTCONV_ERR_VALUE;
    if (c.max_norm > 0 && !c.norm) return WTCONV_ERR_NULL;
    const size_t e = elem_size(c.dtype), es = c.bits == 8 ? 1 : 4;
    int with = 0, without = 0;  // tensors with a master copy
    for (int i = 0; i < count; ++i) {
        const adamw_tensor& t = tensors[i];
        if (t.n == 0) continue;
        if ((rc = check_ptr(t.p, e)) || (rc = check_ptr(t.g, e)) || (rc = check_ptr(t.m, es)) ||
            (rc = check_ptr(t.v, es)))
            return rc;
        if (c.bits == 8 && ((rc = check_ptr(t.ms, 4)) || (rc = check_ptr(t.vs, 4)))) return rc;
        if (t.w && (rc = check_ptr(t.w, 4))) return rc;
        ++(t.w ? with : without);
    }
    if (with && without) return WTCONV_ERR_NULL;
    if ((rc = check_ptr(step, 4))) return rc;
    if (!aligned(c.lr_dev, 4) || !aligned(c.grad_scale_dev, 4) || !aligned(c.norm, 4))
        return WTCONV_ERR_ALIGN;
    if ((rc = check_ws(tensors, count, workspace, ws_bytes))) return rc;
    return hip_status(adw::step(c, tensors, count, step, static_cast<adw::Ctl*>(workspace),
                                static_cast<hipStream_t>(stream)));
}

}  // extern "C"

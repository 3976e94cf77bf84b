/*
 * adamw.h -- C ABI of one AdamW step over many tensors at once, with the
 * moments held in 32 bits or in 8, and of the global gradient norm that clips
 * it, for AMD Instinct MI355X (gfx950).
 *
 * For every element, with the gradient g already multiplied by grad_scale and
 * by the clipping factor below (Loshchilov and Hutter, "Decoupled Weight Decay
 * Regularization", arXiv 1711.05101, algorithm 2), t counting from 1:
 *
 *   m = beta1 m + (1 - beta1) g          v = beta2 v + (1 - beta2) g^2
 *   p = p (1 - lr weight_decay) - lr (m / (1 - beta1^t)) / (sqrt(v / (1 - beta2^t)) + eps)
 *
 * The arithmetic is fp32; p and g are of `dtype`.  A tensor may have a master
 * copy w of its parameters in fp32: then w is updated and p is w, rounded.
 * Without one, a 16-bit p is updated in fp32 and rounded, to nearest even.
 *
 * bits = 32: m and v are fp32.  bits = 8: m and s = sqrt(v) are held as e4m3
 * codes (the OCP format with 448 as its largest value) with one fp32 scale for
 * each ADAMW_BLOCK consecutive elements of a tensor, the last block shorter;
 * value = code * scale.  The update uses the new m and v before they are held.
 *
 * A code depends on the last bit of what it is formed from, so with bits = 8
 * codes and scales are defined to that bit.  Each operation below is in fp32 and
 * rounded to nearest even by itself, each coefficient is the fp32 nearest to its
 * value, and g is the gradient as stored:
 *
 *   f = grad_scale * min(1, max_norm / (norm + 1e-6))   (grad_scale without clipping)
 *   g = g f    m = beta1 (code scale) + (1 - beta1) g
 *   r = code scale    s = sqrt(beta2 (r r) + ((1 - beta2) g) g)
 *   scale = T (1/448)    x = |value| (1 / scale)        (T: the block's largest |value|)
 *   u = x's step to the next code, a power of two       code = floor(x / u + d) u, at most 448
 *
 * That is, x is rounded down to a code if the fraction of the step to the next
 * code that it has covered, plus a dither d in [0, 1), stays below 1, else up; so
 * its mean over the steps is x, and moments move that change by less than half a
 * step at a time.  This holds for T too, whose x is 448 or, by the roundings of
 * its scale, up to two units in the last place less: then a d below 2^-20 takes
 * it to 416.  No generator is involved:
 *
 *   d = (((k * 2654435769 + t * 3242174889 + turn) mod 2^32) >> 8) / 2^24
 *
 * for element k of its tensor at step t; turn is 0 for m and 2^31 for s
 * (multiples of the golden ratio and of the inverse plastic number, whose
 * sequences fill the unit interval evenly).  An s that is not 0 takes the
 * lowest code rather than 0, so that no element divides by eps alone.  Blocks
 * whose scale is below 2^-126 are held as zeros.  A moment that is not finite is
 * held as NaN and leaves the rest of its block alone.  The parameter moves by m
 * and s to fp32 accuracy, as with bits = 32; its last bits are not defined.
 *
 * Ownership, threading, streams and error codes are those of wtconv.h.  The
 * tensor lists are host arrays and are read before the call returns; any
 * alignment of an element is taken; tensors may not overlap.  Everything that
 * changes from step to step is read on the device, so both calls can be
 * captured into a graph.  Results do not depend on timing.
 */
#ifndef ADAMW_H
#define ADAMW_H

#include <stddef.h>

#include "wtconv.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { ADAMW_F32 = 0, ADAMW_F16 = 1, ADAMW_BF16 = 2 } adamw_dtype;

#define ADAMW_BLOCK 256

typedef struct {
    void* p;       /* parameters, n of dtype */
    const void* g; /* gradient, n of dtype */
    float* w;      /* master parameters, n; for every tensor of a call or for none (NULL) */
    void* m;       /* n fp32, or n codes */
    void* v;       /* n fp32, or n codes of sqrt(v) */
    float* ms;     /* bits = 8: scales of m, ceil(n / ADAMW_BLOCK) */
    float* vs;     /* bits = 8: scales of sqrt(v) */
    long long n;
} adamw_tensor;

typedef struct {
    int dtype; /* adamw_dtype of p and g */
    int bits;  /* 32 or 8 */
    double lr, beta1, beta2, eps, weight_decay;
    double grad_scale; /* gradients are multiplied by it (1 / loss scale) */
    double max_norm;   /* > 0: clip, with `norm`; 0: do not */
    /* device values, each may be NULL: */
    const float* lr_dev;         /* used in place of lr */
    const float* grad_scale_dev; /* used in place of grad_scale */
    const float* norm;           /* global norm of grad_scale * g over every tensor of the step */
} adamw_config;

/* Bytes of device workspace both calls need for these tensors. */
int adamw_workspace_size(const adamw_tensor* tensors, int count, size_t* bytes);

/*
 * *norm = grad_scale * the 2-norm of all gradients together (g and n of each
 * tensor are used), summed in fp64 in a fixed order.
 */
int adamw_grad_norm(int dtype, const adamw_tensor* tensors, int count, double grad_scale,
                    const float* grad_scale_dev, float* norm, void* workspace, size_t ws_bytes,
                    void* stream);

/*
 * One step over all tensors.  *step (device) is the number of steps taken so
 * far; it is advanced.  With config->norm, gradients are also multiplied by
 * min(1, max_norm / (norm + 1e-6)) where max_norm > 0, and a norm that is not
 * finite leaves every tensor and *step as they are.
 */
int adamw_step(const adamw_config* config, const adamw_tensor* tensors, int count, int* step,
               void* workspace, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ADAMW_H */

/*
 * rmsnorm.h -- C ABI of the root-mean-square norm with the residual's addition
 * for AMD Instinct MI355X (gfx950), in the activations' type or in 8 bits.
 *
 * Per row of C elements (Zhang and Sennrich, arXiv 1910.07467):
 *
 *   s = x + residual                  rounded to the residual's type: `total` (s = x without it)
 *   rstd = 1 / sqrt(mean(s^2) + eps)
 *   y = s rstd w
 *
 * What is normed is the rounded sum, which later layers read and the backward
 * pass is given.  In 8 bits, with one scale per row:
 *
 *   scale = max |y| / 448             codes = y (1 / scale) in e4m3, to nearest even
 *
 * (a row whose scale would be below 2^-126 has scale 0 and codes 0, a row of no
 * elements rstd NaN and scale 0; a NaN has the code NaN).  A code depends on the last bit of what it is formed from, so codes and
 * scales are defined to that bit from rstd: each operation, (s rstd) w and the
 * others as written, is in fp32 and rounded to nearest even by itself, and a product
 * beyond 448 is taken as 448.  The inverse and the product are rounded once each, so
 * that y / scale may lie within 2^-23 of itself of a tie between two codes and have
 * the further one (one value in a million; a division instead took 8% of the call for
 * 16384 rows of 4096 bf16 with a residual, 19% without).
 *
 * Gradients, for dy of y and dtotal of `total`, with n = s rstd:
 *
 *   g = dy w       ds = rstd (g - n mean(g n)) + dtotal       dw = sum over rows of dy n
 *
 * and ds is the gradient of x and of the residual alike.
 *
 * Rows are [B][T][C] gscan_views: a pointer, the stride of the batch and the
 * stride of a row, in elements; elements within a row are adjacent, and any
 * alignment of an element is taken.  x, y, dy and dx are `dtype`; residual,
 * total, dtotal and dresidual are `rdtype`, which is `dtype` or GSCAN_F32.  w [C],
 * rstd [B][T], scale [B][T] and dw [C] are fp32 and contiguous.
 *
 * Arithmetic is fp32, each output is rounded once, to nearest even; dw is closed
 * in fp64, and every sum is taken in a fixed order: results are bitwise
 * reproducible for a given shape.
 *
 * Ownership, threading, streams, overlaps and error codes are those of sscan.h;
 * `total` may be the residual's own buffer.
 */
#ifndef RMSNORM_H
#define RMSNORM_H

#include <stddef.h>

#include "gscan.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    int B, T, C;       /* B * T rows of C elements (C <= 2^20) */
    int dtype, rdtype; /* gscan_dtype of the activations, and of the residual stream */
    float eps;         /* >= 0, finite */
} rmsnorm_shape;

/* Sizes: B * T up to 2^31 - 1 rows (WTCONV_ERR_SHAPE beyond). */

/* Bytes of device workspace that rmsnorm_bwd needs (the forward needs none). */
int rmsnorm_workspace_size(const rmsnorm_shape* s, size_t* bytes);

/* residual and total are both given or both NULL; rstd may be NULL (not wanted). */
int rmsnorm_fwd(const rmsnorm_shape* s, const gscan_view* x, const gscan_view* residual,
                const float* w, const gscan_view* y, const gscan_view* total, float* rstd,
                void* stream);

/* The same with codes (a view of bytes) and scales for y. */
int rmsnorm_fwd_e4m3(const rmsnorm_shape* s, const gscan_view* x, const gscan_view* residual,
                     const float* w, const gscan_view* codes, float* scale,
                     const gscan_view* total, float* rstd, void* stream);

/*
 * Gradients from what was normed (`kept`, of rdtype: total, or x where there was
 * no residual) and rstd.  dtotal may be NULL (zeros).  dx (dtype) or dresidual
 * (rdtype) may be NULL (not wanted), dw too.
 */
int rmsnorm_bwd(const rmsnorm_shape* s, const gscan_view* kept, const float* w, const float* rstd,
                const gscan_view* dy, const gscan_view* dtotal, const gscan_view* dx,
                const gscan_view* dresidual, float* dw, void* workspace, size_t ws_bytes,
                void* stream);

#ifdef __cplusplus
}
#endif

#endif /* RMSNORM_H */

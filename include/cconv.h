/*
 * cconv.h -- C ABI of a short causal depthwise convolution over token
 * sequences for AMD Instinct MI355X (gfx950), as it stands before a selective
 * state space scan (sscan.h).
 *
 * Per sequence and channel c, with K taps (1..8) and the K - 1 inputs before
 * the first position in h0 (zeros without it), at position t:
 *
 *   v_t = bias[c] + sum_k w[c][k] x_{t-K+1+k}         y_t = silu(v_t), or v_t
 *
 * and `last` holds the K - 1 inputs up to the end, oldest first, from which the
 * sequence can be continued.  Gradients, for dy_t of y_t and dlast of `last`:
 *
 *   dv_t = dy_t silu'(v_t)                            dx_t = sum_k w[c][k] dv_{t+K-1-k} (+ dlast)
 *   dw[c][k] = sum_{b,t} dv_t x_{t-K+1+k}             dbias[c] = sum_{b,t} dv_t
 *
 * dh0 is dx of the inputs in h0.
 *
 * x, y, dy and dx are gscan_views [B][T][C] of `dtype`: a pointer, the stride of
 * the batch and the stride of a position, in elements; channels are adjacent.
 * Any alignment of an element is taken.  h0, last, dlast and dh0 are
 * [B][K-1][C] of `dtype`, w [C][K] and bias [C] and their gradients fp32, all
 * contiguous.  bias and h0 may be NULL.
 *
 * lengths, where given, holds B int32 values in device memory: sequence b has
 * lengths[b] valid positions, its first (values outside 0..T are taken as the
 * nearer end).  y and dx are zero beyond them, and x and dy are not read there.
 *
 * Arithmetic is fp32, each output is rounded once, to nearest even; `last` is
 * copied.  Sums over positions are taken in a fixed order, and closed in fp64:
 * results are bitwise reproducible for a given shape.
 *
 * Ownership, threading, streams, overlaps and error codes are those of sscan.h.
 */
#ifndef CCONV_H
#define CCONV_H

#include <stddef.h>

#include "gscan.h"

#ifdef __cplusplus
extern "C" {
#endif

#define CCONV_MAX_TAPS 8

typedef struct {
    int B, T, C, K; /* sequences, positions (T <= 2^30), channels, taps (1..8) */
    int dtype;      /* gscan_dtype of the activations */
    int silu;       /* 0: y = v, otherwise y = silu(v) */
} cconv_shape;

/*
 * Sizes: B * C up to 2^31, C * K up to 2^27 (WTCONV_ERR_SHAPE beyond).  What one
 * launch does not hold is refused with WTCONV_ERR_UNSUPPORTED:
 * B * ceil(C / 128) * (ceil(T / 128) + 1) has to be below 2^24, and so has, for
 * cconv_bwd with a bias, ceil(C * K / 16) + ceil(C / 16).
 */

/* Bytes of device workspace that cconv_bwd needs (cconv_fwd needs none). */
int cconv_workspace_size(const cconv_shape* s, size_t* bytes);

/* y and `last` (NULL: not wanted; it is empty for K = 1). */
int cconv_fwd(const cconv_shape* s, const gscan_view* x, const float* w, const float* bias,
              const void* h0, const int* lengths, const gscan_view* y, void* last, void* stream);

/* Every gradient; dlast may be NULL (zeros), dh0 may be NULL (not wanted), dbias
 * is NULL where bias is.  Gradients are overwritten. */
int cconv_bwd(const cconv_shape* s, const gscan_view* x, const float* w, const float* bias,
              const void* h0, const int* lengths, const gscan_view* dy, const void* dlast,
              const gscan_view* dx, float* dw, float* dbias, void* dh0, void* workspace,
              size_t ws_bytes, void* stream);

/*
 * One position of B sequences whose last K - 1 inputs live in a cache
 * [S][K-1][C] of `dtype`: cache[slots[b]] is read, moved on by x[b] and written
 * back, and y[b] follows.  slots (int32, device) may be NULL: sequence b uses
 * row b, and S must be at least B.  A sequence whose slot is outside 0..S-1 is
 * passed over: its y is zero and no row changes.  Slots that repeat give
 * undefined rows.  T of the shape is not used.  The views are [B][C]: sb is the
 * row stride, sr is not used.
 */
int cconv_step(const cconv_shape* s, int S, const gscan_view* x, const float* w, const float* bias,
               void* cache, const int* slots, const gscan_view* y, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* CCONV_H */

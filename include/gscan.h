/*
 * gscan.h -- C ABI of a gated linear recurrence over long sequences for AMD
 * Instinct MI355X (gfx950): a mixer over a whole plane or token sequence, to
 * stand beside the local mixing of the WTConv layer.
 *
 * Per sequence b and channel c, with the gates r, i and the input x at each
 * position t (the real-gated linear recurrent unit of De et al., "Griffin",
 * arXiv 2402.19427, section 2.4):
 *
 *   L_t = -decay * softplus(lam[c]) * sig(r_t)          a_t = exp(L_t)
 *   w_t = sqrt(1 - a_t^2)                               (from expm1: no cancellation)
 *   h_t = a_t * h_{t-1} + w_t * sig(i_t) * x_t          h_{-1} = h0[b,c], or 0
 *
 * Gradients, for dh_t of h_t and dh_last of the last state:
 *
 *   g_t = dh_t + a_{t+1} g_{t+1}                        (dh_last joins the last g)
 *   dx_t = g_t w_t sig(i_t)
 *   di_t = g_t w_t x_t sig(i_t) sig(-i_t)
 *   e_t = g_t (a_t h_{t-1} - sig(i_t) x_t a_t^2 / w_t)  (the gradient of L_t; the second
 *                                                        term is 0 where w_t = 0)
 *   dr_t = e_t L_t sig(-r_t)
 *   dlam[c] = -decay sig(lam[c]) * sum_{b,t} e_t sig(r_t)        dh0 = a_0 g_0
 *
 * Layouts (`layout`): GSCAN_BCT, [B][C][T] with time contiguous -- NCHW planes
 * with H*W = T, in raster order -- or GSCAN_BTC, [B][T][C] with channels
 * contiguous.  Every activation is a gscan_view: a pointer, the stride of the
 * batch and the stride of a row (of a channel in BCT, of a position in BTC),
 * in elements; elements within a row are adjacent.  x, r and i may so be parts
 * of one projection, and dx, dr and di parts of its gradient.  Any alignment
 * of an element is taken.
 *
 * reverse != 0 runs the recurrence from the last position to the first.
 *
 * lengths, where given, holds B int32 values in device memory: sequence b has
 * lengths[b] valid positions (values outside 0..T are taken as the nearer
 * end), its first ones in memory, in either direction.  h, dx, dr and di are
 * zero beyond them, what x, r, i and dh hold there is not read, and the last
 * state is that after the valid positions (h0 where there are none).
 *
 * lam, h0, h_last, dh_last, dh0, dlam and the states are fp32; [C] or [B][C],
 * contiguous.  Activations are `dtype`.  Arithmetic is fp32 throughout: each
 * output is rounded once, to nearest even; sums over positions of one state
 * or gradient are taken in a fixed order and dlam is closed in fp64, so
 * results are bitwise reproducible for a given shape.
 *
 * Ownership, threading, streams and error codes are those of wtconv.h: the
 * caller owns every buffer, the calls only enqueue kernels on `stream`, keep
 * nothing, and can be captured into a graph.  An output may not overlap an
 * input, another output, the states or the workspace (views that interleave
 * within one buffer, of the same strides and with no element in common, are
 * taken), nor itself.
 */
#ifndef GSCAN_H
#define GSCAN_H

#include <stddef.h>

#include "wtconv.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { GSCAN_F32 = 0, GSCAN_F16 = 1, GSCAN_BF16 = 2 } gscan_dtype;
typedef enum { GSCAN_BCT = 0, GSCAN_BTC = 1 } gscan_layout;

typedef struct {
    int B, C, T;  /* sequences, channels, positions (T <= 2^30) */
    int layout;   /* gscan_layout of every activation */
    int dtype;    /* gscan_dtype of every activation */
    int reverse;  /* 0: forwards in memory, otherwise backwards */
    float decay;  /* > 0, finite (8 in the published form) */
} gscan_shape;

typedef struct {
    void* p;          /* element [0][0][0] */
    long long sb, sr; /* strides of the batch and of a row, in elements, >= 0 */
} gscan_view;

/*
 * Sizes: T up to 2^30, B * C up to 2^25 (WTCONV_ERR_SHAPE beyond).  What one
 * launch does not hold is refused with WTCONV_ERR_UNSUPPORTED: tokens unless
 * ceil(C / 64) * B * ceil(T / 256) is below 2^23 (2^31 positions of up to 64
 * channels), and planes of up to 1024 rows (B * C) unless B * C *
 * ceil(T / 4096) is below 2^23 (2^35 positions).  Planes of more rows are
 * taken, whatever their length, and so are single positions.
 */

/* Bytes of the states gscan_fwd writes for gscan_bwd (what h held before each
 * of the tiles the kernels walk in). */
int gscan_states_size(const gscan_shape* s, size_t* bytes);

/* Bytes of device workspace gscan_fwd and gscan_bwd need (the maximum of both). */
int gscan_workspace_size(const gscan_shape* s, size_t* bytes);

/*
 * h and h_last from x, r, i, lam and h0 (NULL: zeros); lengths may be NULL.
 * states: gscan_states_size() bytes, or NULL where no gradient is wanted.
 * h_last may be NULL.
 */
int gscan_fwd(const gscan_shape* s, const gscan_view* x, const gscan_view* r,
              const gscan_view* i, const float* lam, const float* h0, const int* lengths,
              const gscan_view* h, float* h_last, float* states, void* workspace,
              size_t ws_bytes, void* stream);

/*
 * Every gradient from the inputs of gscan_fwd, the states it wrote and dh;
 * dh_last may be NULL (zeros), dh0 may be NULL (not wanted).  h is not needed:
 * it is formed again from the states.  Gradients are overwritten.
 */
int gscan_bwd(const gscan_shape* s, const gscan_view* x, const gscan_view* r,
              const gscan_view* i, const float* lam, const float* states, const int* lengths,
              const gscan_view* dh, const float* dh_last, const gscan_view* dx,
              const gscan_view* dr, const gscan_view* di, float* dlam, float* dh0,
              void* workspace, size_t ws_bytes, void* stream);

/*
 * One position of B sequences whose states live in a cache [S][C] fp32:
 * state[slots[b]] is read, advanced and written back, and h[b] is its rounded
 * value.  slots (int32, device) may be NULL: sequence b uses row b, and S must
 * be at least B.  A sequence whose slot is outside 0..S-1 is passed over: its h
 * is zero and no state changes.  Slots that repeat give undefined states.
 * The views are [B][C]: sb is the row stride, sr is not used.
 */
int gscan_step(int B, int C, int S, int dtype, float decay, const gscan_view* x,
               const gscan_view* r, const gscan_view* i, const float* lam, float* state,
               const int* slots, const gscan_view* h, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GSCAN_H */

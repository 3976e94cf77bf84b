/*
 * sscan.h -- C ABI of a selective state space scan over token sequences for
 * AMD Instinct MI355X (gfx950): a recurrence whose step, input and output maps
 * depend on the token, with N states per channel (Gu and Dao,
 * arXiv 2312.00752, section 3).
 *
 * Per sequence, channel d of group k = d / (D / G) and state n, at position t:
 *
 *   delta_t = softplus(dt_t + dt_bias[d])        A = -exp(a_log[d][n])
 *   h_t[n]  = exp(delta_t A) h_{t-1}[n] + delta_t x_t b_t[k][n]     h_{-1} = h0, or 0
 *   s_t     = sum_n c_t[k][n] h_t[n] + d[d] x_t
 *   y_t     = s_t silu(z_t)                      silu(v) = v sig(v); y_t = s_t without z
 *
 * Gradients, for dy_t of y_t and dh_last of the last state:
 *
 *   ds_t = dy_t silu(z_t)                        dz_t = dy_t s_t silu'(z_t)
 *   g_t  = ds_t c_t + exp(delta_{t+1} A) g_{t+1}             (dh_last joins the last g)
 *   db_t = sum_{d in k} g_t delta_t x_t          dc_t = sum_{d in k} ds_t h_t
 *   q_t  = g_t exp(delta_t A) h_{t-1}            w_t = sum_n g_t b_t
 *   dx_t = delta_t w_t + d ds_t                  ddt_t = (sum_n A q_t + x_t w_t) sig(dt_t + dt_bias)
 *   da_log = A sum_{b,t} delta_t q_t             dd = sum_{b,t} ds_t x_t
 *   ddt_bias = sum_{b,t} ddt_t                   dh0 = exp(delta_0 A) g_0
 *
 * Activations (`dtype`) are gscan_views: a pointer, the stride of the batch and
 * the stride of a position, in elements; elements within a position are
 * adjacent.  x, dt, z, y and their gradients are [B][T][D], b, c and theirs
 * [B][T][G*N].  They may so be parts of projections.  Any alignment of an
 * element is taken.
 *
 * a_log [D][N], d [D], dt_bias [D], h0, h_last, dh_last, dh0 ([B][D][N]) and
 * the parameters' gradients are fp32 and contiguous.  d, z, dt_bias and h0 may be
 * NULL: that term is absent.
 *
 * lengths, where given, holds B int32 values in device memory: sequence b has
 * lengths[b] valid positions, its first (values outside 0..T are taken as the
 * nearer end).  Outputs and gradients are zero beyond them, nothing of an input
 * is read there, and the last state is that after the valid positions (h0 where
 * there are none).
 *
 * Arithmetic is fp32 throughout; each output is rounded once, to nearest even.
 * Sums over positions, channels and sequences are taken in a fixed order (those
 * of the parameters are closed in fp64), so results are bitwise reproducible for
 * a given shape.
 *
 * Ownership, threading, streams and error codes are those of wtconv.h: the
 * caller owns every buffer, the calls only enqueue kernels on `stream`, keep
 * nothing, and can be captured into a graph.  An output may not overlap an
 * input, another output, the states or the workspace (views that interleave
 * within one buffer, of the same strides and with no element in common, are
 * taken), nor itself.
 */
#ifndef SSCAN_H
#define SSCAN_H

#include <stddef.h>

#include "gscan.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SSCAN_MAX_STATES 64

typedef struct {
    int B, T, D, N, G; /* sequences, positions (T <= 2^30), channels, states (1..64), groups (G divides D) */
    int dtype;         /* gscan_dtype of every activation */
} sscan_shape;

/*
 * Sizes: B * D and D * N up to 2^25, B * D * N up to 2^31, G * N up to 2^20
 * (WTCONV_ERR_SHAPE beyond).  What one launch does not hold is refused with
 * WTCONV_ERR_UNSUPPORTED: G * ceil(D / G / 64) * B has to be below 2^20 (a 32 for
 * the 64 where N > 16), and B * ceil(T / 16) below 2^31; and so are strides of a
 * position above 2^26.
 */

/* Bytes of the states sscan_fwd writes for sscan_bwd: h before each 16
 * positions. */
int sscan_states_size(const sscan_shape* s, size_t* bytes);

/* Bytes of device workspace that sscan_fwd, and with `backward` sscan_bwd, needs. */
int sscan_workspace_size(const sscan_shape* s, int backward, size_t* bytes);

/* y and h_last.  states: sscan_states_size() bytes, or NULL where no gradient is
 * wanted.  h_last may be NULL. */
int sscan_fwd(const sscan_shape* s, const gscan_view* x, const gscan_view* dt, const float* a_log,
              const gscan_view* b, const gscan_view* c, const float* d, const gscan_view* z,
              const float* dt_bias, const float* h0, const int* lengths, const gscan_view* y,
              float* h_last, float* states, void* workspace, size_t ws_bytes, void* stream);

/* Every gradient from the inputs of sscan_fwd, the states it wrote and dy;
 * dh_last may be NULL (zeros), dh0 may be NULL (not wanted), and dd, dz and
 * ddt_bias are NULL where d, z and dt_bias are.  Gradients are overwritten. */
int sscan_bwd(const sscan_shape* s, const gscan_view* x, const gscan_view* dt, const float* a_log,
              const gscan_view* b, const gscan_view* c, const float* d, const gscan_view* z,
              const float* dt_bias, const float* states, const int* lengths, const gscan_view* dy,
              const float* dh_last, const gscan_view* dx, const gscan_view* ddt, float* da_log,
              const gscan_view* db, const gscan_view* dc, float* dd, const gscan_view* dz,
              float* ddt_bias, float* dh0, void* workspace, size_t ws_bytes, void* stream);

/*
 * One position of B sequences whose states live in a cache [S][D][N] fp32:
 * state[slots[b]] is read, advanced and written back, and y[b] follows.  slots
 * (int32, device) may be NULL: sequence b uses row b, and S must be at least B.
 * A sequence whose slot is outside 0..S-1 is passed over: its y is zero and no
 * state changes.  Slots that repeat give undefined states.  T of the shape is
 * not used.  The views are [B][D] and [B][G*N]: sb is the row stride, sr is not
 * used.
 */
int sscan_step(const sscan_shape* s, int S, const gscan_view* x, const gscan_view* dt,
               const float* a_log, const gscan_view* b, const gscan_view* c, const float* d,
               const gscan_view* z, const float* dt_bias, float* state, const int* slots,
               const gscan_view* y, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SSCAN_H */

/*
 * gdn_qk_norm.h -- the norm of every head's query and key with the position
 * rotation, in one pass over them.
 *
 * For a row x of d channels (one token's one head), with weights w:
 *
 *   r = (s + eps)^(-1/2),  s = sum x_i^2 / d  (or sum x_i^2, GDN_NORM_L2),
 *   y = rotate(w x r)
 *
 * The rotation turns the first rot channels in pairs by the angles of the
 * row's position p, given as tables of their cosines and sines:
 *
 *   (u, v) -> (u cos[p,i] - v sin[p,i], u sin[p,i] + v cos[p,i]),
 *
 * pair i being channels (i, i + rot/2), or (2i, 2i + 1) with
 * GDN_NORM_INTERLEAVED.
 *
 * Status codes, dtypes and gdn_strerror are gdn.h's.  All pointers are
 * DEVICE pointers on the current HIP device unless stated.
 */
#ifndef GDN_QK_NORM_H
#define GDN_QK_NORM_H

#include <stdint.h>

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Flags. */
#define GDN_NORM_L2 1          /* unit length: the sum of squares, not their mean */
#define GDN_NORM_INTERLEAVED 2 /* pairs of neighbouring channels                  */

/*
 * gdn_qk_norm_fwd -- forward pass.
 *
 *   q    : (B, T, Hq, d)   dtype    row-major, contiguous
 *   k    : (B, T, Hk, d)   dtype
 *   cos, sin : (P, rot/2)  float32, required when rot > 0
 *   pos  : (B, T)          int32    each token's position, or NULL: token t of
 *                                   each sequence has position t
 *   wq, wk : (d,)          float32  weights of the queries' and the keys'
 *                                   norms; each may be NULL (ones)
 *   qo, ko : like q and k  dtype    written; rounded to nearest even for bf16
 * A packed batch is B = 1 with its rows' positions in pos.  A row whose
 * position lies outside [0, P) -- -1 marks padding -- is set to zero (rot > 0
 * only: otherwise no position is read).
 *
 * Sizes: B, T >= 0, Hq, Hk in [1, 65535], d in {32, 64, 128, 256}
 *   (GDN_ERR_UNSUPPORTED otherwise); rot even, in [0, d]; P >= 1 when
 *   rot > 0; B * T < 2^31 tokens and fewer than 2^36 rows.  eps >= 0 and finite.
 * dtype: GDN_F32 or GDN_BF16; arithmetic fp32, the tables' angles exact for
 *   any position they hold.
 * flags: GDN_NORM_* or 0; any other bit is GDN_ERR_INVALID_ARG.
 * Pointers: q, k, qo and ko are required when B * T > 0; all are 16-byte
 *   aligned, pos 4-byte.  No output may overlap an input or another output.
 *   (GDN_ERR_INVALID_ARG otherwise.)
 *
 * Behaviour: host-side arguments are validated first; on any error a
 * negative status is returned, nothing is launched and the outputs are left
 * as they were.  On success the work is queued on `stream` and GDN_OK is
 * returned; results are valid once the stream has been synchronised.  The
 * library allocates nothing and keeps no pointer.  A row's bits depend on
 * the row, its position and the weights alone.  A row of zeros with eps 0
 * gives NaN, as the formula does; non-finite values stay within their row.
 * Squares are fp32: a row whose sum of them overflows (values of some 1e19)
 * gives zeros, and below 1e-19 an eps of 0 can give infinities.
 */
int gdn_qk_norm_fwd(const void* q, const void* k, const float* cos,
                    const float* sin, const int32_t* pos, const float* wq,
                    const float* wk, void* qo, void* ko, int B, int T, int Hq,
                    int Hk, int d, int rot, int P, float eps, void* stream,
                    int dtype, int flags);

/*
 * gdn_qk_norm_bwd -- gradients of <dqo, qo> + <dko, ko> for gdn_qk_norm_fwd's
 * outputs, from its inputs alone: with g the gradient turned back by the
 * angles, u = x r and m = d (1 with GDN_NORM_L2),
 *
 *   dx = r (w g - u (sum_i w_i g_i u_i) / m),   dw = sum over rows of g u.
 *
 * Arguments and layouts as for gdn_qk_norm_fwd, plus
 *   dqo, dko : like qo and ko  dtype
 *   dq, dk   : like q and k    dtype    written; zero where qo, ko are set to zero
 *   dwq, dwk : (d,)            float32  written, each NULL if not wanted; the
 *              gradient of the weights whether or not they were given; zeros
 *              for B * T == 0
 *   workspace: DEVICE buffer of at least gdn_qk_norm_workspace_size(...)
 *              bytes, 16-byte aligned, the caller's; overwritten, needed until
 *              the stream has passed the call; may be NULL when neither dwq
 *              nor dwk is wanted.  Calls that may overlap in time need
 *              workspaces of their own.
 * The weights' sums are taken in fp32 in a fixed order.  No gradient for the
 * tables.  Everything else is gdn_qk_norm_fwd's.
 */
int gdn_qk_norm_bwd(const void* q, const void* k, const float* cos,
                    const float* sin, const int32_t* pos, const float* wq,
                    const float* wk, const void* dqo, const void* dko, void* dq,
                    void* dk, float* dwq, float* dwk, int B, int T, int Hq,
                    int Hk, int d, int rot, int P, float eps, void* stream,
                    int dtype, int flags, void* workspace,
                    long long workspace_bytes);

/*
 * gdn_qk_norm_workspace_size -- bytes of workspace gdn_qk_norm_bwd needs for
 * the weights' gradients.  Negative: a status code.
 */
long long gdn_qk_norm_workspace_size(int B, int T, int Hq, int Hk, int d);

#ifdef __cplusplus
}
#endif

#endif /* GDN_QK_NORM_H */

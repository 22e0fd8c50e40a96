/*
 * gdn_linear.h -- linear attention with one fixed decay per head: the
 * recurrence of gdn.h without its erase term,
 *
 *   S_t = a_h S_{t-1} + k_t v_t^T,   o_t = S_t^T q_t,   a_h = exp(g_h),
 *
 * per head and per sequence, with the state S of shape (dk, dv).  The read
 * uses the state after the step's write and no 1/sqrt(dk) scale is applied,
 * as in gdn.h.  The state lies as gdn.h's h0 / hT do (key rows x value
 * columns), so both rules' states can live in one pool (gdn_pool.h).
 *
 * Status codes, dtypes and gdn_strerror are gdn.h's.  All pointers are
 * DEVICE pointers on the current HIP device unless stated.
 */
#ifndef GDN_LINEAR_H
#define GDN_LINEAR_H

#include <stdint.h>

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * gdn_linear_fwd -- forward pass, chunkwise form (prompts, training).
 *
 * Dense mode (cu_seqlens == NULL): B sequences of T tokens each.
 *   q, k : (B, T, H, dk)  dtype     row-major, contiguous
 *   v    : (B, T, H, dv)  dtype
 *   g    : (H,)           float32   natural-log decay, g <= 0; -inf is a
 *                                   state that forgets at every token
 *   out  : (B, T, H, dv)  dtype     written; rounded to nearest even for bf16
 * Packed mode (cu_seqlens != NULL): the tensors drop the leading B, T is the
 *   number of rows, cu_seqlens a DEVICE int32 array of B+1 offsets; sequence
 *   n is rows [cu_seqlens[n], cu_seqlens[n+1]), an independent recurrence.
 *   Offsets are taken into [0, T] and an end before its begin is an empty
 *   sequence, so no offset reads or writes outside the tensors.  Every
 *   sequence has its own rows and state whatever the offsets' order, but where
 *   one lies before an earlier one nothing is cut into segments (see below),
 *   and sequences that overlap race on out (not on hT).  Rows of no sequence
 *   are left as they were.
 * State, both modes: h0 (B, H, dk, dv) float32 or NULL (zero); hT the same
 *   shape, written; hT may be h0 itself (not a part of it).  A sequence of
 *   length 0 gets hT = h0 (or zeros).
 *
 * Sizes: B >= 0, T >= 0, H >= 1; dk, dv in {32, 64, 128}; T * H * max(dk, dv)
 *   * element size < 2^31 (GDN_ERR_INVALID_ARG): a sequence's rows are
 *   addressed with 32 bits, and a packed batch, whose lengths the host does
 *   not know, may hold one sequence of all T rows, so that there the bound is
 *   the whole batch's (a larger one goes in several calls); H <= 65535, B * H <
 *   2^18 and, dense, B * T < 2^31.  dtype: GDN_F32 or GDN_BF16.
 * Pointers: q, k, v and out are required when T > 0 and B > 0, g and hT when
 *   B > 0.  All are 16-byte aligned (GDN_ERR_INVALID_ARG otherwise; g and
 *   cu_seqlens 4-byte).  No output may overlap an input or another output,
 *   hT == h0 apart (GDN_ERR_INVALID_ARG).
 * workspace: DEVICE buffer of at least gdn_linear_workspace_size(...) bytes,
 *   16-byte aligned, the caller's; overwritten, needed until the stream has
 *   passed the call; NULL where that size is 0.  Calls that may overlap in
 *   time need workspaces of their own.
 *
 * Behaviour: host-side arguments are validated first; on any error a
 * negative status is returned, nothing is launched and the outputs are left
 * as they were.  On success the work is queued on `stream` and GDN_OK is
 * returned; results are valid once the stream has been synchronised.  The
 * library allocates nothing and keeps no pointer.  Identical calls give
 * identical bits on one device (no atomics, fixed reduction order); how a
 * batch is cut into segments goes by its sizes (B, T, H, dk, dv), the dtype,
 * whether it is packed and the direction, so the same sequence in another
 * batch may differ by rounding.
 *
 * Segments.  A long sequence of a batch with fewer chains than the device has
 * compute units is cut into segments that run side by side (a packed one
 * where its offsets ascend).  A first launch
 * forms the state that each segment leaves, from which the next ones start;
 * rows whose decay to the segment's end is below e^-40 are left out of it (as
 * gdn_fwd's halos are bounded), non-finite ones among them.  With hT == h0
 * nothing is cut.
 *
 * Arithmetic: GDN_BF16: every product on the bf16 matrix cores with fp32
 * accumulation; the state is rounded to bf16 as an operand of the outputs
 * only, the masked scores are taken as two bf16 terms (16 bits), and the
 * decayed values that enter the state as three, all of their 24 bits.  GDN_F32: fp32
 * throughout.  The state is carried in fp32 in both, and a constant decay's rounding does not add up
 * over a long sequence.  Non-finite inputs propagate within their own head
 * and sequence, to the rows of the same chunk (32 rows at most) before them
 * too.  A positive g is computed as it stands, as long as the decay over 64
 * rows, exp(64 g), is finite in fp32 and the states are.
 */
int gdn_linear_fwd(const void* q, const void* k, const void* v, const float* g,
                   const float* h0, const int32_t* cu_seqlens, void* out,
                   float* hT, int B, int T, int H, int dk, int dv,
                   void* stream, int dtype, void* workspace,
                   long long workspace_bytes);

/*
 * gdn_linear_workspace_size -- bytes of workspace that gdn_linear_fwd
 * (backward == 0) or gdn_linear_bwd (backward != 0) needs for these sizes;
 * packed != 0: a packed batch of T rows.  The states of the segments that
 * long sequences are cut into, where a batch has too few chains to fill the
 * device; 0 where nothing is cut.  Negative: a status code.
 */
long long gdn_linear_workspace_size(int B, int T, int H, int dk, int dv,
                                    int packed, int dtype, int backward);

/*
 * gdn_linear_bwd -- gradients of <dout, out> + <dhT, hT> for
 * gdn_linear_fwd's outputs, from its inputs alone.
 *
 * With the state gradient G_t = q_t dout_t^T + a G_{t+1}, dhT standing in the
 * place of a G_{t+1} at the last token:
 *   dq_t = S_t dout_t,  dk_t = G_t v_t,  dv_t = G_t^T k_t,  dh0 = a G_first
 * (dhT for an empty sequence).  g is a constant of the model: it gets no
 * gradient.
 *
 * Arguments and layouts as for gdn_linear_fwd, plus
 *   dout   : like out              dtype
 *   dhT    : (B, H, dk, dv)        float32, or NULL (zero)
 *   dq, dk : like q                dtype    written
 *   dv     : like v                dtype    written
 *   dh0    : (B, H, dk, dv)        float32  written, or NULL (not wanted); the
 *            gradient of h0 whether or not h0 was given.
 * dh0 may be dhT itself.  Rows of no sequence are left as they were in dq, dk
 * and dv.  Everything else is gdn_linear_fwd's.
 */
int gdn_linear_bwd(const void* q, const void* k, const void* v, const float* g,
                   const float* h0, const int32_t* cu_seqlens, const void* dout,
                   const float* dhT, void* dq, void* dk, void* dv, float* dh0,
                   int B, int T, int H, int dk_, int dv_, void* stream,
                   int dtype, void* workspace, long long workspace_bytes);

/*
 * gdn_linear_fwd_recurrent -- the same operation token by token, for
 * decoding and other short sequences, fp32 arithmetic throughout (bf16
 * storage widened on load, the output rounded to nearest even).  Arguments
 * as for gdn_linear_fwd, without the workspace; any g.  Rows and states are
 * addressed with 64 bits: no limit on a sequence's bytes, but fewer than 2^31
 * rows, and B * H * dv < 2^29.
 */
int gdn_linear_fwd_recurrent(const void* q, const void* k, const void* v,
                             const float* g, const float* h0,
                             const int32_t* cu_seqlens, void* out, float* hT,
                             int B, int T, int H, int dk, int dv, void* stream,
                             int dtype);

#ifdef __cplusplus
}
#endif

#endif /* GDN_LINEAR_H */

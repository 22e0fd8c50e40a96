/*
 * gdn_conv.h -- the short causal convolution that a recurrent layer puts
 * before its recurrence: depthwise over W tokens, with SiLU.
 *
 *   y_t[d] = bias[d] + sum_{i < W} w[d,i] x_{t-W+1+i}[d],  out = y SiLU'd or y,
 *   SiLU(y) = y / (1 + exp(-y))
 *
 * per sequence; the W - 1 tokens before its first are its initial state.
 *
 * Status codes, dtypes and gdn_strerror are gdn.h's.  All pointers are
 * DEVICE pointers on the current HIP device unless stated.
 */
#ifndef GDN_CONV_H
#define GDN_CONV_H

#include <stdint.h>

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Flags. */
#define GDN_CONV_SILU 1 /* the output goes through SiLU */

/*
 * gdn_conv_fwd -- forward pass over whole sequences.
 *
 * Dense mode (cu_seqlens == NULL): B sequences of T tokens each.
 *   x    : (B, T, D)     dtype    row-major, contiguous
 *   w    : (D, W)        float32  w[d, W-1] multiplies the token itself
 *   bias : (D,)          float32, or NULL
 *   out  : (B, T, D)     dtype    written; rounded to nearest even for bf16
 * Packed mode (cu_seqlens != NULL): x and out drop the leading B, T is the
 *   number of rows, cu_seqlens a DEVICE int32 array of B+1 non-decreasing
 *   offsets; sequence n is rows [cu_seqlens[n], cu_seqlens[n+1]).  Offsets are
 *   taken into [0, T] and an end before its begin is an empty sequence; where
 *   offsets fall, which rows belong to which sequence is unspecified, but
 *   nothing outside the tensors is read or written.  Rows of no sequence are
 *   left as they were.
 * State, both modes: h0 (B, W-1, D) dtype, the tokens before the first, oldest
 *   first, or NULL (zeros); hT the same shape, written with the last W - 1
 *   tokens (of h0 and x); hT may be h0 itself (not a part of it).  A sequence
 *   of length 0 gets hT = h0 (or zeros).
 *
 * Sizes: B >= 0, T >= 0, D >= 1, W in {2, 3, 4} (GDN_ERR_UNSUPPORTED
 *   otherwise); at most 2^30 rows, D < 2^20, B < 2^24, B * ceil(D / 64) <
 *   2^25.
 * dtype: GDN_F32 or GDN_BF16; arithmetic fp32.
 * flags: 0 or GDN_CONV_SILU; any other bit is GDN_ERR_INVALID_ARG.
 * Pointers: x and out are required when B > 0 and T > 0, w and hT when B > 0;
 *   all are 16-byte aligned, cu_seqlens and slots 4-byte
 *   (GDN_ERR_INVALID_ARG).  No output may overlap an input or another output,
 *   hT == h0 apart (GDN_ERR_INVALID_ARG).
 *
 * Behaviour: host-side arguments are validated first; on any error a
 * negative status is returned, nothing is launched and the outputs are left
 * as they were.  On success the work is queued on `stream` and GDN_OK is
 * returned; results are valid once the stream has been synchronised.  The
 * library allocates nothing and keeps no pointer.  Identical calls give
 * identical bits; a token's output does not depend on the batch around it.
 * Non-finite inputs propagate to the W tokens that they enter, and no others.
 */
int gdn_conv_fwd(const void* x, const float* w, const float* bias,
                 const void* h0, const int32_t* cu_seqlens, void* out,
                 void* hT, int B, int T, int D, int W, void* stream, int dtype,
                 int flags);

/*
 * gdn_conv_bwd -- gradients of <dout, out> + <dhT, hT> for gdn_conv_fwd's
 * outputs, from its inputs alone (the convolution is formed again).
 *
 * Arguments and layouts as for gdn_conv_fwd, plus
 *   dout  : like out           dtype
 *   dhT   : (B, W-1, D)        dtype, or NULL (zero)
 *   dx    : like x             dtype    written
 *   dw    : (D, W)             float32  written
 *   dbias : (D,)               float32  written, or NULL (not wanted)
 *   dh0   : (B, W-1, D)        dtype    written, or NULL (not wanted); the
 *           gradient of h0 whether or not h0 was given
 *   workspace: DEVICE buffer of at least gdn_conv_workspace_size(...) bytes,
 *           16-byte aligned, the caller's; overwritten, needed until the
 *           stream has passed the call.  Calls that may overlap in time need
 *           workspaces of their own.
 * dx, dw and dbias are written for B == 0 and T == 0 too (dw and dbias with
 * zeros).  Rows of no sequence are left as they were in dx.  The parameters'
 * sums over the tokens are taken in fp32 in a fixed order.  Everything else is
 * gdn_conv_fwd's.
 */
int gdn_conv_bwd(const void* x, const float* w, const float* bias,
                 const void* h0, const int32_t* cu_seqlens, const void* dout,
                 const void* dhT, void* dx, float* dw, float* dbias, void* dh0,
                 int B, int T, int D, int W, void* stream, int dtype, int flags,
                 void* workspace, long long workspace_bytes);

/*
 * gdn_conv_workspace_size -- bytes of workspace gdn_conv_bwd needs for these
 * sizes; packed != 0: a packed batch of T rows.  Negative: a status code.
 */
long long gdn_conv_workspace_size(int B, int T, int D, int W, int packed,
                                  int dtype);

/*
 * gdn_conv_fwd_pool -- the same convolution for decoding, on states in a
 * pool: sequence n starts from the state in slot slots[n] and leaves its last
 * W - 1 tokens there.
 *
 *   x, w, bias, cu_seqlens, out, B, T, D, W, stream, dtype, flags: as for
 *           gdn_conv_fwd; packed offsets may be anything: each sequence is
 *           computed by itself, and those that overlap race on out alone
 *   pool  : (nslots, W-1, D) dtype, read and written in place
 *   slots : (B,) DEVICE int32.  A sequence whose slot lies outside
 *           [0, nslots) -- -1 marks the padding rows of a fixed-size batch --
 *           or is already an earlier sequence's changes no state, and its
 *           rows of out are set to zero.
 *
 * out and the pool may not overlap an input or each other.  Slots are read on
 * the device when the work runs, so a captured graph takes the slots and
 * states of each replay.  Everything else is gdn_conv_fwd's.
 */
int gdn_conv_fwd_pool(const void* x, const float* w, const float* bias,
                      void* pool, const int32_t* slots,
                      const int32_t* cu_seqlens, void* out, int nslots, int B,
                      int T, int D, int W, void* stream, int dtype, int flags);

#ifdef __cplusplus
}
#endif

#endif /* GDN_CONV_H */

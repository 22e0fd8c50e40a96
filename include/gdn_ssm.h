/*
 * gdn_ssm.h -- the selective state space scan: a recurrence whose decay is
 * each channel's and token's own, with the layer's skip and gate.
 *
 * Per sequence and channel d of D, with N states and its group's keys (channel
 * d belongs to group d / (D / G)):
 *
 *   s_t = softplus(dt_t + dt_bias)         (or dt_t + dt_bias),
 *   h_t[n] = exp(s_t A[n]) h_{t-1}[n] + s_t x_t b_t[n],   A = -exp(A_log[d, :]),
 *   y_t = sum_n c_t[n] h_t[n] + Dskip[d] x_t,   out_t = y_t SiLU(z_t),
 *
 * softplus(v) = log(1 + exp(v)), SiLU(z) = z / (1 + exp(-z)).  The recurrence
 * of gdn_diag_fwd (gdn.h) decays all channels of a head alike; here every
 * channel has its own step s_t.
 *
 * Status codes, dtypes and gdn_strerror are gdn.h's.  All pointers are
 * DEVICE pointers on the current HIP device unless stated.
 */
#ifndef GDN_SSM_H
#define GDN_SSM_H

#include <stdint.h>

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Flags. */
#define GDN_SSM_SOFTPLUS 1 /* the step goes through softplus */

/*
 * gdn_ssm_fwd -- forward pass over whole sequences (prompts, training).
 *
 * Dense mode (cu_seqlens == NULL): B sequences of T tokens each.
 *   x, dt  : (B, T, D)     dtype    row-major, contiguous
 *   b, c   : (B, T, G, N)  dtype    write and read keys
 *   A_log  : (D, N)        float32
 *   Dskip  : (D,)          float32, or NULL (no skip term)
 *   z      : (B, T, D)     dtype, or NULL (no gate)
 *   dt_bias: (D,)          float32, or NULL
 *   out    : (B, T, D)     dtype    written; rounded to nearest even for bf16
 * Packed mode (cu_seqlens != NULL): the tensors drop the leading B, T is the
 *   number of rows, cu_seqlens a DEVICE int32 array of B+1 non-decreasing
 *   offsets; sequence n is rows [cu_seqlens[n], cu_seqlens[n+1]).  Offsets are
 *   taken into [0, T] and an end before its begin is an empty sequence; where
 *   offsets fall, the results of the sequences concerned are unspecified, but
 *   nothing outside the tensors is read or written.  Rows of no sequence are
 *   left as they were.
 * State, both modes: h0 (B, D, N) float32 or NULL (zero); hT the same shape,
 *   written; hT may be h0 itself (not a part of it).  A sequence of length 0
 *   gets hT = h0 (or zeros).
 *
 * Sizes: B >= 0, T >= 0, D >= 1, G >= 1 a divisor of D; N in {16, 32, 64}
 *   (GDN_ERR_UNSUPPORTED otherwise); at most 2^30 rows, D < 2^20, B < 2^24,
 *   B * D < 2^28, B * ceil(D N / 1024) < 2^24, B * G * ceil(D / (64 G)) < 2^26.
 *   dtype: GDN_F32 or GDN_BF16.
 * flags: 0 or GDN_SSM_SOFTPLUS; any other bit is GDN_ERR_INVALID_ARG.
 * Pointers: x, dt, b, c and out are required when B > 0 and T > 0, A_log and
 *   hT when B > 0; all are 16-byte aligned, cu_seqlens 4-byte
 *   (GDN_ERR_INVALID_ARG).  No output may overlap an input or another output,
 *   hT == h0 apart (GDN_ERR_INVALID_ARG).
 * workspace: DEVICE buffer of at least gdn_ssm_workspace_size(...) bytes,
 *   16-byte aligned, the caller's; overwritten, needed until the stream has
 *   passed the call; NULL where that size is 0.  Calls that may overlap in
 *   time need workspaces of their own.
 *
 * Behaviour: host-side arguments are validated first; on any error a
 * negative status is returned, nothing is launched and the outputs are left
 * as they were.  On success the work is queued on `stream` and GDN_OK is
 * returned; results are valid once the stream has been synchronised.  The
 * library allocates nothing and keeps no pointer.  Identical calls give
 * identical bits on one device (no atomics, fixed order); how sequences are
 * cut goes by the sizes, the dtype and whether the batch is packed, so the
 * same sequence in another batch may differ by rounding.
 *
 * Segments.  Where there are too few channels and sequences to fill the
 * device, sequences are cut into segments that run side by side: a first
 * launch forms the state that each segment leaves from a zero state and the
 * sum of its steps, a second joins them (h' = exp(A sum s) h + that state:
 * exact, whatever the decay), a third computes the segments from their states.
 * Of a packed batch, whose lengths only the device knows, segments are at most
 * one and a half of a wave's even shares of the rows long (or 64 rows), so that
 * a long sequence among many short ones is cut too; a batch of some hundred rows
 * is taken token by token, whole.
 *
 * Arithmetic: fp32 throughout, bf16 storage widened on load.  Non-finite
 * inputs propagate along their own channel and, through b and c, their own
 * token.  An infinity may come out as NaN behind its token: in a cut sequence
 * where the decay over a segment is zero, in hT, and backwards in every
 * gradient that it reaches.
 */
int gdn_ssm_fwd(const void* x, const void* dt, const void* b, const void* c,
                const float* A_log, const float* Dskip, const void* z,
                const float* dt_bias, const float* h0,
                const int32_t* cu_seqlens, void* out, float* hT, int B, int T,
                int D, int G, int N, void* stream, int dtype, int flags,
                void* workspace, long long workspace_bytes);

/*
 * gdn_ssm_workspace_size -- bytes of workspace that gdn_ssm_fwd (backward ==
 * 0) or gdn_ssm_bwd (backward != 0) needs for these sizes; packed != 0: a
 * packed batch of T rows.  Negative: a status code.
 */
long long gdn_ssm_workspace_size(int B, int T, int D, int G, int N, int packed,
                                 int dtype, int backward);

/*
 * gdn_ssm_bwd -- gradients of <dout, out> + <dhT, hT> for gdn_ssm_fwd's
 * outputs, from its inputs alone (the states are formed again).
 *
 * With the output's gradient dy_t = dout_t SiLU(z_t), the state's is l_t = c_t
 * dy_t + exp(s_{t+1} A) l_{t+1}, dhT standing behind the last token, and
 *   db_t = sum_d l_t s_t x_t,   dc_t = sum_d dy_t h_t     (over a group's channels),
 *   ds_t = sum_n l_t (A exp(s_t A) h_{t-1} + x_t b_t),    dx_t = s_t sum_n l_t b_t + Dskip dy_t,
 *   dA_log = A sum_t l_t s_t exp(s_t A) h_{t-1},          dD = sum_t dy_t x_t,
 *   ddt_t = ds_t sigmoid(dt_t + dt_bias) (or ds_t),       ddt_bias = sum_t ddt_t,
 *   dz_t = dout_t y_t SiLU'(z_t),                         dh0 = exp(s_1 A) l_1.
 *
 * Arguments and layouts as for gdn_ssm_fwd, plus
 *   dout : like out         dtype
 *   dhT  : (B, D, N)        float32, or NULL (zero)
 *   dx, ddt : like x        dtype    written
 *   db, dc  : like b        dtype    written
 *   dA_log  : (D, N)        float32  written
 *   dD      : (D,)          float32  written, or NULL (not wanted)
 *   dz      : like z        dtype    written, or NULL (not wanted); only with z
 *   ddt_bias: (D,)          float32  written, or NULL (not wanted)
 *   dh0     : (B, D, N)     float32  written, or NULL (not wanted); the
 *             gradient of h0 whether or not h0 was given.
 * dh0 may be dhT itself.  The parameters' gradients are written for B == 0 and
 * T == 0 too (zeros).  Rows of no sequence are left as they were.  Sums over
 * tokens and channels are taken in fp32 in a fixed order.  Everything else is
 * gdn_ssm_fwd's; sequences are always cut, into segments of 8 to 24 tokens.
 * Where a state or its gradient is not finite, the parameters' gradients of its
 * channel may be NaN.
 */
int gdn_ssm_bwd(const void* x, const void* dt, const void* b, const void* c,
                const float* A_log, const float* Dskip, const void* z,
                const float* dt_bias, const float* h0,
                const int32_t* cu_seqlens, const void* dout, const float* dhT,
                void* dx, void* ddt, void* db, void* dc, float* dA_log,
                float* dD, void* dz, float* ddt_bias, float* dh0, int B, int T,
                int D, int G, int N, void* stream, int dtype, int flags,
                void* workspace, long long workspace_bytes);

/*
 * gdn_ssm_fwd_recurrent_pool -- the same recurrence token by token for
 * decoding, on states in a pool: sequence n starts from the state in slot
 * slots[n] and leaves its final state there.
 *
 *   x .. dt_bias, cu_seqlens, out, B, T, D, G, N, stream, dtype, flags: as for
 *           gdn_ssm_fwd; packed offsets may be anything: each sequence is
 *           computed by itself, and those that overlap race on out alone
 *   pool  : (nslots, D, N) float32, read and written in place
 *   slots : (B,) DEVICE int32.  A sequence whose slot lies outside
 *           [0, nslots) -- -1 marks the padding rows of a fixed-size batch --
 *           or is already an earlier sequence's changes no state, and its
 *           rows of out are set to zero.
 *
 * out and the pool may not overlap an input or each other.  Slots are read on
 * the device when the work runs, so a captured graph takes the slots and
 * states of each replay.  Everything else is gdn_ssm_fwd's.
 */
int gdn_ssm_fwd_recurrent_pool(const void* x, const void* dt, const void* b,
                               const void* c, const float* A_log,
                               const float* Dskip, const void* z,
                               const float* dt_bias, float* pool,
                               const int32_t* slots, const int32_t* cu_seqlens,
                               void* out, int nslots, int B, int T, int D,
                               int G, int N, void* stream, int dtype,
                               int flags);

#ifdef __cplusplus
}
#endif

#endif /* GDN_SSM_H */

/*
 * gdn_pool.h -- a pool of recurrent states, for serving: sequences come, go
 * and fork while their states stay in the slots of one buffer.
 *
 * A pool is a contiguous (slots, H, dk, dv) float32 array, one slot a
 * sequence's state in the layout of gdn.h's h0 / hT; several layers' pools
 * may lie behind one another.  The token-by-token forms here read and write
 * a sequence's state in its slot; gdn_state_move copies, forks, clears and
 * gathers slots.
 *
 * Status codes, dtypes and gdn_strerror are gdn.h's.  All pointers are
 * DEVICE pointers on the current HIP device unless stated.
 */
#ifndef GDN_POOL_H
#define GDN_POOL_H

#include <stdint.h>

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * gdn_fwd_recurrent_pool -- gdn_fwd_recurrent (the gated delta rule token by
 * token) on states in a pool: sequence n starts from the state in slot
 * slots[n] and leaves its final state there.
 *
 *   q, k, v, g, beta, out, cu_seqlens, B, T, H, dk, dv, dtype, stream: as for
 *          gdn_fwd_recurrent; packed offsets are taken into [0, T] and an end
 *          before its begin is an empty sequence, and rows of no sequence are
 *          left as they were.
 *   pool : (nslots, H, dk, dv) float32, read and written in place
 *   slots: (B,) DEVICE int32.  A sequence whose slot lies outside
 *          [0, nslots) -- -1 marks the padding rows of a fixed-size batch --
 *          or is already an earlier sequence's changes no state, and its
 *          rows of out are set to zero.
 *
 * pool, q, k, v and out are 16-byte aligned; out and the pool may not overlap
 * an input or each other; H <= 65535, B * H * dv < 2^29
 * (GDN_ERR_INVALID_ARG).  Other arguments' errors, determinism and ownership are
 * gdn_fwd_recurrent's.  Arithmetic fp32 throughout.  Slots are read on the
 * device when the work runs, so a captured graph takes the slots and states
 * of each replay.
 */
int gdn_fwd_recurrent_pool(const void* q, const void* k, const void* v,
                           const float* g, const float* beta, float* pool,
                           const int32_t* slots, const int32_t* cu_seqlens,
                           void* out, int nslots, int B, int T, int H, int dk,
                           int dv, void* stream, int dtype);

/*
 * gdn_linear_fwd_recurrent_pool -- the same for linear attention with a
 * decay per head: gdn_linear_fwd_recurrent (gdn_linear.h), g of shape (H,).
 */
int gdn_linear_fwd_recurrent_pool(const void* q, const void* k, const void* v,
                                  const float* g, float* pool,
                                  const int32_t* slots,
                                  const int32_t* cu_seqlens, void* out,
                                  int nslots, int B, int T, int H, int dk,
                                  int dv, void* stream, int dtype);

/*
 * gdn_state_move -- pool[o, dst[i]] = pool[o, src[i]] for every i < n and
 * o < outer, all at once: every source is read as it was before the call.
 * One source may go to many targets (a fork), targets may be sources (a
 * beam's reordering, cycles included), and src[i] == -1 clears its target.
 *
 *   pool : (outer, slots, slot_bytes / 16) blocks of 16 bytes, 16-byte
 *          aligned; any contents (bytes are copied as they are)
 *   src, dst : HOST int32 arrays of n entries, read before the call returns:
 *          the scheduler that owns the slots knows them on the host, so
 *          every index is checked here, and no index array has to be copied.
 *          src in [-1, slots), dst in [0, slots), no dst twice
 *          (GDN_ERR_INVALID_ARG otherwise, and nothing is launched).
 *   slot_bytes : > 0, a multiple of 16, at most 2^36.
 *
 * No workspace: the pairs are put in an order in which every slot is read
 * before it is written, a cycle through registers.  The work is queued on
 * `stream`, in one launch for up to some 300 pairs; a captured graph repeats
 * the pairs it was captured with.  GDN_ERR_LAUNCH also where the host runs
 * out of memory for the order.
 */
int gdn_state_move(void* pool, long long outer, long long slots,
                   long long slot_bytes, const int32_t* src,
                   const int32_t* dst, int n, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_POOL_H */

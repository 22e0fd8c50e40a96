// Token-by-token recurrences on states in a pool of slots, and the moving of
// slots, for gfx950.
//
// Recurrence kernel.  Per token of a chain (sequence, head), with the state M
// of dk rows and dv columns:
//
//   linear attention  M <- a M + k v^T,                        o = M^T q
//   gated delta rule  M <- a M + k u^T, u = beta (v - a M^T k), o = M^T q
//
// A workgroup owns one chain's tile of CW value columns and keeps it in
// registers for the whole sequence: a thread holds four neighbouring columns
// of R neighbouring rows, so every state access is a 16-byte one and a wave's
// covers whole 128-byte lines.  The sums over the rows go through the lanes
// (DPP and permutes) and then through LDS, once a token: the delta rule's
// two sums M^T k and M^T q are taken of the old state together, since
// o = a M^T q + u (k . q).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <new>

#include "gdn_checks.h"
#include "gdn_linear.h"
#include "gdn_move_plan.h"
#include "gdn_pool.h"

namespace {

typedef float f4 __attribute__((ext_vector_type(4)));

struct PoolParams {
  const void* q;
  const void* k;
  const void* v;
  const float* g;
  const float* beta;
  const float* h0;       // null: zero states
  float* hT;
  const int32_t* slots;  // null: sequence n has state n
  const int32_t* cu;
  void* out;
  int B, T, H, dv, nslots, tiles;
};

__device__ static inline float widen(float x) { return x; }
__device__ static inline float widen(__bf16 x) { return (float)x; }

template <typename TI>
__device__ static inline f4 load4(const TI* p) {
  typedef TI t4 __attribute__((ext_vector_type(4)));
  const t4 x = *reinterpret_cast<const t4*>(p);
  return f4{widen(x[0]), widen(x[1]), widen(x[2]), widen(x[3])};
}

template <typename TI>
__device__ static inline void store4(TI* p, f4 x) {
  typedef TI t4 __attribute__((ext_vector_type(4)));
  *reinterpret_cast<t4*>(p) = t4{(TI)x[0], (TI)x[1], (TI)x[2], (TI)x[3]};  // to nearest even
}

// Sum of x over the lanes that hold the same columns (LC lanes apart).
template <int LC>
__device__ static inline f4 sum_rows(f4 x) {
#pragma unroll
  for (int d = LC; d < 64; d *= 2)
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] += __shfl_xor(x[e], d);
  return x;
}

template <typename TI, int DK, int CW, int NT, bool DELTA>
__global__ __launch_bounds__(NT) void pool_recurrent_kernel(const PoolParams p) {
  constexpr int LC = CW / 4;       // lanes across the columns
  constexpr int RG = NT / LC;      // groups of rows
  constexpr int R = DK / RG;       // rows a thread
  constexpr int NW = NT / 64;      // waves
  static_assert(RG * R == DK && LC <= 64 && 64 % LC == 0, "tile");
  // k and q of a token, widened; the waves' partial sums.  Two of each, taken
  // in turn, so that one barrier after each hand-over is enough.
  __shared__ __attribute__((aligned(16))) float kq[2][2][DK];
  __shared__ __attribute__((aligned(16))) float part[2][2][NW][CW];
  __shared__ float kqdot[2][NW];
  __shared__ int taken;

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int tile = blockIdx.x % p.tiles, chain = blockIdx.x / p.tiles;
  const int n = chain / p.H, h = chain % p.H;
  long row0;
  int len;
  if (p.cu) {
    const int b = min(max(p.cu[n], 0), p.T), e = min(max(p.cu[n + 1], b), p.T);
    row0 = b;
    len = e - b;
  } else {
    row0 = (long)n * p.T;
    len = p.T;
  }
  int slot = n;
  bool live = true;
  if (p.slots) {
    slot = p.slots[n];
    live = (unsigned)slot < (unsigned)p.nslots;
  }
  const int c0 = (tid % LC) * 4, col = tile * CW + c0;
  const int r0 = tid / LC * R;
  const long sbase = (((long)slot * p.H + h) * DK + r0) * p.dv + col;

  f4 M[R];
#pragma unroll
  for (int r = 0; r < R; ++r) M[r] = f4{0.f, 0.f, 0.f, 0.f};
  if (live && p.h0) {
#pragma unroll
    for (int r = 0; r < R; ++r) M[r] = *reinterpret_cast<const f4*>(p.h0 + sbase + (long)r * p.dv);
  }
  if (p.slots) {  // an earlier sequence with the same slot keeps it (looked for while the state is on its way)
    if (tid == 0) taken = 0;
    __syncthreads();
    for (int i = tid; i < n; i += NT)
      if (p.slots[i] == slot) taken = 1;
    __syncthreads();
    live = live && !taken;
  }
  TI* out = static_cast<TI*>(p.out);
  if (!live) {
    for (int t = 0; t < len; ++t)
      if (tid < LC) store4(out + ((row0 + t) * p.H + h) * p.dv + col, f4{0.f, 0.f, 0.f, 0.f});
    return;
  }

  const TI* q = static_cast<const TI*>(p.q);
  const TI* k = static_cast<const TI*>(p.k);
  const TI* v = static_cast<const TI*>(p.v);
  // A constant decay's rounding would add up over the tokens, always to the
  // same side: it is taken as two terms.
  float a = 0.f, a_lo = 0.f;
  if (!DELTA && len > 0) {
    const double d = exp((double)p.g[h]);
    a = (float)d;
    a_lo = d > 1e-30 && d < 1e30 ? (float)(d - (double)a) : 0.f;
  }
  // A token's k and q (shared out among the threads), v, and the delta
  // rule's decay and rate, fetched while the token before is worked on.
  constexpr int KQ = (2 * DK + NT - 1) / NT;
  TI kq_next[KQ];
  f4 v_next;
  float g_next = 0.f, b_next = 0.f;
  auto fetch = [&](int t) {
    const long th = (row0 + t) * p.H + h;
#pragma unroll
    for (int j = 0; j < KQ; ++j) {
      const int i = tid + j * NT;
      if (2 * DK % NT == 0 || i < 2 * DK) kq_next[j] = i < DK ? k[th * DK + i] : q[th * DK + i - DK];
    }
    v_next = load4(v + th * p.dv + col);
    if constexpr (DELTA) {
      g_next = p.g[th];
      b_next = p.beta[th];
    }
  };
  if (len > 0) fetch(0);
  for (int t = 0; t < len; ++t) {
    const int s = t & 1;
    const long th = (row0 + t) * p.H + h;
#pragma unroll
    for (int j = 0; j < KQ; ++j) {
      const int i = tid + j * NT;
      if (2 * DK % NT == 0 || i < 2 * DK) kq[s][i / DK][i % DK] = widen(kq_next[j]);
    }
    const f4 vc = v_next;
    const float b = b_next;
    if constexpr (DELTA) a = __expf(g_next);
    if (t + 1 < len) fetch(t + 1);
    __syncthreads();
    float kr[R], qr[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      kr[r] = kq[s][0][r0 + r];
      qr[r] = kq[s][1][r0 + r];
    }
    f4 o = {0.f, 0.f, 0.f, 0.f};
    if constexpr (DELTA) {
      f4 pk = {0.f, 0.f, 0.f, 0.f};
      float d = 0.f;
#pragma unroll
      for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          pk[e] = __builtin_fmaf(M[r][e], kr[r], pk[e]);
          o[e] = __builtin_fmaf(M[r][e], qr[r], o[e]);
        }
        d = __builtin_fmaf(kr[r], qr[r], d);
      }
      pk = sum_rows<LC>(pk);
      o = sum_rows<LC>(o);
#pragma unroll
      for (int w = LC; w < 64; w *= 2) d += __shfl_xor(d, w);
      if constexpr (NW > 1) {
        if (lane < LC) {
          *reinterpret_cast<f4*>(&part[s][0][wave][c0]) = pk;
          *reinterpret_cast<f4*>(&part[s][1][wave][c0]) = o;
        }
        if (lane == 0) kqdot[s][wave] = d;
        __syncthreads();
        pk = o = f4{0.f, 0.f, 0.f, 0.f};
        d = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          pk += *reinterpret_cast<const f4*>(&part[s][0][w][c0]);
          o += *reinterpret_cast<const f4*>(&part[s][1][w][c0]);
          d += kqdot[s][w];
        }
      }
      const f4 u = b * (vc - a * pk);
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e) M[r][e] = __builtin_fmaf(a, M[r][e], u[e] * kr[r]);
      o = a * o + u * d;
      if (tid < LC) store4(out + th * p.dv + col, o);
    } else {
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          M[r][e] = __builtin_fmaf(a, M[r][e], __builtin_fmaf(a_lo, M[r][e], vc[e] * kr[r]));
          o[e] = __builtin_fmaf(M[r][e], qr[r], o[e]);
        }
      o = sum_rows<LC>(o);
      if constexpr (NW > 1) {
        if (lane < LC) *reinterpret_cast<f4*>(&part[s][1][wave][c0]) = o;
        __syncthreads();
        if (tid < LC) {
          o = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int w = 0; w < NW; ++w) o += *reinterpret_cast<const f4*>(&part[s][1][w][c0]);
        }
      }
      if (tid < LC) store4(out + th * p.dv + col, o);
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) *reinterpret_cast<f4*>(p.hT + sbase + (long)r * p.dv) = M[r];
}

template <typename TI, int DK, int CW, int NT, bool DELTA>
void launch_tile(PoolParams p, hipStream_t s) {
  p.tiles = p.dv / CW;
  const long wgs = (long)p.B * p.H * p.tiles;
  hipLaunchKernelGGL((pool_recurrent_kernel<TI, DK, CW, NT, DELTA>), dim3((unsigned)wgs), dim3(NT), 0, s, p);
}

// A chain's columns are one workgroup's, unless that leaves compute units
// idle: then each 32 columns are (one sequence of 4 tokens, H = 16, dk = dv =
// 128 bf16: the kernel takes 6.0 us against 7.7).
template <typename TI, int DK, bool DELTA>
void launch_dk(const PoolParams& p, hipStream_t s) {
  if ((long)p.B * p.H < 256 && p.dv > 32) launch_tile<TI, DK, 32, DK == 128 ? 256 : 64, DELTA>(p, s);
  else if (p.dv == 128) launch_tile<TI, DK, 128, 256, DELTA>(p, s);
  else if (p.dv == 64) launch_tile<TI, DK, 64, DK == 32 ? 128 : 256, DELTA>(p, s);
  else launch_tile<TI, DK, 32, DK == 128 ? 256 : 64, DELTA>(p, s);
}

template <bool DELTA>
int launch(const PoolParams& p, int dk, int dtype, hipStream_t s) {
  switch (dk) {
    case 32: dtype == GDN_BF16 ? launch_dk<__bf16, 32, DELTA>(p, s) : launch_dk<float, 32, DELTA>(p, s); break;
    case 64: dtype == GDN_BF16 ? launch_dk<__bf16, 64, DELTA>(p, s) : launch_dk<float, 64, DELTA>(p, s); break;
    default: dtype == GDN_BF16 ? launch_dk<__bf16, 128, DELTA>(p, s) : launch_dk<float, 128, DELTA>(p, s); break;
  }
  return hipGetLastError() == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}

template <bool DELTA>
int recurrent(const void* q, const void* k, const void* v, const float* g, const float* beta, const float* h0,
              const int32_t* slots, const int32_t* cu, void* out, float* hT, int nslots, int B, int T, int H, int dk,
              int dv, void* stream, int dtype) {
  const bool pooled = slots != nullptr;
  if (B < 0 || T < 0 || H < 1 || dk < 1 || dv < 1) return GDN_ERR_INVALID_ARG;
  if (dtype != GDN_F32 && dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
  if (T > 0 && B > 0 && (!q || !k || !v || !g || (DELTA && !beta) || !out)) return GDN_ERR_INVALID_ARG;
  if (B > 0 && !hT) return GDN_ERR_INVALID_ARG;
  if ((dk != 32 && dk != 64 && dk != 128) || (dv != 32 && dv != 64 && dv != 128)) return GDN_ERR_UNSUPPORTED;
  const long long rows = (cu ? 1LL : (long long)B) * T, held = pooled ? nslots : B;
  // workgroups (at most 2^24 of 256 threads in a grid), tokens, states
  if ((long long)B * H * (dv / 32) >= 1LL << 24 || rows > 0x7fffffffLL || H > 65535) return GDN_ERR_INVALID_ARG;
  if (misaligned({q, k, v, out, h0, hT}, 16) || misaligned({g, beta, cu, slots}, 4)) return GDN_ERR_INVALID_ARG;
  const long long e = dtype == GDN_BF16 ? 2 : 4, state = held * H * dk * dv * 4;
  if (clash({{out, rows * H * dv * e}, {hT, state}},
            {{q, rows * H * dk * e}, {k, rows * H * dk * e}, {v, rows * H * dv * e},
             {g, DELTA ? rows * H * 4 : 4LL * H}, {beta, rows * H * 4}, {cu, 4LL * (B + 1)}, {slots, 4LL * B},
             {h0 == hT ? nullptr : h0, state}}))
    return GDN_ERR_INVALID_ARG;
  if (B == 0) return GDN_OK;
  const PoolParams p = {q, k, v, g, beta, h0, hT, slots, cu, out, B, T, H, dv, nslots, 1};
  return launch<DELTA>(p, dk, dtype, static_cast<hipStream_t>(stream));
}

// ------------------------------------------------------------ moving slots --
//
// The pairs are put in an order that needs no second copy (gdn_move_plan.h).
// A thread carries the same bytes of every slot of its group through the
// whole list, so the order needs no barrier, and since no slot is written
// before its last reading the loads of several steps can be on their way at
// once.  Bound by memory: one read of each source, one write of each target.

constexpr int MOVE_NT = 256;
constexpr int MOVE_V = 4;       // 16-byte pieces a thread carries

__global__ __launch_bounds__(MOVE_NT) void move_kernel(f4* __restrict__ pool, const long pieces, const long slots,
                                                      const MoveList m) {
  const int group = blockIdx.y;
  f4* base = pool + (long)blockIdx.z * slots * pieces;
  const long at = (long)blockIdx.x * MOVE_NT * MOVE_V + threadIdx.x;
  f4 reg[MOVE_V], kept[MOVE_V];
#pragma unroll
  for (int i = 0; i < MOVE_V; ++i) reg[i] = kept[i] = f4{0.f, 0.f, 0.f, 0.f};
  int last = STEP_ZERO;  // what reg holds
  for (int t = m.begin[group]; t < m.begin[group + 1]; ++t) {
    const int src = m.src[t], dst = m.dst[t];
    if (src != last) {
      last = src;
#pragma unroll
      for (int i = 0; i < MOVE_V; ++i) {
        const long x = at + i * MOVE_NT;
        if (src == STEP_KEPT) reg[i] = kept[i];
        else if (src == STEP_ZERO) reg[i] = f4{0.f, 0.f, 0.f, 0.f};
        else if (x < pieces) reg[i] = base[src * pieces + x];
      }
    }
    if (dst == STEP_KEPT) {
#pragma unroll
      for (int i = 0; i < MOVE_V; ++i) kept[i] = reg[i];
    } else {
#pragma unroll
      for (int i = 0; i < MOVE_V; ++i) {
        const long x = at + i * MOVE_NT;
        if (x < pieces) base[dst * pieces + x] = reg[i];
      }
    }
  }
}

int move_slots(f4* pool, long long outer, long long slots, long long pieces, const int32_t* src, const int32_t* dst,
               int n, hipStream_t stream) {
  MovePlan plan;  // whole before its first launch is queued
  if (!plan_moves(plan, slots, src, dst, n)) return GDN_ERR_INVALID_ARG;
  const unsigned tiles = (unsigned)((pieces + MOVE_NT * MOVE_V - 1) / (MOVE_NT * MOVE_V));
  for (const auto& l : plan.launches)
    for (long long o = 0; o < outer; o += 65535) {
      const unsigned z = (unsigned)std::min<long long>(65535, outer - o);
      hipLaunchKernelGGL(move_kernel, dim3(tiles, l.second, z), dim3(MOVE_NT), 0, stream, pool + o * slots * pieces,
                         (long)pieces, (long)slots, l.first);
      if (hipGetLastError() != hipSuccess) return GDN_ERR_LAUNCH;
    }
  return GDN_OK;
}

}  // namespace

extern "C" int gdn_fwd_recurrent_pool(const void* q, const void* k, const void* v, const float* g, const float* beta,
                                      float* pool, const int32_t* slots, const int32_t* cu_seqlens, void* out,
                                      int nslots, int B, int T, int H, int dk, int dv, void* stream, int dtype) {
  if (nslots < 0 || (B > 0 && !slots)) return GDN_ERR_INVALID_ARG;
  return recurrent<true>(q, k, v, g, beta, pool, slots, cu_seqlens, out, pool, nslots, B, T, H, dk, dv, stream, dtype);
}

extern "C" int gdn_linear_fwd_recurrent_pool(const void* q, const void* k, const void* v, const float* g, float* pool,
                                             const int32_t* slots, const int32_t* cu_seqlens, void* out, int nslots,
                                             int B, int T, int H, int dk, int dv, void* stream, int dtype) {
  if (nslots < 0 || (B > 0 && !slots)) return GDN_ERR_INVALID_ARG;
  return recurrent<false>(q, k, v, g, nullptr, pool, slots, cu_seqlens, out, pool, nslots, B, T, H, dk, dv, stream,
                          dtype);
}

extern "C" int gdn_linear_fwd_recurrent(const void* q, const void* k, const void* v, const float* g, const float* h0,
                                        const int32_t* cu_seqlens, void* out, float* hT, int B, int T, int H, int dk,
                                        int dv, void* stream, int dtype) {
  return recurrent<false>(q, k, v, g, nullptr, h0, nullptr, cu_seqlens, out, hT, B, B, T, H, dk, dv, stream, dtype);
}

extern "C" int gdn_state_move(void* pool, long long outer, long long slots, long long slot_bytes, const int32_t* src,
                              const int32_t* dst, int n, void* stream) {
  if (outer < 0 || slots < 0 || slots > 0x7fffffffLL || slot_bytes <= 0 || slot_bytes % 16 || n < 0)
    return GDN_ERR_INVALID_ARG;
  if (n > 0 && (!src || !dst || (!pool && outer > 0))) return GDN_ERR_INVALID_ARG;
  if (misaligned(pool, 16) || slot_bytes > 1LL << 36) return GDN_ERR_INVALID_ARG;  // 64 GiB a slot: the grid's width
  if (n == 0) return GDN_OK;
  try {
    return move_slots(static_cast<f4*>(pool), outer, slots, slot_bytes / 16, src, dst, n,
                      static_cast<hipStream_t>(stream));
  } catch (const std::bad_alloc&) {
    return GDN_ERR_LAUNCH;
  }
}

// Norms of every head's query and key with the position rotation, forwards
// and backwards, for gfx950.
//
// A row of d channels is d / 8 lanes wide, eight neighbouring channels (16
// bytes of bf16) a lane.  The sum of squares goes through the lanes by DPP.
// The rotation needs a channel's partner rot/2 further on (or before): with
// rot/2 a multiple of 8 that is another whole vector of the same row, read
// again (it hits the first cache; a shuffle of eight values costs more), with
// neighbouring pairs it is in the lane's own vector.
//
// Bound by memory: each row once in and once out.  What would come on top are
// the tables and weights, 32 to 96 bytes a lane against a row's 32: a lane
// keeps its weights for all its rows and its angles for up to `heads` heads of
// one token.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "gdn_checks.h"
#include "gdn_qk_norm.h"
#include "gdn_rows.h"

namespace {

constexpr int NT = 256;  // threads of a workgroup

struct NormParams {
  const void* x[2];  // queries, keys
  const void* g[2];  // their outputs' gradients (backwards)
  void* y[2];        // outputs, or the inputs' gradients
  const float* w[2];
  float* part[2];    // partial sums of the weights' gradients, one row of d a workgroup; null: not wanted
  const float* cos;
  const float* sin;
  const int32_t* pos;
  long tokens;
  int T, H[2], heads[2];  // heads a unit (a token's run of heads)
  int wgs[2];             // workgroups for queries and for keys
  int rot, P;
  float eps, scale;       // r = (scale sum x^2 + eps)^-1/2
};

// How a row's channels are paired.
enum Pairs { NONE, HALVES, HALVES_ODD, NEIGHBOURS };

// The eight channels' angles and partners: y_i = own_i cos_i + partner_i sin_i
// (sin with its sign; channels that are not turned have cos 1, sin 0).
struct Angles {
  Vals<8> c, s;
};

template <int PAIRS, bool BACK>
__device__ static inline Angles angles_of(const NormParams& p, long at, int c0) {
  Angles a;
  const int half = p.rot >> 1;
  const float* cs = p.cos + at * half;
  const float* sn = p.sin + at * half;
  if constexpr (PAIRS == HALVES) {
    if (c0 < p.rot) {
      const int i = c0 < half ? c0 : c0 - half;
      a.c = load_vals<float, 8>(cs + i);
      a.s = load_vals<float, 8>(sn + i);
      const float sign = (c0 < half) != BACK ? -1.f : 1.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) a.s[e] *= sign;
      return a;
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int ch = c0 + e;
    a.c[e] = 1.f;
    a.s[e] = 0.f;
    if constexpr (PAIRS == HALVES_ODD) {
      if (ch < p.rot) {
        const int i = ch < half ? ch : ch - half;
        a.c[e] = cs[i];
        a.s[e] = (ch < half) != BACK ? -sn[i] : sn[i];
      }
    } else if constexpr (PAIRS == NEIGHBOURS) {
      if (ch < p.rot) {
        a.c[e] = cs[ch >> 1];
        a.s[e] = ((e & 1) == 0) != BACK ? -sn[ch >> 1] : sn[ch >> 1];
      }
    }
  }
  return a;
}

// The first channel of the lane's partners (HALVES), its own if none.
__device__ static inline int partner0(const NormParams& p, int c0) {
  const int half = p.rot >> 1;
  return c0 < half ? c0 + half : c0 < p.rot ? c0 - half : c0;
}

// The partners' values of the lane's eight channels, as they are stored.
template <typename TS, int PAIRS>
__device__ static inline typename Raw<TS, 8>::type partners(const NormParams& p, const TS* row,
                                                            const typename Raw<TS, 8>::type& own, int c0) {
  typename Raw<TS, 8>::type q = own;
  const int half = p.rot >> 1;
  if constexpr (PAIRS == HALVES) {
    q = load_raw<TS, 8>(row + partner0(p, c0));
  } else if constexpr (PAIRS == HALVES_ODD) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int ch = c0 + e;
      q[e] = row[ch < half ? ch + half : ch < p.rot ? ch - half : ch];
    }
  } else if constexpr (PAIRS == NEIGHBOURS) {
#pragma unroll
    for (int e = 0; e < 8; ++e) q[e] = own[e ^ 1];
  }
  return q;
}

template <typename TI, int D, int PAIRS, bool BACK>
__global__ __launch_bounds__(NT) void norm_kernel(const NormParams p) {
  constexpr int LR = D / 8;  // lanes a row
  constexpr int GROUPS = NT / LR;
  // Rows of one token in flight at once; backwards, with three vectors a row, two
  // leave more waves (4 x 4,096 tokens, 16 + 4 heads of 128, neighbours paired:
  // 58 us a call, 67 with four).
  constexpr int FLIGHT = BACK ? 2 : 4;
  const int side = (int)blockIdx.x < p.wgs[0] ? 0 : 1;
  const int wg = blockIdx.x - (side ? p.wgs[0] : 0), nwg = p.wgs[side];
  const int tid = threadIdx.x, c0 = tid % LR * 8, group = tid / LR;
  const int H = p.H[side], heads = p.heads[side], chunks = (H + heads - 1) / heads;
  const TI* __restrict__ x = static_cast<const TI*>(p.x[side]);
  const TI* __restrict__ g = static_cast<const TI*>(p.g[side]);
  TI* __restrict__ y = static_cast<TI*>(p.y[side]);

  // Forwards the partner's weight is needed too; backwards the gradient is
  // turned back before it meets the weights.
  Vals<8> w, wp;
#pragma unroll
  for (int e = 0; e < 8; ++e) w[e] = wp[e] = 1.f;
  if (p.w[side]) {
    const Raw<float, 8>::type own = load_raw<float, 8>(p.w[side] + c0);
    w = widen<float, 8>(own);
    if constexpr (!BACK) wp = widen<float, 8>(partners<float, PAIRS>(p, p.w[side], own, c0));
  }
  Vals<8> dw;
#pragma unroll
  for (int e = 0; e < 8; ++e) dw[e] = 0.f;

  const long units = p.tokens * chunks;
  for (long u = (long)wg * GROUPS + group; u < units; u += (long)nwg * GROUPS) {
    const long token = u / chunks;
    const int h0 = (int)(u - token * chunks) * heads, h1 = min(h0 + heads, H);
    bool inside = true;
    Angles a;
    if constexpr (PAIRS != NONE) {
      long at = p.pos ? (long)p.pos[token] : token % p.T;
      inside = at >= 0 && at < p.P;
      a = angles_of<PAIRS, BACK>(p, inside ? at : 0, c0);
    }
    const long base = (token * H + h0) * D;
    for (int h = h0; h < h1; h += FLIGHT) {
      const long row = base + (long)(h - h0) * D;
      typename Raw<TI, 8>::type vr[FLIGHT], qr[FLIGHT], tr[FLIGHT];
#pragma unroll
      for (int f = 0; f < FLIGHT; ++f)
        if (h + f < h1) {
          vr[f] = load_raw<TI, 8>(x + row + f * D + c0);
          if constexpr (BACK) {
            tr[f] = load_raw<TI, 8>(g + row + f * D + c0);
            qr[f] = partners<TI, PAIRS>(p, g + row + f * D, tr[f], c0);
          } else {
            qr[f] = partners<TI, PAIRS>(p, x + row + f * D, vr[f], c0);
          }
        }
#pragma unroll
      for (int f = 0; f < FLIGHT; ++f)
        if (h + f < h1) {
          Vals<8> v = widen<TI, 8>(vr[f]);
          const Vals<8> q = widen<TI, 8>(qr[f]);
          float ss = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(v[e], v[e], ss);
          ss = sum_lanes<LR>(ss);
          const float r = 1.f / sqrtf(__builtin_fmaf(ss, p.scale, p.eps));
          Vals<8> o;
          if constexpr (!BACK) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              o[e] = v[e] * r * w[e];
              if constexpr (PAIRS != NONE) o[e] = __builtin_fmaf(q[e] * r * wp[e], a.s[e], o[e] * a.c[e]);
            }
          } else {
            const Vals<8> t = widen<TI, 8>(tr[f]);
            Vals<8> gw;
            float dot = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              float gv = t[e];
              if constexpr (PAIRS != NONE) gv = __builtin_fmaf(q[e], a.s[e], gv * a.c[e]);
              const float unit = v[e] * r;
              if (inside) dw[e] = __builtin_fmaf(gv, unit, dw[e]);
              gw[e] = gv * w[e];
              dot = __builtin_fmaf(gw[e], unit, dot);
              v[e] = unit;
            }
            dot = sum_lanes<LR>(dot) * p.scale;
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = r * __builtin_fmaf(-v[e], dot, gw[e]);
          }
          if (!inside)
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = 0.f;
          store_vals<TI, 8>(y + row + f * D + c0, o);
        }
    }
  }

  if constexpr (BACK) {
    if (p.part[side]) {
      __shared__ float sums[GROUPS][D + 8];
#pragma unroll
      for (int e = 0; e < 8; ++e) sums[group][c0 + e] = dw[e];
      __syncthreads();
      if (tid < D) {
        float s = 0.f;
        for (int i = 0; i < GROUPS; ++i) s += sums[i][tid];
        p.part[side][(long)wg * D + tid] = s;
      }
    }
  }
}

// The partial sums' sums: 32 channels of one side a workgroup, 32 threads each
// (one workgroup a side took 14 us for 2,048 rows of 128, these 5).
__global__ __launch_bounds__(1024) void norm_weights_kernel(const NormParams p, int d, float* dwq, float* dwk) {
  __shared__ float sums[32][32];
  const int side = blockIdx.y, c = threadIdx.x & 31, k = threadIdx.x >> 5;
  float* out = side ? dwk : dwq;
  if (!out) return;
  const float* part = p.part[side] + blockIdx.x * 32 + c;
  float a = 0.f;
#pragma unroll 8
  for (int i = k; i < p.wgs[side]; i += 32) a += part[(long)i * d];
  sums[k][c] = a;
  __syncthreads();
  if (k) return;
  for (int i = 1; i < 32; ++i) a += sums[i][c];
  out[blockIdx.x * 32 + c] = a;
}

// ------------------------------------------------------------------- host --

// Workgroups for the queries (or keys): enough rows in flight to fill the
// device, and few enough that the weights' partial sums are small.
constexpr int MOST_WGS = 2048;

int heads_a_unit(long long tokens, int H, int d) {
  // Angles are read once a unit: as many heads as leave some 8,192 waves'
  // worth of units, up to 8.
  const long long waves = tokens * H * (d / 8) / 64;
  int heads = 1;
  while (heads < 8 && heads < H && waves / (heads * 2) >= 8192) heads *= 2;
  return heads;
}

int workgroups(long long tokens, int H, int heads, int d) {
  const long long units = tokens * ((H + heads - 1) / heads), groups = NT / (d / 8);
  return (int)std::max(1LL, std::min<long long>(MOST_WGS, (units + groups - 1) / groups));
}

template <typename TI, int D, bool BACK>
void launch_pairs(const NormParams& p, int pairs, hipStream_t s) {
  const dim3 grid(p.wgs[0] + p.wgs[1]);
  switch (pairs) {
    case NONE: hipLaunchKernelGGL((norm_kernel<TI, D, NONE, BACK>), grid, dim3(NT), 0, s, p); break;
    case HALVES: hipLaunchKernelGGL((norm_kernel<TI, D, HALVES, BACK>), grid, dim3(NT), 0, s, p); break;
    case HALVES_ODD: hipLaunchKernelGGL((norm_kernel<TI, D, HALVES_ODD, BACK>), grid, dim3(NT), 0, s, p); break;
    default: hipLaunchKernelGGL((norm_kernel<TI, D, NEIGHBOURS, BACK>), grid, dim3(NT), 0, s, p); break;
  }
}

template <bool BACK>
void launch(const NormParams& p, int d, int pairs, int dtype, hipStream_t s) {
  const bool bf = dtype == GDN_BF16;
  switch (d) {
    case 32: bf ? launch_pairs<__bf16, 32, BACK>(p, pairs, s) : launch_pairs<float, 32, BACK>(p, pairs, s); break;
    case 64: bf ? launch_pairs<__bf16, 64, BACK>(p, pairs, s) : launch_pairs<float, 64, BACK>(p, pairs, s); break;
    case 128: bf ? launch_pairs<__bf16, 128, BACK>(p, pairs, s) : launch_pairs<float, 128, BACK>(p, pairs, s); break;
    default: bf ? launch_pairs<__bf16, 256, BACK>(p, pairs, s) : launch_pairs<float, 256, BACK>(p, pairs, s); break;
  }
}

int sizes_checked(int B, int T, int Hq, int Hk, int d) {
  if (B < 0 || T < 0 || Hq < 1 || Hk < 1 || Hq > 65535 || Hk > 65535 || d < 1) return GDN_ERR_INVALID_ARG;
  const long long tokens = (long long)B * T;
  if (tokens > 0x7fffffffLL || tokens * std::max(Hq, Hk) >= 1LL << 36) return GDN_ERR_INVALID_ARG;
  if (d != 32 && d != 64 && d != 128 && d != 256) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

// One call, forwards (g null) or backwards.
int norm(const void* const x[2], const float* cos, const float* sin, const int32_t* pos, const float* const w[2],
         const void* const g[2], void* const y[2], float* const dw[2], int B, int T, int Hq, int Hk, int d, int rot,
         int P, float eps, void* stream, int dtype, int flags, void* workspace, long long workspace_bytes, bool back) {
  if (dtype != GDN_F32 && dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
  if (flags & ~(GDN_NORM_L2 | GDN_NORM_INTERLEAVED)) return GDN_ERR_INVALID_ARG;
  const int rc = sizes_checked(B, T, Hq, Hk, d);
  if (rc != GDN_OK) return rc;
  if (rot < 0 || rot > d || rot % 2 || !(eps >= 0.f) || !std::isfinite(eps)) return GDN_ERR_INVALID_ARG;
  if (rot > 0 && (!cos || !sin || P < 1)) return GDN_ERR_INVALID_ARG;
  const long long tokens = (long long)B * T;
  if (tokens > 0 && (!x[0] || !x[1] || !y[0] || !y[1] || (back && (!g[0] || !g[1])))) return GDN_ERR_INVALID_ARG;
  if (misaligned({x[0], x[1], y[0], y[1], g[0], g[1], cos, sin, w[0], w[1], dw[0], dw[1], workspace}, 16) ||
      misaligned(pos, 4))
    return GDN_ERR_INVALID_ARG;
  const bool weights = dw[0] || dw[1];
  const long long need = weights ? gdn_qk_norm_workspace_size(B, T, Hq, Hk, d) : 0;
  if (need > 0 && (!workspace || workspace_bytes < need)) return GDN_ERR_INVALID_ARG;
  const long long e = dtype == GDN_BF16 ? 2 : 4, q = tokens * Hq * d * e, k = tokens * Hk * d * e;
  const long long table = rot > 0 ? (long long)P * (rot / 2) * 4 : 0;
  if (clash({{y[0], q}, {y[1], k}, {dw[0], 4LL * d}, {dw[1], 4LL * d}, {need > 0 ? workspace : nullptr, need}},
            {{x[0], q}, {x[1], k}, {g[0], q}, {g[1], k}, {cos, table}, {sin, table}, {rot > 0 ? pos : nullptr, tokens * 4},
             {w[0], 4LL * d}, {w[1], 4LL * d}}))
    return GDN_ERR_INVALID_ARG;
  if (tokens == 0 && !weights) return GDN_OK;
  hipStream_t s = static_cast<hipStream_t>(stream);
  NormParams p = {};
  for (int i = 0; i < 2; ++i) {
    p.x[i] = x[i];
    p.g[i] = g[i];
    p.y[i] = y[i];
    p.w[i] = w[i];
    p.H[i] = i ? Hk : Hq;
    p.heads[i] = heads_a_unit(tokens, p.H[i], d);
    p.wgs[i] = tokens > 0 ? workgroups(tokens, p.H[i], p.heads[i], d) : 0;
  }
  if (weights) {
    p.part[0] = dw[0] ? static_cast<float*>(workspace) : nullptr;
    p.part[1] = dw[1] ? static_cast<float*>(workspace) + (long)p.wgs[0] * d : nullptr;
  }
  p.cos = cos;
  p.sin = sin;
  p.pos = pos;
  p.tokens = tokens;
  p.T = T;
  p.rot = rot;
  p.P = P;
  p.eps = eps;
  p.scale = flags & GDN_NORM_L2 ? 1.f : 1.f / (float)d;
  const int pairs = rot == 0 ? NONE : flags & GDN_NORM_INTERLEAVED ? NEIGHBOURS : rot % 16 ? HALVES_ODD : HALVES;
  if (tokens > 0) back ? launch<true>(p, d, pairs, dtype, s) : launch<false>(p, d, pairs, dtype, s);
  if (weights)
    hipLaunchKernelGGL(norm_weights_kernel, dim3(d / 32, 2), dim3(1024), 0, s, p, d, dw[0], dw[1]);
  return hipGetLastError() == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}

}  // namespace

extern "C" long long gdn_qk_norm_workspace_size(int B, int T, int Hq, int Hk, int d) {
  const int rc = sizes_checked(B, T, Hq, Hk, d);
  if (rc != GDN_OK) return rc;
  const long long tokens = (long long)B * T;
  if (tokens == 0) return 0;
  long long rows = 0;
  for (int H : {Hq, Hk}) rows += workgroups(tokens, H, heads_a_unit(tokens, H, d), d);
  return rows * d * 4;
}

extern "C" int gdn_qk_norm_fwd(const void* q, const void* k, const float* cos, const float* sin, const int32_t* pos,
                               const float* wq, const float* wk, void* qo, void* ko, int B, int T, int Hq, int Hk, int d,
                               int rot, int P, float eps, void* stream, int dtype, int flags) {
  const void* const x[2] = {q, k};
  const void* const g[2] = {nullptr, nullptr};
  const float* const w[2] = {wq, wk};
  void* const y[2] = {qo, ko};
  float* const dw[2] = {nullptr, nullptr};
  return norm(x, cos, sin, pos, w, g, y, dw, B, T, Hq, Hk, d, rot, P, eps, stream, dtype, flags, nullptr, 0, false);
}

extern "C" int gdn_qk_norm_bwd(const void* q, const void* k, const float* cos, const float* sin, const int32_t* pos,
                               const float* wq, const float* wk, const void* dqo, const void* dko, void* dq, void* dk,
                               float* dwq, float* dwk, int B, int T, int Hq, int Hk, int d, int rot, int P, float eps,
                               void* stream, int dtype, int flags, void* workspace, long long workspace_bytes) {
  const void* const x[2] = {q, k};
  const void* const g[2] = {dqo, dko};
  const float* const w[2] = {wq, wk};
  void* const y[2] = {dq, dk};
  float* const dw[2] = {dwq, dwk};
  return norm(x, cos, sin, pos, w, g, y, dw, B, T, Hq, Hk, d, rot, P, eps, stream, dtype, flags, workspace,
              workspace_bytes, true);
}

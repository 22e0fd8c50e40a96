// Depthwise causal convolution over W tokens with SiLU, forwards, backwards
// and on states in a pool, for gfx950.
//
// A lane owns V channels -- neighbours, 16 bytes of them, where D allows, else
// 64 apart, so that a wave's loads are whole lines at any alignment -- and walks
// down a segment of its sequence with the last W - 1 tokens in registers, so that
// a token is read once and, at a segment's start, W - 1 of them a second time.
// Bound by memory: x in, out out.
//
// Backwards the convolution is formed again (dy needs y), and a second window
// holds the last W - 1 dy: a token's dx is complete W - 1 tokens later, so a
// segment goes that far into the next one.  The parameters' gradients are
// summed by lane over its rows, then over the four waves of a workgroup, and a
// second launch adds the workgroups'.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "gdn_checks.h"
#include "gdn_conv.h"
#include "gdn_rows.h"

namespace {

constexpr int WAVES = 4;  // of a workgroup, each with a segment of its own

struct ConvParams {
  const void* x;
  const float* w;
  const float* bias;
  const void* h0;       // pooled: the pool
  const int32_t* cu;
  const int32_t* slots; // null: sequence n has state n
  void* out;
  void* hT;
  const void* dout;
  const void* dhT;
  void* dx;
  void* dh0;
  float* part;          // (workgroups, W + 1, D): sums for dw, then for dbias
  int B, T, D, nslots;
  int L, nseg;          // rows a segment, segments a dense sequence; 0: whole sequences
  long segments;
  int tiles;            // of 64 V channels
  int silu;
};

// A lane's V channels and its access to rows.  NEXT: neighbours, read and
// written at once; else 64 apart, the last tile's lanes behind D reading
// channel D - 1 and writing nothing.
template <typename TI, int V, bool NEXT>
struct Channels {
  int first, D;
  uint32_t place[NEXT ? 1 : V];  // in a row, bytes
  typedef typename std::conditional<NEXT, typename Raw<TI, V>::type, Vals<V>>::type raw;
  __device__ Channels(int tile, int lane, int D_) : first(tile * 64 * V + (NEXT ? lane * V : lane)), D(D_) {
    if constexpr (NEXT) place[0] = (uint32_t)first * sizeof(TI);
    else
#pragma unroll
      for (int i = 0; i < V; ++i) place[i] = (uint32_t)min(at(i), D - 1) * sizeof(TI);
  }
  __device__ int at(int i) const { return NEXT ? first + i : first + 64 * i; }
  __device__ bool has(int i) const { return NEXT ? first < D : at(i) < D; }
  __device__ raw load(const TI* row) {
    if constexpr (NEXT) {
      uintptr_t a = reinterpret_cast<uintptr_t>(row);
      asm("" : "+s"(a), "+v"(place[0]));
      return *(const __attribute__((address_space(1))) typename Raw<TI, V>::type*)(
          (const __attribute__((address_space(1))) char*)a + place[0]);
    } else {
      raw x;
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = __builtin_bit_cast(float, Row<TI>::load(row, place[i]));
      return x;
    }
  }
  __device__ Vals<V> widen(const raw& r) const {
    if constexpr (NEXT) return ::widen<TI, V>(r);
    else {
      Vals<V> x;
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = Row<TI>::widen(__builtin_bit_cast(uint32_t, r[i]));
      return x;
    }
  }
  __device__ Vals<V> get(const TI* row) { return widen(load(row)); }
  __device__ void put(TI* row, const Vals<V>& x) {
    if constexpr (NEXT) store_vals<TI, V>(row + first, x);
    else
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (has(i)) Row<TI>::store(row, place[i], x[i]);
  }
  // The same of fp32 vectors over the channels.
  __device__ Vals<V> param(const float* p) const {
    if constexpr (NEXT) return load_vals<float, V>(p + first);
    else {
      Vals<V> x;
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = p[min(at(i), D - 1)];
      return x;
    }
  }
};

template <int W, int V>
struct Taps {
  Vals<V> w[W], bias;
  template <typename TI, bool NEXT>
  __device__ Taps(const ConvParams& p, const Channels<TI, V, NEXT>& ch) {
    if constexpr (NEXT) {
      // V W neighbouring floats; V is a multiple of 4
      const float* at = p.w + (long)ch.first * W;
#pragma unroll
      for (int k = 0; k < V * W; k += 4) {
        const Vals<4> four = load_vals<float, 4>(at + k);
#pragma unroll
        for (int e = 0; e < 4; ++e) w[(k + e) % W][(k + e) / W] = four[e];
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][i] = p.w[(long)min(ch.at(i), p.D - 1) * W + j];
    }
#pragma unroll
    for (int i = 0; i < V; ++i) bias[i] = 0.f;
    if (p.bias) bias = ch.param(p.bias);
  }
  // The convolution at a token from the W - 1 before it and itself, oldest first.
  __device__ Vals<V> at(const Vals<V> (&before)[W - 1], const Vals<V>& x) const {
    Vals<V> y = bias;
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) y[i] = __builtin_fmaf(before[j][i], w[j][i], y[i]);
#pragma unroll
    for (int i = 0; i < V; ++i) y[i] = __builtin_fmaf(x[i], w[W - 1][i], y[i]);
    return y;
  }
};

template <int W, int V>
__device__ static inline void push(Vals<V> (&window)[W - 1], const Vals<V>& x) {
#pragma unroll
  for (int j = 0; j + 1 < W - 1; ++j) window[j] = window[j + 1];
  window[W - 2] = x;
}

// The W - 1 tokens before place t0 of a sequence whose first row is at x; the
// ones before its first are h's, or zeros.
template <int W, typename TI, int V, bool NEXT>
__device__ static inline void window_at(Vals<V> (&window)[W - 1], Channels<TI, V, NEXT>& ch, const TI* x, const TI* h,
                                        int t0) {
#pragma unroll
  for (int j = 0; j < W - 1; ++j) {
    const int t = t0 - (W - 1) + j;
    if (t >= 0) window[j] = ch.get(x + (long)t * ch.D);
    else if (h) window[j] = ch.get(h + (long)(t + W - 1) * ch.D);
    else
#pragma unroll
      for (int i = 0; i < V; ++i) window[j][i] = 0.f;
  }
}

// Rows on their way at once (4 x 4,096 x 1,280 bf16: forwards 17.8 us a call and
// backwards 32.6; 18.1 and 32.5 with two, 18.4 and 37.1 with eight; 4 x 2,048 x
// 1,024 fp32 forwards 12.8, 13.3 and 13.9).
constexpr int FLIGHT = 4;

// A wave's unit: a segment (uniform, and the compiler is told so) and a tile.
__device__ static inline long unit_of(const ConvParams& p) {
  return (long)(blockIdx.x / p.tiles) * WAVES + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
}

template <typename TI, int W, int V, bool NEXT>
__global__ __launch_bounds__(64 * WAVES) void conv_kernel(const ConvParams p) {
  const long unit = unit_of(p);
  if (unit >= p.segments) return;
  const Segment s = p.L ? segment_of(p.cu, p.B, p.T, p.L, p.nseg, unit) : sequence_of(p.cu, p.T, (int)unit);
  if (s.n < 0) return;
  SlotSearch search = p.slots ? SlotSearch(p.slots, s.n) : SlotSearch();
  const int D = p.D;
  Channels<TI, V, NEXT> ch(blockIdx.x % p.tiles, threadIdx.x & 63, D);
  const bool inside = ch.has(0);
  const TI* x = static_cast<const TI*>(p.x) + s.row0 * D;
  TI* out = static_cast<TI*>(p.out) + s.row0 * D;
  // The state is on its way while its slot is looked for among the earlier ones.
  const long at = (long)(p.slots ? __builtin_amdgcn_readfirstlane(search.slot) : s.n) * (W - 1) * D;
  const TI* h = p.h0 && (!p.slots || search.in(p.nslots)) ? static_cast<const TI*>(p.h0) + at : nullptr;
  Vals<V> window[W - 1];
  if (inside) window_at<W>(window, ch, x - (long)s.t0 * D, h, s.t0);
  const bool known = !p.slots || search.own(p.slots, p.nslots, s.n);
  if (!inside) return;
  if (!known) {
    Vals<V> zero;
#pragma unroll
    for (int i = 0; i < V; ++i) zero[i] = 0.f;
    for (int t = 0; t < s.len; ++t) ch.put(out + (long)t * D, zero);
    return;
  }
  const Taps<W, V> taps(p, ch);
  typename Channels<TI, V, NEXT>::raw next[FLIGHT];
#pragma unroll
  for (int f = 0; f < FLIGHT; ++f)
    if (f < s.len) next[f] = ch.load(x + (long)f * D);
  for (int t = 0; t < s.len; t += FLIGHT)
#pragma unroll
    for (int f = 0; f < FLIGHT; ++f)
      if (t + f < s.len) {
        const Vals<V> xv = ch.widen(next[f]);
        if (t + FLIGHT + f < s.len) next[f] = ch.load(x + (long)(t + FLIGHT + f) * D);
        Vals<V> y = taps.at(window, xv);
        if (p.silu)
#pragma unroll
          for (int i = 0; i < V; ++i) y[i] *= sigmoid(y[i]);
        ch.put(out + (long)(t + f) * D, y);
        push<W, V>(window, xv);
      }
  // The final state, by the wave that has read the initial one: hT may be h0.
  if (s.first()) {
    if (!s.last()) window_at<W>(window, ch, x, h, s.total);
    TI* hT = static_cast<TI*>(p.hT) + at;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) ch.put(hT + (long)j * D, window[j]);
  }
}

template <typename TI, int W, int V, bool NEXT>
__global__ __launch_bounds__(64 * WAVES) void conv_bwd_kernel(const ConvParams p) {
  __shared__ float sums[WAVES - 1][W + 1][64 * V];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, D = p.D;
  Channels<TI, V, NEXT> ch(blockIdx.x % p.tiles, lane, D);
  const long unit = unit_of(p);
  Segment s = {0, -1, 0, 0, 0};
  if (unit < p.segments) s = segment_of(p.cu, p.B, p.T, p.L, p.nseg, unit);
  Vals<V> dw[W], db;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    db[i] = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) dw[j][i] = 0.f;
  }
  if (s.n >= 0 && ch.has(0)) {
    const TI* x = static_cast<const TI*>(p.x) + s.row0 * D;
    const TI* dout = static_cast<const TI*>(p.dout) + s.row0 * D;
    TI* dx = static_cast<TI*>(p.dx) + s.row0 * D;
    const long at = (long)s.n * (W - 1) * D;
    const TI* h = p.h0 ? static_cast<const TI*>(p.h0) + at : nullptr;
    const TI* dhT = p.dhT ? static_cast<const TI*>(p.dhT) + at : nullptr;
    TI* dh0 = p.dh0 ? static_cast<TI*>(p.dh0) + at : nullptr;
    Vals<V> window[W - 1], dys[W - 1];
    window_at<W>(window, ch, x - (long)s.t0 * D, h, s.t0);
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) dys[j][i] = 0.f;
    const Taps<W, V> taps(p, ch);
    // rows of the segment and, for their dx, the W - 1 that follow
    const int rows = s.len + W - 1, there = s.total - s.t0, here = min(rows, there);
    typename Channels<TI, V, NEXT>::raw xn[FLIGHT], gn[FLIGHT];
#pragma unroll
    for (int f = 0; f < FLIGHT; ++f)
      if (f < here) {
        xn[f] = ch.load(x + (long)f * D);
        gn[f] = ch.load(dout + (long)f * D);
      }
    for (int t = 0; t < rows; t += FLIGHT) {
      // (all of a turn's loads at its beginning: a seventh more a call where each
      // row's follows the row before)
      typename Channels<TI, V, NEXT>::raw xr[FLIGHT], gr[FLIGHT];
#pragma unroll
      for (int f = 0; f < FLIGHT; ++f) {
        const int u = t + FLIGHT + f;
        xr[f] = xn[f];
        gr[f] = gn[f];
        if (u < here) {
          xn[f] = ch.load(x + (long)u * D);
          gn[f] = ch.load(dout + (long)u * D);
        }
      }
#pragma unroll
      for (int f = 0; f < FLIGHT; ++f) {
        const int u = t + f;
        if (u >= rows) break;
        Vals<V> dy, xv;
#pragma unroll
        for (int i = 0; i < V; ++i) dy[i] = xv[i] = 0.f;
        if (u < there) {
          xv = ch.widen(xr[f]);
          dy = ch.widen(gr[f]);
          if (p.silu) {
            const Vals<V> y = taps.at(window, xv);
#pragma unroll
            for (int i = 0; i < V; ++i) {
              const float q = sigmoid(y[i]);
              dy[i] *= q * __builtin_fmaf(y[i], 1.f - q, 1.f);
            }
          }
        }
        if (u < s.len)
#pragma unroll
          for (int i = 0; i < V; ++i) {
            db[i] += dy[i];
            dw[W - 1][i] = __builtin_fmaf(dy[i], xv[i], dw[W - 1][i]);
#pragma unroll
            for (int j = 0; j < W - 1; ++j) dw[j][i] = __builtin_fmaf(dy[i], window[j][i], dw[j][i]);
          }
        // the gradient W - 1 tokens back: the row's own tap is the last
        const int e = u - (W - 1);  // from the segment's start
        if (e >= 0 || s.first()) {
          Vals<V> d;
#pragma unroll
          for (int i = 0; i < V; ++i) {
            d[i] = dy[i] * taps.w[0][i];
#pragma unroll
            for (int j = 0; j < W - 1; ++j) d[i] = __builtin_fmaf(dys[j][i], taps.w[W - 1 - j][i], d[i]);
          }
          const int k = e - (there - (W - 1));  // its place in the final state
          if (dhT && k >= 0) {
            const Vals<V> more = ch.get(dhT + (long)k * D);
#pragma unroll
            for (int i = 0; i < V; ++i) d[i] += more[i];
          }
          if (e >= 0) ch.put(dx + (long)e * D, d);
          else if (dh0) ch.put(dh0 + (long)u * D, d);
        }
        push<W, V>(window, xv);
        push<W, V>(dys, dy);
      }
    }
  }
  if (wave) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
      for (int j = 0; j < W; ++j) sums[wave - 1][j][i * 64 + lane] = dw[j][i];
      sums[wave - 1][W][i * 64 + lane] = db[i];
    }
  }
  __syncthreads();
  if (wave == 0 && ch.has(0)) {
    float* part = p.part + (long)(blockIdx.x / p.tiles) * (W + 1) * D;
#pragma unroll
    for (int j = 0; j <= W; ++j) {
      Vals<V> a = j < W ? dw[j < W ? j : 0] : db;
#pragma unroll
      for (int k = 0; k < WAVES - 1; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) a[i] += sums[k][j][i * 64 + lane];
      if constexpr (NEXT) store_vals<float, V>(part + (long)j * D + ch.first, a);
      else
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (ch.has(i)) part[(long)j * D + ch.at(i)] = a[i];
    }
  }
}

// Sums over the workgroups' rows: 64 columns a workgroup, 16 threads each.
__global__ __launch_bounds__(1024) void conv_weights_kernel(const float* part, int rows, int D, int W, float* dw,
                                                           float* dbias) {
  __shared__ float sums[16][64];
  const int lane = threadIdx.x & 63, k = threadIdx.x >> 6;
  const long cols = (long)(W + 1) * D, c = (long)blockIdx.x * 64 + lane;
  float a = 0.f;
  if (c < cols)
#pragma unroll 8
    for (int i = k; i < rows; i += 16) a += part[i * cols + c];
  sums[k][lane] = a;
  __syncthreads();
  if (k == 0 && c < cols) {
    for (int i = 1; i < 16; ++i) a += sums[i][lane];
    const int j = (int)(c / D), d = (int)(c % D);
    if (j < W) dw[(long)d * W + j] = a;
    else if (dbias) dbias[d] = a;
  }
}

// ------------------------------------------------------------------- host --

// Rows a segment: 32 (each reads up to 2 (W - 1) rows more of what its
// neighbours read), fewer where that leaves less than some three waves for each
// vector unit.  Whole forward calls: 8 x 4,096 x 1,280 bf16 34 us with 32 rows,
// 40 with 16; 4 x 4,096 18 with 16, 21 with 32; 4 x 2,048 x 1,024 fp32 13 with 8,
// 18 with 16.
int rows_a_segment(long long rows, int D, int V, bool back) {
  int L = 32;
  const long long tiles = (D + 64 * V - 1) / (64 * V);
  while (L > (back ? 8 : 4) && rows / L * tiles < (back ? 2048 : 3000)) L /= 2;
  return L;
}

// Channels a lane: 16 bytes of neighbours forwards, 8 bytes of bf16 backwards
// (two windows and the sums in registers) where every row starts aligned to
// them, else four, 64 apart (6 x 32,530 rows of 271 channels, W 3: 75 us forwards
// and 120 backwards, 112 and 174 with one channel a lane), or one where there are
// not more than a wave's.
struct Width {
  int V;
  bool next;
};

Width channels(int D, int dtype, bool back) {
  const int want = dtype == GDN_F32 || back ? 4 : 8;
  if (D % want == 0) return {want, true};
  return {D > 64 ? 4 : 1, false};
}

int sizes_checked(int B, int T, int D, int W, bool packed, int dtype) {
  if (B < 0 || T < 0 || D < 1 || W < 1 || (dtype != GDN_F32 && dtype != GDN_BF16)) return GDN_ERR_INVALID_ARG;
  if ((packed ? 1LL : (long long)B) * T > MOST_ROWS || D >= 1 << 20 || B >= 1 << 24) return GDN_ERR_INVALID_ARG;
  if (W < 2 || W > 4) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

// A launch's units and grid (fewer than 2^24 workgroups: a grid holds fewer
// than 2^32 threads; segments get longer for that); false where it would be
// wider.
bool plan(ConvParams& p, int V, bool back, bool whole, unsigned& grid) {
  const long long rows = (p.cu ? 1LL : p.B) * (long long)p.T;
  p.tiles = (p.D + 64 * V - 1) / (64 * V);
  if (whole) {
    p.L = p.nseg = 0;
    p.segments = p.B;
  } else {
    p.L = rows_a_segment(rows, p.D, V, back);
    while (p.L < 1 << 20 && slots_of(p.cu != nullptr, p.B, p.T, p.L) / WAVES * p.tiles >= 1LL << 23) p.L *= 2;
    p.nseg = segments_of(p.T, p.L);
    p.segments = slots_of(p.cu != nullptr, p.B, p.T, p.L);
  }
  const long long wgs = (p.segments + WAVES - 1) / WAVES * p.tiles;
  grid = (unsigned)wgs;
  return wgs < 1LL << 24;
}

template <typename TI, int V, bool NEXT, bool BACK>
void launch(const ConvParams& p, int W, unsigned grid, hipStream_t s) {
  const dim3 g(grid), b(64 * WAVES);
  if constexpr (BACK) {
    if (W == 2) hipLaunchKernelGGL((conv_bwd_kernel<TI, 2, V, NEXT>), g, b, 0, s, p);
    else if (W == 3) hipLaunchKernelGGL((conv_bwd_kernel<TI, 3, V, NEXT>), g, b, 0, s, p);
    else hipLaunchKernelGGL((conv_bwd_kernel<TI, 4, V, NEXT>), g, b, 0, s, p);
  } else {
    if (W == 2) hipLaunchKernelGGL((conv_kernel<TI, 2, V, NEXT>), g, b, 0, s, p);
    else if (W == 3) hipLaunchKernelGGL((conv_kernel<TI, 3, V, NEXT>), g, b, 0, s, p);
    else hipLaunchKernelGGL((conv_kernel<TI, 4, V, NEXT>), g, b, 0, s, p);
  }
}

template <typename TI, bool BACK>
void launch_width(const ConvParams& p, Width w, int W, unsigned grid, hipStream_t s) {
  constexpr int MOST = BACK || sizeof(TI) == 4 ? 4 : 8;
  if (w.next) launch<TI, MOST, true, BACK>(p, W, grid, s);
  else if (w.V == 4) launch<TI, 4, false, BACK>(p, W, grid, s);
  else launch<TI, 1, false, BACK>(p, W, grid, s);
}

int forward(ConvParams p, int W, int dtype, int flags, void* stream) {
  const bool pooled = p.slots != nullptr;
  const int rc = sizes_checked(p.B, p.T, p.D, W, p.cu != nullptr, dtype);
  if (rc == GDN_ERR_INVALID_ARG || (flags & ~GDN_CONV_SILU)) return GDN_ERR_INVALID_ARG;
  if (p.B > 0 && (!p.w || !p.hT || (p.T > 0 && (!p.x || !p.out)))) return GDN_ERR_INVALID_ARG;
  if (rc != GDN_OK) return rc;
  if (misaligned({p.x, p.w, p.bias, p.h0, p.out, p.hT}, 16) || misaligned({p.cu, p.slots}, 4))
    return GDN_ERR_INVALID_ARG;
  const long long e = dtype == GDN_BF16 ? 2 : 4, rows = (p.cu ? 1LL : p.B) * (long long)p.T;
  const long long state = (pooled ? p.nslots : p.B) * (long long)(W - 1) * p.D * e;
  if (clash({{p.out, rows * p.D * e}, {p.hT, state}},
            {{p.x, rows * p.D * e}, {p.w, 4LL * p.D * W}, {p.bias, 4LL * p.D}, {p.cu, 4LL * (p.B + 1)},
             {p.slots, 4LL * p.B}, {p.h0 == p.hT ? nullptr : p.h0, state}}))
    return GDN_ERR_INVALID_ARG;
  if (p.B == 0) return GDN_OK;
  p.silu = flags & GDN_CONV_SILU;
  const Width w = channels(p.D, dtype, false);
  unsigned grid;
  if (!plan(p, w.V, false, pooled, grid)) return GDN_ERR_INVALID_ARG;
  hipStream_t s = static_cast<hipStream_t>(stream);
  dtype == GDN_BF16 ? launch_width<__bf16, false>(p, w, W, grid, s) : launch_width<float, false>(p, w, W, grid, s);
  return hipGetLastError() == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}

}  // namespace

extern "C" int gdn_conv_fwd(const void* x, const float* w, const float* bias, const void* h0,
                            const int32_t* cu_seqlens, void* out, void* hT, int B, int T, int D, int W, void* stream,
                            int dtype, int flags) {
  ConvParams p = {};
  p.x = x; p.w = w; p.bias = bias; p.h0 = h0; p.cu = cu_seqlens; p.out = out; p.hT = hT;
  p.B = B; p.T = T; p.D = D;
  return forward(p, W, dtype, flags, stream);
}

extern "C" int gdn_conv_fwd_pool(const void* x, const float* w, const float* bias, void* pool, const int32_t* slots,
                                 const int32_t* cu_seqlens, void* out, int nslots, int B, int T, int D, int W,
                                 void* stream, int dtype, int flags) {
  if (nslots < 0 || (B > 0 && !slots)) return GDN_ERR_INVALID_ARG;
  ConvParams p = {};
  p.x = x; p.w = w; p.bias = bias; p.h0 = pool; p.hT = pool; p.slots = slots; p.cu = cu_seqlens; p.out = out;
  p.B = B; p.T = T; p.D = D; p.nslots = nslots;
  return forward(p, W, dtype, flags, stream);
}

extern "C" long long gdn_conv_workspace_size(int B, int T, int D, int W, int packed, int dtype) {
  const int rc = sizes_checked(B, T, D, W, packed != 0, dtype);
  if (rc != GDN_OK) return rc;
  ConvParams p = {};
  p.B = B; p.T = T; p.D = D;
  p.cu = packed ? reinterpret_cast<const int32_t*>(16) : nullptr;  // only asked whether there is one
  unsigned grid;
  if (!plan(p, channels(D, dtype, true).V, true, false, grid)) return GDN_ERR_INVALID_ARG;
  return (long long)(grid / p.tiles) * (W + 1) * D * 4;
}

extern "C" int gdn_conv_bwd(const void* x, const float* w, const float* bias, const void* h0,
                            const int32_t* cu_seqlens, const void* dout, const void* dhT, void* dx, float* dw,
                            float* dbias, void* dh0, int B, int T, int D, int W, void* stream, int dtype, int flags,
                            void* workspace, long long workspace_bytes) {
  const bool packed = cu_seqlens != nullptr;
  const int rc = sizes_checked(B, T, D, W, packed, dtype);
  if (rc == GDN_ERR_INVALID_ARG || (flags & ~GDN_CONV_SILU) || !dw) return GDN_ERR_INVALID_ARG;
  if (B > 0 && (!w || (T > 0 && (!x || !dout || !dx)))) return GDN_ERR_INVALID_ARG;
  if (rc != GDN_OK) return rc;
  if (misaligned({x, w, bias, h0, dout, dhT, dx, dw, dbias, dh0, workspace}, 16) || misaligned(cu_seqlens, 4))
    return GDN_ERR_INVALID_ARG;
  const long long need = gdn_conv_workspace_size(B, T, D, W, packed, dtype);
  if (need < 0) return (int)need;
  if (need > 0 && (!workspace || workspace_bytes < need)) return GDN_ERR_INVALID_ARG;
  const long long e = dtype == GDN_BF16 ? 2 : 4, rows = (packed ? 1LL : B) * (long long)T;
  const long long state = (long long)B * (W - 1) * D * e, data = rows * D * e, taps = 4LL * D * W;
  if (clash({{dx, data}, {dw, taps}, {dbias, 4LL * D}, {dh0, state}, {workspace, need}},
            {{x, data}, {w, taps}, {bias, 4LL * D}, {cu_seqlens, 4LL * (B + 1)}, {h0, state}, {dout, data},
             {dhT, state}}))
    return GDN_ERR_INVALID_ARG;
  ConvParams p = {};
  p.x = x; p.w = w; p.bias = bias; p.h0 = h0; p.cu = cu_seqlens; p.dout = dout; p.dhT = dhT; p.dx = dx; p.dh0 = dh0;
  p.part = static_cast<float*>(workspace);
  p.B = B; p.T = T; p.D = D;
  p.silu = flags & GDN_CONV_SILU;
  const Width v = channels(D, dtype, true);
  unsigned grid;
  if (!plan(p, v.V, true, false, grid)) return GDN_ERR_INVALID_ARG;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (grid > 0) {
    dtype == GDN_BF16 ? launch_width<__bf16, true>(p, v, W, grid, s) : launch_width<float, true>(p, v, W, grid, s);
  }
  const long long cols = (long long)(W + 1) * D;
  hipLaunchKernelGGL(conv_weights_kernel, dim3((unsigned)((cols + 63) / 64)), dim3(1024), 0, s, p.part,
                     (int)(grid / p.tiles), D, W, dw, dbias);
  return hipGetLastError() == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}

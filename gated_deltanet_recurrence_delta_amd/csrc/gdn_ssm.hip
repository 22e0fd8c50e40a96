// The selective state space scan, forwards, backwards and on states in a
// pool, for gfx950.
//
// Per token, channel and state: a = exp(s A), h = a h + s x b, y += c h.  The
// decay is each channel's, state's and token's own, so nothing of it is a
// matrix product; what bounds the kernels is the vector unit: four
// instructions and an exponential for each of B T D N state updates, against
// some ten bytes of memory for each N of them.
//
// Forwards a lane owns a channel and holds its N states in registers; the
// token's keys, the same for all channels of a group, come through the scalar
// unit and cost no vector instruction.  Where channels and sequences are too
// few to fill the device, sequences are cut into segments (gdn_ssm.h).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "gdn_checks.h"
#include "gdn_rows.h"
#include "gdn_ssm.h"

namespace {

typedef float f4 __attribute__((ext_vector_type(4)));

constexpr float LOG2E = 1.44269504f;

struct SsmParams {
  const void* x;
  const void* dt;
  const void* b;
  const void* c;
  const float* A_log;
  const float* Dskip;
  const void* z;
  const float* dt_bias;
  const float* h0;       // pooled: the pool
  const int32_t* cu;
  const int32_t* slots;  // null: sequence n has state n
  void* out;
  float* hT;
  const void* dout;
  const float* dhT;
  void* dx;
  void* ddt;
  void* db;
  void* dc;
  float* dA_log;
  float* dD;
  void* dz;
  float* ddt_bias;
  float* dh0;
  float* E;      // (segments, D, N): the state a segment leaves from zero; then the state it starts from
  float* R;      // the same for the state's gradient, backwards in time
  float* S;      // (segments, D): the sum of a segment's steps
  float* keys;   // (tiles of workgroups, rows, G, 2, N): partial sums for db and dc
  float* sums;   // (runs of segments, D, N + 2): partial sums for dA_log, dD and ddt_bias
  int B, T, D, G, N, Dg, nslots;
  int L, nseg;   // rows a segment, segments a dense sequence
  long segments;
  int inner;     // forwards, packed: so many places for segments that are not their sequence's last, by the rows L apart
                 // (inner_segment_of); 0: segments are found by their slots
  int run, runs; // backwards: segments a workgroup, and workgroups' runs
  long rows;
  int softplus;
};

// ------------------------------------------------------------------- steps --

// log(1 + exp(v)) = max(v, 0) + log(1 + e), e = exp(-|v|), and with q = e / (2
// + e), log(1 + e) = 2 atanh(q): an odd polynomial of degree 9 in q <= 1/3,
// within 8e-9 relative.  Small steps keep their relative precision, which
// log2(1 + e) would lose.
__device__ static inline float softplus(float v) {
  const float e = __builtin_amdgcn_exp2f(__builtin_fabsf(v) * -LOG2E);
  const float q = e * __builtin_amdgcn_rcpf(2.f + e), w = q * q;
  float y = __builtin_fmaf(w, 0.281577796f, 0.279651582f);
  y = __builtin_fmaf(w, y, 0.400245965f);
  y = __builtin_fmaf(w, y, 0.666663229f);
  y = __builtin_fmaf(w, y, 2.f);
  return __builtin_fmaf(q, y, __builtin_fmaxf(v, 0.f));
}

__device__ static inline float step_of(float v, int soft) {
  const float s = softplus(v);  // no branch
  return soft ? s : v;
}

// A times log2(e), for decays as powers of two.  A finite number even where
// exp(A_log) is none: a step of zero (which tokens behind a segment's last take)
// leaves a state as it is.
__device__ static inline float rate_of(float A_log) {
  const float a = -LOG2E * expf(A_log);
  return a < -3e38f ? -3e38f : a;
}

// exp(A_log) as the factor of a gradient, a finite number likewise: where the
// sum over the tokens is zero, as it is for a state that keeps nothing, so is the
// product.
__device__ static inline float rate_factor(float A_log) {
  const float a = expf(A_log);
  return a > 3e38f ? 3e38f : a;
}

// -------------------------------------------------------------------- keys --

// Sixteen values of a token's key through the scalar unit: the address is the
// same in all lanes, and the constant address space says that nothing writes
// there while the kernel runs.
template <typename TI>
struct Keys16 {
  typedef uint32_t words __attribute__((ext_vector_type(sizeof(TI) * 4)));
  words w;
  __device__ void load(const TI* p) {
    w = *(const __attribute__((address_space(4))) words*)(uintptr_t)p;
  }
  // Makes the loaded values be there at this point of the instruction stream.
  // Scalar loads return in any order, so that a wait for one is a wait for all:
  // the next ones are to be issued behind it.
  __device__ void arrive() { asm volatile("" : "+s"(w)); }
  __device__ float operator[](int i) const {
    // (a value first: a bit cast of a vector's element itself took element 0)
    const uint32_t u = sizeof(TI) == 4 ? w[i] : i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16;
    return __builtin_bit_cast(float, u);
  }
};

// ---------------------------------------------------------- a lane a channel --

// Tokens on their way at once.
constexpr int FLIGHT = 4;

// A wave's place: a segment, a group and 64 of its channels.
struct Place {
  Segment s;
  long slot;
  int g, d;
  bool active;  // the lane's channel is one of the group's
};

// A workgroup is one wave: no wave waits for another, and any number of tiles is
// spread evenly.
template <bool LAST>
__device__ static inline Place place_of(const SsmParams& p) {
  const int lane = threadIdx.x & 63, tiles = (p.Dg + 63) >> 6;
  Place w;
  int k = blockIdx.x;
  const int c = k % tiles * 64 + lane;
  k /= tiles;
  w.g = k % p.G;
  w.slot = k / p.G;
  if (!p.inner) {
    w.s = segment_of(p.cu, p.B, p.T, p.L, p.nseg, w.slot);
  } else {
    // the sequences' last segments, then (alone where LAST is false) the others
    const int u = (int)w.slot, first = LAST ? p.B : 0;
    if (u < first) w.s = last_segment_of(p.cu, p.T, p.L, u, w.slot);
    else w.s = inner_segment_of(p.cu, p.B, p.T, p.L, u - first, w.slot);
  }
  w.active = c < p.Dg;
  w.d = w.g * p.Dg + min(c, p.Dg - 1);
  return w;
}

template <int N>
__device__ static inline void load_states(Vals<N>& h, const float* p) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const Vals<4> q = load_vals<float, 4>(p + i);
#pragma unroll
    for (int e = 0; e < 4; ++e) h[i + e] = q[e];
  }
}

template <int N>
__device__ static inline void store_states(float* p, const Vals<N>& h) {
#pragma unroll
  for (int i = 0; i < N; i += 4) store_vals<float, 4>(p + i, Vals<4>{{h[i], h[i + 1], h[i + 2], h[i + 3]}});
}

// Sixteen of a token's write and read keys.
template <typename TI, bool READ>
struct KeyPair {
  Keys16<TI> b, c;
  __device__ void load(const TI* bk, const TI* ck) {
    b.load(bk);
    if constexpr (READ) c.load(ck);
  }
  __device__ void arrive() {
    b.arrive();
    if constexpr (READ) c.arrive();
  }
};

// Forwards.  OUTPUT: the outputs from the segment's start state (E if the
// sequence is cut, else h0).  Otherwise the state that a segment leaves from
// zero, and the sum of its steps; what follows the last segment is hT, which
// the outputs' launch gives.
//
// Bound by the vector unit's instructions: a state's update takes 27.5 cycles of it
// (a multiplication for the exponent, the exponential's 9.7, a product, two fused
// ones).  8 x 4,096 tokens of 1,280 channels, N 16: 254 us, 42% of it the states that
// segments leave and 5% the join; 117 would be one pass's updates.
template <typename TI, int N, bool OUTPUT>
__global__ __launch_bounds__(64) void ssm_kernel(const SsmParams p) {
  const Place w = place_of<OUTPUT>(p);
  if (w.s.n < 0 || (!OUTPUT && w.s.last()) || !w.active) return;
  const int D = p.D, d = w.d;
  Vals<N> A, h;
  load_states<N>(A, p.A_log + (long)d * N);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    A[i] = rate_of(A[i]);
    h[i] = 0.f;
  }
  if constexpr (OUTPUT) {
    if (p.E && !(w.s.first() && w.s.last())) load_states<N>(h, p.E + (w.slot * D + d) * N);
    else if (p.h0) load_states<N>(h, p.h0 + ((long)w.s.n * D + d) * N);
  }
  const float bias = p.dt_bias ? p.dt_bias[d] : 0.f, skip = OUTPUT && p.Dskip ? p.Dskip[d] : 0.f;
  uint32_t lane = (uint32_t)d * sizeof(TI);
  const long at = w.s.row0 * D;
  const TI* x = static_cast<const TI*>(p.x) + at;
  const TI* dt = static_cast<const TI*>(p.dt) + at;
  const TI* z = (p.z ? static_cast<const TI*>(p.z) : static_cast<const TI*>(p.x)) + at;
  TI* out = static_cast<TI*>(p.out) + (OUTPUT ? at : 0);
  const int len = w.s.len;
  float S = 0.f;

  if (len > 0) {
    uint32_t xn[FLIGHT], dn[FLIGHT], zn[FLIGHT];
#pragma unroll
    for (int f = 0; f < FLIGHT; ++f) {
      const long o = (long)min(f, len - 1) * D;
      xn[f] = Row<TI>::load(x + o, lane);
      dn[f] = Row<TI>::load(dt + o, lane);
      if (OUTPUT) zn[f] = Row<TI>::load(z + o, lane);
    }
    // The keys of the next sixteen states are on their way while these are
    // worked on: two sets, taken in turn.
    const long KS = (long)p.G * N;
    const TI* bk = static_cast<const TI*>(p.b) + (w.s.row0 * p.G + w.g) * N;
    const TI* ck = static_cast<const TI*>(p.c) + (w.s.row0 * p.G + w.g) * N;
    KeyPair<TI, OUTPUT> keys[2];
    keys[0].load(bk, ck);
    for (int t = 0; t < len; t += FLIGHT) {
      // Tokens behind the segment's last take a step of zero: the states stay.
      // (No branch on the way, or what is to be in flight sinks below it: tokens
      // behind the last store the last one's output once more.)
      float y_last = 0.f;
#pragma unroll
      for (int f = 0; f < FLIGHT; ++f) {
        const float xv = Row<TI>::widen(xn[f]), v = Row<TI>::widen(dn[f]) + bias, soft = softplus(v);
        const float zv = OUTPUT ? Row<TI>::widen(zn[f]) : 0.f;
        const long o = (long)min(t + FLIGHT + f, len - 1) * D;
        xn[f] = Row<TI>::load(x + o, lane);
        dn[f] = Row<TI>::load(dt + o, lane);
        if (OUTPUT) zn[f] = Row<TI>::load(z + o, lane);
        const float s = t + f < len ? p.softplus ? soft : v : 0.f, u = s * xv;
        float y = 0.f;
        if constexpr (!OUTPUT) S += s;
#pragma unroll
        for (int n = 0; n < N; n += 16) {
          KeyPair<TI, OUTPUT>&now = keys[(f * (N / 16) + n / 16) & 1], &next = keys[(f * (N / 16) + n / 16 + 1) & 1];
          // (behind the last token: its own again)
          const long step = n + 16 < N ? 16 : (t + f + 1 < len ? KS : 0) - (N - 16);
          bk += step;
          ck += step;
          now.arrive();
          __builtin_amdgcn_sched_barrier(0);
          next.load(bk, ck);
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float a = __builtin_amdgcn_exp2f(s * A[n + i]);
            h[n + i] = __builtin_fmaf(a, h[n + i], u * now.b[i]);
            if constexpr (OUTPUT) y = __builtin_fmaf(now.c[i], h[n + i], y);
          }
        }
        if constexpr (OUTPUT) {
          const float gate = zv * sigmoid(zv);
          y = __builtin_fmaf(skip, xv, y) * (p.z ? gate : 1.f);
          y_last = t + f < len ? y : y_last;
          Row<TI>::store(out + (long)min(t + f, len - 1) * D, lane, y_last);
        }
      }
    }
  }
  if constexpr (OUTPUT) {
    if (w.s.last()) store_states<N>(p.hT + ((long)w.s.n * D + d) * N, h);
  } else {
    store_states<N>(p.E + (w.slot * D + d) * N, h);
    p.S[w.slot * D + d] = S;
  }
}

// Joins the segments of each sequence, a thread for each state and each of
// GROUPS parts of its segments: the parts are folded, then walked from the
// state that the ones before leave.  Forwards E, the state each segment leaves
// from zero, becomes the one it starts from; backwards in time R, likewise, for
// the state's gradient (blockIdx.y == 1).
//
// Bound by the latency of a chain of loads: 200 segments of 20,480 states take
// 25 us in one part.
template <int GROUPS>
__global__ __launch_bounds__(256) void ssm_join_kernel(const SsmParams p) {
  constexpr int STATES = 256 / GROUPS, F = 16;  // segments on their way at once
  __shared__ float ends[GROUPS][STATES], sums[GROUPS][STATES];
  const long DN = (long)p.D * p.N;
  const int lane = threadIdx.x % STATES, group = threadIdx.x / STATES;
  const bool back = blockIdx.y;
  long from = (long)blockIdx.x * STATES, to = p.B * DN, stride = (long)gridDim.x * STATES;
  if (p.inner) {  // some workgroups for each row k L, and work where it is the first such row of a cut sequence
    const int parts = gridDim.x / p.inner, row = (int)(blockIdx.x / parts) * p.L, n = sequence_at(p.cu, p.B, p.T, row);
    if (n < 0) return;
    const int b = taken(p.cu[n], 0, p.T), e = taken(p.cu[n + 1], b, p.T);
    if (row < b || row - b >= p.L || e - b <= p.L) return;
    from = n * DN + (long)(blockIdx.x % parts) * STATES;
    to = (n + 1) * DN;
    stride = (long)parts * STATES;
  }
  for (long id0 = from; id0 < to; id0 += stride) {
    const long id = min(id0 + lane, to - 1);
    const int n = (int)(id / DN);
    const long r = id - n * DN;
    const int d = (int)(r / p.N);
    long slot = (long)n * p.nseg;
    int count = p.T > 0 ? p.nseg : 0;
    if (p.cu) {
      const int b = taken(p.cu[n], 0, p.T), e = taken(p.cu[n + 1], b, p.T);
      slot = b / p.L + n;
      count = (int)min((long)(e - b + p.L - 1) / p.L, max(p.segments - slot, 0L));
    }
    const float A = rate_of(p.A_log[r]);
    float* state = (back ? p.R : p.E) + r;
    const float* first = back ? p.dhT : p.h0;
    const int part = (count + GROUPS - 1) / GROUPS, i0 = min(group * part, count), i1 = min(i0 + part, count);
    const long step = back ? -1 : 1, begin = back ? slot + count - 1 : slot;
    // (read before the parts meet: the last part's thread writes dh0, which may be dhT itself)
    const float begun = first ? first[id] : 0.f;
    float h = 0.f, e[F], s[F];
    auto load = [&](int i) {
#pragma unroll
      for (int f = 0; f < F; ++f) {
        const long k = begin + step * min(i + f, i1 - 1);
        e[f] = state[k * DN];
        s[f] = p.S[k * p.D + d];
      }
    };
    if constexpr (GROUPS > 1) {
      float S = 0.f;
      for (int i = i0; i < i1; i += F) {
        load(i);
#pragma unroll
        for (int f = 0; f < F; ++f)
          if (i + f < i1) {
            h = __builtin_fmaf(__builtin_amdgcn_exp2f(A * s[f]), h, e[f]);
            S += s[f];
          }
      }
      __syncthreads();  // the sums of the states before have been read
      ends[group][lane] = h;
      sums[group][lane] = S;
      __syncthreads();
    }
    h = begun;
    if constexpr (GROUPS > 1)
      for (int g = 0; g < group; ++g) h = __builtin_fmaf(__builtin_amdgcn_exp2f(A * sums[g][lane]), h, ends[g][lane]);
    if (id0 + lane >= to) continue;
    for (int i = i0; i < i1; i += F) {
      load(i);
#pragma unroll
      for (int f = 0; f < F; ++f)
        if (i + f < i1) {
          state[(begin + step * (i + f)) * DN] = h;
          // a forward call's last segment has no state of its own here, and none is needed
          h = __builtin_fmaf(__builtin_amdgcn_exp2f(A * s[f]), h, e[f]);
        }
    }
    if (group != GROUPS - 1) continue;
    if (back && p.dh0) p.dh0[id] = h;
  }
}

// --------------------------------------------------------- token by token --

template <int J>
__device__ static inline float from_quad(float x) {
  return dpp<J * 0x55>(x);
}

__device__ static inline Vals<4> quad(float x) {
  return {{from_quad<0>(x), from_quad<1>(x), from_quad<2>(x), from_quad<3>(x)}};
}

// Four sums over a quad's lanes: lane j gets the j-th, over all LC lanes where
// that is more than four.
template <int LC>
__device__ static inline float sum_own(const Vals<4>& v, bool odd, bool high) {
  const float a = (odd ? v[1] : v[0]) + dpp<0xB1>(odd ? v[0] : v[1]);
  const float b = (odd ? v[3] : v[2]) + dpp<0xB1>(odd ? v[2] : v[3]);
  float r = (high ? b : a) + dpp<0x4E>(high ? a : b);
  if constexpr (LC == 8) r += __int_as_float(__builtin_amdgcn_ds_swizzle(__float_as_int(r), (4 << 10) | 0x1f));
  if constexpr (LC == 16) {
    r += dpp<0x128>(r);  // row_ror 8
    r += dpp<0x124>(r);  // row_ror 4
  }
  return r;
}

// Few tokens on states read and written once: a lane holds four neighbouring
// states (16 bytes), so that a wave's accesses cover whole lines; N / 4 lanes
// are a channel.  Tokens are taken four a turn: lane 4 i + j forms the step and
// gate of the turn's token j and writes its output, and what the others need of
// them comes by DPP, so that a token costs a lane some 45 instructions, not 95.
// TURNS turns are on their way at once.
//
// Bound by memory for one token each (N 16: 128 sequences of 1,280 channels 7.9 us,
// 4.7 at a large copy's rate; 512 of 2,560 channels 41 to 43 us, 37 at that rate); for
// longer sequences of few channels by one wave's instructions, some 0.13 us a token.
template <typename TI, int N, int TURNS, int TOKENS, bool STREAM>
__global__ __launch_bounds__(256) void ssm_recurrent_kernel(const SsmParams p) {
  constexpr int LC = N / 4, CH = 256 / LC;
  const int tiles = (p.D + CH - 1) / CH;
  const int n = blockIdx.x / tiles, tile = blockIdx.x % tiles;
  const int slice = threadIdx.x % LC, d = tile * CH + threadIdx.x / LC, own = slice & (TOKENS - 1);
  const bool odd = slice & 1, high = slice & 2;
  const Segment s = sequence_of(p.cu, p.T, n);
  const int D = p.D, len = s.len;
  const bool inside = d < D;
  // The state is on its way while its slot is looked for among the earlier ones.
  SlotSearch search = p.slots ? SlotSearch(p.slots, n) : SlotSearch();
  const long sat = ((long)(p.slots ? search.slot : n) * D + d) * N + slice * 4;
  Vals<4> h = {{0.f, 0.f, 0.f, 0.f}}, A = h;
  float bias = 0.f, skip = 0.f;
  if (inside) {
    if (p.h0 && (!p.slots || search.in(p.nslots))) {
      const f4* from = reinterpret_cast<const f4*>(p.h0 + sat);
      f4 q;
      if constexpr (STREAM) q = __builtin_nontemporal_load(from);
      else q = *from;
      h = Vals<4>{{q[0], q[1], q[2], q[3]}};
    }
    A = load_vals<float, 4>(p.A_log + (long)d * N + slice * 4);
    if (p.dt_bias) bias = p.dt_bias[d];
    if (p.Dskip) skip = p.Dskip[d];
  }
  const TI* x = static_cast<const TI*>(p.x) + s.row0 * D + d;
  const TI* dt = static_cast<const TI*>(p.dt) + s.row0 * D + d;
  const TI* z = p.z ? static_cast<const TI*>(p.z) + s.row0 * D + d : x;
  const long key = (s.row0 * p.G + d / p.Dg) * N + slice * 4, KS = (long)p.G * N;
  const TI* bk = static_cast<const TI*>(p.b) + key;
  const TI* ck = static_cast<const TI*>(p.c) + key;
  TI xn[TURNS], dn[TURNS], zn[TURNS];
  typename Raw<TI, 4>::type bn[TURNS][TOKENS], cn[TURNS][TOKENS];
  auto load = [&](int k, int t) {
    const long o = (long)min(t + own, len - 1) * D;
    xn[k] = x[o];
    dn[k] = dt[o];
    zn[k] = z[o];
#pragma unroll
    for (int f = 0; f < TOKENS; ++f) {
      const long u = min(t + f, len - 1) * KS;
      bn[k][f] = load_raw<TI, 4>(bk + u);
      cn[k][f] = load_raw<TI, 4>(ck + u);
    }
  };
  // What a turn's tokens need of their own: formed while the turn before is
  // worked on.  Tokens behind the last take a step of zero.
  struct Own {
    float step, u, skip, gate;
  };
  if (inside && len > 0)
#pragma unroll
    for (int k = 0; k < TURNS; ++k) load(k, TOKENS * k);
  const bool known = !p.slots || search.own(p.slots, p.nslots, n);
  if (!inside) return;
  TI* out = static_cast<TI*>(p.out) + s.row0 * D + d;
  if (!known) {
    for (int t = slice; t < len; t += LC) out[(long)t * D] = (TI)0.f;
    return;
  }
  auto own_of = [&](int k, int t) {
    const float xv = (float)xn[k], zv = (float)zn[k], step = step_of((float)dn[k] + bias, p.softplus);
    const float gate = zv * sigmoid(zv), st = t + own < len ? step : 0.f;
    return Own{st, st * xv, skip * xv, p.z ? gate : 1.f};
  };
  Own now = {0.f, 0.f, 0.f, 0.f};
  if (len > 0) now = own_of(0, 0);
#pragma unroll
  for (int i = 0; i < 4; ++i) A[i] = rate_of(A[i]);
  for (int t0 = 0; t0 < len; t0 += TOKENS * TURNS)
#pragma unroll
    for (int k = 0; k < TURNS; ++k) {
      const int t = t0 + TOKENS * k;
      if (t >= len) break;
      Vals<4> b[TOKENS], c[TOKENS], y = {{0.f, 0.f, 0.f, 0.f}};
#pragma unroll
      for (int f = 0; f < TOKENS; ++f) {
        b[f] = widen<TI, 4>(bn[k][f]);
        c[f] = widen<TI, 4>(cn[k][f]);
      }
      const Own own_now = now;
      if (t + TOKENS * TURNS < len) {
        load(k, t + TOKENS * TURNS);
        if constexpr (TURNS == 1) now = own_of(0, t + TOKENS);
      }
      if constexpr (TURNS > 1) now = own_of((k + 1) % TURNS, t + TOKENS);
      const Vals<4> sv = TOKENS == 1 ? Vals<4>{{own_now.step}} : quad(own_now.step);
      const Vals<4> uv = TOKENS == 1 ? Vals<4>{{own_now.u}} : quad(own_now.u);
#pragma unroll
      for (int f = 0; f < TOKENS; ++f)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          h[i] = __builtin_fmaf(__builtin_amdgcn_exp2f(sv[f] * A[i]), h[i], uv[f] * b[f][i]);
          y[f] = __builtin_fmaf(c[f][i], h[i], y[f]);
        }
      const float o = (own_now.skip + (TOKENS == 1 ? sum_lanes<LC>(y[0]) : sum_own<LC>(y, odd, high))) * own_now.gate;
      if (slice < TOKENS && t + own < len) out[(long)(t + own) * D] = (TI)o;
    }
  f4* to = reinterpret_cast<f4*>(p.hT + sat);
  const f4 q = {h[0], h[1], h[2], h[3]};
  if constexpr (STREAM) __builtin_nontemporal_store(q, to);
  else *to = q;
}

// ---------------------------------------------------------------- backwards --
//
// Segments of at most some 25 tokens.  A first launch forms, for sixteen states of a
// channel, what a segment leaves from zero: the state E going forwards and,
// going backwards in time, the state's gradient, R = sum_t exp(A (s_1 + .. +
// s_t)) c_t dy_t, which one forward walk gives too.  The join makes of them the
// state a segment starts from and the gradient that reaches its end.

template <typename TI>
__device__ static inline void bwd_map(const SsmParams& p, long k, int tiles, int parts) {
  const int lane = threadIdx.x & 63, part = (int)(k % parts);
  k /= parts;
  const int tile = (int)(k % tiles);
  k /= tiles;
  const int g = (int)(k % p.G);
  const long slot = k / p.G;
  const Segment s = segment_of(p.cu, p.B, p.T, p.L, p.nseg, slot);
  if (s.n < 0) return;
  const int c = tile * 64 + lane, D = p.D, d = g * p.Dg + min(c, p.Dg - 1), N = p.N;
  const long KS = (long)p.G * N, sat = (slot * D + d) * N + part * 16;
  Vals<16> A, E, P, R;
  load_states<16>(A, p.A_log + (long)d * N + part * 16);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    A[i] = rate_of(A[i]);
    E[i] = R[i] = 0.f;
    P[i] = 1.f;
  }
  const float bias = p.dt_bias ? p.dt_bias[d] : 0.f;
  uint32_t at = (uint32_t)d * sizeof(TI);
  const TI* x = static_cast<const TI*>(p.x) + s.row0 * D;
  const TI* dt = static_cast<const TI*>(p.dt) + s.row0 * D;
  const TI* z = (p.z ? static_cast<const TI*>(p.z) : static_cast<const TI*>(p.x)) + s.row0 * D;
  const TI* dout = static_cast<const TI*>(p.dout) + s.row0 * D;
  const TI* bk = static_cast<const TI*>(p.b) + (s.row0 * p.G + g) * N + part * 16;
  const TI* ck = static_cast<const TI*>(p.c) + (s.row0 * p.G + g) * N + part * 16;
  const int len = s.len;
  float S = 0.f;
  if (len > 0) {
    uint32_t xn[FLIGHT], dn[FLIGHT], zn[FLIGHT], gn[FLIGHT];
    auto load = [&](int f, int t) {
      const long o = (long)min(t, len - 1) * D;
      xn[f] = Row<TI>::load(x + o, at);
      dn[f] = Row<TI>::load(dt + o, at);
      zn[f] = Row<TI>::load(z + o, at);
      gn[f] = Row<TI>::load(dout + o, at);
    };
#pragma unroll
    for (int f = 0; f < FLIGHT; ++f) load(f, f);
    KeyPair<TI, true> keys[2];
    keys[0].load(bk, ck);
    // as ssm_kernel: no branch, tokens behind the last take a step of zero and
    // have no gradient
    for (int t = 0; t < len; t += FLIGHT)
#pragma unroll
      for (int f = 0; f < FLIGHT; ++f) {
        const bool there = t + f < len;
        const float zv = Row<TI>::widen(zn[f]), xv = Row<TI>::widen(xn[f]), gate = zv * sigmoid(zv);
        const float step = step_of(Row<TI>::widen(dn[f]) + bias, p.softplus), st = there ? step : 0.f, u = st * xv;
        const float dy = there ? Row<TI>::widen(gn[f]) * (p.z ? gate : 1.f) : 0.f;
        load(f, t + FLIGHT + f);
        S += st;
        KeyPair<TI, true>&now = keys[f & 1], &next = keys[(f + 1) & 1];
        const long more = t + f + 1 < len ? KS : 0;
        bk += more;
        ck += more;
        now.arrive();
        __builtin_amdgcn_sched_barrier(0);
        next.load(bk, ck);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float a = __builtin_amdgcn_exp2f(st * A[i]);
          E[i] = __builtin_fmaf(a, E[i], u * now.b[i]);
          P[i] *= a;
          R[i] = __builtin_fmaf(P[i], dy * now.c[i], R[i]);
        }
      }
  }
  if (c >= p.Dg) return;
  store_states<16>(p.E + sat, E);
  store_states<16>(p.R + sat, R);
  if (part == 0) p.S[slot * D + d] = S;
}

template <typename TI>
__global__ __launch_bounds__(256) void ssm_bwd_maps_kernel(const SsmParams p) {
  // units: (segment, group, tile of 64 channels, sixteen of the states)
  const int tiles = (p.Dg + 63) >> 6, parts = p.N / 16;
  const long units = p.segments * p.G * tiles * parts;
  for (long k = (long)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); k < units;
       k += (long)gridDim.x * 4)
    bwd_map<TI>(p, k, tiles, parts);
}

// The gradients.  A wave has 1024 / N channels and all their states; a lane has
// a block of four channels (its group's) by four states (its slice's), so that
// half of both sums, over states and over channels, is within the lane.  Lane
// 4 i + j also owns channel j of its group for what is the channel's alone: the
// step, the gate, the stores.  Those values go to the other lanes by DPP.
//
// A segment is at most NB blocks of BT tokens.  A walk forwards keeps the states
// at the blocks' starts; then, from the last block on, a block's states are formed
// again and kept in registers, and its tokens are taken backwards.
//
// Bound by the vector unit's instructions, three exponentials a state's update
// among them (5,003 rows of 640 channels, N 32: 138 to 146 us, the maps 52, against 71 for
// both passes forwards).

// More tokens a block need more registers, more blocks more LDS (a workgroup of
// four waves has 80 KB of it and 256 registers, so that two share a compute
// unit), and shorter segments more joining (4 x 4,096 x 1,280, N 16, whole
// calls: 4 x 6 513 us, 4 x 5 542, 5 x 6 522, 6 x 5 541, 8 x 4 560).
template <int N>
struct Blocks {
  static constexpr int BT = 4, NB = N == 16 ? 6 : 5, BL = BT * NB;
};
int most_blocks(int N) { return N == 16 ? Blocks<16>::NB : N == 32 ? Blocks<32>::NB : Blocks<64>::NB; }

// a and b become (a's lanes below 32, b's below 32) and (a's from 32 on, b's
// from 32 on): their sum then holds a's over both halves in the lower lanes
// and b's in the upper ones, one instruction and one addition for two sums.
// swap_rows does the same within each half, sixteen lanes by sixteen.
__device__ static inline void swap_halves(float& a, float& b) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  a = __uint_as_float(r[0]);
  b = __uint_as_float(r[1]);
}
__device__ static inline void swap_rows(float& a, float& b) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  a = __uint_as_float(r[0]);
  b = __uint_as_float(r[1]);
}

template <typename TI, int N, bool GATE, int WAVES>
__global__ __launch_bounds__(64 * WAVES, 2) void ssm_bwd_kernel(const SsmParams p) {
  constexpr int BT = Blocks<N>::BT, NB = Blocks<N>::NB, BL = BT * NB, NT = 64 * WAVES;
  constexpr int LC = N / 4;            // lanes a channel
  constexpr int CT = 1024 / N;         // channels a wave
  __shared__ __attribute__((aligned(16))) float key[BL][2][N];
  __shared__ __attribute__((aligned(16))) float start[WAVES][NB - 2][16][64];
  __shared__ __attribute__((aligned(16))) float part[2][WAVES][BT][2][N];

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int tiles = (p.Dg + CT - 1) / CT, teams = (tiles + WAVES - 1) / WAVES;
  int k = blockIdx.x;
  const int team = k % teams;
  k /= teams;
  const int g = k % p.G, run = k / p.G;
  const int D = p.D, tile = team * WAVES + wave;
  const int slice = lane % LC, group = lane / LC;
  const bool odd = lane & 1, high = lane & 2;
  // channels of the lane's block, and its own
  const int c0 = tile * CT + group * 4, cown = c0 + (lane & 3);
  // Lanes behind the group's last channel work on copies of it, with inputs and
  // gradients of zero, so that they add nothing to the sums over channels.
  const bool real = cown < p.Dg, mine = real && slice < 4;
  const int own = g * p.Dg + min(cown, p.Dg - 1);
  // places in a row of channels (bytes) and in a segment's states (floats)
  uint32_t lane_at = (uint32_t)own * sizeof(TI), state_at[4];
  const uint32_t mine_at = mine ? lane_at : 1u << 30;  // (no row has that many bytes)
#pragma unroll
  for (int c = 0; c < 4; ++c) state_at[c] = (uint32_t)(g * p.Dg + min(c0 + c, p.Dg - 1)) * N + slice * 4;

  float A[4][4], dA[4][4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const Vals<4> a = load_vals<float, 4>(p.A_log + state_at[c]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      A[c][j] = rate_of(a[j]);
      dA[c][j] = 0.f;
    }
  }
  const float bias = p.dt_bias ? p.dt_bias[own] : 0.f, skip = p.Dskip ? p.Dskip[own] : 0.f;
  float dD = 0.f, dbias = 0.f;
  const TI* xs = static_cast<const TI*>(p.x);
  const TI* dts = static_cast<const TI*>(p.dt);
  const TI* zs = static_cast<const TI*>(p.z);
  const TI* gs = static_cast<const TI*>(p.dout);
  const TI* bs = static_cast<const TI*>(p.b);
  const TI* cs = static_cast<const TI*>(p.c);
  int turn = 0;

  for (int r = 0; r < p.run; ++r) {
    const long slot = (long)run * p.run + r;
    if (slot >= p.segments) break;
    const Segment s = segment_of(p.cu, p.B, p.T, p.L, p.nseg, slot);
    if (s.n < 0 || s.len == 0) continue;
    const long row0 = s.row0;
    const int len = s.len;
    __syncthreads();  // the keys of the segment before have been read
    for (int i = tid; i < len * N; i += NT) {
      const int t = i / N, n = i % N;
      const long o = ((row0 + t) * p.G + g) * N + n;
      key[t][0][n] = (float)bs[o];
      key[t][1][n] = (float)cs[o];
    }
    __syncthreads();

    float h[4][4], l[4][4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const Vals<4> e = load_vals<float, 4>(p.E + slot * D * N + state_at[c]);
      const Vals<4> q = load_vals<float, 4>(p.R + slot * D * N + state_at[c]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        h[c][j] = e[j];
        l[c][j] = q[j];  // exp(s A) times the next token's gradient
      }
    }
    const int blocks = (len + BT - 1) / BT;
    // the states at the blocks' starts
    const long at = row0 * D;
#pragma unroll 1
    for (int blk = 0; blk < blocks - 1; ++blk) {
      uint32_t xr[BT], dr[BT];
#pragma unroll
      for (int i = 0; i < BT; ++i) {
        const long o = at + (long)(blk * BT + i) * D;
        xr[i] = Row<TI>::load(xs + o, lane_at);
        dr[i] = Row<TI>::load(dts + o, lane_at);
      }
#pragma unroll
      for (int i = 0; i < BT; ++i) {
        const float st = step_of(Row<TI>::widen(dr[i]) + bias, p.softplus);
        const Vals<4> sv = quad(st), uv = quad(st * Row<TI>::widen(xr[i]));
        const Vals<4> b = load_vals<float, 4>(&key[blk * BT + i][0][slice * 4]);
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            h[c][j] = __builtin_fmaf(__builtin_amdgcn_exp2f(sv[c] * A[c][j]), h[c][j], uv[c] * b[j]);
      }
      if (blk + 1 < blocks - 1)
#pragma unroll
        for (int e = 0; e < 16; ++e) start[wave][blk][e][lane] = h[e >> 2][e & 3];
    }

#pragma unroll 1
    for (int blk = blocks - 1; blk >= 0; --blk) {
      const int t0 = blk * BT, cnt = min(BT, len - t0);
      if (blk < blocks - 1) {
        if (blk > 0) {
#pragma unroll
          for (int e = 0; e < 16; ++e) h[e >> 2][e & 3] = start[wave][blk - 1][e][lane];
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const Vals<4> e = load_vals<float, 4>(p.E + slot * D * N + state_at[c]);
#pragma unroll
            for (int j = 0; j < 4; ++j) h[c][j] = e[j];
          }
        }
      }
      // forwards: the states before each token; outputs for the gate's gradient
      float before[BT][4][4], dyo[BT], sto[BT];
      uint32_t xr[BT], dr[BT], gr[BT], zr[BT];
#pragma unroll
      for (int i = 0; i < BT; ++i) {
        const long o = at + (long)min(t0 + i, len - 1) * D;
        xr[i] = Row<TI>::load(xs + o, lane_at);
        dr[i] = Row<TI>::load(dts + o, lane_at);
        gr[i] = Row<TI>::load(gs + o, lane_at);
        if (GATE) zr[i] = Row<TI>::load(zs + o, lane_at);
      }
#pragma unroll
      for (int i = 0; i < BT; ++i) {
        // token by token: what the compiler would load ahead, it has no registers for
        __builtin_amdgcn_sched_barrier(0);
        const int t = min(t0 + i, len - 1);
        const bool there = i < cnt && real;
        xr[i] = there ? xr[i] : 0;
        const float x = Row<TI>::widen(xr[i]), z = GATE ? Row<TI>::widen(zr[i]) : 0.f, q = sigmoid(z);
        const float step = step_of(Row<TI>::widen(dr[i]) + bias, p.softplus), st = i < cnt ? step : 0.f;
        float dy = there ? Row<TI>::widen(gr[i]) : 0.f;
        sto[i] = st;
        const Vals<4> sv = quad(st), uv = quad(st * x);
        const Vals<4> b = load_vals<float, 4>(&key[t][0][slice * 4]);
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            before[i][c][j] = h[c][j];
            h[c][j] = __builtin_fmaf(__builtin_amdgcn_exp2f(sv[c] * A[c][j]), h[c][j], uv[c] * b[j]);
          }
        if constexpr (GATE) {
          const Vals<4> c4 = load_vals<float, 4>(&key[t][1][slice * 4]);
          Vals<4> y;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            y[c] = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) y[c] = __builtin_fmaf(c4[j], h[c][j], y[c]);
          }
          const float yo = __builtin_fmaf(skip, x, sum_own<LC>(y, odd, high));
          Row<TI>::store_inside(static_cast<TI*>(p.dz) + at + (long)t * D,
                                i < cnt && p.dz ? D * (int)sizeof(TI) : 0, mine_at,
                                dy * yo * (q * __builtin_fmaf(z, 1.f - q, 1.f)));
        }
        dyo[i] = GATE ? dy * z * q : dy;
      }
      // Backwards.  The empty assembly hides that a token's keys, steps and decays
      // are those of above: kept since then, they would take 36 registers a token.
      // No branch within: it would draw sums behind it, and their terms with them.
#pragma unroll
      for (int i = BT - 1; i >= 0; --i) {
        __builtin_amdgcn_sched_barrier(0);
        // (tokens behind the last: a step and gradients of zero, nothing stored)
        int t = min(t0 + i, len - 1);
        asm("" : "+s"(t));
        const int bytes = i < cnt ? D * (int)sizeof(TI) : 0;
        const float xo = Row<TI>::widen(xr[i]);
        float st = sto[i];
        asm("" : "+v"(st));
        const Vals<4> sv = quad(st), uv = quad(st * xo), gv = quad(dyo[i]);
        const Vals<4> b = load_vals<float, 4>(&key[t][0][slice * 4]), cc = load_vals<float, 4>(&key[t][1][slice * 4]);
        Vals<4> lb, mA, db, dc;
#pragma unroll
        for (int c = 0; c < 4; ++c) lb[c] = mA[c] = db[c] = dc[c] = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float now = i == BT - 1 ? h[c][j] : before[i + 1 < BT ? i + 1 : i][c][j];
            const float lv = __builtin_fmaf(cc[j], gv[c], l[c][j]);
            db[j] = __builtin_fmaf(lv, uv[c], db[j]);
            lb[c] = __builtin_fmaf(lv, b[j], lb[c]);
            dc[j] = __builtin_fmaf(now, gv[c], dc[j]);
            l[c][j] = lv * __builtin_amdgcn_exp2f(sv[c] * A[c][j]);
            const float m = l[c][j] * before[i][c][j];
            mA[c] = __builtin_fmaf(m, A[c][j], mA[c]);
            dA[c][j] = __builtin_fmaf(m, sv[c], dA[c][j]);
            asm volatile("" : "+v"(dA[c][j]));  // or these sums would be formed behind the loop, of kept terms
          }
        }
        const float lbo = sum_own<LC>(lb, odd, high), mAo = sum_own<LC>(mA, odd, high);
        const long o = at + (long)t * D;
        // A is held times log2(e)
        float ds = __builtin_fmaf(xo, lbo, mAo * 0.693147181f);
        const float slope = sigmoid(Row<TI>::widen(dr[i]) + bias);
        ds *= p.softplus ? slope : 1.f;
        const float dx = __builtin_fmaf(st, lbo, skip * dyo[i]);
        Row<TI>::store_inside(static_cast<TI*>(p.dx) + o, bytes, mine_at, dx);
        Row<TI>::store_inside(static_cast<TI*>(p.ddt) + o, bytes, mine_at, ds);
        dD = __builtin_fmaf(dyo[i], xo, dD);
        dbias += i < cnt ? ds : 0.f;
        // the sums over the channels' lanes, LC apart
        swap_halves(db[0], db[2]);
        swap_halves(db[1], db[3]);
        swap_halves(dc[0], dc[2]);
        swap_halves(dc[1], dc[3]);
        float d0 = db[0] + db[2], d1 = db[1] + db[3], e0 = dc[0] + dc[2], e1 = dc[1] + dc[3];
        swap_rows(d0, d1);
        swap_rows(e0, e1);
        float sd = d0 + d1, se = e0 + e1;
        // lanes 0..15 hold state 0 of the slice, 16..31 state 1, 32..47 state 2, 48..63 state 3
        if constexpr (LC <= 8) {
          sd += dpp<0x128>(sd);
          se += dpp<0x128>(se);
        }
        if constexpr (LC == 4) {
          sd += dpp<0x124>(sd);
          se += dpp<0x124>(se);
        }
        // (lanes of the same state hold the same bits)
        part[turn][wave][i][0][slice * 4 + (lane >> 4)] = sd;
        part[turn][wave][i][1][slice * 4 + (lane >> 4)] = se;
      }
      __syncthreads();
      for (int e = tid; e < cnt * 2 * N; e += NT) {
        const float* q = &part[turn][0][0][0][0] + e;
        constexpr int W = BT * 2 * N;
        const float v = WAVES == 2 ? q[0] + q[W] : (q[0] + q[W]) + (q[2 * W] + q[3 * W]);
        const int i = e / (2 * N), which = e / N % 2, n = e % N;
        const long o = ((row0 + t0 + i) * p.G + g) * N + n;
        if (teams == 1) static_cast<TI*>(which ? p.dc : p.db)[o] = (TI)v;
        else p.keys[(((long)team * p.rows + row0 + t0 + i) * p.G + g) * 2 * N + which * N + n] = v;
      }
      turn ^= 1;
    }
  }

  float* sums = p.sums + (long)run * D * (N + 2);
#pragma unroll
  for (int c = 0; c < 4; ++c)
    if (c0 + c < p.Dg)
      store_vals<float, 4>(sums + state_at[c], Vals<4>{{dA[c][0], dA[c][1], dA[c][2], dA[c][3]}});
  if (mine) {
    sums[(long)D * N + own] = dD;
    sums[(long)D * (N + 1) + own] = dbias;
  }
}

// What the workgroups' sums leave to do, in one launch: the parameters' gradients,
// 64 of them a workgroup, 16 threads each; and behind those workgroups, where a
// group's channels are several workgroups', db and dc.  Rows of no sequence are
// left as they were.
template <typename TI>
__global__ __launch_bounds__(1024) void ssm_sums_kernel(const SsmParams p, int teams) {
  __shared__ float sums[16][64];
  const long DN = (long)p.D * p.N, cols = DN + 2L * p.D;
  const int own = (int)((cols + 63) / 64);
  if ((int)blockIdx.x >= own) {
    const long GN = (long)p.G * p.N, total = p.rows * GN * 2;
    for (long e = (long)(blockIdx.x - own) * 1024 + threadIdx.x; e < total; e += (long)(gridDim.x - own) * 1024) {
      const int n = (int)(e % p.N), which = (int)(e / p.N % 2);
      const long rg = e / (2 * p.N), row = rg / p.G;
      if (p.cu && (row < p.cu[0] || row >= p.cu[p.B])) continue;
      float a = 0.f;
      for (int q = 0; q < teams; ++q) a += p.keys[(long)q * total + e];
      static_cast<TI*>(which ? p.dc : p.db)[rg * p.N + n] = (TI)a;
    }
    return;
  }
  const int lane = threadIdx.x & 63, k = threadIdx.x >> 6;
  const long c = (long)blockIdx.x * 64 + lane;
  float a = 0.f;
  if (c < cols)
#pragma unroll 4
    for (int i = k; i < p.runs; i += 16) a += p.sums[i * cols + c];
  sums[k][lane] = a;
  __syncthreads();
  if (k == 0 && c < cols) {
    for (int i = 1; i < 16; ++i) a += sums[i][lane];
    if (c < DN) p.dA_log[c] = -rate_factor(p.A_log[c]) * a;
    else if (c < DN + p.D) {
      if (p.dD) p.dD[c - DN] = a;
    } else if (p.ddt_bias) {
      p.ddt_bias[c - DN - p.D] = a;
    }
  }
}

// ------------------------------------------------------------------- host --

// a grid holds fewer than 2^32 threads; the launches that may need more loop
constexpr long long MOST_WGS = (1LL << 24) - 1;

inline long long up16(long long x) { return (x + 15) & ~15LL; }

int tiles_of(int Dg, int channels) { return (Dg + channels - 1) / channels; }

int sizes_checked(int B, int T, int D, int G, int N, bool packed, int dtype) {
  if (B < 0 || T < 0 || D < 1 || G < 1 || N < 1 || D % G || (dtype != GDN_F32 && dtype != GDN_BF16))
    return GDN_ERR_INVALID_ARG;
  if ((packed ? 1LL : (long long)B) * T > MOST_ROWS || D >= 1 << 20 || B >= 1 << 24 || (long long)B * D >= 1 << 28)
    return GDN_ERR_INVALID_ARG;
  if (N != 16 && N != 32 && N != 64) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

// How a forward call runs.
struct Cut {
  bool recurrent;  // token by token, lanes across the states
  int L, nseg;
  long long segments;
  int inner;      // see SsmParams
  bool cut() const { return segments > 0; }
};

// The waves that the device's 1,024 vector units hold at once, by the states that a
// lane keeps in registers: no more, or some units get another and the rest wait for
// it (8 x 4,096 x 1,280, N 16: 255 us, 265 with 4,096 and 268 with 8,192; 4 x 4,096,
// N 32: 283, 285 with 5,120; 2 x 4,096, N 64: 299, 331 with 4,096).  One sequence can
// lose by it, by its shorter segments: 1 x 8,192 x 2,048, N 16: 124, 120 with 4,096.
long long most_waves(int N) { return N == 16 ? 5120 : N == 32 ? 4096 : 2048; }

Cut cut_of(int B, int T, int D, int G, int N, bool packed) {
  Cut c = {false, std::max(T, 1), 1, 0, 0};
  if (B == 0) return c;
  const long long tiles = (long long)G * tiles_of(D / G, 64), chains = B * tiles;
  // Enough waves without a cut: one launch, a lane a channel, and a second reading
  // saved (60 x 1,280 channels, N 16: 256 tokens 124 us, 158 cut in three; at 48
  // sequences 94 and 122, but N 32 224 and 228, and 1,043 and 774 for 1,024 tokens).
  const bool uncut = !packed && chains > 1024;
  // Token by token, N / 4 lanes a channel in one launch: as long as that takes less
  // than the cut's three (N 16: 20 us against 17 for 128 tokens of few channels,
  // 38 and 41 for 256 of 8 x 1,280; N 64: 29 and 32 for 192 of few, 169 and 204 for
  // 512 of 8 x 1,280); where sequences are not cut, for single tokens (160 x 1,280,
  // N 32: 13 us against 18, for two tokens 20 and 19; of 400 sequences 31 and 34, 45
  // and 33; N 64 of 60 sequences 11 and 19, 15 and 19).
  if (T <= (uncut ? 1 : 64 + 2 * N + std::min(chains, 160LL) * N / 16)) {
    c.recurrent = true;
    return c;
  }
  if (uncut) return c;
  const long long rows = packed ? T : (long long)B * T;
  // Rows a segment for so many waves; of packed sequences the last segments are short.
  auto length = [&](long long waves) {
    const long long segments = std::max(1LL, packed ? waves / tiles - B / 2 : waves / chains * B);
    const long long each = segments / std::max(B, 1);  // of a dense sequence: one at least
    const long long L = packed ? (rows + segments - 1) / segments : (T + each - 1) / each;
    return (L + FLIGHT - 1) / FLIGHT * FLIGHT;
  };
  // No more than 2,048 waves where segments go below 20 rows, and no fewer rows than
  // 8 (2 x 2,013 x 96, N 64: 57 us with 8, 71 with 20; 1,000 x 128, N 16: 20 and 28;
  // 8,192 x 256: 42 with the 16 of 2,048 waves, 53 with 8, 43 with 20).
  c.L = (int)std::max(length(most_waves(N)), std::min(20LL, std::max(8LL, length(2048))));
  // Of packed sequences no segment is longer than half as much again as a wave's even
  // share of the rows (or than 64 rows), however many sequences there are: one may be
  // nearly all of them (511 of 32 tokens and one of 48,000, 1,280 channels, N 16: 0.6 ms,
  // 16.7 uncut; N 64: 3.0 and 81).  What even ones pay is two launches that find
  // nothing (512 of 125 tokens: 277 us, 272 uncut; N 64: 1,177 and 1,171).
  if (packed) {
    const long long share = (3 * rows * tiles / (2 * most_waves(N)) + FLIGHT - 1) / FLIGHT * FLIGHT;
    c.L = (int)std::min<long long>(c.L, std::max(64LL, share));
    while (c.L < T && (slots_of(true, B, T, c.L) + 1) * tiles > 4 * MOST_WGS) c.L *= 2;
  }
  if (c.L >= T) {
    c.L = T;
    return c;
  }
  c.nseg = segments_of(T, c.L);
  c.segments = slots_of(packed, B, T, c.L);
  if (packed && c.nseg < B) c.inner = c.nseg;
  return c;
}

// The pieces of a workspace.
struct Space {
  long long E, R, S, keys, sums, bytes;
};

Space space_of(long long segments, long long runs, long long rows, int D, int G, int N, int teams, bool back) {
  Space w = {};
  const long long state = up16(segments * D * N * 4);
  w.E = 0;
  w.R = w.E + state;
  w.S = w.R + (back ? state : 0);
  w.keys = w.S + up16(segments * D * 4);
  w.sums = w.keys + (back && teams > 1 ? up16(rows * G * 2 * N * 4 * teams) : 0);
  w.bytes = w.sums + (back ? up16(runs * D * (N + 2) * 4) : 0);
  return w;
}

struct BackPlan {
  long long segments, runs, rows;
  int L, nseg, run, waves, teams;
};

BackPlan back_plan(int B, int T, int D, int G, int N, bool packed) {
  BackPlan b;
  b.rows = (packed ? 1LL : B) * (long long)T;
  const int tiles = tiles_of(D / G, 1024 / N);
  // Four waves a workgroup, or two where the last one of a group's would
  // otherwise have two to work for nothing.
  b.waves = (tiles + 3) / 4 * 4 - tiles >= 2 ? 2 : 4;
  b.teams = tiles_of(tiles, b.waves);
  // Segments of as many blocks as there may be, or of so few that all waves still
  // run at once: where the device is not full, a segment's time is the call's (149
  // tokens of 561 channels: 12.5 us with two blocks, 31.5 with six; 4 x 487 of 780
  // 14 and 32).
  const long long wide = (long long)b.teams * G, places = 2048 / b.waves;
  for (int blocks = 2;; ++blocks) {
    b.L = blocks * Blocks<16>::BT;
    b.segments = B > 0 ? slots_of(packed, B, T, b.L) : 0;
    if (blocks == most_blocks(N) || b.segments * wide <= places) break;
  }
  b.nseg = segments_of(T, b.L);
  // A workgroup takes a run of segments (few partial sums of the parameters'
  // gradients), as long as the device's places (eight waves a compute unit)
  // are in the end filled as well as by shorter ones.
  const int first = (int)std::max(1LL, b.segments * wide / (8 * places));
  long long best = 0;
  for (int run = first; run < first + 64; ++run) {
    // (a workgroup's beginning and end take about half a segment's time)
    const long long rounds = ((b.segments + run - 1) / run * wide + places - 1) / places * (2 * run + 1);
    if (run > first && rounds > best) continue;
    best = rounds;
    b.run = run;
  }
  b.runs = (b.segments + b.run - 1) / b.run;
  return b;
}

template <typename TI>
void launch_outputs(const SsmParams& p, unsigned grid, bool output, hipStream_t s) {
  const dim3 g(grid), b(64);
  switch (p.N) {
    case 16:
      if (output) hipLaunchKernelGGL((ssm_kernel<TI, 16, true>), g, b, 0, s, p);
      else hipLaunchKernelGGL((ssm_kernel<TI, 16, false>), g, b, 0, s, p);
      break;
    case 32:
      if (output) hipLaunchKernelGGL((ssm_kernel<TI, 32, true>), g, b, 0, s, p);
      else hipLaunchKernelGGL((ssm_kernel<TI, 32, false>), g, b, 0, s, p);
      break;
    default:
      if (output) hipLaunchKernelGGL((ssm_kernel<TI, 64, true>), g, b, 0, s, p);
      else hipLaunchKernelGGL((ssm_kernel<TI, 64, false>), g, b, 0, s, p);
  }
}

// Few states of many segments take eight threads each (20,480 states of 200
// segments: 16 us instead of 25) or 32 (1,056 of 730: 8 instead of 19; but 6,400
// of 485 25 instead of 15, in pieces of 32 bytes); many states keep the device busy
// with one (245,760 of some 13 segments: 14 us, 51 with eight).  Of more sequences
// than places for inner segments only the cut ones are looked for, some 4,096
// workgroups in all: most end at once (3,000 sequences of 40 tokens and 256 channels:
// calls of 114 us, 108 without a cut, 120 with twice as many and 113 with half; with
// 20,000 tokens behind 3,000 sequences of 5: 201, 171 and 298).
void launch_join(const SsmParams& p, int directions, hipStream_t s) {
  const long long DN = (long long)p.D * p.N, states = p.B * DN, each = p.segments / p.B;
  const int groups = states < 65536 && each > 64 ? states < 4096 && each > 256 ? 32 : 8 : 1;
  const long long wgs = p.inner ? p.inner * std::max(1LL, std::min((DN + 255) / 256, 4096LL / p.inner))
                                : std::min(MOST_WGS, (states * groups + 255) / 256);
  const dim3 grid((unsigned)wgs, directions);
  if (groups == 32) hipLaunchKernelGGL((ssm_join_kernel<32>), grid, dim3(256), 0, s, p);
  else if (groups == 8) hipLaunchKernelGGL((ssm_join_kernel<8>), grid, dim3(256), 0, s, p);
  else hipLaunchKernelGGL((ssm_join_kernel<1>), grid, dim3(256), 0, s, p);
}

// Two turns of four tokens in flight, one where sequences have no more in the mean, and
// turns of a single token where they have that: fewer registers, more waves (one
// token of 128 sequences, 1,280 channels: 7.9 us against 9.5).  Of packed sequences the
// mean is all that is known: 256 of a token each 11.2 us, 16.0 with turns of four and
// 19.9 with two of them in flight; one of 100 tokens, 156 of one and 99 empty ones 48,
// 23.9 and 21.0, since the long one then waits for every token's loads.
// Single tokens' states go past the eight second-level caches, read and written, where
// they are more than those hold, 32 MB (1,280 channels, N 16: 512 sequences 23.3 us,
// 25.8 through the caches; 256 sequences 12.8 and 12.2).
template <typename TI, int N>
void launch_recurrent_n(const SsmParams& p, unsigned grid, hipStream_t s) {
  const dim3 g(grid), b(256);
  const bool stream = (long long)p.B * p.D * p.N * 4 >= 32LL << 20;
  if (p.rows <= p.B) {
    if (stream) hipLaunchKernelGGL((ssm_recurrent_kernel<TI, N, 1, 1, true>), g, b, 0, s, p);
    else hipLaunchKernelGGL((ssm_recurrent_kernel<TI, N, 1, 1, false>), g, b, 0, s, p);
  } else if (p.rows <= 4LL * p.B) {
    hipLaunchKernelGGL((ssm_recurrent_kernel<TI, N, 1, 4, false>), g, b, 0, s, p);
  } else {
    hipLaunchKernelGGL((ssm_recurrent_kernel<TI, N, 2, 4, false>), g, b, 0, s, p);
  }
}

template <typename TI>
void launch_recurrent(const SsmParams& p, unsigned grid, hipStream_t s) {
  if (p.N == 16) launch_recurrent_n<TI, 16>(p, grid, s);
  else if (p.N == 32) launch_recurrent_n<TI, 32>(p, grid, s);
  else launch_recurrent_n<TI, 64>(p, grid, s);
}

template <typename TI, bool GATE, int WAVES>
void launch_bwd_n(const SsmParams& p, unsigned grid, hipStream_t s) {
  const dim3 g(grid), b(64 * WAVES);
  if (p.N == 16) hipLaunchKernelGGL((ssm_bwd_kernel<TI, 16, GATE, WAVES>), g, b, 0, s, p);
  else if (p.N == 32) hipLaunchKernelGGL((ssm_bwd_kernel<TI, 32, GATE, WAVES>), g, b, 0, s, p);
  else hipLaunchKernelGGL((ssm_bwd_kernel<TI, 64, GATE, WAVES>), g, b, 0, s, p);
}

template <typename TI>
void launch_bwd(const SsmParams& p, int waves, unsigned grid, hipStream_t s) {
  if (waves == 2) p.z ? launch_bwd_n<TI, true, 2>(p, grid, s) : launch_bwd_n<TI, false, 2>(p, grid, s);
  else p.z ? launch_bwd_n<TI, true, 4>(p, grid, s) : launch_bwd_n<TI, false, 4>(p, grid, s);
}

int forward(SsmParams p, int dtype, int flags, void* workspace, long long workspace_bytes, void* stream) {
  const bool pooled = p.slots != nullptr, packed = p.cu != nullptr;
  const int rc = sizes_checked(p.B, p.T, p.D, p.G, p.N, packed, dtype);
  if (rc == GDN_ERR_INVALID_ARG || (flags & ~GDN_SSM_SOFTPLUS)) return GDN_ERR_INVALID_ARG;
  if (p.B > 0 && (!p.A_log || !p.hT || (p.T > 0 && (!p.x || !p.dt || !p.b || !p.c || !p.out))))
    return GDN_ERR_INVALID_ARG;
  if (rc != GDN_OK) return rc;
  if (misaligned({p.x, p.dt, p.b, p.c, p.A_log, p.Dskip, p.z, p.dt_bias, p.h0, p.out, p.hT, workspace}, 16) ||
      misaligned({p.cu, p.slots}, 4))
    return GDN_ERR_INVALID_ARG;
  Cut cut = cut_of(p.B, p.T, p.D, p.G, p.N, packed);
  if (pooled) cut = Cut{true, std::max(p.T, 1), 1, 0, 0};
  const Space w = space_of(cut.segments, 0, 0, p.D, p.G, p.N, 1, false);
  const long long need = cut.cut() ? w.bytes : 0;
  if (need > 0 && (!workspace || workspace_bytes < need)) return GDN_ERR_INVALID_ARG;
  p.rows = (packed ? 1LL : p.B) * (long long)p.T;
  const long long e = dtype == GDN_BF16 ? 2 : 4, data = p.rows * p.D * e, keys = p.rows * p.G * p.N * e;
  const long long state = (pooled ? p.nslots : p.B) * (long long)p.D * p.N * 4;
  if (clash({{p.out, data}, {p.hT, state}, {need > 0 ? workspace : nullptr, need}},
            {{p.x, data}, {p.dt, data}, {p.z, data}, {p.b, keys}, {p.c, keys}, {p.A_log, 4LL * p.D * p.N},
             {p.Dskip, 4LL * p.D}, {p.dt_bias, 4LL * p.D}, {p.cu, 4LL * (p.B + 1)}, {p.slots, 4LL * p.B},
             {p.h0 == p.hT ? nullptr : p.h0, state}}))
    return GDN_ERR_INVALID_ARG;
  if (p.B == 0) return GDN_OK;
  p.Dg = p.D / p.G;
  p.softplus = flags & GDN_SSM_SOFTPLUS;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool bf = dtype == GDN_BF16;
  if (cut.recurrent) {
    const long long wgs = (long long)p.B * tiles_of(p.D, 1024 / p.N);
    if (wgs > MOST_WGS) return GDN_ERR_INVALID_ARG;
    bf ? launch_recurrent<__bf16>(p, (unsigned)wgs, s) : launch_recurrent<float>(p, (unsigned)wgs, s);
    return hipGetLastError() == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH;
  }
  p.L = cut.L;
  p.nseg = cut.nseg;
  p.segments = cut.cut() ? cut.segments : slots_of(packed, p.B, p.T, p.L);
  p.inner = cut.inner;
  const long long tiles = (long long)p.G * tiles_of(p.Dg, 64);
  const long long wgs = (p.inner ? (long long)p.B + p.inner : p.segments) * tiles;
  if (wgs > 4 * MOST_WGS) return GDN_ERR_INVALID_ARG;  // of 64 threads
  if (cut.cut()) {
    char* base = static_cast<char*>(workspace);
    p.E = reinterpret_cast<float*>(base + w.E);
    p.S = reinterpret_cast<float*>(base + w.S);
    const unsigned first = (unsigned)((p.inner ? p.inner : p.segments) * tiles);
    bf ? launch_outputs<__bf16>(p, first, false, s) : launch_outputs<float>(p, first, false, s);
    launch_join(p, 1, s);
  }
  bf ? launch_outputs<__bf16>(p, (unsigned)wgs, true, s) : launch_outputs<float>(p, (unsigned)wgs, true, s);
  return hipGetLastError() == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}

}  // namespace

extern "C" long long gdn_ssm_workspace_size(int B, int T, int D, int G, int N, int packed, int dtype, int backward) {
  const int rc = sizes_checked(B, T, D, G, N, packed != 0, dtype);
  if (rc != GDN_OK) return rc;
  if (!backward) {
    const Cut c = cut_of(B, T, D, G, N, packed != 0);
    return c.cut() ? space_of(c.segments, 0, 0, D, G, N, 1, false).bytes : 0;
  }
  const BackPlan b = back_plan(B, T, D, G, N, packed != 0);
  return space_of(b.segments, b.runs, b.rows, D, G, N, b.teams, true).bytes;
}

extern "C" int gdn_ssm_fwd(const void* x, const void* dt, const void* b, const void* c, const float* A_log,
                           const float* Dskip, const void* z, const float* dt_bias, const float* h0,
                           const int32_t* cu_seqlens, void* out, float* hT, int B, int T, int D, int G, int N,
                           void* stream, int dtype, int flags, void* workspace, long long workspace_bytes) {
  SsmParams p = {};
  p.x = x; p.dt = dt; p.b = b; p.c = c; p.A_log = A_log; p.Dskip = Dskip; p.z = z; p.dt_bias = dt_bias;
  p.h0 = h0; p.cu = cu_seqlens; p.out = out; p.hT = hT;
  p.B = B; p.T = T; p.D = D; p.G = G; p.N = N;
  return forward(p, dtype, flags, workspace, workspace_bytes, stream);
}

extern "C" int gdn_ssm_fwd_recurrent_pool(const void* x, const void* dt, const void* b, const void* c,
                                          const float* A_log, const float* Dskip, const void* z, const float* dt_bias,
                                          float* pool, const int32_t* slots, const int32_t* cu_seqlens, void* out,
                                          int nslots, int B, int T, int D, int G, int N, void* stream, int dtype,
                                          int flags) {
  if (nslots < 0 || (B > 0 && !slots)) return GDN_ERR_INVALID_ARG;
  SsmParams p = {};
  p.x = x; p.dt = dt; p.b = b; p.c = c; p.A_log = A_log; p.Dskip = Dskip; p.z = z; p.dt_bias = dt_bias;
  p.h0 = pool; p.hT = pool; p.slots = slots; p.cu = cu_seqlens; p.out = out; p.nslots = nslots;
  p.B = B; p.T = T; p.D = D; p.G = G; p.N = N;
  return forward(p, dtype, flags, nullptr, 0, stream);
}

extern "C" int gdn_ssm_bwd(const void* x, const void* dt, const void* b, const void* c, const float* A_log,
                           const float* Dskip, const void* z, const float* dt_bias, const float* h0,
                           const int32_t* cu_seqlens, const void* dout, const float* dhT, void* dx, void* ddt, void* db,
                           void* dc, float* dA_log, float* dD, void* dz, float* ddt_bias, float* dh0, int B, int T,
                           int D, int G, int N, void* stream, int dtype, int flags, void* workspace,
                           long long workspace_bytes) {
  const bool packed = cu_seqlens != nullptr;
  const int rc = sizes_checked(B, T, D, G, N, packed, dtype);
  if (rc == GDN_ERR_INVALID_ARG || (flags & ~GDN_SSM_SOFTPLUS) || !A_log || !dA_log) return GDN_ERR_INVALID_ARG;
  if (B > 0 && T > 0 && (!x || !dt || !b || !c || !dout || !dx || !ddt || !db || !dc)) return GDN_ERR_INVALID_ARG;
  if (dz && !z) return GDN_ERR_INVALID_ARG;
  if (rc != GDN_OK) return rc;
  if (misaligned({x, dt, b, c, A_log, Dskip, z, dt_bias, h0, dout, dhT, dx, ddt, db, dc, dA_log, dD, dz, ddt_bias, dh0,
                  workspace}, 16) || misaligned(cu_seqlens, 4))
    return GDN_ERR_INVALID_ARG;
  const BackPlan plan = back_plan(B, T, D, G, N, packed);
  const Space w = space_of(plan.segments, plan.runs, plan.rows, D, G, N, plan.teams, true);
  if (w.bytes > 0 && (!workspace || workspace_bytes < w.bytes)) return GDN_ERR_INVALID_ARG;
  const long long e = dtype == GDN_BF16 ? 2 : 4, data = plan.rows * D * e, keys = plan.rows * G * N * e;
  const long long state = (long long)B * D * N * 4, rates = 4LL * D * N, vec = 4LL * D;
  if (clash({{dx, data}, {ddt, data}, {db, keys}, {dc, keys}, {dA_log, rates}, {dD, vec}, {dz, data}, {ddt_bias, vec},
             {dh0, state}, {workspace, w.bytes}},
            {{x, data}, {dt, data}, {b, keys}, {c, keys}, {A_log, rates}, {Dskip, vec}, {z, data}, {dt_bias, vec},
             {h0, state}, {cu_seqlens, 4LL * (B + 1)}, {dout, data}, {dh0 == dhT ? nullptr : dhT, state}}))
    return GDN_ERR_INVALID_ARG;
  SsmParams p = {};
  p.x = x; p.dt = dt; p.b = b; p.c = c; p.A_log = A_log; p.Dskip = Dskip; p.z = z; p.dt_bias = dt_bias;
  p.h0 = h0; p.cu = cu_seqlens; p.dout = dout; p.dhT = dhT; p.dx = dx; p.ddt = ddt; p.db = db; p.dc = dc;
  p.dA_log = dA_log; p.dD = dD; p.dz = dz; p.ddt_bias = ddt_bias; p.dh0 = dh0;
  char* base = static_cast<char*>(workspace);
  p.E = reinterpret_cast<float*>(base + w.E);
  p.R = reinterpret_cast<float*>(base + w.R);
  p.S = reinterpret_cast<float*>(base + w.S);
  p.keys = reinterpret_cast<float*>(base + w.keys);
  p.sums = reinterpret_cast<float*>(base + w.sums);
  p.B = B; p.T = T; p.D = D; p.G = G; p.N = N; p.Dg = D / G;
  p.L = plan.L;
  p.nseg = plan.nseg;
  p.segments = plan.segments;
  p.run = plan.run;
  p.runs = (int)plan.runs;
  p.rows = plan.rows;
  p.softplus = flags & GDN_SSM_SOFTPLUS;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool bf = dtype == GDN_BF16;
  const long long maps = std::min(MOST_WGS, (plan.segments * G * tiles_of(p.Dg, 64) * (N / 16) + 3) / 4);
  const long long wgs = plan.runs * G * plan.teams;
  const long long cols = (long long)D * (N + 2);
  if (wgs > MOST_WGS) return GDN_ERR_INVALID_ARG;
  if (plan.segments > 0) {
    if (bf) hipLaunchKernelGGL((ssm_bwd_maps_kernel<__bf16>), dim3((unsigned)maps), dim3(256), 0, s, p);
    else hipLaunchKernelGGL((ssm_bwd_maps_kernel<float>), dim3((unsigned)maps), dim3(256), 0, s, p);
    launch_join(p, 2, s);
    bf ? launch_bwd<__bf16>(p, plan.waves, (unsigned)wgs, s) : launch_bwd<float>(p, plan.waves, (unsigned)wgs, s);
  }
  // (a workgroup for 64 of the parameters' gradients, at most 4,096 more for db and dc)
  const long long keyed = plan.segments > 0 && plan.teams > 1 ? plan.rows * G * 2 * N : 0;
  const dim3 grid((unsigned)((cols + 63) / 64 + std::min(4096LL, (keyed + 1023) / 1024)));
  if (bf) hipLaunchKernelGGL((ssm_sums_kernel<__bf16>), grid, dim3(1024), 0, s, p, plan.teams);
  else hipLaunchKernelGGL((ssm_sums_kernel<float>), grid, dim3(1024), 0, s, p, plan.teams);
  return hipGetLastError() == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}

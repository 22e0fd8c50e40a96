// Device-side building blocks of the operators around the recurrences: rows
// read and written in vectors and computed in fp32, sums over neighbouring
// lanes, and the segments of packed sequences.  Internal header: every
// definition sits in an unnamed namespace of the including file.
#ifndef GDN_ROWS_H
#define GDN_ROWS_H

#include <hip/hip_runtime.h>
#include <limits.h>
#include <stdint.h>

namespace {

// ------------------------------------------------------------------ vectors --

template <typename TI, int V>
struct Raw {
  typedef TI type __attribute__((ext_vector_type(V)));
};
template <typename TI>
struct Raw<TI, 1> {
  typedef TI type;
};

template <int V>
struct Vals {
  float v[V];
  __device__ float& operator[](int i) { return v[i]; }
  __device__ float operator[](int i) const { return v[i]; }
};

template <typename TI, int V>
__device__ static inline typename Raw<TI, V>::type load_raw(const TI* p) {
  return *reinterpret_cast<const typename Raw<TI, V>::type*>(p);
}

template <typename TI, int V>
__device__ static inline Vals<V> widen(const typename Raw<TI, V>::type& r) {
  Vals<V> x;
  if constexpr (V == 1) x[0] = (float)r;
  else
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = (float)r[i];
  return x;
}

template <typename TI, int V>
__device__ static inline Vals<V> load_vals(const TI* p) {
  return widen<TI, V>(load_raw<TI, V>(p));
}

// Rounded to nearest even where TI is bf16.
template <typename TI, int V>
__device__ static inline void store_vals(TI* p, const Vals<V>& x) {
  if constexpr (V == 1) {
    *p = (TI)x[0];
  } else {
    typename Raw<TI, V>::type r;
    if constexpr (sizeof(TI) == 2) {
      // pair by pair: a packed conversion each
      typedef float f2 __attribute__((ext_vector_type(2)));
      typedef __bf16 b2 __attribute__((ext_vector_type(2)));
      typedef uint32_t u __attribute__((ext_vector_type(V / 2)));
      u w;
#pragma unroll
      for (int i = 0; i < V / 2; ++i)
        w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{x[2 * i], x[2 * i + 1]}, b2));
      r = __builtin_bit_cast(typename Raw<TI, V>::type, w);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) r[i] = x[i];
    }
    *reinterpret_cast<typename Raw<TI, V>::type*>(p) = r;
  }
}

template <int BYTES>
struct Bits {
  typedef uint32_t type;
};
template <>
struct Bits<2> {
  typedef uint16_t type;
};

// A lane's value in a row of one of the token tensors.  The row's address, the
// same in all lanes, is kept in scalar registers (the assembly is empty; without
// it the sum is formed in vector registers, three instructions a load), and the
// value in 32 bits (two of 16 would be packed, and waited for, on the way).
template <typename TI>
struct Row {
  typedef typename Bits<sizeof(TI)>::type bits;
  typedef __attribute__((address_space(1))) bits* place;
  __device__ static place at(const TI* row, uint32_t& lane) {
    uintptr_t a = reinterpret_cast<uintptr_t>(row);
    asm("" : "+s"(a), "+v"(lane));
    return (place)((__attribute__((address_space(1))) char*)a + lane);
  }
  __device__ static uint32_t load(const TI* row, uint32_t& lane) { return *at(row, lane); }
  __device__ static void store(TI* row, uint32_t& lane, float x) { *at(row, lane) = __builtin_bit_cast(bits, (TI)x); }
  // Of the lanes whose place is inside the row of `bytes` bytes, without a branch.
  __device__ static void store_inside(TI* row, int bytes, uint32_t lane, float x) {
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(row, 0, bytes, 0x00020000);
    const bits b = __builtin_bit_cast(bits, (TI)x);
    if constexpr (sizeof(TI) == 2) __builtin_amdgcn_raw_buffer_store_b16(b, r, lane, 0, 0);
    else __builtin_amdgcn_raw_buffer_store_b32(b, r, lane, 0, 0);
  }
  __device__ static float widen(uint32_t x) { return __builtin_bit_cast(float, sizeof(TI) == 2 ? x << 16 : x); }
};

// --------------------------------------------------------------- functions --

// 1 / (1 + exp(-x)); exp2 and the reciprocal are within 1 ulp.  The product with
// log2(e), its rounding (1.44 |x| 2^-24) and the constant's (0.33 |x| 2^-24), moves
// exp2's argument by up to 1.77 |x| 2^-24, the exponential by 1.23 |x| 2^-24 of itself
// and the result by 1 / (1 + exp(x)) of that.
__device__ static inline float sigmoid(float x) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(x * -1.44269504f));
}

// ------------------------------------------------------------- cross-lane --

template <int CTRL>
__device__ static inline float dpp(float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xF, 0xF, true));
}

// Sum over groups of L neighbouring lanes, in every lane of the group; the
// same value, bit for bit, in each (sums of two are symmetric).
template <int L>
__device__ static inline float sum_lanes(float x) {
  if constexpr (L >= 2) x += dpp<0xB1>(x);   // quad_perm 1 0 3 2
  if constexpr (L >= 4) x += dpp<0x4E>(x);   // quad_perm 2 3 0 1
  if constexpr (L >= 8) x += dpp<0x141>(x);  // mirror of 8 lanes: the other quad
  if constexpr (L >= 16) x += dpp<0x140>(x); // mirror of 16 lanes: the other eight
  if constexpr (L >= 32) x += __shfl_xor(x, 16);
  if constexpr (L >= 64) x += __shfl_xor(x, 32);
  return x;
}

// ---------------------------------------------------------------- segments --
//
// A launch works on segments of up to L rows, one a slot.  Dense sequences
// have nseg slots each.  Of packed ones, sequence n has the slots from
// begin(n) / L + n on: ceil(length / L) of them fit before the next one's, an
// empty sequence has one, and the slots of all are fewer than T / L + B + 1.

struct Segment {
  long row0;   // the segment's first row
  int n;       // sequence, -1: none
  int t0;      // the first row's place in its sequence
  int len;     // rows (0 for the one segment of an empty sequence)
  int total;   // rows of the sequence
  __device__ bool first() const { return t0 == 0; }
  __device__ bool last() const { return t0 + len == total; }
};

// Rows of a call: places within a sequence and a few rows behind it are ints.
constexpr long long MOST_ROWS = 1LL << 30;

inline int segments_of(long long T, long long L) { return (int)(T > L ? (T + L - 1) / L : 1); }

inline long long slots_of(bool packed, long long B, long long T, long long L) {
  return packed ? T / L + B : B * segments_of(T, L);
}

__device__ static inline int taken(int x, int lo, int hi) { return min(max(x, lo), hi); }

// How many of the first numbers below B a condition holds for, which holds for none
// behind the first that it fails for: a search that looks at 64 of them at once.
// All 64 lanes take part, with one condition.
template <typename F>
__device__ static inline int leading(int B, F holds) {
  const int lane = threadIdx.x & 63;
  int lo = 0, hi = B;
  while (lo < hi) {
    const int step = (hi - lo + 63) >> 6;
    const long at = lo + (long)lane * step;
    const bool before = at < hi && holds((int)(at < hi ? at : lo));
    const int c = __popcll(__ballot(before));
    if (step == 1) return lo + c;
    if (c == 0) return lo;
    hi = (int)min((long)hi, lo + (long)c * step);
    lo += (c - 1) * step + 1;
  }
  return lo;
}

__device__ static inline Segment segment_of(const int32_t* cu, int B, int T, int L, int nseg, long slot) {
  Segment s;
  int i;
  if (cu) {
    s.n = leading(B, [&](int n) { return taken(cu[n], 0, T) / L + (long)n <= slot; }) - 1;
    if (s.n < 0) return Segment{0, -1, 0, 0, 0};
    const int b = taken(cu[s.n], 0, T), e = taken(cu[s.n + 1], b, T);
    s.total = e - b;
    s.row0 = b;
    i = (int)(slot - b / L - s.n);
  } else {
    s.n = (int)(slot / nseg);
    s.total = T;
    s.row0 = (long)s.n * T;
    i = (int)(slot % nseg);
  }
  const long t0 = (long)i * L;
  if (i < 0 || (i > 0 && t0 >= s.total)) return Segment{0, -1, 0, 0, 0};
  s.t0 = (int)t0;
  s.row0 += t0;
  s.len = min(L, s.total - s.t0);
  return s;
}

// The last sequence that begins at or before a row, -1: none.
__device__ static inline int sequence_at(const int32_t* cu, int B, int T, int row) {
  return leading(B, [&](int n) { return taken(cu[n], 0, T) <= row; }) - 1;
}

// Of a packed batch the k-th segment that is not its sequence's last: each holds
// one row whose number is a multiple of L, so that there are rows / L at most,
// however many sequences there are; n = -1 where row k L is in none.
__device__ static inline Segment inner_segment_of(const int32_t* cu, int B, int T, int L, int k, long& slot) {
  const int row = (int)min((long)k * L, (long)T);
  const int n = sequence_at(cu, B, T, row);
  if (n < 0) return Segment{0, -1, 0, 0, 0};
  const int b = taken(cu[n], 0, T), total = taken(cu[n + 1], b, T) - b;
  const int i = (row - b) / L, t0 = i * L;
  if (row < b || L >= total - t0) return Segment{0, -1, 0, 0, 0};
  slot = b / L + n + (long)i;
  return Segment{(long)b + t0, n, t0, L, total};
}

// The last segment of sequence n of a packed batch.
__device__ static inline Segment last_segment_of(const int32_t* cu, int T, int L, int n, long& slot) {
  const int b = taken(cu[n], 0, T), total = taken(cu[n + 1], b, T) - b;
  const int i = max(total - 1, 0) / L, t0 = i * L;
  slot = b / L + n + (long)i;
  return Segment{(long)b + t0, n, t0, total - t0, total};
}

// A whole sequence as one segment; any offsets.
__device__ static inline Segment sequence_of(const int32_t* cu, int T, int n) {
  if (!cu) return Segment{(long)n * T, n, 0, T, T};
  const int b = taken(cu[n], 0, T), e = taken(cu[n + 1], b, T);
  return Segment{b, n, 0, e - b, e - b};
}

// Looks for sequence n's slot among the earlier ones'.  All 64 lanes take part,
// with one n.  The first loads are issued at once, so that a caller can issue its
// own behind them before it asks for the answer (a token each of 512 sequences of
// 2,560 channels: the scan 60 us with 64 slots a turn and the state's loads behind
// the answer, 43 so and with its states past the caches; the convolution 9.8 and 8.8).
struct SlotSearch {
  static constexpr int MANY = 4;
  int slot, seen[MANY];
  __device__ SlotSearch() : slot(0) {}
  __device__ SlotSearch(const int32_t* slots, int n) : slot(slots[n]) { load(slots, n, 0); }
  __device__ void load(const int32_t* slots, int n, int first) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int k = 0; k < MANY; ++k)
      if (first + 64 * k < n) seen[k] = slots[min(first + 64 * k + lane, n)];
  }
  __device__ bool in(int nslots) const { return (unsigned)slot < (unsigned)nslots; }
  // In the pool, and not an earlier sequence's.
  __device__ bool own(const int32_t* slots, int nslots, int n) {
    const int lane = threadIdx.x & 63;
    if (!in(nslots)) return false;
    for (int first = 0; first < n; first += 64 * MANY) {
      if (first) load(slots, n, first);
      bool same = false;
#pragma unroll
      for (int k = 0; k < MANY; ++k)
        if (first + 64 * k < n) same |= first + 64 * k + lane < n && seen[k] == slot;
      if (__ballot(same)) return false;
    }
    return true;
  }
};

}  // namespace

#endif  // GDN_ROWS_H

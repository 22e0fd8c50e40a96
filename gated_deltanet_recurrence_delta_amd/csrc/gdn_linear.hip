// Linear attention with one fixed decay per head, chunkwise, for gfx950:
//
//   S_t = a S_{t-1} + k_t v_t^T,   o_t = S_t^T q_t,   a = exp(g_h).
//
// Forward and backward are one operation on three row streams x, y, z with a
// state S of dx rows and dz columns,
//
//   out_i = sum_{j <= i} a^(i-j) (x_i . y_j) z_j + a^(i+1) S0^T x_i,
//   S_end = a^n S0 + sum_j a^(n-1-j) y_j z_j^T:
//
//   outputs   x, y, z = q, k, v      S0 = h0        S_end = hT
//   dq        x, y, z = dout, v, k   S0 = h0^T
//   dk        x, y, z = v, dout, q   S0 = dhT^T     from the last row to the
//   dv        x, y, z = k, q, dout   S0 = dhT       first; S_end = dh0
//
// where backwards the state is met after the row's own decay, not before it:
// out_i takes a^i S0 and S_end takes a^(n-j) y_j z_j^T.
//
// Chunks of C rows: with P = (X Y^T) . a^(i-j) (j <= i),
//   O = P Z + diag(a^(i+1)) X S,   S <- a^C S + (diag(a^(C-1-j)) Y)^T Z.
//
// A workgroup walks the chunks of one chain (or of a segment of it) with the
// whole state in registers: each wave owns 16 state columns, all dx rows of
// them, so the state's accumulators are the outputs' operand as they stand
// and nothing of the state goes through LDS.  The scores are formed
// transposed, Y X^T, so that their accumulators are an operand too; their
// 16 x 16 blocks are shared out among the waves and handed over through LDS,
// one chunk ahead of their use.  The waves copy the rows to LDS themselves,
// two chunks ahead, and one barrier a chunk hands over rows and scores.
//
// Bound by memory: every row is read once by one workgroup, or twice where
// its chain is cut (two launches, see segment_chunks).  B=4 H=16 T=4096,
// dx = dz = 128 bf16 (medians): 41 us for the segments' states, 63 us for the
// outputs, 64 KB for each 64 rows of a workgroup in 3.2 us, 5.1 TB/s over the
// device (a copy of the same size reaches 4.7); 11 us of each launch are its
// start, the first chunks' way and the last stores.  The outputs' launch reads
// 218 MB from memory and writes 71, what its rows and states are.  512 chains
// uncut (2.1 GB): 472 us, 4.5 TB/s.
//
// What was tried in its place, for the same call: workgroups of 32 state
// columns, four to a chain, need no segments, but read x and y four times
// over, which L2 gives at 11 TB/s and no more: 98 us in one launch.  Two
// workgroups on a CU with half the rows in flight each: 71 us for the
// outputs.  A wave of its own for the copies, scores behind a barrier of
// their own: 66 us.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "gdn_checks.h"
#include "gdn_device.h"
#include "gdn_linear.h"
#include "gdn_linear_places.h"

namespace {

struct Role {
  const char* x;
  const char* y;
  const char* z;
  char* out;
  const float* s0;   // null: zero
  float* sT;         // null: not wanted
  int s0_transposed;
  int reverse;
};

struct LinParams {
  Role role[3];
  const float* g;
  const int32_t* cu;  // null: dense
  f32x4* ws;          // end states of the segments
  int B, T, H, nrole;
  int segc;           // chunks of a segment, an even number; 0: nothing is cut
  int nslots;         // places of (sequence, segment)
  int nseg;           // of them a dense sequence's
};

template <typename TI, int DX, int DZ, int PASS>
struct LK {
  using Frag = typename Mma<TI>::frag;
  static constexpr bool B16 = sizeof(TI) == 2;
  static constexpr int ES = sizeof(TI), SLAB = Mma<TI>::SLAB, E = Mma<TI>::E;
  // Rows of a chunk, 16-row blocks.  bf16: 32 (64 rows at dx = dz = 128 take
  // 272 us where these take 260, 64,711 packed rows of 16 heads).  fp32: 16,
  // which leaves room for two workgroups on a CU (dx = 128, dz = 32, 512
  // chains of 4,096 rows: 594 us, with 32 rows 1,089), but 32 at 128 x 128,
  // where there is room for one either way (256 chains of 4,096 rows: 713 us,
  // with 16 rows 779).
  // The end states of segments, which need no scores, take twice the rows in
  // bf16: half the decays of the state (32,768 rows of 16 heads at 128 x 128:
  // 184 us, with 32 rows in both 199).
  static constexpr int UNIT = B16 || (DX == 128 && DZ == 128) ? 32 : 16;  // of segments
  static constexpr int C = UNIT * (PASS == 1 && B16 ? 2 : 1), NB = C / 16;
  static constexpr int NW = DZ / 16, NT = 64 * NW;             // waves, threads
  static constexpr int GR = DX * ES / 16, ZGR = DZ * ES / 16;  // 16-byte granules of a row
  static constexpr int NS = DX / SLAB, NJS = C / SLAB, TPS = SLAB / 16, NU = DX / 16;
  // LDS: NBUF chunks of (x,) y and z, the scores of two chunks, and decays of
  // scores.
  static constexpr int YB = C * DX * ES, ZB = C * DZ * ES, AT_Y = PASS == 0 ? YB : 0, AT_Z = AT_Y + YB, SB = AT_Z + ZB;
  static constexpr int NBUF = PASS == 0 ? 3 : 4;
  // bf16 terms that the decayed z are taken as where they enter the state:
  // their 24 bits (two terms would leave 2^-18 of each value, and spare 2% of
  // a pass that memory bounds)
  static constexpr int TERMS = B16 ? 3 : 1;
  // Fragments of scores, rows 16 ib and on against SLAB columns from SLAB js on.
  __host__ __device__ static constexpr int frag_at(int ib, int js) {
    int n = js;
    for (int i = 0; i < ib; ++i) n += i / TPS + 1;
    return n;
  }
  // In bf16 they are two terms, 16 bits: with the state's and the outputs' own
  // roundings a third one would show, and two more products a chunk do not.
  static constexpr int PT = B16 ? 2 : 1, NFR = PT * frag_at(NB, 0);
  static constexpr int PB = PASS == 0 ? NFR * 1024 : 0, DB = PASS == 0 ? 2048 : 0;
  static constexpr int AT_P = NBUF * SB, AT_D = AT_P + 2 * PB, LDS = AT_D + DB;
  static constexpr int Y_INS = YB / 1024, Z_INS = ZB / 1024;  // copies of 1 KB
  static constexpr int GROUP = (DX < DZ ? DX : DZ) * ES < 128 ? 2 : 1;  // heads whose rows share a 128-byte line
  // A wave's copies a chunk, at least, and its stores.
  static constexpr int COPIES = (Y_INS >= NW ? (PASS == 0 ? 2 : 1) * Y_INS / NW : 0) + (Z_INS >= NW ? Z_INS / NW : 0);
  static constexpr int STORES = PASS == 0 ? NB : 0;
  static_assert(2 * COPIES + STORES < 64, "operations in flight are counted in six bits");
  // In 16-bit storage a transposing read takes four neighbouring values of a
  // row, half a granule.  The halves alternate from granule to granule, so
  // that a read covers all banks: accumulator row m = 4 q + e of tile t of a
  // slab is x value 8 q + 4 (t ^ (q & 1)) + e, and a lane's eight values of
  // two tiles are neighbours.
  __device__ static inline int half_of(int t, int q) { return 4 * (t ^ (q & 1)); }
  __device__ static inline int x_of(int t, int q) { return B16 ? 8 * q + half_of(t, q) : 4 * q; }
  __device__ static inline int swz_y(int r) { return swz_kq<GR>(r); }
  // A transposing read of z takes 32 bytes of each of eight rows.
  __device__ static inline int swz_z(int r) {
    if constexpr (!B16) return 0;
    else if constexpr (ZGR >= 16) return 8 * (r & 1) + 4 * ((r >> 1) & 1) + 2 * ((r >> 2) & 1);
    else if constexpr (ZGR >= 8) return 4 * ((r >> 1) & 1) + 2 * ((r >> 2) & 1);
    else return 2 * ((r >> 2) & 1);
  }
};

// A state's decay over n rows.  A constant factor's rounding would add up
// over the chunks, always to the same side: near one it is applied as
// m + (a^n - 1) m, whose rounding goes either way.
struct Decay {
  float f;
  bool near_one;
};
__device__ static inline Decay decay_of(double d) { return {(float)(d > 0.5 ? d - 1.0 : d), d > 0.5}; }
__device__ static inline double pow_of(float g, long n) { return n == 0 ? 1.0 : exp((double)g * (double)n); }
template <bool NEAR_ONE, int N>
__device__ static inline void apply(const float f, f32x4 (&m)[N]) {
#pragma unroll
  for (int u = 0; u < N; ++u)
#pragma unroll
    for (int e = 0; e < 4; ++e) m[u][e] = NEAR_ONE ? __builtin_fmaf(m[u][e], f, m[u][e]) : m[u][e] * f;
}

// What four values' rounding to bf16 (two packed pairs) left of them, exactly.
__device__ static inline f32x4 left_over(f32x4 x, u32x2 t) {
  return f32x4{x[0] - __uint_as_float(t[0] << 16), x[1] - __uint_as_float(t[0] & 0xffff0000u),
               x[2] - __uint_as_float(t[1] << 16), x[3] - __uint_as_float(t[1] & 0xffff0000u)};
}

// Where a workgroup's chain and segment lie.
struct Span {
  long th0;  // token-head of the sequence's first row
  int n, seg, slot, h, ri, len, nch, c0, c1;
};

// Rows further back than this many nats of decay are left out of a segment's
// end state: e^-40 of their own share, as the halos of the delta rule's
// segments are bounded.
constexpr double FORGOTTEN = 40.0;

// 16 bytes a lane from the buffer to LDS, from `at` on.  From assembly: the
// copy writes LDS only, and as a builtin it would make the compiler wait for
// all of a wave's copies before each of its own LDS reads.  The waits stand
// before the barriers that hand a chunk over.  (The wait states are for a
// descriptor or an address that a vector instruction has just put into scalar
// registers: the compiler does not look into the assembly.)
__device__ static inline void lds_copy(unsigned at, int off, __amdgpu_buffer_rsrc_t r) {
#ifdef __HIP_DEVICE_COMPILE__
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :
               : "s"(at), "v"(off), "s"(r)
               : "m0");
#endif
}

// A wave's share of the copies of one stream's chunks to LDS: INS copies a
// chunk among NW waves, rows of G16 granules.
template <int INS, int NW, int G16>
struct Copier {
  static constexpr int MINE = (INS + NW - 1) / NW;
  static_assert(INS % NW == 0 || INS < NW, "even shares");
  __amdgpu_buffer_rsrc_t rsrc;
  unsigned off[MINE], step, at;
  bool any;

  // `base`: the sequence's first row; `place(row, granule)`: where a granule of a row lies in the buffer's row
  template <typename F>
  __device__ inline Copier(const char* base, int stride, int len, int rev, unsigned first, int rows, int w,
                           const char* lds, F place) {
    const int lane = threadIdx.x & 63;
    rsrc = make_rsrc(base, (long)(len - 1) * stride + G16 * 16);
    any = INS >= NW || w < INS;
    at = (unsigned)(uintptr_t)(const __attribute__((address_space(3))) char*)lds + w * MINE * 1024;
    step = (unsigned)(rev ? -rows : rows) * (unsigned)stride;
#pragma unroll
    for (int k = 0; k < MINE; ++k) {
      const int G = (w * MINE + k) * 64 + lane, r = G / G16;
      // Rows outside the sequence lie outside the descriptor (a negative
      // offset wraps far behind it) and read as zeros.
      off[k] = (rev ? (unsigned)(len - 1) - first - r : first + r) * (unsigned)stride + 16 * place(r, G % G16);
    }
  }
  // The next chunk to `shift` bytes behind the first buffer; without `in`,
  // zeros, so that the loop over the chunks has no branch for its last one.
  __device__ inline void issue(int shift, bool in) {
    if (INS >= NW || any) {
#pragma unroll
      for (int k = 0; k < MINE; ++k) {
        lds_copy(at + shift + k * 1024, in ? (int)off[k] : -16, rsrc);
        off[k] += step;
      }
    }
  }
};

// A wave's part.
template <typename TI, int DX, int DZ, int PASS>
__device__ static inline void compute(const LinParams& p, const Span& sp, const float gh, const int w, char* lds,
                                      double* sPow, float* sIn) {
  using K = LK<TI, DX, DZ, PASS>;
  using Frag = typename K::Frag;
  constexpr int C = K::C;
  const Role& role = p.role[sp.ri];
  const int lane = threadIdx.x & 63, m16 = lane & 15, q4 = lane >> 4;
  const int H = p.H, rev = role.reverse, len = sp.len;
  char* const sP = lds + K::AT_P;
  char* const sD = lds + K::AT_D;
  const int z_at = 16 * w + m16;  // the lane's state column
  const int x_stride = H * DX * K::ES, z_stride = H * DZ * K::ES;
  const unsigned row0 = (unsigned)sp.c0 * C;
  auto place_y = [](int r, int g) { return g ^ K::swz_y(r); };
  auto place_z = [](int r, int g) { return g ^ K::swz_z(r); };
  const long x0 = sp.th0 * DX * K::ES;
  Copier<K::Y_INS, K::NW, K::GR> cx(role.x + x0, x_stride, len, rev, row0, C, w, lds, place_y);
  Copier<K::Y_INS, K::NW, K::GR> cy(role.y + x0, x_stride, len, rev, row0, C, w, lds + K::AT_Y, place_y);
  Copier<K::Z_INS, K::NW, K::ZGR> cz(role.z + sp.th0 * DZ * K::ES, z_stride, len, rev, row0, C, w, lds + K::AT_Z,
                                     place_z);
  auto issue = [&](int slot, bool in) {
    if constexpr (PASS == 0) cx.issue(slot * K::SB, in);
    cy.issue(slot * K::SB, in);
    cz.issue(slot * K::SB, in);
  };
#pragma unroll
  for (int i = 0; i < K::NBUF - 1; ++i) issue(i, sp.c0 + i < sp.c1);

  // The decay's powers, while the first chunks are on their way.
  const int tid = threadIdx.x;
  if (tid <= C) {
    const double a = pow_of(gh, tid);
    sPow[tid] = a;
    sIn[C - tid] = (float)a;
  } else if (tid < 2 * C) {
    sIn[tid] = 0.f;
  }
  lds_barrier();

  // The state: tile u has x rows x_at(u) and on.
  f32x4 M[K::NU];
  auto x_at = [&](int u) { return u / K::TPS * K::SLAB + K::x_of(u % K::TPS, q4); };
  auto ws_at = [&](int sl) {
    return p.ws + (((long)sl * H + sp.h) * p.nrole + sp.ri) * (DX * DZ / 4) + w * K::NU * 64 + lane;
  };
#pragma unroll
  for (int u = 0; u < K::NU; ++u) M[u] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (sp.c0 == 0) {
    if (role.s0) {
      const float* s0 = role.s0 + ((long)sp.n * H + sp.h) * DX * DZ;
#pragma unroll
      for (int u = 0; u < K::NU; ++u) {
        if (role.s0_transposed) {
          M[u] = *reinterpret_cast<const f32x4*>(s0 + z_at * DX + x_at(u));
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) M[u][e] = s0[(x_at(u) + e) * DZ + z_at];
        }
      }
    }
  } else if (PASS == 0) {
    const Decay a = decay_of(pow_of(gh, (long)p.segc * K::UNIT));
    const double nats = -(double)gh * p.segc * K::UNIT;
    const int first = nats * sp.seg > FORGOTTEN ? max(sp.slot - sp.seg, sp.slot - 1 - (int)(FORGOTTEN / nats))
                                                : sp.slot - sp.seg;
    auto add = [&](int s) {
      const f32x4* src = ws_at(s);
#pragma unroll
      for (int u = 0; u < K::NU; ++u) M[u] += src[u * 64];
    };
    if (a.near_one && __builtin_isinf(a.f)) {
      // A growing state may be zero in segments over which the growth is past
      // fp32: it grows chunk by chunk, and zeros stay zeros.
      const float f = (float)(sPow[C] - 1.0);
      for (int s = first; s < sp.slot; ++s) {
        for (int c = 0; c < p.segc; ++c) apply<true>(f, M);
        add(s);
      }
    } else {
      for (int s = first; s < sp.slot; ++s) {
        if (a.near_one) apply<true>(a.f, M);
        else apply<false>(a.f, M);
        add(s);
      }
    }
  }

  // The state's power of the decay at output row i = 16 ib + m16; backwards
  // one lower, as the inputs' at row j are one higher.
  float gam[K::NB];
  const Decay step = decay_of(sPow[C]);
  const __amdgpu_buffer_rsrc_t ro = make_rsrc(role.out + sp.th0 * DZ * K::ES, (long)(len - 1) * z_stride + DZ * K::ES);
  unsigned o_off = 0;
  const unsigned o_step = (unsigned)(rev ? -C : C) * (unsigned)z_stride;
  const unsigned o_blk = (unsigned)(rev ? -16 : 16) * (unsigned)z_stride;
  if constexpr (PASS == 0) {
#pragma unroll
    for (int ib = 0; ib < K::NB; ++ib) gam[ib] = (float)sPow[16 * ib + m16 + 1 - rev];
    const unsigned i = (unsigned)sp.c0 * C + m16;
    o_off = (rev ? (unsigned)(len - 1) - i : i) * (unsigned)z_stride + (16 * w + 4 * q4) * K::ES;
    // The decays of a block of scores (row 16 ib + m16, column 16 jb + 4 q4 +
    // e) on the diagonal and beside it; and the zeros beside diagonal blocks.
    for (int d = w; d < 2; d += K::NW) {
      f32x4 v;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int n = 16 * d + m16 - 4 * q4 - e;
        v[e] = n >= 0 ? (float)sPow[min(n, C)] : 0.f;  // past C: beside the diagonal of a chunk of one block, unused
      }
      lds_st(sD, (d * 64 + lane) * 16, v);
    }
    for (int f = w; f < 2 * K::NFR; f += K::NW) lds_st(sP, (f * 64 + lane) * 16, f32x4{0.f, 0.f, 0.f, 0.f});
  }
  const int tr_r = 4 * q4 + (m16 >> 2), tr_g = m16 & 3;
  const int x_row = m16 * (K::GR * 16);
  auto x_granule = [&](int s) { return (((K::SLAB * K::ES / 16) * s + q4) ^ K::swz_y(m16)) * 16; };
  // This wave's blocks of a chunk's scores, transposed and masked.
  auto scores = [&](const char* at_chunk, char* to) {
    auto block = [&](int ib, int jb) {
      const char* bX = at_chunk + 16 * ib * (K::GR * 16);
      const char* bY = at_chunk + K::AT_Y + 16 * jb * (K::GR * 16);
      f32x4 P = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < K::NS; ++s)
        P = Mma<TI>::mma(lds_ld<Frag>(bY, x_row + x_granule(s)), lds_ld<Frag>(bX, x_row + x_granule(s)), P);
      static_assert(PASS == 1 || K::NB <= 2, "two tables of decays");
      const f32x4 decay = lds_ld<f32x4>(sD, ((ib - jb) * 64 + lane) * 16);
#pragma unroll
      for (int e = 0; e < 4; ++e) P[e] *= decay[e];
      char* at = to + (K::PT * K::frag_at(ib, jb / K::TPS) * 64 + lane) * 16;
      if constexpr (K::B16) {
        const u32x2 first = __builtin_bit_cast(u32x2, cvt4(P));
        lds_st(at, 8 * (jb & 1), first);
        lds_st(at, 1024 + 8 * (jb & 1), cvt4(left_over(P, first)));
      } else {
        lds_st(at, 0, P);
      }
    };
    constexpr int BLOCKS = K::NB * (K::NB + 1) / 2;
#pragma unroll
    for (int b0 = 0; b0 < BLOCKS; b0 += K::NW) {
      const int b = b0 + w;
      if (b0 + K::NW <= BLOCKS || b < BLOCKS) {
        const int ib = b >= 1;
        block(ib, b - ib * (ib + 1) / 2);
      }
    }
  };

  if constexpr (PASS == 0) {  // two chunks
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
    lds_barrier();
    scores(lds, sP);
  } else {
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(K::COPIES));
  }
  lds_barrier();

  // A chunk's z columns as fragments over the rows (for two 16-row blocks:
  // rows 4 q4 and on of the first, then of the second, as the scores'
  // accumulators lie), and as they enter the state: decayed, in 16-bit
  // storage as TERMS terms.
  struct ZCols {
    Frag f[K::NJS], t[K::NJS][K::TERMS];
  };
  auto load_z = [&](const char* bZ, ZCols& z) {
#pragma unroll
    for (int js = 0; js < K::NJS; ++js) {
      if constexpr (K::B16) {
        const char* at = bZ + tr_r * (K::ZGR * 16) + (((2 * w + (tr_g >> 1)) ^ K::swz_z(tr_r)) * 16) + 8 * (tr_g & 1);
        const bf16x4 lo = lds_read_tr(at, 32 * js * (K::ZGR * 16));
        const bf16x4 hi = lds_read_tr(at, (32 * js + 16) * (K::ZGR * 16));
        z.f[js] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) z.f[js][e] = lds_ld<float>(bZ, ((16 * js + 4 * q4 + e) * DZ + z_at) * 4);
      }
    }
  };
  auto decay_z = [&](int rows, ZCols& z) {  // rows behind the last have zeros
    const float* in_pow = sIn + C - (rows - 1 + rev) + 4 * q4;
#pragma unroll
    for (int js = 0; js < K::NJS; ++js) {
      if constexpr (K::B16) {
        f32x4 a, b;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          a[e] = (float)z.f[js][e] * in_pow[32 * js + e];
          b[e] = (float)z.f[js][4 + e] * in_pow[32 * js + 16 + e];
        }
#pragma unroll
        for (int i = 0; i < K::TERMS; ++i) {
          const u32x2 ta = __builtin_bit_cast(u32x2, cvt4(a)), tb = __builtin_bit_cast(u32x2, cvt4(b));
          z.t[js][i] = __builtin_bit_cast(Frag, u32x4{ta[0], ta[1], tb[0], tb[1]});
          if (i + 1 < K::TERMS) {
            a = left_over(a, ta);
            b = left_over(b, tb);
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) z.t[js][0][e] = z.f[js][e] * in_pow[16 * js + e];
      }
    }
  };

  // One chunk: its outputs and its share of the state; and the next chunk's z
  // made ready, vector work that runs beside this one's matrix products.
  int slot = 0;
  auto chunk = [&](auto near_one, const int c, const ZCols& z, ZCols& zn) {
    const char* bX = lds + slot * K::SB;
    const char* bY = bX + K::AT_Y;
    issue(slot == 0 ? K::NBUF - 1 : slot - 1, c + K::NBUF - 1 < sp.c1);
    slot = slot == K::NBUF - 1 ? 0 : slot + 1;
    load_z(lds + slot * K::SB + K::AT_Z, zn);

    // the next chunk's scores (behind the last chunk there are zeros)
    if constexpr (PASS == 0) scores(lds + slot * K::SB, sP + (~(c - sp.c0) & 1) * K::PB);

    f32x4 O[K::NB];
    if constexpr (PASS == 0) {
      // The state's part of the outputs, transposed.  In bf16 the state is one
      // term, rounded as the outputs themselves are.  Two terms take the
      // outputs' error from 2.0e-3 to their own rounding's 1.7e-3 (a norm, on
      // random rows), and a seventh more time (64,711 packed rows of 16 heads,
      // dx = dz = 128: 287 us, with one term 249).
      Frag Mf[K::NS];
#pragma unroll
      for (int s = 0; s < K::NS; ++s) {
        if constexpr (K::B16) {
          const u32x2 a = __builtin_bit_cast(u32x2, cvt4(M[2 * s])), b = __builtin_bit_cast(u32x2, cvt4(M[2 * s + 1]));
          const bool odd = q4 & 1;  // tile 0 has the lane's upper four rows
          Mf[s] = __builtin_bit_cast(
              Frag, u32x4{odd ? b[0] : a[0], odd ? b[1] : a[1], odd ? a[0] : b[0], odd ? a[1] : b[1]});
        } else {
          Mf[s] = M[s];
        }
      }
#pragma unroll
      for (int ib = 0; ib < K::NB; ++ib) {
        O[ib] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < K::NS; ++s) {
          O[ib] = Mma<TI>::mma(Mf[s], lds_ld<Frag>(bX + 16 * ib * (K::GR * 16), x_row + x_granule(s)), O[ib]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) O[ib][e] *= gam[ib];
      }
      const char* bP = sP + ((c - sp.c0) & 1) * K::PB;
      // the chunk's own part
#pragma unroll
      for (int ib = 0; ib < K::NB; ++ib) {
#pragma unroll
        for (int js = 0; js * K::TPS <= ib; ++js)
#pragma unroll
          for (int t = K::PT - 1; t >= 0; --t)
            O[ib] = Mma<TI>::mma(z.f[js], lds_ld<Frag>(bP, ((K::PT * K::frag_at(ib, js) + t) * 64 + lane) * 16), O[ib]);
        if constexpr (K::B16)
          __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, cvt4(O[ib])), ro, (int)(o_off + ib * o_blk), 0,
                                                0);
        else
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, O[ib]), ro, (int)(o_off + ib * o_blk), 0, 0);
      }
      o_off += o_step;
    }

    // the state: decayed, and the chunk's y z^T
    const int rows = min(C, len - c * C);
    // a shorter last chunk: its decay is no further from one, or comes once only
    const float last = (float)(decltype(near_one)::value ? sPow[rows] - 1.0 : sPow[rows]);
    apply<decltype(near_one)::value != 0>(rows < C ? last : step.f, M);
    decay_z(max(1, min(C, len - (c + 1) * C)), zn);
#pragma unroll
    for (int js = 0; js < K::NJS; ++js) {
      constexpr int UB = K::NU < 4 ? K::NU : 4;  // tiles at a time: independent products one behind another
#pragma unroll
      for (int u0 = 0; u0 < K::NU; u0 += UB) {
        Frag y[UB];
#pragma unroll
        for (int v = 0; v < UB; ++v) {
          const int u = u0 + v;
          if constexpr (K::B16) {
            const char* at = bY + tr_r * (K::GR * 16) + (((4 * (u / 2) + tr_g) ^ K::swz_y(tr_r)) * 16) +
                             2 * K::half_of(u & 1, tr_g);
            const bf16x4 lo = lds_read_tr(at, 32 * js * (K::GR * 16));
            const bf16x4 hi = lds_read_tr(at, (32 * js + 16) * (K::GR * 16));
            y[v] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
          } else {
            const int x = u * 16 + m16;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int r = 16 * js + 4 * q4 + e;
              y[v][e] = lds_ld<float>(bY, r * (K::GR * 16) + (((x >> 2) ^ K::swz_y(r)) * 16) + (x & 3) * 4);
            }
          }
        }
#pragma unroll
        for (int i = K::TERMS - 1; i >= 0; --i)
#pragma unroll
          for (int v = 0; v < UB; ++v) M[u0 + v] = Mma<TI>::mma(y[v], z.t[js][i], M[u0 + v]);
      }
    }
    // The chunk after the next has to be there: behind its copies are this
    // chunk's stores, or the copies of the one after it.
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(PASS == 0 ? K::STORES : K::COPIES));
    lds_barrier();
  };
  auto walk = [&](auto near_one) {
    ZCols za, zb;
    load_z(lds + K::AT_Z, za);
    decay_z(max(1, min(C, len - sp.c0 * C)), za);
    for (int c = sp.c0; c < sp.c1;) {
      chunk(near_one, c, za, zb);
      if (++c >= sp.c1) break;
      chunk(near_one, c, zb, za);
      ++c;
    }
  };
  // One loop for each kind of decay: a choice inside it would cost a copy of the state a chunk.
  if (step.near_one) walk(IC<1>{});
  else walk(IC<0>{});
  __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));  // no copy outlives the workgroup's LDS

  if constexpr (PASS == 1) {
    f32x4* dst = ws_at(sp.slot);
#pragma unroll
    for (int u = 0; u < K::NU; ++u) dst[u * 64] = M[u];
  } else if (role.sT && sp.c1 >= sp.nch) {
    float* sT = role.sT + ((long)sp.n * H + sp.h) * DX * DZ;
#pragma unroll
    for (int u = 0; u < K::NU; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) sT[(x_at(u) + e) * DZ + z_at] = M[u][e];
  }
}

// The place of a workgroup in a packed batch (one for all of its threads:
// what follows from it stays in scalar registers).
template <int PASS, int NT>
__device__ static inline Place packed_place(const Packed& b, int rows, int at, PlaceBoard& board) {
  const int tid = threadIdx.x;
  const Places<PASS> places = {b, rows, at};
  places.begin(tid, board);
  __syncthreads();
  places.look(tid, NT, board);
  __syncthreads();
  places.settle(tid, NT, board);
  __syncthreads();
  const Place r = places.place(board);
  __syncthreads();
  return {__builtin_amdgcn_readfirstlane(r.n), __builtin_amdgcn_readfirstlane(r.seg),
          __builtin_amdgcn_readfirstlane(r.uncut) != 0};
}

// PASS 0: outputs (and end states); PASS 1: the end states of the segments
// that others follow, each from zero (a sequence's first from S0).
template <typename TI, int DX, int DZ, int PASS>
__global__ __launch_bounds__((LK<TI, DX, DZ, PASS>::NT), 2) void linear_kernel(const LinParams p) {
  using K = LK<TI, DX, DZ, PASS>;
  constexpr int C = K::C;
  __shared__ __attribute__((aligned(16))) char lds[K::LDS];
  __shared__ double sPow[C + 1];
  __shared__ float sIn[2 * C];  // the decay's powers from C down to 0, then zeros
  static_assert(K::NT >= 2 * C, "a thread for each");
  static_assert(K::LDS >= (int)sizeof(PlaceBoard), "the board is in the same memory");

  const int tid = threadIdx.x;
  // Consecutive workgroups go to the XCDs in turn: each XCD has every eighth
  // group of chains, and the roles of a chain, which read the same rows, are
  // neighbours on one.  A group is the heads whose rows share a 128-byte line.
  constexpr int G = K::GROUP;
  const int k = blockIdx.x >> 3, kc = k / p.nrole;
  const int chain = (kc / G * 8 + (blockIdx.x & 7)) * G + kc % G;
  Span sp;
  sp.ri = k % p.nrole;
  if (chain >= p.nslots * p.H) return;
  const int place = chain / p.H;
  sp.h = chain % p.H;
  long row0;
  bool cut = p.segc != 0;
  if (p.cu) {
    const int rows = cut ? p.segc * K::UNIT : p.T + 1;
    const Packed batch = {p.cu, p.B, p.T};
    const Place at = packed_place<PASS, K::NT>(batch, rows, place, *reinterpret_cast<PlaceBoard*>(lds));
    if (at.n < 0) return;
    const Rows r = rows_of(batch, at.n);
    cut = cut && !at.uncut;
    row0 = r.begin;
    sp.n = at.n;
    sp.seg = at.seg;
    sp.len = r.len;
    sp.slot = r.begin / rows + sp.seg;
  } else {
    sp.n = place / p.nseg;
    sp.seg = place % p.nseg;
    row0 = (long)sp.n * p.T;
    sp.len = p.T;
    sp.slot = place;
  }
  sp.th0 = row0 * p.H + sp.h;
  sp.nch = (sp.len + C - 1) / C;
  const int segc = p.segc / (C / K::UNIT);  // whole: segments have an even number of units
  sp.c0 = sp.seg * segc;
  sp.c1 = cut ? min(sp.nch, sp.c0 + segc) : sp.nch;
  if (sp.seg > 0 && sp.c0 >= sp.nch) return;
  const float gh = p.g[sp.h];
  if constexpr (PASS == 1) {
    if (sp.c1 >= sp.nch) return;  // nothing follows
    const double nats = -(double)gh * C;
    if (nats * (sp.c1 - sp.c0) > FORGOTTEN) sp.c0 = max(sp.c0, sp.c1 - 1 - (int)(FORGOTTEN / nats));
  }
  compute<TI, DX, DZ, PASS>(p, sp, gh, __builtin_amdgcn_readfirstlane(tid >> 6), lds, sPow, sIn);
}

// ------------------------------------------------------------------- host --

constexpr int CUS = 256;    // of an MI355X
constexpr int SEG_MIN = 4;  // chunks a segment has at least
constexpr int PACKED_SEG_MIN = 4;

int chunk_rows(int dx, int dz, int dtype) { return dtype == GDN_BF16 || (dx == 128 && dz == 128) ? 32 : 16; }  // LK::UNIT

// Chunks of a segment, or 0: a sequence is cut where a batch has fewer
// chains than the device holds workgroups.  What a cut costs is a first
// launch over y and z, some 0.6 of the second's time a chunk; what it brings
// is shorter rounds of workgroups.
int segment_chunks(int B, int T, int H, int dx, int dz, int roles, bool packed, int dtype) {
  const long rows = chunk_rows(dx, dz, dtype), chains = (long)B * H * roles, room = CUS;
  if (chains <= 0 || T == 0) return 0;
  if (packed) {
    // lengths are not known here: no segment is longer than an even share
    const long all = ((long)T + rows - 1) / rows;
    const long share = (std::max<long>(PACKED_SEG_MIN, (all * H * roles + room - 1) / room) + 1) / 2 * 2;
    return share < all ? (int)share : 0;
  }
  const long nch = ((long)T + rows - 1) / rows;
  long best = 0, least = 0;
  for (long n = 1; n <= 32 && (n == 1 || nch / n >= SEG_MIN); ++n) {
    const long segc = ((nch + n - 1) / n + 1) / 2 * 2, segs = (nch + segc - 1) / segc;  // an even number
    long cost = 10 * ((chains * segs + room - 1) / room) * (segc + 1);
    if (n > 1) cost += 6 * ((chains * (segs - 1) + room - 1) / room) * (segc + 1) + 20;
    if (n == 1 || cost < least) {
      least = cost;
      best = segs == 1 ? 0 : segc;
    }
  }
  return (int)best;
}

// Places of (sequence, segment) in a launch, by pass.
long segment_places(int B, int T, bool packed, int segc, int chunk, int pass) {
  if (!segc) return B;
  const long rows = (long)segc * chunk;
  return packed ? T / rows + (pass == 0 ? B : 0) : B * (((long)T + rows - 1) / rows);
}

long workgroups(long places, const LinParams& p) {
  return (places * p.H + 15) / 16 * 16 * p.nrole;  // whole groups on each of the eight XCDs
}

template <typename TI, int DX, int DZ>
int launch_pass(LinParams p, hipStream_t s) {
  const int chunk = LK<TI, DX, DZ, 0>::UNIT;
  const bool packed = p.cu != nullptr;
  const long places[2] = {segment_places(p.B, p.T, packed, p.segc, chunk, 0),
                          segment_places(p.B, p.T, packed, p.segc, chunk, 1)};
  if (workgroups(places[0], p) >= 1L << 22) return GDN_ERR_INVALID_ARG;
  p.nseg = p.segc && !packed ? (int)(places[0] / p.B) : 1;
  if (p.segc && places[1] > 0) {
    p.nslots = (int)places[1];
    hipLaunchKernelGGL((linear_kernel<TI, DX, DZ, 1>), dim3((unsigned)workgroups(places[1], p)),
                       dim3(LK<TI, DX, DZ, 1>::NT), 0, s, p);
    if (hipGetLastError() != hipSuccess) return GDN_ERR_LAUNCH;
  }
  p.nslots = (int)places[0];
  hipLaunchKernelGGL((linear_kernel<TI, DX, DZ, 0>), dim3((unsigned)workgroups(places[0], p)),
                     dim3(LK<TI, DX, DZ, 0>::NT), 0, s, p);
  return hipGetLastError() == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}

template <typename TI, int DX>
int launch_dz(const LinParams& p, int dz, hipStream_t s) {
  switch (dz) {
    case 32: return launch_pass<TI, DX, 32>(p, s);
    case 64: return launch_pass<TI, DX, 64>(p, s);
    default: return launch_pass<TI, DX, 128>(p, s);
  }
}

int launch(const LinParams& p, int dx, int dz, int dtype, hipStream_t s) {
  const bool b16 = dtype == GDN_BF16;
  switch (dx) {
    case 32: return b16 ? launch_dz<__bf16, 32>(p, dz, s) : launch_dz<float, 32>(p, dz, s);
    case 64: return b16 ? launch_dz<__bf16, 64>(p, dz, s) : launch_dz<float, 64>(p, dz, s);
    default: return b16 ? launch_dz<__bf16, 128>(p, dz, s) : launch_dz<float, 128>(p, dz, s);
  }
}

// Sizes of both directions: 0, or the status to return.
int check_sizes(int B, int T, int H, int dk, int dv, bool packed, int dtype) {
  if (B < 0 || T < 0 || H < 1 || H > 65535 || dk < 1 || dv < 1) return GDN_ERR_INVALID_ARG;
  if (dtype != GDN_F32 && dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
  if ((dk != 32 && dk != 64 && dk != 128) || (dv != 32 && dv != 64 && dv != 128)) return GDN_ERR_UNSUPPORTED;
  // 32-bit offsets in a sequence's rows; the grid
  if ((long long)T * H * std::max(dk, dv) * (dtype == GDN_BF16 ? 2 : 4) > 0x7fffffffLL) return GDN_ERR_INVALID_ARG;
  if ((long long)B * H >= 1LL << 18) return GDN_ERR_INVALID_ARG;
  if (!packed && (long long)B * T > 0x7fffffffLL) return GDN_ERR_INVALID_ARG;
  return GDN_OK;
}

struct Plan {
  int segc;
  long long bytes;
};

// One launch of `roles` roles of states dx x dz.
Plan plan(int B, int T, int H, int dx, int dz, int roles, bool packed, int dtype) {
  const int segc = segment_chunks(B, T, H, dx, dz, roles, packed, dtype);
  if (!segc) return {0, 0};
  return {segc, segment_places(B, T, packed, segc, chunk_rows(dx, dz, dtype), 1) * H * roles * dx * dz * 4LL};
}

}  // namespace

extern "C" long long gdn_linear_workspace_size(int B, int T, int H, int dk, int dv, int packed, int dtype,
                                               int backward) {
  const int rc = check_sizes(B, T, H, dk, dv, packed != 0, dtype);
  if (rc != GDN_OK) return rc;
  if (!backward) return plan(B, T, H, dk, dv, 1, packed != 0, dtype).bytes;
  if (dk == dv) return plan(B, T, H, dk, dv, 3, packed != 0, dtype).bytes;
  return plan(B, T, H, dv, dk, 2, packed != 0, dtype).bytes + plan(B, T, H, dk, dv, 1, packed != 0, dtype).bytes;
}

extern "C" int gdn_linear_fwd(const void* q, const void* k, const void* v, const float* g, const float* h0,
                              const int32_t* cu_seqlens, void* out, float* hT, int B, int T, int H, int dk, int dv,
                              void* stream, int dtype, void* workspace, long long workspace_bytes) {
  const bool packed = cu_seqlens != nullptr;
  const int rc = check_sizes(B, T, H, dk, dv, packed, dtype);
  if (rc != GDN_OK) return rc;
  if (B > 0 && (!g || !hT || (T > 0 && (!q || !k || !v || !out)))) return GDN_ERR_INVALID_ARG;
  Plan pl = plan(B, T, H, dk, dv, 1, packed, dtype);
  if (pl.bytes > 0 && (!workspace || workspace_bytes < pl.bytes)) return GDN_ERR_INVALID_ARG;
  if (misaligned({q, k, v, h0, out, hT, workspace}, 16) || misaligned({g, cu_seqlens}, 4)) return GDN_ERR_INVALID_ARG;
  const long long th = (packed ? 1LL : B) * T * H, e = dtype == GDN_BF16 ? 2 : 4, state = (long long)B * H * dk * dv * 4;
  if (clash({{out, th * dv * e}, {hT, state}, {workspace, pl.bytes}},
            {{q, th * dk * e}, {k, th * dk * e}, {v, th * dv * e}, {g, 4LL * H}, {cu_seqlens, 4LL * (B + 1)},
             {h0 == hT ? nullptr : h0, state}}))
    return GDN_ERR_INVALID_ARG;
  if (B == 0) return GDN_OK;
  if (h0 == hT) pl.segc = 0;  // in place: a later segment's end would be written while an earlier one reads its start
  LinParams p = {};
  p.role[0] = {(const char*)q, (const char*)k, (const char*)v, (char*)out, h0, hT, 0, 0};
  p.g = g;
  p.cu = cu_seqlens;
  p.ws = static_cast<f32x4*>(workspace);
  p.B = B;
  p.T = T;
  p.H = H;
  p.nrole = 1;
  p.segc = pl.segc;
  return launch(p, dk, dv, dtype, static_cast<hipStream_t>(stream));
}

extern "C" int gdn_linear_bwd(const void* q, const void* k, const void* v, const float* g, const float* h0,
                              const int32_t* cu_seqlens, const void* dout, const float* dhT, void* dq, void* dk,
                              void* dv, float* dh0, int B, int T, int H, int dk_, int dv_, void* stream, int dtype,
                              void* workspace, long long workspace_bytes) {
  const bool packed = cu_seqlens != nullptr;
  const int rc = check_sizes(B, T, H, dk_, dv_, packed, dtype);
  if (rc != GDN_OK) return rc;
  if (B > 0 && (!g || (T > 0 && (!q || !k || !v || !dout || !dq || !dk || !dv)))) return GDN_ERR_INVALID_ARG;
  const long long need = gdn_linear_workspace_size(B, T, H, dk_, dv_, packed, dtype, 1);
  if (need > 0 && (!workspace || workspace_bytes < need)) return GDN_ERR_INVALID_ARG;
  if (misaligned({q, k, v, h0, dout, dhT, dq, dk, dv, dh0, workspace}, 16) || misaligned({g, cu_seqlens}, 4))
    return GDN_ERR_INVALID_ARG;
  const long long th = (packed ? 1LL : B) * T * H, e = dtype == GDN_BF16 ? 2 : 4,
                  state = (long long)B * H * dk_ * dv_ * 4;
  if (clash({{dq, th * dk_ * e}, {dk, th * dk_ * e}, {dv, th * dv_ * e}, {dh0, state}, {workspace, need}},
            {{q, th * dk_ * e}, {k, th * dk_ * e}, {v, th * dv_ * e}, {dout, th * dv_ * e}, {g, 4LL * H},
             {cu_seqlens, 4LL * (B + 1)}, {h0, state}, {dhT == dh0 ? nullptr : dhT, state}}))
    return GDN_ERR_INVALID_ARG;
  if (B == 0) return GDN_OK;
  LinParams p = {};
  const Role rq = {(const char*)dout, (const char*)v, (const char*)k, (char*)dq, h0, nullptr, 1, 0};
  const Role rk = {(const char*)v, (const char*)dout, (const char*)q, (char*)dk, dhT, nullptr, 1, 1};
  const Role rv = {(const char*)k, (const char*)q, (const char*)dout, (char*)dv, dhT, dh0, 0, 1};
  p.g = g;
  p.cu = cu_seqlens;
  p.ws = static_cast<f32x4*>(workspace);
  p.B = B;
  p.T = T;
  p.H = H;
  hipStream_t s = static_cast<hipStream_t>(stream);
  // dk reads dhT while dv's workgroups write dh0: in place, dv comes in a launch of its own behind it
  const bool in_place = dh0 && dh0 == dhT;
  if (dk_ == dv_ && !in_place) {
    p.role[0] = rq;
    p.role[1] = rk;
    p.role[2] = rv;
    p.nrole = 3;
    p.segc = plan(B, T, H, dk_, dv_, 3, packed, dtype).segc;
    return launch(p, dk_, dv_, dtype, s);
  }
  const Plan first = plan(B, T, H, dv_, dk_, 2, packed, dtype);
  const bool fits = dk_ != dv_;  // the workspace of equal widths is that of one launch: leave these two uncut
  p.role[0] = rq;
  p.role[1] = rk;
  p.nrole = 2;
  p.segc = fits ? first.segc : 0;
  const int rc2 = launch(p, dv_, dk_, dtype, s);
  if (rc2 != GDN_OK) return rc2;
  p.role[0] = rv;
  p.nrole = 1;
  p.segc = fits && !in_place ? plan(B, T, H, dk_, dv_, 1, packed, dtype).segc : 0;
  p.ws = reinterpret_cast<f32x4*>(static_cast<char*>(workspace) + (fits ? first.bytes : 0));
  return launch(p, dk_, dv_, dtype, s);
}

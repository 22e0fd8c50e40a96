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
// Chunks of 64 rows: with P = (X Y^T) . a^(i-j) (j <= i),
//   O = P Z + diag(a^(i+1)) X S,   S <- a^64 S + (diag(a^(63-j)) Y)^T Z.
//
// A workgroup owns a chain's tile of 32 state columns and walks the chunks.
// X Y^T is then formed once for each 32 columns; in exchange the chain's
// tiles give four times the workgroups, no chain has to be cut while there
// are enough of them, and the tiles' shared rows come from their XCD's L2.
// Each of four waves owns 16 rows of the outputs and a part of the state's
// rows.  The scores are formed transposed, Y X^T, so that their accumulators
// are the second product's operand as they stand; the state's accumulators
// are the third's, and go round through LDS once a chunk because each wave
// needs all of them.  A fifth wave copies the chunks to LDS, and one barrier
// a chunk hands them and the state over.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "gdn_checks.h"
#include "gdn_device.h"
#include "gdn_linear.h"

namespace {

constexpr int C = 64;    // rows of a chunk
constexpr int ZT = 32;   // state columns of a workgroup
constexpr int NWC = 4;   // computing waves

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
  int B, T, H, nrole, tiles;
  int segc;           // chunks of a segment; 0: nothing is cut
  int nslot;          // segment slots: of a dense sequence, or of the packed batch
};

template <typename TI, int DX>
struct LK {
  using Frag = typename Mma<TI>::frag;
  static constexpr bool B16 = sizeof(TI) == 2;
  static constexpr int ES = sizeof(TI), SLAB = Mma<TI>::SLAB, E = Mma<TI>::E;
  static constexpr int GR = DX * ES / 16, ZGR = ZT * ES / 16;  // 16-byte granules of a row
  static constexpr int NS = DX / SLAB, NJS = C / SLAB;
  static constexpr int YB = C * DX * ES, ZB = C * ZT * ES, MB = NS * 2 * 1024;
  static constexpr int Y_INS = YB / 1024, Z_INS = ZB / 1024;
  static constexpr int NBUF = 3 * (YB + ZB) + 2 * MB <= 80 * 1024 ? 3 : 2;
  // State tiles of a wave: SPW slabs of x rows, ZPW 16-column blocks, TPS
  // accumulators a slab.
  static constexpr int SPW = NS >= 4 ? NS / 4 : 1, ZPW = NS >= 4 ? 2 : 1, TPS = SLAB / 16;
  static constexpr int NU = SPW * ZPW * TPS;
  __device__ static inline int slab_of(int w, int i) { return NS >= 4 ? w * SPW + i : (NS == 2 ? w >> 1 : 0); }
  __device__ static inline int zb_of(int w, int i) { return NS >= 4 ? i : w & 1; }
  __device__ static inline bool has_state(int w) { return NS > 1 || w < 2; }
  // Accumulator row 4 q + e of state tile t of a slab: with two tiles a slab
  // a lane's eight rows are neighbours, as a fragment wants them.
  __device__ static inline int x_of(int t, int q) { return B16 ? 8 * q + 4 * t : 4 * q; }
  // State column of MFMA row or column m of block zb: a lane's output columns are neighbours.
  __device__ static inline int z_of(int zb, int m) { return B16 ? 8 * (m >> 2) + 4 * zb + (m & 3) : 16 * zb + m; }
  __device__ static inline int swz_y(int r) { return swz_kq<GR>(r); }
  __device__ static inline int swz_z(int r) { return B16 ? (r >> 1) & 3 : 0; }
};

// exp(n g), and what its rounding to 32 bits leaves: a constant factor's
// rounding would add up over the chunks, always to the same side.
struct Pow {
  float hi, lo;
};
__device__ static inline Pow split_pow(double d) {
  const float hi = (float)d;
  return {hi, d > 1e-30 && d < 1e30 ? (float)(d - (double)hi) : 0.f};
}
__device__ static inline double pow_of(float g, long n) { return n == 0 ? 1.0 : exp((double)g * (double)n); }
__device__ static inline f32x4 decayed(f32x4 m, Pow a) {
  f32x4 r;
#pragma unroll
  for (int e = 0; e < 4; ++e) r[e] = __builtin_fmaf(a.hi, m[e], a.lo * m[e]);
  return r;
}

template <typename V>
__device__ static inline V buf_load16(__amdgpu_buffer_rsrc_t r, int off) {
  return __builtin_bit_cast(V, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}

// PASS 0: outputs (and end states); PASS 1: the end states of the segments
// that others follow, each from zero (a sequence's first from S0).
template <typename TI, int DX, int PASS>
__global__ __launch_bounds__(64 * (NWC + 1)) void linear_kernel(const LinParams p) {
  using K = LK<TI, DX>;
  using Frag = typename K::Frag;
  __shared__ __attribute__((aligned(16))) char sY[K::NBUF * K::YB];
  __shared__ __attribute__((aligned(16))) char sZ[K::NBUF * K::ZB];
  __shared__ __attribute__((aligned(16))) char sM[PASS == 0 ? 2 * K::MB : 16];
  __shared__ double sPow[C + 1];
  __shared__ int sSeq;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int H = p.H, DZ = p.tiles * ZT;

  // ---- which chain, segment, role and tile
  const int item = xcd_remap(blockIdx.x, gridDim.x);
  const int tile = item % p.tiles, ri = item / p.tiles % p.nrole;
  const int sh = item / p.tiles / p.nrole, h = sh % H, slot = sh / H;
  const Role role = p.role[ri];
  int n, seg;
  if (!p.cu || p.segc == 0) {
    const int per = p.segc ? p.nslot : 1;
    n = slot / per;
    seg = slot % per;
  } else {
    // Packed and cut: sequence n has slots floor(begin / rows of a segment) + n and on.
    if (tid == 0) sSeq = -1;
    __syncthreads();
    const int rows = p.segc * C;
    for (int i = tid; i < p.B; i += 64 * (NWC + 1)) {
      const int b = min(max(p.cu[i], 0), p.T), e = min(max(p.cu[i + 1], b), p.T);
      const int first = b / rows + i, count = max(1, (e - b + rows - 1) / rows);
      if (slot >= first && slot < first + count) sSeq = i;
    }
    __syncthreads();
    n = sSeq;
    if (n < 0) return;
    seg = slot - (min(max(p.cu[n], 0), p.T) / rows + n);
  }
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
  const int nch = (len + C - 1) / C;
  const int c0 = seg * p.segc, c1 = p.segc ? min(nch, c0 + p.segc) : nch;
  if (seg > 0 && c0 >= nch) return;
  if (PASS == 1 && c1 >= nch) return;  // nothing follows

  const float gh = p.g[h];
  if (tid <= C) sPow[tid] = pow_of(gh, tid);
  __syncthreads();

  const long th0 = row0 * H + h;  // token-head of the sequence's first row
  const int rev = role.reverse;
  const int x_stride = H * DX * K::ES, z_stride = H * DZ * K::ES;

  if (wave == NWC) {
    // ------------------------------------------------------------- loader --
    const __amdgpu_buffer_rsrc_t ry = make_rsrc(role.y + th0 * DX * K::ES, (long)(len - 1) * x_stride + DX * K::ES);
    const __amdgpu_buffer_rsrc_t rz =
        make_rsrc(role.z + (th0 * DZ + tile * ZT) * K::ES, (long)(len - 1) * z_stride + ZT * K::ES);
    int y_off[K::Y_INS], z_off[K::Z_INS];
#pragma unroll
    for (int i = 0; i < K::Y_INS; ++i) {
      const int G = i * 64 + lane, r = G / K::GR;
      y_off[i] = (rev ? -r : r) * x_stride + ((G % K::GR) ^ K::swz_y(r)) * 16;
    }
#pragma unroll
    for (int i = 0; i < K::Z_INS; ++i) {
      const int G = i * 64 + lane, r = G / K::ZGR;
      z_off[i] = (rev ? -r : r) * z_stride + ((G % K::ZGR) ^ K::swz_z(r)) * 16;
    }
    // Rows outside the sequence lie outside the descriptors (a negative
    // offset wraps far behind them) and read as zeros; so do the chunks
    // behind the last, asked for to keep the count of copies even.
    auto issue = [&](int c) {
      const int s = (c - c0) % K::NBUF;
      const unsigned at = rev ? (unsigned)(len - 1) - (unsigned)c * C : (unsigned)c * C;
      const unsigned ya = at * (unsigned)x_stride, za = at * (unsigned)z_stride;
#pragma unroll
      for (int i = 0; i < K::Y_INS; ++i)
        copy_to_lds(ry, sY + s * K::YB + i * 1024, c < c1 ? (int)(ya + (unsigned)y_off[i]) : -16);
#pragma unroll
      for (int i = 0; i < K::Z_INS; ++i)
        copy_to_lds(rz, sZ + s * K::ZB + i * 1024, c < c1 ? (int)(za + (unsigned)z_off[i]) : -16);
    };
    constexpr int INS = K::Y_INS + K::Z_INS;
    if (c0 < c1) {
#pragma unroll
      for (int i = 0; i < K::NBUF - 1; ++i) issue(c0 + i);
      __builtin_amdgcn_s_waitcnt(waitcnt_vm((K::NBUF - 2) * INS));
    }
    lds_barrier();
    for (int c = c0; c < c1; ++c) {
      issue(c + K::NBUF - 1);
      __builtin_amdgcn_s_waitcnt(waitcnt_vm((K::NBUF - 2) * INS));
      lds_barrier();
    }
    return;
  }

  // ----------------------------------------------------------- computing --
  const int w = wave, m16 = lane & 15, q4 = lane >> 4;
  const int off = rev;  // the state's powers are one lower backwards, the inputs' one higher

  // The state.
  f32x4 M[K::NU];
#pragma unroll
  for (int u = 0; u < K::NU; ++u) M[u] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto at_state = [&](int u, int e, int& x, int& z) {
    const int si = u / (K::ZPW * K::TPS), zi = u / K::TPS % K::ZPW, t = u % K::TPS;
    x = K::slab_of(w, si) * K::SLAB + K::x_of(t, q4) + e;
    z = tile * ZT + K::z_of(K::zb_of(w, zi), m16);
  };
  const bool has = K::has_state(w);
  auto load_s0 = [&]() {
    const float* s0 = role.s0 + ((long)n * H + h) * DX * DZ;
#pragma unroll
    for (int u = 0; u < K::NU; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        int x, z;
        at_state(u, e, x, z);
        M[u][e] = s0[role.s0_transposed ? z * DX + x : x * DZ + z];
      }
  };
  auto ws_at = [&](int sl) { return p.ws + ((((long)sl * H + h) * p.nrole + ri) * p.tiles + tile) * (DX * ZT / 4); };
  if (has) {
    if (seg == 0) {
      if (role.s0) load_s0();
    } else if (PASS == 0) {
      const Pow step = split_pow(pow_of(gh, (long)p.segc * C));
      for (int s = slot - seg; s < slot; ++s) {
        const f32x4* src = ws_at(s) + w * 64 * K::NU + lane;
#pragma unroll
        for (int u = 0; u < K::NU; ++u) M[u] = decayed(M[u], step) + src[u * 64];
      }
    }
  }
  auto publish = [&](int buf) {
    if (!has) return;
#pragma unroll
    for (int si = 0; si < K::SPW; ++si)
#pragma unroll
      for (int zi = 0; zi < K::ZPW; ++zi) {
        const int u = (si * K::ZPW + zi) * K::TPS;
        lds_st(sM + buf * K::MB, ((K::slab_of(w, si) * 2 + K::zb_of(w, zi)) * 64 + lane) * 16,
               Mma<TI>::from_acc(M[u], M[u + K::TPS - 1]));
      }
  };

  // Powers of the decay: the scores' (row i = 16 w + m16, column j = 16 jb +
  // 4 q4 + e), the state's at row i, the inputs' at row j.
  f32x4 D[4], W[4];
  float gam = 0.f;
  auto input_powers = [&](int rows) {
#pragma unroll
    for (int jb = 0; jb < 4; ++jb)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int d = rows - 1 - (16 * jb + 4 * q4 + e) + off;
        W[jb][e] = d >= 0 ? (float)sPow[d] : 0.f;
      }
  };
  if constexpr (PASS == 0) {
#pragma unroll
    for (int jb = 0; jb < 4; ++jb)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int d = 16 * (w - jb) + m16 - 4 * q4 - e;
        D[jb][e] = d >= 0 ? (float)sPow[d] : 0.f;
      }
    gam = (float)sPow[16 * w + m16 + 1 - off];
  }
  input_powers(C);
  Pow step = split_pow(sPow[C]);

  const __amdgpu_buffer_rsrc_t rx = make_rsrc(role.x + th0 * DX * K::ES, (long)(len - 1) * x_stride + DX * K::ES);
  const __amdgpu_buffer_rsrc_t ro =
      make_rsrc(role.out + (th0 * DZ + tile * ZT) * K::ES, (long)(len - 1) * z_stride + ZT * K::ES);
  auto row_of = [&](int c) {
    const unsigned i = (unsigned)c * C + 16 * w + m16;
    return rev ? (unsigned)(len - 1) - i : i;
  };
  Frag X[K::NS], Xn[K::NS];
  auto load_x = [&](int c, Frag* x) {
    const unsigned r = row_of(c) * (unsigned)x_stride + K::E * K::ES * q4;
#pragma unroll
    for (int s = 0; s < K::NS; ++s) x[s] = buf_load16<Frag>(rx, (int)(r + s * K::SLAB * K::ES));
  };
  if constexpr (PASS == 0) {
    if (c0 < c1) load_x(c0, X);
    publish(0);
  }
  lds_barrier();

  for (int c = c0; c < c1; ++c) {
    const char* bY = sY + (c - c0) % K::NBUF * K::YB;
    const char* bZ = sZ + (c - c0) % K::NBUF * K::ZB;
    if (PASS == 0 && c + 1 < c1) load_x(c + 1, Xn);

    // z columns as fragments over the rows (for two 16-row blocks: rows 4 q4
    // and on of the first, then of the second, as the scores' accumulators lie)
    Frag Zf[2][K::NJS];
#pragma unroll
    for (int zb = 0; zb < 2; ++zb)
#pragma unroll
      for (int js = 0; js < K::NJS; ++js) {
        if constexpr (K::B16) {
          const int r = 32 * js + 4 * q4 + (m16 >> 2), g = m16 & 3;
          const bf16x4 lo = lds_read_tr(bZ, r * 64 + ((g ^ K::swz_z(r)) * 16) + 8 * zb);
          const bf16x4 hi = lds_read_tr(bZ, (r + 16) * 64 + ((g ^ K::swz_z(r + 16)) * 16) + 8 * zb);
          Zf[zb][js] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            Zf[zb][js][e] = lds_ld<float>(bZ, ((16 * js + 4 * q4 + e) * ZT + K::z_of(zb, m16)) * 4);
        }
      }

    if constexpr (PASS == 0) {
      // scores, transposed and masked
      f32x4 P[4];
#pragma unroll
      for (int jb = 0; jb < 4; ++jb) {
        P[jb] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (jb <= w) {
          const int r = 16 * jb + m16;
#pragma unroll
          for (int s = 0; s < K::NS; ++s) {
            const Frag y = lds_ld<Frag>(bY, r * (K::GR * 16) + (((K::SLAB * K::ES / 16) * s + q4) ^ K::swz_y(r)) * 16);
            P[jb] = Mma<TI>::mma(y, X[s], P[jb]);
          }
          P[jb] *= D[jb];
        }
      }
      // outputs, transposed: the state's part, then the chunk's own
      f32x4 O[2];
      const char* bM = sM + ((c - c0) & 1) * K::MB;
#pragma unroll
      for (int zb = 0; zb < 2; ++zb) {
        O[zb] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < K::NS; ++s)
          O[zb] = Mma<TI>::mma(lds_ld<Frag>(bM, ((s * 2 + zb) * 64 + lane) * 16), X[s], O[zb]);
        O[zb] *= gam;
#pragma unroll
        for (int js = 0; js < K::NJS; ++js)
          if (js * K::TPS <= w)
            O[zb] = Mma<TI>::mma(Zf[zb][js], Mma<TI>::from_acc(P[js * K::TPS], P[js * K::TPS + K::TPS - 1]), O[zb]);
      }
      const unsigned at = row_of(c) * (unsigned)z_stride;
      if constexpr (K::B16) {
        const u32x2 lo = __builtin_bit_cast(u32x2, cvt4(O[0])), hi = __builtin_bit_cast(u32x2, cvt4(O[1]));
        __builtin_amdgcn_raw_buffer_store_b128(u32x4{lo[0], lo[1], hi[0], hi[1]}, ro, (int)(at + 16 * q4), 0, 0);
      } else {
#pragma unroll
        for (int zb = 0; zb < 2; ++zb)
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, O[zb]), ro, (int)(at + 64 * zb + 16 * q4),
                                                 0, 0);
      }
    }

    // the state: decayed rows y z^T; in 16-bit storage the decayed z are taken as two terms
    if (has) {
      const int rows = len - c * C;
      if (rows < C) {  // the last chunk
        input_powers(rows);
        step = split_pow(sPow[rows]);
      }
#pragma unroll
      for (int u = 0; u < K::NU; ++u) M[u] = decayed(M[u], step);
      Frag Zh[K::ZPW][K::NJS], Zl[K::ZPW][K::NJS];
#pragma unroll
      for (int zi = 0; zi < K::ZPW; ++zi)
#pragma unroll
        for (int js = 0; js < K::NJS; ++js) {
          Frag zf = Zf[zi][js];
          if constexpr (K::ZPW == 1) {
#pragma unroll
            for (int e = 0; e < K::E; ++e) zf[e] = K::zb_of(w, 0) ? Zf[1][js][e] : Zf[0][js][e];
          }
          if constexpr (K::B16) {
            f32x4 a, b;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              a[e] = (float)zf[e] * W[2 * js][e];
              b[e] = (float)zf[4 + e] * W[2 * js + 1][e];
            }
            Zh[zi][js] = Mma<TI>::from_acc(a, b);
            f32x4 ra, rb;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              ra[e] = a[e] - (float)Zh[zi][js][e];
              rb[e] = b[e] - (float)Zh[zi][js][4 + e];
            }
            Zl[zi][js] = Mma<TI>::from_acc(ra, rb);
          } else {
            Zh[zi][js] = zf * W[js];
          }
        }
#pragma unroll
      for (int si = 0; si < K::SPW; ++si)
#pragma unroll
        for (int t = 0; t < K::TPS; ++t)
#pragma unroll
          for (int js = 0; js < K::NJS; ++js) {
            Frag y;
            if constexpr (K::B16) {
              const int r = 32 * js + 4 * q4 + (m16 >> 2), g = 4 * K::slab_of(w, si) + (m16 & 3);
              const bf16x4 lo = lds_read_tr(bY, r * (K::GR * 16) + ((g ^ K::swz_y(r)) * 16) + 8 * t);
              const bf16x4 hi = lds_read_tr(bY, (r + 16) * (K::GR * 16) + ((g ^ K::swz_y(r + 16)) * 16) + 8 * t);
              y = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
            } else {
              const int x = K::slab_of(w, si) * 16 + m16;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int r = 16 * js + 4 * q4 + e;
                y[e] = lds_ld<float>(bY, r * (K::GR * 16) + (((x >> 2) ^ K::swz_y(r)) * 16) + (x & 3) * 4);
              }
            }
#pragma unroll
            for (int zi = 0; zi < K::ZPW; ++zi) {
              const int u = (si * K::ZPW + zi) * K::TPS + t;
              M[u] = Mma<TI>::mma(y, Zh[zi][js], M[u]);
              if constexpr (K::B16) M[u] = Mma<TI>::mma(y, Zl[zi][js], M[u]);
            }
          }
    }
    if constexpr (PASS == 0) {
      publish((c - c0 + 1) & 1);
#pragma unroll
      for (int s = 0; s < K::NS; ++s) X[s] = Xn[s];
    }
    lds_barrier();
  }

  if (!has) return;
  if constexpr (PASS == 1) {
    f32x4* dst = ws_at(slot) + w * 64 * K::NU + lane;
#pragma unroll
    for (int u = 0; u < K::NU; ++u) dst[u * 64] = M[u];
  } else if (role.sT && c1 >= nch) {
    float* sT = role.sT + ((long)n * H + h) * DX * DZ;
#pragma unroll
    for (int u = 0; u < K::NU; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        int x, z;
        at_state(u, e, x, z);
        sT[x * DZ + z] = M[u][e];
      }
  }
}

// ------------------------------------------------------------------- host --

// Where a batch has fewer workgroups than the device has compute units, its
// sequences are cut into segments whose states a first launch forms.
constexpr int CUS = 256;      // of an MI355X
constexpr int SEG_MIN = 8;    // chunks a segment has at least

int segment_chunks(int B, int T, int H, int dz, int roles) {
  const long items = (long)B * H * (dz / ZT) * roles;
  const int nch = (int)(((long)T + C - 1) / C);
  if (items <= 0 || items >= CUS || nch < 2 * SEG_MIN) return 0;
  const int want = (int)std::min<long>((2 * CUS + items - 1) / items, nch / SEG_MIN);
  return want > 1 ? (nch + want - 1) / want : 0;
}

long segment_slots(int B, int T, bool packed, int segc) {
  if (!segc) return B;
  if (packed) return T / ((long)segc * C) + B;
  return (long)B * ((((long)T + C - 1) / C + segc - 1) / segc);
}

template <typename TI, int DX>
int launch_dx(LinParams p, hipStream_t s) {
  const long slots = segment_slots(p.B, p.T, p.cu != nullptr, p.segc);
  p.nslot = p.segc && !p.cu ? (int)(slots / p.B) : 1;
  const long wgs = slots * p.H * p.nrole * p.tiles;
  if (wgs <= 0) return GDN_OK;
  if (wgs >= 1L << 23) return GDN_ERR_INVALID_ARG;
  const dim3 grid((unsigned)wgs), block(64 * (NWC + 1));
  if (p.segc) {
    hipLaunchKernelGGL((linear_kernel<TI, DX, 1>), grid, block, 0, s, p);
    if (hipGetLastError() != hipSuccess) return GDN_ERR_LAUNCH;
  }
  hipLaunchKernelGGL((linear_kernel<TI, DX, 0>), grid, block, 0, s, p);
  return hipGetLastError() == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}

int launch(const LinParams& p, int dx, int dtype, hipStream_t s) {
  const bool b16 = dtype == GDN_BF16;
  switch (dx) {
    case 32: return b16 ? launch_dx<__bf16, 32>(p, s) : launch_dx<float, 32>(p, s);
    case 64: return b16 ? launch_dx<__bf16, 64>(p, s) : launch_dx<float, 64>(p, s);
    default: return b16 ? launch_dx<__bf16, 128>(p, s) : launch_dx<float, 128>(p, s);
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
Plan plan(int B, int T, int H, int dx, int dz, int roles, bool packed) {
  const int segc = segment_chunks(B, T, H, dz, roles);
  if (!segc) return {0, 0};
  return {segc, segment_slots(B, T, packed, segc) * H * roles * dx * dz * 4LL};
}

}  // namespace

extern "C" long long gdn_linear_workspace_size(int B, int T, int H, int dk, int dv, int packed, int dtype,
                                               int backward) {
  const int rc = check_sizes(B, T, H, dk, dv, packed != 0, dtype);
  if (rc != GDN_OK) return rc;
  if (!backward) return plan(B, T, H, dk, dv, 1, packed != 0).bytes;
  if (dk == dv) return plan(B, T, H, dk, dv, 3, packed != 0).bytes;
  return plan(B, T, H, dv, dk, 2, packed != 0).bytes + plan(B, T, H, dk, dv, 1, packed != 0).bytes;
}

extern "C" int gdn_linear_fwd(const void* q, const void* k, const void* v, const float* g, const float* h0,
                              const int32_t* cu_seqlens, void* out, float* hT, int B, int T, int H, int dk, int dv,
                              void* stream, int dtype, void* workspace, long long workspace_bytes) {
  const bool packed = cu_seqlens != nullptr;
  const int rc = check_sizes(B, T, H, dk, dv, packed, dtype);
  if (rc != GDN_OK) return rc;
  if (B > 0 && (!g || !hT || (T > 0 && (!q || !k || !v || !out)))) return GDN_ERR_INVALID_ARG;
  Plan pl = plan(B, T, H, dk, dv, 1, packed);
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
  p.tiles = dv / ZT;
  p.segc = pl.segc;
  return launch(p, dk, dtype, static_cast<hipStream_t>(stream));
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
    p.tiles = dv_ / ZT;
    p.segc = plan(B, T, H, dk_, dv_, 3, packed).segc;
    return launch(p, dk_, dtype, s);
  }
  const Plan first = plan(B, T, H, dv_, dk_, 2, packed);
  const bool fits = dk_ != dv_;  // the workspace of equal widths is that of one launch: leave these two uncut
  p.role[0] = rq;
  p.role[1] = rk;
  p.nrole = 2;
  p.tiles = dk_ / ZT;
  p.segc = fits ? first.segc : 0;
  const int rc2 = launch(p, dv_, dtype, s);
  if (rc2 != GDN_OK) return rc2;
  p.role[0] = rv;
  p.nrole = 1;
  p.tiles = dv_ / ZT;
  p.segc = fits && !in_place ? plan(B, T, H, dk_, dv_, 1, packed).segc : 0;
  p.ws = reinterpret_cast<f32x4*>(static_cast<char*>(workspace) + (fits ? first.bytes : 0));
  return launch(p, dk_, dtype, s);
}

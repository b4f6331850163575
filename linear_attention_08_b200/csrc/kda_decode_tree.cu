// KDA outputs of a tree of drafted tokens over a recurrent state (sm_100a).
//
// Place t of a tree follows place par(t) < t, or the committed state S0.  The
// recurrence along a token's path is one chunk of the chunked form ("LLM -
// Semianalysis, Kimi K3 아키텍처" (charstring.tistory.com/2557), Methods 1)
// whose causal mask "s <= t" becomes "s is t or an ancestor of t" (s ~ t):
//
//   Gam_t = Gam_par(t) + g_t                                  (per key channel)
//   Kt_t = exp(Gam_t) k_t,  Qt_t = exp(Gam_t) q_t,  Kh_s = exp(-Gam_s) k_s
//   L_ts = beta_t Kt_t . Kh_s  (s ~ t, s != t),   P_ts = Qt_t . Kh_s  (s ~ t)
//   (I + L) Vn = Diag(beta) (V - Kt S0)
//   O = Qt S0 + P Vn
//
// L and P are the gated products with exp(Gam_t - Gam_s), which is at most one;
// the factors exp(-Gam_s) alone are not, so a unit whose Kh leaves 10^36 or whose
// Gam leaves +-80 forms L and P pair by pair from the differences instead.
//
// Layout: one CTA per (sequence, head).  Everything is computed transposed,
// O^T = S0^T Qt^T + Vn^T P^T, with value columns as the rows of m16n8k8 products:
//   - the A operand S0^T comes straight from the row-major FP32 state in HBM into
//     the registers of the warp that owns the columns (a lane reads float4s of
//     four columns; which tile row a column is and which k index a state row is
//     are free choices), no shared memory, no transposition;
//   - the accumulators of Kt S0 have the layout of an A operand, so V - Kt S0, Vn
//     and the outputs stay in registers from the first product to the store.
// Shared memory holds the token rows (Kt, Qt, Kh) and the T x T matrices.  The
// contractions are small and the state crosses HBM once, so the kernel is bound
// by memory; the warp-level products need no tensor-memory round trip per unit
// and no staging of the state, which the 5th-generation tile products (operands
// in shared memory, accumulators in tensor memory) would.
//
// Arithmetic: TF32 products with FP32 accumulation for BF16 inputs (operands are
// rounded to nearest, 2^-12 of a value, against 2^-9 when out is rounded).  FP32
// inputs split each operand in two TF32 terms and add three products, and carry
// Gam as an unevaluated sum of two FP32 numbers, for FP32 accuracy.
#include "kda_common.cuh"

namespace kda {
namespace {

constexpr int kMaxNodes = 64;
constexpr float kGamLimit = 80.f;
constexpr float kFactorLimit = 1e36f;

__device__ __forceinline__ uint32_t tf32_rn(float x) {
  uint32_t r;
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
  return r;
}

// One operand value: rounded to TF32, and for X3 what the rounding left.
template <bool X3> struct Op {
  uint32_t hi, lo;
  __device__ __forceinline__ Op() {}
  __device__ __forceinline__ explicit Op(float x) {
    hi = tf32_rn(x);
    if (X3) lo = tf32_rn(x - __uint_as_float(hi));
  }
};

__device__ __forceinline__ void mma_raw(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <bool X3>
__device__ __forceinline__ void mma(float (&c)[4], const Op<X3> &a0, const Op<X3> &a1,
                                    const Op<X3> &a2, const Op<X3> &a3, const Op<X3> &b0,
                                    const Op<X3> &b1) {
  if (X3) {
    mma_raw(c, a0.lo, a1.lo, a2.lo, a3.lo, b0.hi, b1.hi);
    mma_raw(c, a0.hi, a1.hi, a2.hi, a3.hi, b0.lo, b1.lo);
  }
  mma_raw(c, a0.hi, a1.hi, a2.hi, a3.hi, b0.hi, b1.hi);
}

// Position of key channel c in a token row: the four channels 4 m + j (m = 0..3)
// of a group of 16 that lane j of a quad needs lie side by side.
__device__ __forceinline__ int spot(int c) { return (c & ~15) | ((c & 3) << 2) | ((c >> 2) & 3); }

// E consecutive elements as floats (2 or 4).
template <int E> __device__ __forceinline__ void load_row(const __nv_bfloat16 *p, float *x) {
  uint32_t w[E / 2];
  if (E == 4) {
    const uint2 u = __ldg(reinterpret_cast<const uint2 *>(p));
    w[0] = u.x;
    w[E / 2 - 1] = u.y;
  } else {
    w[0] = __ldg(reinterpret_cast<const uint32_t *>(p));
  }
#pragma unroll
  for (int i = 0; i < E / 2; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <int E> __device__ __forceinline__ void load_row(const float *p, float *x) {
  if (E == 4) {
    const float4 u = __ldg(reinterpret_cast<const float4 *>(p));
    x[0] = u.x; x[1] = u.y; x[E - 2] = u.z; x[E - 1] = u.w;
  } else {
    const float2 u = __ldg(reinterpret_cast<const float2 *>(p));
    x[0] = u.x; x[1] = u.y;
  }
}
template <int E> __device__ __forceinline__ void store_row(__nv_bfloat16 *p, const float *x) {
  uint32_t w[E / 2];
#pragma unroll
  for (int i = 0; i < E / 2; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&b);
  }
  if (E == 4) *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[E / 2 - 1]);
  else *reinterpret_cast<uint32_t *>(p) = w[0];
}
template <int E> __device__ __forceinline__ void store_row(float *p, const float *x) {
  if (E == 4) *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[E - 2], x[E - 1]);
  else *reinterpret_cast<float2 *>(p) = make_float2(x[0], x[1]);
}

// NT: tiles of 8 places (places past T are empty ones).
template <int DK, int DV, int NT, typename TIn> struct TreeCfg {
  static constexpr bool X3 = sizeof(TIn) == 4;
  static constexpr int MT = NT == 8 || X3 ? 1 : 2;  // 16-column tiles per warp (registers)
  static constexpr int E = 2 * MT;                  // value columns per lane
  static constexpr int WARPS = DV / (16 * MT);
  static constexpr int THREADS = 32 * WARPS;
  static constexpr int T8 = 8 * NT;
  static constexpr int NB = NT < 2 ? 1 : NT / 2;    // diagonal blocks
  static constexpr int BT = NT < 2 ? 1 : 2;         // tiles per diagonal block
  static constexpr int LDK = DK + 16;               // 16-byte reads of 8 rows: distinct banks
  static constexpr int LDT = T8 + (T8 == 8 ? 0 : 8);   // = 8 or 24 modulo 32: 8-byte reads
  static constexpr int LDB = 8 * BT + (BT == 1 ? 0 : 8);
  // shared memory, in floats
  static constexpr int KT = 0, QT = KT + T8 * LDK, KH = QT + T8 * LDK;
  static constexpr int LM = KH + T8 * LDK, PM = LM + T8 * LDT;
  static constexpr int MI = PM + T8 * LDT;          // (I + L)^-1 of the diagonal blocks
  static constexpr int BE = MI + NB * 8 * BT * LDB;
  static constexpr int TOTAL = BE + T8;
  static constexpr size_t BYTES = (size_t)TOTAL * 4;
};

template <int DK, int DV, int NT, typename TIn>
__global__ void __launch_bounds__(TreeCfg<DK, DV, NT, TIn>::THREADS)
decode_tree_kernel(const TIn *__restrict__ q, const TIn *__restrict__ k,
                   const TIn *__restrict__ v, const float *__restrict__ g,
                   const float *__restrict__ beta, const float *__restrict__ state,
                   const int32_t *__restrict__ parents, TIn *__restrict__ out, int T, int H) {
  using Cfg = TreeCfg<DK, DV, NT, TIn>;
  constexpr bool X3 = Cfg::X3;
  constexpr int MT = Cfg::MT, E = Cfg::E, T8 = Cfg::T8, LDK = Cfg::LDK, LDT = Cfg::LDT;
  constexpr int LDB = Cfg::LDB, BT = Cfg::BT, NB = Cfg::NB, THREADS = Cfg::THREADS;
  extern __shared__ __align__(16) float sm[];
  float *s_kt = sm + Cfg::KT, *s_qt = sm + Cfg::QT, *s_kh = sm + Cfg::KH;
  float *s_L = sm + Cfg::LM, *s_P = sm + Cfg::PM, *s_M = sm + Cfg::MI, *s_beta = sm + Cfg::BE;
  __shared__ unsigned long long s_anc[kMaxNodes];   // ancestors and self; 0: an empty place
  __shared__ int s_par[kMaxNodes], s_jump[kMaxNodes];

  const int64_t unit = blockIdx.x;
  const int n = (int)(unit / H), h = (int)(unit % H);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gid = lane >> 2, j = lane & 3;
  const int64_t row0 = (int64_t)n * T * H + h;      // token t is row row0 + t H

  // ---- the state's columns of this warp: rows 4 m + j, columns col .. col + E - 1 ----
  const int col = 16 * MT * warp + E * gid;
  float s0[DK / 4][E];
  {
    const float *src = state + unit * (DK * DV) + (int64_t)j * DV + col;
#pragma unroll
    for (int m = 0; m < DK / 4; ++m) {
      if (E == 4)
        asm volatile("ld.global.cs.v4.f32 {%0,%1,%2,%3}, [%4];"
                     : "=f"(s0[m][0]), "=f"(s0[m][1]), "=f"(s0[m][E - 2]), "=f"(s0[m][E - 1])
                     : "l"(src + m * 4 * DV));
      else
        asm volatile("ld.global.cs.v2.f32 {%0,%1}, [%2];"
                     : "=f"(s0[m][0]), "=f"(s0[m][1])
                     : "l"(src + m * 4 * DV));
    }
  }

  // ---- ancestors by pointer doubling (one warp) ----
  if (warp == 0) {
    for (int t = lane; t < kMaxNodes; t += 32) {
      int up = -2;
      if (t < T) up = parents ? parents[(int64_t)n * T + t] : t - 1;
      if (up < -1 || up >= t) up = -2;
      s_par[t] = up;
      s_jump[t] = up;
      s_anc[t] = 1ull << t;
    }
    __syncwarp();
    // after the step of size d every mask holds the last 2 d places of its path
    for (int d = 1; d < T; d <<= 1) {
      unsigned long long m[2];
      int up[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int t = lane + 32 * e, a = s_jump[t];
        m[e] = s_anc[t] | (a >= 0 ? s_anc[a] : 0ull);
        up[e] = a >= 0 ? s_jump[a] : a;
      }
      __syncwarp();
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        s_anc[lane + 32 * e] = m[e];
        s_jump[lane + 32 * e] = up[e];
      }
      __syncwarp();
    }
    for (int t = lane; t < kMaxNodes; t += 32)      // a path that ends in an empty place
      if (s_jump[t] != -1) s_anc[t] = 0;
    for (int t = lane; t < T8; t += 32)
      s_beta[t] = t < T && s_anc[t] != 0 ? beta[row0 + (int64_t)t * H] : 0.f;
  }
  __syncthreads();

  // ---- Gam along the paths; Kt, Qt, Kh ----
  bool wide = false;   // factors out of range: L and P pair by pair
  for (int c = tid; c < DK; c += THREADS) {
    const int p = spot(c);
    constexpr int U = 8;
    float gam = 0.f, low = 0.f;          // of the place before, kept for chains
    for (int t0 = 0; t0 < T8; t0 += U) {
      float gv[U], kv[U], qv[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int t = t0 + i;
        gv[i] = kv[i] = qv[i] = 0.f;
        if (t < T) {
          const int64_t at = (row0 + (int64_t)t * H) * DK + c;
          gv[i] = __ldg(g + at);
          kv[i] = to_f32(k[at]);
          qv[i] = to_f32(q[at]);
        }
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int t = t0 + i, up = s_par[t];
        const bool live = s_anc[t] != 0;
        float b = 0.f, bl = 0.f;
        if (up == t - 1 && t > 0) {
          b = gam;
          bl = low;
        } else if (up >= 0) {
          // until every place has been reached, Kh's rows hold Gam (and Qt's its low part)
          b = s_kh[up * LDK + p];
          if (X3) bl = s_qt[up * LDK + p];
        }
        const float gt = live ? gv[i] : 0.f;
        gam = b + gt;
        if (X3) {   // two-sum: the rounding of b + g_t
          const float z = gam - b;
          low = bl + ((b - (gam - z)) + (gt - z));
        }
        s_kh[t * LDK + p] = gam;
        if (X3) s_qt[t * LDK + p] = low;
        s_kt[t * LDK + p] = live ? kv[i] : 0.f;
        if (!X3) s_qt[t * LDK + p] = live ? qv[i] : 0.f;
      }
    }
    for (int t = 0; t < T8; ++t) {
      const float G = s_kh[t * LDK + p], kc = s_kt[t * LDK + p];
      float down, up, qc;
      if (X3) {
        const float lo = s_qt[t * LDK + p];
        qc = t < T && s_anc[t] != 0 ? to_f32(q[(row0 + (int64_t)t * H) * DK + c]) : 0.f;
        down = expf(G);
        down += down * lo;
        up = expf(-G);
        up -= up * lo;
      } else {
        qc = s_qt[t * LDK + p];
        down = __expf(G);
        up = __expf(-G);
      }
      const float kt = kc * down, qt = qc * down, kh = kc * up;
      wide |= !(fabsf(kh) < kFactorLimit) || !(fabsf(G) <= kGamLimit);
      s_kt[t * LDK + p] = X3 ? kt : __uint_as_float(tf32_rn(kt));
      s_qt[t * LDK + p] = X3 ? qt : __uint_as_float(tf32_rn(qt));
      s_kh[t * LDK + p] = X3 ? kh : __uint_as_float(tf32_rn(kh));
    }
  }
  wide = __syncthreads_or(wide);

  // ---- L and P: tile (a, b) of 8 x 8 places, rows Kt and Qt of one tile in one product ----
  if (!wide) {
    for (int tile = warp; tile < NT * (NT + 1) / 2; tile += Cfg::WARPS) {
      int a = 0;
      while ((a + 1) * (a + 2) / 2 <= tile) ++a;
      const int b = tile - a * (a + 1) / 2;
      float c[4] = {0.f, 0.f, 0.f, 0.f}, c2[4] = {0.f, 0.f, 0.f, 0.f};
      const float *pk = s_kt + (8 * a + gid) * LDK + 4 * j;
      const float *pq = s_qt + (8 * a + gid) * LDK + 4 * j;
      const float *ph = s_kh + (8 * b + gid) * LDK + 4 * j;
#pragma unroll
      for (int i = 0; i < DK / 16; ++i) {
        const float4 x = *reinterpret_cast<const float4 *>(pk + 16 * i);
        const float4 y = *reinterpret_cast<const float4 *>(pq + 16 * i);
        const float4 z = *reinterpret_cast<const float4 *>(ph + 16 * i);
        mma<X3>(c, Op<X3>(x.x), Op<X3>(y.x), Op<X3>(x.y), Op<X3>(y.y), Op<X3>(z.x), Op<X3>(z.y));
        mma<X3>(c2, Op<X3>(x.z), Op<X3>(y.z), Op<X3>(x.w), Op<X3>(y.w), Op<X3>(z.z), Op<X3>(z.w));
      }
      const int t = 8 * a + gid;
      const unsigned long long anc = s_anc[t];
      const float bt = s_beta[t];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int s = 8 * b + 2 * j + e;
        const bool on = (anc >> s) & 1;
        s_L[t * LDT + s] = on && s != t ? bt * (c[e] + c2[e]) : 0.f;
        s_P[t * LDT + s] = on ? c[2 + e] + c2[2 + e] : 0.f;
      }
    }
  } else {
    // One warp per place: the path upwards, with the decay between its ends summed
    // from the near one, so that no large sums are subtracted.
    for (int t = warp; t < T8; t += Cfg::WARPS) {
      for (int s = lane; s <= (t | 7); s += 32) s_L[t * LDT + s] = s_P[t * LDT + s] = 0.f;
      __syncwarp();
      const int64_t rt = (row0 + (int64_t)t * H) * DK + lane;
      float kt[DK / 32], qt[DK / 32], d[DK / 32];
      const bool live = s_anc[t] != 0;
#pragma unroll
      for (int c = 0; c < DK / 32; ++c) {
        kt[c] = live ? to_f32(k[rt + 32 * c]) : 0.f;
        qt[c] = live ? to_f32(q[rt + 32 * c]) : 0.f;
        d[c] = 0.f;
      }
      for (int s = live ? t : -1; s >= 0; s = s_par[s]) {
        const int64_t rs = (row0 + (int64_t)s * H) * DK + lane;
        float kk = 0.f, qk = 0.f;
#pragma unroll
        for (int c = 0; c < DK / 32; ++c) {
          const float x = to_f32(k[rs + 32 * c]) * expf(d[c]);
          kk += kt[c] * x;
          qk += qt[c] * x;
          d[c] += g[rs + 32 * c];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          kk += __shfl_xor_sync(0xffffffffu, kk, o);
          qk += __shfl_xor_sync(0xffffffffu, qk, o);
        }
        if (lane == 0) {
          s_L[t * LDT + s] = s != t ? s_beta[t] * kk : 0.f;
          s_P[t * LDT + s] = qk;
        }
      }
    }
  }
  __syncthreads();

  // ---- inverses of the diagonal blocks of I + L: lane = column, forward substitution ----
  for (int b = warp; b < NB; b += Cfg::WARPS) {
    constexpr int B = 8 * BT;
    const float *L = s_L + b * B * LDT + b * B;
    float x[B];
#pragma unroll
    for (int t = 0; t < B; ++t) {
      float y0 = t == lane ? 1.f : 0.f, y1 = 0.f;
#pragma unroll
      for (int s = 0; s < t; ++s) {
        if (s & 1) y1 -= L[t * LDT + s] * x[s];
        else y0 -= L[t * LDT + s] * x[s];
      }
      x[t] = y0 + y1;
    }
    if (lane < B)
#pragma unroll
      for (int t = 0; t < B; ++t) s_M[(b * B + t) * LDB + lane] = x[t];
  }

  // ---- Kt S0 - V, transposed: accumulators hold columns x places ----
  const TIn *vp = v + row0 * DV + col;
  float vn[NT][MT][4];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int t = 8 * i + 2 * j + e;
      float x[E];
#pragma unroll
      for (int c = 0; c < E; ++c) x[c] = 0.f;
      if (t < T && s_anc[t] != 0) load_row<E>(vp + (int64_t)t * H * DV, x);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        vn[i][m][e] = -x[2 * m];
        vn[i][m][2 + e] = -x[2 * m + 1];
      }
    }
  }
#pragma unroll
  for (int a = 0; a < DK / 16; ++a) {
    Op<X3> A[2][MT][4];   // the two k8 tiles of these 16 state rows
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        A[w][m][0] = Op<X3>(s0[4 * a + 2 * w][2 * m]);
        A[w][m][1] = Op<X3>(s0[4 * a + 2 * w][2 * m + 1]);
        A[w][m][2] = Op<X3>(s0[4 * a + 2 * w + 1][2 * m]);
        A[w][m][3] = Op<X3>(s0[4 * a + 2 * w + 1][2 * m + 1]);
      }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const float4 x = *reinterpret_cast<const float4 *>(s_kt + (8 * i + gid) * LDK + 16 * a + 4 * j);
      const Op<X3> b0(x.x), b1(x.y), b2(x.z), b3(x.w);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        mma<X3>(vn[i][m], A[0][m][0], A[0][m][1], A[0][m][2], A[0][m][3], b0, b1);
        mma<X3>(vn[i][m], A[1][m][0], A[1][m][1], A[1][m][2], A[1][m][3], b2, b3);
      }
    }
  }
  __syncthreads();   // the blocks' inverses

  // acc += (rows of W)(vn)^T for one tile of places: W[8 r + gid][8 s + 2 j, + 1] in shared memory
  const auto apply = [&](float (&acc)[MT][4], const float (&x)[MT][4], const float *W, float sign) {
    const float2 w = *reinterpret_cast<const float2 *>(W);
    const Op<X3> b0(sign * w.x), b1(sign * w.y);
#pragma unroll
    for (int m = 0; m < MT; ++m)
      mma<X3>(acc[m], Op<X3>(x[m][0]), Op<X3>(x[m][2]), Op<X3>(x[m][1]), Op<X3>(x[m][3]), b0, b1);
  };

  // ---- (I + L) Vn = beta (V - Kt S0), block by block ----
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    float r[BT][MT][4];
#pragma unroll
    for (int i = 0; i < BT; ++i) {
      const float2 bt = *reinterpret_cast<const float2 *>(s_beta + 8 * (BT * b + i) + 2 * j);
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          r[i][m][e] = -(e & 1 ? bt.y : bt.x) * vn[BT * b + i][m][e];
          vn[BT * b + i][m][e] = 0.f;
        }
#pragma unroll
      for (int s = 0; s < BT * b; ++s)
        apply(r[i], vn[s], s_L + (8 * (BT * b + i) + gid) * LDT + 8 * s + 2 * j, -1.f);
    }
#pragma unroll
    for (int i = 0; i < BT; ++i)
#pragma unroll
      for (int s = 0; s <= i; ++s)
        apply(vn[BT * b + i], r[s], s_M + (8 * (BT * b + i) + gid) * LDB + 8 * s + 2 * j, 1.f);
  }

  // ---- O = Qt S0 + P Vn, a block of places at a time ----
  TIn *op = out + row0 * DV + col;
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    float o[BT][MT][4];
#pragma unroll
    for (int i = 0; i < BT; ++i)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][m][e] = 0.f;
#pragma unroll
    for (int a = 0; a < DK / 16; ++a) {
#pragma unroll
      for (int i = 0; i < BT; ++i) {
        const float4 x = *reinterpret_cast<const float4 *>(
            s_qt + (8 * (BT * b + i) + gid) * LDK + 16 * a + 4 * j);
        const Op<X3> b0(x.x), b1(x.y), b2(x.z), b3(x.w);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          mma<X3>(o[i][m], Op<X3>(s0[4 * a][2 * m]), Op<X3>(s0[4 * a][2 * m + 1]),
                  Op<X3>(s0[4 * a + 1][2 * m]), Op<X3>(s0[4 * a + 1][2 * m + 1]), b0, b1);
          mma<X3>(o[i][m], Op<X3>(s0[4 * a + 2][2 * m]), Op<X3>(s0[4 * a + 2][2 * m + 1]),
                  Op<X3>(s0[4 * a + 3][2 * m]), Op<X3>(s0[4 * a + 3][2 * m + 1]), b2, b3);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < BT; ++i) {
      const int tile = BT * b + i;
#pragma unroll
      for (int s = 0; s <= tile; ++s)
        apply(o[i], vn[s], s_P + (8 * tile + gid) * LDT + 8 * s + 2 * j, 1.f);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int t = 8 * tile + 2 * j + e;
        if (t < T) {
          const bool live = s_anc[t] != 0;
          float x[E];
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            x[2 * m] = live ? o[i][m][e] : 0.f;
            x[2 * m + 1] = live ? o[i][m][2 + e] : 0.f;
          }
          store_row<E>(op + (int64_t)t * H * DV, x);
        }
      }
    }
  }
}

template <int DK, int DV, int NT, typename TIn>
cudaError_t launch_nt(const void *q, const void *k, const void *v, const float *g,
                      const float *beta, const float *state, const int32_t *parents, void *out,
                      int T, int64_t units, int H, cudaStream_t stream) {
  using Cfg = TreeCfg<DK, DV, NT, TIn>;
  const auto kern = decode_tree_kernel<DK, DV, NT, TIn>;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg::BYTES);
  if (e != cudaSuccess) return e;
  kern<<<(unsigned)units, Cfg::THREADS, Cfg::BYTES, stream>>>(
      (const TIn *)q, (const TIn *)k, (const TIn *)v, g, beta, state, parents, (TIn *)out, T, H);
  return cudaGetLastError();
}

template <int DK, int DV, typename TIn>
cudaError_t launch_d(const void *q, const void *k, const void *v, const float *g,
                     const float *beta, const float *state, const int32_t *parents, void *out,
                     int T, int64_t units, int H, cudaStream_t stream) {
  // one instance per power of two of 8-place tiles
#define KDA_NT(NT_) \
  launch_nt<DK, DV, NT_, TIn>(q, k, v, g, beta, state, parents, out, T, units, H, stream)
  if (T <= 8) return KDA_NT(1);
  if (T <= 16) return KDA_NT(2);
  if (T <= 32) return KDA_NT(4);
  return KDA_NT(8);
#undef KDA_NT
}

}  // namespace

template <typename TIn>
cudaError_t launch_decode_tree_t(int dk, int dv, const void *q, const void *k, const void *v,
                                 const float *g, const float *beta, const float *state,
                                 const int32_t *parents, void *out, int T, int64_t units, int H,
                                 cudaStream_t stream) {
#define KDA_DT(DK_, DV_)      \
  if (dk == DK_ && dv == DV_) \
    return launch_d<DK_, DV_, TIn>(q, k, v, g, beta, state, parents, out, T, units, H, stream);
  KDA_DT(32, 32) KDA_DT(32, 64) KDA_DT(32, 128)
  KDA_DT(64, 32) KDA_DT(64, 64) KDA_DT(64, 128)
  KDA_DT(128, 32) KDA_DT(128, 64) KDA_DT(128, 128)
#undef KDA_DT
  return cudaErrorInvalidValue;
}

cudaError_t launch_decode_tree(int dtype, int dk, int dv, const void *q, const void *k,
                               const void *v, const float *g, const float *beta,
                               const float *state, const int32_t *parents, void *out, int T,
                               int64_t units, int H, cudaStream_t stream) {
  if (dtype == KDA_DTYPE_BF16)
    return launch_decode_tree_t<__nv_bfloat16>(dk, dv, q, k, v, g, beta, state, parents, out, T,
                                               units, H, stream);
  return launch_decode_tree_t<float>(dk, dv, q, k, v, g, beta, state, parents, out, T, units, H,
                                     stream);
}

}  // namespace kda

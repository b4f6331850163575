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
// Gam leaves +-80 forms L and P pair by pair from the differences instead (deep trees with
// gates near -5; 128 x 32 heads x 61 places, D = 64 in BF16: 989 us instead of 209).
//
// Layout: one CTA per (sequence, head).  Everything is computed transposed,
// O^T = S0^T Qt^T + Vn^T P^T, with value columns as the rows of m16n8k8 products:
//   - the A operand S0^T comes straight from the row-major FP32 state in HBM into
//     the registers of the warp that owns the columns (a lane reads pairs of
//     columns; which tile row a column is and which k index a state row is
//     are free choices), no shared memory, no transposition;
//   - the accumulators of Kt S0 have the layout of an A operand, so V - Kt S0, Vn
//     and the outputs stay in registers from the first product to the store.
// Shared memory holds the token rows (Kt, Qt, Kh) and the T x T matrices.  BF16 with
// D_k = D_v = 128 runs the tensor-memory kernel of kda_decode_tree_tc.cu, which needs
// value columns for all 128 lanes of an accumulator; this one serves the other head
// sizes, and FP32, whose three products per product the warp-level instructions take
// with operands split in registers.  It is bound by issue slots and by the round trips
// to memory (parents, then all rows at once): 512 x 32 heads x 16 places of D = 64 in
// BF16 take 132 us against 72 at the copy rate, of D = 128 in FP32 617 against 267.
//
// Arithmetic: TF32 products with FP32 accumulation for BF16 inputs (operands are
// rounded to about the nearest, 2^-10.5 of a value at most and 2^-11.7 rms, against
// 2^-9 when out is rounded).  FP32 inputs split each operand in two TF32 terms and add
// three products, and carry Gam as an unevaluated sum of two FP32 numbers, for FP32
// accuracy.
#include "kda_common.cuh"
#include "kda_launch.cuh"
#include "kda_tf32.cuh"

namespace kda {
namespace {

constexpr float kGamLimit = 80.f;
constexpr float kFactorLimit = 0x1p120f;
// At Gam = -80 an element of Kt is 1.8e-35 of k's: a subnormal number for small rows of q and
// k, and for FP32 inputs its second TF32 term, 2^-12 of it, is one for most (16 places with
// gates of -5, q of size 10^-2: 1e-4 off).  So Kh is held divided by a power of two, and
// - FP32: Kt and Qt enter L and P times that, by the split in two terms; terms keep 2^-24 of an
//   element down to 2^-26, and rows too large for it go pair by pair;
// - BF16: Kt and Qt are held times it, V and P as well, and divided again on the way to Vn and
//   out (states or outputs above 10^31 overflow).
template <bool X3> __device__ constexpr float lift() { return X3 ? 0x1p40f : 0x1p24f; }

// Rounded by the conversion instruction.
__device__ __forceinline__ float rn_tf32(float x) {
  uint32_t r;
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
  return __uint_as_float(r);
}
// An operand of the products.  For X3 it is an FP32 value, split into two TF32
// terms where it is used; otherwise it is a value made ready for the cut to TF32 when it
// was made (operand<X3>), whose bits go in as they are.
template <bool X3> __device__ __forceinline__ float operand(float x) { return X3 ? x : to_tf32(x); }
template <bool X3> struct Op {
  uint32_t hi, lo;
  __device__ __forceinline__ explicit Op(float x) {
    if (X3) {
      const float h = cut_tf32(x);
      hi = __float_as_uint(h);
      lo = __float_as_uint(x - h);      // exact; cut in the product, 2^-21 of x
    } else {
      hi = __float_as_uint(x);
    }
  }
  // Of an element of Kt or Qt, times the lift (BF16: it is held so).
  static __device__ __forceinline__ Op lifted(float x) {
    Op r(x);
    if (X3) {
      const float h = __uint_as_float(__float_as_uint(x * (kTf32 * lift<X3>())) & 0xffffe000u);
      r.hi = __float_as_uint(h);
      r.lo = __float_as_uint(fmaf(x, lift<X3>(), -h));
    }
    return r;
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

// What a few products add to an accumulator.  The tensor cores cut, not round, what they
// add to their accumulators (over 48 products of one sum that was 1.6e-6 of the outputs),
// so for X3 a short sum starts from zero and is added by an FP32 addition: 2.0e-7, for 4 %
// of the time.
template <bool X3> struct Sum {
  float c[4];
  __device__ __forceinline__ explicit Sum(const float (&acc)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) c[e] = X3 ? 0.f : acc[e];
  }
  __device__ __forceinline__ void add_to(float (&acc)[4]) const {
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] = X3 ? acc[e] + c[e] : c[e];
  }
};

// Token rows lie in shared memory without padding, in 16-byte units whose low
// three index bits are exclusive-ored with this function of the row: reads of
// units 4 a + j of rows 8 i + gid, and writes of unit gid (or half a unit) of rows
// 8 i + 2 j + e, touch distinct banks.
__device__ __forceinline__ int swizzle(int row) { return ((row & 6) ^ ((row & 1) << 2)); }

// Two consecutive elements, as loaded and as floats.
template <typename T> struct Pair;
template <> struct Pair<__nv_bfloat16> {
  uint32_t x = 0u;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) { x = *reinterpret_cast<const uint32_t *>(p); }
  __device__ __forceinline__ float2 get() const {
    return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
  }
};
template <> struct Pair<float> {
  float2 x = {0.f, 0.f};
  __device__ __forceinline__ void load(const float *p) { x = *reinterpret_cast<const float2 *>(p); }
  __device__ __forceinline__ float2 get() const { return x; }
};
__device__ __forceinline__ void store_pair(__nv_bfloat16 *p, float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  *reinterpret_cast<uint32_t *>(p) = *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ void store_pair(float *p, float a, float b) {
  *reinterpret_cast<float2 *>(p) = make_float2(a, b);
}

// Sets of places: 32 bits do for up to four tiles.
template <int NT> struct MaskOf { using T = uint32_t; };
template <> struct MaskOf<8> { using T = unsigned long long; };

// NT: tiles of 8 places (places past T are empty ones).
template <int DK, int DV, int NT, typename TIn> struct TreeCfg {
  static constexpr bool X3 = sizeof(TIn) == 4;
  static constexpr int WARPS = DV / 16;             // 16 value columns each, two per lane
  // Rows are loaded into registers as soon as the paths are known, all at once (before the
  // operands' rounding was a product, 512 x 32 heads x 16 places of D = 64, BF16: 147 us, 223
  // when they were loaded where they are used; 128 x 32 x 61 places: 218 and 396), except
  // where the registers cost the second CTA of an SM (FP32, 256 x 32 x 30 places: D = 64/128
  // 542 us, 512 without; 32/128 445 and 437).
  static constexpr bool AHEAD = !(X3 && NT == 4 && WARPS == 8 && DK < 128);
  static constexpr int THREADS = 32 * WARPS;
  static constexpr int T8 = 8 * NT;
  static constexpr int NB = NT < 2 ? 1 : NT / 2;    // diagonal blocks
  static constexpr int BT = NT < 2 ? 1 : 2;         // tiles per diagonal block
  static constexpr int LDT = T8 + (T8 == 8 ? 0 : 8);   // = 8 or 24 modulo 32: 8-byte accesses
  static constexpr int LDB = 8 * BT + (BT == 1 ? 0 : 8);
  // shared memory, in floats
  static constexpr int KT = 0, QT = KT + T8 * DK, KH = QT + T8 * DK;
  static constexpr int LM = KH + T8 * DK, PM = LM + T8 * LDT;
  static constexpr int MI = PM + T8 * LDT;          // (I + L)^-1 of the diagonal blocks
  static constexpr int BE = MI + NB * 8 * BT * LDB;
  static constexpr int TOTAL = BE + T8;
  static constexpr size_t BYTES = (size_t)TOTAL * 4;
};

template <int DK, int DV, int NT, typename TIn>
__global__ void __launch_bounds__(TreeCfg<DK, DV, NT, TIn>::THREADS)
decode_tree_kernel(const TIn *q, const TIn *k,
                   const TIn *v, const float *g,
                   const float *beta, const float *state,
                   const int32_t *parents, TIn *__restrict__ out, int T, int H) {
  using Cfg = TreeCfg<DK, DV, NT, TIn>;
  using Mask = typename MaskOf<NT>::T;
  constexpr bool X3 = Cfg::X3;
  constexpr float kHeld = X3 ? 1.f : lift<X3>();   // what Kt, Qt, V and P are held times
  constexpr int T8 = Cfg::T8, LDT = Cfg::LDT, E = 2;
  constexpr bool AHEAD = Cfg::AHEAD;
  constexpr int LDB = Cfg::LDB, BT = Cfg::BT, NB = Cfg::NB;
  extern __shared__ __align__(16) float sm[];
  float *s_kt = sm + Cfg::KT, *s_qt = sm + Cfg::QT, *s_kh = sm + Cfg::KH;
  float *s_L = sm + Cfg::LM, *s_P = sm + Cfg::PM, *s_M = sm + Cfg::MI, *s_beta = sm + Cfg::BE;
  __shared__ Mask s_anc[T8];           // ancestors and self; 0: an empty place
  __shared__ int s_par[T8], s_jump[T8], s_tiles;

  const int64_t unit = blockIdx.x;
  const int n = (int)(unit / H), h = (int)(unit % H);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gid = lane >> 2, j = lane & 3;
  const int64_t row0 = (int64_t)n * T * H + h;      // token t is row row0 + t H

  launch_dependents();
  wait_for_inputs();
  int up[T8 > 32 ? 2 : 1];             // predecessors of places lane (and lane + 32)
  float bt[T8 > 32 ? 2 : 1];
  if (warp == 0) {
#pragma unroll
    for (int e = 0; e < (T8 > 32 ? 2 : 1); ++e) {
      const int t = lane + 32 * e;
      up[e] = -2;
      bt[e] = 0.f;
      if (t < T) {
        up[e] = parents ? parents[(int64_t)n * T + t] : t - 1;
        bt[e] = beta[row0 + (int64_t)t * H];
      }
    }
  }

  // ---- the state's columns of this warp: rows 16 a + 4 j + m, columns col, col + 1 ----
  const int col = 16 * warp + E * gid;
  float s0[DK / 4][E];
  {
    const float *src = state + unit * (DK * DV) + (int64_t)(4 * j) * DV + col;
#pragma unroll
    for (int m = 0; m < DK / 4; ++m)
      asm volatile("ld.global.cs.v2.f32 {%0,%1}, [%2];"
                   : "=f"(s0[m][0]), "=f"(s0[m][1])
                   : "l"(src + ((m >> 2) * 16 + (m & 3)) * DV));
  }

  // ---- ancestors by pointer doubling (one warp): after the step of size d every
  //      mask holds the last 2 d places of its path ----
  if (warp == 0) {
    if (T8 <= 32) {
      if (up[0] < -1 || up[0] >= lane) up[0] = -2;
      int jump = up[0];
      uint32_t m = 1u << lane;
      for (int d = 1; d < T; d <<= 1) {
        const uint32_t mo = __shfl_sync(0xffffffffu, m, jump & 31);
        const int jo = __shfl_sync(0xffffffffu, jump, jump & 31);
        if (jump >= 0) { m |= mo; jump = jo; }
      }
      if (jump != -1) m = 0;                           // a path that ends in an empty place
      if (lane < T8) { s_anc[lane] = (Mask)m; s_par[lane] = up[0]; }
    } else {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int t = lane + 32 * e;
        int &u = up[T8 > 32 ? e : 0];
        if (u < -1 || u >= t) u = -2;
        if (t < T8) {
          s_par[t] = u;
          s_jump[t] = u;
          s_anc[t] = (Mask)1 << (t < T8 ? t : 0);
        }
      }
      __syncwarp();
      for (int d = 1; d < T; d <<= 1) {
        Mask m[2];
        int jo[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int t = (lane + 32 * e) % T8, a = s_jump[t];
          m[e] = s_anc[t] | (a >= 0 ? s_anc[a] : (Mask)0);
          jo[e] = a >= 0 ? s_jump[a] : a;
        }
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          s_anc[(lane + 32 * e) % T8] = m[e];
          s_jump[(lane + 32 * e) % T8] = jo[e];
        }
        __syncwarp();
      }
      for (int t = lane; t < T8; t += 32)
        if (s_jump[t] != -1) s_anc[t] = 0;
    }
    __syncwarp();
    // tiles up to the last token that is there; the rest is not computed
    int last = -1;
#pragma unroll
    for (int e = 0; e < (T8 > 32 ? 2 : 1); ++e) {
      const int t = lane + 32 * e;
      if (t < T8) {
        const bool live = s_anc[t] != 0;
        s_beta[t] = live ? bt[e] : 0.f;
        if (live) last = t;
      }
    }
    last = __reduce_max_sync(0xffffffffu, last);
    if (lane == 0) s_tiles = (last + 8) >> 3;
  }
  __syncthreads();
  const int tiles = s_tiles;

  // The lane's places 8 i + 2 j + e.
  const auto place = [&](int i, int e) { return 8 * i + 2 * j + e; };
  const TIn *vp = v + row0 * DV + col;
  Pair<TIn> rv[AHEAD ? 2 * NT : 1];
  if (AHEAD) {
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (i < tiles && s_anc[place(i, e)] != 0) rv[AHEAD ? 2 * i + e : 0].load(vp + (int64_t)place(i, e) * H * DV);
  }

  // ---- Gam along the paths, Kt, Qt, Kh.  Gam^T = g^T A^T with A the 0/1 matrix of
  //      ancestors, a product as well: a lane brings g, and gets Gam, of its places
  //      in two channels.  g goes in as two TF32 terms (2^-23 of it is
  //      lost); for X3 as multiples of 1/8, whose sums are exact, and two terms for
  //      the rest, with sums of their own. ----
  bool wide = false;   // factors out of range: L and P pair by pair
  for (int cw = warp; cw < DK / 16; cw += Cfg::WARPS) {
    const int c0 = 16 * cw + E * gid;
    const int64_t at0 = row0 * DK + c0, step = (int64_t)H * DK;
    Pair<float> rg[AHEAD ? 2 * NT : 1];
    Pair<TIn> rk[AHEAD ? 2 * NT : 1], rq[AHEAD ? 2 * NT : 1];
    if (AHEAD) {
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (i < tiles && s_anc[place(i, e)] != 0) {
            const int64_t at = at0 + place(i, e) * step;
            rg[AHEAD ? 2 * i + e : 0].load(g + at);
            rk[AHEAD ? 2 * i + e : 0].load(k + at);
            rq[AHEAD ? 2 * i + e : 0].load(q + at);
          }
    }
    float gam[NT][4], low[X3 ? NT : 1][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        gam[i][e] = 0.f;
        if (X3) low[X3 ? i : 0][e] = 0.f;
      }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      if (i >= tiles) break;
      float x[2][E];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        Pair<float> y;
        if (AHEAD) y = rg[AHEAD ? 2 * i + e : 0];
        else if (s_anc[place(i, e)] != 0) y.load(g + at0 + place(i, e) * step);
        x[e][0] = y.get().x;
        x[e][1] = y.get().y;
      }
      uint32_t hi[4], lo[4], lo2[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float y = x[e >> 1][e & 1];             // a0, a1: place 2 j; a2, a3: place 2 j + 1
        if (X3) {
          y = max_nan(y, -128.f);               // exp(-128) is 0 in FP32 already
          const float r = rintf(y * 8.f) * 0.125f;
          hi[e] = __float_as_uint(r);
          y -= r;
          const float l = cut_tf32(y);
          lo[e] = __float_as_uint(l);
          lo2[e] = __float_as_uint(y - l);
        } else {
          y = max_nan(y, -1e5f);                // finite: it meets zeros in the product
          const float h = cut_tf32(y);
          hi[e] = __float_as_uint(h);
          lo[e] = __float_as_uint(y - h);
        }
      }
#pragma unroll
      for (int r = i; r < NT; ++r) {
        const uint32_t bits = (uint32_t)(s_anc[8 * r + gid] >> (8 * i + 2 * j));
        const uint32_t b0 = bits & 1 ? 0x3f800000u : 0u, b1 = bits & 2 ? 0x3f800000u : 0u;
        mma_raw(gam[r], hi[0], hi[1], hi[2], hi[3], b0, b1);
        mma_raw(X3 ? low[X3 ? r : 0] : gam[r], lo[0], lo[1], lo[2], lo[3], b0, b1);
        if (X3) mma_raw(low[X3 ? r : 0], lo2[0], lo2[1], lo2[2], lo2[3], b0, b1);
      }
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      if (i >= tiles) break;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int t = place(i, e);
        Pair<TIn> yk, yq;
        if (AHEAD) {
          yk = rk[AHEAD ? 2 * i + e : 0];
          yq = rq[AHEAD ? 2 * i + e : 0];
        } else if (s_anc[t] != 0) {
          yk.load(k + at0 + t * step);
          yq.load(q + at0 + t * step);
        }
        float kv[E] = {yk.get().x, yk.get().y}, qv[E] = {yq.get().x, yq.get().y}, kh[E];
#pragma unroll
        for (int c = 0; c < E; ++c) {
          float G = gam[i][2 * c + e], down, inv;
          if (X3) {
            const float b = low[X3 ? i : 0][2 * c + e];
            const float sum = G + b, rest = b - (sum - G);
            G = sum;
            down = expf(G);
            down += down * rest;
            inv = expf(-G);
            inv = (inv - inv * rest) * (1.f / lift<X3>());
          } else {                              // and made ready for the cut
            down = __expf(G) * (kTf32 * lift<X3>());
            inv = __expf(-G) * (kTf32 / lift<X3>());
          }
          kh[c] = kv[c] * inv;
          float top = fabsf(kh[c]);
          if (X3) top = fmaxf(top, fmaxf(fabsf(kv[c]), fabsf(qv[c])));
          kv[c] *= down;
          qv[c] *= down;
          wide |= !(top < kFactorLimit / lift<X3>()) || !(fabsf(G) <= kGamLimit);
        }
        const int at = t * DK + ((((c0 >> 2) ^ swizzle(t)) << 2) | (c0 & 3));
        store_pair(s_kt + at, kv[0], kv[1]);
        store_pair(s_qt + at, qv[0], qv[1]);
        store_pair(s_kh + at, kh[0], kh[1]);
      }
    }
  }

  // ---- -V, transposed: what the products below are added to (columns x places) ----
  float vn[NT][4];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int t = place(i, e);
      Pair<TIn> y;
      if (AHEAD) y = rv[AHEAD ? 2 * i + e : 0];
      else if (s_anc[t] != 0) y.load(vp + (int64_t)t * H * DV);
      vn[i][e] = y.get().x * -kHeld;
      vn[i][2 + e] = y.get().y * -kHeld;
    }
  wide = __syncthreads_or(wide);

  // Where this lane's 16-byte units of channels 16 a + 4 j lie in a row 8 i + gid.
  const int even = gid * DK + ((j ^ swizzle(gid)) << 2), odd = even ^ 16;
  const auto unit_at = [&](const float *rows, int i, int a) {
    return *reinterpret_cast<const float4 *>(rows + 8 * i * DK + 32 * (a >> 1) + (a & 1 ? odd : even));
  };
  // L as the diagonal blocks' inverses need it, -L as an operand elsewhere.
  const auto put = [&](int t, int s, float lt, float pt) {
    s_L[t * LDT + s] = t / (8 * BT) == s / (8 * BT) ? lt : operand<X3>(-lt);
    s_P[t * LDT + s] = X3 ? pt : pt * (kTf32 * kHeld);
  };

  // ---- L and P: tile (a, b) of 8 x 8 places, rows Kt and Qt of one tile in one product ----
  if (!wide) {
    for (int tile = warp; tile < tiles * (tiles + 1) / 2; tile += Cfg::WARPS) {
      int a = 0;
      while ((a + 1) * (a + 2) / 2 <= tile) ++a;
      const int b = tile - a * (a + 1) / 2;
      float c[4] = {0.f, 0.f, 0.f, 0.f}, c2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < DK / 16; ++i) {
        const float4 x = unit_at(s_kt, a, i), y = unit_at(s_qt, a, i), z = unit_at(s_kh, b, i);
        const auto up = [](float e) { return Op<X3>::lifted(e); };
        Sum<X3> s1(c), s2(c2);
        mma<X3>(s1.c, up(x.x), up(y.x), up(x.y), up(y.y), Op<X3>(z.x), Op<X3>(z.y));
        mma<X3>(s2.c, up(x.z), up(y.z), up(x.w), up(y.w), Op<X3>(z.z), Op<X3>(z.w));
        s1.add_to(c);
        s2.add_to(c2);
      }
      const int t = 8 * a + gid;
      const Mask anc = s_anc[t];
      const float bt = s_beta[t];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int s = 8 * b + 2 * j + e;
        const bool on = (anc >> s) & 1;
        put(t, s, on && s != t ? bt * (c[e] + c2[e]) : 0.f, on ? c[2 + e] + c2[2 + e] : 0.f);
      }
    }
  } else {
    // One warp per place: the path upwards, with the decay between its ends summed
    // from the near one, so that no large sums are subtracted.
    for (int t = warp; t < 8 * tiles; t += Cfg::WARPS) {
      for (int s = lane; s <= (t | 7); s += 32) put(t, s, 0.f, 0.f);
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
        if (lane == 0) put(t, s, s != t ? s_beta[t] * kk : 0.f, qk);
      }
    }
  }
  __syncthreads();

  // ---- M = (I + L)^-1 of the diagonal blocks, a lane per row, from M (I + L) = I:
  //      once entry s is final, row s of L takes it out of the entries before ----
  if (warp < (NB + 1) / 2) {
    constexpr int B = 8 * BT;
    const int b = min(2 * warp + (lane >> 4), NB - 1), r = lane & 15;
    const float *L = s_L + b * B * LDT + b * B;
    float x[B];
#pragma unroll
    for (int s = 0; s < B; ++s) x[s] = s == r ? 1.f : 0.f;
    if (B * b < 8 * tiles) {
#pragma unroll
      for (int s = B - 1; s > 0; --s) {
        if (BT == 2 && s >= 8 && 8 * (2 * b + 1) >= 8 * tiles) continue;   // rows not computed
#pragma unroll
        for (int e = 0; e < s; e += 4) {
          const float4 l = *reinterpret_cast<const float4 *>(L + s * LDT + e);
          x[e] -= x[s] * l.x;
          if (e + 1 < s) x[e + 1] -= x[s] * l.y;
          if (e + 2 < s) x[e + 2] -= x[s] * l.z;
          if (e + 3 < s) x[e + 3] -= x[s] * l.w;
        }
      }
    }
    if (r < B && (lane < 16 || NB > 1))
#pragma unroll
      for (int s = 0; s < B; s += 4)
        *reinterpret_cast<float4 *>(s_M + (b * B + r) * LDB + s) =
            make_float4(operand<X3>(x[s]), operand<X3>(x[s + 1]), operand<X3>(x[s + 2]),
                        operand<X3>(x[s + 3]));
  }

  // ---- Kt S0 - V and Qt S0, transposed, in one pass over the state ----
  float o[NT][4];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
#pragma unroll
  for (int a = 0; a < DK / 16; ++a) {
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        // The conversion instruction is slower than the product of operand(), but with 64
        // elements per lane the code around it comes out no slower, and faster for four tiles
        // of places (256 x 32 heads x 30 places, BF16: D = 128/32 276 us against 312, 128/64
        // 250 both; 512 x 32 x 16: 128/32 213 against 211, 64/128 309 against 252).
        float &x = s0[4 * a + m][e];
        x = !X3 && DK == 128 ? rn_tf32(x) : operand<X3>(x);
      }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      if (i >= tiles) break;
      const float4 x = unit_at(s_kt, i, a), y = unit_at(s_qt, i, a);
      const Op<X3> x0(x.x), x1(x.y), x2(x.z), x3(x.w), y0(y.x), y1(y.y), y2(y.z), y3(y.w);
      const Op<X3> a0(s0[4 * a][0]), a1(s0[4 * a][1]), a2(s0[4 * a + 1][0]), a3(s0[4 * a + 1][1]);
      const Op<X3> d0(s0[4 * a + 2][0]), d1(s0[4 * a + 2][1]), d2(s0[4 * a + 3][0]),
          d3(s0[4 * a + 3][1]);
      Sum<X3> sv(vn[i]), so(o[i]);
      mma<X3>(sv.c, a0, a1, a2, a3, x0, x1);
      mma<X3>(so.c, a0, a1, a2, a3, y0, y1);
      mma<X3>(sv.c, d0, d1, d2, d3, x2, x3);
      mma<X3>(so.c, d0, d1, d2, d3, y2, y3);
      sv.add_to(vn[i]);
      so.add_to(o[i]);
    }
  }
  __syncthreads();   // the blocks' inverses

  // acc += x (rows of W)^T for one tile of places: W[8 r + gid][8 s + 2 j, + 1]
  const auto apply = [&](float (&acc)[4], const float (&x)[4], const float *W) {
    const float2 w = *reinterpret_cast<const float2 *>(W);
    Sum<X3> sum(acc);
    mma<X3>(sum.c, Op<X3>(x[0]), Op<X3>(x[2]), Op<X3>(x[1]), Op<X3>(x[3]), Op<X3>(w.x), Op<X3>(w.y));
    sum.add_to(acc);
  };

  // ---- (I + L) Vn = beta (V - Kt S0), block by block ----
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    if (BT * b >= tiles) break;
    float r[BT][4];
#pragma unroll
    for (int i = 0; i < BT; ++i) {
      float2 bt2 = *reinterpret_cast<const float2 *>(s_beta + 8 * (BT * b + i) + 2 * j);
      bt2 = make_float2(bt2.x * (-1.f / kHeld), bt2.y * (-1.f / kHeld));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        r[i][e] = (e & 1 ? bt2.y : bt2.x) * vn[BT * b + i][e];
        vn[BT * b + i][e] = 0.f;
      }
      if (BT * b + i < tiles) {
#pragma unroll
        for (int s = 0; s < BT * b; ++s)
          apply(r[i], vn[s], s_L + (8 * (BT * b + i) + gid) * LDT + 8 * s + 2 * j);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) r[i][e] = operand<X3>(r[i][e]);
    }
#pragma unroll
    for (int i = 0; i < BT; ++i) {
#pragma unroll
      for (int s = 0; s <= i; ++s)
        apply(vn[BT * b + i], r[s], s_M + (8 * (BT * b + i) + gid) * LDB + 8 * s + 2 * j);
#pragma unroll
      for (int e = 0; e < 4; ++e) vn[BT * b + i][e] = operand<X3>(vn[BT * b + i][e]);
    }
  }

  // ---- O = Qt S0 + P Vn ----
  TIn *op = out + row0 * DV + col;
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    if (i < tiles) {
#pragma unroll
      for (int s = 0; s <= i; ++s) apply(o[i], vn[s], s_P + (8 * i + gid) * LDT + 8 * s + 2 * j);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int t = place(i, e);
      if (t < T) {
        const bool live = s_anc[t] != 0;
        store_pair(op + (int64_t)t * H * DV, live ? o[i][e] * (1.f / kHeld) : 0.f,
                   live ? o[i][2 + e] * (1.f / kHeld) : 0.f);
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
  return launch_dependent(kern, (unsigned)units, Cfg::THREADS, Cfg::BYTES, 1, stream, (const TIn *)q,
                          (const TIn *)k, (const TIn *)v, g, beta, state, parents, (TIn *)out, T, H);
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
#define KDA_DT(DK_, DV_)                                                                          \
  if (dk == DK_ && dv == DV_)                                                                     \
    return launch_d<DK_, DV_, TIn>(q, k, v, g, beta, state, parents, out, T, units, H, stream);
  KDA_DT(32, 32) KDA_DT(32, 64) KDA_DT(32, 128)
  KDA_DT(64, 32) KDA_DT(64, 64) KDA_DT(64, 128)
  KDA_DT(128, 32) KDA_DT(128, 64)
  if constexpr (sizeof(TIn) == 4) KDA_DT(128, 128)   // BF16: the tensor-memory kernel
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

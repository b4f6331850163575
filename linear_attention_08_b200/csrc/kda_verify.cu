// Verification of drafted tokens against the target's probabilities, from
// given random numbers.
//
// For one sequence, context c is the committed prefix (-1) or a drafted token;
// p_c and d_c are the target's and the draft's distributions after it.  With
// r = p_c and R = 1, the successors of c are tried in the order of their places:
//
//   token x at place i is accepted when r(x) > 0 and u_i R d_c(x) < r(x)
//   accepted: c = i, r = p_i, R = 1
//   refused:  r = max(r - R d_c, 0), R = sum(r)
//
// and when no successor is left the next token is the smallest j with
// r(0) + ... + r(j) > u_last sum(r).  (r / R is what is left of the target's
// distribution; the test and the draw do not change when r and R are scaled
// together, so r is not divided by R, and may double with every refusal:
// a + |a| = 2 max(a, 0) is one FP64 addition, a maximum four instructions.)
// Accepted and drawn tokens then follow the target's distribution exactly, for
// one drafted token per context (a chain) and for several drawn from d_c (a
// tree).  Without a draft distribution (tokens from a lookup, not a sample) d_c
// is one at the token itself: a refusal sets r(x) = 0 and takes p_c(x) from R.
//
// Sums and comparisons are FP64: a token's border in the cumulative sum has to come
// out the same whatever order the sum is taken in, and FP32 would move one draw in
// some hundreds at 10^5 tokens.  The probabilities' bits, shifted into place, are
// their values times 2^-896 in FP64; the conversion instruction has a quarter of the
// rate of the FP64 additions and was the bound (passes over 48 x 50256 FP32
// elements after a refusal: 7 to 13 us before, 5 to 8 us now).
//
// Work: all successors' p and d are gathered at once, so a path of accepted
// tokens reads no rows; only the last context's rows (and those of a context
// with a refusal and a later successor) are read whole.  A cluster of 1 to 8
// CTAs takes one sequence; its CTAs hold one slice of the vocabulary each, add
// their sums over distributed shared memory, and the CTA whose slice holds the
// border finds the token.  No atomics and no workspace: the result does not
// depend on scheduling, and calls on any streams do not share anything.
//
// 64 chains of 7 tokens, 131072 BF16 elements: 14.0 us, 5.1 at the copy rate; without a
// draft 12.2.  48 trees of 24 places, 50257 FP32 elements: 19 to 24 us (the sequence with
// most refusals sets the time), 3.0 at the copy rate; without a draft 14.5.
#include <cooperative_groups.h>

#include "kda_common.cuh"
#include "kda_launch.cuh"

namespace kda {
namespace {

namespace cg = cooperative_groups;

constexpr int kVThreads = 512;
constexpr int kVWarps = kVThreads / 32;
constexpr int kVMaxNodes = 64;
constexpr int kVMaxCluster = 8;

// Elements of one 16-byte load.
template <typename P> constexpr int kVec = 16 / (int)sizeof(P);

// x times 2^-896, exactly, for x >= 0: an FP32 number's exponent and fraction in the
// FP64 fields, subnormal ones too.  Whatever is not positive counts as zero.
constexpr double kUnscale = 0x1p896;
__device__ __forceinline__ double scaled(float x) {
  const uint32_t b = __float_as_uint(fmaxf(x, 0.f));
  return __hiloint2double((int)(b >> 3), (int)(b << 29));
}
__device__ __forceinline__ double scaled_bf16(uint32_t bits) {   // of the upper half
  return __hiloint2double((int)(__float_as_uint(fmaxf(__uint_as_float(bits), 0.f)) >> 3), 0);
}

// 16 bytes, or an element, of global memory (which a called function does not know p to be in).
__device__ __forceinline__ uint4 load16(const void *p) {
  uint4 x;
  asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "l"(p));
  return x;
}
__device__ __forceinline__ void load1(const float *p, float &x) {
  asm volatile("ld.global.f32 %0, [%1];" : "=f"(x) : "l"(p));
}
__device__ __forceinline__ void load1(const __nv_bfloat16 *p, __nv_bfloat16 &x) {
  unsigned short b;
  asm volatile("ld.global.u16 %0, [%1];" : "=h"(b) : "l"(p));
  x = __ushort_as_bfloat16(b);
}

// W neighbouring elements as one load gives them (one, or 16 bytes), and their values.
template <typename P, int W> struct Raw;
template <> struct Raw<float, 4> {
  uint4 x;
  __device__ __forceinline__ void load(const float *p) { x = load16(p); }
  __device__ __forceinline__ void clear() { x = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void get(double (&f)[4]) const {
    f[0] = scaled(__uint_as_float(x.x)); f[1] = scaled(__uint_as_float(x.y));
    f[2] = scaled(__uint_as_float(x.z)); f[3] = scaled(__uint_as_float(x.w));
  }
};
template <> struct Raw<__nv_bfloat16, 8> {
  uint4 x;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) { x = load16(p); }
  __device__ __forceinline__ void clear() { x = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void get(double (&f)[8]) const {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = scaled_bf16(w[i] << 16);
      f[2 * i + 1] = scaled_bf16(w[i] & 0xffff0000u);
    }
  }
};
template <typename P> struct Raw<P, 1> {
  P x;
  __device__ __forceinline__ void load(const P *p) { load1(p, x); }
  __device__ __forceinline__ void clear() { x = from_f32<P>(0.f); }
  __device__ __forceinline__ void get(double (&f)[1]) const { f[0] = scaled(to_f32(x)); }
};

// What is left of a context's target distribution after its refusals, by case:
// kWhole: none; kMinus: one, 2 max(p - d, 0); kMany: several with a draft;
// kGone: without a draft, the refused tokens' elements are zero.
enum Mode { kWhole, kMinus, kMany, kGone };
struct Rest {
  bool draft;             // refusals subtract the draft's row (else zero a token)
  int m;                  // refusals so far
  const double *sum;      // R before each of them (1 before the first)
  const int32_t *gone;    // the refused tokens
  __device__ __forceinline__ Mode mode() const {
    return m == 0 ? kWhole : !draft ? kGone : m == 1 ? kMinus : kMany;
  }
  // r of B times W neighbouring elements, those of one b from `at` + b `step` on, from p
  // and d; all times 2^-896.
  template <int MODE, int B, int W>
  __device__ __forceinline__ void of(double (&r)[B][W], const double (&d)[B][W], int at,
                                     int step) const {
    if (MODE == kWhole) return;
    const int n = MODE == kMinus ? 1 : m;
#pragma unroll 1
    for (int l = 0; l < n; ++l) {
      const double R = MODE == kMany ? -sum[l] : -1.0;
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const int x = MODE == kGone ? gone[l] - (at + b * step) : 0;
#pragma unroll
        for (int e = 0; e < W; ++e) {
          if (MODE == kGone) {
            r[b][e] = x == e ? 0.0 : r[b][e];
          } else {
            r[b][e] = MODE == kMany ? fma(R, d[b][e], r[b][e]) : r[b][e] - d[b][e];
            r[b][e] += fabs(r[b][e]);
          }
        }
      }
    }
  }
};

// Sum of the rest over [lo, hi) over the calling lanes' strided loads of W
// elements, B of them in flight; hi - lo is a multiple of W.
template <typename P, int MODE, int W>
__device__ __forceinline__ double sum_w(const P *p, const P *d, const Rest &rest, int lo, int hi,
                                        int lane) {
  constexpr int B = W == 1 ? 8 : 4, G = 8 / W;
  constexpr bool D = MODE == kMinus || MODE == kMany;
  double acc = 0.0;
#pragma unroll 1
  for (int i = lo + lane * W; i < hi; i += B * 32 * W) {
    Raw<P, W> p0[B], d0[B];
#pragma unroll
    for (int j = 0; j < B; ++j) {
      const int at = i + j * 32 * W;
      if (at < hi) {
        p0[j].load(p + at);
        if (D) d0[j].load(d + at);
      } else {
        p0[j].clear();
        if (D) d0[j].clear();
      }
    }
#pragma unroll
    for (int j = 0; j < B; j += G) {       // G loads' elements at once
      double r[G][W], y[G][W];
#pragma unroll
      for (int b = 0; b < G; ++b) {
        p0[j + b].get(r[b]);
        if (D) d0[j + b].get(y[b]);
      }
      rest.of<MODE, G, W>(r, y, i + j * 32 * W, 32 * W);
#pragma unroll
      for (int b = 0; b < G; ++b) {
#pragma unroll
        for (int o = 1; o < W; o <<= 1)    // pairs first: short chains of FP64 additions
#pragma unroll
          for (int e = 0; e + o < W; e += 2 * o) r[b][e] += r[b][e + o];
      }
#pragma unroll
      for (int o = 1; o < G; o <<= 1)
#pragma unroll
        for (int b = 0; b + o < G; b += 2 * o) r[b][0] += r[b + o][0];
      acc += r[0][0];
    }
  }
  return acc;
}

// The same with 16-byte loads where the rows allow them (a row starts where its
// element type aligns, no more), else, and behind the last whole one, by elements.
template <typename P, int MODE>
__device__ __noinline__ double sum_mode(const P *p, const P *d, const Rest &rest, int lo, int hi,
                                        int lane) {
  constexpr int V = kVec<P>;
  constexpr bool D = MODE == kMinus || MODE == kMany;
  uintptr_t bits = reinterpret_cast<uintptr_t>(p + lo);
  if (D) bits |= reinterpret_cast<uintptr_t>(d + lo);
  const int whole = (bits & 15u) == 0 ? (hi - lo) / V * V : 0;
  double acc = 0.0;
  if (whole) acc = sum_w<P, MODE, V>(p, d, rest, lo, lo + whole, lane);
  if (lo + whole < hi) acc += sum_w<P, MODE, 1>(p, d, rest, lo + whole, hi, lane);
  return acc;
}
template <typename P>
__device__ __forceinline__ double rest_sum(const P *p, const P *d, const Rest &rest, int lo,
                                           int hi, int lane) {
  switch (rest.mode()) {
    case kWhole: return sum_mode<P, kWhole>(p, d, rest, lo, hi, lane);
    case kMinus: return sum_mode<P, kMinus>(p, d, rest, lo, hi, lane);
    case kMany: return sum_mode<P, kMany>(p, d, rest, lo, hi, lane);
    default: return sum_mode<P, kGone>(p, d, rest, lo, hi, lane);
  }
}
// One element's, unscaled.
__device__ __forceinline__ double rest_one(const Rest &rest, float p, float d, int at) {
  double r[1][1] = {{scaled(p)}};
  const double y[1][1] = {{scaled(d)}};
  if (rest.draft) rest.of<kMany, 1, 1>(r, y, at, 0);
  else rest.of<kGone, 1, 1>(r, y, at, 0);
  return r[0][0] * kUnscale;
}

// The part that the border lies in, of N whose sums the lanes hold: the first whose
// cumulative sum, from `base` on, passes it, else the last with anything in it (a random
// number of 1), -1 when there is none.  `before`: the sum ahead of it.  Whole warps.
template <int N>
__device__ __forceinline__ int find_part(double mine, double base, double border, double &before) {
  const int lane = threadIdx.x & 31;
  double incl = mine;
#pragma unroll
  for (int o = 1; o < N; o <<= 1) {
    const double x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  const uint32_t some = __ballot_sync(0xffffffffu, mine > 0.0);
  const uint32_t past = __ballot_sync(0xffffffffu, mine > 0.0 && base + incl > border);
  const int part = past ? __ffs(past) - 1 : 31 - __clz(some);
  const double ahead = __shfl_sync(0xffffffffu, incl, part > 0 ? part - 1 : 0);
  before = base + (part > 0 ? ahead : 0.0);
  return part;
}

template <typename P>
__global__ void __launch_bounds__(kVThreads, 2)
verify_tree_kernel(const P *target, const P *draft,
                   const int32_t *tokens, const int32_t *parents,
                   const float *uniforms, int32_t *__restrict__ accept_node,
                   int32_t *__restrict__ accept_len, int32_t *__restrict__ out_tokens, int T,
                   int vocab) {
  __shared__ int32_t s_tok[kVMaxNodes], s_par[kVMaxNodes], s_path[kVMaxNodes], s_gone[kVMaxNodes];
  __shared__ float s_u[kVMaxNodes + 1];
  __shared__ float s_p[kVMaxNodes], s_d[kVMaxNodes];
  __shared__ double s_sum[kVMaxNodes];
  __shared__ double s_warp[kVWarps], s_scan[kVWarps];
  __shared__ double s_tot[2][kVMaxCluster];   // the CTAs' sums, one buffer per parity of the pass
  __shared__ int s_last[kVWarps];

  launch_dependents();
  cg::cluster_group cluster = cg::this_cluster();
  const int CS = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  if (CS > 1) cluster.barrier_arrive();   // the others' shared memory exists once all have started
  const int64_t n = blockIdx.x / CS;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const P *trow = target + n * (T + 1) * (int64_t)vocab;
  const P *drow = draft ? draft + n * T * (int64_t)vocab : nullptr;

  // Slices of whole 16-byte vectors: CTA, then warp.
  constexpr int V = kVec<P>;
  const int piece = ((vocab + CS * kVWarps - 1) / (CS * kVWarps) + V - 1) / V * V;
  const auto bound = [&](int w) {   // start of warp slice w of the whole cluster
    const int64_t b = (int64_t)w * piece;
    return (int)(b < vocab ? b : vocab);
  };

  wait_for_inputs();
  if (tid <= T) s_u[tid] = uniforms[n * (T + 1) + tid];
  if (tid < T) {
    const int x = tokens[n * T + tid];
    int up = parents ? parents[n * T + tid] : tid - 1;
    if (up < -1 || up >= tid) up = -2;        // an empty place: never a successor
    const bool in = x >= 0 && x < vocab;      // a token outside the vocabulary has no probability
    s_tok[tid] = x;
    s_par[tid] = up;
    s_p[tid] = up >= -1 && in ? to_f32(trow[(int64_t)(up + 1) * vocab + x]) : 0.f;
    // (a NaN is zero here, too)
    s_d[tid] = drow && up >= -1 && in ? fmaxf(to_f32(drow[(int64_t)(up + 1) * vocab + x]), 0.f) : 1.f;
  }
  __syncthreads();
  if (CS > 1) cluster.barrier_wait();

  // Every thread of the cluster takes the same decisions from here on.
  Rest rest{drow != nullptr, 0, s_sum, s_gone};
  int cur = -1, count = 0, pass = 0;
  double R = 1.0;
  // Sums of the rest over warps, CTAs and the cluster.
  const auto sum_rest = [&] {
    const int w = rank * kVWarps + warp;
    double x = rest_sum<P>(trow + (int64_t)(cur + 1) * vocab,
                           rest.draft ? drow + (int64_t)min(cur + 1, T - 1) * vocab : nullptr, rest,
                           bound(w), bound(w + 1), lane) * kUnscale;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if (lane == 0) s_warp[warp] = x;
    __syncthreads();
    const int buf = pass++ & 1;
    if (tid < CS) {
      double t[kVWarps];
#pragma unroll
      for (int i = 0; i < kVWarps; ++i) t[i] = s_warp[i];
#pragma unroll
      for (int o = 1; o < kVWarps; o <<= 1)
#pragma unroll
        for (int i = 0; i < kVWarps; i += 2 * o) t[i] += t[i + o];
      cluster.map_shared_rank(&s_tot[buf][0], tid)[rank] = t[0];
    }
    if (CS > 1) cluster.sync();
    else __syncthreads();
    double t = 0.0;
    for (int i = 0; i < CS; ++i) t += s_tot[buf][i];
    return t;
  };

  for (int i = 0; i < T; ++i) {
    if (s_par[i] != cur) continue;
    if (rest.draft && rest.m > 0) R = sum_rest();
    const double r = rest_one(rest, s_p[i], s_d[i], s_tok[i]);
    if (r > 0.0 && (double)s_u[i] * R * (double)s_d[i] < r) {
      if (tid == 0) s_path[count] = i;
      ++count;
      cur = i;
      rest.m = 0;
      R = 1.0;
    } else {
      __syncthreads();   // the rest's lists are read by every thread
      if (tid == 0) {
        s_sum[rest.m] = R;
        s_gone[rest.m] = s_tok[i];
      }
      if (!rest.draft) R -= r;
      ++rest.m;
      __syncthreads();
    }
  }
  double total = sum_rest();
  if (!(total > 0.0) && rest.m > 0) {   // nothing is left: the target's own row
    rest.m = 0;
    total = sum_rest();
  }
  const int buf = (pass - 1) & 1;

  if (rank == 0) {
    if (tid == 0) {
      accept_node[n] = cur;
      accept_len[n] = count;
    }
    for (int i = tid; i <= T; i += kVThreads)
      if (i != count) out_tokens[n * (T + 1) + i] = i < count ? s_tok[s_path[i]] : -1;
  }

  // The CTA, then the warp slice, that the border lies in: the first whose
  // cumulative sum passes it, else (a random number of 1) the last with a part.
  const double border = (double)s_u[T] * total;
  double before;
  const int owner = find_part<kVMaxCluster>(lane < CS ? s_tot[buf][lane] : 0.0, 0.0, border, before);
  if (owner < 0) {   // no token has a probability
    if (rank == 0 && tid == 0) out_tokens[n * (T + 1) + count] = -1;
    return;
  }
  if (owner != rank) return;
  const int wown = max(0, find_part<kVWarps>(lane < kVWarps ? s_warp[lane] : 0.0, before, border, before));
  // The warp slice over the whole CTA: a contiguous piece per thread, its sum,
  // the threads' prefix sums, then the one piece that holds the border.
  const int lo = bound(rank * kVWarps + wown), hi = bound(rank * kVWarps + wown + 1);
  const int each = (hi - lo + kVThreads - 1) / kVThreads;
  const int a = min(lo + tid * each, hi), b = min(a + each, hi);
  const P *p = trow + (int64_t)(cur + 1) * vocab;
  const P *d = rest.draft && rest.m > 0 ? drow + (int64_t)min(cur + 1, T - 1) * vocab : nullptr;
  double mine = 0.0;
  int last = -1;
  for (int i = a; i < b; ++i) {
    const double r = rest_one(rest, to_f32(p[i]), d ? to_f32(d[i]) : 0.f, i);
    mine += r;
    if (r > 0.0) last = i;
  }
  double incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  const int wlast = __reduce_max_sync(0xffffffffu, last);
  if (lane == 31) s_scan[warp] = incl;
  if (lane == 0) s_last[warp] = wlast;
  __syncthreads();
  double all = lane < kVWarps ? s_scan[lane] : 0.0;    // the warps' sums up to each
#pragma unroll
  for (int o = 1; o < kVWarps; o <<= 1) {
    const double x = __shfl_up_sync(0xffffffffu, all, o);
    if (lane >= o) all += x;
  }
  const double ahead = __shfl_sync(0xffffffffu, all, warp > 0 ? warp - 1 : 0);
  const double start = before + (warp > 0 ? ahead : 0.0);
  const int all_last = __reduce_max_sync(0xffffffffu, lane < kVWarps ? s_last[lane] : -1);
  // first token whose cumulative sum passes the border, or the slice's last
  int hit = INT32_MAX;
  double c = start + (incl - mine);
  for (int i = a; i < b; ++i) {
    const double r = rest_one(rest, to_f32(p[i]), d ? to_f32(d[i]) : 0.f, i);
    c += r;
    if (r > 0.0 && c > border) { hit = i; break; }
  }
  hit = __reduce_min_sync(0xffffffffu, hit);
  __syncthreads();
  if (lane == 0) s_last[warp] = hit;
  __syncthreads();
  if (tid == 0) {
    for (int i = 0; i < kVWarps; ++i) hit = min(hit, s_last[i]);
    out_tokens[n * (T + 1) + count] = hit == INT32_MAX ? all_last : hit;
  }
}

}  // namespace

cudaError_t launch_verify_tree(bool bf16, const void *target, const void *draft,
                               const int32_t *tokens, const int32_t *parents,
                               const float *uniforms, int32_t *accept_node, int32_t *accept_len,
                               int32_t *out_tokens, int N, int T, int vocab, int num_sms,
                               cudaStream_t stream) {
  // CTAs per sequence: as many as keep the grid within the two CTAs that an SM holds
  // (a lone sequence is bound by what its few SMs can load) and leave each a 16-byte
  // load per thread, at most the portable cluster size.  Twice as many: 64 chains of
  // 131072 elements 21 us instead of 15, 48 trees of 50257 elements no different.
  int cs = kVMaxCluster;
  const int least = kVThreads * (bf16 ? kVec<__nv_bfloat16> : kVec<float>);
  while (cs > 1 && ((int64_t)N * cs > 2 * (int64_t)num_sms || vocab <= (cs / 2) * least)) cs >>= 1;
  const unsigned grid = (unsigned)((int64_t)N * cs);
  if (bf16)
    return launch_dependent(verify_tree_kernel<__nv_bfloat16>, grid, kVThreads, 0, (unsigned)cs, stream,
                            (const __nv_bfloat16 *)target, (const __nv_bfloat16 *)draft, tokens, parents,
                            uniforms, accept_node, accept_len, out_tokens, T, vocab);
  return launch_dependent(verify_tree_kernel<float>, grid, kVThreads, 0, (unsigned)cs, stream,
                          (const float *)target, (const float *)draft, tokens, parents, uniforms,
                          accept_node, accept_len, out_tokens, T, vocab);
}

}  // namespace kda

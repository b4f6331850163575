// Commit of an accepted path: each sequence's state is moved from before its
// tree of drafted tokens to the state after one of them.
//
// The path state -> ... -> accepted token is found by walking the parents, and
// the recurrence runs along it in FP32,
//
//   A = Diag(alpha_t) S;  y = A^T k_t;  u = beta_t (v_t - y);  S = A + k_t u^T
//
// The state crosses HBM once in each direction however long the path is, which
// is what bounds the kernel: 128 KB per (sequence, head) at D = 128 against
// 3 D^2 FP32 operations per token, so about twelve tokens hide behind the
// traffic.  Columns of S do not mix, so a warp owns 16 whole columns: its lanes
// are 4 float4 column groups x 8 row residues, the reduction over rows stays
// inside the warp, and the warps run the whole path without a block barrier
// except where the next group of tokens is staged.
#include "kda_common.cuh"

namespace kda {
namespace {

constexpr int kGroup = 8;        // tokens staged at a time

// Value columns of one CTA.
template <int DV> constexpr int kCols = DV < 64 ? DV : 64;

template <int DK, int DV, typename TIn>
__global__ void __launch_bounds__(2 * kCols<DV>, 640 / (2 * kCols<DV>))
tree_commit_kernel(const TIn *__restrict__ k, const TIn *__restrict__ v,
                   const float *__restrict__ g, const float *__restrict__ beta,
                   const float *state, float *state_out, const int32_t *__restrict__ parents,
                   const int32_t *__restrict__ accept_node, int T, int H) {
  constexpr int COLS = kCols<DV>, PARTS = DV / COLS;
  constexpr int THREADS = 2 * COLS;           // 16 columns per warp
  constexpr int V4 = DV / 4;
  constexpr int ROWS = DK / 8;                // float4s per thread
  __shared__ float2 s_ak[kGroup][DK];         // (alpha, k)
  __shared__ float s_v[kGroup][COLS];
  __shared__ float s_b[kGroup];

  const int64_t unit = blockIdx.x / PARTS;
  const int part = blockIdx.x % PARTS;
  const int n = (int)(unit / H), h = (int)(unit % H);
  const int tid = threadIdx.x, lane = tid & 31;
  const int cg = 4 * (tid >> 5) + (lane & 3);  // float4 column
  const int ks = lane >> 2;                    // rows ks, ks + 8, ...

  const int32_t node = __ldg(accept_node + n);
  int32_t up0 = -2, up1 = -2;                  // predecessors of places lane and lane + 32
  if (parents) {
    if (lane < T) up0 = __ldg(parents + (int64_t)n * T + lane);
    if (lane + 32 < T) up1 = __ldg(parents + (int64_t)n * T + lane + 32);
  }
  // In place, a sequence without an accepted token is not touched; otherwise the
  // state is loaded before anything is known of the path.
  const bool named = node >= 0 && node < T;
  if (state_out == state && !named) return;
  const float4 *src = reinterpret_cast<const float4 *>(state) + unit * (DK * V4) + part * (COLS / 4);
  float4 *dst = reinterpret_cast<float4 *>(state_out) + unit * (DK * V4) + part * (COLS / 4);
  float4 s[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) s[i] = __ldcs(src + (ks + 8 * i) * V4 + cg);

  // The path as a set of places (a token's place is above its predecessor's), found
  // by every warp for itself: no shared memory, no barrier.
  unsigned long long path = 0;
  if (named && parents) {
    for (int i = node; i >= 0;) {              // at most T steps: i decreases
      path |= 1ull << i;
      const int up = __shfl_sync(0xffffffffu, i < 32 ? up0 : up1, i & 31);
      if (up < -1 || up >= i) { path = 0; break; }   // it holds an empty place
      i = up;
    }
  } else if (named) {
    path = ~0ull >> (63 - node);
  }
  if (state_out == state && path == 0) return;

  const int64_t row0 = (int64_t)n * T * H + h;
  for (bool first = true; path != 0; first = false) {
    const int m = min(kGroup, __popcll(path));
    if (!first) __syncthreads();
    const unsigned long long all = path;
#pragma unroll
    for (int e0 = 0; e0 < DK + COLS; e0 += THREADS) {
      const int e = e0 + tid;
      unsigned long long rest = all;
#pragma unroll 4
      for (int j = 0; j < kGroup; ++j) {
        if (j < m && e < DK + COLS) {
          const int64_t row = row0 + (int64_t)(__ffsll(rest) - 1) * H;
          if (e < DK) s_ak[j][e] = make_float2(expf(g[row * DK + e]), to_f32(k[row * DK + e]));
          else s_v[j][e - DK] = to_f32(v[row * DV + part * COLS + (e - DK)]);
          if (e == 0) s_b[j] = beta[row];
        }
        rest &= rest - 1;
      }
      path = rest;
    }
    __syncthreads();
    for (int j = 0; j < m; ++j) {
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < ROWS; ++i) {
        const float2 ak = s_ak[j][ks + 8 * i];
        s[i].x *= ak.x; s[i].y *= ak.x; s[i].z *= ak.x; s[i].w *= ak.x;
        y.x += ak.y * s[i].x; y.y += ak.y * s[i].y; y.z += ak.y * s[i].z; y.w += ak.y * s[i].w;
      }
      // Sum over the 8 row residues: each step halves the columns a lane
      // keeps, so a lane ends with one column (7 shuffles, not 12).
      const bool b4 = lane & 16, b3 = lane & 8;
      float p0 = b4 ? y.z : y.x, p1 = b4 ? y.w : y.y;
      p0 += __shfl_xor_sync(0xffffffffu, b4 ? y.x : y.z, 16);
      p1 += __shfl_xor_sync(0xffffffffu, b4 ? y.y : y.w, 16);
      float w = b3 ? p1 : p0;
      w += __shfl_xor_sync(0xffffffffu, b3 ? p0 : p1, 8);
      w += __shfl_xor_sync(0xffffffffu, w, 4);
      const float u = s_b[j] * (s_v[j][4 * cg + (b4 ? 2 : 0) + (b3 ? 1 : 0)] - w);
      const float u8 = __shfl_xor_sync(0xffffffffu, u, 8);
      const float ua = b3 ? u8 : u, ub = b3 ? u : u8;
      const float ua16 = __shfl_xor_sync(0xffffffffu, ua, 16);
      const float ub16 = __shfl_xor_sync(0xffffffffu, ub, 16);
      const float4 u4 = b4 ? make_float4(ua16, ub16, ua, ub) : make_float4(ua, ub, ua16, ub16);
#pragma unroll
      for (int i = 0; i < ROWS; ++i) {
        const float kc = s_ak[j][ks + 8 * i].y;
        s[i].x += kc * u4.x; s[i].y += kc * u4.y; s[i].z += kc * u4.z; s[i].w += kc * u4.w;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < ROWS; ++i) __stcs(dst + (ks + 8 * i) * V4 + cg, s[i]);
}

template <typename TIn>
cudaError_t launch_t(int dk, int dv, const void *k, const void *v, const float *g,
                     const float *beta, const float *state, float *state_out,
                     const int32_t *parents, const int32_t *accept_node, int T, int64_t units,
                     int H, cudaStream_t stream) {
#define KDA_TC(DK_, DV_)                                                                         \
  if (dk == DK_ && dv == DV_) {                                                                  \
    tree_commit_kernel<DK_, DV_, TIn><<<(unsigned)(units * (DV_ / kCols<DV_>)), 2 * kCols<DV_>, 0, stream>>>( \
        (const TIn *)k, (const TIn *)v, g, beta, state, state_out, parents, accept_node, T, H);  \
    return cudaGetLastError();                                                                   \
  }
  KDA_TC(32, 32) KDA_TC(32, 64) KDA_TC(32, 128)
  KDA_TC(64, 32) KDA_TC(64, 64) KDA_TC(64, 128)
  KDA_TC(128, 32) KDA_TC(128, 64) KDA_TC(128, 128)
#undef KDA_TC
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_tree_commit(int dtype, int dk, int dv, const void *k, const void *v,
                               const float *g, const float *beta, const float *state,
                               float *state_out, const int32_t *parents,
                               const int32_t *accept_node, int T, int64_t units, int H,
                               cudaStream_t stream) {
  if (dtype == KDA_DTYPE_BF16)
    return launch_t<__nv_bfloat16>(dk, dv, k, v, g, beta, state, state_out, parents, accept_node,
                                   T, units, H, stream);
  return launch_t<float>(dk, dv, k, v, g, beta, state, state_out, parents, accept_node, T, units,
                         H, stream);
}

}  // namespace kda

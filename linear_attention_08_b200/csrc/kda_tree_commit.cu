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
// 3 D^2 FP32 operations per token.  Columns of S do not mix, so a CTA takes up to
// 64 columns of a unit, a warp 16 of them: its lanes are 4 float4 column groups x 8
// row residues, and the reduction over rows stays inside the warp.
//
// CTAs are persistent and work on the next unit's loads while they compute: every
// thread copies the elements it will hold into shared memory (its own slots, no
// barrier), takes them into registers when the unit begins, and starts the next
// unit's copies into the same slots.  accept_node and parents are read two units
// ahead, the path's first rows one unit ahead.  (Without this a CTA waited in turn
// for accept_node, the state and the rows: 512 x 32 units in 416 us.  With it 354, 94 %
// of the copy rate, in a burst; 366 to 384 under the power cap.)
#include "kda_common.cuh"
#include "kda_launch.cuh"

namespace kda {
namespace {

constexpr int kGroup = 4;        // tokens staged at a time

template <int DK, int DV, typename TIn> struct CommitCfg {
  static constexpr int COLS = DV < 64 ? DV : 64, PARTS = DV / COLS;   // value columns of a CTA
  static constexpr int THREADS = 2 * COLS;      // 16 columns per warp
  static constexpr int ROWS = DK / 8;           // float4s per thread
  // 16-byte pieces of one token's g, k, v
  static constexpr int CG = DK / 4, CK = DK * (int)sizeof(TIn) / 16, CV = COLS * (int)sizeof(TIn) / 16;
  static constexpr int CT = CG + CK + CV;
  // CTAs per SM by shared memory and by registers (the elements and about 56 more)
  static constexpr int SMEM = DK * COLS * 4 + kGroup * (DK * 16 + COLS * 4 + CT * 16 + 8);
  static constexpr int FIT = 227 * 1024 / (SMEM + 1024);
  static constexpr int REGS = 65536 / (THREADS * (4 * ROWS + 56));
  static constexpr int PER_SM = FIT < REGS ? FIT : REGS;
};

__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// Two FP32 numbers per register pair: Blackwell's packed products take one instruction
// for both.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 pack2(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack2(f32x2 x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}

// Place of the j-th token of a path, from the state on (a token's place is above its
// predecessor's).
__device__ __forceinline__ int nth(unsigned long long path, int j) {
  for (; j > 0; --j) path &= path - 1;
  return __ffsll(path) - 1;
}

template <int DK, int DV, typename TIn>
__global__ void __launch_bounds__(CommitCfg<DK, DV, TIn>::THREADS, CommitCfg<DK, DV, TIn>::PER_SM)
tree_commit_kernel(const TIn *k, const TIn *v, const float *g, const float *beta,
                   const float *state, float *state_out, const int32_t *parents,
                   const int32_t *accept_node, int T, int H, int64_t items) {
  using C = CommitCfg<DK, DV, TIn>;
  constexpr int COLS = C::COLS, PARTS = C::PARTS, THREADS = C::THREADS, ROWS = C::ROWS;
  constexpr int V4 = DV / 4;
  __shared__ ulonglong2 s_state[ROWS][THREADS];   // the next unit's elements
  __shared__ uint4 s_raw[kGroup][C::CT];      // its path's first rows: g, k, v
  __shared__ float s_rb[kGroup];              // and beta
  __shared__ float4 s_ak[kGroup][DK];         // (alpha, alpha, k, k): pairs as they are used
  __shared__ float s_v[kGroup][COLS];
  __shared__ float s_b[kGroup];

  const int tid = threadIdx.x, lane = tid & 31;
  const int cg = 4 * (tid >> 5) + (lane & 3);  // float4 column
  const int ks = lane >> 2;                    // rows ks, ks + 8, ...
  const bool in_place = state_out == state;
  const int64_t G = gridDim.x;

  // An item is the columns of one CTA: PARTS of them per unit.
  int node = -1, up0 = -2, up1 = -2;           // predecessors of places lane and lane + 32
  const auto read_ahead = [&](int64_t item) {
    if (item >= items) return;
    const int64_t n = item / PARTS / H;
    node = accept_node[n];
    if (parents) {
      if (lane < T) up0 = parents[n * T + lane];
      if (lane + 32 < T) up1 = parents[n * T + lane + 32];
    }
  };
  // The path as a set of places, found by every warp for itself.
  const auto find_path = [&] {
    unsigned long long path = 0;
    if (node < 0 || node >= T) return path;
    if (!parents) return ~0ull >> (63 - node);
    for (int i = node; i >= 0;) {              // at most T steps: i decreases
      path |= 1ull << i;
      const int up = __shfl_sync(0xffffffffu, i < 32 ? up0 : up1, i & 31);
      if (up < -1 || up >= i) return 0ull;     // it holds an empty place
      i = up;
    }
    return path;
  };
  const auto elements = [&](int64_t item) {    // this thread's, in float4s
    return item / PARTS * (DK * V4) + item % PARTS * (COLS / 4) + (int64_t)ks * V4 + cg;
  };
  const auto first_row = [&](int64_t item) {
    const int64_t unit = item / PARTS;
    return unit / H * T * H + unit % H;
  };
  const auto start_state = [&](int64_t item) {
    const float4 *src = reinterpret_cast<const float4 *>(state) + elements(item);
#pragma unroll
    for (int i = 0; i < ROWS; ++i) copy16(smem_u32(&s_state[i][tid]), src + i * 8 * V4);
  };
  const auto start_rows = [&](int64_t item, unsigned long long path) {
    const int m = min(kGroup, __popcll(path));
    const int64_t row0 = first_row(item);
    for (int e = tid; e < m * C::CT; e += THREADS) {
      const int j = e / C::CT, c = e % C::CT;
      const int64_t row = row0 + (int64_t)nth(path, j) * H;
      const void *from = c < C::CG ? static_cast<const void *>(g + row * DK + c * 4)
                         : c < C::CG + C::CK
                             ? static_cast<const void *>(k + row * DK + (c - C::CG) * (16 / (int)sizeof(TIn)))
                             : static_cast<const void *>(v + row * DV + item % PARTS * COLS +
                                                         (c - C::CG - C::CK) * (16 / (int)sizeof(TIn)));
      copy16(smem_u32(&s_raw[j][c]), from);
    }
    if (tid < m) copy4(smem_u32(&s_rb[tid]), beta + row0 + (int64_t)nth(path, tid) * H);
  };

  launch_dependents();
  wait_for_inputs();
  int64_t item = blockIdx.x;
  read_ahead(item);
  if (!in_place) start_state(item);            // nothing of the path decides whether it is read
  unsigned long long path = find_path();
  start_rows(item, path);
  if (in_place && path != 0) start_state(item);
  read_ahead(item + G);
  for (; item < items; item += G) {
    const int64_t next = item + G;
    const unsigned long long next_path = next < items ? find_path() : 0ull;
    read_ahead(next + G);
    const bool active = path != 0 || !in_place;
    ulonglong2 s[ROWS];
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();                           // the others' copies of rows; the last unit's are used up
    if (active) {
#pragma unroll
      for (int i = 0; i < ROWS; ++i) s[i] = s_state[i][tid];
    }
    int m = min(kGroup, __popcll(path));
    for (int e = tid; e < m * DK; e += THREADS) {
      const int j = e / DK, c = e % DK;
      const float al = expf(reinterpret_cast<const float *>(&s_raw[j][0])[c]);
      const float kc = to_f32(reinterpret_cast<const TIn *>(&s_raw[j][C::CG])[c]);
      s_ak[j][c] = make_float4(al, al, kc, kc);
    }
    for (int e = tid; e < m * COLS; e += THREADS)
      s_v[e / COLS][e % COLS] = to_f32(reinterpret_cast<const TIn *>(&s_raw[e / COLS][C::CG + C::CK])[e % COLS]);
    if (tid < m) s_b[tid] = s_rb[tid];
    // Every warp has read the path for itself, and a caller who rewrites accept_node or parents
    // while the kernel runs makes them disagree; what barriers depend on is decided together.
    bool more = __syncthreads_or(__popcll(path) > kGroup);
    if (next < items) {
      if (!in_place || next_path != 0) start_state(next);
      start_rows(next, next_path);
    }
    for (;;) {
      for (int j = 0; j < m; ++j) {
        f32x2 ya = 0, yb = 0;
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
          const ulonglong2 ak = *reinterpret_cast<const ulonglong2 *>(&s_ak[j][ks + 8 * i]);
          s[i].x = mul2(s[i].x, ak.x);
          s[i].y = mul2(s[i].y, ak.x);
          ya = fma2(ak.y, s[i].x, ya);
          yb = fma2(ak.y, s[i].y, yb);
        }
        const float2 y01 = unpack2(ya), y23 = unpack2(yb);
        const float4 y = make_float4(y01.x, y01.y, y23.x, y23.y);
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
        const f32x2 u01 = b4 ? pack2(ua16, ub16) : pack2(ua, ub);
        const f32x2 u23 = b4 ? pack2(ua, ub) : pack2(ua16, ub16);
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
          const f32x2 kc = reinterpret_cast<const ulonglong2 *>(&s_ak[j][ks + 8 * i])->y;
          s[i].x = fma2(kc, u01, s[i].x);
          s[i].y = fma2(kc, u23, s[i].y);
        }
      }
      // the path's further tokens, read when they are needed
      if (!more) break;
      for (int j = 0; j < m; ++j) path &= path - 1;
      m = min(kGroup, __popcll(path));
      const int64_t row0 = first_row(item);
      __syncthreads();
      for (int e = tid; e < m * (DK + COLS); e += THREADS) {
        const int j = e / (DK + COLS), c = e % (DK + COLS);
        const int64_t row = row0 + (int64_t)nth(path, j) * H;
        if (c < DK) {
          const float al = expf(g[row * DK + c]), kc = to_f32(k[row * DK + c]);
          s_ak[j][c] = make_float4(al, al, kc, kc);
        } else s_v[j][c - DK] = to_f32(v[row * DV + item % PARTS * COLS + (c - DK)]);
        if (c == 0) s_b[j] = beta[row];
      }
      more = __syncthreads_or(__popcll(path) > kGroup);
    }
    if (active) {
      float4 *dst = reinterpret_cast<float4 *>(state_out) + elements(item);
#pragma unroll
      for (int i = 0; i < ROWS; ++i) {
        const float2 a = unpack2(s[i].x), b = unpack2(s[i].y);
        __stcs(dst + i * 8 * V4, make_float4(a.x, a.y, b.x, b.y));
      }
    }
    path = next_path;
  }
}

template <typename TIn>
cudaError_t launch_t(int dk, int dv, const void *k, const void *v, const float *g,
                     const float *beta, const float *state, float *state_out,
                     const int32_t *parents, const int32_t *accept_node, int T, int64_t units,
                     int H, cudaStream_t stream) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0)
    sms = 148;
#define KDA_TC(DK_, DV_)                                                                          \
  if (dk == DK_ && dv == DV_) {                                                                   \
    using C = CommitCfg<DK_, DV_, TIn>;                                                           \
    const int64_t items = units * C::PARTS, slots = (int64_t)C::PER_SM * sms;                     \
    const cudaError_t e = cudaFuncSetAttribute(tree_commit_kernel<DK_, DV_, TIn>,                 \
                                               cudaFuncAttributePreferredSharedMemoryCarveout,    \
                                               (int)cudaSharedmemCarveoutMaxShared);              \
    if (e != cudaSuccess) return e;                                                               \
    return launch_dependent(tree_commit_kernel<DK_, DV_, TIn>,                                    \
                            (unsigned)(items < slots ? items : slots), C::THREADS, 0, 1, stream,  \
                            (const TIn *)k, (const TIn *)v, g, beta, state, state_out, parents,   \
                            accept_node, T, H, items);                                            \
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

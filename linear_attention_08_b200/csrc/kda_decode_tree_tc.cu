// KDA outputs of a tree of drafted tokens on the 5th-generation tensor cores
// (sm_100a), for BF16 q/k/v with D_k = D_v = 128; other shapes run
// kda_decode_tree.cu, whose header has the formulas (Gam, Kt, Qt, Kh, L, P).
//
// With u_t = (Vn)_t, KK_ts = Kt_t . Kh_s and X = [Kt; Qt], for tokens s ~ t:
//
//   D3 = g^T A^T, A_ts = [s ~ t]     Gam, transposed              (M = 128, N = TP, K = TP)
//   D2 = X Kh^T                      KK and P before the mask     (M = 128, N = TP, K = 128)
//   D1 = S0^T X^T                    columns: Kt S0, then Qt S0   (M = 128, N = 2 TP, K = 128)
//   u_t = beta_t (v_t - D1[K_t] - sum_{s < t} KK_ts u_s)
//   D1 += U [KK; P]^T                16 tokens at a time: what later tokens need, and the outputs
//
// All but the third line are products of the tensor cores.  A thread owns one value
// column (one lane of the accumulators) and finds u of 16 tokens in registers, with KK
// broadcast from shared memory.  The products are TF32 with FP32 accumulation, operands
// rounded to about the nearest (2^-10.5 at most, 2^-11.7 rms, below the 2^-9 of the
// outputs' rounding); g goes in as two TF32 terms (2^-22 of it is lost).
//
// S0^T is an A operand and lies in tensor memory: a lane is a value column and reads
// its column of the row-major state from shared memory without bank conflicts, so no
// operand tile of the state is formed.  The state's buffer is free again as soon as it
// is in tensor memory, at the start of a unit, and the next unit's 64 KB arrive while
// this one is computed.  A producer warp runs ahead: it finds the sets of ancestors and
// brings the rows of tokens that are there; those of empty places are filled with zeros.
//
// One CTA per unit is launched, and a CTA that runs takes over those that have not
// started (launch control): units of ragged trees differ in cost by a factor of two.
// TP = 16: two CTAs of 128 + 32 threads per SM, so that one computes while the other waits
// for a product.  TP = 32, 64: these buffers leave room for one CTA, of 256 + 32 threads; X
// holds 32 tokens, and the second 32 take the place of g.
//
// 512 x 32 heads x 16 places: 237 us in a burst, 226 at the copy rate (264 to 288 under the
// power cap).  Units whose decays leave +-80 form KK and P pair by pair (deep trees with
// gates near -5), which is what they then spend their time on: 128 x 32 heads x 61 places
// 1525 us instead of 259.
#include "kda_common.cuh"
#include "kda_launch.cuh"
#include "kda_tc_util.cuh"
#include "kda_tf32.cuh"
#include "kda_tma.cuh"

namespace kda {
namespace {

constexpr int kD = 128;
constexpr int kBlk = 16;                  // tokens solved in registers at a time
constexpr float kGamBound = 80.f;         // beyond: KK and P pair by pair
constexpr float kFactorBound = 1e36f;
// At Gam = -80 an element of Kt is 1.8e-35 of k's, and rows of q or k of size 10^-5 would be
// subnormal numbers.  So X holds Kt and Qt times 2^24, Kh and S0^T are times 2^-24, and the
// products come out as they are: exact, but for elements of S0 below 2^-102 and rows above
// 10^31.
constexpr float kLift = 24.f, kSink = 0x1p-24f;

// TP: token places of the buffers.
template <int TP> struct TreeTc {
  static constexpr int WG = TP == 16 ? 1 : 2;            // warpgroups that compute
  static constexpr int WORKERS = 128 * WG;
  static constexpr int THREADS = WORKERS + 32;
  static constexpr int TH = TP < 32 ? TP : 32;           // tokens in X at a time (a part)
  static constexpr int NH = TP / TH;
  static constexpr int OB = TP / kBlk / WG;              // blocks of outputs per warpgroup
  static constexpr int XR = 2 * TH;                      // rows of X
  static constexpr int ROWS = 2 * TP;                    // rows of [KK; P], part by part
  // shared memory, bytes
  static constexpr uint32_t SF = 0;                      // the state
  static constexpr uint32_t X = SF + kD * kD * 4;        // [Kt; Qt] of a part: K-major tile
  static constexpr uint32_t AN = X;                      // before: A of the paths, K-major tile
  static constexpr uint32_t KH = X + XR * kD * 4;        // Kh: K-major tile of TP rows
  static constexpr uint32_t KP = NH == 1 ? KH : X;       // after: [KK; P], K-major tile
  static constexpr uint32_t RG = KH + TP * kD * 4;       // rows of g, q, k, v
  static constexpr uint32_t X1 = RG;                     // after: X of part 1
  static constexpr uint32_t RQ = RG + TP * 512;
  static constexpr uint32_t RK = RQ + TP * 256;
  static constexpr uint32_t RV = RK + TP * 256;
  static constexpr uint32_t ANC = RV + TP * 256;         // two units' ancestor sets,
  static constexpr uint32_t ALL = ANC + 2 * TP * 8;      // sets of tokens,
  static constexpr uint32_t PAR = ALL + 2 * 8;           // predecessors
  static constexpr uint32_t BETA = PAR + 2 * TP * 4;     // and beta
  static constexpr uint32_t NEXT = BETA + 2 * TP * 4;    // answer of the launch control
  static constexpr uint32_t ROW = NEXT + 16;             // two units' first rows, -1 at the end
  static constexpr uint32_t WIDE = ROW + 16;
  static constexpr uint32_t QUIT = WIDE + 8;
  static constexpr uint32_t SLOT = QUIT + 4;
  static constexpr uint32_t BAR = SLOT + 4;
  static constexpr uint32_t TOTAL = BAR + 14 * 8;
  static_assert(X % 1024 == 0 && KH % 1024 == 0 && NEXT % 16 == 0 && BAR % 8 == 0, "alignment");
  static_assert(ROWS * 128 * ((TP + 31) / 32) <= (NH == 1 ? TP : XR) * kD * 4, "[KK; P]");
  static_assert(NH == 1 || (RG % 1024 == 0 && XR * kD * 4 <= TP * 512), "X in g's place");
  static_assert(TP * 128 * ((TP + 31) / 32) <= XR * kD * 4, "A in X's place");
  // the A operand of D2 reads 128 rows, those past X into lanes that nobody reads
  static_assert((NH == 1 ? X : X1) + (kD / 32 - 1) * XR * 128 + 128 * 128 <= TOTAL, "rows past the operand");
  // tensor memory, columns
  static constexpr uint32_t S = 0;                       // S0^T
  static constexpr uint32_t D1 = 128;                    // part by part: Kt S0, Qt S0
  static constexpr uint32_t AG = D1 + ROWS;              // g: high terms, low terms
  static constexpr uint32_t D2 = AG;                     // after: part 0 (TH columns), part 1 (TP)
  static constexpr uint32_t D3 = AG + 2 * TP;
  static constexpr uint32_t U = D3 + TP;
  static constexpr uint32_t COLS = U + kBlk <= 256 ? 256 : 512;
  static_assert(U + kBlk <= 512 && (NH == 1 ? TH : TH + TP) <= 2 * TP, "tensor memory");
};

enum TreeBar {
  kFullQkg, kFullV, kFullS, kEmptyQkg, kEmptyV, kEmptyS, kMmaG, kMmaA, kMmaB,
  kMmaA1, kMmaB1, kMmaU, kMmaO, kNext, kBars
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(valid ? 16 : 0)
               : "memory");
}
// An arrival once the calling thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// Ask for a CTA of this grid that has not started; it then never does, and its work is
// the caller's.  The answer is 16 bytes, announced on an mbarrier.
__device__ __forceinline__ void ask_next(uint32_t answer, uint32_t bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
          answer),
      "r"(bar)
      : "memory");
}
// Its number, or -1 when none is left (after which nothing more may be asked).
__device__ __forceinline__ int read_next(uint32_t answer) {
  int r;
  asm volatile(
      "{\n\t.reg .b128 a;\n\t.reg .pred p;\n\t"
      "mov.b32 %0, -1;\n\t"
      "ld.shared.b128 a, [%1];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, a;\n\t}"
      : "=&r"(r)
      : "r"(answer)
      : "memory");
  return r;
}

// Instruction descriptor of kind::tf32, both operands K-major: as idesc_bf16 with
// format 2 (TF32) of a and b.
constexpr uint32_t idesc_tf32(int M, int N) {
  return (1u << 4) | (2u << 7) | (2u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void mma_tf32_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::tf32 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_tf32_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::tf32 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Descriptor of K-step s (8 columns) of a K-major tile from the one of its first step:
// the steps lie at fixed distances.
__device__ __forceinline__ uint64_t step_desc(uint64_t first, int rows, int s) {
  return first + (uint64_t)(((s >> 2) * rows * 128 + (s & 3) * 32) >> 4);
}

// Byte offset of 32-bit element (row, col) of a K-major tile with `rows` rows.
__device__ __forceinline__ uint32_t tile32(int rows, int row, int col) {
  return (uint32_t)((col >> 5) * rows * 128 + row * 128 + ((((col & 31) >> 2) ^ (row & 7)) << 4) +
                    (col & 3) * 4);
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// Barrier of the computing threads with a common "or".
template <int N> __device__ __forceinline__ bool bar_or(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x), "n"(N)
      : "memory");
  return r != 0;
}

template <int TP>
__global__ void __launch_bounds__(TreeTc<TP>::THREADS, TP == 16 ? 2 : 1)
decode_tree_tc_kernel(const __nv_bfloat16 *q, const __nv_bfloat16 *k, const __nv_bfloat16 *v,
                      const float *g, const float *beta, const float *state,
                      const int32_t *parents, __nv_bfloat16 *__restrict__ out, int T, int H,
                      int32_t *dev_status, uint64_t wait_ns) {
  using C = TreeTc<TP>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t sraw = smem_u32(smem_raw);
  const uint32_t sb = (sraw + 1023u) & ~1023u;
  uint8_t *sp = smem_raw + (sb - sraw);
  uint64_t *bars = reinterpret_cast<uint64_t *>(sp + C::BAR);
  volatile int *s_quit = reinterpret_cast<int *>(sp + C::QUIT);
  volatile int *s_wide = reinterpret_cast<int *>(sp + C::WIDE);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);   // known to be uniform
  const auto bar_at = [&](int b) { return sb + C::BAR + 8 * b; };

  if (tid == 0) {
    for (int i = 0; i < kBars; ++i)   // rows: a lane's copies each, and the masks
      mbar_init(bars + i, i == kEmptyQkg || i == kEmptyV || i == kEmptyS ? C::WORKERS / 32
                          : i == kFullQkg || i == kFullV               ? 33
                                                                       : 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    *s_quit = 0;
    s_wide[0] = s_wide[1] = 0;
  }
  // Tensor memory is taken after the kernel ahead has ended, and before the next one may
  // start: a block that held some while it waits could keep it from the one it waits for.
  wait_for_inputs();
  if (warp == 0) tc::tmem_alloc(sb + C::SLOT, C::COLS);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  launch_dependents();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t *>(sp + C::SLOT), 0);

  if (warp == C::WORKERS / 32) {
    // ------------------------------------------------------------ producer
    // A wait ends when the computing threads have given up, too.
    const auto wait = [&](int b, uint32_t phase) {
      if (mbar_try_wait(bars + b, phase)) return true;
      const uint64_t t0 = globaltimer();
      while (!mbar_try_wait(bars + b, phase))
        if (*s_quit || globaltimer() - t0 > wait_ns) return false;
      return true;
    };
    const auto load_state = [&](int64_t u) {
      if (lane == 0) {
        mbar_expect_tx(bar_at(kFullS), kD * kD * 4);
        bulk_load(sb + C::SF, state + (size_t)u * kD * kD, kD * kD * 4, bar_at(kFullS));
      }
    };
    constexpr int E = TP > 32 ? 2 : 1;    // places per lane
    volatile int64_t *s_row = reinterpret_cast<int64_t *>(sp + C::ROW);
    int u = blockIdx.x;
    uint32_t states = 0;                  // copies of states begun
    int asked = -1;                       // phase of an answer to come
    bool ended = false;
    for (uint32_t i = 0;; ++i) {
      // the state's buffer is free once the unit before has it in tensor memory (and the
      // one before that, which had this set of masks, is done)
      const int buf = i & 1;
      if (i > 0 && !wait(kEmptyS, (i - 1) & 1)) break;
      const int n = u / H, h = u % H;
      const int64_t row0 = (int64_t)n * T * H + h;
      if (lane == 0) s_row[buf] = row0;
      load_state(u);
      states = i + 1;
      if (lane == 0) {
        mbar_expect_tx(bar_at(kNext), 16);
        ask_next(sb + C::NEXT, bar_at(kNext));
      }
      asked = i & 1;
      // ancestors by pointer doubling: after the step of size d every mask holds the
      // last 2 d places of its path
      int up[E], jump[E];
      unsigned long long m[E];
      float bt[E];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int t = lane + 32 * e;
        up[e] = -2;
        bt[e] = 0.f;
        if (t < T) {
          up[e] = parents ? parents[(int64_t)n * T + t] : t - 1;
          bt[e] = beta[row0 + (int64_t)t * H];
        }
      }
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int t = lane + 32 * e;
        if (up[e] < -1 || up[e] >= t) up[e] = -2;
        jump[e] = up[e];
        m[e] = 1ull << t;
      }
      for (int d = 1; d < T; d <<= 1) {
        unsigned long long mo[E];
        int jo[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int src = jump[e] & 31;
          mo[e] = __shfl_sync(0xffffffffu, m[0], src);
          jo[e] = __shfl_sync(0xffffffffu, jump[0], src);
          if (E > 1) {
            const unsigned long long m1 = __shfl_sync(0xffffffffu, m[E - 1], src);
            const int j1 = __shfl_sync(0xffffffffu, jump[E - 1], src);
            if (jump[e] >= 32) { mo[e] = m1; jo[e] = j1; }
          }
        }
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (jump[e] >= 0) { m[e] |= mo[e]; jump[e] = jo[e]; }
      }
      bool live[E];
      unsigned long long all = 0;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        live[e] = jump[e] == -1;          // else the path ends in an empty place
        all |= (unsigned long long)__ballot_sync(0xffffffffu, live[e]) << (32 * e);
      }
      const int rows = all ? (64 - __clzll(all) + kBlk - 1) / kBlk * kBlk : 0;
      // the rows' buffers: free once the unit before has formed its operands
      if (i > 0 && !wait(kEmptyQkg, (i - 1) & 1)) break;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int t = lane + 32 * e;
        if (t < TP) {
          reinterpret_cast<unsigned long long *>(sp + C::ANC)[buf * TP + t] = live[e] ? m[e] : 0ull;
          reinterpret_cast<int *>(sp + C::PAR)[buf * TP + t] = live[e] ? up[e] : -2;
          reinterpret_cast<float *>(sp + C::BETA)[buf * TP + t] = live[e] ? bt[e] : 0.f;
        }
      }
      if (lane == 0) reinterpret_cast<unsigned long long *>(sp + C::ALL)[buf] = all;
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + kFullQkg);
      // 16 bytes per lane: a row of g, then rows of k and q at once
      const bool isq = lane >= 16;
      const __nv_bfloat16 *kq = (isq ? q : k) + 8 * (lane & 15);
      const uint32_t dkq = sb + (isq ? C::RQ : C::RK) + 16 * (lane & 15);
#pragma unroll 4
      for (int t = 0; t < rows; ++t) {
        const bool there = (all >> t) & 1;
        const int64_t at = there ? (row0 + (int64_t)t * H) * kD : 0;
        cp_async16(sb + C::RG + t * 512 + 16 * lane, g + at + 4 * lane, there);
        cp_async16(dkq + t * 256, kq + at, there);
      }
      cp_async_arrive(bar_at(kFullQkg));
      if (i > 0 && !wait(kEmptyV, (i - 1) & 1)) break;
      if (lane == 0) mbar_arrive(bars + kFullV);
#pragma unroll 4
      for (int t0 = 0; t0 < rows; t0 += 2) {   // two rows at once
        const int t = t0 + isq;
        const bool there = (all >> t) & 1;
        const int64_t at = there ? (row0 + (int64_t)t * H) * kD : 0;
        cp_async16(sb + C::RV + t * 256 + 16 * (lane & 15), v + at + 8 * (lane & 15), there);
      }
      cp_async_arrive(bar_at(kFullV));
      // the next unit, asked for a unit ago
      if (!wait(kNext, i & 1)) break;
      asked = -1;
      u = read_next(sb + C::NEXT);
      tc::fence_smem_to_async();          // read before it is written again
      __syncwarp();
      if (u < 0) {
        ended = wait(kEmptyS, i & 1);   // (so this unit's state has arrived)
        if (ended && lane == 0) {
          s_row[buf ^ 1] = -1;
          mbar_arrive(bars + kFullS);
        }
        break;
      }
    }
    // copies in flight end before the memory is released
    cp_async_wait_all();
    if (!ended) wait_timed(bars + kFullS, (states - 1) & 1, wait_ns);
    if (asked >= 0) wait_timed(bars + kNext, (uint32_t)asked, wait_ns);
  } else {
    // ------------------------------------------------------------ computing threads
    const int hw = warp >> 2;                        // warpgroup
    const int col = tid & 127;                       // value column = lane of tensor memory
    const uint32_t tl = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const float *rg = reinterpret_cast<const float *>(sp + C::RG) + col;
    const __nv_bfloat16 *rq = reinterpret_cast<const __nv_bfloat16 *>(sp + C::RQ) + col;
    const __nv_bfloat16 *rk = reinterpret_cast<const __nv_bfloat16 *>(sp + C::RK) + col;
    const __nv_bfloat16 *rv = reinterpret_cast<const __nv_bfloat16 *>(sp + C::RV) + col;
    const uint64_t x_desc[2] = {tc::desc_kmajor(sb + C::X, C::XR, 0), tc::desc_kmajor(sb + C::X1, C::XR, 0)};
    const uint64_t an_desc = tc::desc_kmajor(sb + C::AN, TP, 0);
    const uint64_t kh_desc = tc::desc_kmajor(sb + C::KH, TP, 0);
    const uint64_t kp_desc = tc::desc_kmajor(sb + C::KP, C::ROWS, 0);
    const auto release = [&](int b) {                // a buffer's next copy may start
      tc::fence_smem_to_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + b);
    };
    bool bad = false, aborted = false;
    uint32_t pend = 0;                               // products in flight, by barrier
    uint32_t phases = 0;                             // the next phase of each product's barrier
    // Wait for the products before a commit to barrier b.
    const auto done = [&](int b) {
      bad |= !wait_timed(bars + b, (phases >> b) & 1, wait_ns);
      if (!bad) {
        phases ^= 1u << b;
        pend &= ~(1u << b);
      }
      tc::fence_after_sync();
    };
    // A unit's outputs: blocks hw, hw + WG, ... of its tokens.
    float o[C::OB][kBlk];
    unsigned long long o_all = 0;
    __nv_bfloat16 *o_at = out;
    const int64_t o_step = (int64_t)H * kD;
    const auto put_out = [&] {
#pragma unroll
      for (int e = 0; e < C::OB; ++e) {
        const int t0 = kBlk * (hw + C::WG * e), left = T - t0;
        const uint32_t live = (uint32_t)(o_all >> t0);
        __nv_bfloat16 *at = o_at + t0 * o_step;
#pragma unroll
        for (int j = 0; j < kBlk; ++j) {
          if (j < left) *at = __float2bfloat16_rn((live >> j) & 1 ? o[e][j] : 0.f);
          at += o_step;
        }
      }
    };
    uint32_t i = 0;
    for (;; ++i) {
      const uint32_t ph = i & 1;
      const unsigned long long *s_anc = reinterpret_cast<unsigned long long *>(sp + C::ANC) + ph * TP;
      const int *s_par = reinterpret_cast<int *>(sp + C::PAR) + ph * TP;
      const float *s_beta = reinterpret_cast<float *>(sp + C::BETA) + ph * TP;

      // ---- S0^T into tensor memory ----
      bad |= !wait_timed(bars + kFullS, ph, wait_ns);
      const int64_t row0 = *reinterpret_cast<volatile int64_t *>(sp + C::ROW + 8 * ph);
      if (!bad && row0 < 0) {
        bar_or<C::WORKERS>(false);         // a thread whose wait has run out is at its next barrier
        break;
      }
      {
        const float *sf = reinterpret_cast<const float *>(sp + C::SF) + col;
#pragma unroll
        for (int b = 0; b < 4 / C::WG; ++b) {
          const int k0 = 32 * (b * C::WG + hw);
          float x[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) x[e] = sf[(k0 + e) * kD] * (kTf32 * kSink);
          tc::tmem_st32(tl + C::S + (uint32_t)k0, x);
        }
        tc::tmem_wait_st();
        release(kEmptyS);
      }

      // ---- Gam along the paths: g (a thread per channel) and A ----
      bad |= !wait_timed(bars + kFullQkg, ph, wait_ns);
      const unsigned long long all = *reinterpret_cast<volatile unsigned long long *>(sp + C::ALL + 8 * ph);
      const int last = all ? 64 - __clzll(all) : 0;                     // places up to the last token,
      const int nb = (last + kBlk - 1) / kBlk;                          // blocks
      const int nh = (nb * kBlk + C::TH - 1) / C::TH;                   // and parts
      for (int b = hw; b < nb && b < TP / kBlk; b += C::WG) {
        float x[kBlk], y[kBlk];
#pragma unroll
        for (int j = 0; j < kBlk; ++j) {
          // finite where it may be -inf: it meets zeros in the product
          y[j] = max_nan(rg[(kBlk * b + j) * kD], -1e5f);
          x[j] = __uint_as_float((__float_as_uint(y[j]) + 0x1000u) & 0xffffe000u);
          y[j] -= x[j];
        }
        tc::tmem_st16(tl + C::AG + (uint32_t)(kBlk * b), x);
        tc::tmem_st16(tl + C::AG + (uint32_t)(TP + kBlk * b), y);
      }
      for (int e = tid; e < TP * TP / 4; e += C::WORKERS) {
        const int t = e / (TP / 4), s0 = 4 * (e % (TP / 4));
        const uint32_t bits = (uint32_t)(s_anc[t] >> s0);
        *reinterpret_cast<float4 *>(sp + C::AN + tile32(TP, t, s0)) =
            make_float4(bits & 1 ? 1.f : 0.f, bits & 2 ? 1.f : 0.f, bits & 4 ? 1.f : 0.f,
                        bits & 8 ? 1.f : 0.f);
      }
      tc::tmem_wait_st();
      tc::fence_smem_to_async();
      tc::fence_before_sync();
      // (every thread is past the last unit's [KK; P], too, where Kh will be)
      if (bar_or<C::WORKERS>(bad)) { aborted = true; break; }
      if (warp == 3 && elect_one()) {
        tc::fence_after_sync();
        for (int b = 0; b < nb; ++b)
#pragma unroll
          for (int s = 0; s < kBlk / 8; ++s) {
            const uint64_t d = step_desc(an_desc, TP, kBlk / 8 * b + s);
            mma_tf32_ts(tmem + C::D3, tmem + C::AG + kBlk * b + 8 * s, d, idesc_tf32(128, TP), b + s > 0);
            mma_tf32_ts(tmem + C::D3, tmem + C::AG + TP + kBlk * b + 8 * s, d, idesc_tf32(128, TP), 1);
          }
        tc::mma_commit(bar_at(kMmaG));
      }
      __syncwarp();
      pend |= 1u << kMmaG;
      done(kMmaG);

      // ---- X = [Kt; Qt] and Kh, then D2 = X Kh^T and D1 = S0^T X^T, part by part ----
      bool wide = false;   // factors out of range: KK and P pair by pair
#pragma unroll
      for (int hf = 0; hf < C::NH; ++hf) {
        if (hf > 0 && hf >= nh) break;
        const int j0 = kBlk * hw, t0 = C::TH * hf + j0;
        if (t0 < kBlk * nb) {
          float Gt[kBlk];
          tc::tmem_ld16(tl + C::D3 + (uint32_t)t0, Gt);
          tc::tmem_wait_ld();
          const uint32_t within = (uint32_t)(((col & 31) >> 2) << 4);
          uint8_t *xt = sp + (hf == 0 ? C::X : C::X1) + (col >> 5) * C::XR * 128 + j0 * 128 + (col & 3) * 4;
          uint8_t *kt = sp + C::KH + (col >> 5) * TP * 128 + t0 * 128 + (col & 3) * 4;
#pragma unroll
          for (int j = 0; j < kBlk; ++j) {
            if (j == kBlk / 2 && t0 + j >= last) break;   // (what the rows held is masked)
            const float kv = __bfloat162float(rk[(t0 + j) * kD]), qv = __bfloat162float(rq[(t0 + j) * kD]);
            // powers of two, times kTf32 and the lift
            const float down = exp2_approx(fmaf(Gt[j], 1.44269504f, kLog2Tf32 + kLift));
            const float d = kv * exp2_approx(fmaf(Gt[j], -1.44269504f, kLog2Tf32 - kLift));
            wide |= !(fabsf(Gt[j]) <= kGamBound && fabsf(d) < kFactorBound);
            const uint32_t at = (within ^ ((j & 7) << 4)) + j * 128;
            *reinterpret_cast<float *>(xt + at) = kv * down;
            *reinterpret_cast<float *>(xt + at + C::TH * 128) = qv * down;
            *reinterpret_cast<float *>(kt + at) = d;
          }
        }
        if (wide) s_wide[ph] = 1;
        if (C::NH == 1 || nh <= 1) release(kEmptyQkg);
        else tc::fence_smem_to_async();
        tc::fence_before_sync();
        if (bar_or<C::WORKERS>(bad)) { aborted = true; break; }
        // Two warps issue, one product each.
        if (warp == 1 && elect_one()) {
          tc::fence_after_sync();
#pragma unroll
          for (int s = 0; s < kD / 8; ++s)
            mma_tf32_ss(tmem + C::D2 + C::TH * hf, step_desc(x_desc[hf], C::XR, s),
                        step_desc(kh_desc, TP, s), idesc_tf32(128, C::TH * (hf + 1)), s > 0);
          tc::mma_commit(bar_at(hf == 0 ? kMmaA : kMmaA1));
        } else if (warp == 2 && elect_one()) {
          tc::fence_after_sync();
#pragma unroll
          for (int s = 0; s < kD / 8; ++s)
            mma_tf32_ts(tmem + C::D1 + C::XR * hf, tmem + C::S + 8 * s,
                        step_desc(x_desc[hf], C::XR, s), idesc_tf32(128, C::XR), s > 0);
          tc::mma_commit(bar_at(hf == 0 ? kMmaB : kMmaB1));
        }
        __syncwarp();
        pend |= hf == 0 ? 1u << kMmaA | 1u << kMmaB : 1u << kMmaA1 | 1u << kMmaB1;
        if (hf + 1 >= nh && i > 0) put_out();   // the last unit's outputs, while the products run
      }
      if (aborted) break;

      // ---- KK and P, masked.  Row of token t in the tile: XR (t / TH) + t % TH, and TH
      //      below it for P ----
      const bool pairwise = s_wide[ph] != 0;
      done(kMmaA);
      if (C::NH > 1) done(kMmaB);          // the tile takes X's place
      if (tid == 0) s_wide[ph ^ 1] = 0;
      if (!pairwise) {
#pragma unroll
        for (int hf = 0; hf < C::NH; ++hf) {
          constexpr int HALF = C::TH / C::WG;        // 16 columns; twice that in part 1
          if (hf > 0 && hf < nh) done(kMmaA1);
          if (hf < nh && col < C::XR) {              // whole warps
            const int t = C::TH * hf + (col & (C::TH - 1));
            unsigned long long on = s_anc[t];
            if (col < C::TH) on &= ~(1ull << t);
#pragma unroll
            for (int p = 0; p <= hf; ++p) {
              const int s0 = HALF * (C::WG * p + hw);
              float x[HALF];
              tc::tmem_ldw<HALF>(tl + C::D2 + (uint32_t)(C::TH * hf + s0), x);
              tc::tmem_wait_ld();
              const uint32_t bits = (uint32_t)(on >> s0);
#pragma unroll
              for (int s = 0; s < HALF; s += 4) {
                float y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  y[e] = (bits >> (s + e)) & 1 ? cut_tf32(x[s + e]) : 0.f;
                *reinterpret_cast<float4 *>(sp + C::KP + tile32(C::ROWS, C::XR * hf + col, s0 + s)) =
                    make_float4(y[0], y[1], y[2], y[3]);
              }
            }
          }
        }
      } else {
        if (C::NH > 1 && nh > 1) done(kMmaA1);
        // One warp per place: the path upwards, with the decay between its ends summed
        // from the near one, so that no large sums are subtracted.
        for (int t = warp; t < kBlk * nb; t += C::WORKERS / 32) {
          const int row = C::XR * (t / C::TH) + t % C::TH;
          const auto kp = [&](int r, int s) {
            return reinterpret_cast<float *>(sp + C::KP + tile32(C::ROWS, r, s));
          };
          for (int s = lane; s < TP; s += 32) *kp(row, s) = *kp(row + C::TH, s) = 0.f;
          __syncwarp();
          const bool live = (all >> t) & 1;
          const int64_t rt = (row0 + (int64_t)t * H) * kD + lane;
          float ka[4], qa[4], d[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            ka[c] = live ? to_f32(k[rt + 32 * c]) : 0.f;
            qa[c] = live ? to_f32(q[rt + 32 * c]) : 0.f;
            d[c] = 0.f;
          }
          for (int s = live ? t : -1; s >= 0; s = s_par[s]) {
            const int64_t rs = (row0 + (int64_t)s * H) * kD + lane;
            float kk = 0.f, qk = 0.f;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const float x = to_f32(k[rs + 32 * c]) * expf(d[c]);
              kk += ka[c] * x;
              qk += qa[c] * x;
              d[c] += g[rs + 32 * c];
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
              kk += __shfl_xor_sync(0xffffffffu, kk, o);
              qk += __shfl_xor_sync(0xffffffffu, qk, o);
            }
            if (lane == 0) {
              if (s != t) *kp(row, s) = cut_tf32(kk);
              *kp(row + C::TH, s) = cut_tf32(qk);
            }
          }
        }
      }
      tc::fence_smem_to_async();
      bad |= !wait_timed(bars + kFullV, ph, wait_ns);
      if (C::NH == 1) done(kMmaB);
      if (C::NH > 1 && nh > 1) {
        done(kMmaB1);
        release(kEmptyQkg);                // X of part 1 lay in g's place
      }
      tc::fence_before_sync();
      if (bar_or<C::WORKERS>(bad)) { aborted = true; break; }
      tc::fence_after_sync();

      // ---- u of 16 tokens at a time, and what they add to D1 ----
      if (hw == 0) {
        for (int b = 0; b < nb; ++b) {
          const int part = kBlk * b / C::TH, r0 = C::XR * part + kBlk * b % C::TH;
          float x[kBlk], ks[kBlk];
          tc::tmem_ld16(tl + C::D1 + (uint32_t)r0, ks);
          tc::tmem_wait_ld();
          const uint8_t *kp = sp + C::KP + (TP > 32 ? (b >> 1) * C::ROWS * 128 : 0) + r0 * 128;
          const uint32_t flip = TP > kBlk ? (b & 1) * 64 : 0;   // column chunks 4 .. 7 of a row
#pragma unroll
          for (int j = kBlk / 2; j < kBlk; ++j) x[j] = 0.f;
#pragma unroll
          for (int j = 0; j < kBlk; ++j) {
            if (j == kBlk / 2 && kBlk * b + j >= last) break;
            // four sums, and u of the token before last: short chains
            float a = __bfloat162float(rv[(kBlk * b + j) * kD]) - ks[j], a1 = 0.f, a2 = 0.f, a3 = 0.f, end = 0.f;
#pragma unroll
            for (int s4 = 0; s4 < j; s4 += 4) {
              const uint32_t at = (uint32_t)(j * 128) + ((uint32_t)(((s4 >> 2) ^ (j & 7)) << 4) ^ flip);
              const float4 kk = *reinterpret_cast<const float4 *>(kp + at);
              if (s4 < j - 1) a -= kk.x * x[s4];
              if (s4 + 1 < j - 1) a1 -= kk.y * x[s4 + 1];
              if (s4 + 2 < j - 1) a2 -= kk.z * x[s4 + 2];
              if (s4 + 3 < j - 1) a3 -= kk.w * x[s4 + 3];
              if (s4 + 4 >= j) end = (j - 1) % 4 == 0 ? kk.x : (j - 1) % 4 == 1 ? kk.y : (j - 1) % 4 == 2 ? kk.z : kk.w;
            }
            a = (a + a1) + (a2 + a3);
            if (j > 0) a -= end * x[j > 0 ? j - 1 : 0];
            x[j] = s_beta[kBlk * b + j] * a;
          }
#pragma unroll
          for (int j = 0; j < kBlk; ++j) x[j] = to_tf32(x[j]);
          tc::tmem_st16(tl + C::U, x);
          tc::tmem_wait_st();
          tc::fence_before_sync();
          asm volatile("barrier.cta.sync 2, 128;" ::: "memory");
          if (warp == 0 && elect_one()) {
            // tokens of this part and the later ones
            tc::fence_after_sync();
            const uint64_t d = step_desc(kp_desc, C::ROWS, kBlk / 8 * b) + (uint64_t)(C::XR * part * 128 >> 4);
            const uint32_t id = C::NH > 1 && nh > part + 1 ? idesc_tf32(128, 2 * C::XR) : idesc_tf32(128, C::XR);
#pragma unroll
            for (int s = 0; s < kBlk / 8; ++s)
              mma_tf32_ts(tmem + C::D1 + C::XR * part, tmem + C::U + 8 * s, d + (uint64_t)(2 * s), id, 1);
            tc::mma_commit(bar_at(b + 1 < nb ? kMmaU : kMmaO));
          }
          __syncwarp();
          if (b + 1 < nb) {
            pend |= 1u << kMmaU;
            done(kMmaU);
          }
        }
        if (nb == 0 && tid == 0) tc::mma_commit(bar_at(kMmaO));
      }
      release(kEmptyV);
      pend |= 1u << kMmaO;
      done(kMmaO);

      // ---- the outputs, kept until the next unit's products run ----
#pragma unroll
      for (int e = 0; e < C::OB; ++e) {
        const int b = hw + C::WG * e;
        if (b < nb)
          tc::tmem_ld16(tl + C::D1 + (uint32_t)(C::XR * (kBlk * b / C::TH) + C::TH + kBlk * b % C::TH), o[e]);
      }
      tc::tmem_wait_ld();
      o_all = all;
      o_at = out + row0 * kD + col;
    }
    if (i > 0 && !aborted) put_out();
    if (aborted || bad) {
      report(dev_status, KDA_ERR_TIMEOUT);
      *s_quit = 1;
      // products still in flight end before the memory is released
      for (int b = kMmaG; b <= kMmaO; ++b)
        if ((pend >> b) & 1) wait_timed(bars + b, (phases >> b) & 1, wait_ns);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 0) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, C::COLS);
  }
}

template <int TP>
cudaError_t launch_tp(const void *q, const void *k, const void *v, const float *g,
                      const float *beta, const float *state, const int32_t *parents, void *out,
                      int T, int64_t units, int H, int32_t *dev_status, cudaStream_t stream) {
  using C = TreeTc<TP>;
  const auto kern = decode_tree_tc_kernel<TP>;
  const size_t smem = C::TOTAL + 1024;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout,
                           (int)cudaSharedmemCarveoutMaxShared);
  if (e != cudaSuccess) return e;
  return launch_dependent(kern, (unsigned)units, C::THREADS, smem, 1, stream, (const __nv_bfloat16 *)q,
                          (const __nv_bfloat16 *)k, (const __nv_bfloat16 *)v, g, beta, state, parents,
                          (__nv_bfloat16 *)out, T, H, dev_status, 2000000000ull);
}

}  // namespace

bool decode_tree_tc_supported(int dtype, int dk, int dv) {
  return dtype == KDA_DTYPE_BF16 && dk == kD && dv == kD;
}

cudaError_t launch_decode_tree_tc(const void *q, const void *k, const void *v, const float *g,
                                  const float *beta, const float *state, const int32_t *parents,
                                  void *out, int T, int64_t units, int H, int32_t *dev_status,
                                  cudaStream_t stream) {
#define KDA_TP(TP_) \
  launch_tp<TP_>(q, k, v, g, beta, state, parents, out, T, units, H, dev_status, stream)
  if (T <= 16) return KDA_TP(16);
  if (T <= 32) return KDA_TP(32);
  return KDA_TP(64);
#undef KDA_TP
}

}  // namespace kda

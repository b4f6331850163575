// The 8-bit state cache: states quantised as they are written into slots, and
// read back as FP32.
//
// Prefix caching keeps FP32 states of 4 D_k D_v bytes per head ("LLM -
// Semianalysis, Kimi K3 아키텍처" (charstring.tistory.com/2557), Methods 3).  One
// byte per element holds four times as many of them.  The decay is per key
// channel, so the rows of a state differ in size by orders of magnitude: each
// row (key channel) carries its own FP32 scale,
//
//   scale = max_v |S[c][v]| * (1 / top)   (top = 448 for E4M3, 127 for INT8)
//   code  = round(S[c][v] / scale)        (to nearest, ties to even; clamped to +-top)
//   value = code * scale
//
// in FP32, with 1 / top, the product and the quotient each correctly rounded, so that
// the codes are reproducible to the bit.  A row of zeros, or one so small that its scale
// underflows to zero, stores zeros; a row that holds an infinity or a NaN stores a NaN
// scale and reads back as NaN.
//
// Both kernels are bound by memory: 5/4 of the FP32 bytes cross HBM once.  One
// CTA takes one (state, head), every thread's loads are issued before the first
// use, and a row lies in one warp (D_v / 4 lanes of float4), so its maximum is a
// reduction inside it.  512 x 32 states of 128 x 128: store 203 us, load 206 us, 205 at
// the copy rate.  The store takes three CTAs per SM (80 registers; 226 us with the two
// that 86 registers allow), and products instead of quotients (318 us with them).  Small
// states are farther off (4096 x 8 of 32 x 32: 62 us, 26 at the copy rate): a CTA has
// 4 KB, and looks through the slots of all later entries for its own.
#include <cuda_fp8.h>
#include <math_constants.h>

#include "kda_common.cuh"
#include "kda_launch.cuh"
#include "kda_tf32.cuh"

namespace kda {
namespace {

constexpr int kCacheThreads = 256;

template <bool E4M3> __device__ __forceinline__ float code_top() { return E4M3 ? 448.f : 127.f; }

// Four codes of one row, packed in memory order, by the quotients.
template <bool E4M3> __device__ __noinline__ uint32_t encode4_exact(float4 x, float scale) {
  const float top = code_top<E4M3>();
  float y[4] = {x.x / scale, x.y / scale, x.z / scale, x.w / scale};
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = fminf(fmaxf(y[i], -top), top);
  if (E4M3) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[0], y[1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[2], y[3]), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
  }
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) r |= (uint32_t)(uint8_t)(int8_t)__float2int_rn(y[i]) << (8 * i);
  return r;
}

// Four codes from products with one factor.  INT8: 1.5 * 2^23 + x f, rounded once,
// holds the nearest integer in its low byte.
template <bool E4M3> __device__ __forceinline__ uint32_t encode4_by(float4 x, float f) {
  if (E4M3) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x.x * f, x.y * f), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x.z * f, x.w * f), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
  }
  constexpr float kBase = 12582912.f;
  const uint32_t lo = __byte_perm(__float_as_uint(__fmaf_rn(x.x, f, kBase)),
                                  __float_as_uint(__fmaf_rn(x.y, f, kBase)), 0x0040);
  const uint32_t hi = __byte_perm(__float_as_uint(__fmaf_rn(x.z, f, kBase)),
                                  __float_as_uint(__fmaf_rn(x.w, f, kBase)), 0x0040);
  return __byte_perm(lo, hi, 0x5410);
}

// The codes are those of the rounded quotients x / scale, at a third of their cost:
// with factors at least 5 * 2^-24 (relative) below and above 1 / scale, x times one
// of them lies on each side of the rounded quotient (its own rounding, the
// reciprocal's and the product's are 4 * 2^-24 together), and rounding to codes is
// monotone.  Where both give one code, it is the quotient's; else (of normal numbers 14
// vectors of four in 10^5 for INT8, 5 for E4M3) the quotients are formed.
struct Factor {
  float lo, hi;
  bool sure;             // the scale is large enough for its reciprocal to be a normal number
  __device__ __forceinline__ explicit Factor(float scale) {
    const float r = __frcp_rn(scale);
    lo = r * (1.f - 0x1p-21f);
    hi = r * (1.f + 0x1p-21f);
    sure = scale >= 0x1p-100f;
  }
};
template <bool E4M3>
__device__ __forceinline__ uint32_t encode4(float4 x, float scale, const Factor &f) {
  const uint32_t a = encode4_by<E4M3>(x, f.lo), b = encode4_by<E4M3>(x, f.hi);
  if (f.sure && a == b) return a;
  return scale > 0.f ? encode4_exact<E4M3>(x, scale) : 0u;   // false for a NaN scale too
}

// Read once, behind the wait for the kernel ahead.
__device__ __forceinline__ float4 load_once(const float4 *p) {
  float4 x;
  asm volatile("ld.global.cs.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
               : "l"(p)
               : "memory");
  return x;
}
__device__ __forceinline__ uint32_t load_once(const uint32_t *p) {
  uint32_t x;
  asm volatile("ld.global.cs.u32 %0, [%1];" : "=r"(x) : "l"(p) : "memory");
  return x;
}

template <bool E4M3> __device__ __forceinline__ float4 decode4(uint32_t c, float scale) {
  float4 x;
  if (E4M3) {
    const __half2 lo(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c & 0xffffu), __NV_E4M3));
    const __half2 hi(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c >> 16), __NV_E4M3));
    const float2 a = __half22float2(lo), b = __half22float2(hi);
    x = make_float4(a.x, a.y, b.x, b.y);
  } else {
    x = make_float4((float)(int8_t)(c & 0xffu), (float)(int8_t)((c >> 8) & 0xffu),
                    (float)(int8_t)((c >> 16) & 0xffu), (float)(int8_t)(c >> 24));
  }
  return make_float4(x.x * scale, x.y * scale, x.z * scale, x.w * scale);
}

template <int DK, int DV, bool E4M3>
__global__ void __launch_bounds__(kCacheThreads, 3)
state_store_kernel(const float *states, const int32_t *slots,
                   uint32_t *__restrict__ cache, float *__restrict__ scales, int N, int H,
                   int64_t num_slots) {
  constexpr int V4 = DV / 4;                          // lanes of one row
  constexpr int RPP = kCacheThreads / V4;             // rows per pass
  constexpr int ITER = DK / RPP;
  static_assert(DK % RPP == 0 && ITER >= 1, "tile mismatch");
  const int64_t unit = blockIdx.x;
  const int n = (int)(unit / H), h = (int)(unit % H);
  const int tid = threadIdx.x, cg = tid % V4, rg = tid / V4;
  launch_dependents();
  wait_for_inputs();
  const int32_t slot = slots[n];
  if (slot < 0 || (int64_t)slot >= num_slots) return;
  const float4 *src = reinterpret_cast<const float4 *>(states) + unit * (DK * V4);
  float4 x[ITER];
#pragma unroll
  for (int i = 0; i < ITER; ++i) x[i] = load_once(src + (rg + i * RPP) * V4 + cg);
  // A slot named twice keeps the last entry's state, whichever CTA runs first.
  int later = 0;
  for (int j = n + 1 + tid; j < N; j += kCacheThreads) later |= slots[j] == slot;
  if (__syncthreads_or(later)) return;
  const int64_t dst_unit = (int64_t)slot * H + h;
  uint32_t *dst = cache + dst_unit * (DK * V4);
  float *sc = scales + dst_unit * DK;
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    const int r = rg + i * RPP;
    // The bits of non-negative numbers are ordered like them, infinity and NaN last.
    uint32_t m = __float_as_uint(max_nan(max_nan(fabsf(x[i].x), fabsf(x[i].y)),
                                         max_nan(fabsf(x[i].z), fabsf(x[i].w))));
    if (V4 == 32) {
      m = __reduce_max_sync(0xffffffffu, m);
    } else {
#pragma unroll
      for (int o = 1; o < V4; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
    const float scale = m < 0x7f800000u ? __uint_as_float(m) * (1.f / code_top<E4M3>()) : CUDART_NAN_F;
    dst[r * V4 + cg] = encode4<E4M3>(x[i], scale, Factor(scale));
    if (cg == 0) sc[r] = scale;
  }
}

template <int DK, int DV, bool E4M3>
__global__ void __launch_bounds__(kCacheThreads)
state_load_kernel(const uint32_t *cache, const float *scales,
                  const int32_t *slots, float *__restrict__ states, int H,
                  int64_t num_slots) {
  constexpr int V4 = DV / 4;
  constexpr int RPP = kCacheThreads / V4;
  constexpr int ITER = DK / RPP;
  const int64_t unit = blockIdx.x;
  const int n = (int)(unit / H), h = (int)(unit % H);
  const int tid = threadIdx.x, cg = tid % V4, rg = tid / V4;
  launch_dependents();
  wait_for_inputs();
  const int32_t slot = slots[n];
  float4 *dst = reinterpret_cast<float4 *>(states) + unit * (DK * V4);
  if (slot < 0 || (int64_t)slot >= num_slots) {   // no cached prefix: the zero state
#pragma unroll
    for (int i = 0; i < ITER; ++i)
      __stcs(dst + (rg + i * RPP) * V4 + cg, make_float4(0.f, 0.f, 0.f, 0.f));
    return;
  }
  const int64_t src_unit = (int64_t)slot * H + h;
  const uint32_t *src = cache + src_unit * (DK * V4);
  const float *sc = scales + src_unit * DK;
  uint32_t c[ITER];
  float s[ITER];
#pragma unroll
  for (int i = 0; i < ITER; ++i) c[i] = load_once(src + (rg + i * RPP) * V4 + cg);
#pragma unroll
  for (int i = 0; i < ITER; ++i) s[i] = sc[rg + i * RPP];
#pragma unroll
  for (int i = 0; i < ITER; ++i)
    __stcs(dst + (rg + i * RPP) * V4 + cg, decode4<E4M3>(c[i], s[i]));
}

template <int DK, int DV>
cudaError_t launch_d(bool store, bool e4m3, float *states, const int32_t *slots, void *cache,
                     float *scales, int N, int H, int64_t num_slots, cudaStream_t stream) {
  const unsigned grid = (unsigned)((int64_t)N * H);
  uint32_t *c = static_cast<uint32_t *>(cache);
  if (store)
    return launch_dependent(e4m3 ? state_store_kernel<DK, DV, true> : state_store_kernel<DK, DV, false>, grid,
                            kCacheThreads, 0, 1, stream, states, slots, c, scales, N, H, num_slots);
  return launch_dependent(e4m3 ? state_load_kernel<DK, DV, true> : state_load_kernel<DK, DV, false>, grid,
                          kCacheThreads, 0, 1, stream, c, scales, slots, states, H, num_slots);
}

}  // namespace

cudaError_t launch_state_cache(bool store, bool e4m3, int dk, int dv, float *states,
                               const int32_t *slots, void *cache, float *scales, int N, int H,
                               int64_t num_slots, cudaStream_t stream) {
#define KDA_SC(DK_, DV_) \
  if (dk == DK_ && dv == DV_) \
    return launch_d<DK_, DV_>(store, e4m3, states, slots, cache, scales, N, H, num_slots, stream);
  KDA_SC(32, 32) KDA_SC(32, 64) KDA_SC(32, 128)
  KDA_SC(64, 32) KDA_SC(64, 64) KDA_SC(64, 128)
  KDA_SC(128, 32) KDA_SC(128, 64) KDA_SC(128, 128)
#undef KDA_SC
  return cudaErrorInvalidValue;
}

}  // namespace kda

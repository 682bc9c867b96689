// kvc_paged_math.cuh -- arithmetic shared by the tensor-core kernels of the paged batch.
#pragma once
#include "kvc_attn_common.cuh"

namespace kvc {
namespace paged {

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// Maxima that keep a NaN, so that a row with a NaN score ends as NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// 2^x of a pair on the FMA pipe: x is clamped to [-126, 128] and split as n + f, n = rint(x)
// (the 1.5 * 2^23 shift), f in [-0.5, 0.5]; 2^f is a quartic with p(0) = 1, fitted by iteratively
// reweighted least squares on the relative error (at most 2.9e-6 in fp32, 3.4e-7 on average);
// n goes into the exponent field. At 128 that gives +inf, as every larger x and a NaN do then: no term that
// passes fp32, and none of a product that is no number, comes out finite.
__device__ __forceinline__ uint64_t exp2_pair(uint64_t x2) {
  constexpr float kShift = 12582912.0f;
  float x0, x1;
  up2(x2, x0, x1);
  const uint64_t xc = pk2(fmaxf(fminf(x0, 128.f), -126.f), fmaxf(fminf(x1, 128.f), -126.f));
  const uint64_t t = add2(xc, pk2(kShift, kShift));
  const uint64_t n = add2(t, pk2(-kShift, -kShift));
  const uint64_t f = fma2(n, pk2(-1.f, -1.f), xc);
  uint64_t q = fma2(pk2(0.009582852944731712f, 0.009582852944731712f), f,
                    pk2(0.055906426161527634f, 0.055906426161527634f));
  q = fma2(q, f, pk2(0.24024099111557007f, 0.24024099111557007f));
  q = fma2(q, f, pk2(0.6931241750717163f, 0.6931241750717163f));
  q = fma2(q, f, pk2(1.0f, 1.0f));
  float q0, q1, t0, t1;
  up2(q, q0, q1);
  up2(t, t0, t1);
  return pk2(__uint_as_float(__float_as_uint(q0) + (__float_as_uint(t0) << 23)),
             __uint_as_float(__float_as_uint(q1) + (__float_as_uint(t1) << 23)));
}
// The same on the MUFU.
__device__ __forceinline__ uint64_t exp2_pair_mufu(uint64_t x2) {
  float x0, x1;
  up2(x2, x0, x1);
  return pk2(ex2(x0), ex2(x1));
}

template <int N>
__device__ __forceinline__ void reg_dealloc() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_alloc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

}  // namespace paged
}  // namespace kvc

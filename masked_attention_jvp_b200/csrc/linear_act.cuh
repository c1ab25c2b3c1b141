// Activations of the linear operators, their derivatives, and the pieces of the
// epilogue that the fused, the split and the few-row kernels share.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "ptx_sm100.cuh"

namespace caj {
namespace lin {

constexpr int kActNone = 0, kActGeluTanh = 1, kActGelu = 2, kActSilu = 3;

__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// act(z), and with SLOPE its derivative.
//   silu        z s,               s (1 + z (1 - s)),         s = 1 / (1 + e^-z)
//   gelu_tanh   0.5 z (1 + tanh u) = z s with s = 1 / (1 + e^-2u), u = a (z + b z^3);
//               s + z s (1 - s) 2 u',                         u' = a (1 + 3 b z^2)
//   gelu        z F(z),            F(z) + z e^(-z^2/2) / sqrt(2 pi), F the normal's cdf
// The exponential and the reciprocal are the hardware's approximations (relative
// error about 2^-22, far under the outputs' bf16); where e^-x overflows, s is 0.
template <int ACT, bool SLOPE>
__device__ __forceinline__ float act(float z, float &slope) {
  if constexpr (ACT == kActNone) {
    slope = 1.f;
    return z;
  } else if constexpr (ACT == kActGelu) {
    const float cdf = 0.5f + 0.5f * erff(z * 0.70710678f);
    if constexpr (SLOPE) slope = fmaf(z * 0.39894228f, ptx::ex2(z * z * -0.72134752f), cdf);
    return z * cdf;
  } else {
    constexpr float kLog2e = 1.44269504f, kA = 0.79788456f, kB = 0.044715f;
    const float z2 = z * z;
    const float arg = ACT == kActSilu ? z * -kLog2e : z * fmaf(z2, -2.f * kA * kB * kLog2e, -2.f * kA * kLog2e);
    const float s = rcp(1.f + ptx::ex2(arg));
    const float y = z * s;
    if constexpr (SLOPE) {
      const float d = ACT == kActSilu ? 1.f : fmaf(z2, 6.f * kA * kB, 2.f * kA);
      slope = fmaf(y * (1.f - s), d, s);
    }
    return y;
  }
}

// v = act(v) for M values; with SLOPE sl = act'(v).
template <int ACT, bool SLOPE, int M>
__device__ __forceinline__ void act_of(float (&v)[M], float (&sl)[M]) {
#pragma unroll
  for (int i = 0; i < M; ++i) v[i] = act<ACT, SLOPE>(v[i], sl[i]);
}
template <bool SLOPE, int M>
__device__ __forceinline__ void act_all(int32_t which, float (&v)[M], float (&sl)[M]) {
  if (which == kActGeluTanh)
    act_of<kActGeluTanh, SLOPE>(v, sl);
  else if (which == kActSilu)
    act_of<kActSilu, SLOPE>(v, sl);
  else if (which == kActGelu)
    act_of<kActGelu, SLOPE>(v, sl);
  else if (SLOPE)
    act_of<kActNone, SLOPE>(v, sl);
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

}  // namespace lin
}  // namespace caj

// Eight consecutive channels of bf16 or fp32 storage as fp32 registers: the unit
// of work of the memory-bound kernels (one or two 16-byte accesses).
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

namespace caj {
namespace v8 {

template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  uint4 a;
};
template <>
struct Raw<float> {
  uint4 a, b;
};

// Streaming (read-once) load of 8 elements from a 16-byte aligned address.
template <typename T>
__device__ __forceinline__ Raw<T> load(const T *p) {
  Raw<T> r;
  r.a = __ldcs(reinterpret_cast<const uint4 *>(p));
  if constexpr (sizeof(T) == 4) r.b = __ldcs(reinterpret_cast<const uint4 *>(p) + 1);
  return r;
}
template <typename T>
__device__ __forceinline__ Raw<T> zero() {
  Raw<T> r;
  r.a = make_uint4(0, 0, 0, 0);
  if constexpr (sizeof(T) == 4) r.b = make_uint4(0, 0, 0, 0);
  return r;
}
template <typename T>
__device__ __forceinline__ void store(T *p, const Raw<T> &r) {
  __stcs(reinterpret_cast<uint4 *>(p), r.a);
  if constexpr (sizeof(T) == 4) __stcs(reinterpret_cast<uint4 *>(p) + 1, r.b);
}

__device__ __forceinline__ void unpack(const Raw<__nv_bfloat16> &r, float (&f)[8]) {
  const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void unpack(const Raw<float> &r, float (&f)[8]) {
  f[0] = __uint_as_float(r.a.x); f[1] = __uint_as_float(r.a.y);
  f[2] = __uint_as_float(r.a.z); f[3] = __uint_as_float(r.a.w);
  f[4] = __uint_as_float(r.b.x); f[5] = __uint_as_float(r.b.y);
  f[6] = __uint_as_float(r.b.z); f[7] = __uint_as_float(r.b.w);
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {  // round to nearest even
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void pack(const float (&f)[8], Raw<__nv_bfloat16> &r) {
  r.a = make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}
__device__ __forceinline__ void pack(const float (&f)[8], Raw<float> &r) {
  r.a = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  r.b = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7]));
}

__device__ __forceinline__ void from_float(float x, float &o) { o = x; }
__device__ __forceinline__ void from_float(float x, __nv_bfloat16 &o) { o = __float2bfloat16_rn(x); }

}  // namespace v8
}  // namespace caj

// 8-bit activation checkpoints: the format, and its arithmetic on the device.
//
// A row of C values is kept as ceil(C/32) blocks of 32 codes: whole numbers c in
// [-127, 127], and one byte s per block. The value is c * 2^(s - 127), with the
// smallest s >= 0 for which the block's largest magnitude is at most
// 127 * 2^(s - 127), but at most kMaxScale: magnitudes above kTop = 127 * 2^121
// (3.376e38) become it, since the next step up would decode to infinity. Codes are padded with zeros to whole blocks, scale bytes to
// whole groups of four, so a block is one aligned 32-byte sector and the scales
// of 128 values one aligned 32-bit word.
//
// Why whole numbers under a power of two: a code has 7 significant bits, so every
// decoded value is exactly a bf16 number, and the backward's products read the
// checkpoint on the bf16 tensor cores without a second rounding. Scaling by a
// power of two is exact too, so the only rounding is value -> code, to nearest
// even: at most half a step, 2^(s - 128). For normal values a block of 32 has its
// largest near 2.2 standard deviations, an rms error of about 0.7% of the
// standard deviation (e4m3 with the same scale byte: about 2.6%).
// A block with an infinity or a NaN gets s = 255 and zero codes, and decodes to
// NaN throughout (0 * inf): a broken activation stays visible.
#pragma once
#include <stdint.h>

#include "ptx_sm100.cuh"

namespace caj {
namespace ck {

constexpr int kBlock = 32;
constexpr uint32_t kMaxScale = 248;
constexpr float kTop = 127.f * 0x1p121f;

// Blocks of a row of `cols` values, and its scale bytes.
__host__ __device__ inline int32_t blocks_of(int32_t cols) { return (cols + kBlock - 1) / kBlock; }
__host__ __device__ inline int32_t scale_bytes(int32_t cols) { return (blocks_of(cols) + 3) & ~3; }

// The scale byte for a block whose largest magnitude has the bits `amax_bits`.
// In units of its own exponent, the magnitude is in [1, 2) and 127/64 = 1.984375
// (mantissa 0x7E0000) is the most that seven bits hold.
__device__ __forceinline__ uint32_t scale_of(uint32_t amax_bits) {
  const uint32_t e = amax_bits >> 23;
  if (e == 255u) return 255u;
  const int32_t s = int32_t(e) - 6 + ((amax_bits & 0x7FFFFFu) > 0x7E0000u ? 1 : 0);
  return s > 0 ? min(uint32_t(s), kMaxScale) : 0u;
}
// At the largest scale, values above kTop saturate.
template <int M>
__device__ __forceinline__ void saturate(float (&f)[M], uint32_t s) {
  if (s < kMaxScale) return;
#pragma unroll
  for (int i = 0; i < M; ++i) f[i] = fminf(fmaxf(f[i], -kTop), kTop);
}
// 2^(127 - s), the factor from values to codes, for s <= kMaxScale (a block with
// s = 255 stores zero codes instead).
__device__ __forceinline__ float up_of(uint32_t s) { return __uint_as_float((254u - s) << 23); }
// 2^(s - 127); infinity for s = 255, subnormal for s = 0.
__device__ __forceinline__ float unit_of(uint32_t s) { return __uint_as_float(s ? s << 23 : 0x400000u); }

// Largest magnitude of M values; NaN if one is NaN (max.NaN keeps it).
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
template <int M>
__device__ __forceinline__ float max_mag(const float (&f)[M]) {
  float m[4] = {0.f, 0.f, 0.f, 0.f};  // four chains
#pragma unroll
  for (int i = 0; i < M; ++i) m[i & 3] = max_nan(m[i & 3], fabsf(f[i]));
  return max_nan(max_nan(m[0], m[1]), max_nan(m[2], m[3]));
}

// |x| as ordered bits (NaN above infinity above every number).
__device__ __forceinline__ uint32_t mag_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// Code of x, |x * up| <= 127: adding 1.5 * 2^23 rounds to the nearest whole
// number, ties to even, and leaves it in the low byte (one fma: the product with a
// power of two is exact, or too small to matter).
__device__ __forceinline__ uint32_t code_word(float x, float up) {
  return __float_as_uint(__fmaf_rn(x, up, 12582912.f));
}
__device__ __forceinline__ uint32_t pack_codes4(float a, float b, float c, float d, float up) {
  const uint32_t ab = __byte_perm(code_word(a, up), code_word(b, up), 0x0040);
  const uint32_t cd = __byte_perm(code_word(c, up), code_word(d, up), 0x0040);
  return __byte_perm(ab, cd, 0x5410);
}
// A block's codes at the largest scale, where values may saturate (rare: kept out of line).
__device__ __noinline__ inline void pack_saturated_block(float *f, uint32_t *w) {
  const float up = up_of(kMaxScale);
  for (int i = 0; i < kBlock; ++i) f[i] = fminf(fmaxf(f[i], -kTop), kTop);
  for (int i = 0; i < kBlock / 4; ++i) w[i] = pack_codes4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3], up);
}
__device__ __forceinline__ void pack_saturated(const float (&v)[kBlock], uint32_t (&w)[kBlock / 4]) {
  float f[kBlock];
  uint32_t o[kBlock / 4];
#pragma unroll
  for (int i = 0; i < kBlock; ++i) f[i] = v[i];
  pack_saturated_block(f, o);
#pragma unroll
  for (int i = 0; i < kBlock / 4; ++i) w[i] = o[i];
}
// Four codes -> two pairs of values: byte ^ 0x80 under the exponent of 2^23 is
// 2^23 + 128 + c; in packed arithmetic. (One fma with -(2^23 + 128) * unit instead would
// overflow from unit 2^105 on.) unit = infinity: 0 * infinity = NaN, as the format wants.
__device__ __forceinline__ void unpack_codes4(uint32_t w, float unit, uint64_t &ab, uint64_t &cd) {
  const uint32_t u = w ^ 0x80808080u;
  const uint64_t off = ptx::f2(8388736.f, 8388736.f), un = ptx::f2(unit, unit);
  ab = ptx::mul2(ptx::sub2(ptx::f2(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440)),
                                   __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7441))), off), un);
  cd = ptx::mul2(ptx::sub2(ptx::f2(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7442)),
                                   __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7443))), off), un);
}
__device__ __forceinline__ void unpack_codes4(uint32_t w, float unit, float &a, float &b, float &c, float &d) {
  uint64_t ab, cd;
  unpack_codes4(w, unit, ab, cd);
  ptx::f2_split(ab, a, b);
  ptx::f2_split(cd, c, d);
}

}  // namespace ck
}  // namespace caj

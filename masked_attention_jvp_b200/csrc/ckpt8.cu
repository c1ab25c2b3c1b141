// 8-bit activation checkpoints: packing rows of bf16 or fp32 values into codes and
// scale bytes, and back (format and rounding: ckpt8.cuh).
//
// Memory-bound: 3.03 bytes a value for bf16 (2 in, 1.03 out, or the reverse).
// Vector form: packing, two lanes hold a block, sixteen values each (16-byte loads and
// stores), and the block's largest magnitude is one shuffle away; unpacking, four lanes,
// eight values each, so that a warp's 16-byte stores are neighbours.
// Each thread takes kUnroll blocks a grid apart, with all loads issued first, to
// keep enough bytes in flight.
// Rows whose 16-byte vectors do not line up (C not a multiple of 8, or a base or
// row stride that is not 16-byte aligned) take the lane form: one lane per value,
// coalesced 2- or 4-byte accesses, the maximum by one redux instruction.
// 32760 x 1536 bf16 on B200: PACKED us packed, UNPACKED us unpacked in the vector form;
// 32760 x 1545 ODDP and ODDU us in the lane form.
#include <cuda_runtime.h>

#include "ckpt8.cuh"
#include "kernels.h"
#include "vec8.cuh"

namespace caj {
namespace {

constexpr int kUnroll = 2, kUnpackUnroll = 4;
constexpr int kThreads = 256;

// Scale byte of block `blk`; the row's last block also zeroes the padding bytes.
__device__ __forceinline__ void store_scale(uint8_t *row, int32_t blk, int32_t nb, int32_t ns, uint32_t s) {
  row[blk] = uint8_t(s);
  if (blk == nb - 1)
    for (int32_t i = nb; i < ns; ++i) row[i] = 0;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) pack_vec_kernel(const Ckpt8Params p) {
  const uint32_t nb = uint32_t(p.nb), total = p.total;
  const uint32_t step = gridDim.x * (kThreads / 2);
  const uint32_t first = blockIdx.x * (kThreads / 2) + (threadIdx.x >> 1);
  const int part = threadIdx.x & 1;
  v8::Raw<T> raw[kUnroll][2];
  uint32_t row[kUnroll], blk[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const uint64_t g = uint64_t(first) + uint64_t(u) * step;
    row[u] = g < total ? uint32_t(g) / nb : 0xFFFFFFFFu;
    blk[u] = uint32_t(g) - row[u] * nb;
    const int32_t c = int32_t(blk[u]) * ck::kBlock + 16 * part;
    const T *src = static_cast<const T *>(p.x) + size_t(row[u]) * p.ld + c;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      raw[u][h] = v8::zero<T>();
      if (g < total && c + 8 * h < p.cols) raw[u][h] = v8::load(src + 8 * h);  // cols is a multiple of 8 here
    }
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    float f[2][8];
    v8::unpack(raw[u][0], f[0]);
    v8::unpack(raw[u][1], f[1]);
    float m = ck::max_nan(ck::max_mag(f[0]), ck::max_mag(f[1]));
    m = ck::max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    if (row[u] == 0xFFFFFFFFu) continue;
    const uint32_t s = ck::scale_of(__float_as_uint(m));
    uint4 codes = make_uint4(0, 0, 0, 0);
    if (s != 255u) {
      const float up = ck::up_of(s);
      ck::saturate(f[0], s);
      ck::saturate(f[1], s);
      codes.x = ck::pack_codes4(f[0][0], f[0][1], f[0][2], f[0][3], up);
      codes.y = ck::pack_codes4(f[0][4], f[0][5], f[0][6], f[0][7], up);
      codes.z = ck::pack_codes4(f[1][0], f[1][1], f[1][2], f[1][3], up);
      codes.w = ck::pack_codes4(f[1][4], f[1][5], f[1][6], f[1][7], up);
    }
    const size_t base = (size_t(row[u]) * nb + blk[u]) * ck::kBlock + 16 * part;
    __stcs(reinterpret_cast<uint4 *>(p.codes + base), codes);
    if (part == 0) store_scale(p.scales + size_t(row[u]) * p.ns, int32_t(blk[u]), p.nb, p.ns, s);
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) unpack_vec_kernel(const Ckpt8Params p) {
  const uint32_t nb = uint32_t(p.nb), total = p.total;
  const uint32_t step = gridDim.x * (kThreads / 4);
  const uint32_t first = blockIdx.x * (kThreads / 4) + (threadIdx.x >> 2);
  const int part = threadIdx.x & 3;
  uint2 codes[kUnpackUnroll];
  uint32_t row[kUnpackUnroll], scale[kUnpackUnroll];
  int32_t col[kUnpackUnroll];
#pragma unroll
  for (int u = 0; u < kUnpackUnroll; ++u) {
    const uint64_t g = uint64_t(first) + uint64_t(u) * step;
    row[u] = g < total ? uint32_t(g) / nb : 0xFFFFFFFFu;
    const uint32_t blk = uint32_t(g) - row[u] * nb;
    col[u] = int32_t(blk) * ck::kBlock + 8 * part;
    codes[u] = make_uint2(0, 0);
    scale[u] = 0;
    if (g < total) {
      codes[u] = __ldcs(reinterpret_cast<const uint2 *>(p.codes + (size_t(row[u]) * nb + blk) * ck::kBlock + 8 * part));
      scale[u] = __ldg(p.scales + size_t(row[u]) * p.ns + blk);
    }
  }
#pragma unroll
  for (int u = 0; u < kUnpackUnroll; ++u) {
    if (row[u] == 0xFFFFFFFFu || col[u] >= p.cols) continue;
    const float unit = ck::unit_of(scale[u]);
    float f[8];
    ck::unpack_codes4(codes[u].x, unit, f[0], f[1], f[2], f[3]);
    ck::unpack_codes4(codes[u].y, unit, f[4], f[5], f[6], f[7]);
    v8::Raw<T> r;
    v8::pack(f, r);
    v8::store(static_cast<T *>(p.out) + size_t(row[u]) * p.ld + col[u], r);
  }
}

// One lane per value: a warp takes a run of up to eight blocks of one row.
constexpr int kRun = 8;

template <typename T>
__global__ void __launch_bounds__(kThreads) pack_lane_kernel(const Ckpt8Params p) {
  const uint32_t runs = (uint32_t(p.nb) + kRun - 1) / kRun;
  const uint32_t unit = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const uint32_t row = unit / runs;
  if (row >= p.rows) return;
  const int32_t blk0 = int32_t(unit - row * runs) * kRun;
  const T *x = static_cast<const T *>(p.x) + size_t(row) * p.ld + blk0 * ck::kBlock + lane;
  int8_t *codes = p.codes + (size_t(row) * p.nb + blk0) * ck::kBlock + lane;
  const int32_t left = p.cols - blk0 * ck::kBlock - lane, blocks = min(kRun, p.nb - blk0);
  float v[kRun];
#pragma unroll
  for (int j = 0; j < kRun; ++j) v[j] = 32 * j < left ? v8::to_float(x[32 * j]) : 0.f;
  uint32_t mine = 0;  // lane j keeps the scale of block j
#pragma unroll
  for (int j = 0; j < kRun; ++j) {
    const uint32_t s = ck::scale_of(__reduce_max_sync(0xFFFFFFFFu, ck::mag_bits(v[j])));
    if (lane == j) mine = s;
    if (j >= blocks) continue;
    float f[1] = {v[j]};
    ck::saturate(f, s);
    codes[32 * j] = s == 255u ? int8_t(0) : int8_t(ck::code_word(f[0], ck::up_of(s)) & 0xFFu);
  }
  if (lane < kRun && blk0 + lane < p.ns)  // runs start at multiples of 8: padding bytes included
    p.scales[size_t(row) * p.ns + blk0 + lane] = uint8_t(lane < blocks ? mine : 0u);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) unpack_lane_kernel(const Ckpt8Params p) {
  const uint32_t runs = (uint32_t(p.nb) + kRun - 1) / kRun;
  const uint32_t unit = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const uint32_t row = unit / runs;
  if (row >= p.rows) return;
  const int32_t blk0 = int32_t(unit - row * runs) * kRun;
  T *out = static_cast<T *>(p.out) + size_t(row) * p.ld + blk0 * ck::kBlock + lane;
  const int8_t *codes = p.codes + (size_t(row) * p.nb + blk0) * ck::kBlock + lane;
  const int32_t left = p.cols - blk0 * ck::kBlock - lane;
  int8_t code[kRun];
#pragma unroll
  for (int j = 0; j < kRun; ++j) code[j] = 32 * j < left ? codes[32 * j] : int8_t(0);
  uint32_t scale = 0;
  if (lane < kRun && blk0 + lane < p.nb) scale = p.scales[size_t(row) * p.ns + blk0 + lane];
#pragma unroll
  for (int j = 0; j < kRun; ++j) {
    const float unit_j = ck::unit_of(__shfl_sync(0xFFFFFFFFu, scale, j));
    if (32 * j >= left) continue;
    T o;
    v8::from_float(float(code[j]) * unit_j, o);
    out[32 * j] = o;
  }
}

template <typename T>
cudaError_t launch(const Ckpt8Params &p, bool unpack, bool vec, cudaStream_t stream) {
  const uint64_t units = vec ? p.total : uint64_t(p.rows) * ((p.nb + kRun - 1) / kRun);
  const uint32_t per_cta = !vec ? kThreads / 32 : unpack ? kThreads / 4 * kUnpackUnroll : kThreads / 2 * kUnroll;
  const unsigned grid = unsigned((units + per_cta - 1) / per_cta);
  if (unpack) {
    if (vec)
      unpack_vec_kernel<T><<<grid, kThreads, 0, stream>>>(p);
    else
      unpack_lane_kernel<T><<<grid, kThreads, 0, stream>>>(p);
  } else {
    if (vec)
      pack_vec_kernel<T><<<grid, kThreads, 0, stream>>>(p);
    else
      pack_lane_kernel<T><<<grid, kThreads, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_ckpt8(const Ckpt8Params &p, bool unpack, bool bf16, cudaStream_t stream) {
  const void *base = unpack ? p.out : p.x;
  const int64_t size = bf16 ? 2 : 4;
  const bool vec = p.cols % 8 == 0 && (reinterpret_cast<uintptr_t>(base) & 15u) == 0 && (p.ld * size) % 16 == 0;
  return bf16 ? launch<__nv_bfloat16>(p, unpack, vec, stream) : launch<float>(p, unpack, vec, stream);
}

}  // namespace caj

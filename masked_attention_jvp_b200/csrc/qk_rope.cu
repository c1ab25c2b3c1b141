// Rotary angles, and the norm + rotation of queries and keys with its tangent and
// its gradient.
//
// Per token and head, with r = sqrt(mean(x^2) + eps) over the head (or over the
// whole token, or with no norm at all) and R the rotation by the position's angles:
//   y  = R (g * x / r),   ty = R (g * (tx / r - x mean(x tx) / r^3))
// and for a gradient dq of y, with u = R^T dq:
//   dx = g u / r - x mean(x g u) / r^3,   dg = sum over tokens (and heads) of u x / r
// v is laid out anew and nothing else. Inputs are token-major [B, N, H D] with any
// distance between tokens (slices of one fused projection), outputs are the
// attention's [B, H, N, D]; the backward goes the other way.
//
// Everything here moves data: each element is read and written once, in 16-byte
// accesses, with fp32 arithmetic between (sums of squares, means and the gains'
// gradients too). A thread owns eight channels of one head for a run of tokens, so
// gains stay in registers; D/8 neighbouring lanes hold a head and reduce by
// shuffles. Pairs of the half layout (channels i and i + P) sit P/8 lanes apart and
// meet by a shuffle; interleaved pairs (2i, 2i + 1) are in one thread.
#include <cuda_runtime.h>

#include "ckpt8.cuh"
#include "kernels.h"
#include "vec8.cuh"

namespace caj {
namespace {

constexpr int kNormNone = 0, kNormHead = 1, kNormToken = 2;

// ------------------------------------------------------------- rotary angles
// cos and sin of pos * freq, scaled by mscale. The product is kept exactly, as a
// double and its rounding error (one fma), and reduced by multiples of pi/2 held
// in two doubles, so an angle of 10^9 radians is as exact as one of 1. The rest,
// |r| <= pi/4, goes through the Taylor series in fp32: sin to r^9 (the next term
// is below 2e-9 r), cos to r^10 (below 2e-10).
// Written once (8 bytes a pair), so bound by its stores; the 64-bit part is about
// ten instructions a pair, well under the 64 a clock that an SM issues.
__device__ __forceinline__ void cos_sin(double pos, double freq, float mscale, float &c, float &s) {
  const double hi = __dmul_rn(pos, freq), lo = __fma_rn(pos, freq, -hi);
  // 1.5 * 2^52 rounds to the nearest whole number, whose low bits it leaves in the mantissa
  const double shifted = __fma_rn(hi, 0.63661977236758134308, 6755399441055744.0);
  const int quadrant = __double2loint(shifted);
  const double k = shifted - 6755399441055744.0;
  double r = __fma_rn(-k, 1.5707963267948965580, hi);       // pi/2, leading 53 bits
  r = __fma_rn(-k, 6.1232339957367658860e-17, r) + lo;      // and the next 53
  const float x = float(r), x2 = x * x;
  float sn = fmaf(x2, 2.7557319e-6f, -1.9841270e-4f);
  sn = fmaf(x2, sn, 8.3333333e-3f);
  sn = fmaf(x2, sn, -1.6666667e-1f);
  sn = fmaf(x2 * x, sn, x);
  float cs = fmaf(x2, -2.7557319e-7f, 2.4801587e-5f);
  cs = fmaf(x2, cs, -1.3888889e-3f);
  cs = fmaf(x2, cs, 4.1666667e-2f);
  cs = fmaf(x2, cs, -0.5f);
  cs = fmaf(x2, cs, 1.f);
  const float a = quadrant & 1 ? cs : sn, b = quadrant & 1 ? sn : cs;
  s = (quadrant & 2 ? -a : a) * mscale;
  c = ((quadrant + 1) & 2 ? -b : b) * mscale;
}

// A thread owns V neighbouring pairs (V = 4: 16-byte stores) and walks over the
// positions, so frequencies and axes stay in registers.
template <typename I, int V>
__global__ void __launch_bounds__(256) rope_table_kernel(const RopeTableParams p) {
  const int32_t cols = p.P / V;  // threads across a row of pairs
  const int64_t id = int64_t(blockIdx.x) * 256 + threadIdx.x;
  const int64_t row0 = id / cols, step = int64_t(gridDim.x) * 256 / cols;  // a whole number of rows
  const int32_t i = int32_t(id - row0 * cols) * V;
  double freq[V];
  int32_t ax[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    freq[e] = __ldg(p.freq + i + e);
    ax[e] = p.axis ? __ldg(p.axis + i + e) : 0;
    if (ax[e] < 0 || ax[e] >= p.A) freq[e] = __longlong_as_double(0x7FF8000000000000ll), ax[e] = 0;  // NaN
  }
  for (int64_t n = row0; n < p.N; n += step) {
    float c[V], s[V];
#pragma unroll
    for (int e = 0; e < V; ++e)
      cos_sin(double(__ldg(static_cast<const I *>(p.pos) + n * p.A + ax[e])), freq[e], p.mscale, c[e], s[e]);
    const int64_t at = n * p.P + i;
    if constexpr (V == 4) {
      __stcs(reinterpret_cast<float4 *>(p.cos + at), make_float4(c[0], c[1], c[2], c[3]));
      __stcs(reinterpret_cast<float4 *>(p.sin + at), make_float4(s[0], s[1], s[2], s[3]));
    } else {
      p.cos[at] = c[0];
      p.sin[at] = s[0];
    }
  }
}

// ------------------------------------------------------------ norm + rotation
struct Lane {       // a thread's place in its tensor
  int32_t V, T;     // 8-channel vectors of a token, tokens a block takes at a time
  int32_t t, vec;   // this thread's token among T, and its vector
  bool on;
  int32_t head, d0;
};
__device__ __forceinline__ Lane lane_of(int32_t H, int32_t D) {
  Lane l;
  l.V = H * D / 8;
  l.T = int32_t(blockDim.x) / l.V;
  l.t = int32_t(threadIdx.x) / l.V;
  l.vec = int32_t(threadIdx.x) - l.t * l.V;
  l.on = l.t < l.T;
  l.head = 8 * l.vec / D;
  l.d0 = 8 * l.vec - l.head * D;
  return l;
}

// Cosines and sines for a thread's eight channels: interleaved four pairs (repeated
// for nothing: only the first four are read), half eight.
struct Angle {
  float c[8], s[8];
};
__device__ __forceinline__ void load4(const float *p, float *f) {
  const float4 a = __ldg(reinterpret_cast<const float4 *>(p));
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
}
__device__ __forceinline__ void load_angle(const QkRopeParams &p, int32_t n, int32_t d0, Angle &a) {
  const size_t row = size_t(n) * p.P;
  if (p.half) {
    const int32_t i = d0 < p.P ? d0 : d0 - p.P;
    load4(p.cos + row + i, a.c);
    load4(p.cos + row + i + 4, a.c + 4);
    load4(p.sin + row + i, a.s);
    load4(p.sin + row + i + 4, a.s + 4);
  } else {
    load4(p.cos + row + d0 / 2, a.c);
    load4(p.sin + row + d0 / 2, a.s);
  }
}
// Rotates a thread's eight channels; `sign` -1 turns back. Every lane of the warp
// comes here (the half layout shuffles), `turns` says whether its channels rotate.
__device__ __forceinline__ void rotate(float (&x)[8], const Angle &a, bool half, bool turns, bool first,
                                       int32_t hop, float sign) {
  if (half) {
    const int src = int(threadIdx.x & 31) + (turns ? (first ? hop : -hop) : 0);
    const float sg = first ? -sign : sign;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float other = __shfl_sync(0xFFFFFFFFu, x[i], src);
      if (turns) x[i] = fmaf(x[i], a.c[i], sg * a.s[i] * other);
    }
  } else if (turns) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float u = x[2 * i], w = x[2 * i + 1], s = sign * a.s[i];
      x[2 * i] = fmaf(u, a.c[i], -w * s);
      x[2 * i + 1] = fmaf(u, s, w * a.c[i]);
    }
  }
}

// Sums of a thread's M values over the norm's group: the head's lanes, or all
// vectors of the token through shared memory (`red`: [T][heads][M] floats).
template <int M>
__device__ __forceinline__ void group_sums(float (&v)[M], const Lane &l, int32_t norm, int32_t D, int32_t H,
                                           float *red) {
  for (int o = D / 16; o > 0; o >>= 1) {
#pragma unroll
    for (int i = 0; i < M; ++i) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], o);
  }
  if (norm != kNormToken) return;
  __syncthreads();  // the sums of the round before have been read
  if (l.on && l.d0 == 0) {
#pragma unroll
    for (int i = 0; i < M; ++i) red[(l.t * H + l.head) * M + i] = v[i];
  }
  __syncthreads();
  if (!l.on) return;
#pragma unroll
  for (int i = 0; i < M; ++i) v[i] = 0.f;
  for (int h = 0; h < H; ++h) {
#pragma unroll
    for (int i = 0; i < M; ++i) v[i] += red[(l.t * H + h) * M + i];
  }
}

__device__ __forceinline__ void load_gain(const float *g, const QkRopeParams &p, const Lane &l, float (&o)[8]) {
  const float *src = g + (p.gain_full ? 8 * l.vec : l.d0);
  load4(src, o);
  load4(src + 4, o + 4);
}

// Forward. Grid: token groups of T * U, and for each the tensors q, k, v next to each
// other, so that v's copies fill the memory's time while q and k are computed.
template <typename T, bool TAN, int U>
__global__ void __launch_bounds__(1024) qk_rope_fwd_kernel(const QkRopeParams p) {
  extern __shared__ float red[];
  const int which = int(blockIdx.x) % p.tensors;
  const int32_t group = int32_t(blockIdx.x) / p.tensors;
  const int32_t H = which == 0 ? p.Hq : p.Hk, D = p.D;
  const Lane l = lane_of(H, D);
  const int32_t rows = p.B * p.N;
  const T *x = static_cast<const T *>(p.x[which]), *tx = static_cast<const T *>(p.tx[which]);
  T *y = static_cast<T *>(p.y[which]), *ty = static_cast<T *>(p.ty[which]);
  const int64_t tok0 = int64_t(group) * l.T * U + l.t;

  v8::Raw<T> raw[U], traw[U];
  bool on[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t tok = tok0 + int64_t(u) * l.T;
    on[u] = l.on && tok < rows;
    raw[u] = v8::zero<T>();
    traw[u] = v8::zero<T>();
    if (on[u]) {
      raw[u] = v8::load(x + tok * p.ld[which] + 8 * l.vec);
      if (TAN) traw[u] = v8::load(tx + tok * p.tld[which] + 8 * l.vec);
    }
  }
  float g[8];
  const bool normed = which < 2 && p.norm != kNormNone;
  if (normed && l.on) load_gain(p.g[which], p, l, g);
  const bool turns = l.d0 < 2 * p.P, first = l.d0 < p.P;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int32_t tok = int32_t(tok0 + int64_t(u) * l.T);
    const int32_t b = on[u] ? tok / p.N : 0, n = on[u] ? tok - b * p.N : 0;
    const size_t out = ((size_t(b) * H + l.head) * p.N + n) * D + l.d0;
    if (which == 2) {
      if (on[u]) {
        v8::store(y + out, raw[u]);
        if (TAN) v8::store(ty + out, traw[u]);
      }
      continue;
    }
    float f[8], tf[8];
    v8::unpack(raw[u], f);
    if (TAN) v8::unpack(traw[u], tf);
    if (normed) {
      float sums[TAN ? 2 : 1];
      sums[0] = 0.f;
      if constexpr (TAN) sums[1] = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sums[0] = fmaf(f[i], f[i], sums[0]);
        if constexpr (TAN) sums[1] = fmaf(f[i], tf[i], sums[1]);
      }
      group_sums(sums, l, p.norm, D, H, red);
      const float inv_len = 1.f / float(p.norm == kNormHead ? D : H * D);
      const float inv = rsqrtf(fmaf(sums[0], inv_len, p.eps));
      if constexpr (TAN) {
        const float k3 = inv * inv * inv * (sums[1] * inv_len);
#pragma unroll
        for (int i = 0; i < 8; ++i) tf[i] = g[i] * fmaf(tf[i], inv, -f[i] * k3);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] *= g[i] * inv;
    }
    Angle a;
    if (turns && on[u]) load_angle(p, n, l.d0, a);
    rotate(f, a, p.half, turns, first, p.P / 8, 1.f);
    if (TAN) rotate(tf, a, p.half, turns, first, p.P / 8, 1.f);
    if (on[u]) {
      v8::Raw<T> o;
      v8::pack(f, o);
      v8::store(y + out, o);
      if (TAN) {
        v8::pack(tf, o);
        v8::store(ty + out, o);
      }
    }
  }
}

// Backward. p.blocks blocks for each tensor (q, k, v next to each other) walk over the
// token groups, so the gains' gradient stays in registers for a block's whole run; block
// i leaves its partial dg in p.partial[which][i].
// CK: x comes from an 8-bit checkpoint.
template <typename T, bool CK, int U>
__global__ void __launch_bounds__(1024) qk_rope_bwd_kernel(const QkRopeParams p) {
  extern __shared__ float red[];
  const int which = int(blockIdx.x) % p.tensors;
  const int32_t group = int32_t(blockIdx.x) / p.tensors;
  const int32_t H = which == 0 ? p.Hq : p.Hk, D = p.D;
  const Lane l = lane_of(H, D);
  const int32_t rows = p.B * p.N;
  const T *dy = static_cast<const T *>(p.dy[which]);
  T *dx = static_cast<T *>(p.dx[which]);
  const bool normed = which < 2 && p.norm != kNormNone;
  const int32_t ns = ck::scale_bytes(H * D);
  const int8_t *codes = static_cast<const int8_t *>(p.x[which]);
  const bool turns = l.d0 < 2 * p.P, first = l.d0 < p.P;
  float g[8], dg[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) g[i] = dg[i] = 0.f;
  if (normed && l.on) load_gain(p.g[which], p, l, g);
  const float inv_len = 1.f / float(p.norm == kNormHead ? D : H * D);

  for (int64_t base = int64_t(group) * l.T * U; base < rows; base += int64_t(p.blocks) * l.T * U) {
    v8::Raw<T> raw[U], xr[U];
    uint2 cw[U];
    uint32_t sc[U];
    bool on[U];
    int32_t nn[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t tok = base + int64_t(u) * l.T + l.t;
      on[u] = l.on && tok < rows;
      raw[u] = v8::zero<T>();
      if (!CK) xr[u] = v8::zero<T>();
      cw[u] = make_uint2(0, 0);
      sc[u] = 0;
      nn[u] = 0;
      if (on[u]) {
        const int32_t b = int32_t(tok) / p.N;
        nn[u] = int32_t(tok) - b * p.N;
        raw[u] = v8::load(dy + ((size_t(b) * H + l.head) * p.N + nn[u]) * D + l.d0);
        if (normed) {
          if (CK) {
            cw[u] = __ldcs(reinterpret_cast<const uint2 *>(codes + size_t(tok) * H * D + 8 * l.vec));
            sc[u] = __ldg(p.x_scales[which] + size_t(tok) * ns + l.vec / 4);
          } else {
            xr[u] = v8::load(static_cast<const T *>(p.x[which]) + tok * p.ld[which] + 8 * l.vec);
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      T *out = dx + (base + int64_t(u) * l.T + l.t) * int64_t(H) * D + 8 * l.vec;
      if (which == 2) {
        if (on[u]) v8::store(out, raw[u]);
        continue;
      }
      float f[8];
      v8::unpack(raw[u], f);
      Angle a;
      if (turns && on[u]) load_angle(p, nn[u], l.d0, a);
      rotate(f, a, p.half, turns, first, p.P / 8, -1.f);
      if (normed) {
        float xv[8], sums[2] = {0.f, 0.f};
        if (CK) {
          const float unit = ck::unit_of(sc[u]);
          ck::unpack_codes4(cw[u].x, unit, xv[0], xv[1], xv[2], xv[3]);
          ck::unpack_codes4(cw[u].y, unit, xv[4], xv[5], xv[6], xv[7]);
        } else {
          v8::unpack(xr[u], xv);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          sums[0] = fmaf(xv[i], xv[i], sums[0]);
          sums[1] = fmaf(xv[i], g[i] * f[i], sums[1]);
        }
        group_sums(sums, l, p.norm, D, H, red);
        const float inv = rsqrtf(fmaf(sums[0], inv_len, p.eps));
        const float k3 = inv * inv * inv * (sums[1] * inv_len);
        if (on[u]) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            dg[i] = fmaf(f[i], xv[i] * inv, dg[i]);
            f[i] = fmaf(g[i] * f[i], inv, -xv[i] * k3);
          }
        }
      }
      if (on[u]) {
        v8::Raw<T> o;
        v8::pack(f, o);
        v8::store(out, o);
      }
    }
  }
  if (!normed) return;
  // this block's dg: over its T tokens a round, and over the heads where they share a gain
  __syncthreads();
  if (l.on) {
#pragma unroll
    for (int i = 0; i < 8; ++i) red[(l.t * l.V + l.vec) * 8 + i] = dg[i];
  }
  __syncthreads();
  const int32_t len = p.gain_full ? H * D : D, width = H * D;
  float *part = p.partial[which] + size_t(group) * len;
  for (int32_t c = int32_t(threadIdx.x); c < len; c += int32_t(blockDim.x)) {
    float s = 0.f;
    for (int32_t t = 0; t < l.T; ++t)
      for (int32_t i = c; i < width; i += len) s += red[t * width + i];
    part[c] = s;
  }
}

// Sums the blocks' partial dg in a fixed order: 8 slices of the blocks, then the slices.
__global__ void __launch_bounds__(256) gain_grad_kernel(const QkRopeParams p) {
  __shared__ float s[8][32];
  const int which = blockIdx.y;
  const int32_t len = p.gain_full ? (which ? p.Hk : p.Hq) * p.D : p.D;
  const int32_t c = int32_t(blockIdx.x) * 32 + int32_t(threadIdx.x & 31), slice = int32_t(threadIdx.x >> 5);
  float acc = 0.f;
  if (c < len) {
#pragma unroll 8
    for (int32_t b = slice; b < p.blocks; b += 8) acc += p.partial[which][size_t(b) * len + c];
  }
  s[slice][threadIdx.x & 31] = acc;
  __syncthreads();
  if (slice == 0 && c < len) {
#pragma unroll
    for (int i = 1; i < 8; ++i) acc += s[i][threadIdx.x & 31];
    p.dg[which][c] = acc;
  }
}

// Threads of a block: whole tokens of the wider tensor, near 256.
int32_t threads_for(const QkRopeParams &p) {
  const int32_t V = (p.Hq > p.Hk ? p.Hq : p.Hk) * p.D / 8;
  const int32_t t = V >= 256 ? 1 : 256 / V;
  return (V * t + 31) & ~31;
}

template <typename T>
cudaError_t launch_fwd(const QkRopeParams &p, cudaStream_t stream) {
  const int32_t threads = threads_for(p);
  const bool tan = p.tx[0] != nullptr;
  const int32_t U = tan ? 2 : 4;
  const int32_t Vmax = (p.Hq > p.Hk ? p.Hq : p.Hk) * p.D / 8;
  const int32_t per = threads / Vmax * U;  // the narrower tensor takes more tokens a block
  const unsigned grid = unsigned((int64_t(p.B) * p.N + per - 1) / per) * unsigned(p.tensors);
  const size_t smem = p.norm == kNormToken ? size_t(threads) / (p.D / 8) * (tan ? 2 : 1) * sizeof(float) : 0;
  if (tan)
    qk_rope_fwd_kernel<T, true, 2><<<grid, threads, smem, stream>>>(p);
  else
    qk_rope_fwd_kernel<T, false, 4><<<grid, threads, smem, stream>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_bwd(const QkRopeParams &p, cudaStream_t stream) {
  const int32_t threads = threads_for(p);
  const unsigned grid = unsigned(p.blocks * p.tensors);
  const size_t smem = p.norm == kNormNone ? 0 : size_t(threads) * 8 * sizeof(float);
  if (p.x_scales[0])
    qk_rope_bwd_kernel<T, true, 2><<<grid, threads, smem, stream>>>(p);
  else
    qk_rope_bwd_kernel<T, false, 2><<<grid, threads, smem, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || p.norm == kNormNone) return e;
  const int32_t len = p.gain_full ? (p.Hq > p.Hk ? p.Hq : p.Hk) * p.D : p.D;
  gain_grad_kernel<<<dim3(unsigned((len + 31) / 32), 2), 256, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

namespace {
// The grid's threads are a whole number of rows: a multiple of `cols` blocks.
template <typename I, int V>
cudaError_t launch_table(const RopeTableParams &p, cudaStream_t stream) {
  const int64_t cols = p.P / V, most = 148 * 32;
  const int64_t want = (p.N * cols + 255) / 256;
  int64_t blocks = want < most ? want : most;
  blocks = (blocks + cols - 1) / cols * cols;
  rope_table_kernel<I, V><<<unsigned(blocks), 256, 0, stream>>>(p);
  return cudaGetLastError();
}
}  // namespace

cudaError_t launch_rope_table(const RopeTableParams &p, bool pos64, cudaStream_t stream) {
  const bool vec = p.P % 4 == 0 && ((reinterpret_cast<uintptr_t>(p.cos) | reinterpret_cast<uintptr_t>(p.sin)) & 15u) == 0;
  if (vec) return pos64 ? launch_table<int64_t, 4>(p, stream) : launch_table<int32_t, 4>(p, stream);
  return pos64 ? launch_table<int64_t, 1>(p, stream) : launch_table<int32_t, 1>(p, stream);
}

// Blocks of the backward a tensor: fixed by the sizes alone, so that the order of
// the gains' sums is too. Four blocks an SM for the three tensors together.
int32_t qk_rope_bwd_blocks(int32_t B, int32_t N, int32_t Hq, int32_t Hk, int32_t D) {
  QkRopeParams p{};
  p.Hq = Hq; p.Hk = Hk; p.D = D;
  const int32_t V = (Hq > Hk ? Hq : Hk) * D / 8;
  const int64_t groups = (int64_t(B) * N + threads_for(p) / V * 2 - 1) / (threads_for(p) / V * 2);
  const int64_t most = 148 * 4;
  return int32_t(groups < most ? groups : most);
}

cudaError_t launch_qk_rope_fwd(const QkRopeParams &p, bool bf16, cudaStream_t stream) {
  return bf16 ? launch_fwd<__nv_bfloat16>(p, stream) : launch_fwd<float>(p, stream);
}
cudaError_t launch_qk_rope_bwd(const QkRopeParams &p, bool bf16, cudaStream_t stream) {
  return bf16 ? launch_bwd<__nv_bfloat16>(p, stream) : launch_bwd<float>(p, stream);
}

}  // namespace caj

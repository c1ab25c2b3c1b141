// Internal launch interface between the C-ABI front end (api.cpp) and the CUDA
// translation units. Not part of the public header.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "mask_schedule.h"

namespace caj {

// Query-tile height of both kernels' work decomposition (rows per tile).
constexpr int kBlockM = 128;
// Key-tile width of the tensor-core kernel.
constexpr int kBlockN = 64;
// Largest number of query tiles per head the launch order table can hold.
constexpr int kMaxQTiles = 4096;

// Device error word values (first error wins). Low byte: where a wait gave up.
enum DeviceError : uint32_t {
  kErrNone = 0,
  kErrTimeoutBase = 0x100,     // | wait site
  kErrSmemMisaligned = 0x200,  // dynamic shared memory not 1 KiB aligned
  kErrTileKind = 0x300,        // a query tile outside the kind its launch covers
};

// Wait site of the signal barrier (kErrTimeoutBase | site when it gives up).
constexpr uint32_t kSiteSignalBarrier = 0xF0;

// Query tiles of one launch of the tensor-core forward. With clean-tangent-zero
// teacher forcing (tq, tk, tv vanish on rows < L) a call runs as two launches,
// one per kind of query tile: each kernel instantiation carries only its own
// kind's code, with no runtime branch on the kind.
enum TileKind : int32_t {
  kTilesAll = 0,       // dense tangents, every query tile
  kTilesNoisyCTZ = 1,  // clean-tangent-zero: tiles with a noisy row (q1 > L)
  kTilesCleanCTZ = 2,  // clean-tangent-zero: tiles of clean rows only (primal only)
};

// Largest number of sequence slices one output map scatters to: the GPUs of
// one NVSwitch domain.
constexpr int kMaxShards = 8;

// Where the output rows of a launch go. The packed sequence of N rows is cut
// into `shards` equal slices of `shard_len` rows; slice r lives in buffers
// o[r], to[r], lse[r], tlse[r]. In context-parallel (Ulysses) attention slice r
// belongs to rank r and those buffers are its memory, reached over NVLink, so
// the epilogue itself performs the output all-to-all. Head h of the launch
// (bh = b * heads + h) is head head_base + h of the heads_total heads each slice
// holds. O, tO: [B, heads_total, shard_len, D], or [B, shard_len, heads_total, D]
// when token_major (the input layout of the output projection). LSE, tLSE:
// [B, heads_total, shard_len]. One slice with head_base = 0 and
// heads_total = heads is the plain [B, H, N, D] output.
struct OutMap {
  void *o[kMaxShards], *to[kMaxShards];
  float *lse[kMaxShards], *tlse[kMaxShards];
  int32_t shards, shard_len;
  int32_t heads, head_base, heads_total;
  int32_t token_major;
};

// Output row q of head bh: its slice, its O/tO row (in units of D elements)
// and its LSE/tLSE element.
struct OutRow {
  int32_t shard;
  size_t row, stat;
};

__host__ __device__ inline OutRow slice_row(const OutMap &m, int32_t bh, int32_t q) {
  const int32_t b = bh / m.heads, h = m.head_base + bh % m.heads;
  const int32_t r = q / m.shard_len, ql = q - r * m.shard_len;
  OutRow o;
  o.shard = r;
  o.stat = (size_t(b) * m.heads_total + h) * m.shard_len + ql;
  o.row = m.token_major ? (size_t(b) * m.shard_len + ql) * m.heads_total + h : o.stat;
  return o;
}

// Element offset of output row q of head bh (= b H + h) in a one-slice output:
// [B, H, N, D] when out_heads == 0, else token-major [B, N, H, D] with
// H = out_heads. Equal to slice_row of the one-slice map, times D.
__host__ __device__ inline size_t out_row(int32_t bh, int32_t q, int32_t N, int32_t out_heads, int D) {
  if (out_heads == 0) return (size_t(bh) * N + q) * D;
  const int32_t b = bh / out_heads, h = bh % out_heads;
  return ((size_t(b) * N + q) * out_heads + h) * D;
}

struct Sm100Params {
  CUtensorMap tm_q, tm_tq, tm_k, tm_tk, tm_v, tm_tv;  // 3-D maps over [B*H, N, D]
  void *o, *to;          // one-slice output: [B*H, N, D] bf16
  float *lse, *tlse;     // [B*H, N]
  MaskGeom geom;
  int32_t BH;
  int32_t n_qtiles;
  float scale;           // softmax scale
  float scale_log2e;     // scale * log2(e)
  uint64_t timeout_ns;   // bounded-wait limit
  int32_t fault_mode;    // test hook: 1 = skip the query-tile copies
  int32_t tile_kind;     // TileKind: the query tiles this launch covers
  int32_t out_heads;     // H when O, tO are token-major [B, N, H, D]; 0: [B, H, N, D]
  uint16_t qtile_order[kMaxQTiles];  // heaviest query tiles first
  // Sequence slices of a context-parallel output. shards == 0: the launch
  // writes the one-slice output above; otherwise the scattering
  // instantiations write through this map and o, to, lse, tlse are unused.
  OutMap scatter;
};

struct SimtParams {
  const void *q, *k, *v, *tq, *tk, *tv;
  OutMap out;  // where O, tO (fp32) and LSE, tLSE rows go
  MaskGeom geom;
  int32_t BH;
  float scale;
};

struct PrologueParams {
  const void *xq, *xk, *xv, *txq, *txk, *txv;  // [B, N, H*D] bf16
  const float *gq, *gk;                        // [H*D]
  const float *rope_cos, *rope_sin;            // [N, D/2]
  void *q, *k, *v, *tq, *tk, *tv;              // [B, H, N, D] bf16
  int32_t B, N, H, D;
  float eps;
  int32_t per_head;
};

struct BwdParams {
  // dq kernel: streamed K, V (64-row boxes); Q and dO rows are read into TMEM;
  // dkdv kernel: resident V (128-row box), streamed Q, dO (64-row boxes); K
  // rows are read into TMEM
  CUtensorMap tm_k_s, tm_v_s, tm_v_r, tm_q_s, tm_do_s;
  const void *q, *k;      // [B*H, N, D] bf16
  const void *o, *dout;   // [B*H, N, D] bf16 (o for Delta only)
  const float *lse;       // [B*H, N] natural log, from the forward
  float *delta;           // [B*H, N] Delta = <dO, O> (written by the pre-pass)
  void *dq, *dk, *dv;     // [B*H, N, D] bf16
  MaskGeom geom;
  int32_t BH;
  int32_t n_row_tiles;    // ceil(N / 128), for both query and key tiles
  float scale;
  uint64_t timeout_ns;
  uint16_t row_order[kMaxQTiles];  // query tiles, heaviest first (dq kernel)
  uint16_t col_order[kMaxQTiles];  // key tiles, heaviest first (dkdv kernel)
  int32_t fault_mode;     // test hook: 1 = the producers issue no copies
};

// Output projection in primal-tangent form: y = x W^T + b, ty = tx W^T.
// 2-D bf16 maps, innermost dimension first, 128-byte swizzle:
//   tm_x, tm_tx over [M, K], box 64 x 128 (a CTA's half of a 256-row tile);
//   tm_w over [C, K], box 64 x 128 (a CTA's half of a 256-row weight tile);
//   tm_y, tm_ty over [M, C], box 64 x 32 (the epilogue's store box).
struct OutProjParams {
  CUtensorMap tm_x, tm_tx, tm_w, tm_y, tm_ty;
  const void *bias;      // [C] bf16 or null
  int32_t M, K, C;
  uint64_t timeout_ns;
  int32_t fault_mode;    // test hook: 1 = the producer issues no copies
};

// Rotary tables: cos, sin [N, P] of pos[n][axis[i]] * freq[i].
struct RopeTableParams {
  const void *pos;       // [N, A] int32 or int64
  const double *freq;    // [P]
  const int32_t *axis;   // [P], or null: all 0
  float *cos, *sin;      // [N, P]
  int64_t N;
  int32_t A, P;
  double mscale;
};

// Norm + rotation of q and k (and v's new layout), forward or backward; index 0, 1, 2
// is q, k, v.
struct QkRopeParams {
  const void *x[3], *tx[3];    // [B, N, heads * D], token distance ld / tld elements
  void *y[3], *ty[3];          // [B, heads, N, D]
  const void *dy[3];           // backward: [B, heads, N, D]
  void *dx[3];                 // [B, N, heads * D]
  const uint8_t *x_scales[2];  // backward: x[] holds an 8-bit checkpoint's codes, these its scales
  float *dg[2], *partial[2];   // gains' gradient; [blocks][gain length]
  int64_t ld[3], tld[3];
  const float *g[2];           // [D], or [heads * D] with gain_full
  const float *cos, *sin;      // [N, P]
  int32_t B, N, Hq, Hk, D, P;
  float eps;
  int32_t norm, half, gain_full;
  int32_t blocks;              // backward: all blocks, those of every share of the heads
  int32_t share_heads;         // heads a block has (set by the launch)
  int32_t ring, angle_slots;   // backward: tokens in a thread's ring of copies, slots for angles (set by the launch)
};

// Matrix products of the linear operators; the operands' maps have 128-byte-swizzled
// boxes of 64 bf16 columns (K-major A: 128 rows, 64 with tangents; K-major B: half a
// tile's columns; MN-major: 64).
constexpr int32_t kLinearFewRows = 32;  // rows (tangents counted) up to which W is streamed
struct LinearProblem {
  int32_t M, N;                                   // output rows and columns
  int32_t m_tiles, n_tiles, k_blocks;             // 0 tiles: not wanted
  int32_t splits, split_blocks;                   // parts of the contraction, blocks of a part
  int64_t part_rows;                              // rows of a part's buffer
};
struct LinearParams {
  CUtensorMap tm_a, tm_a2, tm_b;   // forward: x, tx, W; gradients: dz (64 x 64 boxes), -, W
  CUtensorMap tm_b2;               // gradients: x
  CUtensorMap tm_y, tm_y2;         // y, ty or dx, dW; 64-byte-swizzled boxes of 32 columns x 32 rows
  CUtensorMap tm_part, tm_part2;   // splits > 1: fp32 parts (of dW: the second), boxes of 16 x 32
  LinearProblem prob[2];           // the forward (or dx), and dW
  const void *x, *tx, *w;          // few rows: x, tx, W themselves; tx also says whether there are tangents
  const void *bias, *res, *tres;   // bf16 or null
  void *y, *ty;                    // [M, N] bf16; gradients: dx, dW
  float *part, *part2;             // [splits][1 or 2][part_rows][N]
  int8_t *codes;                   // z's 8-bit checkpoint, or null
  uint8_t *scales;
  int64_t ld_x, ld_tx, ld_res, ld_tres;
  int32_t K, tile_cols;
  int32_t nb, ns;
  int32_t act;
  int32_t fault_mode;              // test hook: 1 = the producer issues no copies
  uint64_t timeout_ns;
};
struct LinearDzParams {
  const void *dy;         // [M, C] bf16, rows ld_dy apart
  const int8_t *codes;    // z's checkpoint (act != none)
  const uint8_t *scales;
  void *dz;               // [M, C] bf16, rows ld_dz apart (act != none)
  float *partial;         // [chunks][C], or null
  int64_t M, ld_dy, ld_dz;
  int32_t C, nb, ns, act, chunk_rows;
  int32_t late;           // beside the products that went before (act = none: nothing of theirs is read)
};

// 8-bit checkpoints of `rows` rows: nb blocks and ns scale bytes a row, total = rows * nb.
struct Ckpt8Params {
  const void *x;       // pack: rows of `cols` values, ld elements apart
  void *out;           // unpack: likewise
  int8_t *codes;       // [rows, 32 nb]
  uint8_t *scales;     // [rows, ns]
  int64_t ld;
  uint32_t total, rows;
  int32_t cols, nb, ns;
};

// Signal barrier of a context-parallel group: pads[r] is rank r's pad of
// kMaxShards words as mapped in this process.
struct SignalParams {
  uint32_t *pads[kMaxShards];
  int32_t shards, rank;
  uint32_t epoch;
  uint64_t timeout_ns;
};

// Runs `set` (a per-device kernel attribute setting, e.g. its shared-memory
// limit) the first time a call site launches on the current device: function
// attributes hold per device, so a process that drives several GPUs sets them
// on each. `done` is the call site's bit set of devices (ordinals below 64).
template <class F>
inline cudaError_t once_per_device(std::atomic<uint64_t> &done, F set) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? (uint64_t(1) << dev) : 0;
  if (bit && (done.load() & bit)) return cudaSuccess;
  e = set();
  if (e == cudaSuccess && bit) done.fetch_or(bit);
  return e;
}

// Each returns the launch's cudaError_t (cudaSuccess when enqueued).
cudaError_t launch_fwd_jvp_sm100(const Sm100Params &p, int D, cudaStream_t stream);
cudaError_t launch_fwd_jvp_simt_f32(const SimtParams &p, int D, cudaStream_t stream);
cudaError_t launch_qk_norm_rope_jvp(const PrologueParams &p, cudaStream_t stream);
cudaError_t launch_attn_bwd_sm100(const BwdParams &p, int D, cudaStream_t stream);
cudaError_t read_and_clear_bwd_error(uint32_t *out);
cudaError_t launch_rope_table(const RopeTableParams &p, bool pos64, cudaStream_t stream);
cudaError_t launch_qk_rope_fwd(const QkRopeParams &p, bool bf16, cudaStream_t stream);
cudaError_t launch_qk_rope_bwd(const QkRopeParams &p, bool bf16, cudaStream_t stream);
int32_t qk_rope_bwd_blocks(int32_t B, int32_t N, int32_t Hq, int32_t Hk, int32_t D, int32_t norm);
cudaError_t launch_linear_fwd(const LinearParams &p, cudaStream_t stream);
// Up to two matrices of `rows` rows of `vecs` 16-byte vectors, copied to rows of another pitch
// (in vectors).
struct CopyRowsParams {
  const void *src[2];
  void *dst[2];
  int64_t ld_src[2], ld_dst[2];
  int64_t rows;
  int32_t vecs[2];
};
cudaError_t launch_copy_rows(const CopyRowsParams &p, int32_t matrices, cudaStream_t stream);
// `sums`: column sums alone (late), to run beside the products
cudaError_t launch_linear_grads(const LinearParams &p, const LinearDzParams *sums, cudaStream_t stream);
cudaError_t launch_linear_dz(const LinearDzParams &p, cudaStream_t stream);
cudaError_t launch_linear_db(const LinearDzParams &p, float *db, bool late, cudaStream_t stream);
int32_t linear_dz_chunk_rows(int64_t M, int32_t C);
cudaError_t read_and_clear_linear_error(uint32_t *out);
cudaError_t launch_ckpt8(const Ckpt8Params &p, bool unpack, bool bf16, cudaStream_t stream);
cudaError_t launch_signal_barrier(const SignalParams &p, cudaStream_t stream);
cudaError_t launch_out_proj_sm100(const OutProjParams &p, cudaStream_t stream);
cudaError_t read_and_clear_proj_error(uint32_t *out);
cudaError_t read_and_clear_signal_error(uint32_t *out);

// Device error word access (defined next to the kernels that write it).
cudaError_t read_and_clear_device_error(cudaStream_t stream, uint32_t *out);

}  // namespace caj

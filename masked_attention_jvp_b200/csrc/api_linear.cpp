// C-ABI front end of the linear operators (products with bias, activation and
// residual, their tangents and gradients): argument checks, the split of the
// contraction, tensor maps and workspaces (contracts: include/causaljvp.h).
#include <algorithm>

#include "api_internal.h"
#include "ckpt8.cuh"
#include "kernels.h"

using caj::aligned_to;

namespace {

caj_status done(cudaError_t e) { return e == cudaSuccess ? CAJ_OK : caj::cuda_fail(e); }

constexpr int64_t kTileRows = 256, kBlock = 64;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t padded(int64_t bytes) { return size_t((bytes + 255) & ~int64_t(255)); }

struct Plan {
  caj::LinearProblem prob;
  int64_t units, part_bytes;
  double unit_us, parts_us;
};
constexpr int64_t kPairs = 74;  // pairs of SMs, each at one tile (or part of one) at a time
constexpr int32_t kMaxSplits = 32;

// rows x cols outputs (and as many tangents), contraction of `depth` in `splits` parts, tiles
// of `tile_cols` columns. The estimates weigh one shape against another; they were fitted to
// the times on B200 of 154 shapes of each product (33 to 32760 tokens, 256 to 8192 channels),
// every width and up to 10 parts: the choice by them takes 0.7% longer than each shape's
// best forward and 1.0% longer backward, where figures from a few long products had taken
// 2.4% and 4.0%. A 64-wide block of the contraction takes a pair 0.35 us at
// 256 columns, 0.225 at 160 and 0.205 at 128, a tile 0.5 to 1 us besides. Parts cost 8
// bytes an output at 8 TB/s and a launch that adds them.
bool can_split(int32_t k_blocks, int32_t splits) {  // no part without blocks
  if (splits > k_blocks) return false;
  const int32_t per = (k_blocks + splits - 1) / splits;
  return (k_blocks + per - 1) / per == splits;
}
Plan plan_tiles(int64_t rows, int64_t cols, int64_t depth, bool tangent, int32_t tile_cols, int64_t splits) {
  Plan p{};
  const int64_t tile_rows = tangent ? kTileRows / 2 : kTileRows, ops = tangent ? 2 : 1;
  const int64_t m_tiles = ceil_div(rows, tile_rows), n_tiles = ceil_div(cols, tile_cols);
  const int64_t k_blocks = ceil_div(depth, kBlock), per = ceil_div(k_blocks, splits);
  const double block_us = tile_cols == 256 ? 0.35 : tile_cols == 160 ? 0.225 : 0.205;
  p.units = m_tiles * n_tiles * splits;
  p.unit_us = block_us * double(per) + (tile_cols == 256 ? 1.0 : tile_cols == 160 ? 0.8 : 0.5);
  if (splits > 1) p.parts_us = 1.0 + 0.3 * double(splits) + double(8 * splits * ops) * double(rows * cols) / 8e6;
  p.prob = {int32_t(rows), int32_t(cols), int32_t(m_tiles), int32_t(n_tiles), int32_t(k_blocks), int32_t(splits),
            int32_t(per), m_tiles * tile_rows};
  p.part_bytes = splits > 1 ? splits * ops * p.prob.part_rows * cols * 4 : 0;
  return p;
}
// One launch over a's units, then b's, dealt out to the pairs in turn: the longest share is
// the first pair's, or that of the first pair to begin with b. The launch that adds parts
// starts later (0.5 us) when no SM is free to hold its blocks before.
double launch_us(const Plan &a, const Plan &b) {
  const int64_t all = a.units + b.units, n = ceil_div(a.units, kPairs), turn = a.units % kPairs;
  const double first = double(n) * a.unit_us + double(ceil_div(all, kPairs) - n) * b.unit_us;
  const int64_t m = a.units / kPairs, of_b = all > turn ? ceil_div(all - turn, kPairs) - m : 0;
  const double parts = a.parts_us + b.parts_us + (a.part_bytes + b.part_bytes > 0 && all > 64 ? 0.5 : 0);
  return std::max(first, double(m) * a.unit_us + double(of_b) * b.unit_us) + parts;
}
// More parts are not looked at once every pair has several units: what imbalance is left is
// less than the parts cost.
bool enough(const Plan &p) { return p.units >= 4 * kPairs; }

// The forward's tiles: the width and split with the least estimate. Measured (primal and
// tangent, 1560 tokens, 1536 x 1536): 78 tiles of 256 columns 26.3 us, 156 of 128 columns
// 20.5, 130 of 160 columns 18.0.
struct FwdPlan : Plan {
  int32_t tile_cols;
};
FwdPlan plan_fwd(int64_t M, int64_t C, int64_t K, bool tangent) {
  FwdPlan best{};
  double best_us = 0;
  for (const int32_t tile_cols : {256, 160, 128}) {
    for (int32_t s = 1; s <= kMaxSplits; ++s) {
      if (!can_split(int32_t(ceil_div(K, kBlock)), s)) continue;
      const Plan p = plan_tiles(M, C, K, tangent, tile_cols, s);
      const double us = launch_us(p, Plan{});
      if (!best.tile_cols || us < best_us) {
        static_cast<Plan &>(best) = p;
        best.tile_cols = tile_cols;
        best_us = us;
      }
      if (enough(p)) break;
    }
  }
  return best;
}
// The gradients' tiles, dW's and then dx's in one launch: of each width dW's split beside an
// unsplit dx, then dx's beside that. Planned for both even where one is wanted, so that a
// gradient does not depend, in its last bits, on whether the other was asked for.
struct GradPlan {
  Plan dx, dw;
  int32_t tile_cols;
};
GradPlan plan_grads(int64_t M, int64_t C, int64_t K) {
  GradPlan best{};
  double best_us = 0;
  for (const int32_t tile_cols : {256, 128}) {
    GradPlan g{plan_tiles(M, K, C, false, tile_cols, 1), plan_tiles(C, K, M, false, tile_cols, 1), tile_cols};
    double us = launch_us(g.dw, g.dx);
    for (int32_t s = 2; s <= kMaxSplits && !enough(g.dw); ++s) {
      if (!can_split(int32_t(ceil_div(M, kBlock)), s)) continue;
      const Plan p = plan_tiles(C, K, M, false, tile_cols, s);
      const double t = launch_us(p, g.dx);
      if (t < us) g.dw = p, us = t;
      if (enough(p)) break;
    }
    for (int32_t s = 2; s <= kMaxSplits && !enough(g.dx); ++s) {
      if (!can_split(int32_t(ceil_div(C, kBlock)), s)) continue;
      const Plan p = plan_tiles(M, K, C, false, tile_cols, s);
      const double t = launch_us(g.dw, p);
      if (t < us) g.dx = p, us = t;
      if (enough(p)) break;
    }
    if (best.tile_cols && us >= best_us) continue;
    best = g;
    best_us = us;
  }
  return best;
}
bool few_rows(int64_t M, bool tangent) { return (tangent ? 2 : 1) * M <= caj::kLinearFewRows; }

bool part_map(CUtensorMap *map, const Plan &pl, bool tangent, void *parts) {
  return pl.prob.splits <= 1 || caj::encode_out_2d(map, parts, int64_t(pl.prob.splits) * (tangent ? 2 : 1) * pl.prob.part_rows,
                                                   pl.prob.N, true);
}

caj_status check_shape(const caj_linear_act_shape *s) {
  if (!s || s->M <= 0 || s->K <= 0 || s->C <= 0) return CAJ_ERR_INVALID_ARG;
  if (s->act < CAJ_ACT_NONE || s->act > CAJ_ACT_SILU) return CAJ_ERR_INVALID_ARG;
  if (s->K % 8 || s->C % 8) return CAJ_ERR_UNSUPPORTED;  // 16-byte rows
  // rows, tiles and parts are counted in 32 bits
  if (s->M > (int64_t(1) << 30) || s->K > (1 << 24) || s->C > (1 << 24)) return CAJ_ERR_UNSUPPORTED;
  const int64_t limit = (int64_t(1) << 31) - 1;
  if (ceil_div(s->M, 128) * ceil_div(std::max(s->K, s->C), 128) > limit / 32) return CAJ_ERR_UNSUPPORTED;
  if (ceil_div(s->K, 128) * ceil_div(s->C, 128) > limit / 32) return CAJ_ERR_UNSUPPORTED;
  if (s->M > limit / ceil_div(std::max(s->K, s->C), 32)) return CAJ_ERR_UNSUPPORTED;  // checkpoint blocks
  return CAJ_OK;
}
bool good_rows(const void *p, int64_t ld, int64_t width) {
  return p && aligned_to(p, 16) && ld >= width && ld % 8 == 0 && ld < (int64_t(1) << 36);
}

// Rows of the workspace's own matrices begin at a 128-byte line, so that a tile's 128-byte
// pieces of them lie in one line each (4485 x 4152 -> 776: gradients 66 us with both operands'
// rows at odd multiples of 16 bytes, 56 with both aligned).
int64_t row_of(int64_t width) { return (width + 63) & ~int64_t(63); }
// A caller's matrix [M, K] in rows at odd multiples of 16 bytes is copied to such rows first
// where the products read it often enough: `reuse` columns of output to each of its rows
// (9360 x 1624 -> 4104 135 to 118 us; 1032 columns 46 to 47, and from 296 channels, whose
// tiles their epilogue bounds, 32 to 37).
bool worth_copying(int64_t M, int64_t K, int64_t ld, int64_t reuse) {
  return ld % 16 != 0 && K >= 768 && reuse >= 2048 && double(M) * double(K) * double(reuse) >= 8e9;
}
// One of a launch's copies.
void add_copy(caj::CopyRowsParams *c, int32_t *n, const void *src, int64_t ld, int64_t M, int64_t K, void *dst) {
  c->src[*n] = src;
  c->dst[*n] = dst;
  c->ld_src[*n] = ld / 8;
  c->ld_dst[*n] = row_of(K) / 8;
  c->rows = M;
  c->vecs[*n] = int32_t(K / 8);
  ++*n;
}
struct FwdSizes {
  size_t parts, x, tx;
};
FwdSizes fwd_sizes(const caj_linear_act_shape *s, bool tangent, const Plan &plan) {
  FwdSizes f{};
  f.parts = padded(plan.part_bytes);
  if (worth_copying(s->M, s->K, s->ldx, s->C)) f.x = padded(s->M * row_of(s->K) * 2);
  if (tangent && worth_copying(s->M, s->K, s->ldtx, s->C)) f.tx = padded(s->M * row_of(s->K) * 2);
  return f;
}

struct BwdSizes {
  GradPlan grads;
  int32_t chunk_rows;
  bool copy_x, copy_dy;
  size_t x, dz, sums, dx_parts, dw_parts, total;
};
BwdSizes bwd_sizes(const caj_linear_act_shape *s, bool x_ckpt, bool want_dx, bool want_dw, bool want_db) {
  BwdSizes b{};
  b.grads = plan_grads(s->M, s->C, s->K);
  if (!want_dx) b.grads.dx = Plan{};
  if (!want_dw) b.grads.dw = Plan{};
  b.chunk_rows = caj::linear_dz_chunk_rows(s->M, s->C);
  b.copy_x = !x_ckpt && want_dw && worth_copying(s->M, s->K, s->ldx, s->C);
  b.copy_dy = s->act == CAJ_ACT_NONE && (want_dx || want_dw) &&
              worth_copying(s->M, s->C, s->ldy, s->K * (int(want_dx) + int(want_dw)));
  if ((x_ckpt && want_dw) || b.copy_x) b.x = padded(s->M * row_of(s->K) * 2);
  if (s->act != CAJ_ACT_NONE || b.copy_dy) b.dz = padded(s->M * row_of(s->C) * 2);
  if (want_db) b.sums = padded(ceil_div(s->M, b.chunk_rows) * s->C * 4);
  b.dx_parts = padded(b.grads.dx.part_bytes);
  b.dw_parts = padded(b.grads.dw.part_bytes);
  b.total = b.x + b.dz + b.sums + b.dx_parts + b.dw_parts;
  return b;
}

}  // namespace

extern "C" {

caj_status caj_linear_act_fwd_workspace(const caj_linear_act_shape *shape, int32_t tangent, size_t *bytes) {
  if (!bytes || (tangent != 0 && tangent != 1)) return CAJ_ERR_INVALID_ARG;
  const caj_status st = check_shape(shape);
  if (st != CAJ_OK) return st;
  *bytes = 0;
  if (few_rows(shape->M, tangent)) return CAJ_OK;
  const FwdSizes f = fwd_sizes(shape, tangent, plan_fwd(shape->M, shape->C, shape->K, tangent));
  *bytes = f.parts + f.x + f.tx;
  return CAJ_OK;
}

caj_status caj_linear_act_fwd(const void *x, const void *tx, const void *w, const void *bias, const void *res,
                              const void *tres, const caj_linear_act_shape *shape, void *y, void *ty,
                              int8_t *pre_codes, uint8_t *pre_scales, void *workspace, size_t workspace_bytes,
                              void *stream) {
  caj_status st = check_shape(shape);
  if (st != CAJ_OK) return st;
  const int64_t M = shape->M, K = shape->K, C = shape->C;
  const bool tan = tx != nullptr;
  if (!good_rows(x, shape->ldx, K) || !w || !aligned_to(w, 16) || !y || !aligned_to(y, 16)) return CAJ_ERR_INVALID_ARG;
  if (tan != (ty != nullptr) || (tan && (!good_rows(tx, shape->ldtx, K) || !aligned_to(ty, 16))))
    return CAJ_ERR_INVALID_ARG;
  if (bias && !aligned_to(bias, 16)) return CAJ_ERR_INVALID_ARG;
  if (res && !good_rows(res, shape->ldres, C)) return CAJ_ERR_INVALID_ARG;
  if (tres && (!tan || !good_rows(tres, shape->ldtres, C))) return CAJ_ERR_INVALID_ARG;
  if (!pre_codes != !pre_scales) return CAJ_ERR_INVALID_ARG;
  if (pre_codes && (!aligned_to(pre_codes, 32) || !aligned_to(pre_scales, 4))) return CAJ_ERR_INVALID_ARG;
  const bool few = few_rows(M, tan);
  const FwdPlan pl = plan_fwd(M, C, K, tan);
  const FwdSizes sizes = few ? FwdSizes{} : fwd_sizes(shape, tan, pl);
  const size_t need = sizes.parts + sizes.x + sizes.tx;
  if (need && (!workspace || !aligned_to(workspace, 16) || workspace_bytes < need)) return CAJ_ERR_INVALID_ARG;
  st = caj::check_device();
  if (st != CAJ_OK) return st;
  caj::LinearParams p{};
  p.x = x;
  p.tx = tx;
  p.w = w;
  p.bias = bias;
  p.res = res;
  p.tres = tres;
  p.y = y;
  p.ty = ty;
  p.codes = pre_codes;
  p.scales = pre_scales;
  p.ld_x = shape->ldx;
  p.ld_tx = shape->ldtx;
  p.ld_res = shape->ldres;
  p.ld_tres = shape->ldtres;
  p.nb = caj::ck::blocks_of(shape->C);
  p.ns = caj::ck::scale_bytes(shape->C);
  p.act = shape->act;
  p.prob[0] = pl.prob;
  p.K = shape->K;
  bool ok = true;
  if (!few) {
    p.tile_cols = pl.tile_cols;
    p.part = static_cast<float *>(workspace);
    p.timeout_ns = caj::wait_timeout_ns();
    p.fault_mode = caj::fault_mode();
    char *at = static_cast<char *>(workspace);
    caj::CopyRowsParams copies{};
    int32_t n = 0;
    int64_t ldx = shape->ldx, ldtx = shape->ldtx;
    if (sizes.x) {
      add_copy(&copies, &n, x, ldx, M, K, at + sizes.parts);
      x = at + sizes.parts;
      ldx = row_of(K);
    }
    if (sizes.tx) {
      add_copy(&copies, &n, tx, ldtx, M, K, at + sizes.parts + sizes.x);
      tx = at + sizes.parts + sizes.x;
      ldtx = row_of(K);
    }
    if (n) st = done(caj::launch_copy_rows(copies, n, static_cast<cudaStream_t>(stream)));
    if (st != CAJ_OK) return st;
    ok = part_map(&p.tm_part, pl, tan, workspace) &&
         caj::encode_map_2d_ld(&p.tm_a, x, M, K, ldx, tan ? 64 : 128) &&
         caj::encode_map_2d_ld(&p.tm_b, w, C, K, K, pl.tile_cols / 2) && caj::encode_out_2d(&p.tm_y, y, M, C, false);
    if (ok && tan)
      ok = caj::encode_map_2d_ld(&p.tm_a2, tx, M, K, ldtx, 64) &&
           caj::encode_out_2d(&p.tm_y2, ty, M, C, false);
  }
  if (!ok) return caj::cuda_fail(cudaErrorInvalidValue);
  return done(caj::launch_linear_fwd(p, static_cast<cudaStream_t>(stream)));
}

caj_status caj_linear_act_bwd_workspace(const caj_linear_act_shape *shape, int32_t x_ckpt, size_t *bytes) {
  if (!bytes || (x_ckpt != 0 && x_ckpt != 1)) return CAJ_ERR_INVALID_ARG;
  const caj_status st = check_shape(shape);
  if (st != CAJ_OK) return st;
  *bytes = bwd_sizes(shape, x_ckpt != 0, true, true, true).total;
  return CAJ_OK;
}

caj_status caj_linear_act_bwd(const void *dy, const void *x, const uint8_t *x_scales, const void *w,
                              const int8_t *pre_codes, const uint8_t *pre_scales, const caj_linear_act_shape *shape,
                              void *dx, void *dw, float *db, void *workspace, size_t workspace_bytes, void *stream) {
  caj_status st = check_shape(shape);
  if (st != CAJ_OK) return st;
  const int64_t M = shape->M, K = shape->K, C = shape->C;
  const bool act = shape->act != CAJ_ACT_NONE;
  if (!dx && !dw && !db) return CAJ_ERR_INVALID_ARG;
  if (!good_rows(dy, shape->ldy, C)) return CAJ_ERR_INVALID_ARG;
  if (dx && (!w || !aligned_to(w, 16) || !aligned_to(dx, 16))) return CAJ_ERR_INVALID_ARG;
  if (dw) {
    if (!aligned_to(dw, 16)) return CAJ_ERR_INVALID_ARG;
    if (x_scales ? (!x || !aligned_to(x, 16) || !aligned_to(x_scales, 4)) : !good_rows(x, shape->ldx, K))
      return CAJ_ERR_INVALID_ARG;
  }
  if (db && !aligned_to(db, 4)) return CAJ_ERR_INVALID_ARG;
  if (act && (!pre_codes || !aligned_to(pre_codes, 16) || !pre_scales || !aligned_to(pre_scales, 4)))
    return CAJ_ERR_INVALID_ARG;
  const BwdSizes b = bwd_sizes(shape, x_scales != nullptr, dx != nullptr, dw != nullptr, db != nullptr);
  if (b.total && (!workspace || !aligned_to(workspace, 256) || workspace_bytes < b.total)) return CAJ_ERR_INVALID_ARG;
  st = caj::check_device();
  if (st != CAJ_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  char *at = static_cast<char *>(workspace);
  void *x_values = at;
  void *dz = at + b.x;
  float *sums = reinterpret_cast<float *>(at + b.x + b.dz);
  char *parts = at + b.x + b.dz + b.sums;

  int64_t ld_dz = row_of(C);
  if (!act && !b.copy_dy) {
    dz = const_cast<void *>(dy);
    ld_dz = shape->ldy;
  }
  // db: the products do not wait for it. Without an activation its sums over dy run beside
  // them, with one the chunks' sums are added after them.
  const bool products = dx || dw;
  caj::LinearDzParams d{};
  if (act || db) {
    d.dy = dy;
    d.codes = pre_codes;
    d.scales = pre_scales;
    d.dz = dz;
    d.partial = db ? sums : nullptr;
    d.M = M;
    d.ld_dy = shape->ldy;
    d.ld_dz = ld_dz;
    d.C = shape->C;
    d.nb = caj::ck::blocks_of(shape->C);
    d.ns = caj::ck::scale_bytes(shape->C);
    d.act = shape->act;
    d.chunk_rows = b.chunk_rows;
    d.late = !act && products;
    if (!d.late) st = done(caj::launch_linear_dz(d, s));
    if (st != CAJ_OK) return st;
  }
  if (!products) return db ? done(caj::launch_linear_db(d, db, false, s)) : CAJ_OK;
  int64_t ld_x = shape->ldx;
  if (dw && x_scales) {
    caj::Ckpt8Params c{};
    c.codes = static_cast<int8_t *>(const_cast<void *>(x));
    c.scales = const_cast<uint8_t *>(x_scales);
    c.out = x_values;
    c.ld = ld_x = row_of(K);
    c.cols = shape->K;
    c.nb = caj::ck::blocks_of(shape->K);
    c.ns = caj::ck::scale_bytes(shape->K);
    c.total = uint32_t(M * c.nb);
    c.rows = uint32_t(M);
    st = done(caj::launch_ckpt8(c, true, true, s));
    if (st != CAJ_OK) return st;
    x = x_values;
  }
  caj::CopyRowsParams copies{};
  int32_t n = 0;
  if (b.copy_x) {
    add_copy(&copies, &n, x, ld_x, M, K, x_values);
    x = x_values;
    ld_x = row_of(K);
  }
  if (b.copy_dy) add_copy(&copies, &n, dy, shape->ldy, M, C, dz);
  if (n) st = done(caj::launch_copy_rows(copies, n, s));
  if (st != CAJ_OK) return st;
  caj::LinearParams p{};
  p.prob[0] = b.grads.dx.prob;
  p.prob[1] = b.grads.dw.prob;
  p.tile_cols = b.grads.tile_cols;
  p.y = dx;
  p.ty = dw;
  p.part = reinterpret_cast<float *>(parts);
  p.part2 = reinterpret_cast<float *>(parts + b.dx_parts);
  p.timeout_ns = caj::wait_timeout_ns();
  p.fault_mode = caj::fault_mode();
  bool ok = caj::encode_map_2d_ld(&p.tm_a, dz, M, C, ld_dz, 64);
  if (dx)
    ok = ok && caj::encode_map_2d_ld(&p.tm_b, w, C, K, K, 64) && caj::encode_out_2d(&p.tm_y, dx, M, K, false) &&
         part_map(&p.tm_part, b.grads.dx, false, p.part);
  if (dw)
    ok = ok && caj::encode_map_2d_ld(&p.tm_b2, x, M, K, ld_x, 64) && caj::encode_out_2d(&p.tm_y2, dw, C, K, false) &&
         part_map(&p.tm_part2, b.grads.dw, false, p.part2);
  if (!ok) return caj::cuda_fail(cudaErrorInvalidValue);
  st = done(caj::launch_linear_grads(p, d.late ? &d : nullptr, s));
  return st == CAJ_OK && db ? done(caj::launch_linear_db(d, db, !d.late, s)) : st;
}

}  // extern "C"

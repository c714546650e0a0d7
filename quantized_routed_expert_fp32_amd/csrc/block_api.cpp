// C entry points of the operators around the feed-forward block: argument
// validation, workspace layout, then the kernel launches.
#include <algorithm>
#include <cmath>

#include "api_checks.h"
#include "block_launch.h"

using namespace moe;

namespace {

constexpr int kMaxExperts = 1024, kMaxPicks = 64;
constexpr int kMaxRank = 256, kMaxAdapters = 1024;
constexpr int64_t kMaxAdapterStride = (int64_t)1 << 40;

int dt_of(int dtype) { return dtype == MOE_FP32 ? (int)DT_F32 : dtype; }

int check_norm(const char* fn, const moe_norm* a) {
  if (!a) return bad(std::string(fn) + ": NULL argument block");
  int st;
  if ((st = check_dim(fn, "rows", a->rows, kMaxRows)) || (st = check_dim(fn, "hidden", a->hidden, kMaxDim)) ||
      (st = check_dtype(fn, a->dtype)))
    return st;
  if (a->x_dtype != a->dtype && a->x_dtype != MOE_FP32)
    return bad(std::string(fn) + ": x_dtype " + std::to_string(a->x_dtype) + " is neither dtype nor MOE_FP32",
               MOE_EUNSUPPORTED);
  if (a->w_dtype != a->dtype && a->w_dtype != MOE_FP32)
    return bad(std::string(fn) + ": w_dtype " + std::to_string(a->w_dtype) + " is neither dtype nor MOE_FP32",
               MOE_EUNSUPPORTED);
  if (!(a->eps >= 1.17549435e-38f && a->eps <= 1.f))
    return bad(std::string(fn) + ": eps=" + std::to_string(a->eps) + " outside 2^-126..1");
  if (a->unit_offset != 0 && a->unit_offset != 1)
    return bad(std::string(fn) + ": unit_offset=" + std::to_string(a->unit_offset) + " is not 0 or 1");
  if (!a->x || !a->w) return bad(std::string(fn) + ": NULL x/w");
  if (!a->residual && a->x_dtype != a->dtype)
    return bad(std::string(fn) + ": x of MOE_FP32 without a residual", MOE_EUNSUPPORTED);
  if ((st = check_ld(fn, "ldx", a->ldx, a->hidden)) ||
      (a->residual && (st = check_ld(fn, "ldresidual", a->ldresidual, a->hidden))))
    return st;
  return MOE_OK;
}

NormArgs norm_args(const moe_norm* a, void* total, int64_t ldtotal) {
  NormArgs n{};
  n.rows = a->rows;
  n.hidden = a->hidden;
  n.x_dt = dt_of(a->x_dtype);
  n.w_dt = dt_of(a->w_dtype);
  n.eps = a->eps;
  n.w_add = (float)a->unit_offset;
  n.x = a->x;
  n.ldx = a->ldx;
  n.res = a->residual;
  n.ldres = a->ldresidual;
  n.w = a->w;
  n.total = total;
  n.ldtotal = ldtotal;
  return n;
}

int check_total(const char* fn, const moe_norm* a, const void* total, int64_t ldtotal) {
  if (!a->residual != !total)
    return bad(std::string(fn) + ": total is given with a residual, and only then");
  return total ? check_ld(fn, "ldtotal", ldtotal, a->hidden) : MOE_OK;
}

int check_balance(const char* fn, int rows, int experts, int k, int dtype, const void* logits, int64_t ld) {
  int st;
  if ((st = check_dim(fn, "rows", rows, kMaxRows)) || (st = check_dim(fn, "experts", experts, kMaxExperts)) ||
      (st = check_dim(fn, "k", k, std::min(experts, kMaxPicks))))
    return st;
  if (dtype != MOE_BF16 && dtype != MOE_FP16 && dtype != MOE_FP32)
    return bad(std::string(fn) + ": dtype " + std::to_string(dtype) + " is not MOE_BF16, MOE_FP16 or MOE_FP32",
               MOE_EUNSUPPORTED);
  if (!logits) return bad(std::string(fn) + ": NULL logits");
  return check_ld(fn, "ldlogits", ld, experts);
}

int check_lora(const char* fn, const moe_lora* a) {
  if (!a) return bad(std::string(fn) + ": NULL argument block");
  int st;
  if ((st = check_dim(fn, "rows", a->rows, kMaxRows)) || (st = check_dim(fn, "in", a->in, kMaxDim)) ||
      (st = check_dim(fn, "out", a->out, kMaxDim)) || (st = check_dim(fn, "rank", a->rank, kMaxRank)) ||
      (st = check_dim(fn, "adapters", a->adapters, kMaxAdapters)) || (st = check_dtype(fn, a->dtype)))
    return st;
  if (!a->x || !a->a || !a->b || !a->scale || !a->ids) return bad(std::string(fn) + ": NULL x/a/b/scale/ids");
  if ((st = check_ld(fn, "ldx", a->ldx, a->in)) || (st = check_ld(fn, "lda", a->lda, a->in)) ||
      (st = check_ld(fn, "ldb", a->ldb, a->rank)))
    return st;
  if (a->stride_a < 0 || a->stride_a > kMaxAdapterStride || a->stride_b < 0 || a->stride_b > kMaxAdapterStride)
    return bad(std::string(fn) + ": stride_a=" + std::to_string(a->stride_a) + ", stride_b=" +
               std::to_string(a->stride_b) + " outside 0..2^40", MOE_ESHAPE);
  return MOE_OK;
}

struct LoraPlan {
  int rp, blocks, max_tiles, splits, seg_rows, max_segs, slots;
  uint64_t hist_off, tiles_off, rows_off, hi_off, lo_off, fac_off, sums_off, segs_off, slot_off, span_off, u_off, top_off, part_off,
      total;
};

// dw: with the gradients of the adapters
LoraPlan plan_lora(const moe_lora* a, bool backward, bool dw) {
  LoraPlan p{};
  if (!backward && lora_by_row(a->rows, a->in, a->out, a->rank)) return p;
  const uint64_t R = a->rows;
  p.rp = (int)up(a->rank, 32);
  p.blocks = (a->rows + LORA_SORT - 1) / LORA_SORT;
  // an adapter's last tile may be short
  p.max_tiles = a->rows / LORA_TILE + std::min(a->adapters + 1, a->rows);
  Bump b;
  p.hist_off = b.take(p.blocks > 1 ? (uint64_t)p.blocks * (a->adapters + 1) * 4 : 0);
  p.tiles_off = b.take((uint64_t)p.max_tiles * 16);
  p.rows_off = b.take((uint64_t)p.max_tiles * LORA_TILE * 4);
  p.hi_off = b.take(R * p.rp * 2);
  p.lo_off = b.take(R * p.rp * 2);
  p.fac_off = b.take(R * 4);
  p.splits = lora_splits(a->rows, backward ? a->out : a->in, a->rank);
  p.sums_off = b.take((uint64_t)p.splits * R * up(a->rank, 4) * 4);
  p.u_off = b.take(R * a->rank * 4);       // t where the caller does not keep it, or u
  if (backward) {
    if (a->dtype == MOE_FP16) p.top_off = b.take((uint64_t)p.max_tiles * (LORA_TILE / 16) * 4 * 2);
  }
  if (dw) {
    // Rows of a segment: as many workgroups as fill the card twice, were the rows one
    // adapter's; every segment more costs its adapter's sums another trip through memory.
    const int64_t tiles = ((a->in + 255) / 256 + (a->out + 255) / 256) * (int64_t)((a->rank + 63) / 64);
    p.seg_rows = (int)std::max<int64_t>(up((a->rows * tiles + 511) / 512, LORA_TILE), 256);
    p.max_segs = a->rows / p.seg_rows + a->adapters;
    // only adapters of several segments have slots: m segments hold over (m - 1) seg_rows >= m / 2 seg_rows rows
    p.slots = 2 * (a->rows / p.seg_rows);
    p.segs_off = b.take((uint64_t)p.max_segs * 16);
    p.slot_off = b.take((uint64_t)p.max_segs * 4);
    p.span_off = b.take((uint64_t)a->adapters * 8);
    p.part_off = b.take((uint64_t)p.slots * a->rank * (a->in + (uint64_t)a->out) * 4);
  }
  p.total = b.at;
  return p;
}

LoraSort sort_args(const moe_lora* a, const LoraPlan& p, uint8_t* w) {
  LoraSort s{};
  s.rows = a->rows;
  s.adapters = a->adapters;
  s.ids = a->ids;
  s.blocks = p.blocks;
  s.hist = reinterpret_cast<int*>(w + p.hist_off);
  s.tiles = reinterpret_cast<int4*>(w + p.tiles_off);
  s.max_tiles = p.max_tiles;
  s.tile_rows = reinterpret_cast<int*>(w + p.rows_off);
  s.seg_rows = p.seg_rows;
  s.max_segs = p.max_segs;
  s.segs = reinterpret_cast<int4*>(w + p.segs_off);
  s.slot = reinterpret_cast<int*>(w + p.slot_off);
  s.span = reinterpret_cast<int2*>(w + p.span_off);
  return s;
}

// src [rows, k] through weights w into the parts of t
LoraShrink shrink_args(const moe_lora* a, const LoraPlan& p, uint8_t* w, int k, const void* src, int64_t ldsrc,
                       const void* weights, int64_t ldw, int64_t stw, float* t) {
  LoraShrink s{};
  s.k = k;
  s.rank = a->rank;
  s.rp = p.rp;
  s.adapters = a->adapters;
  s.src = src;
  s.ldsrc = ldsrc;
  s.w = weights;
  s.ldw = ldw;
  s.stw = stw;
  s.scale = a->scale;
  s.rows = reinterpret_cast<const int*>(w + p.rows_off);
  s.tiles = reinterpret_cast<const int4*>(w + p.tiles_off);
  s.max_tiles = p.max_tiles;
  s.splits = p.splits;
  s.part = reinterpret_cast<float*>(w + p.sums_off);
  s.places = a->rows;
  s.t = t ? t : reinterpret_cast<float*>(w + p.u_off);
  s.hi = reinterpret_cast<uint16_t*>(w + p.hi_off);
  s.lo = reinterpret_cast<uint16_t*>(w + p.lo_off);
  s.fac = reinterpret_cast<float*>(w + p.fac_off);
  return s;
}

LoraExpand expand_args(const moe_lora* a, const LoraPlan& p, uint8_t* w, int cols, const void* weights, int64_t ldw,
                       int64_t stw, const void* base, int64_t ldbase, void* dst, int64_t lddst) {
  LoraExpand e{};
  e.cols = cols;
  e.chunk = lora_chunk(a->rows, cols);
  e.rank = a->rank;
  e.rp = p.rp;
  e.adapters = a->adapters;
  e.w = weights;
  e.ldw = ldw;
  e.stw = stw;
  e.base = base;
  e.ldbase = ldbase;
  e.dst = dst;
  e.lddst = lddst;
  e.rows = reinterpret_cast<const int*>(w + p.rows_off);
  e.tiles = reinterpret_cast<const int4*>(w + p.tiles_off);
  e.max_tiles = p.max_tiles;
  e.hi = reinterpret_cast<const uint16_t*>(w + p.hi_off);
  e.lo = reinterpret_cast<const uint16_t*>(w + p.lo_off);
  e.fac = reinterpret_cast<const float*>(w + p.fac_off);
  return e;
}

}  // namespace

extern "C" {

int moe_norm_forward(const moe_norm* a, void* total, int64_t ldtotal, void* y, int64_t ldy, float* rstd, void* stream) {
  const char* fn = "moe_norm_forward";
  int st = check_norm(fn, a);
  if (st) return st;
  if (!y) return bad(std::string(fn) + ": NULL y");
  if ((st = check_total(fn, a, total, ldtotal)) || (st = check_ld(fn, "ldy", ldy, a->hidden))) return st;
  NormArgs n = norm_args(a, total, ldtotal);
  n.y = y;
  n.ldy = ldy;
  n.rstd = rstd;
  const hipError_t e = launch_norm(a->dtype, n, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_bad(fn, e);
}

int moe_norm_i8(const moe_norm* a, void* total, int64_t ldtotal, int8_t* q, int64_t ldq, float* scale, void* y,
                int64_t ldy, void* stream) {
  const char* fn = "moe_norm_i8";
  int st = check_norm(fn, a);
  if (st) return st;
  if (!q || !scale) return bad(std::string(fn) + ": NULL q/scale");
  if ((st = check_total(fn, a, total, ldtotal)) || (st = check_ld(fn, "ldq", ldq, a->hidden)) ||
      (y && (st = check_ld(fn, "ldy", ldy, a->hidden))))
    return st;
  NormArgs n = norm_args(a, total, ldtotal);
  n.q = q;
  n.ldq = ldq;
  n.scale = scale;
  n.y = y;
  n.ldy = ldy;
  const hipError_t e = launch_norm(a->dtype, n, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_bad(fn, e);
}

int moe_norm_backward_workspace_size(const moe_norm* a, uint64_t* bytes) {
  const char* fn = "moe_norm_backward_workspace_size";
  if (!bytes) return bad(std::string(fn) + ": NULL bytes");
  const int st = check_norm(fn, a);
  if (st) return st;
  *bytes = align256((uint64_t)norm_grad_words(a->rows, a->hidden) * 4);
  return MOE_OK;
}

int moe_norm_backward(const moe_norm* a, const float* rstd, const void* dy, int64_t lddy, const void* dtotal,
                      int64_t lddtotal, void* dx, int64_t lddx, void* dw, void* ws, uint64_t ws_bytes, void* stream) {
  const char* fn = "moe_norm_backward";
  int st = check_norm(fn, a);
  if (st) return st;
  if (a->residual) return bad(std::string(fn) + ": residual given (x is the forward call's total)");
  if (!rstd || !dy) return bad(std::string(fn) + ": NULL rstd/dy");
  if (!dx && !dw) return bad(std::string(fn) + ": no gradient asked for (dx and dw are NULL)");
  if (dtotal && !dx) return bad(std::string(fn) + ": dtotal without dx, the only gradient that it is part of");
  if ((st = check_ld(fn, "lddy", lddy, a->hidden)) || (dtotal && (st = check_ld(fn, "lddtotal", lddtotal, a->hidden))) ||
      (dx && (st = check_ld(fn, "lddx", lddx, a->hidden))))
    return st;
  const uint64_t need = dw ? align256((uint64_t)norm_grad_words(a->rows, a->hidden) * 4) : 0;
  if ((st = check_ws(fn, ws, ws_bytes, need))) return st;
  NormGradArgs g{};
  g.rows = a->rows;
  g.hidden = a->hidden;
  g.w_dt = dt_of(a->w_dtype);
  g.w_add = (float)a->unit_offset;
  g.x = a->x;
  g.ldx = a->ldx;
  g.w = a->w;
  g.rstd = rstd;
  g.dy = dy;
  g.lddy = lddy;
  g.dtotal = dtotal;
  g.lddtotal = lddtotal;
  g.dx = dx;
  g.lddx = lddx;
  g.dw = dw;
  g.part = static_cast<float*>(ws);
  const hipError_t e = launch_norm_grad(a->dtype, g, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_bad(fn, e);
}

int moe_balance_workspace_size(int rows, int experts, uint64_t* bytes) {
  const char* fn = "moe_balance_workspace_size";
  if (!bytes) return bad(std::string(fn) + ": NULL bytes");
  int st;
  if ((st = check_dim(fn, "rows", rows, kMaxRows)) || (st = check_dim(fn, "experts", experts, kMaxExperts))) return st;
  *bytes = align256((uint64_t)balance_part_words(rows, experts) * 4);
  return MOE_OK;
}

int moe_balance_forward(const void* logits, int dtype, int64_t ldlogits, const int32_t* ids, const uint8_t* mask, int rows,
                        int experts, int k, float* losses, int32_t* counts, void* ws, uint64_t ws_bytes, void* stream) {
  const char* fn = "moe_balance_forward";
  int st = check_balance(fn, rows, experts, k, dtype, logits, ldlogits);
  if (st) return st;
  if (!ids || !losses || !counts) return bad(std::string(fn) + ": NULL ids/losses/counts");
  if ((st = check_ws(fn, ws, ws_bytes, align256((uint64_t)balance_part_words(rows, experts) * 4)))) return st;
  BalanceArgs b{};
  b.rows = rows;
  b.experts = experts;
  b.k = k;
  b.logits = logits;
  b.ld = ldlogits;
  b.ids = ids;
  b.mask = mask;
  b.losses = losses;
  b.counts = counts;
  b.part = static_cast<float*>(ws);
  const hipError_t e = launch_balance(dt_of(dtype), b, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_bad(fn, e);
}

int moe_balance_backward(const float* dlosses, const void* logits, int dtype, int64_t ldlogits, const uint8_t* mask,
                         int rows, int experts, int k, const int32_t* counts, void* dlogits, int64_t lddlogits,
                         void* stream) {
  const char* fn = "moe_balance_backward";
  int st = check_balance(fn, rows, experts, k, dtype, logits, ldlogits);
  if (st) return st;
  if (!dlosses || !counts || !dlogits) return bad(std::string(fn) + ": NULL dlosses/counts/dlogits");
  if ((st = check_ld(fn, "lddlogits", lddlogits, experts))) return st;
  BalanceArgs b{};
  b.rows = rows;
  b.experts = experts;
  b.k = k;
  b.logits = logits;
  b.ld = ldlogits;
  b.mask = mask;
  b.counts = const_cast<int32_t*>(counts);
  b.dlosses = dlosses;
  b.dlogits = dlogits;
  b.ldd = lddlogits;
  const hipError_t e = launch_balance_grad(dt_of(dtype), b, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_bad(fn, e);
}

int moe_lora_workspace_size(const moe_lora* a, int kind, uint64_t* bytes) {
  const char* fn = "moe_lora_workspace_size";
  if (!bytes) return bad(std::string(fn) + ": NULL bytes");
  if (kind != MOE_LORA_FORWARD && kind != MOE_LORA_BACKWARD)
    return bad(std::string(fn) + ": kind " + std::to_string(kind) + " is not MOE_LORA_FORWARD or MOE_LORA_BACKWARD");
  const int st = check_lora(fn, a);
  if (st) return st;
  *bytes = plan_lora(a, kind == MOE_LORA_BACKWARD, kind == MOE_LORA_BACKWARD).total;
  return MOE_OK;
}

int moe_lora_forward(const moe_lora* a, const void* base, int64_t ldbase, void* y, int64_t ldy, float* t, void* ws,
                     uint64_t ws_bytes, void* stream) {
  const char* fn = "moe_lora_forward";
  int st = check_lora(fn, a);
  if (st) return st;
  if (!y) return bad(std::string(fn) + ": NULL y");
  if ((base && (st = check_ld(fn, "ldbase", ldbase, a->out))) || (st = check_ld(fn, "ldy", ldy, a->out))) return st;
  const LoraPlan p = plan_lora(a, false, false);
  if ((st = check_ws(fn, ws, ws_bytes, p.total))) return st;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e;
  if (!p.total) {
    LoraRow r{};
    r.rows = a->rows;
    r.in = a->in;
    r.out = a->out;
    r.rank = a->rank;
    r.adapters = a->adapters;
    r.x = a->x;
    r.ldx = a->ldx;
    r.a = a->a;
    r.lda = a->lda;
    r.sta = a->stride_a;
    r.b = a->b;
    r.ldb = a->ldb;
    r.stb = a->stride_b;
    r.scale = a->scale;
    r.ids = a->ids;
    r.base = base;
    r.ldbase = ldbase;
    r.y = y;
    r.ldy = ldy;
    r.t = t;
    e = launch_lora_row(a->dtype, r, s);
    return e == hipSuccess ? MOE_OK : hip_bad(fn, e);
  }
  uint8_t* w = static_cast<uint8_t*>(ws);
  e = launch_lora_sort(sort_args(a, p, w), s);
  if (e == hipSuccess)
    e = launch_lora_shrink(a->dtype, false,
                           shrink_args(a, p, w, a->in, a->x, a->ldx, a->a, a->lda, a->stride_a, t), s);
  if (e == hipSuccess)
    e = launch_lora_expand(a->dtype, false,
                           expand_args(a, p, w, a->out, a->b, a->ldb, a->stride_b, base, ldbase, y, ldy), s);
  return e == hipSuccess ? MOE_OK : hip_bad(fn, e);
}

int moe_lora_backward(const moe_lora* a, const void* dy, int64_t lddy, const float* t, const void* dx_base,
                      int64_t lddx_base, void* dx, int64_t lddx, void* da, void* db, void* ws, uint64_t ws_bytes,
                      void* stream) {
  const char* fn = "moe_lora_backward";
  int st = check_lora(fn, a);
  if (st) return st;
  if (!dy) return bad(std::string(fn) + ": NULL dy");
  if (!da != !db) return bad(std::string(fn) + ": da and db are both given or both NULL");
  if (!dx && !da) return bad(std::string(fn) + ": no gradient asked for (dx and da/db are NULL)");
  if (da && !t) return bad(std::string(fn) + ": NULL t (of the forward call), which db needs");
  if (dx_base && !dx) return bad(std::string(fn) + ": dx_base without dx");
  if ((st = check_ld(fn, "lddy", lddy, a->out)) || (dx_base && (st = check_ld(fn, "lddx_base", lddx_base, a->in))) ||
      (dx && (st = check_ld(fn, "lddx", lddx, a->in))))
    return st;
  const LoraPlan p = plan_lora(a, true, da != nullptr);
  if ((st = check_ws(fn, ws, ws_bytes, p.total))) return st;
  // (dx is written first; dx_base, which it may be, is easily the same tensor as dy)
  if (da && dx && (dx == a->x || dx == dy)) return bad(std::string(fn) + ": dx is x or dy, which da and db are computed from");
  uint8_t* w = static_cast<uint8_t*>(ws);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e = launch_lora_sort(sort_args(a, p, w), s);
  float* u = reinterpret_cast<float*>(w + p.u_off);
  LoraShrink k = shrink_args(a, p, w, a->out, dy, lddy, a->b, a->ldb, a->stride_b, u);
  if (da && a->dtype == MOE_FP16) {
    k.top = reinterpret_cast<uint32_t*>(w + p.top_off);
    k.top2 = k.top + (int64_t)p.max_tiles * (LORA_TILE / 16);
    k.t2 = t;
  }
  if (e == hipSuccess) e = launch_lora_shrink(a->dtype, true, k, s);
  if (e == hipSuccess && dx)
    e = launch_lora_expand(a->dtype, true,
                           expand_args(a, p, w, a->in, a->a, a->lda, a->stride_a, dx_base, lddx_base, dx, lddx), s);
  if (e == hipSuccess && da) {
    LoraGrad g{};
    g.rank = a->rank;
    g.in = a->in;
    g.out = a->out;
    g.adapters = a->adapters;
    g.u = u;
    g.t = t;
    g.x = a->x;
    g.ldx = a->ldx;
    g.dy = dy;
    g.lddy = lddy;
    g.scale = a->scale;
    g.rows = k.rows;
    g.segs = reinterpret_cast<const int4*>(w + p.segs_off);
    g.slot = reinterpret_cast<const int*>(w + p.slot_off);
    g.span = reinterpret_cast<const int2*>(w + p.span_off);
    g.max_segs = p.max_segs;
    g.join = a->rows > p.seg_rows;
    g.top_u = k.top;
    g.top_t = k.top2;
    g.da = da;
    g.db = db;
    g.part = reinterpret_cast<float*>(w + p.part_off);
    e = launch_lora_grad(a->dtype, g, s);
  }
  return e == hipSuccess ? MOE_OK : hip_bad(fn, e);
}

}  // extern "C"

// C entry points of the dense feed-forward operators: argument validation,
// workspace layout, tile choice, then the kernel launches.
#include <algorithm>
#include <string>

#include <hip/hip_runtime.h>

#include "api_checks.h"
#include "dense_launch.h"

using namespace moe;

namespace {

constexpr int kDecodeRows = 16;          // rows the decode form takes
constexpr int kPairRows = 32;            // rows whose dg and du go as high and low parts
// Rows the tile kernels read as they are: 16-byte aligned, whole 16-byte
// chunks. Others are copied to zero-padded rows in the workspace first.
bool plain_rows(const void* p, int64_t ld, int64_t cols, int es) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * es % 16 == 0 && cols * es % 16 == 0;
}

// K steps (128 bytes) of a contiguous contraction
int steps_of(int64_t kbytes) { return (int)((kbytes + 127) / 128); }

uint64_t part_bytes(int splits, int64_t nq, int64_t pcols) {
  return splits > 1 ? (uint64_t)splits * nq * pcols * 4 : 0;
}

struct GluPlan {
  bool decode, pad_x, pad_g, pad_u;
  bool quant, inner;      // x quantised into the workspace, or by the decode kernel itself
  int64_t kp;             // padded row length (elements)
  int tile, splits;
  uint64_t x_off, g_off, u_off, sx_off, part_off, total;
};

GluPlan plan_forward(const moe_glu* a, int dt) {
  GluPlan p{};
  const int es = dt == DT_I8 ? 1 : 2;
  p.decode = a->rows <= kDecodeRows;
  p.inner = dt == DT_I8 && !a->s_x && p.decode && dense_decode_quantises(EPI_GLU, a->rows, a->hidden, a->inter);
  p.quant = dt == DT_I8 && !a->s_x && !p.inner;
  p.kp = up(a->hidden, 16 / es);
  Bump b;
  p.pad_x = !p.quant && !p.decode && !plain_rows(a->x, a->ldx, a->hidden, es);
  p.pad_g = !p.decode && !plain_rows(a->w_gate, a->ldw_gate, a->hidden, es);
  p.pad_u = !p.decode && !plain_rows(a->w_up, a->ldw_up, a->hidden, es);
  if (p.quant || p.pad_x) p.x_off = b.take((uint64_t)a->rows * p.kp * es);
  if (p.quant) p.sx_off = b.take((uint64_t)a->rows * 4);
  if (p.pad_g) p.g_off = b.take((uint64_t)a->inter * p.kp * es);
  if (p.pad_u) p.u_off = b.take((uint64_t)a->inter * p.kp * es);
  p.splits = 1;
  if (!p.decode) {
    p.tile = dense_tile(EPI_GLU, a->inter, a->rows, steps_of(p.kp * es), &p.splits);
    p.part_off = b.take(part_bytes(p.splits, a->rows, 2 * up(a->inter, 4)));
  }
  p.total = b.at;
  return p;
}

struct GradPlan {
  bool pad_x, pad_g, pad_u, pairs;
  int64_t kp, ip;
  int parts;              // rows of D
  int tile_x, splits_x, tile_w, splits_w;
  uint64_t d_off, x_off, g_off, u_off, down_off, part_off, total;
};

GradPlan plan_backward(const moe_glu* a, bool dx, bool dw) {
  GradPlan p{};
  p.kp = up(a->hidden, 8);
  p.ip = up(a->inter, 64);
  Bump b;
  p.pairs = a->rows <= kPairRows;
  p.parts = p.pairs ? (int)up(a->rows, 16) * 2 : a->rows;
  p.d_off = b.take((uint64_t)p.parts * 2 * p.ip * 2);
  p.pad_x = dw && !p.pairs && !plain_rows(a->x, a->ldx, a->hidden, 2);
  p.pad_g = dx && !plain_rows(a->w_gate, a->ldw_gate, a->hidden, 2);
  p.pad_u = dx && !plain_rows(a->w_up, a->ldw_up, a->hidden, 2);
  if (p.pad_x || (dw && p.pairs)) p.x_off = b.take((uint64_t)p.parts * p.kp * 2);   // pairs: a DensePairs copy
  if (p.pad_g) p.g_off = b.take((uint64_t)a->inter * p.kp * 2);
  if (p.pad_u) p.u_off = b.take((uint64_t)a->inter * p.kp * 2);
  if (a->dtype == MOE_FP16) p.down_off = b.take((1 + GRAD_TOPS) * 4);
  p.splits_x = p.splits_w = 1;
  uint64_t part = 0;
  if (dx) {
    p.tile_x = dense_tile(EPI_OUT, a->hidden, p.parts, (int)(2 * p.ip / 64), &p.splits_x);
    part = std::max(part, part_bytes(p.splits_x, a->rows, up(a->hidden, 4)));
  }
  if (dw) {
    p.tile_w = dense_tile(EPI_OUT, a->hidden, (int)(2 * p.ip), (p.parts + 63) / 64, &p.splits_w);
    part = std::max(part, part_bytes(p.splits_w, 2 * p.ip, up(a->hidden, 4)));
  }
  p.part_off = b.take(part);
  p.total = b.at;
  return p;
}

int check_glu(const char* fn, const moe_glu* a, bool i8) {
  if (!a) return bad(std::string(fn) + ": NULL argument block");
  int st;
  if ((st = check_dim(fn, "rows", a->rows, kMaxRows)) || (st = check_dim(fn, "hidden", a->hidden, kMaxDim)) ||
      (st = check_dim(fn, "inter", a->inter, kMaxDim)) || (st = check_dtype(fn, a->dtype)))
    return st;
  if (a->act != MOE_ACT_SILU && a->act != MOE_ACT_GELU_TANH)
    return bad(std::string(fn) + ": act " + std::to_string(a->act) + " is not MOE_ACT_SILU or MOE_ACT_GELU_TANH",
               MOE_EUNSUPPORTED);
  if (!a->x || !a->w_gate || !a->w_up) return bad(std::string(fn) + ": NULL x/w_gate/w_up");
  if (i8 && (!a->s_gate || !a->s_up)) return bad(std::string(fn) + ": NULL s_gate/s_up");
  if (!i8 && (a->s_gate || a->s_up || a->s_x))
    return bad(std::string(fn) + ": scales given to the 16-bit form (moe_glu_i8 takes them)");
  if ((st = check_ld(fn, "ldx", a->ldx, a->hidden)) || (st = check_ld(fn, "ldw_gate", a->ldw_gate, a->hidden)) ||
      (st = check_ld(fn, "ldw_up", a->ldw_up, a->hidden)))
    return st;
  return MOE_OK;
}

// The operands as the tile kernels read them: copied to the workspace where
// the plan says so, by one launch (run).
struct Rows {
  const uint8_t* p;
  int64_t ld;   // bytes
};
struct Padder {
  DensePad j{};
  int n = 0, es;
  Padder(int cols, int64_t kp, int esize) : es(esize) {
    j.cols = cols;
    j.ldd = kp;
  }
  Rows take(bool pad, const void* src, int64_t ld, int rows, uint8_t* dst) {
    if (!pad) return {static_cast<const uint8_t*>(src), ld * es};
    j.src[n] = src;
    j.dst[n] = dst;
    j.ld[n] = ld;
    j.rows[n++] = rows;
    return {dst, j.ldd * es};
  }
  hipError_t run(hipStream_t s) const { return n ? launch_dense_pad(es, j, s) : hipSuccess; }   // a launch of its own
};

int glu_run(const char* fn, const moe_glu* a, int dt, void* h, int64_t ldh, float* gu, void* ws, uint64_t ws_bytes,
            void* stream) {
  if (!h) return bad(std::string(fn) + ": NULL h");
  int st = check_ld(fn, "ldh", ldh, a->inter);
  if (st) return st;
  const GluPlan p = plan_forward(a, dt);
  if ((st = check_ws(fn, ws, ws_bytes, p.total))) return st;
  uint8_t* w = static_cast<uint8_t*>(ws);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const int es = dt == DT_I8 ? 1 : 2;
  Padder pad(a->hidden, p.kp, es);
  Rows x = pad.take(p.pad_x, a->x, a->ldx, a->rows, w + p.x_off);
  const Rows g = pad.take(p.pad_g, a->w_gate, a->ldw_gate, a->inter, w + p.g_off);
  const Rows u = pad.take(p.pad_u, a->w_up, a->ldw_up, a->inter, w + p.u_off);
  hipError_t e;
  if (p.inner) x.ld = a->ldx * 2;
  if (p.quant) {
    e = launch_quant_rows(a->dtype, a->x, a->ldx, a->rows, a->hidden, reinterpret_cast<int8_t*>(w + p.x_off), p.kp,
                          reinterpret_cast<float*>(w + p.sx_off), &pad.j, s);
    x = {w + p.x_off, p.kp};
  } else {
    e = pad.run(s);
  }
  if (e != hipSuccess) return hip_bad(fn, e);
  DenseArgs d{};
  d.p0 = g.p;
  d.p1 = u.p;
  d.q0 = x.p;
  d.ldp0 = g.ld;
  d.ldp1 = u.ld;
  d.ldq = x.ld;
  d.np = a->inter;
  d.nq = a->rows;
  d.kbytes = (int)(p.kp * es);
  d.splits = p.splits;
  d.act = a->act;
  d.out0 = h;
  d.ldo = ldh;
  d.out_dt = a->dtype;
  d.save = gu;
  if (dt == DT_I8) {
    d.sq = p.quant ? reinterpret_cast<const float*>(w + p.sx_off) : a->s_x;
    d.sp0 = a->s_gate;
    d.sp1 = a->s_up;
  }
  d.part = reinterpret_cast<float*>(w + p.part_off);
  d.pcols = 2 * up(a->inter, 4);
  if (p.decode) e = launch_dense_decode(dt, EPI_GLU, p.inner ? a->dtype : DT_I8, DenseDecodeArgs{d, a->hidden}, s);
  else e = launch_dense(dt, EPI_GLU, FORM_NT, p.tile, d, s);
  return e == hipSuccess ? MOE_OK : hip_bad(fn, e);
}

struct LinPlan {
  bool decode, pad_x, pad_w, quant, inner;
  int64_t kp;
  int tile, splits;
  uint64_t x_off, sx_off, w_off, part_off, total;
};

LinPlan plan_linear(const moe_linear* a) {
  LinPlan p{};
  p.decode = a->rows <= kDecodeRows;
  p.inner = !a->s_x && p.decode && dense_decode_quantises(EPI_SCALE, a->rows, a->in, a->out);
  p.quant = !a->s_x && !p.inner;
  p.kp = up(a->in, 16);
  Bump b;
  p.pad_x = !p.quant && !p.decode && !plain_rows(a->x, a->ldx, a->in, 1);
  p.pad_w = !p.decode && !plain_rows(a->w, a->ldw, a->in, 1);
  if (p.quant || p.pad_x) p.x_off = b.take((uint64_t)a->rows * p.kp);
  if (p.quant) p.sx_off = b.take((uint64_t)a->rows * 4);
  if (p.pad_w) p.w_off = b.take((uint64_t)a->out * p.kp);
  p.splits = 1;
  if (!p.decode) {
    p.tile = dense_tile(EPI_SCALE, a->out, a->rows, steps_of(p.kp), &p.splits);
    p.part_off = b.take(part_bytes(p.splits, a->rows, up(a->out, 4)));
  }
  p.total = b.at;
  return p;
}

int check_linear(const char* fn, const moe_linear* a) {
  if (!a) return bad(std::string(fn) + ": NULL argument block");
  int st;
  if ((st = check_dim(fn, "rows", a->rows, kMaxRows)) || (st = check_dim(fn, "in", a->in, kMaxDim)) ||
      (st = check_dim(fn, "out", a->out, kMaxDim)) || (st = check_dtype(fn, a->dtype)))
    return st;
  if (!a->x || !a->w || !a->s_w) return bad(std::string(fn) + ": NULL x/w/s_w");
  if ((st = check_ld(fn, "ldx", a->ldx, a->in)) || (st = check_ld(fn, "ldw", a->ldw, a->in))) return st;
  return MOE_OK;
}

}  // namespace

// Tile (see launch_dense) and K ranges of a product: the choice of least cost
// under a model of a tile's start and end, of a 128-byte K step with one
// workgroup on a CU and with two, of the join of several ranges and of their
// partial sums (bytes through memory). The weights are fitted so that the
// choice agrees with graph replays of 95 products (rows 24..4096, hidden
// 512..8192, inter 512..8192, every tile with 1 to 4 ranges timed for each; all
// 95 are the fit's own, none held back): for 88 of them its time is 0.3% above
// the best timed one on average, 8% at most (1024 x 4096 -> 2048 in 38.2 us
// against 35.3); for the other 7 it takes 6 or 8 ranges, which were not timed. One tile for all would cost more: 700 x
// 4096 -> 2 x 2000 takes 79 us on 256 x 256, 40 on 128 x 128, 33 on it in
// 256-byte steps, 45 on 64 x 64; 512 x 2048 -> 2 x 512 takes 43, 18, 18 and 12.
int moe::dense_tile(int epi, int np, int nq, int steps, int* splits) {
  static const struct {
    int edge, per_cu;
    double step1, step2, fixed;
  } kTile[4] = {{256, 1, 1.60, 1.60, 11.4}, {128, 2, 0.73, 1.12, 7.0}, {64, 2, 0.27, 0.48, 5.1}, {128, 1, 0.56, 0.56, 10.2}};
  constexpr double kJoin = 3.1, kJoinByte = 1e-6 / 6.4;
  const int cus = 256, glu = epi == EPI_GLU ? 2 : 1;
  double best = 0;
  int tile = -1;
  for (int t = 0; t < 4; ++t) {
    const int op = kTile[t].edge / glu;
    const int64_t n = (int64_t)((np + op - 1) / op) * ((nq + kTile[t].edge - 1) / kTile[t].edge);
    for (int s = 1; s <= 8 && (s == 1 || steps >= 4 * s); ++s) {
      const int64_t wgs = n * s, full = wgs / (cus * kTile[t].per_cu), rest = wgs % (cus * kTile[t].per_cu);
      const int st = (steps + s - 1) / s;
      double us = full * (kTile[t].fixed + st * kTile[t].step2);
      if (rest) us += kTile[t].fixed + st * (rest <= cus ? kTile[t].step1 : kTile[t].step2);
      if (s > 1) us += kJoin + kJoinByte * 8 * s * nq * np * glu;
      if (tile < 0 || us < best) {
        best = us;
        tile = t;
        *splits = s;
      }
    }
  }
  return tile;
}

extern "C" {

int moe_glu_workspace_size(const moe_glu* a, int kind, uint64_t* bytes) {
  const char* fn = "moe_glu_workspace_size";
  if (!bytes) return bad(std::string(fn) + ": NULL bytes");
  if (kind < MOE_GLU_FORWARD || kind > MOE_GLU_I8)
    return bad(std::string(fn) + ": kind " + std::to_string(kind) +
               " is not MOE_GLU_FORWARD, MOE_GLU_BACKWARD or MOE_GLU_I8");
  int st = check_glu(fn, a, kind == MOE_GLU_I8);
  if (st) return st;
  *bytes = kind == MOE_GLU_BACKWARD ? plan_backward(a, true, true).total
                                    : plan_forward(a, kind == MOE_GLU_I8 ? DT_I8 : a->dtype).total;
  return MOE_OK;
}

int moe_glu_forward(const moe_glu* a, void* h, int64_t ldh, float* gu, void* ws, uint64_t ws_bytes, void* stream) {
  int st = check_glu("moe_glu_forward", a, false);
  return st ? st : glu_run("moe_glu_forward", a, a->dtype, h, ldh, gu, ws, ws_bytes, stream);
}

int moe_glu_i8(const moe_glu* a, void* h, int64_t ldh, void* ws, uint64_t ws_bytes, void* stream) {
  int st = check_glu("moe_glu_i8", a, true);
  return st ? st : glu_run("moe_glu_i8", a, DT_I8, h, ldh, nullptr, ws, ws_bytes, stream);
}

int moe_glu_backward(const moe_glu* a, const float* gu, const void* dh, int64_t lddh, void* dx, int64_t lddx,
                     void* dw_gate, void* dw_up, void* ws, uint64_t ws_bytes, void* stream) {
  const char* fn = "moe_glu_backward";
  int st = check_glu(fn, a, false);
  if (st) return st;
  if (!gu || !dh) return bad(std::string(fn) + ": NULL gu/dh");
  if (!dw_gate != !dw_up) return bad(std::string(fn) + ": dw_gate and dw_up are both given or both NULL");
  if (!dx && !dw_gate) return bad(std::string(fn) + ": no gradient asked for (dx and dw_gate/dw_up are NULL)");
  if ((st = check_ld(fn, "lddh", lddh, a->inter)) || (dx && (st = check_ld(fn, "lddx", lddx, a->hidden)))) return st;
  const GradPlan p = plan_backward(a, dx != nullptr, dw_gate != nullptr);
  if ((st = check_ws(fn, ws, ws_bytes, p.total))) return st;
  uint8_t* w = static_cast<uint8_t*>(ws);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  Padder pad(a->hidden, p.kp, 2);
  Rows x = pad.take(p.pad_x, a->x, a->ldx, a->rows, w + p.x_off);
  DensePairs px{};
  if (p.pairs && dw_gate) {
    px = {a->x, w + p.x_off, a->ldx, p.kp, a->rows, a->hidden};
    x = {w + p.x_off, p.kp * 2};
  }
  const Rows g = pad.take(p.pad_g, a->w_gate, a->ldw_gate, a->inter, w + p.g_off);
  const Rows u = pad.take(p.pad_u, a->w_up, a->ldw_up, a->inter, w + p.u_off);
  hipError_t e = launch_glu_grad(a->dtype, p.pairs, a->act, dh, lddh, gu, a->rows, a->inter, (int)p.ip, w + p.d_off,
                                 pad.j, px, reinterpret_cast<float*>(w + p.down_off), s);
  if (e != hipSuccess) return hip_bad(fn, e);
  DenseArgs d{};
  d.q0 = w + p.d_off;
  d.ldq = 2 * p.ip * 2;
  d.np = a->hidden;
  d.fold = p.pairs ? a->rows : 0;
  d.down = reinterpret_cast<const float*>(w + p.down_off);
  d.out_dt = a->dtype;
  d.part = reinterpret_cast<float*>(w + p.part_off);
  d.pcols = up(a->hidden, 4);
  if (dx) {
    // dx[r] = sum_i dg[r, i] Wg[i] + du[r, i] Wu[i]: both sums one contraction
    DenseArgs dd = d;
    dd.p0 = g.p;
    dd.p1 = u.p;
    dd.ldp0 = g.ld;
    dd.ldp1 = u.ld;
    dd.nq = p.parts;
    dd.kbytes = (int)(2 * p.ip * 2);
    dd.krows = a->inter;
    dd.segbytes = (int)(p.ip * 2);
    dd.splits = p.splits_x;
    dd.out0 = dx;
    dd.ldo = lddx;
    e = launch_dense(a->dtype, EPI_OUT, FORM_NN, p.tile_x, dd, s);
    if (e != hipSuccess) return hip_bad(fn, e);
  }
  if (dw_gate) {
    // [dWg; dWu] = D^T x
    DenseArgs dd = d;
    dd.p0 = x.p;
    dd.ldp0 = x.ld;
    dd.nq = (int)(2 * p.ip);
    dd.krows = p.parts;
    dd.splits = p.splits_w;
    dd.out0 = dw_gate;
    dd.out1 = dw_up;
    dd.ldo = a->hidden;
    dd.qseg = a->inter;
    dd.qpad = (int)p.ip;
    e = launch_dense(a->dtype, EPI_OUT, FORM_TN, p.tile_w, dd, s);
    if (e != hipSuccess) return hip_bad(fn, e);
  }
  return MOE_OK;
}

int moe_quant_rows(const void* x, int dtype, int rows, int cols, int64_t ldx, int8_t* q, int64_t ldq, float* scale,
                   void* stream) {
  const char* fn = "moe_quant_rows";
  if (!x || !q || !scale) return bad(std::string(fn) + ": NULL x/q/scale");
  if (dtype != MOE_BF16 && dtype != MOE_FP16 && dtype != MOE_FP32)
    return bad(std::string(fn) + ": dtype " + std::to_string(dtype) + " is not MOE_BF16, MOE_FP16 or MOE_FP32",
               MOE_EUNSUPPORTED);
  int st;
  if ((st = check_dim(fn, "rows", rows, kMaxRows)) || (st = check_dim(fn, "cols", cols, kMaxDim)) ||
      (st = check_ld(fn, "ldx", ldx, cols)) || (st = check_ld(fn, "ldq", ldq, cols)))
    return st;
  hipError_t e = launch_quant_rows(dtype == MOE_FP32 ? DT_F32 : dtype, x, ldx, rows, cols, q, ldq, scale, nullptr,
                                   static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MOE_OK : hip_bad(fn, e);
}

int moe_linear_i8_workspace_size(const moe_linear* a, uint64_t* bytes) {
  const char* fn = "moe_linear_i8_workspace_size";
  if (!bytes) return bad(std::string(fn) + ": NULL bytes");
  int st = check_linear(fn, a);
  if (st) return st;
  *bytes = plan_linear(a).total;
  return MOE_OK;
}

int moe_linear_i8(const moe_linear* a, void* y, int64_t ldy, void* ws, uint64_t ws_bytes, void* stream) {
  const char* fn = "moe_linear_i8";
  int st = check_linear(fn, a);
  if (st) return st;
  if (!y) return bad(std::string(fn) + ": NULL y");
  if ((st = check_ld(fn, "ldy", ldy, a->out))) return st;
  const LinPlan p = plan_linear(a);
  if ((st = check_ws(fn, ws, ws_bytes, p.total))) return st;
  uint8_t* w = static_cast<uint8_t*>(ws);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  Padder pad(a->in, p.kp, 1);
  Rows x = pad.take(p.pad_x, a->x, a->ldx, a->rows, w + p.x_off);
  const Rows m = pad.take(p.pad_w, a->w, a->ldw, a->out, w + p.w_off);
  hipError_t e;
  if (p.inner) x.ld = a->ldx * 2;
  if (p.quant) {
    e = launch_quant_rows(a->dtype, a->x, a->ldx, a->rows, a->in, reinterpret_cast<int8_t*>(w + p.x_off), p.kp,
                          reinterpret_cast<float*>(w + p.sx_off), &pad.j, s);
    x = {w + p.x_off, p.kp};
  } else {
    e = pad.run(s);
  }
  if (e != hipSuccess) return hip_bad(fn, e);
  DenseArgs d{};
  d.p0 = m.p;
  d.q0 = x.p;
  d.ldp0 = m.ld;
  d.ldq = x.ld;
  d.np = a->out;
  d.nq = a->rows;
  d.kbytes = (int)p.kp;
  d.splits = p.splits;
  d.out0 = y;
  d.ldo = ldy;
  d.out_dt = a->dtype;
  d.sq = p.quant ? reinterpret_cast<const float*>(w + p.sx_off) : a->s_x;
  d.sp0 = a->s_w;
  d.bias = a->bias;
  d.part = reinterpret_cast<float*>(w + p.part_off);
  d.pcols = up(a->out, 4);
  if (p.decode) e = launch_dense_decode(DT_I8, EPI_SCALE, p.inner ? a->dtype : DT_I8, DenseDecodeArgs{d, a->in}, s);
  else e = launch_dense(DT_I8, EPI_SCALE, FORM_NT, p.tile, d, s);
  return e == hipSuccess ? MOE_OK : hip_bad(fn, e);
}

}  // extern "C"

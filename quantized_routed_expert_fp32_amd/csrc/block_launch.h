// Argument blocks and launchers of the operators around the feed-forward block:
// the norm before it, the balance loss of its router, low-rank adapters beside
// its projections (internal to the library).
#pragma once
#include "dense_launch.h"

namespace moe {

// ------------------------------------------------------------------ norm
// Rows [rows, hidden]; strides in elements.
struct NormArgs {
  int rows, hidden, x_dt, w_dt;     // x: the result's type or DT_F32; w: the same choice
  float eps, w_add;                 // w_add: 1 where the weight counts from 1
  const void* x;
  const void* res;                  // or null
  const void* w;
  void* total;                      // or null
  void* y;                          // or null
  int8_t* q;                        // 8-bit result with scale, or null
  float* scale;
  float* rstd;                      // or null
  int64_t ldx, ldres, ldtotal, ldy, ldq;
};
// dt: type of the result (total, y)
hipError_t launch_norm(int dt, const NormArgs& a, hipStream_t s);

struct NormGradArgs {
  int rows, hidden, w_dt;
  float w_add;
  const void* x;                    // what the forward call normalised
  const void* w;
  const float* rstd;
  const void* dy;
  const void* dtotal;               // or null
  void* dx;                         // or null
  void* dw;                         // or null, of w_dt
  float* part;                      // norm_grad_words(rows, hidden): the workgroups' sums of dw
  int64_t ldx, lddy, lddtotal, lddx;
};
int64_t norm_grad_words(int rows, int hidden);
hipError_t launch_norm_grad(int dt, const NormGradArgs& a, hipStream_t s);

// --------------------------------------------------------------- balance
struct BalanceArgs {
  int rows, experts, k;
  const void* logits;               // [rows, experts], row stride ld
  int64_t ld;
  const int32_t* ids;               // [rows, k]
  const uint8_t* mask;              // [rows] or null
  float* losses;                    // balance, z
  int32_t* counts;                  // [experts + 1], the last one the rows that count
  float* part;                      // balance_part_words(rows, experts) words
  // backward
  const float* dlosses;
  void* dlogits;                    // [rows, experts], row stride ldd
  int64_t ldd;
};
int64_t balance_part_words(int rows, int experts);
hipError_t launch_balance(int dt, const BalanceArgs& a, hipStream_t s);
hipError_t launch_balance_grad(int dt, const BalanceArgs& a, hipStream_t s);

// ------------------------------------------------- low-rank adapters (lora)
// The rows sorted by adapter (in their order inside one), those with none as
// adapter number `adapters`, cut into tiles of LORA_TILE rows of one adapter and,
// for the gradients, segments of seg_rows.
constexpr int LORA_TILE = 64;
constexpr int LORA_SORT = 8192;       // rows of a sorting workgroup
struct LoraSort {
  int rows, adapters;
  const int32_t* ids;
  int blocks;                         // sorting workgroups
  int* hist;                          // [blocks, adapters + 1], blocks > 1
  int4* tiles;                        // [max_tiles]: adapter (-1: none left), first place in the order, rows, number
  int max_tiles;
  int* tile_rows;                     // [max_tiles, LORA_TILE]: the rows of each (its last one again behind them)
  // gradients (seg_rows = 0: none): every adapter has a segment at least
  int seg_rows, max_segs;             // (a multiple of LORA_TILE)
  int4* segs;                         // [max_segs]: adapter (-1), first place, rows, first tile
  int* slot;                          // [max_segs]: where its partial sums go, -1: it is its adapter's only one
  int2* span;                         // [adapters]: first slot, segments (0: one)
};
hipError_t launch_lora_sort(const LoraSort& a, hipStream_t s);

// t[r] = w_i src[r] (k_major: w_i^T src[r]): rows of `rank` sums over k elements
struct LoraShrink {
  int k, rank, rp, adapters;          // rp: rank to a multiple of 32
  const void* src;
  const void* w;                      // [adapters, rank, k]; k-major [adapters, k, rank]
  int64_t ldsrc, ldw, stw;
  const float* scale;
  const int* rows;                    // LoraSort's tile_rows
  const int4* tiles;
  int max_tiles;
  int splits;                         // K ranges (lora_splits)
  float* part;                        // [splits, places, rank to a multiple of 4] sums
  int64_t places;                     // rows
  float* t;                           // fp32 [rows, rank]
  // by place in the order:
  uint16_t* hi;                       // [rows, rp] parts of t over a power of two a row (zero behind rank)
  uint16_t* lo;
  float* fac;                         // [rows] scale times that power
  // for the gradients in fp16: of each 16 rows of each tile the largest |t| (as bits,
  // finite ones only), and the same of t2
  uint32_t* top;                      // or null
  const float* t2;
  uint32_t* top2;
};
int lora_splits(int rows, int k, int rank);
hipError_t launch_lora_shrink(int dt, bool k_major, const LoraShrink& a, hipStream_t s);

// dst[r] = base[r] + fac[r] (w_i t[r]) (k_major: w_i^T t[r]), cols wide
struct LoraExpand {
  int cols, rank, rp, adapters;
  int chunk;                          // columns of a workgroup (lora_chunk)
  const void* w;                      // [adapters, cols, rank]; k-major [adapters, rank, cols]
  const void* base;                   // or null
  void* dst;
  int64_t ldw, stw, ldbase, lddst;
  const int* rows;
  const int4* tiles;
  int max_tiles;
  const uint16_t* hi;
  const uint16_t* lo;
  const float* fac;
};
int lora_chunk(int rows, int cols);
hipError_t launch_lora_expand(int dt, bool k_major, const LoraExpand& a, hipStream_t s);

// da_i = scale_i sum_r u[r] x[r]^T, db_i = scale_i sum_r dy[r] t[r]^T
struct LoraGrad {
  int rank, in, out, adapters;
  const float* u;                     // [rows, rank]
  const float* t;
  const void* x;
  const void* dy;
  int64_t ldx, lddy;
  const float* scale;
  const int* rows;                    // tile_rows
  const int4* segs;
  const int* slot;
  const int2* span;
  int max_segs;
  bool join;                          // an adapter may have several segments
  const uint32_t* top_u;              // fp16
  const uint32_t* top_t;
  void* da;                           // or null, both
  void* db;
  float* part;                        // [slots, rank (in + out)]
};
hipError_t launch_lora_grad(int dt, const LoraGrad& a, hipStream_t s);

// Few rows: everything of a row by one workgroup, in fp32 products
struct LoraRow {
  int rows, in, out, rank, adapters;
  const void* x;
  const void* a;
  const void* b;
  int64_t ldx, lda, sta, ldb, stb;
  const float* scale;
  const int32_t* ids;
  const void* base;                   // or null
  void* y;
  int64_t ldbase, ldy;
  float* t;                           // or null
};
bool lora_by_row(int rows, int in, int out, int rank);
hipError_t launch_lora_row(int dt, const LoraRow& a, hipStream_t s);

}  // namespace moe

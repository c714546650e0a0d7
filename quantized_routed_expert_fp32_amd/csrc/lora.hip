// Low-rank adapters of many requests beside a shared projection: row r has
// adapter i = ids[r], or none,
//   t_r = a_i x_r,  y_r = base_r + scale_i b_i t_r
// and the gradients
//   u_r = b_i^T dy_r,  dx_r = dx_base_r + scale_i a_i^T u_r,
//   da_i = scale_i sum_r u_r x_r^T,  db_i = scale_i sum_r dy_r t_r^T.
//
//  * k_lora_row: few rows, one launch, a workgroup a row.
//  * k_lora_sort: the rows by adapter, cut into tiles of one adapter each.
//  * k_lora_shrink: t or u, the long contraction: operands straight from memory into
//    matrix instructions, its K range over the waves of a workgroup.
//  * k_lora_expand: y or dx, the short contraction, one pass over base and result.
//  * k_lora_grad (k_lora_join): da and db, contractions over an adapter's rows.
// Ranks are small, so all of them are bound by the bytes of x, base, y and the
// gradients (rank 64: 64 flops a byte), and by launches where there are few rows.
// t and u are sums in fp32 and go into their products as a high and a low 16-bit part
// (one part would cost a bf16 result as much error again as its own rounding): the
// matrix units have the time. fp16 parts carry a power of two a row (k_lora_expand)
// or a segment (k_lora_grad), as fp16 has its 11 bits from 2^-14 on only. Sums have
// a fixed order.
#include "block_launch.h"
#include "dense_rows.h"

#include <algorithm>

namespace moe {

constexpr int SORT_WG = 512, SORT_WAVES = SORT_WG / 64, SORT_BINS = 1025;

// ------------------------------------------------------------------- sorting
__device__ __forceinline__ int bin_of(int id, int adapters) { return (uint32_t)id < (uint32_t)adapters ? id : adapters; }

__global__ __launch_bounds__(SORT_WG) void k_lora_hist(LoraSort a) {
  __shared__ int cnt[SORT_BINS];
  const int bins = a.adapters + 1;
  for (int b = threadIdx.x; b < bins; b += SORT_WG) cnt[b] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < LORA_SORT; i += SORT_WG) {
    const int r = blockIdx.x * LORA_SORT + i;
    if (r < a.rows) atomicAdd(&cnt[bin_of(a.ids[r], a.adapters)], 1);
  }
  __syncthreads();
  for (int b = threadIdx.x; b < bins; b += SORT_WG) a.hist[(int64_t)blockIdx.x * bins + b] = cnt[b];
}

struct Scan4 {
  int v[4];
};
// Exclusive prefix sums over the workgroup's threads.
__device__ __forceinline__ Scan4 scan(Scan4 x, Scan4* wave_sum) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  Scan4 s = x;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int o = __shfl_up(s.v[i], d);
      if (lane >= d) s.v[i] += o;
    }
  if (lane == 63) wave_sum[w] = s;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s.v[i] -= x.v[i];
    for (int k = 0; k < w; ++k) s.v[i] += wave_sum[k].v[i];
  }
  return s;
}

// A stable counting sort, 8192 rows a workgroup: counts a wave in LDS, their
// prefix sums, then each wave places its rows in order (a lane's place among the
// wave's lanes of the same adapter from ballots over the id's bits).
__global__ __launch_bounds__(SORT_WG) void k_lora_sort(LoraSort a) {
  constexpr int PER = LORA_SORT / SORT_WG;      // steps of a wave
  constexpr int BPT = (SORT_BINS + SORT_WG - 1) / SORT_WG;
  __shared__ int cnt[SORT_WAVES][SORT_BINS];
  __shared__ int off[SORT_BINS + 1], tile[SORT_BINS + 1], seg[SORT_BINS + 1], slot[SORT_BINS + 1];
  __shared__ Scan4 wave_sum[SORT_WAVES];
  const int bins = a.adapters + 1, lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  for (int i = threadIdx.x; i < SORT_WAVES * SORT_BINS; i += SORT_WG) (&cnt[0][0])[i] = 0;
  __syncthreads();
  const int64_t r0 = (int64_t)blockIdx.x * LORA_SORT + w * (PER * 64) + lane;
  int id[PER];
#pragma unroll
  for (int s = 0; s < PER; ++s) id[s] = r0 + s * 64 < a.rows ? bin_of(a.ids[r0 + s * 64], a.adapters) : -1;
#pragma unroll
  for (int s = 0; s < PER; ++s)
    if (id[s] >= 0) atomicAdd(&cnt[w][id[s]], 1);
  __syncthreads();
  // the bins' rows in the workgroups before this one and in all
  int all[BPT], before[BPT];
  Scan4 sum = {};
  const int b0 = threadIdx.x * BPT;
#pragma unroll
  for (int i = 0; i < BPT; ++i) {
    const int b = b0 + i;
    all[i] = before[i] = 0;
    if (b >= bins) continue;
    if (a.blocks > 1) {
      for (int k = 0; k < a.blocks; ++k) {
        if (k == (int)blockIdx.x) before[i] = all[i];
        all[i] += a.hist[(int64_t)k * bins + b];
      }
    } else {
      for (int k = 0; k < SORT_WAVES; ++k) all[i] += cnt[k][b];
    }
    sum.v[0] += all[i];
    sum.v[1] += (all[i] + LORA_TILE - 1) / LORA_TILE;
    if (a.seg_rows && b < a.adapters) {
      const int segs = max((all[i] + a.seg_rows - 1) / a.seg_rows, 1);
      sum.v[2] += segs;
      sum.v[3] += segs > 1 ? segs : 0;
    }
  }
  Scan4 at = scan(sum, wave_sum);
#pragma unroll
  for (int i = 0; i < BPT; ++i) {
    const int b = b0 + i;
    if (b >= bins) continue;
    off[b] = at.v[0];
    tile[b] = at.v[1];
    seg[b] = at.v[2];
    slot[b] = at.v[3];
    int to = at.v[0] + before[i];
    for (int k = 0; k < SORT_WAVES; ++k) {
      const int n = cnt[k][b];
      cnt[k][b] = to;
      to += n;
    }
    at.v[0] += all[i];
    at.v[1] += (all[i] + LORA_TILE - 1) / LORA_TILE;
    if (a.seg_rows && b < a.adapters) {
      const int segs = max((all[i] + a.seg_rows - 1) / a.seg_rows, 1);
      if (blockIdx.x == 0) a.span[b] = make_int2(at.v[3], segs > 1 ? segs : 0);
      at.v[2] += segs;
      at.v[3] += segs > 1 ? segs : 0;
    }
    if (b == bins - 1) {
      off[bins] = at.v[0];
      tile[bins] = at.v[1];
      seg[bins] = at.v[2];
      slot[bins] = at.v[3];
    }
  }
  __syncthreads();
  const int bits = 32 - __builtin_clz(a.adapters);
#pragma unroll
  for (int s = 0; s < PER; ++s) {
    const bool in = id[s] >= 0;
    uint64_t same = __ballot(in);
    for (int i = 0; i < bits; ++i) {
      const uint64_t set = __ballot(in && (id[s] >> i & 1));
      same &= id[s] >> i & 1 ? set : ~set;
    }
    if (in) {
      const int rank = __popcll(same & ((1ull << lane) - 1));
      const int base = cnt[w][id[s]];
      a.perm[base + rank] = (int)(r0 + s * 64);
      asm volatile("" ::: "memory");             // every lane has read: LDS runs in order
      if (rank == 0) cnt[w][id[s]] = base + __popcll(same);
    }
    asm volatile("" ::: "memory");
  }
  // the tables, shared among the workgroups: the bin of entry e is the last one that starts at or before it
  auto find = [&](const int* starts, int e) {
    int lo = 0, hi = bins;                        // starts[lo] <= e < starts[hi]
    while (hi - lo > 1) {
      const int m = (lo + hi) / 2;
      if (starts[m] <= e) lo = m;
      else hi = m;
    }
    return lo;
  };
  for (int e = blockIdx.x * SORT_WG + threadIdx.x; e < a.max_tiles; e += gridDim.x * SORT_WG) {
    int4 v = make_int4(-1, 0, 0, 0);
    if (e < tile[bins]) {
      const int b = find(tile, e), i = (e - tile[b]) * LORA_TILE;
      v = make_int4(b, off[b] + i, min(LORA_TILE, off[b + 1] - off[b] - i), 0);
    }
    a.tiles[e] = v;
  }
  if (a.seg_rows)
    for (int e = blockIdx.x * SORT_WG + threadIdx.x; e < a.max_segs; e += gridDim.x * SORT_WG) {
      int4 v = make_int4(-1, 0, 0, 0);
      int sl = -1;
      if (e < seg[bins]) {
        const int b = find(seg, e), i = e - seg[b], n = off[b + 1] - off[b];
        v = make_int4(b, off[b] + i * a.seg_rows, min(a.seg_rows, n - i * a.seg_rows),
                      tile[b] + i * (a.seg_rows / LORA_TILE));
        if (seg[b + 1] - seg[b] > 1) sl = slot[b] + i;
      }
      a.segs[e] = v;
      a.slot[e] = sl;
    }
}

// ------------------------------------------------------- operand fragments
// 4 rows of 16 columns a 16-lane group, as a transposed read gives them: lane i
// supplies row i / 4, columns 4 (i % 4).. and gets column i's 4 rows. Two reads make
// a lane's 8 k; `hi` is 4 rows on.
__device__ __forceinline__ u32x4 read_tr(const uint8_t* at, int hi) {
  typedef __attribute__((address_space(3))) i16x4* lp;
  const i16x4 l = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(at));
  const i16x4 h = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(at + hi));
  const uint2 x = __builtin_bit_cast(uint2, l), y = __builtin_bit_cast(uint2, h);
  return u32x4{x.x, x.y, y.x, y.y};
}
// the exponent e of a positive finite v as 2^(e - 1) <= v < 2^e, 0 for 0
__device__ __forceinline__ int exponent(uint32_t bits) { return bits ? __builtin_amdgcn_frexp_expf(__uint_as_float(bits)) : 0; }
// |v| as bits where it is finite
__device__ __forceinline__ uint32_t finite_bits(float v) {
  const uint32_t b = __float_as_uint(v) & 0x7FFFFFFFu;
  return b < 0x7F800000u ? b : 0;
}

// ------------------------------------------------------------------- shrink
// A workgroup: 16 MF rows of one tile, all of the rank in blocks of 16 NF. Its
// W waves take chunks of 64 k in turn, each with all the rows and columns, so no
// operand is loaded twice and nothing waits for another wave; their sums join
// through LDS, half of the waves at a time. In a chunk lane quad c holds k = 32 u +
// 8 c.. of row lane % 16: loads of 16 bytes at any alignment, the next chunk's in
// flight. k-major weights go through a wave's own piece of LDS for the transposed read.
template <int DT, bool KM, int MF, int NF, int W, bool BIG>
__global__ __launch_bounds__(W * 64) void k_lora_shrink(LoraShrink a) {
  constexpr int ROWS = MF * 16, COLS = NF * 16, WG = W * 64;
  constexpr int JOIN = W / 2 * ROWS * COLS * 4;                   // half of the waves' sums
  constexpr int SROW = COLS * 2 + 16, STAGE = KM ? W * 32 * SROW : 0;
  constexpr int FCOLS = BIG ? 256 : COLS;
  constexpr int AREA = JOIN > STAGE ? JOIN : STAGE;
  __shared__ __align__(16) uint8_t area[AREA];
  __shared__ __align__(16) float full[ROWS][FCOLS + 4];
  __shared__ int s_row[ROWS];
  __shared__ uint32_t s_top[2];
  const int4 tile = a.tiles[blockIdx.x];
  const int first = tile.y + blockIdx.y * ROWS, n = min(tile.z - (int)blockIdx.y * ROWS, ROWS);
  if (tile.x < 0 || n <= 0) return;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, quad = lane >> 4;
  const bool none = tile.x == a.adapters;
  if (threadIdx.x < ROWS) s_row[threadIdx.x] = a.perm[first + min((int)threadIdx.x, n - 1)];
  if (threadIdx.x < 2) s_top[threadIdx.x] = 0;
  __syncthreads();
  if (!none) {
    const uint16_t* wi = static_cast<const uint16_t*>(a.w) + tile.x * a.stw;
    const uint16_t* src[MF];
#pragma unroll
    for (int m = 0; m < MF; ++m) src[m] = static_cast<const uint16_t*>(a.src) + s_row[m * 16 + col] * a.ldsrc;
    const int chunks = (a.k + 63) / 64;
    const int64_t end = (int64_t)a.k * 2;
    uint8_t* const stage = area + (KM ? w * 32 * SROW : 0);
#pragma unroll 1
    for (int j0 = 0; j0 < a.rank; j0 += COLS) {
      f32x4 acc[NF][MF];
#pragma unroll
      for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int m = 0; m < MF; ++m) acc[f][m] = f32x4{0.f, 0.f, 0.f, 0.f};
      const uint16_t* wr[NF];
      if constexpr (!KM)
#pragma unroll
        for (int f = 0; f < NF; ++f) wr[f] = wi + min(j0 + f * 16 + col, a.rank - 1) * a.ldw;
      // u: which half of the chunk; k-major: 32 k rows of 2 NF chunks of 16 bytes
      u32x4 xv[2][MF], wv[2][NF];
      auto load = [&](int ch) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int64_t at = (int64_t)ch * 128 + u * 64 + quad * 16;
#pragma unroll
          for (int m = 0; m < MF; ++m) xv[u][m] = load_chunk<2>(src[m], at, end);
#pragma unroll
          for (int f = 0; f < NF; ++f) {
            if constexpr (!KM) {
              wv[u][f] = load_chunk<2>(wr[f], at, end);
            } else {
              const int q = f * 64 + lane, k = ch * 64 + u * 32 + q / (2 * NF), c = q % (2 * NF);
              wv[u][f] = u32x4{0, 0, 0, 0};
              if (k < a.k && j0 + c * 8 < a.rank)
                wv[u][f] = load_chunk<2>(wi + k * a.ldw, (int64_t)(j0 + c * 8) * 2, (int64_t)a.rank * 2);
            }
          }
        }
      };
      if (w < chunks) load(w);
      for (int ch = w; ch < chunks; ch += W) {
        u32x4 x0[2][MF], w0[2][NF];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
          for (int m = 0; m < MF; ++m) x0[u][m] = xv[u][m];
#pragma unroll
          for (int f = 0; f < NF; ++f) w0[u][f] = wv[u][f];
        }
        if (ch + W < chunks) load(ch + W);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if constexpr (KM) {
            asm volatile("" ::: "memory");
#pragma unroll
            for (int f = 0; f < NF; ++f) {
              const int q = f * 64 + lane;
              *reinterpret_cast<u32x4*>(stage + q / (2 * NF) * SROW + q % (2 * NF) * 16) = w0[u][f];
            }
            asm volatile("" ::: "memory");         // the wave's own LDS runs in order
#pragma unroll
            for (int f = 0; f < NF; ++f)
              w0[u][f] = read_tr(stage + (quad * 8 + (col >> 2)) * SROW + f * 32 + (col & 3) * 8, 4 * SROW);
          }
#pragma unroll
          for (int f = 0; f < NF; ++f)
#pragma unroll
            for (int m = 0; m < MF; ++m) acc[f][m] = Elem<DT>::mma16(w0[u][f], x0[u][m], acc[f][m]);
        }
      }
      // lane: row m 16 + col, columns f 16 + quad 4..
#pragma unroll
      for (int half = W / 2; half; half /= 2) {
        __syncthreads();                           // the area is free
        f32x4* buf = reinterpret_cast<f32x4*>(area) + (w % half) * (NF * MF * 64) + lane;
        if (w >= half && w < 2 * half)
#pragma unroll
          for (int f = 0; f < NF; ++f)
#pragma unroll
            for (int m = 0; m < MF; ++m) buf[(f * MF + m) * 64] = acc[f][m];
        __syncthreads();
        if (w < half)
#pragma unroll
          for (int f = 0; f < NF; ++f)
#pragma unroll
            for (int m = 0; m < MF; ++m) acc[f][m] += buf[(f * MF + m) * 64];
      }
      if (w == 0)
#pragma unroll
        for (int f = 0; f < NF; ++f)
#pragma unroll
          for (int m = 0; m < MF; ++m)
            *reinterpret_cast<f32x4*>(&full[m * 16 + col][(BIG ? j0 : 0) + f * 16 + quad * 4]) = acc[f][m];
      __syncthreads();                             // the next block's pieces lie where wave 0 has read
    }
  }
  // a row's sums to memory: WG / ROWS threads a row
  constexpr int TPR = WG / ROWS;
  const int i = threadIdx.x / TPR, g = threadIdx.x % TPR;
  const bool in = i < n;
  const int64_t r = s_row[i];
  uint32_t m = 0, m2 = 0;
  if (!none)
    for (int j = g; j < a.rank; j += TPR) m = max(m, finite_bits(full[i][j]));
  if (a.t2)
    for (int j = g; j < a.rank; j += TPR) m2 = max(m2, finite_bits(a.t2[r * a.rank + j]));
#pragma unroll
  for (int d = TPR / 2; d; d >>= 1) {
    m = max(m, (uint32_t)__shfl_xor((int)m, d));
    m2 = max(m2, (uint32_t)__shfl_xor((int)m2, d));
  }
  if (a.top) {
    if (in && g == 0) {
      atomicMax(&s_top[0], m);                     // a maximum: any order
      atomicMax(&s_top[1], m2);
    }
    __syncthreads();
    if (threadIdx.x < MF) {
      const int at = blockIdx.x * (LORA_TILE / 16) + blockIdx.y * MF + threadIdx.x;
      a.top[at] = s_top[0];
      a.top2[at] = s_top[1];
    }
  }
  if (!in) return;
  // fp16: |t| below 2^14, in one row's own power of two
  const int e = DT == DT_F16 ? exponent(m) - 14 : 0;
  if (g == 0) a.fac[r] = none ? 0.f : __builtin_ldexpf(a.scale[tile.x], e);
  for (int j = g; j < a.rp; j += TPR) {
    const float v = none || j >= a.rank ? 0.f : full[i][j];
    if (a.t && j < a.rank) a.t[r * a.rank + j] = v;
    if (none) continue;
    const float s = DT == DT_F16 ? __builtin_ldexpf(v, -e) : v;
    a.hi[r * a.rp + j] = to16<DT>(s);
    a.lo[r * a.rp + j] = to16<DT>(low_part<DT>(s));
  }
}

// ------------------------------------------------------------------- expand
// A workgroup of four waves: a tile's rows, EXP_COLS columns of the result, a wave
// 64 rows x 32 columns at a time. The weights' rows are dealt to the fragments so
// that a lane ends with 8 consecutive columns of a row (fragment f, place m: column
// 8 (m / 4) + 4 f + m % 4): base and result move 16 bytes a lane, 64 a row. The
// parts' products have sums of their own, joined where the high one is finite: an
// infinite weight times a low part of zero would make a NaN of it. KB: blocks of 32
// of the rank whose parts stay in registers (0: any rank, read each time).
constexpr int EXP_COLS = 512;
template <int DT, bool KM, int KB>
__global__ __launch_bounds__(256) void k_lora_expand(LoraExpand a) {
  constexpr int MF = 4, F = 2, SROW = 80;
  __shared__ __align__(16) uint8_t area[KM ? 4 * 32 * SROW : 16];
  const int4 tile = a.tiles[blockIdx.x];
  if (tile.x < 0) return;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, quad = lane >> 4;
  const bool none = tile.x == a.adapters;
  const int kb = KB ? KB : a.rp / 32;
  int64_t row[MF];
  float fac[MF];
  u32x4 th[KB ? KB : 1][MF], tl[KB ? KB : 1][MF];
#pragma unroll
  for (int m = 0; m < MF; ++m) {
    row[m] = a.perm[tile.y + min(m * 16 + col, tile.z - 1)];
    fac[m] = none ? 0.f : a.fac[row[m]];
  }
  auto parts = [&](int k, u32x4* h, u32x4* l) {
#pragma unroll
    for (int m = 0; m < MF; ++m) {
      h[m] = *reinterpret_cast<const u32x4*>(a.hi + row[m] * a.rp + k * 32 + quad * 8);
      l[m] = *reinterpret_cast<const u32x4*>(a.lo + row[m] * a.rp + k * 32 + quad * 8);
    }
  };
  if constexpr (KB > 0)
    if (!none)
#pragma unroll
      for (int k = 0; k < KB; ++k) parts(k, th[k], tl[k]);
  const uint16_t* wi = static_cast<const uint16_t*>(a.w) + (none ? 0 : tile.x * a.stw);
  uint8_t* const stage = area + (KM ? w * 32 * SROW : 0);
  const int c_end = min(a.cols, (int)(blockIdx.y + 1) * EXP_COLS);
#pragma unroll 1
  for (int c0 = blockIdx.y * EXP_COLS + w * 32; c0 < c_end; c0 += 128) {
    const int c = c0 + quad * 8;                   // the lane's 8 columns
    u32x4 bv[MF];
#pragma unroll
    for (int m = 0; m < MF; ++m) {
      bv[m] = u32x4{0, 0, 0, 0};
      if (a.base && c < a.cols)
        bv[m] = load_chunk<2, true>(static_cast<const uint16_t*>(a.base) + row[m] * a.ldbase, (int64_t)c * 2, (int64_t)a.cols * 2);
    }
    f32x4 hi[F][MF], lo[F][MF];
#pragma unroll
    for (int f = 0; f < F; ++f)
#pragma unroll
      for (int m = 0; m < MF; ++m) hi[f][m] = lo[f][m] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (!none) {
#pragma unroll
      for (int k = 0; k < (KB ? KB : 8); ++k) {
        if (!KB && k >= kb) break;
        u32x4 p[F];
        if constexpr (!KM) {
#pragma unroll
          for (int f = 0; f < F; ++f) {
            const int at = c0 + (col >> 2) * 8 + f * 4 + (col & 3);
            p[f] = load_chunk<2>(wi + min(at, a.cols - 1) * a.ldw, (int64_t)(k * 32 + quad * 8) * 2, (int64_t)a.rank * 2);
          }
        } else {
          // 32 k rows of 4 chunks of 16 bytes
          u32x4 v[2];
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int kr = k * 32 + (q * 64 + lane) / 4, cc = c0 + lane % 4 * 8;
            v[q] = u32x4{0, 0, 0, 0};
            if (kr < a.rank && cc < a.cols) v[q] = load_chunk<2, true>(wi + kr * a.ldw, (int64_t)cc * 2, (int64_t)a.cols * 2);
          }
          asm volatile("" ::: "memory");
#pragma unroll
          for (int q = 0; q < 2; ++q)
            *reinterpret_cast<u32x4*>(stage + (q * 64 + lane) / 4 * SROW + lane % 4 * 16) = v[q];
          asm volatile("" ::: "memory");           // the wave's own LDS runs in order
#pragma unroll
          for (int f = 0; f < F; ++f)
            p[f] = read_tr(stage + (quad * 8 + (col >> 2)) * SROW + (col & 3) * 16 + f * 8, 4 * SROW);
        }
        if constexpr (KB == 0) parts(k, th[0], tl[0]);
#pragma unroll
        for (int f = 0; f < F; ++f)
#pragma unroll
          for (int m = 0; m < MF; ++m) {
            hi[f][m] = Elem<DT>::mma16(p[f], th[KB ? k : 0][m], hi[f][m]);
            lo[f][m] = Elem<DT>::mma16(p[f], tl[KB ? k : 0][m], lo[f][m]);
          }
      }
    }
    if (c >= a.cols) continue;
#pragma unroll
    for (int m = 0; m < MF; ++m) {
      if (m * 16 + col >= tile.z) continue;
      float v[8];
      unpack16<DT>(bv[m], v);
      if (!none)
#pragma unroll
        for (int f = 0; f < F; ++f)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float h = hi[f][m][e];
            v[f * 4 + e] += fac[m] * (__builtin_fabsf(h) < __builtin_inff() ? h + lo[f][m][e] : h);
          }
      const u32x4 o = pack16<DT>(v);
      uint16_t* at = static_cast<uint16_t*>(a.dst) + row[m] * a.lddst + c;
      if (c + 8 <= a.cols) __builtin_memcpy(at, &o, 16);      // at any alignment
      else
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (c + e < a.cols) at[e] = (uint16_t)(o[e / 2] >> (16 * (e & 1)));
    }
  }
}

// ---------------------------------------------------------------- gradients
// A workgroup of four waves: 64 of the rank x 128 columns of one segment's sums over
// its rows, 64 rows a step: the 16-bit rows and the parts of the fp32 ones go through
// LDS (the next step's on their way in registers), both read transposed. da's lanes
// end with 8 consecutive columns of a rank row, db's with 16 consecutive ranks of a
// column's row: the operands change places.
constexpr int GRAD_COLS = 128, GRAD_ROWS = 64;
template <int DT, bool DB>
__device__ __forceinline__ void lora_grad(const LoraGrad& a, int4 seg, int slot, int j0, int c0, uint8_t* sx, uint8_t* st,
                                          uint32_t* s_top) {
  constexpr int XROW = GRAD_COLS * 2 + 16, TROW = 128 + 16;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, col = lane & 15, quad = lane >> 4;
  const int cols = DB ? a.out : a.in;
  const float* tp = DB ? a.t : a.u;
  const uint16_t* xp = static_cast<const uint16_t*>(DB ? a.dy : a.x);
  const int64_t ld = DB ? a.lddy : a.ldx;
  int e = 0;                                       // fp16: parts are |t| 2^-e, below 2^14
  if constexpr (DT == DT_F16) {
    const uint32_t* top = (DB ? a.top_t : a.top_u) + seg.w * (LORA_TILE / 16);
    uint32_t m = 0;
    for (int i = threadIdx.x; i < (seg.z + 15) / 16; i += 256) m = max(m, top[i]);
#pragma unroll
    for (int d = 32; d; d >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
    if (lane == 0) s_top[w] = m;
    __syncthreads();
    e = exponent(max(max(s_top[0], s_top[1]), max(s_top[2], s_top[3]))) - 14;
  }
  // x: 16 chunks a row, 16 rows at a time; t: 4 threads a row, 16 of the rank each
  const int xr = threadIdx.x >> 4, xc = threadIdx.x & 15, tr = threadIdx.x >> 2, tc = (threadIdx.x & 3) * 16;
  u32x4 xv[4];
  float tv[16];
  auto row_of = [&](int i) { return i < seg.z ? a.perm[seg.y + i] : -1; };
  auto load = [&](int i0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = row_of(i0 + xr + i * 16);
      xv[i] = u32x4{0, 0, 0, 0};
      if (r >= 0 && c0 + xc * 8 < cols)
        xv[i] = load_chunk<2, true>(xp + r * ld, (int64_t)(c0 + xc * 8) * 2, (int64_t)cols * 2);
    }
    const int r = row_of(i0 + tr);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u32x4 v = {0, 0, 0, 0};
      if (r >= 0 && j0 + tc + i * 4 < a.rank)
        v = load_chunk<4>(tp + (int64_t)r * a.rank, (int64_t)(j0 + tc + i * 4) * 4, (int64_t)a.rank * 4);
      unpack16<DT_F32>(v, tv + i * 4);
    }
  };
  f32x4 hi[2][4], lo[2][4];                        // [x fragment][t fragment]
#pragma unroll
  for (int f = 0; f < 2; ++f)
#pragma unroll
    for (int j = 0; j < 4; ++j) hi[f][j] = lo[f][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (seg.z > 0) load(0);
  for (int i0 = 0; i0 < seg.z; i0 += GRAD_ROWS) {
    __syncthreads();                               // the last step's readers are done
#pragma unroll
    for (int i = 0; i < 4; ++i) *reinterpret_cast<u32x4*>(sx + (xr + i * 16) * XROW + xc * 16) = xv[i];
    float low[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if constexpr (DT == DT_F16) tv[i] = __builtin_ldexpf(tv[i], -e);
      low[i] = low_part<DT>(tv[i]);
    }
    uint8_t* h = st + tr * TROW + tc * 2;
    uint8_t* l = h + GRAD_ROWS * TROW;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      *reinterpret_cast<u32x4*>(h + i * 16) = pack16<DT>(tv + i * 8);
      *reinterpret_cast<u32x4*>(l + i * 16) = pack16<DT>(low + i * 8);
    }
    __syncthreads();
    if (i0 + GRAD_ROWS < seg.z) load(i0 + GRAD_ROWS);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int kr = k * 32 + quad * 8 + (col >> 2);
      u32x4 x[2], th[4], tl[4];
#pragma unroll
      for (int f = 0; f < 2; ++f)
        x[f] = read_tr(sx + kr * XROW + w * 64 + (DB ? f * 32 + (col & 3) * 8 : (col & 3) * 16 + f * 8), 4 * XROW);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint8_t* at = st + kr * TROW + (DB ? (col & 3) * 32 + j * 8 : j * 32 + (col & 3) * 8);
        th[j] = read_tr(at, 4 * TROW);
        tl[j] = read_tr(at + GRAD_ROWS * TROW, 4 * TROW);
      }
#pragma unroll
      for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          hi[f][j] = DB ? Elem<DT>::mma16(th[j], x[f], hi[f][j]) : Elem<DT>::mma16(x[f], th[j], hi[f][j]);
          lo[f][j] = DB ? Elem<DT>::mma16(tl[j], x[f], lo[f][j]) : Elem<DT>::mma16(x[f], tl[j], lo[f][j]);
        }
    }
  }
  const float scale = a.scale[seg.x];
  auto value = [&](int f, int j, int q) {
    const float h = hi[f][j][q], v = __builtin_fabsf(h) < __builtin_inff() ? h + lo[f][j][q] : h;
    return DT == DT_F16 ? __builtin_ldexpf(v, e) : v;
  };
  // N consecutive values of a row of the result, from column c on of n: rounded, or
  // (one of several segments) as they are
  const int64_t size = (int64_t)a.rank * cols;
  float* part = slot < 0 ? nullptr : a.part + (int64_t)slot * a.rank * (a.in + a.out) + (DB ? (int64_t)a.rank * a.in : 0);
  uint16_t* out = static_cast<uint16_t*>(DB ? a.db : a.da) + seg.x * size;
  auto put8 = [&](int64_t row, int c, int n, const float* v) {
    const int64_t at = row * n + c;
    if (part) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < n) part[at + i] = v[i];
      return;
    }
    float s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = scale * v[i];
    const u32x4 o = pack16<DT>(s);
    if (c + 8 <= n) __builtin_memcpy(out + at, &o, 16);
    else
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < n) out[at + i] = (uint16_t)(o[i / 2] >> (16 * (i & 1)));
  };
  if constexpr (!DB) {
    const int c = c0 + w * 32 + quad * 8;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int rk = j0 + j * 16 + col;
      if (rk >= a.rank || c >= cols) continue;
      float v[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = value(q / 4, j, q % 4);
      put8(rk, c, cols, v);
    }
  } else {
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      const int c = c0 + w * 32 + f * 16 + col;
      if (c >= cols) continue;
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int rk = j0 + quad * 16 + p * 8;
        if (rk >= a.rank) continue;
        float v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = value(f, p * 2 + q / 4, q % 4);
        put8(c, rk, a.rank, v);
      }
    }
  }
}
template <int DT> __global__ __launch_bounds__(256) void k_lora_grad(LoraGrad a, int in_tiles) {
  __shared__ __align__(16) uint8_t sx[GRAD_ROWS * (GRAD_COLS * 2 + 16)], st[2 * GRAD_ROWS * 144];
  __shared__ uint32_t s_top[4];
  const int4 seg = a.segs[blockIdx.x];
  if (seg.x < 0) return;
  const int slot = a.slot[blockIdx.x], j0 = blockIdx.z * 64;
  if ((int)blockIdx.y < in_tiles) lora_grad<DT, false>(a, seg, slot, j0, blockIdx.y * GRAD_COLS, sx, st, s_top);
  else lora_grad<DT, true>(a, seg, slot, j0, (blockIdx.y - in_tiles) * GRAD_COLS, sx, st, s_top);
}
// the sums of adapters of several segments, in order
template <int DT> __global__ __launch_bounds__(256) void k_lora_join(LoraGrad a) {
  const int2 span = a.span[blockIdx.y];
  if (!span.y) return;
  const int64_t na = (int64_t)a.rank * a.in, nb = (int64_t)a.rank * a.out, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= na + nb) return;
  const float* p = a.part + span.x * (na + nb) + i;
  float v = p[0];
  for (int s = 1; s < span.y; ++s) v += p[s * (na + nb)];
  const uint16_t o = to16<DT>(a.scale[blockIdx.y] * v);
  if (i < na) static_cast<uint16_t*>(a.da)[blockIdx.y * na + i] = o;
  else static_cast<uint16_t*>(a.db)[blockIdx.y * nb + i - na] = o;
}

// ------------------------------------------------------------------ few rows
// A workgroup of 16 waves a row. t: a wave a rank row (ranks below 16: several
// waves, a stretch of k each), 16 bytes a lane. y: LPC lanes a column, 8 of the
// rank each, so that the weights are read in one stretch.
template <int DT, int LPC> __global__ __launch_bounds__(1024) void k_lora_row(LoraRow a) {
  __shared__ float s_part[16], s_t[256];
  const int64_t r = blockIdx.x;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int id = a.ids[r];
  const bool none = (uint32_t)id >= (uint32_t)a.adapters;
  if (!none) {
    const uint16_t* x = static_cast<const uint16_t*>(a.x) + r * a.ldx;
    const uint16_t* wa = static_cast<const uint16_t*>(a.a) + id * a.sta;
    const int split = a.rank <= 1 ? 16 : a.rank <= 2 ? 8 : a.rank <= 4 ? 4 : a.rank <= 8 ? 2 : 1;
    const int chunks = (a.in + 7) / 8;
    const int c0 = chunks * (w % split) / split, c1 = chunks * (w % split + 1) / split;
    for (int j = w / split; j < a.rank; j += 16 / split) {
      float v = 0.f;
#pragma unroll 4
      for (int c = c0 + lane; c < c1; c += 64) {
        float f[8], g[8];
        unpack16<DT>(load_chunk<2, true>(x, (int64_t)c * 16, (int64_t)a.in * 2), f);
        unpack16<DT>(load_chunk<2, true>(wa + j * a.lda, (int64_t)c * 16, (int64_t)a.in * 2), g);
#pragma unroll
        for (int i = 0; i < 8; ++i) v += f[i] * g[i];
      }
#pragma unroll
      for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
      if (lane == 0) {
        if (split == 1) s_t[j] = v;
        else s_part[w] = v;
      }
    }
    __syncthreads();
    if (split > 1) {
      if ((int)threadIdx.x < a.rank) {
        float v = s_part[threadIdx.x * split];
        for (int i = 1; i < split; ++i) v += s_part[threadIdx.x * split + i];
        s_t[threadIdx.x] = v;
      }
      __syncthreads();
    }
  }
  if (a.t)
    for (int j = threadIdx.x; j < a.rank; j += 1024) a.t[r * a.rank + j] = none ? 0.f : s_t[j];
  const uint16_t* wb = static_cast<const uint16_t*>(a.b) + (none ? 0 : id * a.stb);
  const float scale = none ? 0.f : a.scale[id];
  const uint16_t* base = a.base ? static_cast<const uint16_t*>(a.base) + r * a.ldbase : nullptr;
  uint16_t* y = static_cast<uint16_t*>(a.y) + r * a.ldy;
  const int g = threadIdx.x % LPC;
  for (int c = threadIdx.x / LPC; c < a.out; c += 1024 / LPC) {
    const float b = base ? Row<DT>::f(base[c]) : 0.f;
    float v = 0.f;
    if (!none) {
      for (int j = g * 8; j < a.rank; j += LPC * 8) {
        float f[8];
        unpack16<DT>(load_chunk<2, true>(wb + c * a.ldb, (int64_t)j * 2, (int64_t)a.rank * 2), f);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (j + i < a.rank) v += f[i] * s_t[j + i];
      }
#pragma unroll
      for (int d = 1; d < LPC; d <<= 1) v += __shfl_xor(v, d);
      v = b + scale * v;
    } else {
      v = b;
    }
    if (g == 0) y[c] = to16<DT>(v);
  }
}

// --------------------------------------------------------------- launchers
hipError_t launch_lora_sort(const LoraSort& a, hipStream_t s) {
  if (a.blocks > 1) {
    hipLaunchKernelGGL(k_lora_hist, dim3(a.blocks), dim3(SORT_WG), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(k_lora_sort, dim3(a.blocks), dim3(SORT_WG), 0, s, a);
  return hipGetLastError();
}

template <int DT, bool KM, int MF, int NF, int W, bool BIG> static hipError_t shrink(const LoraShrink& a, hipStream_t s) {
  hipLaunchKernelGGL((k_lora_shrink<DT, KM, MF, NF, W, BIG>), dim3(a.max_tiles, LORA_TILE / 16 / MF), dim3(W * 64), 0, s, a);
  return hipGetLastError();
}
template <int DT, bool KM, int MF, int W> static hipError_t shrink_rank(const LoraShrink& a, hipStream_t s) {
  if (a.rank <= 16) return shrink<DT, KM, MF, 1, W, false>(a, s);
  if (a.rank <= 32) return shrink<DT, KM, MF, 2, W, false>(a, s);
  if (a.rank <= 64) return shrink<DT, KM, MF, 4, W, false>(a, s);
  return shrink<DT, KM, 1, 4, W, true>(a, s);
}
template <int DT, bool KM> static hipError_t shrink_rows(int rows, const LoraShrink& a, hipStream_t s) {
  // more rows a workgroup read the weights less often, where enough workgroups are left
  if (rows <= 4096) return shrink_rank<DT, KM, 1, 8>(a, s);
  return shrink_rank<DT, KM, 2, 8>(a, s);
}
hipError_t launch_lora_shrink(int dt, bool k_major, int rows, const LoraShrink& a, hipStream_t s) {
  if (dt == DT_BF16) return k_major ? shrink_rows<DT_BF16, true>(rows, a, s) : shrink_rows<DT_BF16, false>(rows, a, s);
  if (dt == DT_F16) return k_major ? shrink_rows<DT_F16, true>(rows, a, s) : shrink_rows<DT_F16, false>(rows, a, s);
  return hipErrorInvalidValue;
}

template <int DT, bool KM> static hipError_t expand(const LoraExpand& a, hipStream_t s) {
  const dim3 grid(a.max_tiles, (a.cols + EXP_COLS - 1) / EXP_COLS);
  if (a.rp == 32) hipLaunchKernelGGL((k_lora_expand<DT, KM, 1>), grid, dim3(256), 0, s, a);
  else if (a.rp == 64) hipLaunchKernelGGL((k_lora_expand<DT, KM, 2>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_lora_expand<DT, KM, 0>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}
hipError_t launch_lora_expand(int dt, bool k_major, const LoraExpand& a, hipStream_t s) {
  if (dt == DT_BF16) return k_major ? expand<DT_BF16, true>(a, s) : expand<DT_BF16, false>(a, s);
  if (dt == DT_F16) return k_major ? expand<DT_F16, true>(a, s) : expand<DT_F16, false>(a, s);
  return hipErrorInvalidValue;
}

template <int DT> static hipError_t grad(const LoraGrad& a, hipStream_t s) {
  const int ti = (a.in + GRAD_COLS - 1) / GRAD_COLS, to = (a.out + GRAD_COLS - 1) / GRAD_COLS;
  hipLaunchKernelGGL((k_lora_grad<DT>), dim3(a.max_segs, ti + to, (a.rank + 63) / 64), dim3(256), 0, s, a, ti);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.join) return e;
  const int64_t n = (int64_t)a.rank * (a.in + (int64_t)a.out);
  hipLaunchKernelGGL((k_lora_join<DT>), dim3((uint32_t)((n + 255) / 256), a.adapters), dim3(256), 0, s, a);
  return hipGetLastError();
}
hipError_t launch_lora_grad(int dt, const LoraGrad& a, hipStream_t s) {
  if (dt == DT_BF16) return grad<DT_BF16>(a, s);
  if (dt == DT_F16) return grad<DT_F16>(a, s);
  return hipErrorInvalidValue;
}

// Where the rows' own reads of the weights (a row's a and b each) stay few
bool lora_by_row(int rows, int in, int out, int rank) { return rows <= 64 && (int64_t)rows * rank * (in + (int64_t)out) <= 8 << 20; }

template <int DT> static hipError_t by_row(const LoraRow& a, hipStream_t s) {
  const dim3 g(a.rows), b(1024);
  if (a.rank <= 8) hipLaunchKernelGGL((k_lora_row<DT, 1>), g, b, 0, s, a);
  else if (a.rank <= 16) hipLaunchKernelGGL((k_lora_row<DT, 2>), g, b, 0, s, a);
  else if (a.rank <= 32) hipLaunchKernelGGL((k_lora_row<DT, 4>), g, b, 0, s, a);
  else hipLaunchKernelGGL((k_lora_row<DT, 8>), g, b, 0, s, a);
  return hipGetLastError();
}
hipError_t launch_lora_row(int dt, const LoraRow& a, hipStream_t s) {
  if (dt == DT_BF16) return by_row<DT_BF16>(a, s);
  if (dt == DT_F16) return by_row<DT_F16>(a, s);
  return hipErrorInvalidValue;
}

}  // namespace moe

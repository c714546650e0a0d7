// Low-rank adapters of many requests beside a shared projection: row r has
// adapter i = ids[r], or none,
//   t_r = a_i x_r,  y_r = base_r + scale_i b_i t_r
// and the gradients
//   u_r = b_i^T dy_r,  dx_r = dx_base_r + scale_i a_i^T u_r,
//   da_i = scale_i sum_r u_r x_r^T,  db_i = scale_i sum_r dy_r t_r^T.
//
//  * k_lora_row: few rows, one launch, a workgroup a row.
//  * k_lora_sort: the rows by adapter, cut into tiles of one adapter each.
//  * k_lora_shrink, k_lora_parts: t or u, the long contraction, its K range over
//    several workgroups whose sums are joined in order.
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

constexpr int EXP_WGS = 1024;          // workgroups of k_lora_expand: four a CU
constexpr int SORT_WG = 1024, SORT_WAVES = SORT_WG / 64, SORT_BINS = 1025;

// ------------------------------------------------------------------- sorting
__device__ __forceinline__ int bin_of(int id, int adapters) { return (uint32_t)id < (uint32_t)adapters ? id : adapters; }

// the wave's lanes with the same id (of so many bits), none for a negative one
__device__ __forceinline__ uint64_t same(int id, int bits) {
  uint64_t m = __ballot(id >= 0);
  for (int i = 0; i < bits; ++i) {
    const uint64_t set = __ballot(id >> i & 1);
    m &= id >> i & 1 ? set : ~set;
  }
  return m;
}

__global__ __launch_bounds__(SORT_WG) void k_lora_hist(LoraSort a) {
  __shared__ int cnt[SORT_BINS];
  const int bins = a.adapters + 1;
  for (int b = threadIdx.x; b < bins; b += SORT_WG) cnt[b] = 0;
  __syncthreads();
  const int bits = 32 - __builtin_clz(a.adapters), lane = threadIdx.x & 63;
  for (int i = threadIdx.x; i < LORA_SORT; i += SORT_WG) {
    const int r = blockIdx.x * LORA_SORT + i;
    const int id = r < a.rows ? bin_of(a.ids[r], a.adapters) : -1;
    const uint64_t m = same(id, bits);
    if (id >= 0 && !(m & ((1ull << lane) - 1))) atomicAdd(&cnt[id], __popcll(m));     // whole numbers: any order
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
// prefix sums, then each wave places its rows. Lanes of the same adapter find each
// other by ballots over the id's bits: runs of one adapter would queue at an LDS
// atomic. One workgroup's latency: 10 us for 777 rows, 14 for
// 4096, 17 for 8192.
__global__ __launch_bounds__(SORT_WG) void k_lora_sort(LoraSort a) {
  constexpr int PER = LORA_SORT / SORT_WG;      // steps of a wave
  constexpr int BPT = (SORT_BINS + SORT_WG - 1) / SORT_WG;
  __shared__ uint16_t cnt[SORT_WAVES][SORT_BINS];   // a wave's counts, then its first places in the workgroup
  __shared__ int off[SORT_BINS + 1], tile[SORT_BINS + 1], seg[SORT_BINS + 1], slot[SORT_BINS + 1], first[SORT_BINS];
  __shared__ Scan4 wave_sum[SORT_WAVES];
  const int bins = a.adapters + 1, lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  for (int b = threadIdx.x; b < bins; b += SORT_WG)
#pragma unroll
    for (int k = 0; k < SORT_WAVES; ++k) cnt[k][b] = 0;
  __syncthreads();
  const int64_t r0 = (int64_t)blockIdx.x * LORA_SORT + w * (PER * 64) + lane;
  int id[PER];
#pragma unroll
  for (int s = 0; s < PER; ++s) id[s] = r0 + s * 64 < a.rows ? bin_of(a.ids[r0 + s * 64], a.adapters) : -1;
  // a row's place among the wave's rows of its adapter; the counts are the wave's own
  const int bits = 32 - __builtin_clz(a.adapters);
  int local[PER];
#pragma unroll
  for (int s = 0; s < PER; ++s) {
    const uint64_t m = same(id[s], bits);
    local[s] = __popcll(m & ((1ull << lane) - 1));
    if (id[s] >= 0) {
      const int n = cnt[w][id[s]];
      asm volatile("" ::: "memory");             // every lane has read: LDS runs in order
      if (local[s] == 0) cnt[w][id[s]] = (uint16_t)(n + __popcll(m));
      local[s] += n;
    }
    asm volatile("" ::: "memory");
  }
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
    first[b] = before[i];
    int to = 0;
    for (int k = 0; k < SORT_WAVES; ++k) {
      const int n = cnt[k][b];
      cnt[k][b] = (uint16_t)to;
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
#pragma unroll
  for (int s = 0; s < PER; ++s)
    if (id[s] >= 0) {
      // place in its adapter's tiles; an adapter's last row stands for the rows that its
      // last tile lacks
      const int b = id[s], q = first[b] + cnt[w][b] + local[s], r = (int)(r0 + s * 64);
      int* to = a.tile_rows + (int64_t)tile[b] * LORA_TILE + q;
      *to = r;
      if (q == off[b + 1] - off[b] - 1)
        for (int i = 1; (q + i) % LORA_TILE; ++i) to[i] = r;
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
      v = make_int4(b, off[b] + i, min(LORA_TILE, off[b + 1] - off[b] - i), e);
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

// 16-bit elements, zero in the place of infinities and NaN: what the low parts meet where
// a result is not finite. A low part of zero, or of the other sign than its high part,
// makes a NaN of the infinity that the high part's product says; so results that are
// not finite (a look at each) are computed again with these.
template <int DT> __device__ __forceinline__ u32x4 finite_or_zero(u32x4 v) {
  constexpr uint32_t EXP = DT == DT_BF16 ? 0x7F80 : 0x7C00;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if ((v[i] & EXP) == EXP) v[i] &= 0xFFFF0000u;
    if ((v[i] >> 16 & EXP) == EXP) v[i] &= 0xFFFFu;
  }
  return v;
}

// ------------------------------------------------------------------- shrink
// A workgroup of four waves: a tile's rows x 16 NF of the rank over one of several K
// ranges, 64 k a step: rows and weights go through LDS, a wave takes 16 rows. The
// loads of the next two steps are in flight in registers, 16 bytes a lane at any
// alignment, whole lines of a row. The K ranges' sums go through memory to
// k_lora_parts. 4096 x 4096 to rank 64: 13 us, and 5.7 for k_lora_parts (joined by
// the last workgroup of a tile instead, 96: every workgroup's fence writes an L2 back);
// 8192 rows 25 to 26 us, 2.6 TB/s of x.
constexpr int SHR_K = 64;
// a row of sums in memory
static __host__ __device__ int sum_ld(int rank) { return (rank + 3) & ~3; }
template <int DT, bool KM, int NF> __global__ __launch_bounds__(256) void k_lora_shrink(LoraShrink a) {
  constexpr int COLS = NF * 16, ROW = SHR_K * 2 + 16;
  constexpr int WROW = KM ? COLS * 2 + 16 : ROW, WBYTES = KM ? SHR_K * WROW : COLS * ROW;
  constexpr int STAGE = LORA_TILE * ROW + WBYTES;
  constexpr int WL = (COLS * SHR_K * 2 / 16 + 255) / 256;         // chunks of weights a thread loads in a step
  __shared__ __align__(16) uint8_t area[2 * STAGE];
  __shared__ int s_row[LORA_TILE];
  const int4 tile = a.tiles[blockIdx.x];
  if (tile.x < 0 || tile.x == a.adapters) return;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, quad = lane >> 4;
  if (threadIdx.x < LORA_TILE) s_row[threadIdx.x] = a.rows[blockIdx.x * LORA_TILE + threadIdx.x];
  __syncthreads();
  const int j0 = blockIdx.y * COLS, z = (int)((blockIdx.z + (uint32_t)tile.w) % gridDim.z);
  const int steps = (a.k + SHR_K - 1) / SHR_K;
  const int t0 = (int)((int64_t)steps * z / gridDim.z), t1 = (int)((int64_t)steps * (z + 1) / gridDim.z);
  const uint16_t* wi = static_cast<const uint16_t*>(a.w) + tile.x * a.stw;
  const int64_t end = (int64_t)a.k * 2;
  // rows: 8 chunks each, 32 rows at a time; rows past the tile's repeat its last one
  const int xr = threadIdx.x >> 3, xc = (threadIdx.x & 7) * 16;
  const uint16_t* src[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) src[i] = static_cast<const uint16_t*>(a.src) + s_row[xr + i * 32] * a.ldsrc;
  struct Step {
    u32x4 x[2], w[WL];
  };
  auto load = [&](Step& s, int t) {
    const int64_t at = (int64_t)t * (SHR_K * 2) + xc;
#pragma unroll
    for (int i = 0; i < 2; ++i) s.x[i] = load_chunk<2, true>(src[i], at, end);
#pragma unroll
    for (int i = 0; i < WL; ++i) {
      const int q = i * 256 + threadIdx.x;
      s.w[i] = u32x4{0, 0, 0, 0};
      if constexpr (!KM) {
        const int r = j0 + q / 8;                // (rank rows past the last: zero)
        if (q / 8 < COLS && r < a.rank) s.w[i] = load_chunk<2, true>(wi + r * a.ldw, at, end);
      } else {
        const int k = t * SHR_K + q / (COLS / 8), c = j0 + q % (COLS / 8) * 8;
        if (q / (COLS / 8) < SHR_K && k < a.k && c < a.rank)
          s.w[i] = load_chunk<2, true>(wi + k * a.ldw, (int64_t)c * 2, (int64_t)a.rank * 2);
      }
    }
  };
  f32x4 acc[NF];
#pragma unroll
  for (int f = 0; f < NF; ++f) acc[f] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto step = [&](const Step& s, int buf) {
    uint8_t* const sx = area + buf * STAGE;
    uint8_t* const sw = sx + LORA_TILE * ROW;
#pragma unroll
    for (int i = 0; i < 2; ++i) *reinterpret_cast<u32x4*>(sx + (xr + i * 32) * ROW + xc) = s.x[i];
#pragma unroll
    for (int i = 0; i < WL; ++i) {
      const int q = i * 256 + threadIdx.x;
      if constexpr (!KM) {
        if (q / 8 < COLS) *reinterpret_cast<u32x4*>(sw + q / 8 * WROW + q % 8 * 16) = s.w[i];
      } else {
        if (q / (COLS / 8) < SHR_K) *reinterpret_cast<u32x4*>(sw + q / (COLS / 8) * WROW + q % (COLS / 8) * 16) = s.w[i];
      }
    }
  };
  auto multiply = [&](int buf) {
    const uint8_t* const sx = area + buf * STAGE;
    const uint8_t* const sw = sx + LORA_TILE * ROW;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const u32x4 x = *reinterpret_cast<const u32x4*>(sx + (w * 16 + col) * ROW + u * 64 + quad * 16);
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        u32x4 p;
        if constexpr (!KM) p = *reinterpret_cast<const u32x4*>(sw + (f * 16 + col) * WROW + u * 64 + quad * 16);
        else p = read_tr(sw + (u * 32 + quad * 8 + (col >> 2)) * WROW + f * 32 + (col & 3) * 8, 4 * WROW);
        acc[f] = Elem<DT>::mma16(p, x, acc[f]);
      }
    }
  };
  // One barrier a step: a buffer is written again two steps on, when every wave
  // has passed the barrier behind its readers.
  Step s[2];
  if (t0 < t1) load(s[0], t0);
  if (t0 + 1 < t1) load(s[1], t0 + 1);
  for (int t = t0; t < t1; t += 2) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (t + i >= t1) break;
      step(s[i], i);
      if (t + i + 2 < t1) load(s[i], t + i + 2);
      __syncthreads();
      multiply(i);
    }
  }
  // lane: row w 16 + col, columns f 16 + quad 4..
  const int i = w * 16 + col;
  float* part = a.part + ((int64_t)z * a.places + tile.y + i) * sum_ld(a.rank);
  if (i < tile.z)
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      const int j = j0 + f * 16 + quad * 4;
      if (j < a.rank) *reinterpret_cast<f32x4*>(part + j) = acc[f];
    }
}

// 16 of a tile's rows, 16 threads each, four of the rank at a time: the K ranges' sums in
// order to t, its largest value, then its parts.
template <int DT> __global__ __launch_bounds__(256) void k_lora_parts(LoraShrink a) {
  __shared__ uint32_t s_top[4][2];
  const int4 tile = a.tiles[blockIdx.x];
  if (tile.x < 0 || (int)blockIdx.y * 16 >= tile.z) return;
  const bool none = tile.x == a.adapters;
  const int i = blockIdx.y * 16 + (threadIdx.x >> 4), g = (threadIdx.x & 15) * 4, ld = sum_ld(a.rank);
  const bool in = i < tile.z;
  const int64_t p = tile.y + min(i, tile.z - 1), r = a.rows[blockIdx.x * LORA_TILE + i];
  float* const tr = a.t + r * a.rank;
  uint32_t m = 0, m2 = 0;
  f32x4 v = {0.f, 0.f, 0.f, 0.f};                  // of the last four (up to rank 64 the only ones)
  if (in)
    for (int j = g; j < a.rank; j += 64) {
      v = f32x4{0.f, 0.f, 0.f, 0.f};
      if (!none) {
        const float* at = a.part + p * ld + j;
        v = *reinterpret_cast<const f32x4*>(at);
#pragma unroll 8
        for (int z = 1; z < a.splits; ++z) v += *reinterpret_cast<const f32x4*>(at + (int64_t)z * a.places * ld);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (j + e >= a.rank) continue;
        tr[j + e] = v[e];
        m = max(m, finite_bits(v[e]));
        if (a.t2) m2 = max(m2, finite_bits(a.t2[r * a.rank + j + e]));
      }
    }
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) {
    m = max(m, (uint32_t)__shfl_xor((int)m, d));
    m2 = max(m2, (uint32_t)__shfl_xor((int)m2, d));
  }
  if (a.top) {
    uint32_t w0 = m, w1 = m2;
#pragma unroll
    for (int d = 16; d < 64; d <<= 1) {
      w0 = max(w0, (uint32_t)__shfl_xor((int)w0, d));
      w1 = max(w1, (uint32_t)__shfl_xor((int)w1, d));
    }
    if ((threadIdx.x & 63) == 0) {
      s_top[threadIdx.x >> 6][0] = w0;
      s_top[threadIdx.x >> 6][1] = w1;
    }
    __syncthreads();
    if (threadIdx.x < 2)
      (threadIdx.x ? a.top2 : a.top)[tile.w * (LORA_TILE / 16) + blockIdx.y] =
          max(max(s_top[0][threadIdx.x], s_top[1][threadIdx.x]), max(s_top[2][threadIdx.x], s_top[3][threadIdx.x]));
  }
  if (!in || none) return;
  // fp16: |t| below 2^14, in one row's own power of two
  const int e = DT == DT_F16 ? exponent(m) - 14 : 0;
  if (g == 0) a.fac[p] = __builtin_ldexpf(a.scale[tile.x], e);
  for (int j = g; j < a.rp; j += 64) {
    float h[4], l[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      // (beyond rank 64: this thread's own stores)
      h[k] = j + k >= a.rank ? 0.f : a.rank <= 64 ? v[k] : tr[j + k];
      if constexpr (DT == DT_F16) h[k] = __builtin_ldexpf(h[k], -e);
      l[k] = low_part<DT>(h[k]);
    }
    *reinterpret_cast<uint2*>(a.hi + p * a.rp + j) = make_uint2(to16<DT>(h[0]) | (uint32_t)to16<DT>(h[1]) << 16,
                                                                to16<DT>(h[2]) | (uint32_t)to16<DT>(h[3]) << 16);
    *reinterpret_cast<uint2*>(a.lo + p * a.rp + j) = make_uint2(to16<DT>(l[0]) | (uint32_t)to16<DT>(l[1]) << 16,
                                                                to16<DT>(l[2]) | (uint32_t)to16<DT>(l[3]) << 16);
  }
}

// ------------------------------------------------------------------- expand
// A workgroup of four waves: a tile's rows (16 a wave), `chunk` columns of the result,
// 64 columns and 32 KB of the rank a step. The weights go through LDS, read from memory
// once for the four; the loads of the next two steps are in flight in registers. The
// weights' rows are dealt to the fragments so that a lane ends with 8 consecutive
// columns of a row, twice (fragment f, place m: column 32 (f / 2) + 8 (m / 4) + 4 (f % 2)
// + m % 4): base and result move 16 bytes a lane, 64 a row, whole lines in two. 8192 x
// rank 64 -> 4096: 45 to 46 us, 2.9 TB/s of base and result, where a copy in the same pattern
// with all loads at the start takes 30; with 2 waves a SIMD instead of 4 it took 55 for 48.
template <int DT, bool KM, int KB> __global__ __launch_bounds__(256, 4) void k_lora_expand(LoraExpand a) {
  constexpr int F = 4, WROW = KM ? 144 : KB * 64 + 16, STAGE = KM ? KB * 32 * WROW : 64 * WROW;
  constexpr int CPR = KM ? 8 : KB * 4, WL = KB;    // chunks of a staged row, loads of a thread
  __shared__ __align__(16) uint8_t area[2 * STAGE];
  const int4 tile = a.tiles[blockIdx.x];
  if (tile.x < 0) return;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, quad = lane >> 4;
  const bool none = tile.x == a.adapters;
  const int i = w * 16 + col;                      // the lane's row of the tile
  const bool in = i < tile.z;
  const int64_t r = a.rows[blockIdx.x * LORA_TILE + i], at = tile.y + min(i, tile.z - 1);
  const uint16_t* const bp = static_cast<const uint16_t*>(a.base) + r * a.ldbase + quad * 8;
  uint16_t* const dp = static_cast<uint16_t*>(a.dst) + r * a.lddst + quad * 8;
  const uint16_t* const wi = static_cast<const uint16_t*>(a.w) + (none ? 0 : tile.x * a.stw);
  const float fac = none ? 0.f : a.fac[at];
  const int nk = none ? 1 : (a.rp + KB * 32 - 1) / (KB * 32);
  u32x4 th[KB], tl[KB];
  auto parts = [&](int kk) {
#pragma unroll
    for (int k = 0; k < KB; ++k) {
      const int j = (kk * KB + k) * 32 + quad * 8;
      th[k] = tl[k] = u32x4{0, 0, 0, 0};
      if (j >= a.rp) continue;
      th[k] = *reinterpret_cast<const u32x4*>(a.hi + at * a.rp + j);
      tl[k] = *reinterpret_cast<const u32x4*>(a.lo + at * a.rp + j);
    }
  };
  if (!none) parts(0);
  // tiles start with different columns, so that neighbours read different weights
  const int y = (int)((blockIdx.y + (uint32_t)tile.w) % gridDim.y);
  const int cb = y * a.chunk, steps = (min(a.cols, cb + a.chunk) - cb + 63) / 64 * nk;
  struct Step {
    u32x4 w[WL], b[2];
  };
  auto load = [&](Step& s, int n) {
    const int c0 = cb + n / nk * 64, kk = n % nk;
    // whether nothing of what the workgroup loads lies behind its rows' ends
    const bool inside = c0 + 64 <= a.cols;
    if (!none) {
      const int q0 = threadIdx.x / CPR, qc = threadIdx.x % CPR * 8;
      constexpr int RPL = 256 / CPR;               // staged rows of a load
      if (inside && (kk + 1) * KB * 32 <= a.rank) {
        const uint16_t* p = KM ? wi + (int64_t)(kk * KB * 32 + q0) * a.ldw + c0 + qc
                               : wi + (int64_t)(c0 + q0) * a.ldw + kk * KB * 32 + qc;
#pragma unroll
        for (int l = 0; l < WL; ++l) __builtin_memcpy(&s.w[l], p + l * RPL * a.ldw, 16);
      } else {
#pragma unroll
        for (int l = 0; l < WL; ++l) {
          const int row = (KM ? kk * KB * 32 : c0) + q0 + l * RPL, e = (KM ? c0 : kk * KB * 32) + qc;
          s.w[l] = u32x4{0, 0, 0, 0};
          if (row < (KM ? a.rank : a.cols) && e < (KM ? a.cols : a.rank))
            s.w[l] = load_chunk<2, true>(wi + row * a.ldw, (int64_t)e * 2, (int64_t)(KM ? a.cols : a.rank) * 2);
        }
      }
    }
    if (kk) return;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      s.b[h] = u32x4{0, 0, 0, 0};
      if (!a.base) continue;
      const int c = c0 + h * 32;
      if (inside) __builtin_memcpy(&s.b[h], bp + c, 16);
      else if (c + quad * 8 < a.cols)
        s.b[h] = load_chunk<2, true>(bp - quad * 8, (int64_t)(c + quad * 8) * 2, (int64_t)a.cols * 2);
    }
  };
  f32x4 acc[F];
  // safe: low parts meet zeros where the weights are not finite
  auto multiply = [&](int buf, bool safe) {
    const uint8_t* const sw = area + buf * STAGE;
#pragma unroll
    for (int k = 0; k < KB; ++k)
#pragma unroll
      for (int f = 0; f < F; ++f) {
        u32x4 p;
        if constexpr (KM)
          p = read_tr(sw + (k * 32 + quad * 8 + (col >> 2)) * WROW + (f >> 1) * 64 + (col & 3) * 16 + (f & 1) * 8, 4 * WROW);
        else
          p = *reinterpret_cast<const u32x4*>(sw + ((f >> 1) * 32 + (col >> 2) * 8 + (f & 1) * 4 + (col & 3)) * WROW +
                                              k * 64 + quad * 16);
        acc[f] = Elem<DT>::mma16(p, th[k], acc[f]);
        if (safe) p = finite_or_zero<DT>(p);
        acc[f] = Elem<DT>::mma16(p, tl[k], acc[f]);
      }
  };
  auto clear = [&]() {
#pragma unroll
    for (int f = 0; f < F; ++f) acc[f] = f32x4{0.f, 0.f, 0.f, 0.f};
  };
  auto finite = [&]() {
    float far = 0.f;
#pragma unroll
    for (int f = 0; f < F; ++f)
#pragma unroll
      for (int e = 0; e < 4; ++e) far = __builtin_fmaf(0.f, acc[f][e], far);
    return far == 0.f;
  };
  auto stage = [&](const Step& s, int buf) {
    constexpr int RPL = 256 / CPR;
    uint8_t* const sw = area + buf * STAGE + threadIdx.x / CPR * WROW + threadIdx.x % CPR * 16;
#pragma unroll
    for (int l = 0; l < WL; ++l) *reinterpret_cast<u32x4*>(sw + l * RPL * WROW) = s.w[l];
  };
  // one value of the result: the row's parts from t0 on, column c of the weights
  auto one_sum = [&](int64_t t0, int c) {
    float v = 0.f;
#pragma unroll 1
    for (int j = 0; j < a.rank; ++j) {
      const float wv = Row<DT>::f(KM ? wi[j * a.ldw + c] : wi[c * a.ldw + j]);
      v += wv * Row<DT>::f(a.hi[t0 + j]);
      if (__builtin_fabsf(wv) < __builtin_inff()) v += wv * Row<DT>::f(a.lo[t0 + j]);
    }
    return v;
  };
  // One barrier a step: a buffer is written again two steps on, when every wave has
  // passed the barrier behind its readers.
  Step s[2];
  u32x4 base[2];
  if (steps > 0) load(s[0], 0);
  if (steps > 1) load(s[1], 1);
  for (int n = 0; n < steps; n += 2) {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      if (n + b >= steps) break;
      const int c0 = cb + (n + b) / nk * 64, kk = (n + b) % nk;
      if (!none) stage(s[b], b);
      if (kk == 0) {
        base[0] = s[b].b[0];
        base[1] = s[b].b[1];
        clear();
      }
      if (n + b + 2 < steps) load(s[b], n + b + 2);
      if (!none) {
        __syncthreads();
        if (nk > 1) parts(kk);
        multiply(b, false);
      }
      if (kk != nk - 1) continue;
      // not finite: again with zeros for the low parts. A rank of several steps: those values
      // alone, from memory, a wave by itself; the others keep the sums that they have.
      if (!none && __any(!finite())) {
        if (nk == 1) {
          clear();
          multiply(b, true);
        } else {
#pragma unroll
          for (int f = 0; f < F; ++f)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (__builtin_fabsf(acc[f][e]) < __builtin_inff()) continue;
              const int c = min(c0 + (f >> 1) * 32 + quad * 8 + (f & 1) * 4 + e, a.cols - 1);
              acc[f][e] = one_sum(at * a.rp, c);
            }
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = c0 + h * 32 + quad * 8;
        float v[8];
        unpack16<DT>(base[h], v);
        if (!none)
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = __builtin_fmaf(fac, acc[h * 2 + e / 4][e % 4], v[e]);
        const u32x4 o = pack16<DT>(v);
        if (!in) continue;
        if (c + 8 <= a.cols) __builtin_memcpy(dp + c0 + h * 32, &o, 16);      // at any alignment
        else
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (c + e < a.cols) dp[c0 + h * 32 + e] = (uint16_t)(o[e / 2] >> (16 * (e & 1)));
      }
    }
  }
}

// ---------------------------------------------------------------- gradients
// A workgroup of four waves: 64 of the rank x 256 columns of one segment's sums over
// its rows (a wave 64 x 64), 64 rows a step: the 16-bit rows and the parts of the fp32
// ones go through LDS (the next step's on their way in registers, the places of the
// one after that too), both read transposed; a row's 32-byte pieces are moved about so
// that the 8 rows that 32 lanes read together meet different banks. da's lanes end with
// 4 consecutive columns of a rank row, db's with 4 ranks of a column's row: the
// operands change places. 8192 rows of 4096, rank 64, both gradients: 69 to 72 us (eight waves
// of 64 x 32 with rows padded instead of moved about, and a mask at every product, 107).
constexpr int GRAD_WG = 256, GRAD_COLS = 256, GRAD_ROWS = 64;
constexpr int GRAD_XROW = GRAD_COLS * 2, GRAD_TROW = 128;      // bytes in LDS
__device__ __forceinline__ int swz_x(int k) { return (k & 3) | (k >> 3 & 1) << 2; }
__device__ __forceinline__ int swz_t(int k) { return (k >> 1 & 1) | (k >> 3 & 1) << 1; }
template <int DT, bool DB>
__device__ __forceinline__ void lora_grad(const LoraGrad& a, int4 seg, int slot, int j0, int c0, uint8_t* sx, uint8_t* st,
                                          uint32_t* s_top, int (*s_rows)[GRAD_ROWS]) {
  constexpr int XROW = GRAD_XROW, TROW = GRAD_TROW;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, col = lane & 15, quad = lane >> 4;
  const int cols = DB ? a.out : a.in;
  const float* tp = DB ? a.t : a.u;
  const uint16_t* xp = static_cast<const uint16_t*>(DB ? a.dy : a.x);
  const int64_t ld = DB ? a.lddy : a.ldx;
  auto place = [&](int i) { return i < seg.z ? a.rows[(int64_t)seg.w * LORA_TILE + i] : -1; };
  int e = 0;                                       // fp16: parts are |t| 2^-e, below 2^14
  if constexpr (DT == DT_F16) {
    const uint32_t* top = (DB ? a.top_t : a.top_u) + seg.w * (LORA_TILE / 16);
    uint32_t m = 0;
    for (int i = threadIdx.x; i < (seg.z + 15) / 16; i += GRAD_WG) m = max(m, top[i]);
#pragma unroll
    for (int d = 32; d; d >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
    if (lane == 0) s_top[w] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < GRAD_WG / 64; ++i) m = max(m, s_top[i]);
    e = exponent(m) - 14;
  }
  // x: 32 chunks a row, 8 rows at a time; t: 4 threads a row, 16 of the rank each
  const int xr = threadIdx.x >> 5, xc = threadIdx.x & 31, tr = threadIdx.x >> 2, tc = threadIdx.x & 3;
  u32x4 xv[8];
  float tv[16];
  int next = -1;
  // whether nothing of what the workgroup loads lies behind its rows' ends
  const bool whole = c0 + GRAD_COLS <= cols && j0 + 64 <= a.rank;
  auto load = [&](const int* rows, int left) {
    if (whole && left >= GRAD_ROWS) {
#pragma unroll
      for (int i = 0; i < 8; ++i) __builtin_memcpy(&xv[i], xp + rows[xr + i * 8] * ld + (c0 + xc * 8), 16);
      const float* t = tp + (int64_t)rows[tr] * a.rank + (j0 + tc * 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) __builtin_memcpy(tv + i * 4, t + i * 4, 16);
      return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = rows[xr + i * 8];
      xv[i] = u32x4{0, 0, 0, 0};
      if (r >= 0 && c0 + xc * 8 < cols) xv[i] = load_chunk<2, true>(xp + r * ld, (int64_t)(c0 + xc * 8) * 2, (int64_t)cols * 2);
    }
    const int r = rows[tr];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u32x4 v = {0, 0, 0, 0};
      if (r >= 0 && j0 + tc * 16 + i * 4 < a.rank)
        v = load_chunk<4>(tp + (int64_t)r * a.rank, (int64_t)(j0 + tc * 16 + i * 4) * 4, (int64_t)a.rank * 4);
      unpack16<DT_F32>(v, tv + i * 4);
    }
  };
  f32x4 acc[4][4];                                 // [x fragment][t fragment]
  auto sums = [&](bool safe) {
#pragma unroll
    for (int f = 0; f < 4; ++f)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[f][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (threadIdx.x < 2 * GRAD_ROWS) s_rows[threadIdx.x / GRAD_ROWS][threadIdx.x % GRAD_ROWS] = place(threadIdx.x);
    __syncthreads();
    if (seg.z > 0) load(s_rows[0], seg.z);
    for (int i0 = 0, step = 0; i0 < seg.z; i0 += GRAD_ROWS, ++step) {
      __syncthreads();                             // the last step's readers are done
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int k = xr + i * 8;
        *reinterpret_cast<u32x4*>(sx + k * XROW + ((xc >> 1) ^ swz_x(k)) * 32 + (xc & 1) * 16) = xv[i];
      }
      float low[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if constexpr (DT == DT_F16) tv[i] = __builtin_ldexpf(tv[i], -e);
        low[i] = safe ? low_part<DT>(tv[i]) : tv[i] - Row<DT>::f(to16<DT>(tv[i]));
      }
      uint8_t* h = st + tr * TROW + (tc ^ swz_t(tr)) * 32;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        *reinterpret_cast<u32x4*>(h + i * 16) = pack16<DT>(tv + i * 8);
        *reinterpret_cast<u32x4*>(h + GRAD_ROWS * TROW + i * 16) = pack16<DT>(low + i * 8);
      }
      if (step && threadIdx.x < GRAD_ROWS) s_rows[(step + 1) & 1][threadIdx.x] = next;
      __syncthreads();
      if (threadIdx.x < GRAD_ROWS) next = place(i0 + 2 * GRAD_ROWS + threadIdx.x);
      if (i0 + GRAD_ROWS < seg.z) load(s_rows[(step + 1) & 1], seg.z - i0 - GRAD_ROWS);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int kr = k * 32 + quad * 8 + (col >> 2);         // kr + 4: the same pieces
        u32x4 x[4];
#pragma unroll
        for (int f = 0; f < 4; ++f) x[f] = read_tr(sx + kr * XROW + ((w * 4 + f) ^ swz_x(kr)) * 32 + (col & 3) * 8, 4 * XROW);
#pragma unroll
        for (int p = 0; p < 2; ++p) {              // the high parts, then the low ones
          if (p && safe)
#pragma unroll
            for (int f = 0; f < 4; ++f) x[f] = finite_or_zero<DT>(x[f]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const u32x4 t = read_tr(st + (p * GRAD_ROWS + kr) * TROW + (j ^ swz_t(kr)) * 32 + (col & 3) * 8, 4 * TROW);
#pragma unroll
            for (int f = 0; f < 4; ++f) acc[f][j] = DB ? Elem<DT>::mma16(t, x[f], acc[f][j]) : Elem<DT>::mma16(x[f], t, acc[f][j]);
          }
        }
      }
    }
    __syncthreads();
  };
  sums(false);
  float far = 0.f;
#pragma unroll
  for (int f = 0; f < 4; ++f)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) far = __builtin_fmaf(0.f, acc[f][j][q], far);
  if (__syncthreads_or(far != 0.f)) sums(true);
  const float scale = seg.z ? a.scale[seg.x] : 0.f;       // (no row: zeros, whatever stands in the scale)
  // four consecutive values of a row of the result, n long, from column c on: rounded,
  // or (one of several segments) as they are
  const int64_t size = (int64_t)a.rank * cols;
  float* part = slot < 0 ? nullptr : a.part + (int64_t)slot * a.rank * (a.in + (int64_t)a.out) + (DB ? (int64_t)a.rank * a.in : 0);
  uint16_t* out = static_cast<uint16_t*>(DB ? a.db : a.da) + seg.x * size;
#pragma unroll
  for (int f = 0; f < 4; ++f)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = DB ? a.rank : cols;
      const int row = DB ? c0 + w * 64 + f * 16 + col : j0 + j * 16 + col;
      const int c = DB ? j0 + j * 16 + quad * 4 : c0 + w * 64 + f * 16 + quad * 4;
      if (row >= (DB ? cols : a.rank) || c >= n) continue;
      float v[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        v[q] = DT == DT_F16 ? __builtin_ldexpf(acc[f][j][q], e) : acc[f][j][q];
        if (!part) v[q] *= scale;
      }
      const int64_t at = (int64_t)row * n + c;
      if (part) {
        if (c + 4 <= n) __builtin_memcpy(part + at, v, 16);    // at any alignment
        else
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (c + q < n) part[at + q] = v[q];
      } else {
        uint16_t b[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) b[q] = to16<DT>(v[q]);
        if (c + 4 <= n) __builtin_memcpy(out + at, b, 8);
        else
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (c + q < n) out[at + q] = b[q];
      }
    }
}
template <int DT> __global__ __launch_bounds__(GRAD_WG, 2) void k_lora_grad(LoraGrad a, int in_tiles) {
  __shared__ __align__(64) uint8_t sx[GRAD_ROWS * GRAD_XROW], st[2 * GRAD_ROWS * GRAD_TROW];
  __shared__ uint32_t s_top[GRAD_WG / 64];
  __shared__ int s_rows[2][GRAD_ROWS];
  const int4 seg = a.segs[blockIdx.x];
  if (seg.x < 0) return;
  const int slot = a.slot[blockIdx.x], j0 = blockIdx.z * 64;
  if ((int)blockIdx.y < in_tiles) lora_grad<DT, false>(a, seg, slot, j0, blockIdx.y * GRAD_COLS, sx, st, s_top, s_rows);
  else lora_grad<DT, true>(a, seg, slot, j0, (blockIdx.y - in_tiles) * GRAD_COLS, sx, st, s_top, s_rows);
}
// the sums of adapters of several segments, in order, four a thread
template <int DT> __global__ __launch_bounds__(256) void k_lora_join(LoraGrad a) {
  const int2 span = a.span[blockIdx.y];
  if (!span.y) return;
  const int64_t na = (int64_t)a.rank * a.in, n = na + (int64_t)a.rank * a.out;
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= n) return;
  const float* p = a.part + span.x * n + i;
  const int m = (int)min(n - i, (int64_t)4);
  float v[4] = {};
  if (m == 4) {
#pragma unroll 4
    for (int s = 0; s < span.y; ++s) {
      float f[4];
      __builtin_memcpy(f, p + s * n, 16);          // at any alignment
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = s ? v[e] + f[e] : f[e];
    }
  } else {
    for (int e = 0; e < m; ++e) {
      v[e] = p[e];
      for (int s = 1; s < span.y; ++s) v[e] += p[s * n + e];
    }
  }
  const float scale = a.scale[blockIdx.y];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int64_t k = i + e;
    if (k >= n) continue;
    if (k < na) static_cast<uint16_t*>(a.da)[blockIdx.y * na + k] = to16<DT>(scale * v[e]);
    else static_cast<uint16_t*>(a.db)[blockIdx.y * (n - na) + k - na] = to16<DT>(scale * v[e]);
  }
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

// K ranges of the long contraction: enough workgroups for two a CU, 256 k each at least
int lora_splits(int rows, int k, int rank) {
  const int tiles = (rows + LORA_TILE - 1) / LORA_TILE * ((rank + 63) / 64);
  return std::max(1, std::min((512 + tiles - 1) / tiles, (k + 255) / 256));
}
template <int DT, bool KM> static hipError_t shrink(const LoraShrink& a, hipStream_t s) {
  const dim3 grid(a.max_tiles, (a.rank + 63) / 64, a.splits), wg(256);
  if (a.rank <= 16) hipLaunchKernelGGL((k_lora_shrink<DT, KM, 1>), grid, wg, 0, s, a);
  else if (a.rank <= 32) hipLaunchKernelGGL((k_lora_shrink<DT, KM, 2>), grid, wg, 0, s, a);
  else hipLaunchKernelGGL((k_lora_shrink<DT, KM, 4>), grid, wg, 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((k_lora_parts<DT>), dim3(a.max_tiles, LORA_TILE / 16), wg, 0, s, a);
  return hipGetLastError();
}
hipError_t launch_lora_shrink(int dt, bool k_major, const LoraShrink& a, hipStream_t s) {
  if (dt == DT_BF16) return k_major ? shrink<DT_BF16, true>(a, s) : shrink<DT_BF16, false>(a, s);
  if (dt == DT_F16) return k_major ? shrink<DT_F16, true>(a, s) : shrink<DT_F16, false>(a, s);
  return hipErrorInvalidValue;
}

template <int DT, bool KM> static hipError_t expand(const LoraExpand& a, hipStream_t s) {
  const dim3 grid(a.max_tiles, (a.cols + a.chunk - 1) / a.chunk);
  if (a.rp == 32) hipLaunchKernelGGL((k_lora_expand<DT, KM, 1>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_lora_expand<DT, KM, 2>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}
// Columns of a workgroup: as few as leave four workgroups a CU
int lora_chunk(int rows, int cols) {
  const int64_t tiles = (rows + LORA_TILE - 1) / LORA_TILE;
  return (int)((cols * tiles / EXP_WGS + 63) / 64 + (cols * tiles < EXP_WGS)) * 64;
}
hipError_t launch_lora_expand(int dt, bool k_major, const LoraExpand& a, hipStream_t s) {
  if (dt == DT_BF16) return k_major ? expand<DT_BF16, true>(a, s) : expand<DT_BF16, false>(a, s);
  if (dt == DT_F16) return k_major ? expand<DT_F16, true>(a, s) : expand<DT_F16, false>(a, s);
  return hipErrorInvalidValue;
}

template <int DT> static hipError_t grad(const LoraGrad& a, hipStream_t s) {
  const int ti = (a.in + GRAD_COLS - 1) / GRAD_COLS, to = (a.out + GRAD_COLS - 1) / GRAD_COLS;
  hipLaunchKernelGGL((k_lora_grad<DT>), dim3(a.max_segs, ti + to, (a.rank + 63) / 64), dim3(GRAD_WG), 0, s, a, ti);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.join) return e;
  const int64_t n = (int64_t)a.rank * (a.in + (int64_t)a.out);
  hipLaunchKernelGGL((k_lora_join<DT>), dim3((uint32_t)((n + 1023) / 1024), a.adapters), dim3(256), 0, s, a);
  return hipGetLastError();
}
hipError_t launch_lora_grad(int dt, const LoraGrad& a, hipStream_t s) {
  if (dt == DT_BF16) return grad<DT_BF16>(a, s);
  if (dt == DT_F16) return grad<DT_F16>(a, s);
  return hipErrorInvalidValue;
}

// Few rows: one launch, each row's weights through one CU, against the tiles' four. It is the
// better one while rank (in + out) of a row stays below 256 Ki, whatever the rows: bf16, 16 rows
// of 4096 -> 4096, rank 16 12 us for 25, rank 32 20 for 25, rank 64 38 for 26; 64 rows of 2048 ->
// 2048, rank 32 13 for 29. The limit here is on all rows' products, and leaves the worse one on
// both sides of that: 4 rows of 4096, rank 256 take 124 us for 32, 64 rows of rank 32 35 for 27.
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

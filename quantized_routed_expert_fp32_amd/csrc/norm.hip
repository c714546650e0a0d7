// Root-mean-square norm of rows with the residual's addition before it:
//   total = x + residual                      (fp32, rounded to the result's type)
//   y = total rstd w,  rstd = 1 / sqrt(mean(total^2) + eps)
// or in 8 bits: v = total w in fp32, s0 = fp32(max|v| / 127), the codes of v / s0 and
// the scale s0 rstd. rstd is common to a row and leaves the codes alone, so they
// depend on no sum's order. And its gradients
//   g = dy w,  dx = rstd (g - total rstd^2 mean(g total)) + dtotal,  dw = sum_r dy total rstd.
//
// A row is held in registers (its total, 16 bits an element) between the sum and
// the result: one pass over memory, which bounds the long calls; the short ones
// are bound by the launch and the row's own latency.
#include "block_launch.h"
#include "dense_rows.h"

namespace moe {

constexpr int NORM_WAVES = 8192;       // waves of a call at most, 32 a CU
// a workgroup's sums of dw: whole chunks
static __host__ __device__ int64_t part_ld(int hidden) { return (int64_t)(hidden + 7) / 8 * 8; }

// ------------------------------------------------------------------- sums
// over the TPR threads that hold a row: a wave, or the whole workgroup
template <int TPR> __device__ __forceinline__ float row_sum(float v, float* red) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
  if constexpr (TPR > 64) {
    __syncthreads();                 // the last sum's readers are done
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int i = 1; i < TPR / 64; ++i) v += red[i];
  }
  return v;
}
template <int TPR> __device__ __forceinline__ uint32_t row_max(uint32_t m, uint32_t* red) {
#pragma unroll
  for (int d = 32; d; d >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
  if constexpr (TPR > 64) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
    __syncthreads();
    m = red[0];
#pragma unroll
    for (int i = 1; i < TPR / 64; ++i) m = max(m, red[i]);
  }
  return m;
}

// ------------------------------------------------------------------ chunks
// A chunk is 8 elements. From 16-bit rows, or from fp32 ones (two loads).
template <int T> __device__ __forceinline__ void load8(const void* row, int c, int cols, float* f) {
  if constexpr (T == DT_F32) {
    unpack16<DT_F32>(load_chunk<4, true>(row, (int64_t)c * 32, (int64_t)cols * 4), f);
    if (c * 8 + 4 < cols) {
      unpack16<DT_F32>(load_chunk<4, true>(row, (int64_t)c * 32 + 16, (int64_t)cols * 4), f + 4);
    } else {
#pragma unroll
      for (int i = 4; i < 8; ++i) f[i] = 0.f;
    }
  } else {
    unpack16<T>(load_chunk<2, true>(row, (int64_t)c * 16, (int64_t)cols * 2), f);
  }
}
// the weights of chunk c, as the products take them
template <int DT> __device__ __forceinline__ void weights8(const void* w, int w_dt, float add, int c, int cols, float* f) {
  if (w_dt == DT_F32) load8<DT_F32>(w, c, cols, f);
  else load8<DT>(w, c, cols, f);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] += add;      // no change where add is 0
}
__device__ __forceinline__ void store_chunk(void* row, int c, int cols, u32x4 v) {
  uint16_t* o = static_cast<uint16_t*>(row) + c * 8;
  if (c * 8 + 8 <= cols) __builtin_memcpy(o, &v, 16);      // at any alignment
  else
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c * 8 + i < cols) o[i] = (uint16_t)(v[i / 2] >> (16 * (i & 1)));
}

// 1 / sqrt(mean + eps) of a row whose elements are held as NC chunks a thread.
// bf16 has the range of fp32, so the squares of a finite row may not: such a row is
// taken times 2^-80 (the mean is then below 2^96, and eps below its rounding).
template <int DT, int TPR, int NC>
__device__ __forceinline__ float row_rstd(const u32x4* held, int cols, float eps, float* red) {
  float ss = 0.f;
#pragma unroll
  for (int h = 0; h < NC; ++h) {
    float f[8];
    unpack16<DT>(held[h], f);
#pragma unroll
    for (int i = 0; i < 8; ++i) ss += f[i] * f[i];
  }
  ss = row_sum<TPR>(ss, red);
  if constexpr (DT == DT_BF16) {
    if (ss == __builtin_inff()) {               // the same for the whole row
      const float down = __builtin_ldexpf(1.f, -80);
      ss = 0.f;
#pragma unroll
      for (int h = 0; h < NC; ++h) {
        float f[8];
        unpack16<DT>(held[h], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss += (f[i] * down) * (f[i] * down);
      }
      ss = row_sum<TPR>(ss, red);
      return down / __builtin_sqrtf(ss / (float)cols);
    }
  }
  return 1.f / __builtin_sqrtf(ss / (float)cols + eps);
}

// ---------------------------------------------------------------- the norm
// A workgroup takes rows blockIdx, blockIdx + gridDim.. one at a time, a chunk (NC,
// beyond 8192 columns) a thread, the next row's loads in flight while a row is reduced
// and written; each thread holds its columns' weights. 8192 x 4096 with a residual:
// 42 to 48 us for 268 MB, 5.6 to 6.4 TB/s (a row without the next one's loads 54 to 62); in
// 8 bits 57. Beyond 16384 columns (NC = 8) a row and the next one are more than the registers
// hold: as many elements take 187 us through scratch, in 8 bits 254, their gradients 430.
template <int DT, int XT, bool I8, int TPR, int NC> __global__ __launch_bounds__(TPR) void k_norm(NormArgs a) {
  __shared__ float red[TPR / 64];
  __shared__ uint32_t redm[TPR / 64];
  constexpr int XL = XT == DT_F32 ? 2 : 1;       // loads of a chunk of x
  const int t = threadIdx.x;
  const int chunks = (a.hidden + 7) / 8;
  u32x4 xs[NC][XL], rs[NC];
  auto load = [&](int64_t r) {
    const char* xr = static_cast<const char*>(a.x) + r * a.ldx * (XT == DT_F32 ? 4 : 2);
    const char* rr = static_cast<const char*>(a.res) + r * a.ldres * 2;
#pragma unroll
    for (int h = 0; h < NC; ++h) {
      const int c = h * TPR + t;
      if (c >= chunks) continue;
#pragma unroll
      for (int l = 0; l < XL; ++l) {
        constexpr int ES = XT == DT_F32 ? 4 : 2;
        xs[h][l] = u32x4{0, 0, 0, 0};
        if (l == 0 || c * 8 + 4 < a.hidden)
          xs[h][l] = load_chunk<ES, true>(xr, ((int64_t)c * XL + l) * 16, (int64_t)a.hidden * ES);
      }
      if (a.res) rs[h] = load_chunk<2, true>(rr, (int64_t)c * 16, (int64_t)a.hidden * 2);
    }
  };
  load(blockIdx.x);
  float w[NC][8];
#pragma unroll
  for (int h = 0; h < NC; ++h) {
    const int c = h * TPR + t;
    if (c < chunks) weights8<DT>(a.w, a.w_dt, a.w_add, c, a.hidden, w[h]);
  }
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    u32x4 held[NC];
#pragma unroll
    for (int h = 0; h < NC; ++h) {
      held[h] = u32x4{0, 0, 0, 0};
      if (h * TPR + t >= chunks) continue;
      if (XT != DT_F32 && !a.res) {
        held[h] = xs[h][0];
        continue;
      }
      float f[8], g[8];
#pragma unroll
      for (int l = 0; l < XL; ++l) unpack16<XT>(xs[h][l], f + 4 * l);
      unpack16<DT>(rs[h], g);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] += g[i];
      held[h] = pack16<DT>(f);
    }
    if (r + gridDim.x < a.rows) load(r + gridDim.x);
    if (a.res) {
      char* tr = static_cast<char*>(a.total) + r * a.ldtotal * 2;
#pragma unroll
      for (int h = 0; h < NC; ++h)
        if (h * TPR + t < chunks) store_chunk(tr, h * TPR + t, a.hidden, held[h]);
    }
    const float rstd = row_rstd<DT, TPR, NC>(held, a.hidden, a.eps, red);
    if (a.rstd && t == 0) a.rstd[r] = rstd;
    char* yr = static_cast<char*>(a.y) + r * a.ldy * 2;
    if (!I8 || a.y) {
#pragma unroll
      for (int h = 0; h < NC; ++h) {
        const int c = h * TPR + t;
        if (c >= chunks) continue;
        float f[8];
        unpack16<DT>(held[h], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = f[i] * rstd * w[h][i];
        store_chunk(yr, c, a.hidden, pack16<DT>(f));
      }
    }
    if constexpr (I8) {
      uint32_t m = 0;
#pragma unroll
      for (int h = 0; h < NC; ++h) {
        const int c = h * TPR + t;
        if (c >= chunks) continue;
        float f[8];
        unpack16<DT>(held[h], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = c * 8 + i < a.hidden ? f[i] * w[h][i] : 0.f;
        m = top_bits<DT_F32, 8>(f, m);
      }
      const RowScale sc(row_max<TPR>(m, redm));
      if (t == 0) a.scale[r] = sc.s * rstd;
      int8_t* qr = a.q + r * a.ldq;
#pragma unroll
      for (int h = 0; h < NC; ++h) {
        const int c = h * TPR + t;
        if (c >= chunks) continue;
        float f[8];
        unpack16<DT>(held[h], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= w[h][i];
        const uint32_t o[2] = {sc.codes4(f), sc.codes4(f + 4)};
        if (c * 8 + 8 <= a.hidden) __builtin_memcpy(qr + c * 8, o, 8);
        else
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (c * 8 + i < a.hidden) qr[c * 8 + i] = (int8_t)(o[i / 4] >> (8 * (i & 3)));
      }
    }
  }
}

// ------------------------------------------------------------- its gradients
// Workgroup b takes rows [b, b + 1) rows / gridDim one at a time, a chunk (NC, beyond
// 8192 columns) a thread; the next row's loads are in flight while a row is reduced
// and written. Each thread holds its columns' weights, and sums their dw over its
// rows in fp32; k_norm_dw adds the workgroups' sums in order. 8192 x 4096 with dtotal:
// 48 us, 5.6 TB/s (several rows at once without loads ahead 148), and 5 for k_norm_dw.
template <int DT, int TPR, int NC> __global__ __launch_bounds__(TPR) void k_norm_grad(NormGradArgs a) {
  __shared__ float red[TPR / 64];
  const int t = threadIdx.x;
  const int chunks = (a.hidden + 7) / 8;
  const int64_t r0 = (int64_t)a.rows * blockIdx.x / gridDim.x, r1 = (int64_t)a.rows * (blockIdx.x + 1) / gridDim.x;
  float dw[NC][8] = {}, w[NC][8];
#pragma unroll
  for (int h = 0; h < NC; ++h) {
    const int c = h * TPR + t;
    if (c < chunks) weights8<DT>(a.w, a.w_dt, a.w_add, c, a.hidden, w[h]);
  }
  u32x4 xs[NC], es[NC], us[NC];
  float rstd = 0.f;
  auto load = [&](int64_t r) {
    const char* xr = static_cast<const char*>(a.x) + r * a.ldx * 2;
    const char* er = static_cast<const char*>(a.dy) + r * a.lddy * 2;
    const char* ur = static_cast<const char*>(a.dtotal) + r * a.lddtotal * 2;
    const int64_t end = (int64_t)a.hidden * 2;
#pragma unroll
    for (int h = 0; h < NC; ++h) {
      const int c = h * TPR + t;
      xs[h] = es[h] = us[h] = u32x4{0, 0, 0, 0};
      if (c >= chunks) continue;
      xs[h] = load_chunk<2, true>(xr, (int64_t)c * 16, end);
      es[h] = load_chunk<2, true>(er, (int64_t)c * 16, end);
      if (a.dtotal) us[h] = load_chunk<2, true>(ur, (int64_t)c * 16, end);
    }
    rstd = a.rstd[r];
  };
  if (r0 < r1) load(r0);
  for (int64_t r = r0; r < r1; ++r) {
    u32x4 xv[NC], ev[NC], uv[NC];
    const float rs = rstd;
#pragma unroll
    for (int h = 0; h < NC; ++h) {
      xv[h] = xs[h];
      ev[h] = es[h];
      uv[h] = us[h];
    }
    if (r + 1 < r1) load(r + 1);
    float dot = 0.f;
#pragma unroll
    for (int h = 0; h < NC; ++h) {
      if (h * TPR + t >= chunks) continue;
      float x[8], e[8];
      unpack16<DT>(xv[h], x);
      unpack16<DT>(ev[h], e);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float n = x[i] * rs;
        dot += e[i] * w[h][i] * n;
        dw[h][i] += e[i] * n;
      }
    }
    if (!a.dx) continue;
    dot = row_sum<TPR>(dot, red) / (float)a.hidden;
    char* dr = static_cast<char*>(a.dx) + r * a.lddx * 2;
#pragma unroll
    for (int h = 0; h < NC; ++h) {
      const int c = h * TPR + t;
      if (c >= chunks) continue;
      float x[8], e[8], u[8];
      unpack16<DT>(xv[h], x);
      unpack16<DT>(ev[h], e);
      unpack16<DT>(uv[h], u);
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = rs * (e[i] * w[h][i] - x[i] * rs * dot) + u[i];
      store_chunk(dr, c, a.hidden, pack16<DT>(e));
    }
  }
  if (!a.dw) return;
  float* part = a.part + (int64_t)blockIdx.x * part_ld(a.hidden);
#pragma unroll
  for (int h = 0; h < NC; ++h) {
    const int c = h * TPR + t;
    if (c >= chunks) continue;
#pragma unroll
    for (int i = 0; i < 8; i += 4) *reinterpret_cast<f32x4*>(part + c * 8 + i) = f32x4{dw[h][i], dw[h][i + 1], dw[h][i + 2], dw[h][i + 3]};
  }
}

// dw[c]: the workgroups' sums, 32 columns a workgroup, four a thread, each in 128
// stretches joined in order
template <int DT> __global__ __launch_bounds__(1024) void k_norm_dw(NormGradArgs a, int parts) {
  __shared__ float red[128][33];
  __shared__ float red2[32][33];
  const int c = blockIdx.x * 32 + (threadIdx.x & 7) * 4, s = threadIdx.x >> 3;
  const int64_t ld = part_ld(a.hidden);
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  if (c < a.hidden) {
    const int p1 = parts * (s + 1) / 128;
#pragma unroll 4
    for (int p = parts * s / 128; p < p1; ++p) v += *reinterpret_cast<const f32x4*>(a.part + p * ld + c);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) red[s][(threadIdx.x & 7) * 4 + i] = v[i];
  __syncthreads();
  const int col = threadIdx.x & 31, g = threadIdx.x >> 5;
  red2[g][col] = (red[g * 4][col] + red[g * 4 + 1][col]) + (red[g * 4 + 2][col] + red[g * 4 + 3][col]);
  __syncthreads();
  const int cc = blockIdx.x * 32 + col;
  if (g || cc >= a.hidden) return;
  float sum = red2[0][col];
#pragma unroll
  for (int i = 1; i < 32; ++i) sum += red2[i][col];
  if (a.w_dt == DT_F32) static_cast<float*>(a.dw)[cc] = sum;
  else static_cast<uint16_t*>(a.dw)[cc] = to16<DT>(sum);
}

// --------------------------------------------------------------- launchers
// Threads of a row: a chunk each, up to 1024
static int row_threads(int hidden) {
  const int chunks = (hidden + 7) / 8;
  int t = 64;
  while (t < chunks && t < 1024) t *= 2;
  return t;
}
template <int DT, int XT, bool I8, int TPR, int NC> static hipError_t norm_run(const NormArgs& a, hipStream_t s) {
  const int most = NORM_WAVES * 64 / TPR;
  hipLaunchKernelGGL((k_norm<DT, XT, I8, TPR, NC>), dim3(a.rows < most ? a.rows : most), dim3(TPR), 0, s, a);
  return hipGetLastError();
}
template <int DT, int XT, bool I8> static hipError_t norm_pick(const NormArgs& a, hipStream_t s) {
  switch (row_threads(a.hidden)) {
    case 64: return norm_run<DT, XT, I8, 64, 1>(a, s);
    case 128: return norm_run<DT, XT, I8, 128, 1>(a, s);
    case 256: return norm_run<DT, XT, I8, 256, 1>(a, s);
    case 512: return norm_run<DT, XT, I8, 512, 1>(a, s);
  }
  const int chunks = (a.hidden + 7) / 8;
  if (chunks <= 1024) return norm_run<DT, XT, I8, 1024, 1>(a, s);
  if (chunks <= 2048) return norm_run<DT, XT, I8, 1024, 2>(a, s);
  if (chunks <= 8192) return norm_run<DT, XT, I8, 1024, 8>(a, s);
  return hipErrorInvalidValue;
}
template <int DT> static hipError_t norm_dt(const NormArgs& a, hipStream_t s) {
  if (a.x_dt == DT_F32) return a.q ? norm_pick<DT, DT_F32, true>(a, s) : norm_pick<DT, DT_F32, false>(a, s);
  return a.q ? norm_pick<DT, DT, true>(a, s) : norm_pick<DT, DT, false>(a, s);
}
hipError_t launch_norm(int dt, const NormArgs& a, hipStream_t s) {
  if (dt == DT_BF16) return norm_dt<DT_BF16>(a, s);
  if (dt == DT_F16) return norm_dt<DT_F16>(a, s);
  return hipErrorInvalidValue;
}

// Workgroups of the gradients: 16 waves a CU. Their sums of dw take up to 8 MiB of the
// workspace for 8192 columns, beyond that (1024 threads a row, so no fewer workgroups) up to
// 64 MiB for 65536.
static int norm_grad_parts(int rows, int hidden) {
  const int most = 4096 * 64 / row_threads(hidden);
  return rows < most ? rows : most;
}
int64_t norm_grad_words(int rows, int hidden) { return norm_grad_parts(rows, hidden) * part_ld(hidden); }
template <int DT, int TPR, int NC> static hipError_t grad_run(const NormGradArgs& a, hipStream_t s) {
  const int parts = norm_grad_parts(a.rows, a.hidden);
  hipLaunchKernelGGL((k_norm_grad<DT, TPR, NC>), dim3(parts), dim3(TPR), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.dw) return e;
  hipLaunchKernelGGL((k_norm_dw<DT>), dim3((a.hidden + 31) / 32), dim3(1024), 0, s, a, parts);
  return hipGetLastError();
}
template <int DT> static hipError_t grad_pick(const NormGradArgs& a, hipStream_t s) {
  switch (row_threads(a.hidden)) {
    case 64: return grad_run<DT, 64, 1>(a, s);
    case 128: return grad_run<DT, 128, 1>(a, s);
    case 256: return grad_run<DT, 256, 1>(a, s);
    case 512: return grad_run<DT, 512, 1>(a, s);
  }
  const int chunks = (a.hidden + 7) / 8;
  if (chunks <= 1024) return grad_run<DT, 1024, 1>(a, s);
  if (chunks <= 2048) return grad_run<DT, 1024, 2>(a, s);
  if (chunks <= 8192) return grad_run<DT, 1024, 8>(a, s);
  return hipErrorInvalidValue;
}
hipError_t launch_norm_grad(int dt, const NormGradArgs& a, hipStream_t s) {
  if (dt == DT_BF16) return grad_pick<DT_BF16>(a, s);
  if (dt == DT_F16) return grad_pick<DT_F16>(a, s);
  return hipErrorInvalidValue;
}

}  // namespace moe

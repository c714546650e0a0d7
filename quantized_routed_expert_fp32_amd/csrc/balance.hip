// Balance of a router: how often each expert was picked, and two losses over the
// rows that count (n of them; all, or those that a mask keeps)
//   f_e = counts_e / (n k),  P_e = 1/n sum_r p_re,  p_r = softmax(l_r)
//   balance = E sum_e f_e P_e,   z = 1/n sum_r lse_r^2,  lse_r = log sum_e exp(l_re)
// with the gradient (the counts are constants to it)
//   dl_re = p_re / n (gb E (f_e - sum_j f_j p_rj) + 2 gz lse_r).
//
// One pass over the logits each way, in registers: bound by their bytes. Both
// compute the softmax from the logits, so that nothing of it is kept (lse in fp32
// would lose bits of p where logits are far from zero). A row lies in 16 lanes (64
// beyond 256 experts), four consecutive logits a lane and load at any alignment (a
// router's logits may stand beside the shared gate's, in rows of 257), and its
// reductions run in the lanes' own rows of 16.
#include "block_launch.h"
#include "dense_rows.h"

namespace moe {

constexpr int BAL_WG = 512;         // threads of a workgroup
constexpr int BAL_PARTS = 256;      // workgroups at most: a sum of each for k_balance_join
constexpr int BAL_ONE = 256;        // rows that one workgroup takes, joined in the same launch

template <int CTRL> __device__ __forceinline__ float lanes(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, false));
}
// Over the G lanes of a row, the same bits in each: neighbours, pairs, quads
// (a half row's mirror), halves (a row's mirror), then across the rows of 16.
template <int G, typename F> __device__ __forceinline__ float over(float v, F f) {
  v = f(v, lanes<0xB1>(v));
  v = f(v, lanes<0x4E>(v));
  v = f(v, lanes<0x141>(v));
  v = f(v, lanes<0x140>(v));
  if constexpr (G == 64) {
    v = f(v, __shfl_xor(v, 16));
    v = f(v, __shfl_xor(v, 32));
  }
  return v;
}
__device__ __forceinline__ float add(float a, float b) { return a + b; }
// NaN stays
__device__ __forceinline__ float top(float a, float b) { return a > b || a != a ? a : b; }

// four logits from column c on, -inf behind the last
template <int T> __device__ __forceinline__ void logits4(const void* row, int c, int n, float* v) {
  typedef typename Row<T>::type E;
  const E* at = static_cast<const E*>(row) + c;
  E b[4];
  if (c + 4 <= n) {
    __builtin_memcpy(b, at, sizeof b);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = Row<T>::f(b[e]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = c + e < n ? Row<T>::f(at[e]) : -__builtin_inff();
  }
}

// e^d of d <= 0 = 2^n 2^f, n the whole number next to d log2 e, f the rest (log2 e in two
// parts, the first one's product exact), 2^f from the hardware. Off by 0.97 ulp at most over all
// fp32 arguments (expf: 0.86), subnormal results by one step. The forward kernel takes 20 us for
// 65536 x 256 fp32, with expf 22. A NaN is lost here (softmax has it).
__device__ __forceinline__ float exp_neg(float d) {
  constexpr float L = 1.44269502f, REST = 1.92596303e-8f;
  d = __builtin_fmaxf(d, -200.f);
  const float n = __builtin_rintf(d * L), f = __builtin_fmaf(d, REST, __builtin_fmaf(d, L, -n));
  return __builtin_ldexpf(__builtin_amdgcn_exp2f(f), (int)n);
}
// p of a row in place of its logits; its logsumexp
template <int G, int NI> __device__ __forceinline__ float softmax(float (&v)[NI][4]) {
  float m = v[0][0];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) m = top(m, v[i][e]);
  m = over<G>(m, top);
  float z = 0.f;
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) z += v[i][e] = exp_neg(v[i][e] - m);
  z = over<G>(z, add) + (m - m);                  // NaN where the largest is not finite
  const float inv = 1.f / z;
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) v[i][e] *= inv;
  return m + logf(z);
}

// A workgroup's sums in the workspace: ep sums of p (fp32), ep counts, lse^2 (64 bits), rows.
// A thread adds its own rows of p in fp32 (in long calls rows / 8192 of them, beyond 256
// experts rows / 2048); everything behind that, and lse^2 from its product on, is added in
// 64 bits: one chain of fp32 additions over a workgroup's 32 groups cost the z loss of 64
// rows 1.0e-7 where its own rounding is 3e-8.
struct Part {
  int ep;
  int64_t words;
  __host__ __device__ explicit Part(int experts) : ep((experts + 3) / 4 * 4), words(2 * ((experts + 3) / 4 * 4) + 4) {}
};

// The workgroups' sums in order, by one workgroup: 16 bytes a load, each column
// in up to 16 stretches.
__device__ __forceinline__ void join(const BalanceArgs& a, int parts) {
  __shared__ double seg[BAL_WG][4];
  __shared__ double loss[BAL_WG / 64];
  __shared__ double zsum;
  __shared__ int rows;
  const Part p(a.experts);
  const int q = p.ep / 4, units = 2 * q;                 // at most 512
  const int segs = min(BAL_WG / units, 16);
  const int u = threadIdx.x % units, s = threadIdx.x / units;
  if (s < segs) {
    const float* at = a.part + u * 4;
    const int p0 = (int)((int64_t)parts * s / segs), p1 = (int)((int64_t)parts * (s + 1) / segs);
    if (u < q) {
      double v[4] = {0, 0, 0, 0};
#pragma unroll 8
      for (int i = p0; i < p1; ++i) {
        const f32x4 f = *reinterpret_cast<const f32x4*>(at + i * p.words);
        for (int e = 0; e < 4; ++e) v[e] += f[e];
      }
      for (int e = 0; e < 4; ++e) seg[threadIdx.x][e] = v[e];
    } else {
      i32x4 v = {0, 0, 0, 0};
#pragma unroll 8
      for (int i = p0; i < p1; ++i) v += *reinterpret_cast<const i32x4*>(at + i * p.words);
      for (int e = 0; e < 4; ++e) seg[threadIdx.x][e] = v[e];          // exact
    }
  }
  if (threadIdx.x < 64) {
    double z = 0;
    int n = 0;
    for (int i = threadIdx.x; i < parts; i += 64) {
      const float* at = a.part + i * p.words + 2 * p.ep;
      z += *reinterpret_cast<const double*>(at);
      n += __float_as_int(at[2]);
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) {
      z += __shfl_xor(z, d);
      n += __shfl_xor(n, d);
    }
    if (threadIdx.x == 0) {
      zsum = z;
      rows = n;
    }
  }
  __syncthreads();
  double mine = 0;
  if ((int)threadIdx.x < q) {
    double v[4] = {0, 0, 0, 0};
    double c[4] = {0, 0, 0, 0};
    for (int i = 0; i < segs; ++i)
      for (int e = 0; e < 4; ++e) {
        v[e] += seg[i * units + u][e];
        c[e] += seg[i * units + q + u][e];
      }
    for (int e = 0; e < 4; ++e)
      if (u * 4 + e < a.experts) {
        a.counts[u * 4 + e] = (int)c[e];
        mine += v[e] * c[e];
      }
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) mine += __shfl_xor(mine, d);
  if ((threadIdx.x & 63) == 0) loss[threadIdx.x >> 6] = mine;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < BAL_WG / 64; ++i) mine += loss[i];
    const double n = rows;
    a.losses[0] = rows ? (float)(mine * a.experts / (n * n * a.k)) : 0.f;
    a.losses[1] = rows ? (float)(zsum / n) : 0.f;
    a.counts[a.experts] = rows;
  }
}

// Workgroup b takes rows [b, b + 1) rows / gridDim, 512 / G at a time.
template <int T, int G, int NI> __global__ __launch_bounds__(BAL_WG) void k_balance(BalanceArgs a) {
  constexpr int GROUPS = BAL_WG / G, COLS = G * NI * 4;
  __shared__ float sp[GROUPS * COLS];               // 8 KiB NI
  __shared__ int hist[COLS];
  __shared__ double sz[GROUPS];
  __shared__ int sn[GROUPS];
  const int g = threadIdx.x % G, grp = threadIdx.x / G;
  for (int c = threadIdx.x; c < COLS; c += BAL_WG) hist[c] = 0;
  __syncthreads();
  const int64_t r0 = (int64_t)a.rows * blockIdx.x / gridDim.x, r1 = (int64_t)a.rows * (blockIdx.x + 1) / gridDim.x;
  float sum[NI][4] = {};
  double z2 = 0;
  int n = 0;
  for (int64_t r = r0 + grp; r < r1; r += GROUPS) {
    if (a.mask && !a.mask[r]) continue;             // (all lanes of the group)
    const char* row = static_cast<const char*>(a.logits) + r * a.ld * (int64_t)sizeof(typename Row<T>::type);
    float v[NI][4];
#pragma unroll
    for (int i = 0; i < NI; ++i) logits4<T>(row, (i * G + g) * 4, a.experts, v[i]);
    for (int j = g; j < a.k; j += G) {
      const int id = a.ids[r * a.k + j];
      if ((uint32_t)id < (uint32_t)a.experts) atomicAdd(&hist[id], 1);      // whole numbers: any order
    }
    const float lse = softmax<G, NI>(v);
    z2 += (double)lse * lse;
    ++n;
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[i][e] += v[i][e];
  }
#pragma unroll
  for (int i = 0; i < NI; ++i)
    *reinterpret_cast<f32x4*>(&sp[grp * COLS + (i * G + g) * 4]) = f32x4{sum[i][0], sum[i][1], sum[i][2], sum[i][3]};
  if (g == 0) {
    sz[grp] = z2;
    sn[grp] = n;
  }
  __syncthreads();
  const Part p(a.experts);
  float* part = a.part + blockIdx.x * p.words;
  for (int c = threadIdx.x; c < p.ep; c += BAL_WG) {
    double v = 0;
    for (int i = 0; i < GROUPS; ++i) v += sp[i * COLS + c];
    part[c] = (float)v;
    part[p.ep + c] = __int_as_float(hist[c]);
  }
  if (threadIdx.x == 0) {
    double z = 0;
    int rows = 0;
    for (int i = 0; i < GROUPS; ++i) {
      z += sz[i];
      rows += sn[i];
    }
    *reinterpret_cast<double*>(part + 2 * p.ep) = z;
    part[2 * p.ep + 2] = __int_as_float(rows);
  }
  if (gridDim.x == 1) {
    __syncthreads();
    join(a, 1);
  }
}
__global__ __launch_bounds__(BAL_WG) void k_balance_join(BalanceArgs a, int parts) { join(a, parts); }

template <int T> __device__ __forceinline__ void put4(void* row, int c, int n, const float* v) {
  typedef typename Row<T>::type E;
  E* at = static_cast<E*>(row) + c;
  E b[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (T == DT_F32) b[e] = v[e];
    else b[e] = to16<T>(v[e]);
  }
  if (c + 4 <= n) __builtin_memcpy(at, b, sizeof b);
  else
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (c + e < n) at[e] = b[e];
}

template <int T, int G, int NI> __global__ __launch_bounds__(256) void k_balance_grad(BalanceArgs a) {
  constexpr int GROUPS = 256 / G;
  const int g = threadIdx.x % G, grp = threadIdx.x / G;
  const int rows = a.counts[a.experts];
  const float n = (float)rows, gb = a.dlosses[0] * (float)a.experts, gz = 2.f * a.dlosses[1];
  float f[NI][4];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int c = (i * G + g) * 4 + e;
      f[i][e] = c < a.experts && rows ? (float)a.counts[c] / (n * (float)a.k) : 0.f;
    }
  for (int64_t r = (int64_t)blockIdx.x * GROUPS + grp; r < a.rows; r += (int64_t)gridDim.x * GROUPS) {
    const bool in = !a.mask || a.mask[r];
    char* out = static_cast<char*>(a.dlogits) + r * a.ldd * (int64_t)sizeof(typename Row<T>::type);
    float v[NI][4] = {};
    if (in) {
      const char* row = static_cast<const char*>(a.logits) + r * a.ld * (int64_t)sizeof(typename Row<T>::type);
#pragma unroll
      for (int i = 0; i < NI; ++i) logits4<T>(row, (i * G + g) * 4, a.experts, v[i]);
      const float lse = softmax<G, NI>(v);
      float dot = 0.f;
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) dot += f[i][e] * v[i][e];
      dot = over<G>(dot, add);
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) v[i][e] *= (gb * (f[i][e] - dot) + gz * lse) / n;
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) put4<T>(out, (i * G + g) * 4, a.experts, v[i]);
  }
}

// --------------------------------------------------------------- launchers
static int balance_parts(int rows) {
  if (rows <= BAL_ONE) return 1;
  return (rows + 31) / 32 < BAL_PARTS ? (rows + 31) / 32 : BAL_PARTS;
}
int64_t balance_part_words(int rows, int experts) { return balance_parts(rows) * Part(experts).words; }

template <int T, int G, int NI> static hipError_t fwd(const BalanceArgs& a, hipStream_t s) {
  const int parts = balance_parts(a.rows);
  hipLaunchKernelGGL((k_balance<T, G, NI>), dim3(parts), dim3(BAL_WG), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || parts == 1) return e;
  hipLaunchKernelGGL(k_balance_join, dim3(1), dim3(BAL_WG), 0, s, a, parts);
  return hipGetLastError();
}
template <int T, int G, int NI> static hipError_t bwd(const BalanceArgs& a, hipStream_t s) {
  const int64_t wgs = ((int64_t)a.rows + 256 / G - 1) / (256 / G);
  hipLaunchKernelGGL((k_balance_grad<T, G, NI>), dim3((uint32_t)(wgs < 2048 ? wgs : 2048)), dim3(256), 0, s, a);
  return hipGetLastError();
}
template <int T> static hipError_t pick(const BalanceArgs& a, bool grad, hipStream_t s) {
  if (a.experts <= 64) return grad ? bwd<T, 16, 1>(a, s) : fwd<T, 16, 1>(a, s);
  if (a.experts <= 128) return grad ? bwd<T, 16, 2>(a, s) : fwd<T, 16, 2>(a, s);
  if (a.experts <= 256) return grad ? bwd<T, 16, 4>(a, s) : fwd<T, 16, 4>(a, s);
  if (a.experts <= 1024) return grad ? bwd<T, 64, 4>(a, s) : fwd<T, 64, 4>(a, s);
  return hipErrorInvalidValue;
}
static hipError_t run(int dt, const BalanceArgs& a, bool grad, hipStream_t s) {
  if (dt == DT_BF16) return pick<DT_BF16>(a, grad, s);
  if (dt == DT_F16) return pick<DT_F16>(a, grad, s);
  if (dt == DT_F32) return pick<DT_F32>(a, grad, s);
  return hipErrorInvalidValue;
}
hipError_t launch_balance(int dt, const BalanceArgs& a, hipStream_t s) { return run(dt, a, false, s); }
hipError_t launch_balance_grad(int dt, const BalanceArgs& a, hipStream_t s) { return run(dt, a, true, s); }

}  // namespace moe

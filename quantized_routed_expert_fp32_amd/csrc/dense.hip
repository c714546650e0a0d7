// Dense feed-forward products beside the routed experts: the gated block
//   g = x Wg^T, u = x Wu^T, h = act(g) u
// in 16 bits, its gradients
//   dg = dh u act'(g), du = dh act(g),
//   dx = dg Wg + du Wu (one contraction over [dg | du]), dWg = dg^T x, dWu = du^T x,
// and products of 8-bit integers with a scale per token and per channel, which
// the gated block takes too.
//
//  * k_dense: all of the products for more than 16 rows, on four workgroup
//    tiles (dense_tile picks one and, for few tiles, a number of K ranges).
//  * k_dense_decode: up to 16 rows, the weights straight from memory into
//    16x16 matrix instructions, one launch.
//  * k_quant_rows (rows to 8 bits), k_glu_grad (dg and du; k_glu_top before it
//    in fp16), k_dense_pad (rows the tiles cannot read in place), k_dense_join
//    (K ranges): one pass over memory each.
// Sums are fp32 (int32 for 8-bit operands, exact), in a fixed order. Rounded
// to 16 bits: the outputs, and dg and du, because the matrix instructions of
// their two products take 16-bit operands (up to 32 rows they go as a high and
// a low part, in tile rows that would be idle); g and u are kept in fp32 for the
// gradients (kept in 16 bits they cost dx and dW as much error again as dg,
// du and the outputs together: 3.1e-3 of their norm in bf16 against 2.4e-3,
// where rounding the outputs alone is 1.7e-3).
//
// What bounds the large products is the card's power, and waits: on normal data
// 16x16 matrix instructions alone run 2.02 PFLOP/s bf16 and 4.26 POP/s 8-bit, the
// 32x32 ones 1.75 and 3.55 (zeros: 2.44 and 4.87 both), which is why every
// product here is 16x16; in the products the matrix units are busy 55 to 67% of
// the cycles, on zeros as on normal data, at a clock of 1.9 to 2.0 GHz on the
// latter. Medians of 23 launches on one card (least in parentheses): the 8192 x
// 4096 x 8192 training step's three products 931 (890), 877 (838) and 922 (882)
// us, 1.18 to 1.31 PFLOP/s, 8192 x 4096 -> 8192 8-bit 283 (237) us, 1.95 to 2.32
// POP/s; on another card, least, 826, 766, 794 and 227. Leaving the loads into
// LDS out of the loop would take 17% off, leaving zeros in the operands 30%. A
// library's products of the same shapes take 832, 916 and 1030 us; its largest
// 8-bit ones run at 2.1 to 2.3 POP/s.
#include "dense_launch.h"

#include <algorithm>
#include <atomic>

namespace moe {

typedef _Float16 f16;
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef f16 f16x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// ------------------------------------------------------------ element types
template <int T> struct Elem;
template <> struct Elem<DT_BF16> {
  typedef f32x4 acc4;
  static constexpr int SIZE = 2;
  static __device__ __forceinline__ acc4 mma16(u32x4 p, u32x4 q, acc4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, p), __builtin_bit_cast(bf16x8, q), c,
                                                   0, 0, 0);
  }
};
template <> struct Elem<DT_F16> {
  typedef f32x4 acc4;
  static constexpr int SIZE = 2;
  static __device__ __forceinline__ acc4 mma16(u32x4 p, u32x4 q, acc4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, p), __builtin_bit_cast(f16x8, q), c, 0,
                                                  0, 0);
  }
};
template <> struct Elem<DT_I8> {
  typedef i32x4 acc4;
  static constexpr int SIZE = 1;
  static __device__ __forceinline__ acc4 mma16(u32x4 p, u32x4 q, acc4 c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, p), __builtin_bit_cast(i32x4, q), c, 0, 0,
                                                 0);
  }
};

// ------------------------------------------------------------- activations
// silu(g) = g s(g); gelu_tanh(g) = g s(w(g)) with w = 2 sqrt(2/pi) (g +
// 0.044715 g^3), since (1 + tanh(w/2)) / 2 = s(w): one sigmoid for both.
constexpr float GELU_C = 1.5957691216057308f;
// v_rcp_f32 and v_exp_f32 are good to one ulp. Below w = FAR the sigmoid is e^w to
// fp32 and soon subnormal, or its inverse infinite, where g e^w still counts: there
// t = e^(w / 2) goes in twice, on either side of the rounding. act_n and act_grad_n
// look once at all of a wave's gates (a minimum a gate; in place of the plain form
// everywhere it would cost 2048 x 2048 -> 2 x 8192 2%, 8-bit 4%; so, 0 to 2%).
constexpr float FAR = -80.f;
__device__ __forceinline__ float act_arg(float g, int act) {
  return act == ACT_SILU ? g : GELU_C * g * (1.f + 0.044715f * g * g);
}
__device__ __forceinline__ float act_slope(float g, int act) {
  return act == ACT_SILU ? 1.f : GELU_C * (1.f + 0.134145f * g * g);
}
__device__ __forceinline__ float sigmoid_f(float w) { return __builtin_amdgcn_rcpf(1.f + __expf(-w)); }
template <int N> __device__ __forceinline__ void act_n(const float* g, int act, float* v) {
  float low = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float w = act_arg(g[i], act);
    v[i] = g[i] * sigmoid_f(w);
    low = __builtin_fminf(low, w);
  }
  if (__any(low < FAR))
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float w = act_arg(g[i], act), t = __expf(0.5f * w);
      if (w < FAR) v[i] = (g[i] * t) * t;
    }
}
// Values and derivatives: p + g p (1 - p) w'; where p (1 - p) is zero the
// second term is (w' may overflow there)
template <int N> __device__ __forceinline__ void act_grad_n(const float* g, int act, float* v, float* d) {
  float low = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float w = act_arg(g[i], act), p = sigmoid_f(w), pp = p * sigmoid_f(-w);
    v[i] = g[i] * p;
    d[i] = p + (pp > 0.f ? g[i] * pp * act_slope(g[i], act) : 0.f * pp);
    low = __builtin_fminf(low, w);
  }
  if (__any(low < FAR))
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float w = act_arg(g[i], act), t = __expf(0.5f * w);
      if (w < FAR) {
        v[i] = (g[i] * t) * t;
        d[i] = t > 0.f ? ((1.f + g[i] * act_slope(g[i], act)) * t) * t : 0.f;
      }
    }
}

// ------------------------------------------------------------------ stores
template <int T> __device__ __forceinline__ uint16_t to16(float v) {
  if constexpr (T == DT_BF16) return __builtin_bit_cast(uint16_t, (__bf16)v);
  else return __builtin_bit_cast(uint16_t, (f16)v);
}
__device__ __forceinline__ uint16_t to16_rt(float v, int dt) {
  return dt == DT_BF16 ? to16<DT_BF16>(v) : to16<DT_F16>(v);
}
// four consecutive outputs of a row, the first at column p of np (global
// stores take any alignment)
__device__ __forceinline__ void store4(void* row, int p, int np, int dt, const float* v) {
  if (dt == DT_F32) {
    float* o = static_cast<float*>(row) + p;
    if (p + 4 <= np) __builtin_memcpy(o, v, 16);
    else
      for (int i = 0; i < 4; ++i)
        if (p + i < np) o[i] = v[i];
    return;
  }
  uint16_t* o = static_cast<uint16_t*>(row) + p;
  uint16_t b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) b[i] = to16_rt(v[i], dt);
  if (p + 4 <= np) __builtin_memcpy(o, b, 8);
  else
    for (int i = 0; i < 4; ++i)
      if (p + i < np) o[i] = b[i];
}
// row q of the product's output, or null when q is padding between the two
__device__ __forceinline__ char* out_row(const DenseArgs& a, int q) {
  if (!a.qpad || q < a.qseg) return static_cast<char*>(a.out0) + q * a.ldo * 2;
  if (q >= a.qpad && q < a.qpad + a.qseg) return static_cast<char*>(a.out1) + (q - a.qpad) * a.ldo * 2;
  return nullptr;
}
// sum * (q * p) of two scales whose product may leave fp32's range where the
// result does not (2^-70 squared, or infinity times a sum of zero): mantissas
// and exponents apart, the same bits as the plain products wherever those stay
// normal numbers. NaN and infinity are their own mantissas.
struct Scale {
  float m;
  int e;
  __device__ __forceinline__ explicit Scale(float s)
      : m(__builtin_amdgcn_frexp_mantf(s)), e(__builtin_amdgcn_frexp_expf(s)) {}
};
__device__ __forceinline__ float scaled(float sum, Scale q, Scale p) {
  return __builtin_amdgcn_ldexpf(sum * (q.m * p.m), q.e + p.e);
}
// What a gradient's sums are multiplied by: fp16 operands carry a power of two (see k_glu_top)
template <int T> __device__ __forceinline__ float grad_down(const DenseArgs& a) {
  if constexpr (T == DT_F16) return *a.down;
  else return 1.f;
}
// The epilogues on four consecutive columns p.. of row q. `s0` and `s1` are
// the sums (gate and up for GLU) as fp32 or int32, `sq` the row's scale.
template <int T, int EPI, typename V>
__device__ __forceinline__ void finish4(const DenseArgs& a, int q, int p, const V* s0, const V* s1, float sq) {
  if (q >= a.nq || p >= a.np) return;
  float v[4], g[4], u[4];
  if constexpr (EPI == EPI_GLU) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (T == DT_I8) {
        const int pi = min(p + i, a.np - 1);
        g[i] = scaled((float)s0[i], Scale(sq), Scale(a.sp0[pi]));
        u[i] = scaled((float)s1[i], Scale(sq), Scale(a.sp1[pi]));
      } else {
        g[i] = s0[i];
        u[i] = s1[i];
      }
    }
    act_n<4>(g, a.act, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] *= u[i];
    if (a.save) {
      float* sv = static_cast<float*>(a.save) + (int64_t)q * 2 * a.np;
      store4(sv, p, a.np, DT_F32, g);
      store4(sv + a.np, p, a.np, DT_F32, u);
    }
  } else if constexpr (EPI == EPI_SCALE) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int pi = min(p + i, a.np - 1);
      v[i] = scaled((float)s0[i], Scale(sq), Scale(a.sp0[pi])) + (a.bias ? a.bias[pi] : 0.f);
    }
  } else {
    const float down = grad_down<T>(a);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = s0[i] * down;
  }
  char* row = out_row(a, q);
  if (row) store4(row, p, a.np, a.out_dt, v);
}

// ------------------------------------------------------- loads into the ring
// A wave-uniform address, in scalar registers.
__device__ __forceinline__ const uint8_t* uniform(const uint8_t* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return reinterpret_cast<const uint8_t*>((uint64_t)hi << 32 | lo);
}
// 64 x 16 bytes from base + off (a lane's own) to LDS [lds, lds + 1024). In
// asm, because the compiler would guard every LDS read against the loads in
// flight by waiting for all of them; it has no register outputs, and reads of
// what it writes are ordered by step_wait. Nor does the compiler look for hazards
// in here: m0 needs its one wait state, and a base that a vector instruction
// wrote (a readlane) would need five. The kernels as built compute every base in
// scalar registers, which a test checks (s_nop 3 in place of s_nop 0 would cover
// it too, and costs the 512 x 2048 -> 2 x 512 forward 5%, the large ones 1%).
__device__ __forceinline__ void dma16(uint32_t lds, uint32_t off, const uint8_t* base) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off), "s"(base)
               : "m0");
}
// the same with a whole address per lane (the last step's masked loads)
__device__ __forceinline__ void dma16_at(uint32_t lds, const uint8_t* src) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(src) : "m0");
}
// the wave's own loads but the newest N have landed, its LDS reads are done;
// then every wave's
template <int N> __device__ __forceinline__ void step_wait() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// 16 zero bytes: what a masked load reads (K behind the operand's end)
__device__ const u32x4 g_zero16 = {0, 0, 0, 0};

// ---------------------------------------------------------------- the product
// Workgroup tile BP x BQ of WP x WQ waves; a K step is KB bytes of a
// k-contiguous row (KB / 2 k of 16 bits). Both operands go from memory straight
// into an LDS ring. k-contiguous operand: rows of KB bytes, 16-byte chunk c of
// row r at position c ^ (r & 7), so the rows that are read together meet
// different banks. k-major operand (the gradients' weights and activations,
// never transposed in memory): rows k of 2 B bytes, 32-byte segment s at s ^
// swz_km(k), so the 4 rows of a transposed read do. Counted at 8192 x 4096 x
// 8192: 1 to 4% of the LDS cycles are conflicts, LDS is busy 27% of the time,
// the matrix units 64 to 67%, the L2 serves 77 to 81% of the loads (a band of 4
// x 8 tiles an XCD: 12 operand tiles for 32 workgroups' 64).
//
// 256 x 256, 8 waves of 64 x 128: 128 accumulators, 2 waves a SIMD to cover
// each other's waits (4 waves of 128 x 128 read a third less LDS but spill: 1398
// us against 940 for the 8192 x 4096 -> 2 x 8192 forward); its epilogue is
// alone on the CU (160 KiB of LDS), 5 us a tile. The smaller tiles fill the CUs
// when there are few rows and are bound by a step's latency (barrier, LDS
// reads); 8 waves on 128 x 128 take 15% off 4, and two k blocks a unit in
// 256-byte steps 20 to 30% off one in 128-byte steps on 64 x 64.
template <int T, int EPI, int FORM, int BP, int BQ, int WP, int WQ, int R, int KB, int KU>
struct Dense {
  static constexpr int RPM = 1;                    // fragment reads a product
  static constexpr bool PKM = FORM != FORM_NT, QKM = FORM == FORM_TN;
  static constexpr int NW = WP * WQ;
  static constexpr int TP = BP / WP, TQ = BQ / WQ, FP = TP / 16, FQ = TQ / 16;
  static constexpr int PB = BP * KB, QB = BQ * KB, UNIT = PB > QB ? PB : QB;   // R ring slots of UNIT bytes
  static constexpr int LP = PB / (NW * 1024), LQ = QB / (NW * 1024);
  static constexpr int NK = KB / 64;               // matrix-instruction k blocks of a step
  static constexpr int QH = KU == 1 && FQ > 2 ? FQ / 2 : 1, QG = FQ / QH, NU = NK / KU * QH;   // units: KU k blocks, QG Q fragments
  static constexpr int CPR = KB / 16, KR = KB / 2;  // chunks of a k-contiguous row; k rows of a step
  typedef typename Elem<T>::acc4 acc_t;
  static_assert(NK / KU % 2 == 0 && NK % KU == 0 && QG * QH == FQ, "units");
  static_assert(LP * NW * 1024 == PB && LQ * NW * 1024 == QB && LP == LQ, "whole loads");
  static_assert(R % 2 == 1 && R >= 5, "ring");

  static __device__ __forceinline__ int swz_kc(int r) { return r & 7; }
  // the same for k and k + 4
  template <int B> static __device__ __forceinline__ int swz_km(int k) {
    return ((k & 3) | ((k >> 3) & 1) << 2) & (B / 16 - 1);
  }
  // whether load i of wave w holds up rows (GLU: rows interleaved 32 gate, 32 up)
  static __device__ __forceinline__ bool is_up(int i, int w) {
    return EPI == EPI_GLU && (((i * NW + w) * (64 / CPR)) >> 5 & 1);
  }
  // source offset of load i of a lane, k-contiguous rows clamped below n
  template <bool KM, int B, int L, bool GLU>
  static __device__ __forceinline__ void offsets(uint32_t* off, int w, int lane, int c0, int n, int64_t ld0, int64_t ld1) {
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const int q = (i * NW + w) * 64 + lane;
      const uint32_t ld = (uint32_t)(GLU && is_up(i, w) ? ld1 : ld0);
      if constexpr (!KM) {
        const int r = q / CPR;
        const int c = (q % CPR) ^ swz_kc(r);
        const int idx = GLU ? c0 + (r >> 6) * 32 + (r & 31) : c0 + r;
        off[i] = (uint32_t)(min(idx, n - 1) - c0) * ld + c * 16;
      } else {
        constexpr int RC = B * 2 / 16;                 // chunks of a k row
        const int k = q / RC, pos = q % RC;
        const int s = (pos >> 1) ^ swz_km<B>(k);
        const int col = c0 + (s * 2 + (pos & 1)) * 8;
        off[i] = (uint32_t)k * ld + (uint32_t)(min(col, (n - 1) & ~7) - c0) * 2;
      }
    }
  }

  // a lane's 16 bytes of row `row`, k block kk: chunk 4 kk + lane / 16
  static __device__ __forceinline__ u32x4 frag_kc(const uint8_t* tile, int row, int kk, int quad) {
    return *reinterpret_cast<const u32x4*>(tile + row * KB + (((kk * 4 + quad) ^ swz_kc(row)) << 4));
  }
  // k-major: the lane's 8 k of column col0 + lane % 16: two 4-row transposed
  // reads; a 16-lane group reads 4 rows of 16 columns, lane i supplying the
  // address of row i / 4, columns 4 (i % 4).. and getting column i's 4 rows
  template <int B>
  static __device__ __forceinline__ u32x4 frag_km(const uint8_t* tile, int col0, int kk, int lane) {
    const int i = lane & 15, g = lane >> 4;
    const int k = kk * 32 + g * 8 + (i >> 2);
    const uint8_t* ad = tile + k * (B * 2) + ((((col0 >> 4) ^ swz_km<B>(k)) << 5) | ((i & 3) << 3));
    typedef __attribute__((address_space(3))) i16x4* lp;
    const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(ad));
    const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(ad + 4 * (B * 2)));
    const uint2 a = __builtin_bit_cast(uint2, lo), b = __builtin_bit_cast(uint2, hi);
    return u32x4{a.x, a.y, b.x, b.y};
  }

  static __device__ __forceinline__ void run(const DenseArgs& a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wp = w % WP, wq = w / WP;
    constexpr int OP = EPI == EPI_GLU ? BP / 2 : BP;    // output columns of a tile
    const int tp = (a.np + OP - 1) / OP, tq = (a.nq + BQ - 1) / BQ;
    // workgroup i runs on XCD i mod 8: each XCD takes a contiguous run of
    // tiles, in bands of GQ tile rows, so that its L2 serves both operands
    int id = blockIdx.x;
    const int tiles = tp * tq;
    {
      const int x = id & 7, j = id >> 3, per = tiles >> 3, rem = tiles & 7;
      id = x * per + min(x, rem) + j;
    }
    constexpr int GQ = 4;
    const int band = id / (GQ * tp), inb = id % (GQ * tp);
    const int gh = min(GQ, tq - band * GQ);
    // (uniform, but a division leaves its result in a vector register)
    const int iq = __builtin_amdgcn_readfirstlane(band * GQ + inb % gh), ip = __builtin_amdgcn_readfirstlane(inb / gh);
    const int c0p = ip * OP, c0q = iq * BQ;
    // K steps that lie whole inside the operands, this workgroup's range of
    // them, and the masked rest (up to one step a segment), which the last
    // range takes. NN: two segments of P rows, gate then up.
    const int z = blockIdx.y;
    const int nws = PKM ? a.krows / KR : a.kbytes / KB;
    const bool rest = PKM ? a.krows % KR != 0 : a.kbytes % KB != 0;
    constexpr int NSEG = FORM == FORM_NN ? 2 : 1;
    const int t0 = __builtin_amdgcn_readfirstlane((int)((int64_t)NSEG * nws * z / a.splits));
    const int t1 = __builtin_amdgcn_readfirstlane((int)((int64_t)NSEG * nws * (z + 1) / a.splits));

    uint32_t offp[LP], offq[LQ];
    offsets<PKM, BP, LP, EPI == EPI_GLU>(offp, w, lane, c0p, a.np, a.ldp0, a.ldp1);
    offsets<QKM, BQ, LQ, false>(offq, w, lane, c0q, a.nq, a.ldq, a.ldq);
    // NN's second segment counts its offsets in its own stride
    uint32_t offp1[FORM == FORM_NN ? LP : 1];
    if constexpr (FORM == FORM_NN) offsets<PKM, BP, LP, false>(offp1, w, lane, c0p, a.np, a.ldp1, a.ldp1);
    const uint8_t* pb0 = a.p0 + (PKM ? (int64_t)c0p * 2 : (int64_t)c0p * a.ldp0);
    const uint8_t* pb1 = a.p1 ? a.p1 + (PKM ? (int64_t)c0p * 2 : (int64_t)c0p * a.ldp1) : nullptr;
    // GLU: the operand each load of this wave reads
    const uint8_t* pbn[LP];
#pragma unroll
    for (int i = 0; i < LP; ++i) pbn[i] = uniform(is_up(i, w) ? pb1 : pb0);
    const uint8_t* qb = a.q0 + (QKM ? (int64_t)c0q * 2 : (int64_t)c0q * a.ldq);
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(
        (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)smem);
    const uint8_t* const zero = reinterpret_cast<const uint8_t*>(&g_zero16);

    // load n of a step's P or Q half into ring slot `slot`: step t of segment sg
    struct Src {
      const uint8_t* b;
      uint32_t lds;
      bool second;
    };
    auto source_p = [&](int sg, int t, int slot) {
      Src r;
      r.lds = lds0 + slot * UNIT + w * 1024;
      r.second = sg;
      r.b = (EPI == EPI_GLU ? nullptr : sg ? pb1 : pb0) +
            (PKM ? (int64_t)t * KR * (sg ? a.ldp1 : a.ldp0) : (int64_t)t * KB);
      return r;
    };
    auto source_q = [&](int sg, int t, int slot) {
      Src r;
      r.lds = lds0 + slot * UNIT + w * 1024;
      r.second = sg;
      r.b = qb + (QKM ? (int64_t)t * KR * a.ldq : (int64_t)t * KB + (sg ? a.segbytes : 0));
      return r;
    };
    auto seg_of = [&](int t) { return NSEG == 2 && t >= nws ? 1 : 0; };
    auto src = [&](bool isp, int t, int slot) {
      const int sg = seg_of(t);
      return isp ? source_p(sg, sg ? t - nws : t, slot) : source_q(sg, sg ? t - nws : t, slot);
    };
    auto base_p = [&](const Src& r, int n) -> const uint8_t* {
      return EPI == EPI_GLU ? pbn[n] + reinterpret_cast<intptr_t>(r.b) : r.b;
    };
    auto off_p = [&](const Src& r, int n) {
      if constexpr (FORM == FORM_NN) return r.second ? offp1[n] : offp[n];
      else return offp[n];
    };
    auto load_p = [&](const Src& r, int n) { dma16(r.lds + n * NW * 1024, off_p(r, n), uniform(base_p(r, n))); };
    auto load_q = [&](const Src& r, int n) { dma16(r.lds + n * NW * 1024, offq[n], uniform(r.b)); };
    // the step behind segment sg's whole ones into slots 0 and 1, zero past the operands' end
    auto load_rest = [&](int sg) {
      const Src rp = source_p(sg, nws, 0), rq = source_q(sg, nws, 1);
      const int kr = a.krows - nws * KR;
      const int kb = (NSEG == 1 ? a.kbytes : sg ? a.kbytes - a.segbytes : a.segbytes) - nws * KB;
#pragma unroll
      for (int n = 0; n < LP; ++n) {
        const int q = (n * NW + w) * 64 + lane;
        const bool inp = PKM ? q / (BP * 2 / 16) < kr : ((q % CPR) ^ swz_kc(q / CPR)) * 16 < kb;
        const bool inq = QKM ? q / (BQ * 2 / 16) < kr : ((q % CPR) ^ swz_kc(q / CPR)) * 16 < kb;
        dma16_at(rp.lds + n * NW * 1024, inp ? base_p(rp, n) + off_p(rp, n) : zero);
        dma16_at(rq.lds + n * NW * 1024, inq ? rq.b + offq[n] : zero);
      }
    };

    acc_t acc[FP][FQ];
#pragma unroll
    for (int i = 0; i < FP; ++i)
#pragma unroll
      for (int j = 0; j < FQ; ++j) acc[i][j] = acc_t{};

    // A unit is KU k blocks (64 bytes of k each) and QG of the wave's Q fragments.
    const int col = lane & 15, quad = lane >> 4;
    u32x4 fp[2][KU][FP], fq[2][KU][QG];
    auto frag_p = [&](int sp, int u, int kb, int i) {
      const uint8_t* pt = smem + sp * UNIT;
      const int kk = u / QH * KU + kb;
      if constexpr (PKM) fp[u / QH & 1][kb][i] = frag_km<BP>(pt, wp * TP + i * 16, kk, lane);
      else fp[u / QH & 1][kb][i] = frag_kc(pt, wp * TP + i * 16 + col, kk, quad);
    };
    auto frag_q = [&](int sq, int u, int kb, int j) {
      const uint8_t* qt = smem + sq * UNIT;
      const int kk = u / QH * KU + kb, jj = u % QH * QG + j;
      if constexpr (QKM) fq[u & 1][kb][j] = frag_km<BQ>(qt, wq * TQ + jj * 16, kk, lane);
      else fq[u & 1][kb][j] = frag_kc(qt, wq * TQ + jj * 16 + col, kk, quad);
    };
    // read x of unit u, in the order its products need them: a k block's P 0,
    // its Qs, its other Ps
    auto frag1 = [&](int sp, int sq, int u, int x) {
      if (u % QH != 0) {
        frag_q(sq, u, x / QG, x % QG);
      } else {
        const int kb = x / (FP + QG), y = x % (FP + QG);
        if (y == 0 || y > QG) frag_p(sp, u, kb, y == 0 ? 0 : y - QG);
        else frag_q(sq, u, kb, y - 1);
      }
    };
    constexpr int NM = KU * FP * QG;
    auto reads = [](int u) { return KU * (u % QH ? QG : FP + QG); };
    auto mma1 = [&](int u, int n) {
      const int kb = n / (FP * QG), i = n / QG % FP, j = n % QG;
      acc_t& c = acc[i][u % QH * QG + j];
      c = Elem<T>::mma16(fp[u / QH & 1][kb][i], fq[u & 1][kb][j], c);
    };

    // Ring of R slots, a step's P and Q halves in turn: half 2 t (P) and 2 t + 1
    // (Q) of step t in slots of their number mod R. Before a step's last unit
    // the wave waits for its own loads of the next step and for its LDS reads;
    // the barrier then makes the next step visible and tells that every wave
    // has read the whole of this one, whose two slots halves 2 t + R (a Q) and
    // 2 t + R + 1 (a P) refill: the Q loads go out between that unit's matrix
    // instructions, the P loads (needed a step later) between those of the next
    // step's units. An odd R keeps half a step more in flight than whole stages
    // in the same memory. The fragments of a unit are read between the products
    // of the one before it; the scheduling barriers keep that order.
    const int halves = 2 * (t1 - t0);
    if (t0 < t1) {
#pragma unroll
      for (int h = 0; h < R; ++h)
        if (h < halves) {
          const Src r = src(h % 2 == 0, t0 + h / 2, h);
#pragma unroll
          for (int n = 0; n < LP; ++n) {
            if (h % 2 == 0) load_p(r, n);
            else load_q(r, n);
          }
        }
      if (halves >= R) step_wait<(R - 2) * LP>();
      else step_wait<0>();
#pragma unroll
      for (int x = 0; x < reads(0); ++x) frag1(0, 1, 0, x);
      // opaque, or the compiler merges these reads with the loop's own
#pragma unroll
      for (int kb = 0; kb < KU; ++kb) {
#pragma unroll
        for (int i = 0; i < FP; ++i) asm volatile("" : "+v"(fp[0][kb][i]));
#pragma unroll
        for (int j = 0; j < QG; ++j) asm volatile("" : "+v"(fq[0][kb][j]));
      }
      int sp = 0, sq = 1;
      Src rp = src(true, t0, 0);
      bool more_p = false;
      for (int t = t0; t < t1; ++t) {
        const int sp1 = sp + 2 >= R ? sp + 2 - R : sp + 2, sq1 = sq + 2 >= R ? sq + 2 - R : sq + 2;
        // unit u's products, between them the reads of unit v of the step in
        // slots fsp, fsq, and some of the loads
        auto unit = [&](int u, int fsp, int fsq, int v, auto loads) {
          const int nf = reads(v);
#pragma unroll
          for (int n = 0; n < NM; ++n) {
            mma1(u, n);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int x = n * RPM; x < (n + 1 == NM ? nf : min((n + 1) * RPM, nf)); ++x) frag1(fsp, fsq, v, x);
            loads(n);
            __builtin_amdgcn_sched_barrier(0);
          }
        };
        constexpr int PHN = (NU - 1) * NM;      // products the P loads spread over
#pragma unroll
        for (int u = 0; u + 1 < NU; ++u)
          unit(u, sp, sq, u + 1, [&](int n) {
            const int m = u * NM + n;
            if (m * LP / PHN != (m + 1) * LP / PHN && more_p) {
#pragma unroll
              for (int l = m * LP / PHN; l < (m + 1) * LP / PHN; ++l) load_p(rp, l);
            }
          });
        const int rel = 2 * (t - t0);
        if (rel + R <= halves) step_wait<(R - 4) * LP>();
        else step_wait<0>();
        const bool more_q = rel + R < halves;
        const Src rq = src(false, t + R / 2, sp);
        more_p = rel + R + 1 < halves;
        rp = src(true, t + R / 2 + 1, sq);
        unit(NU - 1, sp1, sq1, 0, [&](int n) {
          if (n * LQ / NM != (n + 1) * LQ / NM && more_q) {
#pragma unroll
            for (int l = n * LQ / NM; l < (n + 1) * LQ / NM; ++l) load_q(rq, l);
          }
        });
        sp = sp1;
        sq = sq1;
      }
      step_wait<0>();
    }
    if (rest && z == a.splits - 1) {
#pragma unroll 1
      for (int sg = 0; sg < NSEG; ++sg) {
        load_rest(sg);
        step_wait<0>();
#pragma unroll
        for (int u = 0; u < NU; ++u) {
#pragma unroll
          for (int x = 0; x < reads(u); ++x) frag1(0, 1, u, x);
#pragma unroll
          for (int n = 0; n < NM; ++n) mma1(u, n);
        }
        step_wait<0>();
      }
    }

    epilogue(a, acc, smem + w * (R * UNIT / NW / 16 * 16), lane, c0p + (EPI == EPI_GLU ? wp * (TP / 2) : wp * TP),
             c0q + wq * TQ, z);
  }

  // 16 rows of COLS elements of ES bytes, staged by the wave in LDS (rows
  // padded by 16 bytes), to memory: 16 bytes a lane, whole rows, so that a
  // store covers 64-byte runs and more (straight from the accumulators it
  // would be 32 bytes of 16 rows)
  template <int ES, int COLS> static constexpr int row_bytes() { return COLS * ES + 16; }
  template <int ES, int COLS, typename RowOf>
  static __device__ __forceinline__ void flush(const uint8_t* buf, int lane, int q0, int nq, int p0, int np,
                                               RowOf row) {
    constexpr int CH = COLS * ES / 16, N = 16 / ES;
    asm volatile("" ::: "memory");     // other lanes' writes: LDS runs in order
#pragma unroll
    for (int it = 0; it < (16 * CH + 63) / 64; ++it) {
      const int r = (it * 64 + lane) / CH, c = (it * 64 + lane) % CH;
      if (16 * CH % 64 && r >= 16) continue;
      const u32x4 v = *reinterpret_cast<const u32x4*>(buf + r * row_bytes<ES, COLS>() + c * 16);
      const int q = q0 + r, p = p0 + c * N;
      if (q >= nq || p >= np) continue;
      char* o = row(q);
      if (!o) continue;
      o += (int64_t)p * ES;
      if (p + N <= np) __builtin_memcpy(o, &v, 16);      // at any alignment
      else
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (p + e < np) {
            if constexpr (ES == 4) reinterpret_cast<uint32_t*>(o)[e] = v[e];
            else reinterpret_cast<uint16_t*>(o)[e] = (uint16_t)(v[e / 2] >> (16 * (e & 1)));
          }
    }
    asm volatile("" ::: "memory");
  }
  template <int DT> static __device__ __forceinline__ void put4(uint8_t* at, const float* v) {
    if constexpr (DT == DT_F32) *reinterpret_cast<f32x4*>(at) = f32x4{v[0], v[1], v[2], v[3]};
    else
      *reinterpret_cast<uint2*>(at) = make_uint2(to16<DT>(v[0]) | (uint32_t)to16<DT>(v[1]) << 16,
                                                 to16<DT>(v[2]) | (uint32_t)to16<DT>(v[3]) << 16);
  }

  // The wave's TP x TQ part of the tile: in acc[i][j] a lane holds column
  // q = q0 + 16 j + lane % 16, rows p = p0 + 16 i + 4 (lane / 16) + e (GLU: of
  // 4 fragments the first 2 are gate, the others up of the same 32 outputs).
  static __device__ __forceinline__ void epilogue(const DenseArgs& a, acc_t (&acc)[FP][FQ], uint8_t* buf, int lane,
                                                  int p0, int q0, int z) {
    constexpr bool GLU = EPI == EPI_GLU;
    constexpr int OC = GLU ? TP / 2 : TP;              // output columns of the wave
    constexpr int OG = OC / 16;                        // groups of 16
    const int col = lane & 15, quad = lane >> 4;
    auto gate = [](int g) { return GLU ? g / 2 * 4 + g % 2 : g; };
    // Pairs of Q rows (high and low parts): one output row each. Where the high
    // part's sum is not finite the low part's stays out: an infinite weight times
    // a low part of zero, or of the other sign, would turn infinity into NaN.
    const int fold = EPI == EPI_OUT && FORM == FORM_NN ? a.fold : 0, nq = fold ? fold : a.nq;
    const int js = fold ? FQ / 2 : FQ;
    if (fold) {
      q0 /= 2;
#pragma unroll
      for (int i = 0; i < FP; ++i)
#pragma unroll
        for (int j = 0; j < FQ / 2; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float hi = (float)acc[i][2 * j][e];
            acc[i][j][e] = __builtin_fabsf(hi) < __builtin_inff() ? hi + acc[i][2 * j + 1][e] : hi;
          }
    }
    if (a.splits > 1) {
      float* part = a.part + (int64_t)z * nq * a.pcols;
      const int lim = (int)(GLU ? a.pcols / 2 : a.pcols);
#pragma unroll
      for (int j = 0; j < FQ; ++j)
#pragma unroll
        for (int k = 0; k < (GLU ? 2 : 1); ++k) {
          if (j >= js) continue;
#pragma unroll
          for (int g = 0; g < OG; ++g)
            *reinterpret_cast<acc_t*>(buf + col * row_bytes<4, OC>() + (g * 16 + quad * 4) * 4) = acc[gate(g) + 2 * k][j];
          float* base = part + (k ? a.pcols / 2 : 0);
          flush<4, OC>(buf, lane, q0 + 16 * j, nq, p0, lim,
                       [&](int q) { return reinterpret_cast<char*>(base + (int64_t)q * a.pcols); });
        }
      return;
    }
    // the lane's column scales (and bias), all at once
    float sp0[T == DT_I8 ? OG : 1][4], sp1[T == DT_I8 ? OG : 1][4];
    int elo = 0, ehi = 0;                              // their exponents' range
    if constexpr (T == DT_I8) {
      const float* second = GLU ? a.sp1 : a.bias;
#pragma unroll
      for (int g = 0; g < OG; ++g)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int p = min(p0 + g * 16 + quad * 4 + e, a.np - 1);
          sp0[g][e] = a.sp0[p];
          sp1[g][e] = second ? second[p] : 0.f;
          elo = min(elo, min(Scale(sp0[g][e]).e, GLU ? Scale(sp1[g][e]).e : 0));
          ehi = max(ehi, max(Scale(sp0[g][e]).e, GLU ? Scale(sp1[g][e]).e : 0));
        }
    }
    const float down = EPI == EPI_OUT ? grad_down<T>(a) : 1.f;
#pragma unroll
    for (int j = 0; j < FQ; ++j) {
      if (j >= js) continue;
      const int q = q0 + 16 * j;
      float sq = 1.f;
      if constexpr (T == DT_I8) sq = a.sq[min(q + col, nq - 1)];
      float s0[OG][4], s1[OG][4];
#pragma unroll
      for (int g = 0; g < OG; ++g)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s0[g][e] = (float)acc[gate(g)][j][e];
          if constexpr (GLU) s1[g][e] = (float)acc[gate(g) + 2][j][e];
          if constexpr (EPI == EPI_OUT) s0[g][e] *= down;
        }
      if constexpr (T == DT_I8) {
        // the plain products where they are normal numbers for the whole wave
        // (`scaled` everywhere costs 4096 x 4096 -> 2 x 8192 1.5%, this nothing)
        const int eq = Scale(sq).e;
        if (__all(eq + elo >= -124 && eq + ehi <= 128)) {
#pragma unroll
          for (int g = 0; g < OG; ++g)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              s0[g][e] *= sq * sp0[g][e];
              if constexpr (GLU) s1[g][e] *= sq * sp1[g][e];
            }
        } else {
#pragma unroll
          for (int g = 0; g < OG; ++g)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              s0[g][e] = scaled(s0[g][e], Scale(sq), Scale(sp0[g][e]));
              if constexpr (GLU) s1[g][e] = scaled(s1[g][e], Scale(sq), Scale(sp1[g][e]));
            }
        }
        if constexpr (!GLU)
#pragma unroll
          for (int g = 0; g < OG; ++g)
#pragma unroll
            for (int e = 0; e < 4; ++e) s0[g][e] += sp1[g][e];
      }
      if constexpr (GLU && T != DT_I8) {
        if (a.save) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
#pragma unroll
            for (int g = 0; g < OG; ++g)
              put4<DT_F32>(buf + col * row_bytes<4, OC>() + (g * 16 + quad * 4) * 4, k ? s1[g] : s0[g]);
            float* base = static_cast<float*>(a.save) + k * a.np;
            flush<4, OC>(buf, lane, q, nq, p0, a.np,
                         [&](int qq) { return reinterpret_cast<char*>(base + (int64_t)qq * 2 * a.np); });
          }
        }
      }
      if constexpr (GLU) {
        float v[OG][4];
        act_n<OG * 4>(&s0[0][0], a.act, &v[0][0]);
#pragma unroll
        for (int g = 0; g < OG; ++g)
#pragma unroll
          for (int e = 0; e < 4; ++e) s0[g][e] = v[g][e] * s1[g][e];
      }
#pragma unroll
      for (int g = 0; g < OG; ++g) {
        uint8_t* at = buf + col * row_bytes<2, OC>() + (g * 16 + quad * 4) * 2;
        if (a.out_dt == DT_BF16) put4<DT_BF16>(at, s0[g]);
        else put4<DT_F16>(at, s0[g]);
      }
      flush<2, OC>(buf, lane, q, nq, p0, a.np, [&](int qq) { return out_row(a, qq); });
    }
  }
};

template <int T, int EPI, int FORM, int BP, int BQ, int WP, int WQ, int R, int KB, int KU>
__global__ __launch_bounds__(WP * WQ * 64) void k_dense(DenseArgs a) {
  Dense<T, EPI, FORM, BP, BQ, WP, WQ, R, KB, KU>::run(a);
}

// Joins the K ranges of a split product, range 0 first, and runs its epilogue.
template <int T, int EPI>
__global__ __launch_bounds__(256) void k_dense_join(DenseArgs a) {
  const int p = (blockIdx.y * 256 + threadIdx.x) * 4, q = blockIdx.x;
  if (p >= a.np) return;
  typedef typename Elem<T>::acc4 acc4;
  const int64_t stride = (int64_t)gridDim.x * a.pcols;
  const float* r0 = a.part + q * a.pcols + p;
  const float* r1 = r0 + (EPI == EPI_GLU ? a.pcols / 2 : 0);
  acc4 v0 = *reinterpret_cast<const acc4*>(r0), v1 = *reinterpret_cast<const acc4*>(r1);
  for (int z = 1; z < a.splits; ++z) {
    v0 += *reinterpret_cast<const acc4*>(r0 + z * stride);
    if constexpr (EPI == EPI_GLU) v1 += *reinterpret_cast<const acc4*>(r1 + z * stride);
  }
  decltype(v0[0] + 0) s0[4], s1[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    s0[e] = v0[e];
    s1[e] = v1[e];
  }
  finish4<T, EPI>(a, q, p, s0, s1, T == DT_I8 ? a.sq[q] : 1.f);
}

// -------------------------------------------------- rows at any alignment
// 16 bytes of a row from byte `byte` on, of elements of ES bytes, zero from
// byte `end` on. Global loads take any alignment. SHIFT: a chunk that passes the
// end is the row's last 16 bytes, shifted, instead of up to 15 loads (8-bit
// 333 x 1288 -> 776, both operands copied: 10.9 us for 11.6); the decode kernel
// has no registers left for it.
template <int ES, bool SHIFT = false>
__device__ __forceinline__ u32x4 load_chunk(const void* row, int64_t byte, int64_t end) {
  const uint8_t* at = static_cast<const uint8_t*>(row) + byte;
  u32x4 v = {0, 0, 0, 0};
  if (byte + 16 <= end) {
    __builtin_memcpy(&v, at, 16);
  } else if (SHIFT && end >= 16) {
    __builtin_memcpy(&v, static_cast<const uint8_t*>(row) + (end - 16), 16);
    const int n = (int)min(byte + 16 - end, (int64_t)16) * 8;
    uint64_t lo = v[0] | (uint64_t)v[1] << 32, hi = v[2] | (uint64_t)v[3] << 32;
    lo = n < 64 ? lo >> n | hi << 1 << (63 - n) : n < 128 ? hi >> (n - 64) : 0;
    hi = n < 64 ? hi >> n : 0;
    v = u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
  } else {
    uint8_t* b = reinterpret_cast<uint8_t*>(&v);
#pragma unroll
    for (int i = 0; i < 16; i += ES)
      if (byte + i < end) __builtin_memcpy(b + i, at + i, ES);
  }
  return v;
}

// Row r of the operands that are copied to zero-padded rows of 16-byte chunks,
// by a workgroup of 256 (a wave a row took 6.9 us for 2315 rows of 1283, bound by
// its own round trips). The copies ride in the grid of the kernel that has to run
// before the product anyway, where there is one: dx at 777 x 1283 x 769 fp16
// 26.4 us, 29.3 with a launch of their own.
template <int ES> __device__ __forceinline__ void pad_row(const DensePad& j, int r) {
  // Selects, not j.src[o]: an index known at run time moves j into scratch
  // (the copies of 777, 769 and 769 rows of 1283: 5 us, and 13 from scratch).
  const int r1 = r - j.rows[0], r2 = r1 - j.rows[1];
  const int64_t i = r2 >= 0 ? r2 : r1 >= 0 ? r1 : r;
  if (r2 >= j.rows[2]) return;
  const int64_t ld = r2 >= 0 ? j.ld[2] : r1 >= 0 ? j.ld[1] : j.ld[0];
  const uint8_t* src = static_cast<const uint8_t*>(r2 >= 0 ? j.src[2] : r1 >= 0 ? j.src[1] : j.src[0]) + i * ld * ES;
  u32x4* dst = reinterpret_cast<u32x4*>(static_cast<uint8_t*>(r2 >= 0 ? j.dst[2] : r1 >= 0 ? j.dst[1] : j.dst[0]) +
                                        i * j.ldd * ES);
  const int chunks = (int)(j.ldd * ES / 16);
  for (int c = threadIdx.x; c < chunks; c += 256)
    dst[c] = load_chunk<ES, true>(src, (int64_t)c * 16, (int64_t)j.cols * ES);
}

// The rows of x as the product with high and low parts of few rows takes them
// (see DensePairs), a workgroup a row: zero where the low parts meet an element
// that is not finite, whose product with the high part stands alone then
// (infinity times a low part of zero, or of the other sign, is NaN).
template <int DT> __device__ __forceinline__ void pair_row(const DensePairs& x, int r) {
  const int i = (r >> 5) * 16 + (r & 15);
  const bool low = r & 16;
  constexpr uint32_t EXP = DT == DT_BF16 ? 0x7F80 : 0x7C00;
  const uint8_t* src = static_cast<const uint8_t*>(x.src) + i * x.ld * 2;
  u32x4* dst = reinterpret_cast<u32x4*>(static_cast<uint8_t*>(x.dst) + r * x.ldd * 2);
  const int chunks = (int)(x.ldd * 2 / 16);
  for (int c = threadIdx.x; c < chunks; c += 256) {
    u32x4 v = {0, 0, 0, 0};
    if (i < x.rows) v = load_chunk<2, true>(src, (int64_t)c * 16, (int64_t)x.cols * 2);
    if (low)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if ((v[k] & EXP) == EXP) v[k] &= 0xFFFF0000u;
        if ((v[k] >> 16 & EXP) == EXP) v[k] &= 0xFFFFu;
      }
    dst[c] = v;
  }
}

// ---------------------------------------------------------------- quantising
template <int T> struct Row;
template <> struct Row<DT_BF16> {
  typedef uint16_t type;
  static __device__ __forceinline__ float f(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
};
template <> struct Row<DT_F16> {
  typedef uint16_t type;
  static __device__ __forceinline__ float f(uint16_t b) { return (float)__builtin_bit_cast(f16, b); }
};
template <> struct Row<DT_F32> {
  typedef float type;
  static __device__ __forceinline__ float f(float b) { return b; }
};

template <int T> __device__ __forceinline__ void unpack16(u32x4 v, float* f) {
  if constexpr (T == DT_F32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = Row<T>::f((uint16_t)v[i]);
      f[2 * i + 1] = Row<T>::f((uint16_t)(v[i] >> 16));
    }
  }
}

template <int DT> __device__ __forceinline__ u32x4 pack16(const float* f) {
  u32x4 v;
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = to16<DT>(f[2 * k]) | (uint32_t)to16<DT>(f[2 * k + 1]) << 16;
  return v;
}
// what rounding v to 16 bits leaves (nothing where that is not finite)
template <int DT> __device__ __forceinline__ float low_part(float v) {
  const float hi = Row<DT>::f(to16<DT>(v));
  return __builtin_fabsf(hi) < __builtin_inff() ? v - hi : 0.f;
}
// Scale of a row whose largest |x| has the bits m, and its codes: q =
// round-half-even of the exact x / s, |q| <= 127, 0 where s is not positive.
// The fp32 product with the reciprocal (off by less than 1.15e-5: 127 2^-24 from
// the reciprocal's rounding, 2^-18 from a product between 64 and 128) decides,
// four values at a time, unless one of them lies within 2e-5
// of a half-integer or the reciprocal overflows (a subnormal scale); then
// 53-bit quotients do: x - s (n + 1/2) is zero or at least 2^-32 of x, so 53
// bits tell the two apart. (A wider margin sends whole waves there: with 1e-3 the
// 8-bit block of 1 x 2048 -> 2 x 512 takes 5.5 us instead of 5.2.)
struct RowScale {
  float s, inv;
  bool fast;
  __device__ __forceinline__ explicit RowScale(uint32_t m) {
    s = m < 0x7F800000u ? __uint_as_float(m) / 127.f : __builtin_nanf("");
    inv = s > 0.f ? 1.f / s : 0.f;
    fast = s > 0.f && inv < 3e38f;
  }
  __device__ __forceinline__ uint32_t exact(float x) const {
    const double q = __builtin_rint((double)x / (double)s);
    return s > 0.f ? (uint32_t)(int)__builtin_fmin(__builtin_fmax(q, -127.0), 127.0) & 255u : 0u;
  }
  // four codes, the first in the low byte
  __device__ __forceinline__ uint32_t codes4(const float* f) const {
    float n[4], far = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float t = f[e] * inv;
      n[e] = __builtin_rintf(t);
      far = __builtin_fmaxf(far, __builtin_fabsf(t - n[e]));
    }
    uint32_t o = 0;
    if (fast && far < 0.49998f) {
#pragma unroll
      for (int e = 0; e < 4; ++e) o |= ((uint32_t)(int)n[e] & 255u) << (8 * e);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) o |= exact(f[e]) << (8 * e);
    }
    return o;
  }
};
template <int T, int N> __device__ __forceinline__ uint32_t top_bits(const float* f, uint32_t m) {
#pragma unroll
  for (int i = 0; i < N; ++i) m = max(m, __float_as_uint(f[i]) & 0x7FFFFFFFu);
  return m;
}
// --------------------------------------------------------------- decode rows
// nq <= 16: a workgroup of 16 waves computes 16 weight rows (GLU: 8 gate and
// 8 up) against every activation row on 16x16 matrix instructions; the waves
// take 256-byte K chunks in turn (a chunk's loads in flight while the one
// before it is multiplied) and their sums join through LDS. Operands come
// straight from memory at any alignment: bound by the weights' bytes, or by
// latency when there are few. XT = DT_BF16 / DT_F16 (8-bit weights only): x is
// quantised by every workgroup into LDS, while its first weights arrive.
constexpr int DEC_QUANT = 32;     // elements a thread holds while it quantises

template <int T, int EPI, int XT, int NF>
__global__ __launch_bounds__(1024) void k_dense_decode(DenseDecodeArgs da) {
  const DenseArgs& a = da.d;
  typedef typename Elem<T>::acc4 acc4;
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int RED = NF * 16384;
  uint8_t* const red = smem;                       // the waves' sums
  float* const s_sq = reinterpret_cast<float*>(smem + RED);                  // 16 row scales
  uint32_t* const s_top = reinterpret_cast<uint32_t*>(smem + RED + 64);      // 16 waves' maxima
  uint8_t* const s_x = smem + RED + 128;         // quantised rows
  constexpr bool QUANT = XT != DT_I8 && T == DT_I8;
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, c = lane >> 4;
  constexpr int OP = EPI == EPI_GLU ? 8 : 16;
  const int p0 = blockIdx.x * OP * NF;
  const uint8_t* pr[NF];
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    if (EPI == EPI_GLU) {
      const int p = min(p0 + f * OP + (r & 7), a.np - 1);
      pr[f] = r < 8 ? a.p0 + (int64_t)p * a.ldp0 : a.p1 + (int64_t)p * a.ldp1;
    } else {
      pr[f] = a.p0 + (int64_t)min(p0 + f * OP + r, a.np - 1) * a.ldp0;
    }
  }
  const uint8_t* const qr = a.q0 + (int64_t)min(r, a.nq - 1) * a.ldq;
  const int64_t kb = (int64_t)da.k * Elem<T>::SIZE;
  const int chunks = (int)((kb + 255) / 256);
  const int xs = QUANT ? chunks * 256 + 16 : 0;    // bytes of a quantised row in LDS (off a bank period)
  constexpr int U = 4;
  u32x4 pv[2][NF][U], qv[2][U];
  auto load_p = [&](int buf, int ch) {
    const int64_t at = (int64_t)ch * 256 + c * 16;
    if ((int64_t)(ch + 1) * 256 <= kb) {
#pragma unroll
      for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int u = 0; u < U; ++u) __builtin_memcpy(&pv[buf][f][u], pr[f] + at + u * 64, 16);
    } else {
#pragma unroll
      for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int u = 0; u < U; ++u) pv[buf][f][u] = load_chunk<Elem<T>::SIZE>(pr[f], at + u * 64, kb);
    }
  };
  auto load_q = [&](int buf, int ch) {
    const int64_t at = (int64_t)ch * 256 + c * 16;
    if constexpr (QUANT) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        qv[buf][u] = *reinterpret_cast<const u32x4*>(s_x + min(r, a.nq - 1) * xs + at + u * 64);
    } else if ((int64_t)(ch + 1) * 256 <= kb) {
#pragma unroll
      for (int u = 0; u < U; ++u) __builtin_memcpy(&qv[buf][u], qr + at + u * 64, 16);
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u) qv[buf][u] = load_chunk<Elem<T>::SIZE>(qr, at + u * 64, kb);
    }
  };
  if (w < chunks) load_p(0, w);
  if constexpr (QUANT) {
    // threads [t per, (t + 1) per) of the workgroup take row t, per a multiple
    // of 64; each thread 8 elements at a time, held between maximum and codes
    const int per = a.nq == 1 ? 1024 : a.nq == 2 ? 512 : a.nq <= 4 ? 256 : a.nq <= 8 ? 128 : 64;
    const int row = threadIdx.x / per, i0 = threadIdx.x % per;
    const uint16_t* xr = reinterpret_cast<const uint16_t*>(a.q0 + (int64_t)min(row, a.nq - 1) * a.ldq);
    float f[DEC_QUANT / 8][8];
    uint32_t m = 0;
#pragma unroll
    for (int h = 0; h < DEC_QUANT / 8; ++h) {
      const int at = (h * per + i0) * 8;
      u32x4 v = {0, 0, 0, 0};
      if (at < da.k) v = load_chunk<2>(xr, at * 2, da.k * 2);
      unpack16<XT>(v, f[h]);
      m = top_bits<XT, 8>(f[h], m);
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
    if (lane == 0) s_top[w] = m;
    __syncthreads();
    for (int i = 0; i < per / 64; ++i) m = max(m, s_top[row * (per / 64) + i]);
    const RowScale rs(m);
    if (row < a.nq) {
      if (i0 == 0) s_sq[row] = rs.s;
#pragma unroll
      for (int h = 0; h < DEC_QUANT / 8; ++h) {
        const int at = (h * per + i0) * 8;
        if (at < chunks * 256)
          *reinterpret_cast<uint2*>(s_x + row * xs + at) = make_uint2(rs.codes4(f[h]), rs.codes4(f[h] + 4));
      }
    }
    __syncthreads();
  }
  acc4 acc[NF] = {};
  if (w < chunks) load_q(0, w);
  for (int ch = w, i = 0; ch < chunks; ch += 32) {
    // two chunks a round, so that the buffers' indices are constants
#pragma unroll
    for (i = 0; i < 2; ++i) {
      const int cur = ch + 16 * i;
      if (cur >= chunks) break;
      if (cur + 16 < chunks) {
        load_p(i ^ 1, cur + 16);
        load_q(i ^ 1, cur + 16);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int f = 0; f < NF; ++f) acc[f] = Elem<T>::mma16(pv[i][f][u], qv[i][u], acc[f]);
    }
  }
  // lane: q = lane % 16, p = 4 (lane / 16) + e; red[f][w][q][p]
  acc4* rd = reinterpret_cast<acc4*>(red);
#pragma unroll
  for (int f = 0; f < NF; ++f) rd[f * 1024 + w * 64 + r * 4 + c] = acc[f];
  __syncthreads();
  typedef decltype(acc[0][0] + 0) V;
  constexpr int PG = OP / 4, TF = 16 * PG;         // threads of a fragment
  if (threadIdx.x < NF * TF) {
    const int f = threadIdx.x / TF, q = threadIdx.x % TF / PG, g = threadIdx.x % PG;
    acc4 v0 = {}, v1 = {};
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      v0 += rd[f * 1024 + i * 64 + q * 4 + g];
      if constexpr (EPI == EPI_GLU) v1 += rd[f * 1024 + i * 64 + q * 4 + 2 + g];
    }
    V s0[4], s1[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s0[e] = v0[e];
      s1[e] = v1[e];
    }
    float sq = 1.f;
    if constexpr (T == DT_I8) sq = QUANT ? s_sq[min(q, a.nq - 1)] : a.sq[min(q, a.nq - 1)];
    finish4<T, EPI>(a, q, p0 + f * OP + g * 4, s0, s1, sq);
  }
}

// ----------------------------------------------------------- small kernels
template <int ES> __global__ __launch_bounds__(256) void k_dense_pad(DensePad j) { pad_row<ES>(j, blockIdx.x); }

// One workgroup a row, 16 bytes of x a thread at a time; the first QUANT_HOLD
// of a thread stay in registers between the maximum and the codes, longer rows
// are read twice (from the L2). VEC: q's rows are whole 8-byte (fp32: 4-byte)
// groups at such an address. Bound by memory: 3 bytes an element for 16-bit rows.
constexpr int QUANT_HOLD = 4;
template <int T, bool VEC>
__global__ __launch_bounds__(256) void k_quant_rows(const typename Row<T>::type* x, int64_t ldx, int rows, int cols,
                                                    int8_t* q, int64_t ldq, float* scale, DensePad pad) {
  if (blockIdx.x >= (uint32_t)rows) {
    pad_row<1>(pad, blockIdx.x - rows);
    return;
  }
  constexpr int ES = sizeof(typename Row<T>::type), N = 16 / ES;
  __shared__ uint32_t red[4];
  const int64_t r = blockIdx.x;
  const typename Row<T>::type* xr = x + r * ldx;
  const int chunks = (int)((ldq + N - 1) / N);     // past cols they are zero
  auto chunk = [&](int c) { return c * N < cols ? load_chunk<ES>(xr, (int64_t)c * 16, (int64_t)cols * ES) : u32x4{0, 0, 0, 0}; };
  u32x4 hold[QUANT_HOLD];
  // |x| as bits: ordered as the values, infinity and NaN above them all
  uint32_t m = 0;
  auto top = [&](u32x4 v) {
    float f[N];
    unpack16<T>(v, f);
    m = top_bits<T, N>(f, m);
  };
#pragma unroll
  for (int h = 0; h < QUANT_HOLD; ++h) hold[h] = chunk(h * 256 + threadIdx.x);
#pragma unroll
  for (int h = 0; h < QUANT_HOLD; ++h) top(hold[h]);
  for (int c = QUANT_HOLD * 256 + threadIdx.x; c < chunks; c += 256) top(chunk(c));
#pragma unroll
  for (int d = 32; d; d >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
  __syncthreads();
  m = max(max(red[0], red[1]), max(red[2], red[3]));
  const RowScale rs(m);
  if (threadIdx.x == 0) scale[r] = rs.s;
  int8_t* qr = q + r * ldq;
  auto put = [&](int c, u32x4 v) {
    float f[N];
    unpack16<T>(v, f);
    uint32_t o[N / 4];
#pragma unroll
    for (int i = 0; i < N / 4; ++i) o[i] = rs.codes4(f + 4 * i);
    if constexpr (VEC && N == 8) *reinterpret_cast<uint2*>(qr + c * 8) = make_uint2(o[0], o[1]);
    else if constexpr (VEC) *reinterpret_cast<uint32_t*>(qr + c * 4) = o[0];
    else
#pragma unroll
      for (int i = 0; i < N; ++i)
        if ((int64_t)c * N + i < ldq) qr[(int64_t)c * N + i] = (int8_t)(o[i / 4] >> (8 * (i % 4)));
  };
#pragma unroll
  for (int h = 0; h < QUANT_HOLD; ++h) {
    const int c = h * 256 + threadIdx.x;
    if (c < chunks) put(c, hold[h]);
  }
  for (int c = QUANT_HOLD * 256 + threadIdx.x; c < chunks; c += 256) put(c, chunk(c));
}

// dg = dh u act'(g) and du = dh act(g) of 8 elements from column i on, from one
// row's dh, g and u (g + inter); zero behind inter and where the row is not `in`.
template <int DT>
__device__ __forceinline__ void grad8(int act, const uint16_t* dh, const float* g, int i, int inter, bool in, float* dg,
                                      float* du) {
  float e[8], gv[8], uv[8];
  unpack16<DT>(in && i < inter ? load_chunk<2>(dh, i * 2, inter * 2) : u32x4{0, 0, 0, 0}, e);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const bool here = in && i + 4 * k < inter;
    unpack16<DT_F32>(here ? load_chunk<4>(g, (i + 4 * k) * 4, inter * 4) : u32x4{0, 0, 0, 0}, gv + 4 * k);
    unpack16<DT_F32>(here ? load_chunk<4>(g + inter, (i + 4 * k) * 4, inter * 4) : u32x4{0, 0, 0, 0}, uv + 4 * k);
  }
  float v[8], dv[8];
  act_grad_n<8>(gv, act, v, dv);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    dg[k] = e[k] * uv[k] * dv[k];
    du[k] = e[k] * v[k];
  }
}

// fp16 has 11 bits from 2^-14 on only, and gradients are often smaller: dg and
// du go into their products times 2^k, one k a call, and the epilogues multiply
// by 2^-k. k (0 to 100) is the largest that leaves every |dg|, |du| that fp16
// holds below 2^15, so they lose what fp16 does relative to the largest of
// them (2^-39 of it at least: half a subnormal step). Values that are not finite
// or too large for fp16 do not count, and become infinite as they are. This
// kernel finds the largest: each workgroup of four groups of 256 threads, a group
// a stretch of 2048 columns at a time, leaves its maximum in top[block]. It reads
// what k_glu_grad reads again: a backward call of 512 x 2048 x 512 takes 25.7 us
// with it and 21.8 without, 8192 x 4096 x 8192 2,010 and 1,870; without it dWg of
// 512 rows with dh of deviation 1e-6 is 2.7e-2 off in norm, where rounding the
// outputs alone is 1.2e-3. bf16 has the range of fp32 and needs none of this.
__global__ __launch_bounds__(1024) void k_glu_top(int act, const uint16_t* dh, int64_t lddh, const float* gu, int rows,
                                                  int inter, uint32_t* top) {
  __shared__ uint32_t red[16];
  const int ny = (inter + 2047) / 2048, t = threadIdx.x & 255;
  uint32_t m = 0;
  for (int it = blockIdx.x * 4 + (threadIdx.x >> 8); it < rows * ny; it += gridDim.x * 4) {
    const int64_t r = it / ny;
    const int i = (it % ny * 256 + t) * 8;
    if (i >= inter) continue;
    float dg[8], du[8];
    grad8<DT_F16>(act, dh + r * lddh, gu + r * 2 * inter, i, inter, true, dg, du);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float a = __builtin_fabsf(dg[k]), b = __builtin_fabsf(du[k]);
      if (a < 65520.f) m = max(m, __float_as_uint(a));
      if (b < 65520.f) m = max(m, __float_as_uint(b));
    }
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 16; ++w) m = max(m, red[w]);
    top[blockIdx.x] = m;
  }
}
// the k of a call, for every thread of a workgroup of 256
__device__ __forceinline__ int grad_shift(const uint32_t* top, int tops) {
  __shared__ uint32_t red[4];
  uint32_t m = 0;
  for (int c = threadIdx.x; c < tops; c += 256) m = max(m, top[c]);
#pragma unroll
  for (int d = 32; d; d >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
  __syncthreads();
  m = max(max(red[0], red[1]), max(red[2], red[3]));
  return m ? min(max(14 + 127 - (int)(m >> 23), 0), 100) : 0;
}

// [dg | du] from dh and the kept g, u, 8 elements a thread: 14 bytes an
// element through memory, which bounds it (196 us for 8192 x 8192, 4.8 TB/s).
// PAIRS: each row as a high and a low part, in groups of 16 rows of each (see
// DenseArgs::fold), the last group filled up with zero rows. fp16: times 2^k
// (k_glu_top's maxima in top), 2^-k left in `down`.
template <int DT, bool PAIRS>
__global__ __launch_bounds__(256) void k_glu_grad(int act, const uint16_t* dh, int64_t lddh, const float* gu, int rows,
                                                  int inter, int ip, uint16_t* d, DensePad pad, DensePairs px,
                                                  const uint32_t* top, int tops, float* down) {
  const int drows = PAIRS ? (rows + 15) / 16 * 16 : rows;
  if (blockIdx.x >= (uint32_t)drows) {
    const int r = blockIdx.x - drows, pr = PAIRS && px.src ? 2 * drows : 0;
    if (blockIdx.y == 0) {
      if (r < pr) pair_row<DT>(px, r);
      else pad_row<2>(pad, r - pr);
    }
    return;
  }
  const int64_t r = blockIdx.x;
  const int i = (blockIdx.y * 256 + threadIdx.x) * 8;
  float dg[8], du[8];
  grad8<DT>(act, dh + r * lddh, gu + r * 2 * inter, i, inter, !PAIRS || r < rows, dg, du);
  if constexpr (DT == DT_F16) {
    const int k = grad_shift(top, tops);
    if (r == 0 && i == 0) *down = __builtin_ldexpf(1.f, -k);
    const float up = __builtin_ldexpf(1.f, k);
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      dg[n] *= up;
      du[n] *= up;
    }
  }
  if (i >= ip) return;
  const int64_t at = PAIRS ? (r / 16) * 32 + r % 16 : r;
  u32x4* o = reinterpret_cast<u32x4*>(d + at * 2 * ip + i);
  o[0] = pack16<DT>(dg);
  o[ip / 8] = pack16<DT>(du);
  if constexpr (PAIRS) {
    o += 16 * (2 * ip / 8);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      dg[k] = low_part<DT>(dg[k]);
      du[k] = low_part<DT>(du[k]);
    }
    o[0] = pack16<DT>(dg);
    o[ip / 8] = pack16<DT>(du);
  }
}

// --------------------------------------------------------------- launchers
template <int T, int EPI, int FORM, int BP, int BQ, int WP, int WQ, int R, int KB, int KU>
static hipError_t launch_tile(const DenseArgs& a, hipStream_t s) {
  typedef Dense<T, EPI, FORM, BP, BQ, WP, WQ, R, KB, KU> K;
  constexpr int lds = R * K::UNIT;
  constexpr int OP = EPI == EPI_GLU ? BP / 2 : BP;
  auto kern = k_dense<T, EPI, FORM, BP, BQ, WP, WQ, R, KB, KU>;
  const int64_t tiles = (int64_t)((a.np + OP - 1) / OP) * ((a.nq + BQ - 1) / BQ);
  if (tiles > 0x7FFFFFFF) return hipErrorInvalidValue;
  if (lds > 65536) {
    // once a kernel and device (a runtime call of about a microsecond)
    static std::atomic<uint64_t> allowed{0};
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (!(allowed.load(std::memory_order_relaxed) & bit)) {
      e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
      if (e != hipSuccess) return e;
      allowed.fetch_or(bit, std::memory_order_relaxed);
    }
  }
  hipLaunchKernelGGL(kern, dim3((uint32_t)tiles, a.splits), dim3(WP * WQ * 64), lds, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  hipLaunchKernelGGL((k_dense_join<T, EPI>), dim3(FORM == FORM_NN && a.fold ? a.fold : a.nq, (a.np + 1023) / 1024), dim3(256), 0,
                     s, a);
  return hipGetLastError();
}

// tiles: 0 256 x 256; 1 128 x 128, two workgroups a CU; 2 64 x 64, two a CU;
// 3 128 x 128 in steps of 256 bytes (half the barriers), one a CU
template <int T, int EPI, int FORM>
static hipError_t launch_form(int tile, const DenseArgs& a, hipStream_t s) {
  switch (tile) {
    case 0: return launch_tile<T, EPI, FORM, 256, 256, 4, 2, 5, 128, 1>(a, s);
    case 1: return launch_tile<T, EPI, FORM, 128, 128, 2, 4, 5, 128, 1>(a, s);
    case 3: return launch_tile<T, EPI, FORM, 128, 128, 2, 4, 5, 256, 2>(a, s);
    case 2:
      if constexpr (EPI == EPI_GLU) return launch_tile<T, EPI, FORM, 64, 64, 1, 4, 5, 256, 2>(a, s);
      else return launch_tile<T, EPI, FORM, 64, 64, 2, 2, 5, 256, 2>(a, s);
  }
  return hipErrorInvalidValue;
}

hipError_t launch_dense(int dt, int epi, int form, int tile, const DenseArgs& a, hipStream_t s) {
  if (form == FORM_NT && epi == EPI_GLU) {
    if (dt == DT_BF16) return launch_form<DT_BF16, EPI_GLU, FORM_NT>(tile, a, s);
    if (dt == DT_F16) return launch_form<DT_F16, EPI_GLU, FORM_NT>(tile, a, s);
    if (dt == DT_I8) return launch_form<DT_I8, EPI_GLU, FORM_NT>(tile, a, s);
  }
  if (form == FORM_NT && epi == EPI_SCALE && dt == DT_I8) return launch_form<DT_I8, EPI_SCALE, FORM_NT>(tile, a, s);
  if (epi == EPI_OUT) {
    if (dt == DT_BF16 && form == FORM_NN) return launch_form<DT_BF16, EPI_OUT, FORM_NN>(tile, a, s);
    if (dt == DT_F16 && form == FORM_NN) return launch_form<DT_F16, EPI_OUT, FORM_NN>(tile, a, s);
    if (dt == DT_BF16 && form == FORM_TN) return launch_form<DT_BF16, EPI_OUT, FORM_TN>(tile, a, s);
    if (dt == DT_F16 && form == FORM_TN) return launch_form<DT_F16, EPI_OUT, FORM_TN>(tile, a, s);
  }
  return hipErrorInvalidValue;
}

// Whether a decode call quantises x in its own launch: where that costs each
// workgroup little (half of what its threads can hold) and the workgroups run
// in one round. The rule goes by the time on the GPU, which is what a captured
// decode step takes; an eager call of two launches takes 15 to 16 us whatever
// they do, and would gain by one. 1 x 2048 -> 2048: 5.2 us against 3.5 + 2.5 and a launch between;
// 16 x 2048 -> 2 x 512 (twice the bound): 9.6 us against 7.4 in two launches; 1 x
// 4096 -> 2 x 8192 (two rounds): 20.9 against 17.3.
bool dense_decode_quantises(int epi, int rows, int k, int np) {
  return (int64_t)rows * k <= 1024 * DEC_QUANT / 2 && np <= 512 * (epi == EPI_GLU ? 8 : 16);
}

template <int T, int EPI, int XT, int NF>
static hipError_t decode_launch_nf(const DenseDecodeArgs& a, hipStream_t s) {
  constexpr int OP = (EPI == EPI_GLU ? 8 : 16) * NF;
  const size_t lds = NF * 16384 + 128 + (XT != DT_I8 && T == DT_I8 ? (size_t)a.d.nq * ((a.k + 255) / 256 * 256 + 16) : 0);
  hipLaunchKernelGGL((k_dense_decode<T, EPI, XT, NF>), dim3((a.d.np + OP - 1) / OP), dim3(1024), lds, s, a);
  return hipGetLastError();
}
template <int T, int EPI, int XT>
static hipError_t decode_launch(const DenseDecodeArgs& a, hipStream_t s) {
  constexpr int OP = EPI == EPI_GLU ? 8 : 16;
  // Two fragments a workgroup halve the reads of x (from the L2), where enough
  // workgroups are left and x is not small: 16 x 4096 -> 2 x 8192 bf16 30.8 us
  // against 34.8; 2 x 2048 outputs would take 13.9 against 11.0.
  if (XT == DT_I8 && a.d.nq > 4 && a.d.np >= 512 * OP) return decode_launch_nf<T, EPI, XT, XT == DT_I8 ? 2 : 1>(a, s);
  return decode_launch_nf<T, EPI, XT, 1>(a, s);
}

hipError_t launch_dense_decode(int dt, int epi, int xt, const DenseDecodeArgs& a, hipStream_t s) {
  if (dt == DT_BF16 && epi == EPI_GLU) return decode_launch<DT_BF16, EPI_GLU, DT_I8>(a, s);
  if (dt == DT_F16 && epi == EPI_GLU) return decode_launch<DT_F16, EPI_GLU, DT_I8>(a, s);
  if (dt != DT_I8) return hipErrorInvalidValue;
  if (epi == EPI_GLU) {
    if (xt == DT_BF16) return decode_launch<DT_I8, EPI_GLU, DT_BF16>(a, s);
    if (xt == DT_F16) return decode_launch<DT_I8, EPI_GLU, DT_F16>(a, s);
    return decode_launch<DT_I8, EPI_GLU, DT_I8>(a, s);
  }
  if (xt == DT_BF16) return decode_launch<DT_I8, EPI_SCALE, DT_BF16>(a, s);
  if (xt == DT_F16) return decode_launch<DT_I8, EPI_SCALE, DT_F16>(a, s);
  return decode_launch<DT_I8, EPI_SCALE, DT_I8>(a, s);
}

static uint32_t pad_rows(const DensePad* j) { return j ? (uint32_t)(j->rows[0] + j->rows[1] + j->rows[2]) : 0; }

hipError_t launch_dense_pad(int esize, const DensePad& j, hipStream_t s) {
  if (!pad_rows(&j)) return hipSuccess;
  if (esize == 1) hipLaunchKernelGGL((k_dense_pad<1>), dim3(pad_rows(&j)), dim3(256), 0, s, j);
  else hipLaunchKernelGGL((k_dense_pad<2>), dim3(pad_rows(&j)), dim3(256), 0, s, j);
  return hipGetLastError();
}

template <int T>
static void quant_launch(const void* x, int64_t ldx, int rows, int cols, int8_t* q, int64_t ldq, float* scale,
                         const DensePad* pad, hipStream_t s) {
  typedef typename Row<T>::type E;
  constexpr int N = T == DT_F32 ? 4 : 8;
  const bool vec = reinterpret_cast<uintptr_t>(q) % N == 0 && ldq % N == 0;
  const dim3 grid((uint32_t)rows + pad_rows(pad));
  const E* e = static_cast<const E*>(x);
  const DensePad j = pad ? *pad : DensePad{};
  if (vec) hipLaunchKernelGGL((k_quant_rows<T, true>), grid, dim3(256), 0, s, e, ldx, rows, cols, q, ldq, scale, j);
  else hipLaunchKernelGGL((k_quant_rows<T, false>), grid, dim3(256), 0, s, e, ldx, rows, cols, q, ldq, scale, j);
}

hipError_t launch_quant_rows(int dt, const void* x, int64_t ldx, int rows, int cols, int8_t* q, int64_t ldq,
                             float* scale, const DensePad* pad, hipStream_t s) {
  if (dt == DT_BF16) quant_launch<DT_BF16>(x, ldx, rows, cols, q, ldq, scale, pad, s);
  else if (dt == DT_F16) quant_launch<DT_F16>(x, ldx, rows, cols, q, ldq, scale, pad, s);
  else if (dt == DT_F32) quant_launch<DT_F32>(x, ldx, rows, cols, q, ldq, scale, pad, s);
  else return hipErrorInvalidValue;
  return hipGetLastError();
}

template <int DT>
static void grad_launch(bool pairs, int act, const void* dh, int64_t lddh, const float* gu, int rows, int inter, int ip,
                        void* d, const DensePad& pad, const DensePairs& px, float* down, hipStream_t s) {
  const int drows = pairs ? (rows + 15) / 16 * 16 : rows;
  const dim3 grid(drows + (pairs && px.src ? 2 * drows : 0) + pad_rows(&pad), (ip + 2047) / 2048);
  const uint16_t* e = static_cast<const uint16_t*>(dh);
  uint16_t* o = static_cast<uint16_t*>(d);
  uint32_t* top = reinterpret_cast<uint32_t*>(down) + 1;
  int tops = 0;
  if (DT == DT_F16) {
    tops = (int)std::min<int64_t>(((int64_t)rows * ((inter + 2047) / 2048) + 3) / 4, GRAD_TOPS);
    hipLaunchKernelGGL(k_glu_top, dim3(tops), dim3(1024), 0, s, act, e, lddh, gu, rows, inter, top);
  }
  if (pairs)
    hipLaunchKernelGGL((k_glu_grad<DT, true>), grid, dim3(256), 0, s, act, e, lddh, gu, rows, inter, ip, o, pad, px,
                       top, tops, down);
  else
    hipLaunchKernelGGL((k_glu_grad<DT, false>), grid, dim3(256), 0, s, act, e, lddh, gu, rows, inter, ip, o, pad, px,
                       top, tops, down);
}

hipError_t launch_glu_grad(int dt, bool pairs, int act, const void* dh, int64_t lddh, const float* gu, int rows,
                           int inter, int ip, void* d, const DensePad& pad, const DensePairs& px, float* down,
                           hipStream_t s) {
  if (dt == DT_BF16) grad_launch<DT_BF16>(pairs, act, dh, lddh, gu, rows, inter, ip, d, pad, px, down, s);
  else grad_launch<DT_F16>(pairs, act, dh, lddh, gu, rows, inter, ip, d, pad, px, down, s);
  return hipGetLastError();
}

}  // namespace moe

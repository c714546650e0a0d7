// Argument blocks and launchers of the dense feed-forward operators
// (internal to the library).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

enum { DT_BF16 = 0, DT_F16 = 1, DT_I8 = 2, DT_F32 = 3 };   // element types
enum { ACT_SILU = 0, ACT_GELU_TANH = 1 };
// What a product does with its sums: store them (OUT), scale and add the
// bias first (SCALE, 8-bit operands), gate them (GLU)
enum { EPI_OUT = 0, EPI_SCALE = 1, EPI_GLU = 2 };
// Operand forms: NT both with the contraction contiguous; NN the P operand
// with it as the row index; TN both
enum { FORM_NT = 0, FORM_NN = 1, FORM_TN = 2 };

// One product out[q, p] = sum_k Q[q, k] P[p, k]. P is the operand whose
// index runs along the output's rows of memory (weights, or x for the weight
// gradients), Q the other one. Every operand row starts at a 16-byte
// boundary and is 16-byte granular (the padding zero along k).
struct DenseArgs {
  const uint8_t* p0;      // NT: P rows (GLU: gate rows); NN/TN: rows of k
  const uint8_t* p1;      // GLU: up rows; NN: rows of the second segment
  const uint8_t* q0;
  int64_t ldp0, ldp1, ldq;   // bytes
  int np, nq;             // output columns and rows (GLU: np of gate and of up)
  int kbytes;             // NT / NN: bytes of a k-contiguous row in use (multiple of 16)
  int krows;              // NN: k rows of one segment in use; TN: k rows
  int segbytes;           // NN: Q bytes of the first segment
  int splits;             // K ranges (1: the epilogue runs in the product)
  int act;
  // Gradients of few rows: D's rows are pairs of a high and a low 16-bit part, 16
  // high rows, then their 16 low ones, and so on (the last group zero behind the
  // rows). fold = rows (0: no pairs). NN: nq counts the parts, the output has
  // fold rows. (TN: krows counts the parts, P is a DensePairs copy.)
  int fold;
  // outputs
  void* out0;             // [nq, np] (weight gradients: rows below qseg)
  void* out1;             // weight gradients: rows from qpad on
  int64_t ldo;            // elements
  int out_dt;             // DT_BF16 / DT_F16
  int qseg, qpad;         // rows of out0, first row index of out1 (0: one output)
  void* save;             // GLU: fp32 [nq, 2 np] pre-activations, or null
  const float* sq;        // 8-bit: scale of each Q row
  const float* sp0;       // 8-bit: scale of each P row (GLU: gate)
  const float* sp1;       // 8-bit GLU: up
  const float* bias;      // SCALE: [np] or null
  float* part;            // splits > 1: [splits, nq, pcols] sums (int32 for 8-bit)
  int64_t pcols;
  const float* down;      // gradients in fp16: the power of two that divides D's out again
};

// Decode rows (nq <= 16), any alignment: k elements per row. launch_dense_decode's
// xt: DT_I8 (x has the weights' type), or the 16-bit type of an x that the kernel
// quantises itself (8-bit weights, where dense_decode_quantises says so).
struct DenseDecodeArgs {
  DenseArgs d;
  int k;
};

int dense_tile(int epi, int np, int nq, int steps, int* splits);
hipError_t launch_dense(int dt, int epi, int form, int tile, const DenseArgs& a, hipStream_t s);
// Copies of up to three operands (rows of `cols` elements, any start and row
// stride ld) to rows of ldd elements, zero behind cols; rows[o] = 0: none.
struct DensePad {
  const void* src[3];
  void* dst[3];
  int64_t ld[3];
  int rows[3];
  int cols;
  int64_t ldd;   // a multiple of 16 bytes
};

// The copy of rows [rows, cols] of 16 bits (row stride ld) that meets D's high
// and low parts in the product over rows: dst rows of ldd elements, for each
// group of 16 rows the rows, then the same rows with zeros where they are not
// finite; zero behind rows and behind cols. src = null: none.
struct DensePairs {
  const void* src;
  void* dst;
  int64_t ld, ldd;
  int rows, cols;
};

bool dense_decode_quantises(int epi, int rows, int k, int np);
hipError_t launch_dense_decode(int dt, int epi, int xt, const DenseDecodeArgs& a, hipStream_t s);
hipError_t launch_dense_pad(int esize, const DensePad& j, hipStream_t s);
// q[r, 0..ldq) (zero behind cols), scale[r]; and the copies of pad (8-bit
// operands), or null
hipError_t launch_quant_rows(int dt, const void* x, int64_t ldx, int rows, int cols, int8_t* q, int64_t ldq,
                             float* scale, const DensePad* pad, hipStream_t s);
// D[r] = [dg | du], each ip wide (zero behind inter); pairs: see
// DenseArgs::fold; and the copies of pad (16-bit operands) and px (with pairs).
// fp16: D times a power of two, its inverse in *down, in front of GRAD_TOPS
// words of scratch (bf16: down is not used).
constexpr int GRAD_TOPS = 512;
hipError_t launch_glu_grad(int dt, bool pairs, int act, const void* dh, int64_t lddh, const float* gu, int rows,
                           int inter, int ip, void* d, const DensePad& pad, const DensePairs& px, float* down,
                           hipStream_t s);

}  // namespace moe

// Internal launchers of the 8-bit activation operators (act8.cu holds the
// codec, the gated activation and the C entry points, act8_grad.cu the
// gradients' operand passes, act8_gemm.cu the products).
#pragma once
#include "common.cuh"

namespace s4 {

constexpr int64_t kAct8MaxRows = int64_t(1) << 30;     // of any matrix
constexpr int64_t kAct8MaxCols = int64_t(1) << 26;
constexpr int64_t kAct8MaxInner = int64_t(1) << 17;    // 128 * 127 * 2^17 < 2^31: an integer sum stays exact
constexpr int kAct8CodeAlign = 16;                     // bytes, of code rows (TMA)
constexpr int kAct8Digits = 3;                         // base-256 digits of a fixed-point gradient

// A matrix as TMA reads it: `parts` planes of rows x ld elements, `plane`
// rows apart, 16-byte aligned rows.
struct Act8Operand {
  const void* p;
  int64_t ld;                                          // elements
  int64_t plane;                                       // rows from one plane to the next
};

struct Act8Out {
  void* y;                                             // R x M
  int64_t ld;
  int32_t dtype;
  int32_t accumulate;                                  // y += product (in fp32, rounded once)
  const float* row_scale;                              // of R, optional
  const float* col_scale;                              // of M, optional
  const float* bias;                                   // of M, optional
  int32_t col_shift;                                   // halves: column m has col_scale[m >> col_shift]
};

// Where a product raises SHAMPOO4_FLAG_TIMEOUT (may be null), and the limit of
// its waits (0: 2 s).  The loads, whose barriers also tell that nothing is
// under way when a CTA leaves, keep the 2 s.
struct Act8Watch {
  uint32_t* flags = nullptr;
  uint64_t wait_ns = 0;
};

// How an integer product is cut: tiles of `rows` rows by one CTA each (0: by
// pairs of CTAs), the contraction in `shares`.
struct Form { int rows, shares; };
Form act8_codes_form(int64_t M, int64_t R, int64_t K);
Form act8_digits_form(int64_t M, int64_t R, int64_t K);

// All products: Y[r, m] = row_scale[r] col_scale[m] sum_k B[r, k] A[m, k] + bias[m].

// int8 codes both: a is M x K, b is R x K (K contiguous).  after_pass: b was
// written by the kernel enqueued just before on this stream, and a was not;
// the launch may then overlap that kernel's end.  (The others always
// follow their own operand pass.)
shampoo4_status launch_act8_codes(const Act8Operand& a, const Act8Operand& b, int64_t M, int64_t R, int64_t K,
                                  const Act8Out& out, bool after_pass, Act8Watch watch, cudaStream_t st);
// a: codes K x M (M contiguous); b: kAct8Digits planes of R x K digits, most
// significant first: B = 65536 d0 + 256 d1 + d2.
shampoo4_status launch_act8_digits(const Act8Operand& a, const Act8Operand& b, int64_t M, int64_t R, int64_t K,
                                   const Act8Out& out, Act8Watch watch, cudaStream_t st);
// Halves both, operands the sums of their planes: a is K x M in a_parts, b is
// K x R in b_parts: 2 and 1 or 2 (the product of the second planes is left
// out), or 1 and 1.
// shares (act8_halves_shares, one of the least estimated time): with more than
// one, the contraction is cut in that many and out.y receives their sums, fp32,
// R x M each, for the caller to add up.
int act8_halves_shares(int64_t M, int64_t R, int64_t K);
shampoo4_status launch_act8_halves(const Act8Operand& a, int a_parts, const Act8Operand& b, int b_parts, int64_t M,
                                   int64_t R, int64_t K, int shares, const Act8Out& out, Act8Watch watch,
                                   cudaStream_t st);

// The same with one plane each, and b R x K.
shampoo4_status launch_act8_row_halves(const Act8Operand& a, const Act8Operand& b, int64_t M, int64_t R, int64_t K,
                                       const Act8Out& out, Act8Watch watch, cudaStream_t st);

// A gradient as act8_weight_grad and act8_input_grad take it (weight: which).
struct Act8Grad {
  bool weight;
  const void* dy;
  int32_t dtype;
  int64_t lddy;
  const int8_t* codes;
  int64_t ldc;
  const float* scales;
  int32_t group;
  int64_t tokens, out, inner;
  void* y;
  int32_t result;
  int64_t ldy;
  int32_t accumulate;
};
// Everything that can be refused, and the workspace that the run needs.
shampoo4_status act8_grad_check(const Act8Grad& g, size_t* bytes);
shampoo4_status act8_grad_run(const Act8Grad& g, void* ws, Act8Watch watch, cudaStream_t st);

}  // namespace s4

// Internal launchers of the 8-bit activation operators (act8.cu holds the
// codec, the gated activation and the C entry points, act8_gemm.cu the
// products).
#pragma once
#include "common.cuh"

namespace s4 {

constexpr int64_t kAct8MaxDim = int64_t(1) << 30;      // rows or columns of any matrix
constexpr int64_t kAct8MaxInner = int64_t(1) << 17;    // 127^2 * 2^17 < 2^31: the integer sum stays exact
constexpr int kAct8CodeAlign = 16;                     // bytes, of code rows (TMA)

// An operand of a product in bfloat16 parts: value = hi + lo (lo optional).
struct Act8Parts {
  const void* hi;
  const void* lo;
  int64_t ld;                                          // elements
};

struct Act8Out {
  void* y;
  int64_t ld;
  int32_t dtype;
  int32_t accumulate;                                  // y += product (in fp32, rounded once)
  const float* row_scale;                              // optional
  const float* col_scale;                              // optional
  const float* bias;                                   // optional
};

// Y[m, n] = row_scale[m] col_scale[n] sum_k A[m, k] B[n, k] + bias[n] on int8 codes.
shampoo4_status launch_act8_gemm_i8(const int8_t* a, int64_t lda, const int8_t* b, int64_t ldb, int64_t M, int64_t N,
                                    int64_t K, const Act8Out& out, uint32_t* flags, cudaStream_t st);

// Y[m, n] = sum_k A(m, k) B(k, n) on bfloat16 parts; b is K x N row-major, a
// is M x K row-major (a_mn = 0) or K x M row-major (a_mn = 1).  Products
// taken: hi hi, hi lo (when b.lo), lo hi (when a.lo).
shampoo4_status launch_act8_gemm_bf16(const Act8Parts& a, int a_mn, const Act8Parts& b, int64_t M, int64_t N,
                                      int64_t K, const Act8Out& out, uint32_t* flags, cudaStream_t st);

}  // namespace s4

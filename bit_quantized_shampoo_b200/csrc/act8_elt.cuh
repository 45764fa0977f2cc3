// Elements, code rows, work partition and argument checks shared by the
// streaming kernels of the 8-bit activation operators.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <algorithm>
#include <type_traits>
#include "act8.h"
#include "plan.h"

namespace s4 {
namespace {

constexpr int kChunk = 256;                            // columns of a warp's piece of a row, 8 per lane
constexpr int kThreads = 256;

// ---- 8 elements of a row

template <class T> struct Raw8 { uint4 v[sizeof(T) / 2]; };

__device__ __forceinline__ float elt(const Raw8<float>& r, int i) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(r.v);
  return __uint_as_float(w[i]);
}
__device__ __forceinline__ float elt(const Raw8<__nv_bfloat16>& r, int i) {
  const uint32_t w = reinterpret_cast<const uint32_t*>(r.v)[i >> 1];
  return __uint_as_float((i & 1) ? (w & 0xffff0000u) : (w << 16));
}
__device__ __forceinline__ float elt(const Raw8<__half>& r, int i) {
  const uint32_t w = reinterpret_cast<const uint32_t*>(r.v)[i >> 1];
  return __half2float(__ushort_as_half(uint16_t((i & 1) ? (w >> 16) : w)));
}
__device__ __forceinline__ void to_elt(float x, float& o) { o = x; }
__device__ __forceinline__ void to_elt(float x, __nv_bfloat16& o) { o = __float2bfloat16_rn(x); }
__device__ __forceinline__ void to_elt(float x, __half& o) { o = __float2half_rn(x); }

// Columns c .. c + 7 of a row of n (zeros past its end).
template <class T>
__device__ __forceinline__ void load8(const T* row, int64_t c, int64_t n, bool vec, Raw8<T>& r) {
  if (vec && c + 8 <= n) {
    const uint4* p = reinterpret_cast<const uint4*>(row + c);
#pragma unroll
    for (int i = 0; i < int(sizeof(T) / 2); ++i) r.v[i] = __ldg(p + i);
  } else {
    T* e = reinterpret_cast<T*>(r.v);
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = c + i < n ? row[c + i] : T(0.0f);
  }
}
template <class T>
__device__ __forceinline__ void store8(T* row, int64_t c, int64_t n, bool vec, const float (&v)[8]) {
  Raw8<T> r;
  T* e = reinterpret_cast<T*>(r.v);
#pragma unroll
  for (int i = 0; i < 8; ++i) to_elt(v[i], e[i]);
  if (vec && c + 8 <= n) {
    uint4* p = reinterpret_cast<uint4*>(row + c);
#pragma unroll
    for (int i = 0; i < int(sizeof(T) / 2); ++i) p[i] = r.v[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < n) row[c + i] = e[i];
  }
}
// Code rows are 16-byte aligned, so 8 codes at a multiple of 8 are one word pair.
__device__ __forceinline__ void load_codes8(const int8_t* row, int64_t c, int64_t n, uint2& w) {
  if (c + 8 <= n) {
    w = __ldg(reinterpret_cast<const uint2*>(row + c));
  } else {
    w = make_uint2(0u, 0u);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < n) (i < 4 ? w.x : w.y) |= uint32_t(uint8_t(row[c + i])) << (8 * (i & 3));
  }
}
__device__ __forceinline__ void store_codes8(int8_t* row, int64_t c, int64_t n, uint2 w) {
  if (c + 8 <= n) {
    *reinterpret_cast<uint2*>(row + c) = w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < n) row[c + i] = int8_t((i < 4 ? w.x : w.y) >> (8 * (i & 3)));
  }
}
__device__ __forceinline__ float code_at(uint2 w, int i) {
  return float(int8_t((i < 4 ? w.x : w.y) >> (8 * (i & 3))));
}

// Bits of |x|: as integers they order NaN above +Inf above every finite
// magnitude, so an integer maximum also tells a group with NaN or Inf.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }


// Over the group's lanes (a power of two, consecutive, aligned).
__device__ __forceinline__ uint32_t group_max(uint32_t m, int lanes) {
  for (int o = lanes >> 1; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}
// Over the CTA, whatever its shape; slots: one word per warp.
__device__ __forceinline__ uint32_t cta_max(uint32_t m, uint32_t* slots) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  m = __reduce_max_sync(0xffffffffu, m);
  __syncthreads();                                       // the slots' previous use is over
  if (lane == 0) slots[warp] = m;
  __syncthreads();
  return __reduce_max_sync(0xffffffffu, lane < int(blockDim.x >> 5) ? slots[lane] : 0u);
}

// The product enqueued next may be launched now (it waits for this kernel's
// results itself).
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

struct Mat {
  const void* p;
  int64_t ld;
  int32_t vec;       // rows are 16-byte aligned
};
struct Ckpt {
  int8_t* codes;
  int64_t ldc;
  float* scales;     // rows x groups, dense
};

// Pieces of rows as warps: blockDim = (32 wx, wy), blockIdx.x over rows,
// blockIdx.y over column pieces.
struct Piece {
  int64_t row, c;    // this lane's first column
  __device__ __forceinline__ Piece() {
    row = int64_t(blockIdx.x) * blockDim.y + threadIdx.y;
    c = (int64_t(blockIdx.y) * (blockDim.x >> 5) + (threadIdx.x >> 5)) * kChunk + (threadIdx.x & 31) * 8;
  }
};
dim3 piece_block(int64_t cols) {
  unsigned wx = 1;
  while (wx < kThreads / 32 && int64_t(wx) * kChunk < cols) wx *= 2;
  return dim3(32 * wx, kThreads / 32 / wx);
}
bool piece_grid(int64_t rows, int64_t cols, dim3 b, dim3* g) {
  const int64_t per = int64_t(b.x / 32) * kChunk;
  const int64_t gx = (rows + b.y - 1) / b.y, gy = (cols + per - 1) / per;
  if (gx > 0x7fffffffLL || gy > 65535) return false;
  *g = dim3(unsigned(gx), unsigned(gy));
  return true;
}

// ------------------------------------------------------------------ host

int64_t elt_size(int32_t dtype) { return dtype == ACT8_FP32 ? 4 : 2; }
bool dtype_ok(int32_t d) { return d == ACT8_FP32 || d == ACT8_BF16 || d == ACT8_FP16; }
bool group_ok(int32_t g) { return g == 0 || g == 32 || g == 64 || g == 128 || g == 256; }
int64_t group_count(int64_t cols, int32_t group) { return group ? (cols + group - 1) / group : 1; }
bool shape_ok(int64_t rows, int64_t cols) {
  return rows >= 0 && cols >= 0 && rows <= kAct8MaxDim && cols <= kAct8MaxDim;
}
// A float matrix: element-aligned, rows that do not overlap.
bool mat_ok(const void* p, int32_t dtype, int64_t rows, int64_t cols, int64_t ld) {
  return p && dtype_ok(dtype) && aligned(p, size_t(elt_size(dtype))) && (ld >= cols || rows == 1);
}
bool codes_ok(const void* p, int64_t ldc, int64_t cols, const void* scales) {
  return p && scales && aligned(p, kAct8CodeAlign) && ldc % kAct8CodeAlign == 0 && ldc >= cols && aligned(scales, 4);
}
bool row_aligned(const void* p, int64_t ld, int32_t dtype) {
  return aligned(p, 16) && (ld * elt_size(dtype)) % 16 == 0;
}
Mat mat(const void* p, int64_t ld, int32_t dtype) { return Mat{p, ld, row_aligned(p, ld, dtype) ? 1 : 0}; }

// Call f(T*) with a null pointer of the element type.
template <class F>
shampoo4_status by_dtype(int32_t dtype, F f) {
  if (dtype == ACT8_FP32) return f(static_cast<float*>(nullptr));
  if (dtype == ACT8_BF16) return f(static_cast<__nv_bfloat16*>(nullptr));
  return f(static_cast<__half*>(nullptr));
}

}  // namespace
}  // namespace s4

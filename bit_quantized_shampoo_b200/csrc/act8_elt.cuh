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

// Two floats as the operand of a packed fp32 instruction.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Words 0 .. N - 1 of the words w shifted down by `bytes` (0 .. 16): words move by
// selects (the shift is the same for a whole row), bytes by funnel shifts.
template <int N, bool SUBWORD>
__device__ __forceinline__ void shift_down(uint32_t (&w)[N + 5], uint32_t bytes) {
  if (bytes & 16u) {
#pragma unroll
    for (int i = 0; i < N + 1; ++i) w[i] = w[i + 4];
  }
  if (bytes & 8u) {
#pragma unroll
    for (int i = 0; i < N + 3; ++i) w[i] = w[i + 2];
  }
  if (bytes & 4u) {
#pragma unroll
    for (int i = 0; i < N + 4; ++i) w[i] = w[i + 1];
  }
  if (SUBWORD) {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 8u * (bytes & 3u));
  }
}

// Columns c .. c + 7 of a row of n (zeros past its end).  A: rows are 16-byte
// aligned (vec 2: 32-byte, fp32 then moves its 8 elements at once).  Else, of
// any alignment: the aligned 16-byte pieces around the elements, shifted,
// inside the row, and one by one at its ends, so that nothing outside the row
// is read.  (Kernels are built for each: with both in one, the registers of
// the shifts cost aligned data a quarter of its bandwidth.)
template <bool A, class T>
__device__ __forceinline__ void load8(const T* row, int c, int n, int vec, Raw8<T>& r) {
  constexpr int kWords = 2 * int(sizeof(T));            // of 8 elements
  if (A && c + 8 <= n) {
    if (sizeof(T) == 4 && vec == 2) {
      uint32_t* w = reinterpret_cast<uint32_t*>(r.v);
      asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                   : "l"(row + c));
    } else {
      const uint4* p = reinterpret_cast<const uint4*>(row + c);
#pragma unroll
      for (int i = 0; i < int(sizeof(T) / 2); ++i) r.v[i] = __ldg(p + i);
    }
  } else if (!A && c >= 8 && c + 16 <= n) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(row + c);
    const uint4* p = reinterpret_cast<const uint4*>(at & ~uintptr_t(15));
    uint32_t w[kWords + 5];
#pragma unroll
    for (int i = 0; i < kWords / 4 + 1; ++i) {
      const uint4 x = __ldg(p + i);
      w[4 * i] = x.x;
      w[4 * i + 1] = x.y;
      w[4 * i + 2] = x.z;
      w[4 * i + 3] = x.w;
    }
    w[kWords + 4] = 0u;
    shift_down<kWords, sizeof(T) == 2>(w, uint32_t(at) & 15u);
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i) r.v[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  } else {
    T* e = reinterpret_cast<T*>(r.v);
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = c + i < n ? row[c + i] : T(0.0f);
  }
}
__device__ __forceinline__ void round8(const float (&v)[8], Raw8<float>& r) {
  uint32_t* w = reinterpret_cast<uint32_t*>(r.v);
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(v[i]);
}
__device__ __forceinline__ void round8(const float (&v)[8], Raw8<__nv_bfloat16>& r) {
  uint32_t* w = reinterpret_cast<uint32_t*>(r.v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&x);
  }
}
__device__ __forceinline__ void round8(const float (&v)[8], Raw8<__half>& r) {
  uint32_t* w = reinterpret_cast<uint32_t*>(r.v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 x = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&x);
  }
}
// To rows that are 16-byte aligned (vec 2: 32-byte).
template <class T>
__device__ __forceinline__ void store8(T* row, int c, int n, int vec, const float (&v)[8]) {
  Raw8<T> r;
  round8(v, r);
  if (c + 8 <= n) {
    if (sizeof(T) == 4 && vec == 2) {
      const uint32_t* w = reinterpret_cast<const uint32_t*>(r.v);
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                   ::"l"(row + c), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]),
                     "r"(w[7]) : "memory");
    } else {
      uint4* p = reinterpret_cast<uint4*>(row + c);
#pragma unroll
      for (int i = 0; i < int(sizeof(T) / 2); ++i) p[i] = r.v[i];
    }
  } else {
    const T* e = reinterpret_cast<const T*>(r.v);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < n) row[c + i] = e[i];
  }
}
// The same, and without A for rows of any alignment, by a whole warp whose lanes hold
// consecutive pieces of 8 columns (lanes without columns pass n <= c).  Lane l
// stores the aligned 16-byte pieces that begin in its predecessor's elements
// and end in its own; the row's (and the warp's) first and last elements go
// one by one.
template <bool A, class T>
__device__ __forceinline__ void store8_any(T* row, int c, int n, int vec, const float (&v)[8]) {
  if (A) {
    store8(row, c, n, vec, v);
    return;
  }
  constexpr int kWords = 2 * int(sizeof(T)), kPer = 16 / int(sizeof(T));
  Raw8<T> r;
  round8(v, r);
  const uint32_t* own = reinterpret_cast<const uint32_t*>(r.v);
  uint32_t w[kWords + 5];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = __shfl_up_sync(0xffffffffu, own[kWords - 4 + i], 1);
#pragma unroll
  for (int i = 0; i < kWords; ++i) w[4 + i] = own[i];
  w[kWords + 4] = 0u;
  const int lane = threadIdx.x & 31;
  const uintptr_t at = reinterpret_cast<uintptr_t>(row + c);
  const uint32_t lead = uint32_t(at) & 15u;             // bytes from an aligned address to the first element
  const T* e = reinterpret_cast<const T*>(r.v);
  if (c + 8 > n) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < n) row[c + i] = e[i];
    return;
  }
  shift_down<kWords, sizeof(T) == 2>(w, 16u - lead);
  uint4* p = reinterpret_cast<uint4*>(at & ~uintptr_t(15));
#pragma unroll
  for (int i = 0; i < kWords / 4; ++i)
    if (i > 0 || lane > 0 || lead == 0)
      p[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  const int head = kPer - int(lead / sizeof(T));        // own elements in the first aligned piece
  if (lane == 0 && lead != 0) {
#pragma unroll
    for (int i = 0; i < kPer && i < 8; ++i)
      if (i < head) row[c + i] = e[i];
  }
  if (lane == 31 || c + 16 > n) {                       // no successor stores this lane's last elements
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i >= 8 - int(lead / sizeof(T))) row[c + i] = e[i];
  }
}
// Code rows are 16-byte aligned, so 8 codes at a multiple of 8 are one word pair.
__device__ __forceinline__ void load_codes8(const int8_t* row, int c, int n, uint2& w) {
  if (c + 8 <= n) {
    w = __ldg(reinterpret_cast<const uint2*>(row + c));
  } else {
    w = make_uint2(0u, 0u);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < n) (i < 4 ? w.x : w.y) |= uint32_t(uint8_t(row[c + i])) << (8 * (i & 3));
  }
}
__device__ __forceinline__ void store_codes8(int8_t* row, int c, int n, uint2 w) {
  if (c + 8 <= n) {
    *reinterpret_cast<uint2*>(row + c) = w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < n) row[c + i] = int8_t((i < 4 ? w.x : w.y) >> (8 * (i & 3)));
  }
}
// The 8 values code * s (one fp32 multiply each).  A code's byte with its
// sign bit flipped, under the exponent of 2^23, is the float 2^23 + 128 +
// code: cheaper than an integer conversion, and as exact.
__device__ __forceinline__ void values8(uint2 w, float s, float (&v)[8]) {
  const uint64_t s2 = pack2(s, s), off = pack2(-8388736.0f, -8388736.0f);
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const uint32_t b = (i < 4 ? w.x : w.y) ^ 0x80808080u;
    const float x0 = __uint_as_float(__byte_perm(b, 0x4B000000u, 0x7540 | (i & 3)));
    const float x1 = __uint_as_float(__byte_perm(b, 0x4B000000u, 0x7540 | ((i & 3) + 1)));
    unpack2(mul2(add2(pack2(x0, x1), off), s2), v[i], v[i + 1]);
  }
}

// Bits of |x|: as integers they order NaN above +Inf above every finite
// magnitude, so an integer maximum also tells a group with NaN or Inf.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }


// Over the group's lanes (a power of two, consecutive, aligned).
__device__ __forceinline__ uint32_t group_max(uint32_t m, int lanes) {
#pragma unroll
  for (int o = 1; o < 32; o *= 2)
    if (o < lanes) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
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
// The results of the pass enqueued before are there.
__device__ __forceinline__ void wait_for_pass() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

struct Mat {
  const void* p;
  int64_t ld;
  int32_t vec;       // see load8
};
struct Ckpt {
  int8_t* codes;
  int64_t ldc;
  float* scales;     // rows x groups, dense
  int32_t groups, shift;   // column c is in group c >> shift
};

// Pieces of rows as warps: blockDim = (32 wx, wy), blockIdx.x over rows,
// blockIdx.y over column pieces.  A thread takes ROWS rows, wy apart, whose
// loads it issues together.
template <int ROWS>
struct Piece {
  int64_t row;       // the first row
  int c;             // this lane's first column
  __device__ __forceinline__ explicit Piece(unsigned block_y = blockIdx.y) {
    row = int64_t(blockIdx.x) * (blockDim.y * ROWS) + threadIdx.y;
    c = int((block_y * (blockDim.x >> 5) + (threadIdx.x >> 5)) * kChunk + (threadIdx.x & 31) * 8);
  }
  __device__ __forceinline__ int64_t at(int u) const { return row + int64_t(u) * blockDim.y; }
};
dim3 piece_block(int64_t cols) {
  unsigned wx = 1;
  while (wx < kThreads / 32 && int64_t(wx) * kChunk < cols) wx *= 2;
  return dim3(32 * wx, kThreads / 32 / wx);
}
// Whether several rows per thread still leave every SM its 2048 threads.
bool many_pieces(int64_t rows, int64_t cols) { return rows * ((cols + 7) / 8) >= int64_t(4) * 148 * 2048; }
bool piece_grid(int64_t rows, int64_t cols, dim3 b, int rows_per_thread, dim3* g) {
  const int64_t per = int64_t(b.x / 32) * kChunk, rp = int64_t(b.y) * rows_per_thread;
  const int64_t gx = (rows + rp - 1) / rp, gy = (cols + per - 1) / per;
  if (gx > 0x7fffffffLL || gy > 65535) return false;
  *g = dim3(unsigned(gx), unsigned(gy));
  return true;
}

// ------------------------------------------------------------------ host

int64_t elt_size(int32_t dtype) { return dtype == ACT8_FP32 ? 4 : 2; }
bool dtype_ok(int32_t d) { return d == ACT8_FP32 || d == ACT8_BF16 || d == ACT8_FP16; }
bool group_ok(int32_t g) { return g == 0 || g == 32 || g == 64 || g == 128 || g == 256; }
// Column c lies in group c >> group_shift (rows have at most 2^30 columns).
int group_shift(int32_t group) {
  int s = 31;
  if (group)
    for (s = 5; (1 << s) < group; ++s) {}
  return s;
}
int64_t group_count(int64_t cols, int32_t group) { return group ? (cols + group - 1) / group : 1; }
bool shape_ok(int64_t rows, int64_t cols) {
  return rows >= 0 && cols >= 0 && rows <= kAct8MaxRows && cols <= kAct8MaxCols;
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
// 0: element-aligned rows only, 1: 16-byte aligned ones, 2: 32-byte.
int vec_of(const void* p, int64_t ld, int32_t dtype) {
  if (!row_aligned(p, ld, dtype)) return 0;
  return aligned(p, 32) && (ld * elt_size(dtype)) % 32 == 0 ? 2 : 1;
}
Mat mat(const void* p, int64_t ld, int32_t dtype) { return Mat{p, ld, vec_of(p, ld, dtype)}; }

Ckpt ckpt(const int8_t* codes, int64_t ldc, const float* scales, int64_t cols, int32_t group) {
  return Ckpt{const_cast<int8_t*>(codes), ldc, const_cast<float*>(scales), int32_t(group_count(cols, group)),
              group_shift(group)};
}

// Call f(std::true_type) or f(std::false_type).
template <class F>
shampoo4_status by_flag(bool b, F f) { return b ? f(std::true_type{}) : f(std::false_type{}); }

// Call f(T*) with a null pointer of the element type.
template <class F>
shampoo4_status by_dtype(int32_t dtype, F f) {
  if (dtype == ACT8_FP32) return f(static_cast<float*>(nullptr));
  if (dtype == ACT8_BF16) return f(static_cast<__nv_bfloat16*>(nullptr));
  return f(static_cast<__half*>(nullptr));
}

}  // namespace
}  // namespace s4

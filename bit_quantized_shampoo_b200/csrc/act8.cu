// 8-bit activation checkpoints: the codec, the gated activation that keeps
// its inputs in 8 bits, and the C entry points of the products in
// act8_gemm.cu.
//
// A group of columns of a row (or the whole row) holds a = max |x|, the
// scale s = fp32(a / 127) and, per element, the integer nearest to 127 x / a
// (ties to even).  The code is that of the exact quotient: the fast path
// multiplies by RN(127 / a), whose product is within 127 2^-23 < 2^-15 of
// the quotient, and an element that close to a border between two codes is
// decided by one double division (of two fp32 numbers a quotient that is not
// a tie lies at least 2^-26 away from it, far above a double's rounding).
//
// All kernels here stream: the bound is HBM bandwidth.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <algorithm>
#include "act8.h"
#include "plan.h"

namespace s4 {
namespace {

constexpr float kScaleMax = 8454659.0f * 0x1p98f;      // the largest s with 127 s finite in fp32
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

// ---- the code rule

// Bits of |x|: as integers they order NaN above +Inf above every finite
// magnitude, so an integer maximum also tells a group with NaN or Inf.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

struct Group {
  float a;        // max |x|
  float r;        // RN(127 / a); 0 where every code is 0
  float scale;
  bool fast;      // r normal: the fast path holds
  __device__ __forceinline__ explicit Group(uint32_t bits) {
    a = __uint_as_float(bits);
    const bool finite = bits < 0x7f800000u;
    scale = finite ? fminf(__fdiv_rn(a, 127.0f), kScaleMax) : (bits > 0x7f800000u ? __uint_as_float(0x7fc00000u) : a);
    fast = a >= 0x1p-118f || !finite || bits == 0u;
    r = (finite && bits != 0u && fast) ? __fdiv_rn(127.0f, a) : 0.0f;
  }
};

__device__ __noinline__ float code_exact(float x, float a) { return float(rint(127.0 * double(x) / double(a))); }

// The code of x as the low byte of the result.  A group without codes (zero
// or non-finite) has r = 0; x * 0 may be NaN there, hence the select.
__device__ __forceinline__ uint32_t code_of(float x, const Group& g) {
  constexpr float kMagic = 12582912.0f;                 // 1.5 2^23: adding it rounds to an integer, ties to even
  float t = fmaf(x, g.r, kMagic);
  const float d = fmaf(x, g.r, -(t - kMagic));
  if (!g.fast || fabsf(fabsf(d) - 0.5f) < 0x1p-15f) t = code_exact(x, g.a) + kMagic;
  return g.r == 0.0f && g.fast ? 0u : (__float_as_uint(t) & 0xffu);
}
template <class T>
__device__ __forceinline__ uint2 codes8(const Raw8<T>& r, const Group& g) {
  uint32_t b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) b[i] = code_of(elt(r, i), g);
  return make_uint2(b[0] | (b[1] << 8) | (b[2] << 16) | (b[3] << 24), b[4] | (b[5] << 8) | (b[6] << 16) | (b[7] << 24));
}
template <class T>
__device__ __forceinline__ uint32_t absmax8(const Raw8<T>& r) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, abs_bits(elt(r, i)));
  return m;
}
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

// ---- pack

template <class T>
__global__ void __launch_bounds__(kThreads) k_act8_pack_groups(Mat x, Ckpt o, int64_t rows, int64_t cols, int group) {
  const Piece p;
  if (p.row >= rows) return;                             // a whole warp
  Raw8<T> r;
  load8(static_cast<const T*>(x.p) + p.row * x.ld, p.c, cols, x.vec, r);
  const Group g(group_max(absmax8(r), group / 8));
  if (p.c >= cols) return;
  store_codes8(o.codes + p.row * o.ldc, p.c, cols, codes8(r, g));
  if (p.c % group == 0) o.scales[p.row * ((cols + group - 1) / group) + p.c / group] = g.scale;
}

// One scale for the row: a CTA per row.  IT > 0: the row (at most
// IT * 2048 columns) stays in registers between the maximum and the codes;
// IT = 0: it is read twice.
template <class T, int IT>
__global__ void __launch_bounds__(kThreads) k_act8_pack_rows(Mat x, Ckpt o, int64_t rows, int64_t cols) {
  __shared__ uint32_t slots[kThreads / 32];
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const T* xr = static_cast<const T*>(x.p) + row * x.ld;
    int8_t* cr = o.codes + row * o.ldc;
    uint32_t m = 0;
    if (IT > 0) {
      Raw8<T> r[IT > 0 ? IT : 1];
#pragma unroll
      for (int i = 0; i < IT; ++i) load8(xr, (int64_t(i) * kThreads + threadIdx.x) * 8, cols, x.vec, r[i]);
#pragma unroll
      for (int i = 0; i < IT; ++i) m = max(m, absmax8(r[i]));
      const Group g(cta_max(m, slots));
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        const int64_t c = (int64_t(i) * kThreads + threadIdx.x) * 8;
        if (c < cols) store_codes8(cr, c, cols, codes8(r[i], g));
      }
      if (threadIdx.x == 0) o.scales[row] = g.scale;
    } else {
      Raw8<T> r;
      for (int64_t c = threadIdx.x * 8; c < cols; c += kThreads * 8) {
        load8(xr, c, cols, x.vec, r);
        m = max(m, absmax8(r));
      }
      const Group g(cta_max(m, slots));
      for (int64_t c = threadIdx.x * 8; c < cols; c += kThreads * 8) {
        load8(xr, c, cols, x.vec, r);
        store_codes8(cr, c, cols, codes8(r, g));
      }
      if (threadIdx.x == 0) o.scales[row] = g.scale;
    }
  }
}

// ---- unpack, and the bfloat16 parts the products take

template <class T>
__global__ void __launch_bounds__(kThreads) k_act8_unpack(Ckpt k, T* x, int64_t ldx, int vec, int64_t rows,
                                                          int64_t cols, int group, int64_t groups) {
  const Piece p;
  if (p.row >= rows || p.c >= cols) return;
  uint2 w;
  load_codes8(k.codes + p.row * k.ldc, p.c, cols, w);
  const float s = __ldg(k.scales + p.row * groups + (group ? p.c / group : 0));
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = code_at(w, i) * s;
  store8(x + p.row * ldx, p.c, cols, vec, v);
}

// v = hi + lo + O(2^-16 v): hi = RN(v), kept finite when v is (the residual
// of an infinite hi would be infinite too), lo = RN(v - hi).
__device__ __forceinline__ void split(float v, float& hi, float& lo) {
  constexpr float kMax = 3.38953139e38f;                 // the largest finite bfloat16
  hi = __bfloat162float(__float2bfloat16_rn(v));
  if (fabsf(hi) > kMax && fabsf(v) <= 3.402823466e38f) hi = copysignf(kMax, v);
  lo = v - hi;
}

__global__ void __launch_bounds__(kThreads) k_act8_expand(Ckpt k, __nv_bfloat16* hi, __nv_bfloat16* lo, int64_t ld,
                                                          int64_t rows, int64_t cols, int group, int64_t groups) {
  const Piece p;
  if (p.row >= rows || p.c >= cols) return;
  uint2 w;
  load_codes8(k.codes + p.row * k.ldc, p.c, cols, w);
  const float s = __ldg(k.scales + p.row * groups + (group ? p.c / group : 0));
  float h[8], l[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) split(code_at(w, i) * s, h[i], l[i]);
  store8(hi + p.row * ld, p.c, cols, true, h);
  if (lo) store8(lo + p.row * ld, p.c, cols, true, l);
}

template <class T>
__global__ void __launch_bounds__(kThreads) k_act8_split(Mat x, __nv_bfloat16* hi, __nv_bfloat16* lo, int64_t ld,
                                                         int64_t rows, int64_t cols) {
  const Piece p;
  if (p.row >= rows || p.c >= cols) return;
  Raw8<T> r;
  load8(static_cast<const T*>(x.p) + p.row * x.ld, p.c, cols, x.vec, r);
  float h[8], l[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) split(elt(r, i), h[i], l[i]);
  store8(hi + p.row * ld, p.c, cols, true, h);
  if (lo) store8(lo + p.row * ld, p.c, cols, true, l);
}

// ---- the gated activation

__device__ __forceinline__ float sigmoid(float x) { return __fdiv_rn(1.0f, 1.0f + expf(-x)); }

template <class T>
__device__ __forceinline__ void gated8(const Raw8<T>& g, const Raw8<T>& u, T* h, int64_t c, int64_t n, bool vec) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = elt(g, i);
    v[i] = x * sigmoid(x) * elt(u, i);
  }
  store8(h, c, n, vec, v);
}

template <class T>
__global__ void __launch_bounds__(kThreads)
k_act8_swiglu_groups(Mat gate, Mat up, T* h, int64_t ldh, int vech, Ckpt kg, Ckpt ku, int64_t rows, int64_t cols,
                     int group) {
  const Piece p;
  if (p.row >= rows) return;
  Raw8<T> g, u;
  load8(static_cast<const T*>(gate.p) + p.row * gate.ld, p.c, cols, gate.vec, g);
  load8(static_cast<const T*>(up.p) + p.row * up.ld, p.c, cols, up.vec, u);
  const Group gg(group_max(absmax8(g), group / 8)), gu(group_max(absmax8(u), group / 8));
  if (p.c >= cols) return;
  gated8(g, u, h + p.row * ldh, p.c, cols, vech);
  store_codes8(kg.codes + p.row * kg.ldc, p.c, cols, codes8(g, gg));
  store_codes8(ku.codes + p.row * ku.ldc, p.c, cols, codes8(u, gu));
  if (p.c % group == 0) {
    const int64_t s = p.row * ((cols + group - 1) / group) + p.c / group;
    kg.scales[s] = gg.scale;
    ku.scales[s] = gu.scale;
  }
}

// One scale per row: the row is read twice (the second time from L2).
template <class T>
__global__ void __launch_bounds__(kThreads)
k_act8_swiglu_rows(Mat gate, Mat up, T* h, int64_t ldh, int vech, Ckpt kg, Ckpt ku, int64_t rows, int64_t cols) {
  __shared__ uint32_t slots[kThreads / 32];
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const T* gr = static_cast<const T*>(gate.p) + row * gate.ld;
    const T* ur = static_cast<const T*>(up.p) + row * up.ld;
    Raw8<T> g, u;
    uint32_t mg = 0, mu = 0;
    for (int64_t c = threadIdx.x * 8; c < cols; c += kThreads * 8) {
      load8(gr, c, cols, gate.vec, g);
      load8(ur, c, cols, up.vec, u);
      mg = max(mg, absmax8(g));
      mu = max(mu, absmax8(u));
      gated8(g, u, h + row * ldh, c, cols, vech);
    }
    const Group gg(cta_max(mg, slots)), gu(cta_max(mu, slots));
    for (int64_t c = threadIdx.x * 8; c < cols; c += kThreads * 8) {
      load8(gr, c, cols, gate.vec, g);
      load8(ur, c, cols, up.vec, u);
      store_codes8(kg.codes + row * kg.ldc, c, cols, codes8(g, gg));
      store_codes8(ku.codes + row * ku.ldc, c, cols, codes8(u, gu));
    }
    if (threadIdx.x == 0) {
      kg.scales[row] = gg.scale;
      ku.scales[row] = gu.scale;
    }
  }
}

template <class T>
__global__ void __launch_bounds__(kThreads)
k_act8_swiglu_backward(Mat dh, Ckpt kg, Ckpt ku, T* dg, int64_t lddg, int vecg, T* du, int64_t lddu, int vecu,
                       int64_t rows, int64_t cols, int group, int64_t groups) {
  const Piece p;
  if (p.row >= rows || p.c >= cols) return;
  Raw8<T> d;
  uint2 wg, wu;
  load8(static_cast<const T*>(dh.p) + p.row * dh.ld, p.c, cols, dh.vec, d);
  load_codes8(kg.codes + p.row * kg.ldc, p.c, cols, wg);
  load_codes8(ku.codes + p.row * ku.ldc, p.c, cols, wu);
  const int64_t s = p.row * groups + (group ? p.c / group : 0);
  const float sg = __ldg(kg.scales + s), su = __ldg(ku.scales + s);
  float og[8], ou[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float g = code_at(wg, i) * sg, u = code_at(wu, i) * su, x = elt(d, i);
    const float sig = sigmoid(g);
    ou[i] = x * (g * sig);
    og[i] = x * u * (sig * fmaf(g, 1.0f - sig, 1.0f));
  }
  store8(dg + p.row * lddg, p.c, cols, vecg, og);
  store8(du + p.row * lddu, p.c, cols, vecu, ou);
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

shampoo4_status pack(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t ldx, int32_t group, Ckpt o,
                     cudaStream_t st) {
  if (rows == 0 || cols == 0) return SHAMPOO4_OK;
  const Mat m = mat(x, ldx, dtype);
  return by_dtype(dtype, [&](auto* tag) -> shampoo4_status {
    using T = std::remove_pointer_t<decltype(tag)>;
    if (group) {
      const dim3 b = piece_block(cols);
      dim3 g;
      if (!piece_grid(rows, cols, b, &g)) return SHAMPOO4_ERR_INVALID_ARG;
      k_act8_pack_groups<T><<<g, b, 0, st>>>(m, o, rows, cols, group);
    } else {
      const unsigned g = unsigned(std::min<int64_t>(rows, 0x7fffffff));
      if (cols <= 2048) k_act8_pack_rows<T, 1><<<g, kThreads, 0, st>>>(m, o, rows, cols);
      else if (cols <= 4096) k_act8_pack_rows<T, 2><<<g, kThreads, 0, st>>>(m, o, rows, cols);
      else if (cols <= 8192) k_act8_pack_rows<T, 4><<<g, kThreads, 0, st>>>(m, o, rows, cols);
      else if (cols <= 16384) k_act8_pack_rows<T, 8><<<g, kThreads, 0, st>>>(m, o, rows, cols);
      else k_act8_pack_rows<T, 0><<<g, kThreads, 0, st>>>(m, o, rows, cols);
    }
    S4_CUDA(cudaGetLastError());
    return SHAMPOO4_OK;
  });
}

// ---- the gradient products: operands to bfloat16 parts in the workspace

size_t round_up(size_t n, size_t a) { return (n + a - 1) / a * a; }

struct GradPlan {
  int dy_parts, code_parts;
  int64_t ld_dy, ld_code;
  size_t dy_bytes, code_bytes;   // per part
  size_t total;
};
// dy: tokens x out; codes: rows x inner.  A bfloat16 dy is one exact part; a
// fp32 or fp16 one takes two (fp16 exactly, fp32 to 2^-16).  The codes'
// values take two parts (to 2^-16), or one, to bfloat16's half step, when dy
// and the result are bfloat16: a rounding of each product's factor that is
// no larger than the result's own.
GradPlan grad_plan(int32_t dtype, int32_t result, int64_t tokens, int64_t out, int64_t code_rows, int64_t inner) {
  GradPlan p{};
  p.dy_parts = dtype == ACT8_BF16 ? 1 : 2;
  p.code_parts = dtype == ACT8_BF16 && result == ACT8_BF16 ? 1 : 2;
  p.ld_dy = int64_t(round_up(size_t(out), 8));
  p.ld_code = int64_t(round_up(size_t(inner), 8));
  p.dy_bytes = round_up(size_t(tokens) * p.ld_dy * 2, 256);
  p.code_bytes = round_up(size_t(code_rows) * p.ld_code * 2, 256);
  // room for a copy of dy whatever its alignment turns out to be
  p.total = p.dy_parts * p.dy_bytes + p.code_parts * p.code_bytes;
  return p;
}

shampoo4_status expand(const Ckpt& k, int64_t rows, int64_t cols, int32_t group, void* hi, void* lo, int64_t ld,
                       cudaStream_t st) {
  if (rows == 0 || cols == 0) return SHAMPOO4_OK;
  const dim3 b = piece_block(cols);
  dim3 g;
  if (!piece_grid(rows, cols, b, &g)) return SHAMPOO4_ERR_INVALID_ARG;
  k_act8_expand<<<g, b, 0, st>>>(k, static_cast<__nv_bfloat16*>(hi), static_cast<__nv_bfloat16*>(lo), ld, rows, cols,
                                 group, group_count(cols, group));
  S4_CUDA(cudaGetLastError());
  return SHAMPOO4_OK;
}

shampoo4_status split_mat(const void* x, int32_t dtype, int64_t ldx, int64_t rows, int64_t cols, void* hi, void* lo,
                          int64_t ld, cudaStream_t st) {
  if (rows == 0 || cols == 0) return SHAMPOO4_OK;
  const dim3 b = piece_block(cols);
  dim3 g;
  if (!piece_grid(rows, cols, b, &g)) return SHAMPOO4_ERR_INVALID_ARG;
  const Mat m = mat(x, ldx, dtype);
  return by_dtype(dtype, [&](auto* tag) -> shampoo4_status {
    using T = std::remove_pointer_t<decltype(tag)>;
    k_act8_split<T><<<g, b, 0, st>>>(m, static_cast<__nv_bfloat16*>(hi), static_cast<__nv_bfloat16*>(lo), ld, rows,
                                     cols);
    S4_CUDA(cudaGetLastError());
    return SHAMPOO4_OK;
  });
}

// Both gradients: dy (tokens x out) against expanded codes (code_rows x
// inner).  weight: Y[out, inner] = dy^T X; else Y[tokens, inner] = dy W.
shampoo4_status grad(bool weight, const void* dy, int32_t dtype, int64_t lddy, const Ckpt& k, int32_t group,
                     int64_t tokens, int64_t out, int64_t inner, const Act8Out& o, void* ws, size_t ws_bytes,
                     uint32_t* flags, cudaStream_t st) {
  const int64_t code_rows = weight ? tokens : out;
  const int64_t M = weight ? out : tokens;
  if (M == 0 || inner == 0) return SHAMPOO4_OK;
  if (code_rows == 0 && o.accumulate) return SHAMPOO4_OK;
  const GradPlan p = grad_plan(dtype, o.dtype, tokens, out, code_rows, inner);
  if (p.total > 0 && (!ws || !aligned(ws, 256))) return SHAMPOO4_ERR_INVALID_ARG;
  if (ws_bytes < p.total) return SHAMPOO4_ERR_WORKSPACE;
  char* w = static_cast<char*>(ws);
  Act8Parts a{dy, nullptr, lddy}, b{};
  if (dtype != ACT8_BF16 || !row_aligned(dy, lddy, dtype)) {
    a = Act8Parts{w, p.dy_parts == 2 ? w + p.dy_bytes : nullptr, p.ld_dy};
    S4_TRY(split_mat(dy, dtype, lddy, tokens, out, w, p.dy_parts == 2 ? w + p.dy_bytes : nullptr, p.ld_dy, st));
  }
  w += p.dy_parts * p.dy_bytes;
  b = Act8Parts{w, p.code_parts == 2 ? w + p.code_bytes : nullptr, p.ld_code};
  S4_TRY(expand(k, code_rows, inner, group, w, p.code_parts == 2 ? w + p.code_bytes : nullptr, p.ld_code, st));
  return launch_act8_gemm_bf16(a, weight ? 1 : 0, b, M, inner, code_rows, o, flags, st);
}

}  // namespace
}  // namespace s4

// ------------------------------------------------------------------ C ABI

using namespace s4;

extern "C" shampoo4_status act8_pack(const void* d_x, int32_t dtype, int64_t rows, int64_t cols, int64_t ldx,
                                     int32_t group, int8_t* d_codes, int64_t ldc, float* d_scales,
                                     shampoo4_stream_t stream) {
  if (!shape_ok(rows, cols) || !dtype_ok(dtype) || !group_ok(group)) return SHAMPOO4_ERR_INVALID_ARG;
  if (rows == 0 || cols == 0) return SHAMPOO4_OK;
  if (!mat_ok(d_x, dtype, rows, cols, ldx) || !codes_ok(d_codes, ldc, cols, d_scales)) return SHAMPOO4_ERR_INVALID_ARG;
  return pack(d_x, dtype, rows, cols, ldx, group, Ckpt{d_codes, ldc, d_scales}, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" shampoo4_status act8_unpack(const int8_t* d_codes, int64_t ldc, const float* d_scales, int64_t rows,
                                       int64_t cols, int32_t group, void* d_x, int32_t dtype, int64_t ldx,
                                       shampoo4_stream_t stream) {
  if (!shape_ok(rows, cols) || !dtype_ok(dtype) || !group_ok(group)) return SHAMPOO4_ERR_INVALID_ARG;
  if (rows == 0 || cols == 0) return SHAMPOO4_OK;
  if (!mat_ok(d_x, dtype, rows, cols, ldx) || !codes_ok(d_codes, ldc, cols, d_scales)) return SHAMPOO4_ERR_INVALID_ARG;
  const dim3 b = piece_block(cols);
  dim3 g;
  if (!piece_grid(rows, cols, b, &g)) return SHAMPOO4_ERR_INVALID_ARG;
  const Ckpt k{const_cast<int8_t*>(d_codes), ldc, const_cast<float*>(d_scales)};
  return by_dtype(dtype, [&](auto* tag) -> shampoo4_status {
    using T = std::remove_pointer_t<decltype(tag)>;
    k_act8_unpack<T><<<g, b, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
        k, static_cast<T*>(d_x), ldx, row_aligned(d_x, ldx, dtype), rows, cols, group, group_count(cols, group));
    S4_CUDA(cudaGetLastError());
    return SHAMPOO4_OK;
  });
}

static shampoo4_status check_product(int64_t tokens, int64_t out, int64_t inner) {
  if (!shape_ok(tokens, out) || inner < 0 || inner > kAct8MaxInner) return SHAMPOO4_ERR_INVALID_ARG;
  return SHAMPOO4_OK;
}

extern "C" shampoo4_status act8_matmul(const int8_t* d_xc, int64_t ldxc, const float* d_xs, const int8_t* d_wc,
                                       int64_t ldwc, const float* d_ws, const float* d_bias, int64_t tokens,
                                       int64_t out, int64_t inner, void* d_y, int32_t dtype, int64_t ldy,
                                       uint32_t* d_flags, shampoo4_stream_t stream) {
  S4_TRY(check_product(tokens, out, inner));
  if (!dtype_ok(dtype)) return SHAMPOO4_ERR_INVALID_ARG;
  if (tokens == 0 || out == 0) return SHAMPOO4_OK;
  if (!mat_ok(d_y, dtype, tokens, out, ldy) || !aligned(d_bias, 4) || !aligned(d_flags, 4))
    return SHAMPOO4_ERR_INVALID_ARG;
  if (inner > 0 && (!codes_ok(d_xc, ldxc, inner, d_xs) || !codes_ok(d_wc, ldwc, inner, d_ws)))
    return SHAMPOO4_ERR_INVALID_ARG;
  // no columns: no group, so no scale either
  const Act8Out o{d_y, ldy, dtype, 0, inner > 0 ? d_xs : nullptr, inner > 0 ? d_ws : nullptr, d_bias};
  return launch_act8_gemm_i8(d_xc, ldxc, d_wc, ldwc, tokens, out, inner, o, d_flags,
                             reinterpret_cast<cudaStream_t>(stream));
}

extern "C" shampoo4_status act8_linear(const void* d_x, int32_t xdtype, int64_t ldx, const int8_t* d_wc, int64_t ldwc,
                                       const float* d_ws, const float* d_bias, int64_t tokens, int64_t out,
                                       int64_t inner, int8_t* d_xc, int64_t ldxc, float* d_xs, void* d_y,
                                       int32_t ydtype, int64_t ldy, uint32_t* d_flags, shampoo4_stream_t stream) {
  S4_TRY(check_product(tokens, out, inner));
  if (!dtype_ok(xdtype) || !dtype_ok(ydtype)) return SHAMPOO4_ERR_INVALID_ARG;
  if (tokens == 0) return SHAMPOO4_OK;
  if (inner > 0 && (!mat_ok(d_x, xdtype, tokens, inner, ldx) || !codes_ok(d_xc, ldxc, inner, d_xs)))
    return SHAMPOO4_ERR_INVALID_ARG;
  if (out > 0 && (!mat_ok(d_y, ydtype, tokens, out, ldy) || !aligned(d_bias, 4) || !aligned(d_flags, 4) ||
                  (inner > 0 && !codes_ok(d_wc, ldwc, inner, d_ws))))
    return SHAMPOO4_ERR_INVALID_ARG;
  S4_TRY(act8_pack(d_x, xdtype, tokens, inner, ldx, 0, d_xc, ldxc, d_xs, stream));
  return act8_matmul(d_xc, ldxc, d_xs, d_wc, ldwc, d_ws, d_bias, tokens, out, inner, d_y, ydtype, ldy, d_flags,
                     stream);
}

extern "C" shampoo4_status act8_grad_workspace(int32_t weight, int32_t dtype, int32_t result, int64_t tokens,
                                               int64_t out, int64_t inner, size_t* bytes) {
  if (!bytes || !dtype_ok(dtype) || !dtype_ok(result) || !shape_ok(tokens, out) || !shape_ok(0, inner))
    return SHAMPOO4_ERR_INVALID_ARG;
  *bytes = grad_plan(dtype, result, tokens, out, weight ? tokens : out, inner).total;
  return SHAMPOO4_OK;
}

static shampoo4_status grad_call(bool weight, const void* d_dy, int32_t dtype, int64_t lddy, const int8_t* codes,
                                 int64_t ldc, const float* scales, int32_t group, int64_t tokens, int64_t out,
                                 int64_t inner, void* d_y, int32_t result, int64_t ldy, int32_t accumulate,
                                 void* d_ws, size_t ws_bytes, uint32_t* d_flags, shampoo4_stream_t stream) {
  if (!shape_ok(tokens, out) || !shape_ok(0, inner) || !dtype_ok(dtype) || !dtype_ok(result) || !group_ok(group))
    return SHAMPOO4_ERR_INVALID_ARG;
  const int64_t M = weight ? out : tokens, K = weight ? tokens : out;
  if (M == 0 || inner == 0) return SHAMPOO4_OK;
  if (!mat_ok(d_y, result, M, inner, ldy) || !aligned(d_flags, 4)) return SHAMPOO4_ERR_INVALID_ARG;
  if (K > 0 && (!mat_ok(d_dy, dtype, tokens, out, lddy) || !codes_ok(codes, ldc, inner, scales)))
    return SHAMPOO4_ERR_INVALID_ARG;
  const Act8Out o{d_y, ldy, result, accumulate ? 1 : 0, nullptr, nullptr, nullptr};
  return grad(weight, d_dy, dtype, lddy, Ckpt{const_cast<int8_t*>(codes), ldc, const_cast<float*>(scales)}, group,
              tokens, out, inner, o, d_ws, ws_bytes, d_flags, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" shampoo4_status act8_weight_grad(const void* d_dy, int32_t dtype, int64_t lddy, const int8_t* d_xc,
                                            int64_t ldxc, const float* d_xs, int32_t group, int64_t tokens,
                                            int64_t out, int64_t inner, void* d_dw, int32_t result, int64_t lddw,
                                            int32_t accumulate, void* d_workspace, size_t workspace_bytes,
                                            uint32_t* d_flags, shampoo4_stream_t stream) {
  return grad_call(true, d_dy, dtype, lddy, d_xc, ldxc, d_xs, group, tokens, out, inner, d_dw, result, lddw,
                   accumulate, d_workspace, workspace_bytes, d_flags, stream);
}

extern "C" shampoo4_status act8_input_grad(const void* d_dy, int32_t dtype, int64_t lddy, const int8_t* d_wc,
                                           int64_t ldwc, const float* d_ws, int64_t tokens, int64_t out,
                                           int64_t inner, void* d_dx, int32_t result, int64_t lddx,
                                           int32_t accumulate, void* d_workspace, size_t workspace_bytes,
                                           uint32_t* d_flags, shampoo4_stream_t stream) {
  return grad_call(false, d_dy, dtype, lddy, d_wc, ldwc, d_ws, 0, tokens, out, inner, d_dx, result, lddx, accumulate,
                   d_workspace, workspace_bytes, d_flags, stream);
}

extern "C" shampoo4_status act8_swiglu(const void* d_gate, int64_t ldg, const void* d_up, int64_t ldu, int32_t dtype,
                                       int64_t rows, int64_t cols, int32_t group, void* d_h, int64_t ldh,
                                       int8_t* d_gate_codes, int64_t ldgc, float* d_gate_scales, int8_t* d_up_codes,
                                       int64_t lduc, float* d_up_scales, shampoo4_stream_t stream) {
  if (!shape_ok(rows, cols) || !dtype_ok(dtype) || !group_ok(group)) return SHAMPOO4_ERR_INVALID_ARG;
  if (rows == 0 || cols == 0) return SHAMPOO4_OK;
  if (!mat_ok(d_gate, dtype, rows, cols, ldg) || !mat_ok(d_up, dtype, rows, cols, ldu) ||
      !mat_ok(d_h, dtype, rows, cols, ldh) || !codes_ok(d_gate_codes, ldgc, cols, d_gate_scales) ||
      !codes_ok(d_up_codes, lduc, cols, d_up_scales))
    return SHAMPOO4_ERR_INVALID_ARG;
  const dim3 b = piece_block(cols);
  dim3 g;
  if (!piece_grid(rows, cols, b, &g)) return SHAMPOO4_ERR_INVALID_ARG;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const Ckpt kg{d_gate_codes, ldgc, d_gate_scales}, ku{d_up_codes, lduc, d_up_scales};
  const int vh = row_aligned(d_h, ldh, dtype);
  return by_dtype(dtype, [&](auto* tag) -> shampoo4_status {
    using T = std::remove_pointer_t<decltype(tag)>;
    if (group)
      k_act8_swiglu_groups<T><<<g, b, 0, st>>>(mat(d_gate, ldg, dtype), mat(d_up, ldu, dtype), static_cast<T*>(d_h),
                                               ldh, vh, kg, ku, rows, cols, group);
    else
      k_act8_swiglu_rows<T><<<unsigned(std::min<int64_t>(rows, 0x7fffffff)), kThreads, 0, st>>>(
          mat(d_gate, ldg, dtype), mat(d_up, ldu, dtype), static_cast<T*>(d_h), ldh, vh, kg, ku, rows, cols);
    S4_CUDA(cudaGetLastError());
    return SHAMPOO4_OK;
  });
}

extern "C" shampoo4_status act8_swiglu_backward(const void* d_dh, int64_t lddh, int32_t dtype,
                                                const int8_t* d_gate_codes, int64_t ldgc, const float* d_gate_scales,
                                                const int8_t* d_up_codes, int64_t lduc, const float* d_up_scales,
                                                int64_t rows, int64_t cols, int32_t group, void* d_dgate,
                                                int64_t lddg, void* d_dup, int64_t lddu, shampoo4_stream_t stream) {
  if (!shape_ok(rows, cols) || !dtype_ok(dtype) || !group_ok(group)) return SHAMPOO4_ERR_INVALID_ARG;
  if (rows == 0 || cols == 0) return SHAMPOO4_OK;
  if (!mat_ok(d_dh, dtype, rows, cols, lddh) || !mat_ok(d_dgate, dtype, rows, cols, lddg) ||
      !mat_ok(d_dup, dtype, rows, cols, lddu) || !codes_ok(d_gate_codes, ldgc, cols, d_gate_scales) ||
      !codes_ok(d_up_codes, lduc, cols, d_up_scales))
    return SHAMPOO4_ERR_INVALID_ARG;
  const dim3 b = piece_block(cols);
  dim3 g;
  if (!piece_grid(rows, cols, b, &g)) return SHAMPOO4_ERR_INVALID_ARG;
  const Ckpt kg{const_cast<int8_t*>(d_gate_codes), ldgc, const_cast<float*>(d_gate_scales)};
  const Ckpt ku{const_cast<int8_t*>(d_up_codes), lduc, const_cast<float*>(d_up_scales)};
  return by_dtype(dtype, [&](auto* tag) -> shampoo4_status {
    using T = std::remove_pointer_t<decltype(tag)>;
    k_act8_swiglu_backward<T><<<g, b, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
        mat(d_dh, lddh, dtype), kg, ku, static_cast<T*>(d_dgate), lddg, row_aligned(d_dgate, lddg, dtype),
        static_cast<T*>(d_dup), lddu, row_aligned(d_dup, lddu, dtype), rows, cols, group, group_count(cols, group));
    S4_CUDA(cudaGetLastError());
    return SHAMPOO4_OK;
  });
}

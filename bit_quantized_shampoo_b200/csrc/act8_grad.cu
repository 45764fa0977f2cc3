// Gradients of the 8-bit product, Y = X W^T:
//
//   act8_weight_grad   dW[o, i] = sum_t dY[t, o] sx[t] xc[t, i]
//   act8_input_grad    dX[t, i] = sum_o dY[t, o] sw[o] wc[o, i]
//
// The scale belongs to the contraction index, so it has to go into a factor.
// Three ways, chosen by the scales, types and sizes (grad_path):
//
//  digits  One scale per row of codes.  F = dY * scale in fp32 becomes fixed
//          point relative to its largest magnitude over the contraction,
//          q = rint(F * Q / max|F|), Q just below 127 (65536 + 256 + 1), in
//          three signed base-256 digits; the codes stay as they are stored.  Three
//          int8 products with exact int32 sums: the only error is q's
//          rounding (half of max|F| / 2^23 per element) and a few fp32
//          roundings at the end.  1.5 times a bfloat16 product's tensor-core
//          time, against three times for operands split into bfloat16 parts.
//  halves  Scales per group of columns (no common factor per row): each column
//          of dY and each group of the values' columns scaled by a power of
//          two (its largest over the contraction to about 2^14) and taken
//          as a half and a half of what is left, 22 bits and never coarser
//          than 2^-39 of that largest; a 16-bit dY is one half, and so is a
//          value for a bfloat16 result of a bfloat16 dY (2^-11, an eighth of
//          the result's own rounding; as one bfloat16 it would add as much
//          again).  Three products (two, one), summed in fp32 outside the
//          tensor core every 256 k (one: every 1024).  (Three bfloat16
//          parts each, six products, measured 47 us where this took 32 at
//          1537 x 768 x 2305 fp32.)  Also with one scale per row, for a large
//          bfloat16 weight gradient.
//  row     The large bfloat16 input gradient of a bfloat16 dY: F = dY * scale,
//  halves  each row scaled by a power of two (its largest to about 2^14), as
//          one half (2^-11, never coarser than 2^-39 of the row's largest),
//          the codes as halves as they are: one product.
//
// The operand passes of this file stream; their bound is HBM bandwidth.
#include <cooperative_groups.h>
#include "act8_elt.cuh"
#include "quant4.cuh"

namespace cg = cooperative_groups;

namespace s4 {
namespace {

// A little below 127 * 65536 + 127 * 256 + 127 = 8355711, the largest number
// of three digits: no rounding of F * inv passes it.
constexpr float kQMax = 8355704.0f;
constexpr float kTiny = 0x1p-100f;                     // below it the fixed point stays that of kTiny

// Fixed point of a row whose largest magnitude has these bits: the factor to
// q and the scale back, NaN for a row that holds a NaN or an infinity.
struct Fixed {
  float inv, scale;
  __device__ __forceinline__ explicit Fixed(uint32_t bits) {
    const bool finite = bits < 0x7f800000u;
    const float a = fmaxf(__uint_as_float(bits), kTiny);
    inv = finite ? __fdiv_rn(kQMax, a) : 0.0f;
    scale = finite ? __fdiv_rn(a, kQMax) : __uint_as_float(0x7fc00000u);
  }
};
// The three digits of f * inv as the low bytes, least significant first (a
// NaN, from inv = 0 and an infinity, converts to 0).
__device__ __forceinline__ uint32_t digits_of(float f, float inv) {
  return uint32_t(__float2int_rn(f * inv) + 0x808080) ^ 0x808080u;
}

// Byte `b` of four words, the first word's in the low byte.
__device__ __forceinline__ uint32_t bytes4(uint32_t x0, uint32_t x1, uint32_t x2, uint32_t x3, int b) {
  const uint32_t sel = uint32_t(b | ((4 + b) << 4));
  return __byte_perm(__byte_perm(x0, x1, sel), __byte_perm(x2, x3, sel), 0x5410);
}

// Scales c .. c + 7 of n, zeros past the end.
__device__ __forceinline__ void scales8(const float* s, int c, int n, bool vec, float (&v)[8]) {
  if (vec && c + 8 <= n) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(s + c)), b = __ldg(reinterpret_cast<const float4*>(s + c + 4));
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < n ? __ldg(s + c + i) : 0.0f;
  }
}
// Rows of dY as they are (act8_input_grad): a CTA per row, or a warp per row
// of up to 1024 columns, read twice (the second time from cache).  8192 x 4096
// fp16: 37 us, 4.5 TB/s of dY read once and the digits written.
template <class T, bool WARP, bool A>
__global__ void __launch_bounds__(kThreads)
k_act8_digit_rows(Mat dy, const float* __restrict__ scale, int8_t* digits, int64_t ld, float* row_scale, int64_t rows,
                  int cols) {
  let_next_start();
  __shared__ uint32_t slots[kThreads / 32];
  const int64_t row = WARP ? int64_t(blockIdx.x) * blockDim.y + threadIdx.y : int64_t(blockIdx.x);
  if (row >= rows) return;                               // a whole warp, or nobody
  const T* x = static_cast<const T*>(dy.p) + row * dy.ld;
  const int step = int(blockDim.x) * 8;
  const bool vec = (reinterpret_cast<uintptr_t>(scale) & 15) == 0;
  Raw8<T> r;
  float s[8];
  uint32_t m = 0;
#pragma unroll 2
  for (int c = int(threadIdx.x) * 8; c < cols; c += step) {   // past the last column: 0 * 0
    load8<A>(x, c, cols, dy.vec, r);
    scales8(scale, c, cols, vec, s);
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = elt(r, i) * s[i];
    const float a = absmax3_nan(y[0], y[1], y[2]), b = absmax3_nan(y[3], y[4], y[5]);
    m = max(m, abs_bits(max2_nan(absmax3_nan(a, y[6], y[7]), b)));
  }
  if (WARP) __syncwarp();
  const Fixed f(WARP ? __reduce_max_sync(0xffffffffu, m) : cta_max(m, slots));
  if (threadIdx.x == 0) row_scale[row] = f.scale;
  for (int c = int(threadIdx.x) * 8; c < ld; c += step) {               // ld: the padding gets zeros
    load8<A>(x, c, cols, dy.vec, r);
    scales8(scale, c, cols, vec, s);
    uint32_t q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = digits_of(elt(r, i) * s[i], f.inv);
#pragma unroll
    for (int d = 0; d < kAct8Digits; ++d) {
      const int b = kAct8Digits - 1 - d;
      *reinterpret_cast<uint2*>(digits + (d * rows + row) * ld + c) =
          make_uint2(bytes4(q[0], q[1], q[2], q[3], b), bytes4(q[4], q[5], q[6], q[7], b));
    }
  }
}

// Columns of dY as rows of digits (act8_weight_grad): a cluster of up to 8
// CTAs (gridDim.y) per 64 columns, tiles of 128 tokens dealt round robin.  The first sweep finds
// the columns' largest magnitudes (joined over distributed shared memory),
// the second quantizes and transposes through shared memory, so that every
// digit row is written in pieces of 128 bytes.  A thread holds 4 tokens by 8
// columns of a tile.  Bound by issue slots (60% busy) and shared memory as
// much as by HBM: 8192 x 4096 bf16 49 us, 3.4 TB/s of dY and digits.
constexpr int kColTile = 64, kTokTile = 128, kColCluster = 8, kMaxParts = 8;
template <class T, bool A>
__global__ void __launch_bounds__(kThreads, 4)
k_act8_digit_columns(Mat dy, const float* __restrict__ scale, int8_t* digits, int64_t ld, float* row_scale,
                     int64_t tokens, int64_t cols) {
  let_next_start();
  constexpr int kPitch = kTokTile / 4 + 1;              // words
  __shared__ uint32_t colmax[kColTile];
  __shared__ uint32_t tile[kAct8Digits][kColTile][kPitch];
  cg::cluster_group cluster = cg::this_cluster();
  const int64_t n0 = int64_t(blockIdx.x) * kColTile;
  const int cgrp = threadIdx.x & 7, tgrp = threadIdx.x >> 3;     // 8 columns, 4 tokens
  const int c = int(n0) + cgrp * 8;
  const int64_t ntiles = (tokens + kTokTile - 1) / kTokTile;
  const T* x = static_cast<const T*>(dy.p);
  if (threadIdx.x < kColTile) colmax[threadIdx.x] = 0;
  __syncthreads();

  // This thread's 4 tokens by 8 columns of tile tt, and the tokens' scales.
  const bool inside = A && c + 8 <= cols;
  auto fetch = [&](int64_t tt, Raw8<T> (&r)[4], float (&s)[4]) {
    const int64_t t0 = tt * kTokTile + tgrp * 4;
    const T* p = x + t0 * dy.ld;
    if (inside && t0 + 4 <= tokens) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint4* q = reinterpret_cast<const uint4*>(p + j * dy.ld + c);
#pragma unroll
        for (int k = 0; k < int(sizeof(T) / 2); ++k) r[j].v[k] = __ldg(q + k);
        s[j] = __ldg(scale + t0 + j);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        load8<A>(p + j * dy.ld, c, t0 + j < tokens ? int(cols) : 0, dy.vec, r[j]);
        s[j] = t0 + j < tokens ? __ldg(scale + t0 + j) : 0.0f;
      }
    }
  };
  uint32_t m[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) m[i] = 0;
  for (int64_t tt = blockIdx.y; tt < ntiles; tt += gridDim.y) {
    Raw8<T> r[4];
    float s[4];
    fetch(tt, r, s);
    // the maximum of magnitudes, NaN above all: |dy s| by pairs of tokens
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = max2_nan(fabsf(elt(r[0], i) * s[0]), fabsf(elt(r[1], i) * s[1]));
      m[i] = max(m[i], abs_bits(absmax3_nan(a, elt(r[2], i) * s[2], elt(r[3], i) * s[3])));
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {                         // over the warp's 4 token groups, then the CTA
    m[i] = max(m[i], __shfl_xor_sync(0xffffffffu, m[i], 8));
    m[i] = max(m[i], __shfl_xor_sync(0xffffffffu, m[i], 16));
    if ((threadIdx.x & 24) == 0) atomicMax(&colmax[cgrp * 8 + i], m[i]);
  }
  uint32_t all = 0;
  if (gridDim.y > 1) {
    cluster.sync();
    if (threadIdx.x < kColTile)
      for (unsigned k = 0; k < gridDim.y; ++k) all = max(all, *cluster.map_shared_rank(&colmax[threadIdx.x], k));
    cluster.sync();                                     // everyone has read before anyone overwrites or leaves
  } else {
    __syncthreads();
    if (threadIdx.x < kColTile) all = colmax[threadIdx.x];
  }
  if (threadIdx.x < kColTile) {
    colmax[threadIdx.x] = all;
    if (blockIdx.y == 0 && n0 + threadIdx.x < cols) row_scale[n0 + threadIdx.x] = Fixed(all).scale;
  }
  __syncthreads();
  float inv[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) inv[i] = Fixed(colmax[cgrp * 8 + i]).inv;

  for (int64_t tt = blockIdx.y; tt < ntiles; tt += gridDim.y) {
    Raw8<T> r[4];
    float s[4];
    fetch(tt, r, s);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t q[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) q[j] = digits_of(elt(r[j], i) * s[j], inv[i]);
#pragma unroll
      for (int d = 0; d < kAct8Digits; ++d)
        tile[d][cgrp * 8 + i][tgrp] = bytes4(q[0], q[1], q[2], q[3], kAct8Digits - 1 - d);
    }
    __syncthreads();
    const int lane = threadIdx.x & 31;
    const int64_t t = tt * kTokTile + lane * 4;
    const int rows = int(min(int64_t(kColTile), cols - n0));
    if (t < ld) {                                       // ld is a multiple of 16: a word is inside or outside
#pragma unroll
      for (int d = 0; d < kAct8Digits; ++d) {
        int8_t* o = digits + (d * cols + n0) * ld + t;
        for (int n = threadIdx.x >> 5; n < rows; n += kThreads / 32)
          *reinterpret_cast<uint32_t*>(o + n * ld) = tile[d][n][lane];
      }
    }
    __syncthreads();
  }
}

// ---- halves

// Bits of the largest finite magnitudes (elements that are not finite do not
// count: they stay so whatever the factor) of each column of dY and of each
// group's scales: a cluster of up to 8 CTAs per 64 columns and part (of
// gridDim.y / cluster parts, which share the tiles of 128 tokens), joined in
// distributed shared memory; `words` gets a row of ldw per part, dY's columns
// first, the scales' from code_word on.  The grid's first dy_strips are dY's.
// 4096 x 4096 fp32 28 us, 8192 x 4096 bf16 30 to 37, under the next kernel's
// first loads from 20 us on.
__device__ __forceinline__ uint32_t finite_bits(float x) {
  const uint32_t b = abs_bits(x);
  return b < 0x7f800000u ? b : 0u;
}
template <bool A, class T>
__device__ __forceinline__ void column_maxima(const T* x, int64_t ld, int vec, int64_t rows, int cols, int c, int tgrp,
                                              uint32_t (&m)[8]) {
  const int64_t tiles = (rows + kTokTile - 1) / kTokTile;
  for (int64_t tt = blockIdx.y; tt < tiles; tt += gridDim.y) {
    const int64_t t0 = tt * kTokTile + tgrp * 4;
    Raw8<T> r[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) load8<A>(x + (t0 + j) * ld, c, t0 + j < rows ? cols : 0, vec, r[j]);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) m[i] = max(m[i], finite_bits(elt(r[j], i)));
  }
}
template <class T, bool A>
__global__ void __launch_bounds__(kThreads)
k_act8_largest(Mat dy, int cols, unsigned dy_strips, const float* __restrict__ scales, int groups, int64_t rows,
               uint32_t* words, int64_t ldw, int64_t code_word) {
  let_next_start();
  __shared__ uint32_t colmax[kColTile];
  cg::cluster_group cluster = cg::this_cluster();
  const bool codes = blockIdx.x >= dy_strips;
  const int n = codes ? groups : cols, n0 = int(codes ? blockIdx.x - dy_strips : blockIdx.x) * kColTile;
  const int cgrp = threadIdx.x & 7, tgrp = threadIdx.x >> 3;     // 8 columns, 4 tokens
  if (threadIdx.x < kColTile) colmax[threadIdx.x] = 0;
  __syncthreads();
  uint32_t m[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (codes) column_maxima<false>(scales, groups, 0, rows, n, n0 + cgrp * 8, tgrp, m);
  else column_maxima<A>(static_cast<const T*>(dy.p), dy.ld, dy.vec, rows, n, n0 + cgrp * 8, tgrp, m);
#pragma unroll
  for (int i = 0; i < 8; ++i) {                         // over the warp's 4 token groups, then the CTA
    m[i] = max(m[i], __shfl_xor_sync(0xffffffffu, m[i], 8));
    m[i] = max(m[i], __shfl_xor_sync(0xffffffffu, m[i], 16));
    if ((threadIdx.x & 24) == 0) atomicMax(&colmax[cgrp * 8 + i], m[i]);
  }
  const unsigned ctas = cluster.num_blocks();
  cluster.sync();
  if (cluster.block_rank() == 0 && threadIdx.x < kColTile) {
    uint32_t all = 0;
    for (unsigned k = 0; k < ctas; ++k) all = max(all, *cluster.map_shared_rank(&colmax[threadIdx.x], k));
    const int at = n0 + int(threadIdx.x);
    if (at < (n + 7) / 8 * 8) words[int64_t(blockIdx.y / ctas) * ldw + (codes ? code_word : 0) + at] = all;
  }
  cluster.sync();                                        // nobody leaves while its words are read
}

// The e with 2^13 < 2^e x < 2^15 for the x of these bits (0 for zero), within
// the exponents whose powers are normal.  (The bounds cost nothing: 2^126 x is
// a multiple of 2^-23, a half's smallest step is 2^-24.)
__device__ __forceinline__ int power_to(uint32_t bits) {
  return bits == 0u ? 0 : min(max(14 + 127 - int(bits >> 23), -126), 126);
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(uint32_t(127 + e) << 23); }
// A value's largest is its scale's 127-fold, 2^7 of it.
__device__ __forceinline__ int value_power(uint32_t scale_bits) {
  return power_to(scale_bits == 0u ? 0u : min(scale_bits + (7u << 23), 0x7f000000u));
}

// Rows of F = dY * scale as one half each, for act8_input_grad: a CTA per row,
// read twice (the second time from cache).  factor: what undoes a row's power.
// Bound by HBM and the second reading: 8192 x 11008 81 us, 4.5 TB/s of dY read
// once and the halves written.
template <bool A>
__global__ void __launch_bounds__(kThreads)
k_act8_row_halves(Mat dy, const float* __restrict__ scale, __half* o, int64_t ld, float* factor, int cols) {
  let_next_start();
  __shared__ uint32_t slots[kThreads / 32];
  const int64_t row = blockIdx.x;
  const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(dy.p) + row * dy.ld;
  const bool vec = (reinterpret_cast<uintptr_t>(scale) & 15) == 0;
  Raw8<__nv_bfloat16> r;
  float s[8];
  uint32_t m = 0;
#pragma unroll 2
  for (int c = int(threadIdx.x) * 8; c < cols; c += kThreads * 8) {   // past the last column: 0 * 0
    load8<A>(x, c, cols, dy.vec, r);
    scales8(scale, c, cols, vec, s);
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, finite_bits(elt(r, i) * s[i]));
  }
  const int e = power_to(cta_max(m, slots));
  if (threadIdx.x == 0) factor[row] = pow2(-e);
  const float power = pow2(e);
#pragma unroll 2
  for (int c = int(threadIdx.x) * 8; c < cols; c += kThreads * 8) {
    load8<A>(x, c, cols, dy.vec, r);
    scales8(scale, c, cols, vec, s);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = elt(r, i) * s[i] * power;
    store8(o + row * ld, c, cols, 1, v);
  }
}
// Codes as halves, exactly.  11008 x 4096: 28 us, 4.9 TB/s.
__global__ void __launch_bounds__(kThreads) k_act8_code_halves(Ckpt k, __half* o, int64_t ld, int64_t rows, int cols) {
  let_next_start();
  const Piece<4> p;
  if (p.row >= rows || p.c >= cols) return;
  uint2 w[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) load_codes8(k.codes + p.at(u) * k.ldc, p.c, p.at(u) < rows ? cols : 0, w[u]);
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    float v[8];
    values8(w[u], 1.0f, v);
    if (p.at(u) < rows) store8(o + p.at(u) * ld, p.c, cols, 1, v);
  }
  wait_for_pass();                       // nothing of it is read here, but the product relies on both
}

template <int PARTS>
__device__ __forceinline__ void store_halves(const float (&v)[8], const int (&e)[8], __half* o, int64_t plane, int c,
                                             int cols) {
  float hi[8], lo[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = v[i] * pow2(e[i]);
    hi[i] = __half2float(__float2half_rn(x));
    lo[i] = x - hi[i];
  }
  store8(o, c, cols, 1, hi);
  if (PARTS == 2) store8(o + plane, c, cols, 1, lo);
}

// Both operands in one launch: the first code_blocks of blockIdx.y the codes'
// values, the others dY.  A column of dY has its power of two and so has a
// group of the codes' columns, from the maxima; what undoes them goes to
// `factor` (dY's columns, then from code_word on the groups).  Bound by HBM:
// 4096 x 4096 codes and fp32 dY 48 us, 4.6 TB/s; 8192 x 11008 codes and
// 8192 x 4096 bf16, one half each, 90 us.
template <class T, int CODE_PARTS, int kRows, bool A>
__global__ void __launch_bounds__(kThreads)
k_act8_halves(Ckpt k, __half* co, int64_t ldco, int cols_c, Mat dy, __half* dyo, int64_t lddyo, int cols_dy,
              const uint32_t* words, int parts, int64_t ldw, int64_t code_word, float* factor, int64_t rows,
              unsigned code_blocks) {
  let_next_start();
  const bool codes = blockIdx.y < code_blocks;
  const Piece<kRows> p(codes ? blockIdx.y : blockIdx.y - code_blocks);
  if (p.row >= rows || p.c >= (codes ? cols_c : cols_dy)) return;
  constexpr int PARTS = sizeof(T) == 4 ? 2 : 1;
  int e[8];
  if (codes) {
    const int64_t group = p.c >> k.shift;
    uint2 w[kRows];
    float s[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int64_t row = p.at(u);
      load_codes8(k.codes + row * k.ldc, p.c, row < rows ? cols_c : 0, w[u]);
      s[u] = row < rows ? __ldg(k.scales + row * k.groups + group) : 0.0f;
    }
    wait_for_pass();
    uint32_t top = 0;
#pragma unroll 4
    for (int i = 0; i < parts; ++i) top = max(top, __ldcg(words + i * ldw + code_word + group));
    const int power = value_power(top);
    if (p.row == 0 && p.c == group << k.shift) factor[code_word + group] = pow2(-power);
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = power;
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int64_t row = p.at(u);
      float v[8];
      values8(w[u], s[u], v);
      if (row < rows) store_halves<CODE_PARTS>(v, e, co + row * ldco, rows * ldco, p.c, cols_c);
    }
  } else {
    Raw8<T> r[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u)
      load8<A>(static_cast<const T*>(dy.p) + p.at(u) * dy.ld, p.c, p.at(u) < rows ? cols_dy : 0, dy.vec, r[u]);
    wait_for_pass();
    uint32_t top[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 4
    for (int i = 0; i < parts; ++i) {
      const uint4* w = reinterpret_cast<const uint4*>(words + i * ldw + p.c);
      const uint4 a = w[0], b = w[1];
      top[0] = max(top[0], a.x), top[1] = max(top[1], a.y), top[2] = max(top[2], a.z), top[3] = max(top[3], a.w);
      top[4] = max(top[4], b.x), top[5] = max(top[5], b.y), top[6] = max(top[6], b.z), top[7] = max(top[7], b.w);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      e[i] = power_to(top[i]);
      if (p.row == 0 && p.c + i < cols_dy) factor[p.c + i] = pow2(-e[i]);
    }
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int64_t row = p.at(u);
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = elt(r[u], i);
      if (row < rows) store_halves<PARTS>(v, e, dyo + row * lddyo, rows * lddyo, p.c, cols_dy);
    }
  }
}

// The shares' sums, added in order, into the result (512 x 512: 4.6 us).
template <class T>
__global__ void __launch_bounds__(kThreads) k_act8_join(const float* __restrict__ sums, int shares, T* y, int64_t ldy,
                                                        int accumulate, int64_t rows, int cols) {
  const int64_t n = rows * cols;
  for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < n; i += int64_t(gridDim.x) * kThreads) {
    float v = __ldg(sums + i);
    for (int k = 1; k < shares; ++k) v += __ldg(sums + k * n + i);
    T* p = y + i / cols * ldy + i % cols;
    if (accumulate) v += float(*p);
    *p = T(v);
  }
}

// ------------------------------------------------------------------ host

// One scale per row, dY and the result bfloat16: one product of halves, where
// digits take half as long again per row of the result but need no copy of the
// codes; and only on 256 x 256 tiles.  So it wants rows (input gradient, 11008
// inner, 4096 of contraction: 1500 rows 130 us, digits 128; 2048 rows 155, 169)
// and tiles (three per pair of CTAs; 2048 x 3200, 11008 of contraction, 104
// tiles: 163, 157).  The result is the exact one rounded, either way.
enum GradPath { kDigits, kHalves, kRowHalves };
GradPath grad_path(bool weight, int32_t dtype, int32_t result, int32_t group, int64_t rows, int64_t inner) {
  if (group) return kHalves;
  const bool many = rows >= 2048 && ((rows + 255) / 256) * ((inner + 255) / 256) >= 222;
  if (dtype != ACT8_BF16 || result != ACT8_BF16 || !many) return kDigits;
  return weight ? kHalves : kRowHalves;
}

size_t round_up(size_t n, size_t a) { return (n + a - 1) / a * a; }

// Workspace of a gradient: scales (digits) or the result's factors and the
// largest magnitudes (halves), dY (tokens x out) in the form its product takes,
// then, but for digits, the codes' values (code_rows x inner) in 16 bits.
struct GradPlan {
  GradPath path;
  int dy_parts, code_parts;      // halves of an element
  int64_t ld_dy, ld_code;        // elements
  size_t scale_bytes, dy_bytes, code_bytes;
  unsigned ctas, parts;          // halves: the search's clusters, and how many share a strip of columns
  int64_t code_word, ldw;        // of a row of maxima, and of the factors: the first group's, and the length
  int shares;                    // halves: parts of the contraction, and room for their sums
  size_t sum_bytes;
  int64_t dy_strips() const { return (code_word + kColTile - 1) / kColTile; }
  int64_t strips() const { return dy_strips() + (ldw - code_word + kColTile - 1) / kColTile; }
  size_t total() const { return scale_bytes + dy_bytes + code_bytes + sum_bytes; }
};
GradPlan grad_plan(bool weight, int32_t dtype, int32_t result, int32_t group, int64_t tokens, int64_t out,
                   int64_t inner) {
  GradPlan p{};
  p.path = grad_path(weight, dtype, result, group, weight ? out : tokens, inner);
  if (p.path == kDigits) {
    const int64_t rows = weight ? out : tokens, k = weight ? tokens : out;
    p.ld_dy = int64_t(round_up(size_t(k), 16));
    p.scale_bytes = round_up(size_t(rows) * 4, 256);
    p.dy_bytes = round_up(size_t(rows) * p.ld_dy * kAct8Digits, 256);
    return p;
  }
  p.dy_parts = dtype == ACT8_FP32 ? 2 : 1;
  p.code_parts = dtype == ACT8_BF16 && result == ACT8_BF16 ? 1 : 2;
  if (p.path == kRowHalves) {
    p.scale_bytes = round_up(size_t(tokens) * 4, 256);
    p.ld_dy = int64_t(round_up(size_t(out), 8));
    p.ld_code = int64_t(round_up(size_t(inner), 8));
    p.dy_bytes = round_up(size_t(tokens) * p.ld_dy * 2, 256);
    p.code_bytes = round_up(size_t(out) * p.ld_code * 2, 256);
    return p;
  }
  p.code_word = int64_t(round_up(size_t(out), 8));
  p.ldw = p.code_word + int64_t(round_up(size_t(group_count(inner, group)), 8));
  // Enough clusters for every SM's 2048 threads, as far as there are tiles.
  // (65536 x 64: 10.5 us in 8 parts; 16 take 7.9, but the next pass, which
  // reads a row of maxima per part, 12 more.)
  const int64_t tiles = (tokens + kTokTile - 1) / kTokTile, strips = p.strips();
  p.ctas = 1;
  while (p.ctas < kColCluster && int64_t(p.ctas) < tiles) p.ctas *= 2;
  p.parts = unsigned(std::max<int64_t>(1, std::min<int64_t>({kMaxParts, 148 * 8 / (strips * p.ctas), tiles / p.ctas})));
  p.scale_bytes = round_up(size_t(p.parts + 1) * size_t(p.ldw) * 4, 256);
  p.ld_dy = int64_t(round_up(size_t(out), 8));
  p.ld_code = int64_t(round_up(size_t(inner), 8));
  p.dy_bytes = round_up(size_t(tokens) * p.ld_dy * 2 * p.dy_parts, 256);
  p.code_bytes = round_up(size_t(tokens) * p.ld_code * 2 * p.code_parts, 256);
  p.shares = p.code_parts == 2 ? act8_halves_shares(inner, out, tokens) : 1;
  p.sum_bytes = p.shares > 1 ? round_up(size_t(p.shares) * out * inner * 4, 256) : 0;
  return p;
}

// after_pass: the kernel enqueued just before is this call's own pass; this
// one may start under it and waits for it itself.
template <class... P, class... A>
shampoo4_status start(void (*kern)(P...), dim3 grid, dim3 block, dim3 cluster, bool after_pass, cudaStream_t st,
                      A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  unsigned n = 0;
  if (cluster.x * cluster.y > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = cluster.x;
    attr[n].val.clusterDim.y = cluster.y;
    attr[n++].val.clusterDim.z = 1;
  }
  if (after_pass) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  S4_CUDA(cudaLaunchKernelEx(&cfg, kern, P(args)...));
  return SHAMPOO4_OK;
}

shampoo4_status digit_pass(bool weight, const void* dy, int32_t dtype, int64_t lddy, const float* scale,
                           int64_t tokens, int64_t out, int8_t* digits, int64_t ld, float* row_scale,
                           cudaStream_t st) {
  const Mat m = mat(dy, lddy, dtype);
  const int64_t strips = (out + kColTile - 1) / kColTile;
  return by_dtype(dtype, [&](auto* tag) { return by_flag(m.vec != 0, [&](auto flag) -> shampoo4_status {
    using T = std::remove_pointer_t<decltype(tag)>;
    constexpr bool A = decltype(flag)::value;
    if (weight) {
      unsigned ctas = 1;                                // per strip: no more than it has tiles
      while (ctas < kColCluster && int64_t(ctas) * kTokTile < tokens) ctas *= 2;
      return start(k_act8_digit_columns<T, A>, dim3(unsigned(strips), ctas), dim3(kThreads), dim3(1, ctas), false, st,
                   m, scale, digits, ld, row_scale, tokens, out);
    } else {
      if (out <= 1024)
        k_act8_digit_rows<T, true, A><<<unsigned((tokens + 7) / 8), dim3(32, 8), 0, st>>>(m, scale, digits, ld, row_scale,
                                                                                      tokens, int(out));
      else
        k_act8_digit_rows<T, false, A><<<unsigned(tokens), kThreads, 0, st>>>(m, scale, digits, ld, row_scale, tokens,
                                                                          int(out));
      S4_CUDA(cudaGetLastError());
    }
    return SHAMPOO4_OK;
  }); });
}

// dY * scale in rows of halves at dyp, the codes as halves at cp.
shampoo4_status row_halves_pass(const void* dy, int64_t lddy, const Ckpt& k, int64_t tokens, int64_t out,
                                int64_t inner, const GradPlan& p, float* factor, void* dyp, void* cp,
                                cudaStream_t st) {
  const Mat m = mat(dy, lddy, ACT8_BF16);
  const dim3 b = piece_block(inner);
  dim3 g;
  if (!piece_grid(out, inner, b, 4, &g)) return SHAMPOO4_ERR_INVALID_ARG;
  S4_TRY(start(m.vec ? k_act8_row_halves<true> : k_act8_row_halves<false>, dim3(unsigned(tokens)), dim3(kThreads),
               dim3(1), false, st, m, k.scales, static_cast<__half*>(dyp), p.ld_dy, factor, int(out)));
  return start(k_act8_code_halves, g, b, dim3(1), true, st, k, static_cast<__half*>(cp), p.ld_code, out, int(inner));
}

// Both operands as halves at dyp and cp, and the result's factors.
shampoo4_status halves_pass(const void* dy, int32_t dtype, int64_t lddy, const Ckpt& k, int64_t tokens, int64_t out,
                            int64_t inner, const GradPlan& p, float* factor, void* dyp, void* cp, cudaStream_t st) {
  const Mat m = mat(dy, lddy, dtype);
  const dim3 b = piece_block(std::max(out, inner));
  // Four rows per thread, which share the reading of the maxima, where that
  // leaves every SM its 64 warps (a warp takes 256 columns of a row, however
  // few there are: two operands of 65536 x 64 take 30 us, 50 with a row per
  // thread).
  const bool many = tokens * ((out + kChunk - 1) / kChunk + (inner + kChunk - 1) / kChunk) >= int64_t(4) * 148 * 64;
  dim3 g, gc;
  if (!piece_grid(tokens, out, b, many ? 4 : 1, &g) || !piece_grid(tokens, inner, b, many ? 4 : 1, &gc) ||
      g.y + gc.y > 65535)
    return SHAMPOO4_ERR_INVALID_ARG;
  g.y += gc.y;
  uint32_t* words = reinterpret_cast<uint32_t*>(factor + p.ldw);
  return by_dtype(dtype, [&](auto* tag) { return by_flag(m.vec != 0, [&](auto flag) -> shampoo4_status {
    using T = std::remove_pointer_t<decltype(tag)>;
    constexpr bool A = decltype(flag)::value;
    S4_TRY(start(k_act8_largest<T, A>, dim3(unsigned(p.strips()), p.ctas * p.parts), dim3(kThreads), dim3(1, p.ctas),
                 false, st, m, int(out), unsigned(p.dy_strips()), k.scales, k.groups, tokens, words, p.ldw,
                 p.code_word));
    const auto kern = p.code_parts == 1 ? (many ? k_act8_halves<T, 1, 4, A> : k_act8_halves<T, 1, 1, A>)
                                        : (many ? k_act8_halves<T, 2, 4, A> : k_act8_halves<T, 2, 1, A>);
    return start(kern, g, b, dim3(1), true, st, k, static_cast<__half*>(cp), p.ld_code, int(inner), m,
                 static_cast<__half*>(dyp), p.ld_dy, int(out), words, int(p.parts), p.ldw, p.code_word, factor, tokens,
                 gc.y);
  }); });
}

}  // namespace

shampoo4_status act8_grad_check(const Act8Grad& g, size_t* bytes) {
  *bytes = 0;
  if (!shape_ok(g.tokens, g.out) || !shape_ok(0, g.inner) || !dtype_ok(g.dtype) || !dtype_ok(g.result) ||
      !group_ok(g.group))
    return SHAMPOO4_ERR_INVALID_ARG;
  const int64_t M = g.weight ? g.out : g.tokens, K = g.weight ? g.tokens : g.out;
  if (M == 0 || g.inner == 0) return SHAMPOO4_OK;
  if (!mat_ok(g.y, g.result, M, g.inner, g.ldy)) return SHAMPOO4_ERR_INVALID_ARG;
  if (K == 0) return SHAMPOO4_OK;
  if (!mat_ok(g.dy, g.dtype, g.tokens, g.out, g.lddy) || !codes_ok(g.codes, g.ldc, g.inner, g.scales))
    return SHAMPOO4_ERR_INVALID_ARG;
  *bytes = grad_plan(g.weight, g.dtype, g.result, g.group, g.tokens, g.out, g.inner).total();
  return SHAMPOO4_OK;
}

// weight: Y[out, inner] = dY^T X; else Y[tokens, inner] = dY W.
shampoo4_status act8_grad_run(const Act8Grad& g, void* ws, Act8Watch watch, cudaStream_t st) {
  const bool weight = g.weight;
  const int64_t tokens = g.tokens, out = g.out, inner = g.inner;
  const int64_t K = weight ? tokens : out, R = weight ? out : tokens;
  if (R == 0 || inner == 0 || (K == 0 && g.accumulate)) return SHAMPOO4_OK;
  Act8Out o{g.y, g.ldy, g.result, g.accumulate ? 1 : 0, nullptr, nullptr, nullptr, 0};
  if (K == 0) return launch_act8_codes(Act8Operand{}, Act8Operand{}, inner, R, 0, o, false, watch, st);   // zeros
  const GradPlan p = grad_plan(weight, g.dtype, g.result, g.group, tokens, out, inner);
  const Ckpt k = ckpt(g.codes, g.ldc, g.scales, inner, g.group);
  char* w = static_cast<char*>(ws);
  if (p.path == kDigits) {
    float* row_scale = reinterpret_cast<float*>(w);
    int8_t* digits = reinterpret_cast<int8_t*>(w + p.scale_bytes);
    S4_TRY(digit_pass(weight, g.dy, g.dtype, g.lddy, k.scales, tokens, out, digits, p.ld_dy, row_scale, st));
    o.row_scale = row_scale;
    return launch_act8_digits(Act8Operand{k.codes, k.ldc, 0}, Act8Operand{digits, p.ld_dy, R}, inner, R, K, o, watch,
                              st);
  }
  char *dyp = w + p.scale_bytes, *cp = dyp + p.dy_bytes;
  float* factor = reinterpret_cast<float*>(w);
  if (p.path == kRowHalves) {
    S4_TRY(row_halves_pass(g.dy, g.lddy, k, tokens, out, inner, p, factor, dyp, cp, st));
    o.row_scale = factor;
    return launch_act8_row_halves(Act8Operand{cp, p.ld_code, 0}, Act8Operand{dyp, p.ld_dy, 0}, inner, R, K, o, watch,
                                  st);
  }
  S4_TRY(halves_pass(g.dy, g.dtype, g.lddy, k, tokens, out, inner, p, factor, dyp, cp, st));
  o.row_scale = factor;
  o.col_scale = factor + p.code_word;
  o.col_shift = k.shift;
  const Act8Operand a{cp, p.ld_code, K}, b{dyp, p.ld_dy, tokens};
  if (p.shares == 1) return launch_act8_halves(a, p.code_parts, b, p.dy_parts, inner, R, K, 1, o, watch, st);
  float* sums = reinterpret_cast<float*>(cp + p.code_bytes);
  S4_TRY(launch_act8_halves(a, p.code_parts, b, p.dy_parts, inner, R, K, p.shares,
                            Act8Out{sums, inner, ACT8_FP32, 0, o.row_scale, o.col_scale, nullptr, o.col_shift}, watch, st));
  const unsigned ctas = unsigned(std::min<int64_t>((R * inner + kThreads - 1) / kThreads, 148 * 8));
  return by_dtype(o.dtype, [&](auto* tag) -> shampoo4_status {
    using T = std::remove_pointer_t<decltype(tag)>;
    k_act8_join<T><<<ctas, kThreads, 0, st>>>(sums, p.shares, static_cast<T*>(o.y), o.ld, o.accumulate, R, int(inner));
    S4_CUDA(cudaGetLastError());
    return SHAMPOO4_OK;
  });
}

}  // namespace s4

// ------------------------------------------------------------------ C ABI

using namespace s4;

extern "C" shampoo4_status act8_grad_workspace(int32_t weight, int32_t dtype, int32_t result, int64_t tokens,
                                               int64_t out, int64_t inner, int32_t group, size_t* bytes) {
  if (!bytes || !dtype_ok(dtype) || !dtype_ok(result) || !group_ok(group) || !shape_ok(tokens, out) || !shape_ok(0, inner))
    return SHAMPOO4_ERR_INVALID_ARG;
  *bytes = tokens == 0 || out == 0 || inner == 0 ? 0 : grad_plan(weight != 0, dtype, result, group, tokens, out, inner).total();
  return SHAMPOO4_OK;
}

extern "C" shampoo4_status act8_product_form(int32_t call, int32_t dtype, int32_t result, int64_t tokens,
                                             int64_t out, int64_t inner, int32_t group, act8_form* form) {
  if (!form || call < 0 || call > 2 || !dtype_ok(dtype) || !dtype_ok(result) || !group_ok(group) ||
      (call == 2 && group) || !shape_ok(tokens, out) || !shape_ok(0, inner))
    return SHAMPOO4_ERR_INVALID_ARG;
  *form = act8_form{ACT8_WAY_CODES, 0, 0, 0};
  if (tokens == 0 || out == 0 || inner == 0) return SHAMPOO4_OK;
  if (call == 0) {
    const Form f = act8_codes_form(out, tokens, inner);
    *form = act8_form{ACT8_WAY_CODES, f.rows, f.shares, 0};
    return SHAMPOO4_OK;
  }
  const bool weight = call == 1;
  const GradPlan p = grad_plan(weight, dtype, result, group, tokens, out, inner);
  if (p.path == kDigits) {
    const Form f = weight ? act8_digits_form(inner, out, tokens) : act8_digits_form(inner, tokens, out);
    *form = act8_form{ACT8_WAY_DIGITS, f.rows, f.shares, 0};
  } else if (p.path == kRowHalves) {
    *form = act8_form{ACT8_WAY_ROW_HALVES, 0, 1, 1};
  } else {
    *form = act8_form{ACT8_WAY_HALVES, 0, p.shares, p.code_parts};
  }
  return SHAMPOO4_OK;
}

static shampoo4_status grad_call(const Act8Grad& g, void* ws, size_t ws_bytes, uint32_t* flags,
                                 shampoo4_stream_t stream) {
  size_t bytes = 0;
  if (!aligned(flags, 4)) return SHAMPOO4_ERR_INVALID_ARG;
  S4_TRY(act8_grad_check(g, &bytes));
  if (bytes && (!ws || !aligned(ws, 256))) return SHAMPOO4_ERR_INVALID_ARG;
  if (ws_bytes < bytes) return SHAMPOO4_ERR_WORKSPACE;
  return act8_grad_run(g, ws, Act8Watch{flags}, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" shampoo4_status act8_weight_grad(const void* d_dy, int32_t dtype, int64_t lddy, const int8_t* d_xc,
                                            int64_t ldxc, const float* d_xs, int32_t group, int64_t tokens,
                                            int64_t out, int64_t inner, void* d_dw, int32_t result, int64_t lddw,
                                            int32_t accumulate, void* d_workspace, size_t workspace_bytes,
                                            uint32_t* d_flags, shampoo4_stream_t stream) {
  return grad_call(Act8Grad{true, d_dy, dtype, lddy, d_xc, ldxc, d_xs, group, tokens, out, inner, d_dw, result, lddw,
                            accumulate},
                   d_workspace, workspace_bytes, d_flags, stream);
}

extern "C" shampoo4_status act8_input_grad(const void* d_dy, int32_t dtype, int64_t lddy, const int8_t* d_wc,
                                           int64_t ldwc, const float* d_ws, int64_t tokens, int64_t out,
                                           int64_t inner, void* d_dx, int32_t result, int64_t lddx,
                                           int32_t accumulate, void* d_workspace, size_t workspace_bytes,
                                           uint32_t* d_flags, shampoo4_stream_t stream) {
  return grad_call(Act8Grad{false, d_dy, dtype, lddy, d_wc, ldwc, d_ws, 0, tokens, out, inner, d_dx, result, lddx,
                            accumulate},
                   d_workspace, workspace_bytes, d_flags, stream);
}


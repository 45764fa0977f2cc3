// 8-bit activation checkpoints: the codec, the gated activation that keeps
// its inputs in 8 bits, and the C entry points of the forward product
// (act8_gemm.cu).
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
#include "act8_elt.cuh"

namespace s4 {
namespace {

constexpr float kScaleMax = 8454659.0f * 0x1p98f;      // the largest s with 127 s finite in fp32

// ---- the code rule

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
  let_next_start();
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

// ---- unpack

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

static shampoo4_status matmul(const int8_t* xc, int64_t ldxc, const float* xs, const int8_t* wc, int64_t ldwc,
                              const float* ws, const float* bias, int64_t tokens, int64_t out, int64_t inner, void* y,
                              int32_t dtype, int64_t ldy, bool after_pack, uint32_t* flags, cudaStream_t st) {
  // no columns: no group, so no scale either
  const Act8Out o{y, ldy, dtype, 0, inner > 0 ? xs : nullptr, inner > 0 ? ws : nullptr, bias};
  return launch_act8_codes(Act8Operand{wc, ldwc, 0}, Act8Operand{xc, ldxc, 0}, out, tokens, inner, o, after_pack,
                           flags, st);
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
  return matmul(d_xc, ldxc, d_xs, d_wc, ldwc, d_ws, d_bias, tokens, out, inner, d_y, dtype, ldy, false, d_flags,
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
  if (out == 0) return SHAMPOO4_OK;
  return matmul(d_xc, ldxc, d_xs, d_wc, ldwc, d_ws, d_bias, tokens, out, inner, d_y, ydtype, ldy, inner > 0, d_flags,
                reinterpret_cast<cudaStream_t>(stream));
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

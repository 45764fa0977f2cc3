// 8-bit activation checkpoints: the codec, the gated activation that keeps
// its inputs in 8 bits, and the C entry points of the forward product
// (act8_gemm.cu).
//
// A group of columns of a row (or the whole row) holds a = max |x|, the
// scale s = fp32(a / 127) and, per element, the integer nearest to 127 x / a
// (ties to even), the code of the exact quotient.
//
// fp32: two factors bracket 127 / a, and one packed fp32 multiply-add each
// rounds both products to integers; rounding is monotonic, so where the two
// agree the code is that of the quotient between them.  Where they differ (a
// border between two codes lies within 2^-20 of the quotient, exact ties
// included) the sign of 254 |x| - (2 k + 1) a decides, in fp32 with the
// products' exact remainders.
//
// 16-bit types: the factor above 127 / a alone.  With x = mx 2^i and a = ma
// 2^j, mantissas below 2^11, a quotient q that is not a tie is at least
// q / (254 mx) > q 2^-19 away from a border, and the factor is off by less
// than 2^-20 of itself.  A tie, 254 |x| = (2 k + 1) a, needs the prime 127 in
// 2 k + 1 (then k = 63, and the even code is the larger one, where the factor
// rounds to) or in ma; groups with 127 in ma (one in 128) go the fp32 way.
// (Ties are met often: with two factors for all types every fifth warp of
// normal bfloat16 data held one, 190 against 120 us for 16384 x 11008.)
//
// All kernels here stream: the bound is HBM bandwidth, and then instructions
// (the first form, with an IEEE division per lane and a distance test per
// element, issued 25 instructions per element and ran at a third of the
// bandwidth).
#include "act8_elt.cuh"
#include "quant4.cuh"

namespace s4 {
namespace {

constexpr float kScaleMax = 8454659.0f * 0x1p98f;      // the largest s with 127 s finite in fp32

// ---- the code rule

// Within 1 ulp where x and the result are normal, else 0 or infinity (the form
// that keeps subnormals takes several instructions more).
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

struct Group {
  float a;          // max |x|
  uint64_t lo, hi;  // factors below and above 127 / a, twice each; 0 where every code is 0 or decided one by one
  bool ties;        // 127 divides the mantissa of a
  bool apart;       // decided one by one: NaN, infinity, or a magnitude that the factors do not fit
  __device__ __forceinline__ explicit Group(uint32_t bits) {
    a = __uint_as_float(bits);
    apart = bits != 0u && !(a >= 0x1p-100f && a <= 0x1p120f);
    // 127 rcp(a) is within 2^-23 + 2^-24 of 127 / a, at most 3 of its ulps
    const uint32_t r = __float_as_uint(127.0f * rcp_approx(a));
    ties = ((bits & 0x7fffffu) | 0x800000u) % 127u == 0u;
    const bool use = bits != 0u && !apart;
    const float l = use ? __uint_as_float(r - 4) : 0.0f, h = use ? __uint_as_float(r + 4) : 0.0f;
    lo = pack2(l, l);
    hi = pack2(h, h);
  }
  // fp32(a / 127), capped: Markstein's correction (IBM J. Res. Dev. 34(1),
  // 1990) of the product with RN(1/127); a plain division where the residual
  // could underflow.
  __device__ __forceinline__ float scale() const {
    if (!(a < __int_as_float(0x7f800000))) return a > 0.0f ? a : __uint_as_float(0x7fc00000u);
    if (a < 0x1p-90f) return __fdiv_rn(a, 127.0f);
    constexpr float kInv = 1.0f / 127.0f;
    const float q = a * kInv;
    return fminf(fmaf(fmaf(-q, 127.0f, a), kInv, q), kScaleMax);
  }
};

// The 8 codes one by one: groups of tiny or huge magnitude, and the zero
// codes of a group with NaN or infinity.  (Two fp32 numbers' quotient that is
// not a tie lies at least 2^-26 away from one, far above a double's rounding.)
template <class T>
__device__ __noinline__ uint2 codes8_apart(Raw8<T> r, float a) {
  uint32_t b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    b[i] = a < __int_as_float(0x7f800000) ? uint32_t(__double2int_rn(127.0 * double(elt(r, i)) / double(a))) & 0xffu
                                          : 0u;
  return make_uint2(b[0] | (b[1] << 8) | (b[2] << 16) | (b[3] << 24), b[4] | (b[5] << 8) | (b[6] << 16) | (b[7] << 24));
}

constexpr float kMagic = 12582912.0f;                   // 1.5 2^23: adding it rounds to an integer, ties to even

// The code (plus kMagic) of an x between codes: k or k + 1 of its sign, k the
// smaller in magnitude of the two candidates.  254 |x| and (2 k + 1) a as
// rounded products and their exact remainders: the rounded ones are so close
// that they subtract exactly, and the remainders have at most 9 bits.
__device__ __forceinline__ uint32_t between(float x, float a, uint32_t t0, uint32_t t1) {
  const float k = fminf(fabsf(__uint_as_float(t0) - kMagic), fabsf(__uint_as_float(t1) - kMagic));
  const float odd = fmaf(2.0f, k, 1.0f), y = fabsf(x);
  const float u = 254.0f * y, w = odd * a;
  const float d = (u - w) + (fmaf(254.0f, y, -u) - fmaf(odd, a, -w));
  const float up = d > 0.0f || (d == 0.0f && (int(k) & 1)) ? 1.0f : 0.0f;
  return __float_as_uint(copysignf(k + up, x) + kMagic);
}

template <class T>
__device__ __forceinline__ uint2 codes8(const Raw8<T>& r, const Group& g) {
  const uint64_t magic = pack2(kMagic, kMagic);
  if (g.apart) return codes8_apart(r, g.a);
  uint32_t t[8];
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const uint64_t h = fma2(pack2(elt(r, i), elt(r, i + 1)), g.hi, magic);
    t[i] = uint32_t(h);
    t[i + 1] = uint32_t(h >> 32);
  }
  if (sizeof(T) == 4 || g.ties) {
    uint32_t q[8];
    uint32_t differ = 0;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const uint64_t l = fma2(pack2(elt(r, i), elt(r, i + 1)), g.lo, magic);
      q[i] = uint32_t(l);
      q[i + 1] = uint32_t(l >> 32);
      differ |= (t[i] ^ q[i]) | (t[i + 1] ^ q[i + 1]);
    }
    if (differ) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (t[i] != q[i]) t[i] = between(elt(r, i), g.a, t[i], q[i]);
    }
  }
  return make_uint2(__byte_perm(__byte_perm(t[0], t[1], 0x0040), __byte_perm(t[2], t[3], 0x0040), 0x5410),
                    __byte_perm(__byte_perm(t[4], t[5], 0x0040), __byte_perm(t[6], t[7], 0x0040), 0x5410));
}

// max |x| of 8 elements, as bits; NaN above everything.
__device__ __forceinline__ uint32_t absmax8(const Raw8<float>& r) {
  float m = absmax3_nan(elt(r, 0), elt(r, 1), elt(r, 2));
  m = absmax3_nan(m, elt(r, 3), elt(r, 4));
  m = absmax3_nan(m, elt(r, 5), elt(r, 6));
  return abs_bits(max2_nan(m, fabsf(elt(r, 7))));
}
__device__ __forceinline__ uint32_t absmax8(const Raw8<__nv_bfloat16>& r) {
  const __nv_bfloat162* w = reinterpret_cast<const __nv_bfloat162*>(r.v);
  const __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(__habs2(w[0]), __habs2(w[1])),
                                       __hmax2_nan(__habs2(w[2]), __habs2(w[3])));
  return abs_bits(max2_nan(__low2float(m), __high2float(m)));
}
__device__ __forceinline__ uint32_t absmax8(const Raw8<__half>& r) {
  const __half2* w = reinterpret_cast<const __half2*>(r.v);
  const __half2 m = __hmax2_nan(__hmax2_nan(__habs2(w[0]), __habs2(w[1])),
                                __hmax2_nan(__habs2(w[2]), __habs2(w[3])));
  return abs_bits(max2_nan(__low2float(m), __high2float(m)));
}

// ---- pack

// Groups of columns: a lane holds 8 columns of kRows rows, a group's maximum
// goes over its lanes by shuffles, x is read once.  fp32 is bound by HBM
// (16384 x 11008 in groups of 128: 165 us, 5.5 TB/s), the 16-bit types by
// issue slots too (bf16 140 us, 3.9 TB/s; 18 instructions per element).
template <class T, int kRows, bool A>
__global__ void __launch_bounds__(kThreads) k_act8_pack_groups(Mat x, Ckpt o, int64_t rows, int cols) {
  const Piece<kRows> p;
  if (p.row >= rows) return;                             // a whole warp
  Raw8<T> r[kRows];
#pragma unroll
  for (int u = 0; u < kRows; ++u)
    load8<A>(static_cast<const T*>(x.p) + p.at(u) * x.ld, p.c, p.at(u) < rows ? cols : 0, x.vec, r[u]);
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    const int64_t row = p.at(u);
    const Group g(group_max(absmax8(r[u]), 1 << (o.shift - 3)));
    if (row >= rows || p.c >= cols) continue;
    store_codes8(o.codes + row * o.ldc, p.c, cols, codes8(r[u], g));
    if ((p.c & ((1 << o.shift) - 1)) == 0) o.scales[row * o.groups + (p.c >> o.shift)] = g.scale();
  }
}

// One scale for the row.  WARP: a warp per row (up to 1024 columns); else a
// CTA per row.  IT > 0: a thread's at most IT pieces of 8 columns stay in
// registers between the maximum and the codes; IT = 0: the row is read twice.
// Bound by HBM: 16384 x 11008 bf16 98 us, 5.5 TB/s, fp32 144 us, 6.3 TB/s.
template <class T, int IT, bool WARP, bool A>
__global__ void __launch_bounds__(512, 2) k_act8_pack_rows(Mat x, Ckpt o, int64_t rows, int cols) {
  __shared__ uint32_t slots[32];
  let_next_start();
  const int64_t row = WARP ? int64_t(blockIdx.x) * blockDim.y + threadIdx.y : int64_t(blockIdx.x);
  if (row >= rows) return;                               // a whole warp, or nobody
  const T* xr = static_cast<const T*>(x.p) + row * x.ld;
  int8_t* cr = o.codes + row * o.ldc;
  const int step = int(blockDim.x) * 8, first = int(threadIdx.x) * 8;
  uint32_t m = 0;
  if (IT > 0) {
    Raw8<T> r[IT > 0 ? IT : 1];
#pragma unroll
    for (int i = 0; i < IT; ++i) load8<A>(xr, first + i * step, cols, x.vec, r[i]);
#pragma unroll
    for (int i = 0; i < IT; ++i) m = max(m, absmax8(r[i]));
    m = WARP ? __reduce_max_sync(0xffffffffu, m) : cta_max(m, slots);
    const Group g(m);
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int c = first + i * step;
      if (c < cols) store_codes8(cr, c, cols, codes8(r[i], g));
    }
    if (threadIdx.x == 0) o.scales[row] = g.scale();
  } else {
    Raw8<T> r;
    for (int c = first; c < cols; c += step) {
      load8<A>(xr, c, cols, x.vec, r);
      m = max(m, absmax8(r));
    }
    const Group g(cta_max(m, slots));
    for (int c = first; c < cols; c += step) {
      load8<A>(xr, c, cols, x.vec, r);
      store_codes8(cr, c, cols, codes8(r, g));
    }
    if (threadIdx.x == 0) o.scales[row] = g.scale();
  }
}

// ---- unpack

// Bound by HBM: 16384 x 11008 to bf16 90 us, 6.0 TB/s, to fp32 144 us.
template <class T, int kRows, bool A>
__global__ void __launch_bounds__(kThreads) k_act8_unpack(Ckpt k, T* x, int64_t ldx, int vec, int64_t rows, int cols) {
  const Piece<kRows> p;
  if (p.row >= rows || (A && p.c >= cols)) return;       // unaligned stores are a whole warp's
  uint2 w[kRows];
  float s[kRows];
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    const int64_t row = p.at(u);
    load_codes8(k.codes + row * k.ldc, p.c, row < rows ? cols : 0, w[u]);
    s[u] = row < rows && (A || p.c < cols) ? __ldg(k.scales + row * k.groups + (p.c >> k.shift)) : 0.0f;
  }
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    float v[8];
    values8(w[u], s[u], v);
    store8_any<A>(x + p.at(u) * ldx, p.c, p.at(u) < rows ? cols : 0, vec, v);
  }
}

// ---- the gated activation

// 1 / (1 + exp(-x)).  fp32: the accurate exponential, then a reciprocal
// within an ulp (2^-22 in all); 16-bit results: the base-2 exponential unit,
// off by 2^-22 and by the rounding of its argument (up to 88 log2(e) 2^-24),
// below 1e-5, against their half step of 2^-11 or 2^-8.
template <class T>
__device__ __forceinline__ float sigmoid(float x) {
  if (sizeof(T) == 4) return rcp_approx(1.0f + expf(-x));
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.4426950408889634f));
  return rcp_approx(1.0f + e);
}

template <bool A, class T>
__device__ __forceinline__ void gated8(const Raw8<T>& g, const Raw8<T>& u, T* h, int c, int n, int vec) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = elt(g, i);
    v[i] = x * sigmoid<T>(x) * elt(u, i);
  }
  store8_any<A>(h, c, n, vec, v);
}

// Both inputs are read once, for the codes and for h.  Bound by issue slots (71%
// busy: two codes, an exponential and a reciprocal per element, 43
// instructions) and HBM: 8192 x 11008 bf16 in groups of 128 167 us, 4.3 TB/s;
// fp32 231 us, 5.5 TB/s.
template <class T, int kRows, bool A>
__global__ void __launch_bounds__(kThreads)
k_act8_swiglu_groups(Mat gate, Mat up, T* h, int64_t ldh, int vech, Ckpt kg, Ckpt ku, int64_t rows, int cols) {
  const Piece<kRows> p;
  if (p.row >= rows) return;
  Raw8<T> g[kRows], u[kRows];
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int64_t row = p.at(k);
    const int n = row < rows ? cols : 0;
    load8<A>(static_cast<const T*>(gate.p) + row * gate.ld, p.c, n, gate.vec, g[k]);
    load8<A>(static_cast<const T*>(up.p) + row * up.ld, p.c, n, up.vec, u[k]);
  }
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int64_t row = p.at(k);
    const int lanes = 1 << (kg.shift - 3);
    const Group gg(group_max(absmax8(g[k]), lanes)), gu(group_max(absmax8(u[k]), lanes));
    if (row >= rows) continue;                           // a whole warp
    if (p.c < cols) {
      store_codes8(kg.codes + row * kg.ldc, p.c, cols, codes8(g[k], gg));
      store_codes8(ku.codes + row * ku.ldc, p.c, cols, codes8(u[k], gu));
      if ((p.c & ((1 << kg.shift) - 1)) == 0) {
        const int64_t s = row * kg.groups + (p.c >> kg.shift);
        kg.scales[s] = gg.scale();
        ku.scales[s] = gu.scale();
      }
    }
    gated8<A>(g[k], u[k], h + row * ldh, p.c, cols, vech);
  }
}

// One scale per row: the row is read twice (the second time from cache).
// 8192 x 11008 bf16 157 us, fp32 222 us.
template <class T, bool A>
__global__ void __launch_bounds__(kThreads)
k_act8_swiglu_rows(Mat gate, Mat up, T* h, int64_t ldh, int vech, Ckpt kg, Ckpt ku, int64_t rows, int cols) {
  __shared__ uint32_t slots[kThreads / 32];
  const int64_t row = blockIdx.x;
  const T* gr = static_cast<const T*>(gate.p) + row * gate.ld;
  const T* ur = static_cast<const T*>(up.p) + row * up.ld;
  Raw8<T> g, u;
  uint32_t mg = 0, mu = 0;
#pragma unroll 2
  for (int c0 = 0; c0 < cols; c0 += kThreads * 8) {      // all lanes to the end
    const int c = c0 + int(threadIdx.x) * 8;
    load8<A>(gr, c, cols, gate.vec, g);
    load8<A>(ur, c, cols, up.vec, u);
    mg = max(mg, absmax8(g));
    mu = max(mu, absmax8(u));
    gated8<A>(g, u, h + row * ldh, c, cols, vech);
  }
  const Group gg(cta_max(mg, slots)), gu(cta_max(mu, slots));
#pragma unroll 2
  for (int c = int(threadIdx.x) * 8; c < cols; c += kThreads * 8) {
    load8<A>(gr, c, cols, gate.vec, g);
    load8<A>(ur, c, cols, up.vec, u);
    store_codes8(kg.codes + row * kg.ldc, c, cols, codes8(g, gg));
    store_codes8(ku.codes + row * ku.ldc, c, cols, codes8(u, gu));
  }
  if (threadIdx.x == 0) {
    kg.scales[row] = gg.scale();
    ku.scales[row] = gu.scale();
  }
}

// Bound by HBM (fp32: 197 us for 8192 x 11008, 6.4 TB/s) and, for the 16-bit
// types, as much by issue slots (67% busy; bf16 130 us, 5.5 TB/s).
template <class T, int kRows, bool A>
__global__ void __launch_bounds__(kThreads)
k_act8_swiglu_backward(Mat dh, Ckpt kg, Ckpt ku, T* dg, int64_t lddg, int vecg, T* du, int64_t lddu, int vecu,
                       int64_t rows, int cols) {
  const Piece<kRows> p;
  if (p.row >= rows || (A && p.c >= cols)) return;       // unaligned stores are a whole warp's
  Raw8<T> d[kRows];
  uint2 wg[kRows], wu[kRows];
  float sg[kRows], su[kRows];
  const int gi = p.c >> kg.shift;
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int64_t row = p.at(k);
    const int n = row < rows ? cols : 0;
    load8<A>(static_cast<const T*>(dh.p) + row * dh.ld, p.c, n, dh.vec, d[k]);
    load_codes8(kg.codes + row * kg.ldc, p.c, n, wg[k]);
    load_codes8(ku.codes + row * ku.ldc, p.c, n, wu[k]);
    sg[k] = n && (A || p.c < n) ? __ldg(kg.scales + row * kg.groups + gi) : 0.0f;
    su[k] = n && (A || p.c < n) ? __ldg(ku.scales + row * ku.groups + gi) : 0.0f;
  }
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int64_t row = p.at(k);
    const int n = row < rows ? cols : 0;
    float g[8], u[8], og[8], ou[8];
    values8(wg[k], sg[k], g);
    values8(wu[k], su[k], u);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = elt(d[k], i), sig = sigmoid<T>(g[i]);
      ou[i] = x * (g[i] * sig);
      og[i] = x * (u[i] * (sig * fmaf(g[i], 1.0f - sig, 1.0f)));   // the slope first: dh up may pass fp32's range
    }
    store8_any<A>(dg + row * lddg, p.c, n, vecg, og);
    store8_any<A>(du + row * lddu, p.c, n, vecu, ou);
  }
}

shampoo4_status pack(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t ldx, int32_t group, Ckpt o,
                     cudaStream_t st) {
  if (rows == 0 || cols == 0) return SHAMPOO4_OK;
  const Mat m = mat(x, ldx, dtype);
  return by_dtype(dtype, [&](auto* tag) { return by_flag(m.vec != 0, [&](auto flag) -> shampoo4_status {
    using T = std::remove_pointer_t<decltype(tag)>;
    constexpr bool A = decltype(flag)::value;
    const int n = int(cols);
    if (group) {
      const dim3 b = piece_block(cols);
      dim3 g;
      constexpr int kMany = sizeof(T) == 4 ? 2 : 4;
      const bool many = many_pieces(rows, cols);
      if (!piece_grid(rows, cols, b, many ? kMany : 1, &g)) return SHAMPOO4_ERR_INVALID_ARG;
      if (many) k_act8_pack_groups<T, kMany, A><<<g, b, 0, st>>>(m, o, rows, n);
      else k_act8_pack_groups<T, 1, A><<<g, b, 0, st>>>(m, o, rows, n);
    } else if (cols <= 1024) {                           // 8 rows per CTA, a warp each
      const dim3 b(32, 8);
      const unsigned g = unsigned((rows + 7) / 8);
      if (cols <= 256) k_act8_pack_rows<T, 1, true, A><<<g, b, 0, st>>>(m, o, rows, n);
      else if (cols <= 512) k_act8_pack_rows<T, 2, true, A><<<g, b, 0, st>>>(m, o, rows, n);
      else if (cols <= 768) k_act8_pack_rows<T, 3, true, A><<<g, b, 0, st>>>(m, o, rows, n);
      else k_act8_pack_rows<T, 4, true, A><<<g, b, 0, st>>>(m, o, rows, n);
    } else {
      // Few threads with many pieces each in flight: 256 with up to 8 (fp32,
      // whose pieces take twice the registers: 512 with up to 4).  16384 x
      // 11008 bf16: 99 us, against 128 with 704 threads of two pieces.
      const int64_t pieces = (cols + 7) / 8;
      const unsigned g = unsigned(rows);
      const int threads = sizeof(T) == 2 || pieces <= 1024 ? 256 : 512;
      const int it = int(std::min<int64_t>((pieces + threads - 1) / threads, 99));
      const unsigned b = unsigned(std::min<int64_t>(threads, ((pieces + it - 1) / it + 31) / 32 * 32));
      if (it == 1) k_act8_pack_rows<T, 1, false, A><<<g, b, 0, st>>>(m, o, rows, n);
      else if (it == 2) k_act8_pack_rows<T, 2, false, A><<<g, b, 0, st>>>(m, o, rows, n);
      else if (it == 3) k_act8_pack_rows<T, 3, false, A><<<g, b, 0, st>>>(m, o, rows, n);
      else if (it == 4) k_act8_pack_rows<T, 4, false, A><<<g, b, 0, st>>>(m, o, rows, n);
      else if (sizeof(T) == 2 && it <= 6) k_act8_pack_rows<T, 6, false, A><<<g, b, 0, st>>>(m, o, rows, n);
      else if (sizeof(T) == 2 && it <= 8) k_act8_pack_rows<T, 8, false, A><<<g, b, 0, st>>>(m, o, rows, n);
      else k_act8_pack_rows<T, 0, false, A><<<g, 512, 0, st>>>(m, o, rows, n);
    }
    S4_CUDA(cudaGetLastError());
    return SHAMPOO4_OK;
  }); });
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
  return pack(d_x, dtype, rows, cols, ldx, group, ckpt(d_codes, ldc, d_scales, cols, group),
              reinterpret_cast<cudaStream_t>(stream));
}

extern "C" shampoo4_status act8_unpack(const int8_t* d_codes, int64_t ldc, const float* d_scales, int64_t rows,
                                       int64_t cols, int32_t group, void* d_x, int32_t dtype, int64_t ldx,
                                       shampoo4_stream_t stream) {
  if (!shape_ok(rows, cols) || !dtype_ok(dtype) || !group_ok(group)) return SHAMPOO4_ERR_INVALID_ARG;
  if (rows == 0 || cols == 0) return SHAMPOO4_OK;
  if (!mat_ok(d_x, dtype, rows, cols, ldx) || !codes_ok(d_codes, ldc, cols, d_scales)) return SHAMPOO4_ERR_INVALID_ARG;
  const bool many = many_pieces(rows, cols);
  const dim3 b = piece_block(cols);
  dim3 g;
  if (!piece_grid(rows, cols, b, many ? 4 : 1, &g)) return SHAMPOO4_ERR_INVALID_ARG;
  const Ckpt k = ckpt(d_codes, ldc, d_scales, cols, group);
  const int vec = vec_of(d_x, ldx, dtype);
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return by_dtype(dtype, [&](auto* tag) { return by_flag(vec != 0, [&](auto flag) -> shampoo4_status {
    using T = std::remove_pointer_t<decltype(tag)>;
    constexpr bool A = decltype(flag)::value;
    T* x = static_cast<T*>(d_x);
    if (many) k_act8_unpack<T, 4, A><<<g, b, 0, st>>>(k, x, ldx, vec, rows, int(cols));
    else k_act8_unpack<T, 1, A><<<g, b, 0, st>>>(k, x, ldx, vec, rows, int(cols));
    S4_CUDA(cudaGetLastError());
    return SHAMPOO4_OK;
  }); });
}

static shampoo4_status check_product(int64_t tokens, int64_t out, int64_t inner) {
  if (!shape_ok(tokens, out) || inner < 0 || inner > kAct8MaxInner) return SHAMPOO4_ERR_INVALID_ARG;
  return SHAMPOO4_OK;
}

static shampoo4_status matmul(const int8_t* xc, int64_t ldxc, const float* xs, const int8_t* wc, int64_t ldwc,
                              const float* ws, const float* bias, int64_t tokens, int64_t out, int64_t inner, void* y,
                              int32_t dtype, int64_t ldy, bool after_pack, uint32_t* flags, cudaStream_t st) {
  // no columns: no group, so no scale either
  const Act8Out o{y, ldy, dtype, 0, inner > 0 ? xs : nullptr, inner > 0 ? ws : nullptr, bias, 0};
  return launch_act8_codes(Act8Operand{wc, ldwc, 0}, Act8Operand{xc, ldxc, 0}, out, tokens, inner, o, after_pack,
                           Act8Watch{flags}, st);
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
  const bool many = dtype != ACT8_FP32 && many_pieces(rows, cols);
  if (!piece_grid(rows, cols, b, many ? 2 : 1, &g)) return SHAMPOO4_ERR_INVALID_ARG;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const Ckpt kg = ckpt(d_gate_codes, ldgc, d_gate_scales, cols, group);
  const Ckpt ku = ckpt(d_up_codes, lduc, d_up_scales, cols, group);
  const int vh = vec_of(d_h, ldh, dtype);
  const Mat mg = mat(d_gate, ldg, dtype), mu = mat(d_up, ldu, dtype);
  return by_dtype(dtype, [&](auto* tag) { return by_flag(mg.vec && mu.vec && vh, [&](auto flag) -> shampoo4_status {
    using T = std::remove_pointer_t<decltype(tag)>;
    constexpr bool A = decltype(flag)::value;
    T* h = static_cast<T*>(d_h);
    if (group && many)
      k_act8_swiglu_groups<T, 2, A><<<g, b, 0, st>>>(mg, mu, h, ldh, vh, kg, ku, rows, int(cols));
    else if (group)
      k_act8_swiglu_groups<T, 1, A><<<g, b, 0, st>>>(mg, mu, h, ldh, vh, kg, ku, rows, int(cols));
    else
      k_act8_swiglu_rows<T, A><<<unsigned(rows), kThreads, 0, st>>>(mg, mu, h, ldh, vh, kg, ku, rows, int(cols));
    S4_CUDA(cudaGetLastError());
    return SHAMPOO4_OK;
  }); });
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
  const bool many = dtype != ACT8_FP32 && many_pieces(rows, cols);
  if (!piece_grid(rows, cols, b, many ? 2 : 1, &g)) return SHAMPOO4_ERR_INVALID_ARG;
  const Ckpt kg = ckpt(d_gate_codes, ldgc, d_gate_scales, cols, group);
  const Ckpt ku = ckpt(d_up_codes, lduc, d_up_scales, cols, group);
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const Mat m = mat(d_dh, lddh, dtype);
  const int vg = vec_of(d_dgate, lddg, dtype), vu = vec_of(d_dup, lddu, dtype);
  return by_dtype(dtype, [&](auto* tag) { return by_flag(m.vec && vg && vu, [&](auto flag) -> shampoo4_status {
    using T = std::remove_pointer_t<decltype(tag)>;
    constexpr bool A = decltype(flag)::value;
    T *dg = static_cast<T*>(d_dgate), *du = static_cast<T*>(d_dup);
    if (many)
      k_act8_swiglu_backward<T, 2, A><<<g, b, 0, st>>>(m, kg, ku, dg, lddg, vg, du, lddu, vu, rows, int(cols));
    else
      k_act8_swiglu_backward<T, 1, A><<<g, b, 0, st>>>(m, kg, ku, dg, lddg, vg, du, lddu, vu, rows, int(cols));
    S4_CUDA(cudaGetLastError());
    return SHAMPOO4_OK;
  }); });
}

// Products of the 8-bit activation operators on the sm_100a tensor cores:
//
//   act8_matmul        int8 codes x int8 codes, exact int32 sums
//                      (tcgen05.mma kind::i8), scaled in the epilogue
//   act8_weight_grad,  bfloat16 parts x bfloat16 parts, fp32 sums
//   act8_input_grad    (tcgen05.mma kind::f16)
//
// One persistent CTA per SM walks the output tiles (128 x 256).  Operands
// come by TMA into a ring of stages, each holding 128 bytes of K (128 codes
// or 64 bfloat16) of every part; the accumulator is double-buffered in
// tensor memory, so one tile's epilogue runs under the next one's products.
// Warp roles (192 threads): warp 0 issues the loads, warp 1 the MMAs, warps
// 2..5 drain the accumulator.  Every wait is bounded (2 s); on expiry the
// roles raise SHAMPOO4_FLAG_TIMEOUT, wait for what they issued and leave.
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <algorithm>
#include <climits>
#include "act8.h"
#include "plan.h"
#include "tcgen05.cuh"

namespace s4 {
namespace {

enum { kI8 = 0, kBf16 = 1 };
constexpr int kTileM = 128;               // rows of a CTA's accumulator: the TMEM lanes
constexpr int kRowBytes = 128;            // bytes of K per stage (K-major), one swizzle atom row
constexpr int kPitch = 36;                // staging row pitch in words: conflict-free both ways

template <int KIND, bool A_MN, bool B_MN, int BN, int NA, int NB, int STAGES>
struct Cfg {
  static constexpr int kKElems = KIND == kI8 ? 128 : 64;       // K per stage
  static constexpr int kATile = kTileM * kRowBytes;
  static constexpr int kBTile = BN * kRowBytes;
  static constexpr int kStage = NA * kATile + NB * kBTile;
  static constexpr int kEpiWarp = 32 * kPitch * 4;
  static constexpr int kSmem = STAGES * kStage + 4 * kEpiWarp + 1024;
  static constexpr int kTmemCols = 2 * BN;
  static_assert(kSmem <= 227 * 1024, "stages fit in shared memory");
  static_assert(KIND == kBf16 || (!A_MN && !B_MN && NA == 1 && NB == 1), "codes are K-major");
};

struct GemmArgs {
  CUtensorMap a[2], b[2];
  int32_t M, N, kblocks, tiles_m, tiles_n;
  uint32_t* flags;
  Act8Out out;
};

// Instruction descriptor: fp32 sums of bfloat16 (type code 1) or int32 sums
// of signed 8-bit integers (type code 1, accumulator code 2).
template <int KIND>
__host__ __device__ constexpr uint32_t idesc(int M, int N, int a_mn, int b_mn) {
  return ((KIND == kI8 ? 2u : 1u) << 4) | (1u << 7) | (1u << 10) | (uint32_t(a_mn) << 15) | (uint32_t(b_mn) << 16) |
         (uint32_t(N >> 3) << 17) | (uint32_t(M >> 4) << 24);
}

template <int KIND>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
  if (KIND == kI8)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(id), "r"(acc) : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(id), "r"(acc) : "memory");
}

// K-major (128-byte swizzle): rows of 128 B, 8-row groups 1024 B apart, an
// MMA's K (32 bytes) along the row.  MN-major: boxes of 64 elements (128 B)
// by 64 K rows, 8192 B apart; 8-row K groups 1024 B apart, an MMA's K is 16
// rows.
template <bool MN>
__device__ __forceinline__ uint64_t tile_desc(uint32_t base, int kk) {
  return MN ? smem_desc(base + kk * 2048, 8192, 1024, 2) : smem_desc(base + kk * 32, 16, 1024, 2);
}

template <bool MN, int ROWS, int KELEMS>
__device__ __forceinline__ void load_tile(const CUtensorMap* map, int mn0, int k0, uint32_t dst, uint64_t* bar) {
  if (!MN) {
    tma_load_2d(dst, map, k0, mn0, bar);
  } else {
#pragma unroll
    for (int g = 0; g < ROWS / 64; ++g) tma_load_2d(dst + g * 8192, map, mn0 + 64 * g, k0, bar);
  }
}

// Tile t in an order that keeps the tiles in flight close in both operands:
// groups of 8 tile rows, walked column by column.
__device__ __forceinline__ void tile_of(const GemmArgs& g, int t, int& tm, int& tn) {
  const int per = 8 * g.tiles_n;
  const int grp = t / per, r = t - grp * per;
  const int rows = min(8, g.tiles_m - 8 * grp);
  tn = r / rows;
  tm = 8 * grp + (r - tn * rows);
}

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
template <class T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <> __device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }

// Four results (columns c .. c + 3 of one row) into y, rounded once.
template <class T>
__device__ __forceinline__ void store4(T* p, int c, int N, bool vec, bool add, float (&v)[4]) {
  struct alignas(4 * sizeof(T)) V4 { T e[4]; };
  if (vec && c + 4 <= N) {
    if (add) {
      const V4 o = *reinterpret_cast<const V4*>(p);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] += to_f32(o.e[j]);
    }
    V4 r;
#pragma unroll
    for (int j = 0; j < 4; ++j) r.e[j] = from_f32<T>(v[j]);
    *reinterpret_cast<V4*>(p) = r;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (c + j < N) p[j] = from_f32<T>(add ? v[j] + to_f32(p[j]) : v[j]);
  }
}

// Rows m0 .. m0 + 31 and columns n0 .. n0 + BN - 1 by one epilogue warp:
// 32 columns at a time out of tensor memory (lane = row), transposed through
// the warp's staging block, then lane l takes row 4 t + l / 8, columns
// 4 (l % 8) .. + 3, so a store instruction covers four full row segments.
template <int KIND, int BN, class T>
__device__ __forceinline__ void drain(const GemmArgs& g, uint32_t tacc, int m0, int n0, int lane, float* stage) {
  T* y = static_cast<T*>(g.out.y);
  const int64_t ld = g.out.ld;
  const int M = g.M, N = g.N;
  const bool vec = ((reinterpret_cast<uintptr_t>(y) | uintptr_t(ld * int64_t(sizeof(T)))) % (4 * sizeof(T))) == 0;
  const bool add = g.out.accumulate != 0;
  const bool any = g.kblocks > 0;
  const int sr = lane >> 3, sc = 4 * (lane & 7);
  float rs[8];
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    const int r = m0 + 4 * t + sr;
    rs[t] = (g.out.row_scale && r < M) ? __ldg(g.out.row_scale + r) : 1.0f;
  }
#pragma unroll 1
  for (int c0 = 0; c0 < BN && n0 + c0 < N; c0 += 32) {
    uint32_t r[32];
    if (any) {
      tmem_ld32(tacc + uint32_t(c0), r);
    } else {
#pragma unroll
      for (int j = 0; j < 32; ++j) r[j] = 0u;
    }
    __syncwarp();                                        // the previous chunk's reads are done
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
      float4 x;
      if (KIND == kI8)
        x = make_float4(__int2float_rn(int(r[j])), __int2float_rn(int(r[j + 1])), __int2float_rn(int(r[j + 2])),
                        __int2float_rn(int(r[j + 3])));
      else
        x = make_float4(__uint_as_float(r[j]), __uint_as_float(r[j + 1]), __uint_as_float(r[j + 2]),
                        __uint_as_float(r[j + 3]));
      *reinterpret_cast<float4*>(stage + lane * kPitch + j) = x;
    }
    __syncwarp();
    const int c = n0 + c0 + sc;
    float cs[4], bi[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      cs[j] = (g.out.col_scale && c + j < N) ? __ldg(g.out.col_scale + c + j) : 1.0f;
      bi[j] = (g.out.bias && c + j < N) ? __ldg(g.out.bias + c + j) : 0.0f;
    }
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const int row = m0 + 4 * t + sr;
      const float4 x = *reinterpret_cast<const float4*>(stage + (4 * t + sr) * kPitch + sc);
      float v[4] = {x.x, x.y, x.z, x.w};
      if (KIND == kI8) {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = v[j] * rs[t] * cs[j] + bi[j];
      }
      if (row < M && c < N) store4<T>(y + int64_t(row) * ld + c, c, N, vec, add, v);
    }
  }
}

template <int KIND, bool A_MN, bool B_MN, int BN, int NA, int NB, int STAGES>
__global__ void __launch_bounds__(192, 1) k_act8_gemm(const __grid_constant__ GemmArgs g) {
  using C = Cfg<KIND, A_MN, B_MN, BN, NA, NB, STAGES>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t full_bar[STAGES], empty_bar[STAGES], acc_full[2], acc_empty[2], done_bar;
  __shared__ uint32_t tmem_slot;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&acc_full[s], 1);
      mbar_init(&acc_empty[s], 4);
    }
    mbar_init(&done_bar, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)),
                 "r"(C::kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = tmem_slot;
  const int tiles = g.tiles_m * g.tiles_n, kblocks = g.kblocks;

  if (warp == 0) {
    if (lane == 0) {                                        // ---- loads
      int it = 0;
      bool ok = true;
      for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
        int tm, tn;
        tile_of(g, t, tm, tn);
        const int m0 = tm * kTileM, n0 = tn * BN;
        for (int kb = 0; kb < kblocks; ++kb, ++it) {
          const int s = it % STAGES;
          if (!mbar_wait(&empty_bar[s], ((it / STAGES) & 1) ^ 1)) { ok = false; break; }
          uint32_t dst = smem_u32(smem + s * C::kStage);
          mbar_expect_tx(&full_bar[s], C::kStage);
#pragma unroll
          for (int p = 0; p < NA; ++p, dst += C::kATile)
            load_tile<A_MN, kTileM, C::kKElems>(&g.a[p], m0, kb * C::kKElems, dst, &full_bar[s]);
#pragma unroll
          for (int p = 0; p < NB; ++p, dst += C::kBTile)
            load_tile<B_MN, BN, C::kKElems>(&g.b[p], n0, kb * C::kKElems, dst, &full_bar[s]);
        }
      }
      // every stage's last load has been consumed (or, after a timeout, has landed) before the CTA leaves
      for (int i = max(0, it - STAGES); i < it; ++i)
        if (!mbar_wait(ok ? &empty_bar[i % STAGES] : &full_bar[i % STAGES], (i / STAGES) & 1)) ok = false;
      if (!ok && g.flags) atomicOr(g.flags, SHAMPOO4_FLAG_TIMEOUT);
    }
  } else if (warp == 1) {
    if (lane == 0) {                                        // ---- products
      constexpr uint32_t id = idesc<KIND>(kTileM, BN, A_MN, B_MN);
      int it = 0, i = 0;
      bool ok = true;
      for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x, ++i) {
        const int ab = i & 1;
        if (!mbar_wait(&acc_empty[ab], ((i >> 1) & 1) ^ 1)) { ok = false; break; }
        fence_after_sync();
        const uint32_t d = tmem + uint32_t(ab * BN);
        for (int kb = 0; kb < kblocks; ++kb, ++it) {
          const int s = it % STAGES;
          if (!mbar_wait(&full_bar[s], (it / STAGES) & 1)) { ok = false; break; }
          fence_after_sync();
          const uint32_t a0 = smem_u32(smem + s * C::kStage), b0 = a0 + NA * C::kATile;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            mma<KIND>(d, tile_desc<A_MN>(a0, kk), tile_desc<B_MN>(b0, kk), id, (kb | kk) != 0);
            if (NB == 2) mma<KIND>(d, tile_desc<A_MN>(a0, kk), tile_desc<B_MN>(b0 + C::kBTile, kk), id, 1);
            if (NA == 2) mma<KIND>(d, tile_desc<A_MN>(a0 + C::kATile, kk), tile_desc<B_MN>(b0, kk), id, 1);
          }
          mma_commit(&empty_bar[s]);
        }
        if (ok) mma_commit(&acc_full[ab]);
      }
      // all MMAs issued are finished before tensor memory is freed
      mma_commit(&done_bar);
      if (!mbar_wait(&done_bar, 0)) ok = false;
      if (!ok && g.flags) atomicOr(g.flags, SHAMPOO4_FLAG_TIMEOUT);
    }
  } else {                                                  // ---- epilogue, warps 2..5
    const int q = warp & 3;                                 // TMEM lane quarter
    float* stage = reinterpret_cast<float*>(smem + STAGES * C::kStage + q * C::kEpiWarp);
    int i = 0;
    for (int t = blockIdx.x; t < tiles; t += gridDim.x, ++i) {
      const int ab = i & 1;
      if (!mbar_wait(&acc_full[ab], (i >> 1) & 1)) {
        if (g.flags && lane == 0) atomicOr(g.flags, SHAMPOO4_FLAG_TIMEOUT);
        break;
      }
      fence_after_sync();
      int tm, tn;
      tile_of(g, t, tm, tn);
      const uint32_t tacc = tmem + uint32_t(ab * BN) + (uint32_t(32 * q) << 16);
      const int m0 = tm * kTileM + 32 * q, n0 = tn * BN;
      if (g.out.dtype == ACT8_FP32) drain<KIND, BN, float>(g, tacc, m0, n0, lane, stage);
      else if (g.out.dtype == ACT8_BF16) drain<KIND, BN, __nv_bfloat16>(g, tacc, m0, n0, lane, stage);
      else drain<KIND, BN, __half>(g, tacc, m0, n0, lane, stage);
      fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[ab]);
    }
  }
  fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    fence_after_sync();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kTmemCols)
                 : "memory");
  }
}

// ------------------------------------------------------------------ host

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    cudaDriverEntryPointQueryResult q;
    void* p = nullptr;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return fn;
}

// Tensor map of a rows x cols row-major matrix, box of 128 bytes of a row by
// box_rows, 128-byte swizzle, zeros outside.
shampoo4_status encode(CUtensorMap* out, int kind, const void* base, int64_t rows, int64_t cols, int64_t ld,
                       int box_rows) {
  auto fn = encoder();
  if (!fn) return SHAMPOO4_ERR_CUDA;
  const int64_t esize = kind == kI8 ? 1 : 2;
  if ((ld * esize) % 16 != 0 || reinterpret_cast<uintptr_t>(base) % 16 != 0) return SHAMPOO4_ERR_INVALID_ARG;
  cuuint64_t dims[2] = {cuuint64_t(cols), cuuint64_t(rows)};
  cuuint64_t strides[1] = {cuuint64_t(ld * esize)};
  cuuint32_t box[2] = {cuuint32_t(128 / esize), cuuint32_t(box_rows)};
  cuuint32_t estr[2] = {1u, 1u};
  const CUresult r = fn(out, kind == kI8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                        const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? SHAMPOO4_OK : SHAMPOO4_ERR_CUDA;
}

template <int KIND, bool A_MN, bool B_MN, int BN, int NA, int NB, int STAGES>
shampoo4_status launch(GemmArgs& g, int64_t M, int64_t N, int64_t K, cudaStream_t st) {
  using C = Cfg<KIND, A_MN, B_MN, BN, NA, NB, STAGES>;
  auto kern = k_act8_gemm<KIND, A_MN, B_MN, BN, NA, NB, STAGES>;
  g.M = int32_t(M);
  g.N = int32_t(N);
  g.kblocks = int32_t((K + C::kKElems - 1) / C::kKElems);
  const int64_t tm = (M + kTileM - 1) / kTileM, tn = (N + BN - 1) / BN;
  if (tm * tn > INT_MAX / 2) return SHAMPOO4_ERR_INVALID_ARG;
  g.tiles_m = int32_t(tm);
  g.tiles_n = int32_t(tn);
  S4_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem));
  int dev = 0, sms = 0;
  S4_CUDA(cudaGetDevice(&dev));
  S4_CUDA(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
  kern<<<unsigned(std::min<int64_t>(tm * tn, sms)), 192, C::kSmem, st>>>(g);
  S4_CUDA(cudaGetLastError());
  return SHAMPOO4_OK;
}

}  // namespace

shampoo4_status launch_act8_gemm_i8(const int8_t* a, int64_t lda, const int8_t* b, int64_t ldb, int64_t M, int64_t N,
                                    int64_t K, const Act8Out& out, uint32_t* flags, cudaStream_t st) {
  GemmArgs g{};
  g.out = out;
  g.flags = flags;
  if (K > 0) {
    S4_TRY(encode(&g.a[0], kI8, a, M, K, lda, kTileM));
    S4_TRY(encode(&g.b[0], kI8, b, N, K, ldb, 256));
  }
  return launch<kI8, false, false, 256, 1, 1, 4>(g, M, N, K, st);
}

shampoo4_status launch_act8_gemm_bf16(const Act8Parts& a, int a_mn, const Act8Parts& b, int64_t M, int64_t N,
                                      int64_t K, const Act8Out& out, uint32_t* flags, cudaStream_t st) {
  GemmArgs g{};
  g.out = out;
  g.flags = flags;
  if (K > 0) {
    const void* ap[2] = {a.hi, a.lo};
    const void* bp[2] = {b.hi, b.lo};
    for (int p = 0; p < 2; ++p) {
      if (ap[p]) S4_TRY(a_mn ? encode(&g.a[p], kBf16, ap[p], K, M, a.ld, 64)
                             : encode(&g.a[p], kBf16, ap[p], M, K, a.ld, kTileM));
      if (bp[p]) S4_TRY(encode(&g.b[p], kBf16, bp[p], K, N, b.ld, 64));
    }
  }
  const int na = a.lo ? 2 : 1, nb = b.lo ? 2 : 1;
  if (na == 2 && nb == 1) return SHAMPOO4_ERR_INVALID_ARG;   // no caller rounds b while it splits a
  if (a_mn) {
    if (nb == 1) return launch<kBf16, true, true, 256, 1, 1, 4>(g, M, N, K, st);
    if (na == 1) return launch<kBf16, true, true, 256, 1, 2, 2>(g, M, N, K, st);
    return launch<kBf16, true, true, 256, 2, 2, 2>(g, M, N, K, st);
  }
  if (nb == 1) return launch<kBf16, false, true, 256, 1, 1, 4>(g, M, N, K, st);
  if (na == 1) return launch<kBf16, false, true, 256, 1, 2, 2>(g, M, N, K, st);
  return launch<kBf16, false, true, 256, 2, 2, 2>(g, M, N, K, st);
}

}  // namespace s4

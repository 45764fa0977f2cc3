// Products of the 8-bit activation operators on the sm_100a tensor cores,
// all of the form  Y[r, m] = sum_k B[r, k] A[m, k]  with m contiguous in Y:
//
//   act8_matmul / act8_linear   A = weight codes, B = token codes: int8 x int8,
//                               exact int32 sums (tcgen05.mma kind::i8)
//   act8_weight_grad and        A = the stored codes, read in place (their
//   act8_input_grad             contraction index is the row: MN-major), B =
//                               the gradient in three signed base-256 digits
//                               of fixed point: three int8 products with
//                               exact int32 sums, joined in the epilogue
//   the same in 16 bits         A = the codes' values, B = the gradient, each
//                               as one or two scaled halves (kind::f16, fp32
//                               sums)
//
// A pair of CTAs (cta_group::2) owns a tile of 256 columns m by R rows: each
// CTA stages its 128 columns of A and half of the rows of B, and the leader's
// MMAs read both halves, so B crosses each SM's shared memory port once per
// pair.  TMEM lanes are columns m: a warp's 32 lanes write 32 consecutive
// results of a row without a transposing pass.  Digits are stacked along the
// MMA's N, so A is read once for all three.  The accumulator is
// double-buffered in tensor memory: one tile's epilogue runs under the next
// one's products.  The pairs are persistent, one CTA per SM.  Bound by the
// tensor cores, and in a loop by the power cap: 8192 x 11008 x 4096 codes 215
// us alone (3.4 POPS), 227 to 239 in a loop; its weight gradient in digits 648
// us alone (3.4 POPS of three products); 8192 x 4096 x 11008 as one half each
// 478 to 504 us (1.5 PFLOP/s); the tensor pipe is 88 to 92% busy where tiles
// fill the waves.
//
// Warp roles (320 threads): warp 0 issues the TMA loads, warp 1 of the leader
// the MMAs, warps 2..9 drain the accumulator, two per lane quarter with half of
// the rows each.  Every wait is bounded; on expiry a role raises
// SHAMPOO4_FLAG_TIMEOUT and stops, and the pair waits for its MMAs before it
// frees tensor memory and leaves.  The loads' waits are bounded by 2 s whatever
// the others' limit: a CTA leaves when every stage that it filled has been
// read, or 2 s after it issued the last one.
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include "act8.h"
#include "plan.h"
#include "tcgen05.cuh"

namespace s4 {
namespace {

enum { kI8 = 0, kHalf = 1 };
constexpr int kLanes = 128;               // columns m per CTA: the TMEM lanes
constexpr int kPairThreads = 320, kSmallThreads = 192;
constexpr int kRowBytes = 128;            // bytes of a swizzle atom row

// KIND; A_MN/B_MN: the operand's row index (not k) is contiguous; R: rows of
// a tile; PA, PB: 16-bit parts; ND: digit planes of B (stacked along N);
// CG: CTAs per tile; CHUNK: k-blocks per accumulation into registers (0: the
// whole sum in tensor memory).
template <int KIND_, bool A_MN_, bool B_MN_, int R_, int PA_, int PB_, int ND_, int CG_, int STAGES_, int CHUNK_>
struct Cfg {
  static constexpr int KIND = KIND_, R = R_, PA = PA_, PB = PB_, ND = ND_, CG = CG_, STAGES = STAGES_, CHUNK = CHUNK_;
  static constexpr bool A_MN = A_MN_, B_MN = B_MN_;
  static constexpr int kK = KIND == kI8 ? 128 : 64;            // k of a block: a swizzle atom's row
  static constexpr int kN = ND * R;                            // MMA N
  static constexpr int kBRows = R / CG;                        // rows of each digit plane a CTA stages
  static constexpr int kATile = kLanes * kRowBytes;
  static constexpr int kBTile = ND * kBRows * kRowBytes;
  static constexpr int kAPart = A_MN ? kK * kRowBytes : kATile;        // from one part to the next
  static constexpr int kBPart = B_MN ? kK * kRowBytes : kBTile;
  static constexpr int kStage = PA * kATile + PB * kBTile;
  static constexpr int kSmem = STAGES * kStage + 1024;
  // with several parts the products of lower parts (2^-11 of the first and
  // less) have columns of their own: the tensor core truncates each addition
  // at the accumulator's magnitude
  static constexpr bool kSmallApart = PA > 1 || PB > 1;
  static constexpr int kAccCols = kN <= 128 && !kSmallApart ? 128 : 256;   // columns from one accumulator to the other
  static_assert(!kSmallApart || 2 * kN <= kAccCols, "both sums fit");
  static constexpr int kTmemCols = 2 * kAccCols;
  static_assert(kSmem + 16 * R + 512 <= 227 * 1024, "stages, row scales and barriers fit in shared memory");
  static_assert(R % 64 == 0 && kN <= 256 && kN % 32 == 0 && kBRows % 8 == 0 && kBTile % 1024 == 0, "tile shape");
  static_assert(KIND != kI8 || (PA == 1 && PB == 1 && !B_MN), "integer operands");
  static_assert(KIND == kI8 || (ND == 1 && A_MN), "16-bit operands");
};

struct GemmArgs {
  CUtensorMap a, b;
  int32_t M, R, kblocks, tiles_m, tiles_r;
  int32_t shares, share_blocks;            // pairs: parts of the contraction, k-blocks of each
  int64_t share_stride;                    // and elements of Y from one part's sums to the next
  uint32_t* flags;
  uint64_t wait_ns;                        // limit of the MMAs' and the epilogue's waits
  Act8Out out;
};

// Instruction descriptor: fp32 sums (accumulator code 1) of halves (type code
// 0), or int32 sums (code 2) of signed 8-bit integers (1).
template <class C>
__host__ __device__ constexpr uint32_t idesc() {
  return ((C::KIND == kI8 ? 2u : 1u) << 4) | ((C::KIND == kHalf ? 0u : 1u) * ((1u << 7) | (1u << 10))) |
         (uint32_t(C::A_MN) << 15) | (uint32_t(C::B_MN) << 16) | (uint32_t(C::kN >> 3) << 17) |
         (uint32_t((C::CG * kLanes) >> 4) << 24);
}

template <int KIND, int CG>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
#define S4_MMA(group, kind)                                               \
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"          \
               "tcgen05.mma.cta_group::" group ".kind::" kind " [%0], %1, %2, %3, p;\n\t}" \
               ::"r"(d), "l"(a), "l"(b), "r"(id), "r"(acc) : "memory")
  if (KIND == kI8) {
    if (CG == 2) S4_MMA("2", "i8"); else S4_MMA("1", "i8");
  } else {
    if (CG == 2) S4_MMA("2", "f16"); else S4_MMA("1", "f16");
  }
#undef S4_MMA
}

// Shared-memory address of the same variable in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// The kernel before this one on the stream may still run (a programmatic
// launch): from here on its results are visible.  Weight codes are older
// than that kernel, so they are fetched before the wait.
__device__ __forceinline__ void wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Tile load whose bytes count on a barrier of either CTA of the pair.
template <int CG>
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* map, int x, int y, int plane, uint32_t bar) {
  if (CG == 2)
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 "
        "[%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(plane), "r"(bar) : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(plane), "r"(bar) : "memory");
}
// Whether the barrier's phase is complete, without waiting for it.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity) : "memory");
  return ok != 0;
}
// Arrive on the barrier (of every CTA of the pair) once the MMAs issued so far are done.
template <int CG>
__device__ __forceinline__ void commit(uint64_t* bar) {
  if (CG == 2)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
        ::"r"(smem_u32(bar)), "h"(uint16_t(3)) : "memory");
  else
    mma_commit(bar);
}

// K-major (128-byte swizzle): rows of 128 B, 8-row groups 1024 B apart; an
// MMA's k (32 bytes) lies along the row; the planes of a box follow one
// another.  MN-major: boxes of 128 bytes of rows by kK k's by all planes, one
// box per 128 bytes of rows; 8-k groups 1024 B apart, an MMA's k is 32 (int8)
// or 16 (16-bit) box rows.  addr: the tile's shared address / 16 (below 2^14,
// so offsets add without a carry); only the low word depends on it.
template <class C, bool MN, int PLANES>
__device__ __forceinline__ uint64_t tile_desc(uint32_t addr, int kk) {
  constexpr uint32_t kStep = MN ? (C::KIND == kI8 ? 4096 : 2048) : 32, kLead = MN ? PLANES * C::kK * kRowBytes : 16;
  constexpr uint32_t hi = (1024u >> 4) | (1u << 14) | (2u << 29);   // group stride, version, 128-byte swizzle
  const uint32_t lo = (addr + uint32_t(kk) * (kStep >> 4)) | ((kLead >> 4) << 16);
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
  return d;
}
// One lane of a converged warp.
__device__ __forceinline__ bool elected() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// Rows mn0 .. mn0 + rows - 1 by k0 .. k0 + kK - 1 of every plane of an operand.
template <class C, bool MN, int ROWS, int PLANES>
__device__ __forceinline__ void load_tile(const CUtensorMap* map, int mn0, int k0, uint32_t dst, uint32_t bar) {
  if (!MN) {
    load_box<C::CG>(dst, map, k0, mn0, 0, bar);
  } else {
    constexpr int kWide = C::KIND == kI8 ? 128 : 64;                // elements of 128 bytes
#pragma unroll
    for (int g = 0; g < (ROWS + kWide - 1) / kWide; ++g)
      load_box<C::CG>(dst + g * PLANES * C::kK * kRowBytes, map, mn0 + kWide * g, k0, 0, bar);
  }
}

// Tile t in an order that keeps the tiles in flight close in both operands:
// groups of 8 column tiles, walked row tile by row tile.
__device__ __forceinline__ void tile_of(const GemmArgs& g, int t, int& tm, int& tr) {
  const int per = 8 * g.tiles_r;
  const int grp = t / per, x = t - grp * per;
  const int cols = min(8, g.tiles_m - 8 * grp);
  tr = x / cols;
  tm = 8 * grp + (x - tr * cols);
}

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void put(__half* p, float x) { *p = __float2half_rn(x); }

// A chunk of 32 rows (TMEM columns) of this lane's column m.
template <class C>
__device__ __forceinline__ void load_chunk(uint32_t tacc, int i, float (&v)[32]) {
  uint32_t r[32];
  if (C::ND == 1) {
    tmem_ld32(tacc + uint32_t(32 * i), r);
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = C::KIND == kI8 ? __int2float_rn(int(r[j])) : __uint_as_float(r[j]);
    if (C::kSmallApart) {
      tmem_ld32(tacc + uint32_t(C::kN + 32 * i), r);
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] += __uint_as_float(r[j]);
    }
  } else {
    // MMA columns: [CTA half][digit][row of the half]
    constexpr int kPer = C::kBRows / 32;
    const uint32_t c = tacc + uint32_t((i / kPer) * C::ND * C::kBRows + 32 * (i % kPer));
    static_assert(C::ND == 1 || C::kBRows % 32 == 0, "a chunk lies in one half");
    tmem_ld32(c, r);
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = __int2float_rn(int(r[j]));
#pragma unroll
    for (int d = 1; d < C::ND; ++d) {
      tmem_ld32(c + uint32_t(d * C::kBRows), r);
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = fmaf(v[j], 256.0f, __int2float_rn(int(r[j])));
    }
  }
}

// Two 16-bit results in one word.
__device__ __forceinline__ uint32_t pack_pair(__nv_bfloat16*, float lo, float hi) {
  const __nv_bfloat162 x = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&x);
}
__device__ __forceinline__ uint32_t pack_pair(__half*, float lo, float hi) {
  const __half2 x = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&x);
}

// 32 rows r0.. of column m to Y: a store instruction writes 32 consecutive
// columns of a row, or, of 16-bit results whose rows are 4-byte aligned, a
// pair of columns per lane for two rows (neighbouring lanes swap two rows'
// halves).  rs: the rows' scales in shared memory (null: none), read four at a
// time.  A chunk inside the matrix goes out without a test per row.  The
// epilogue is bound by shuffles, shared memory and store instructions: one
// shuffle and one store per row took 5.5 us for a pair's tile of 256 rows, as
// long as 2300 of contraction; this takes 4.3.
template <class T>
__device__ __forceinline__ void store_chunk(const Act8Out& o, int R, int M, int r0, int m, float cs, float bias,
                                            const float* rs, float (&v)[32]) {
  T* y = static_cast<T*>(o.y) + int64_t(r0) * o.ld + m;
  if (rs) {
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
      const float4 s = *reinterpret_cast<const float4*>(rs + j);
      v[j] *= s.x;
      v[j + 1] *= s.y;
      v[j + 2] *= s.z;
      v[j + 3] *= s.w;
    }
  }
#pragma unroll
  for (int j = 0; j < 32; ++j) v[j] = fmaf(v[j], cs, bias);
  const bool whole = !o.accumulate && r0 + 32 <= R && __all_sync(0xffffffffu, m < M);
  if constexpr (sizeof(T) == 2) {
    if (whole && ((reinterpret_cast<uintptr_t>(o.y) | uintptr_t(o.ld * 2)) & 3) == 0) {
      const bool odd = m & 1;
      uint32_t* p = reinterpret_cast<uint32_t*>(y - (odd ? 1 : 0) + (odd ? 2 : 0) * o.ld);   // even lanes rows 4k, odd 4k + 2
      const int64_t step = o.ld / 2;                          // words
#pragma unroll
      for (int j = 0; j < 32; j += 4) {
        const uint32_t a = pack_pair(y, v[j], v[j + 1]), b = pack_pair(y, v[j + 2], v[j + 3]);
        const uint32_t mine = odd ? b : a, other = __shfl_xor_sync(0xffffffffu, odd ? a : b, 1);
        const uint32_t left = odd ? other : mine, right = odd ? mine : other;   // columns m & ~1 and m | 1
        p[j * step] = __byte_perm(left, right, 0x5410);
        p[(j + 1) * step] = __byte_perm(left, right, 0x7632);
      }
      return;
    }
  }
  if (whole) {
#pragma unroll
    for (int j = 0; j < 32; ++j) put(y + int64_t(j) * o.ld, v[j]);
  } else if (m < M) {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (r0 + j < R) {
        T* p = y + int64_t(j) * o.ld;
        put(p, o.accumulate ? v[j] + to_f32(*p) : v[j]);
      }
  }
}
__device__ __forceinline__ void store_any(const Act8Out& o, int R, int M, int r0, int m, float cs, float bias,
                                          const float* rs, float (&v)[32]) {
  if (o.dtype == ACT8_FP32) store_chunk<float>(o, R, M, r0, m, cs, bias, rs, v);
  else if (o.dtype == ACT8_BF16) store_chunk<__nv_bfloat16>(o, R, M, r0, m, cs, bias, rs, v);
  else store_chunk<__half>(o, R, M, r0, m, cs, bias, rs, v);
}
// Written by the pass that this kernel may overlap, so not through the
// read-only path: that holds for memory nobody writes while the kernel runs.
__device__ __forceinline__ float row_scale(const Act8Out& o, int R, int r) {
  return o.row_scale && r < R ? __ldcg(o.row_scale + r) : 1.0f;
}

template <class C>
__global__ void __launch_bounds__(kPairThreads, 1) k_act8_gemm(const __grid_constant__ GemmArgs g) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t full_bar[C::STAGES], empty_bar[C::STAGES], acc_full[2], acc_empty[2], done_bar;
  __shared__ uint32_t tmem_slot;
  __shared__ __align__(16) float row_scales[8][C::R / 2];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = C::CG == 2 ? cta_rank() : 0u;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&acc_full[s], 1);
      mbar_init(&acc_empty[s], 8 * C::CG);
    }
    mbar_init(&done_bar, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    if (C::CG == 2) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)),
                   "r"(C::kTmemCols) : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)),
                   "r"(C::kTmemCols) : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
  }
  fence_before_sync();
  __syncthreads();
  if (C::CG == 2) cluster_sync();
  fence_after_sync();
  const uint32_t tmem = tmem_slot;
  const int shares = C::CHUNK ? g.shares : 1, items = g.tiles_m * g.tiles_r * shares, kblocks = g.kblocks;
  const int first = blockIdx.x / C::CG, step = gridDim.x / C::CG;
  const int chunk = C::CHUNK ? C::CHUNK : max(kblocks, 1);

  if (warp == 0) {
    // ---- loads.  The whole warp walks the loop and one lane issues, a box over
    // all planes of an operand: four boxes a k-block from one lane's branch
    // took longer to issue than the digits' products take (903 against 755 us
    // for the weight gradient of 8192 x 4096 x 11008).
    const uint32_t base = smem_u32(smem);
    int s = 0, filled = 0;
    uint32_t phase = 1;                                     // of the stage's release before this fill
    bool ok = true, ready = false;
    wait_previous();
    for (int t = first; ok && t < items; t += step) {
      int tm, tr;
      tile_of(g, t / shares, tm, tr);
      const int m0 = (tm * C::CG + int(rank)) * kLanes, r0 = tr * C::R + int(rank) * C::kBRows;
      const int kb_end = min(kblocks, (t % shares + 1) * g.share_blocks);
      for (int kb = t % shares * g.share_blocks; kb < kb_end; ++kb) {
        if (!__all_sync(0xffffffffu, ready)) {
          ok = __all_sync(0xffffffffu, mbar_wait(&empty_bar[s], phase));
          if (!ok) break;
        }
        if (elected()) {
          const uint32_t dst = base + uint32_t(s) * C::kStage;
          uint32_t bar = smem_u32(&full_bar[s]);
          if (rank == 0) mbar_expect_tx(&full_bar[s], C::CG * C::kStage);
          if (C::CG == 2) bar = in_cta(bar, 0);
          load_tile<C, C::A_MN, kLanes, C::PA>(&g.a, m0, kb * C::kK, dst, bar);
          load_tile<C, C::B_MN, C::kBRows, C::PB * C::ND>(&g.b, r0, kb * C::kK, dst + C::PA * C::kATile, bar);
        }
        __syncwarp();
        filled = min(filled + 1, C::STAGES);
        if (++s == C::STAGES) {
          s = 0;
          phase ^= 1u;
        }
        ready = mbar_test(&empty_bar[s], phase);
      }
    }
    // every stage this CTA filled has been read before it leaves
    for (; filled > 0 && ok; --filled) {
      int last = s - filled;
      uint32_t ph = phase;
      if (last < 0) {
        last += C::STAGES;
        ph ^= 1u;
      }
      ok = mbar_wait(&empty_bar[last], ph ^ 1u);
    }
    if (!ok && lane == 0 && g.flags) atomicOr(g.flags, SHAMPOO4_FLAG_TIMEOUT);
  } else if (warp == 1) {
    // ---- products.  The whole warp walks the loop, so that descriptors stay
    // in uniform registers, and one lane issues; the next stage's barrier is
    // tried under the MMAs just issued.  (With the loop inside one lane's
    // branch the issue, about 600 clocks a k-block, was the bound: 266 against
    // 234 us at 8192 x 11008 x 4096.)
    if (rank == 0) {
      wait_previous();                                      // the limits count from here on
      constexpr uint32_t id = idesc<C>();
      constexpr int kParts = C::PA > C::PB ? C::PA : C::PB;
      const uint32_t base = smem_u32(smem) >> 4;
      int s = 0, i = 0;
      uint32_t phase = 0;
      bool ok = true, ready = false;                        // ready: the next stage's loads have landed already
      for (int t = first; ok && t < items; t += step) {
        const int kb_end = min(kblocks, (t % shares + 1) * g.share_blocks);
        bool some = true;                                   // no k-blocks at all: an empty sum
        for (int kb = t % shares * g.share_blocks; ok && some; ++i) {
          const int ab = i & 1;
          ok = __all_sync(0xffffffffu, mbar_wait(&acc_empty[ab], ((i >> 1) & 1) ^ 1, g.wait_ns));
          if (!ok) break;
          fence_after_sync();
          const uint32_t d = tmem + uint32_t(ab * C::kAccCols);
          const int k_end = min(kb + chunk, kb_end);
          const int k_first = kb;
          for (; kb < k_end; ++kb) {
            if (!__all_sync(0xffffffffu, ready)) {
              ok = __all_sync(0xffffffffu, mbar_wait(&full_bar[s], phase, g.wait_ns));
              if (!ok) break;
            }
            fence_after_sync();
            const uint32_t a0 = base + uint32_t(s) * (C::kStage >> 4), b0 = a0 + ((C::PA * C::kATile) >> 4);
            if (elected()) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                for (int pa = 0; pa < C::PA; ++pa)
#pragma unroll
                  for (int pb = 0; pb < C::PB; ++pb)
                    if (pa + pb < kParts) {
                      // the first product into each of the two sums overwrites it
                      const bool opens = pa + pb == 0 || (C::PB > 1 ? pa == 0 && pb == 1 : pa == 1);
                      mma<C::KIND, C::CG>(d + (pa + pb > 0 ? C::kN : 0),
                                          tile_desc<C, C::A_MN, C::PA>(a0 + ((pa * C::kAPart) >> 4), kk),
                                          tile_desc<C, C::B_MN, C::PB>(b0 + ((pb * C::kBPart) >> 4), kk),
                                          id,
                                          !(opens && kb == k_first && kk == 0));
                    }
              commit<C::CG>(&empty_bar[s]);
            }
            __syncwarp();
            if (++s == C::STAGES) {
              s = 0;
              phase ^= 1u;
            }
            ready = mbar_test(&full_bar[s], phase);         // under the MMAs just issued
          }
          if (ok && elected()) commit<C::CG>(&acc_full[ab]);
          __syncwarp();
          some = kb < kb_end;
        }
      }
      // all MMAs issued are finished before tensor memory is freed
      if (elected()) {
        if (C::CG == 2)
          asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
              smem_u32(&done_bar)) : "memory");
        else
          mma_commit(&done_bar);
      }
      __syncwarp();
      if (!mbar_wait(&done_bar, 0)) ok = false;
      if (!ok && lane == 0 && g.flags) atomicOr(g.flags, SHAMPOO4_FLAG_TIMEOUT);
    }
  } else {                                                  // ---- epilogue, warps 2..9
    const int q = warp & 3;                                 // TMEM lane quarter
    constexpr int kChunks = C::R / 64;                      // of this warp: half of the tile's
    const int c0 = (warp - 2) / 4 * kChunks;
    int i = 0;
    bool ok = true;
    wait_previous();
    for (int t = first; ok && t < items; t += step) {
      int tm, tr;
      tile_of(g, t / shares, tm, tr);
      const int m = (tm * C::CG + int(rank)) * kLanes + 32 * q + lane, r0 = tr * C::R + 32 * c0;
      const float cs = g.out.col_scale && m < g.M
                           ? __ldcg(g.out.col_scale + (C::KIND == kHalf ? m >> g.out.col_shift : m)) : 1.0f;
      const float bias = g.out.bias && m < g.M ? __ldg(g.out.bias + m) : 0.0f;
      float* rs = g.out.row_scale ? row_scales[warp - 2] : nullptr;   // fetched under the products
      if (rs) {
        __syncwarp();
#pragma unroll
        for (int c = 0; c < kChunks; ++c) rs[32 * c + lane] = row_scale(g.out, g.R, r0 + 32 * c + lane);
        __syncwarp();
      }
      const int share = t % shares, blocks = min(kblocks - share * g.share_blocks, g.share_blocks);
      const int passes = max(1, (blocks + chunk - 1) / chunk);
      Act8Out out = g.out;
      if (C::CHUNK) out.y = static_cast<float*>(out.y) + (shares > 1 ? share * g.share_stride : 0);
      float sum[C::CHUNK ? kChunks : 1][32];
      for (int pass = 0; pass < passes; ++pass, ++i) {
        const int ab = i & 1;
        // the whole warp goes on or stops: what follows is collective
        if (!__all_sync(0xffffffffu, mbar_wait(&acc_full[ab], (i >> 1) & 1, g.wait_ns))) {
          if (g.flags && lane == 0) atomicOr(g.flags, SHAMPOO4_FLAG_TIMEOUT);
          ok = false;
          break;
        }
        fence_after_sync();
        const uint32_t tacc = tmem + uint32_t(ab * C::kAccCols) + (uint32_t(32 * q) << 16);
        if (C::CHUNK) {
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            float v[32];
            if (kblocks > 0) load_chunk<C>(tacc, c0 + c, v);
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const float x = kblocks > 0 ? v[j] : 0.0f;
              sum[c][j] = pass == 0 ? x : sum[c][j] + x;
            }
          }
        } else {
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            if (r0 + 32 * c >= g.R) break;
            float v[32];
            if (kblocks > 0) {
              load_chunk<C>(tacc, c0 + c, v);
            } else {
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] = 0.0f;
            }
            store_any(g.out, g.R, g.M, r0 + 32 * c, m, cs, bias, rs ? rs + 32 * c : nullptr, v);
          }
        }
        fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          if (C::CG == 2)
            // relaxed: the accumulator is in registers (its loads are complete), and a release would
            // wait for the results' stores (54 against 41 us for a 4096 x 4096 weight gradient of 64 tokens)
            asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                in_cta(smem_u32(&acc_empty[ab]), 0)) : "memory");
          else
            mbar_arrive(&acc_empty[ab]);
        }
      }
      if (C::CHUNK && ok) {
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          if (r0 + 32 * c < g.R) {
            if (C::KIND == kHalf) {
              // powers of two, the smaller first: their product may lie outside fp32 where the result
              // does not, and the other way round a step might
#pragma unroll
              for (int j = 0; j < 32; ++j) {
                const float f = rs[32 * c + j];
                sum[c][j] = sum[c][j] * fminf(f, cs) * fmaxf(f, cs);
              }
              store_any(out, g.R, g.M, r0 + 32 * c, m, 1.0f, 0.0f, nullptr, sum[c]);
            } else {
              store_any(out, g.R, g.M, r0 + 32 * c, m, cs, bias, rs ? rs + 32 * c : nullptr, sum[c]);
            }
          }
        }
      }
    }
  }
  fence_before_sync();
  __syncthreads();
  if (C::CG == 2) cluster_sync();
  __syncwarp();
  if (warp == 1) {
    fence_after_sync();
    if (C::CG == 2)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kTmemCols) : "memory");
    else
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kTmemCols) : "memory");
  }
}

// Columns m .. m + 3 of row r to Y.
template <class T>
__device__ __forceinline__ void store_row4(const Act8Out& o, int r, int m, int M, float (&v)[4]) {
  T* p = static_cast<T*>(o.y) + int64_t(r) * o.ld + m;
  struct alignas(4 * sizeof(T)) V4 { T e[4]; };
  if (!o.accumulate && m + 4 <= M && reinterpret_cast<uintptr_t>(p) % (4 * sizeof(T)) == 0) {
    V4 w;
#pragma unroll
    for (int e = 0; e < 4; ++e) put(&w.e[e], v[e]);
    *reinterpret_cast<V4*>(p) = w;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (m + e < M) put(p + e, o.accumulate ? v[e] + to_f32(p[e]) : v[e]);
  }
}

// ---------------------------------------------------------------------------
// Small products (few rows, or too few tiles for the pairs): one CTA per 128
// columns by R rows and per share of the contraction, a cluster of up to 8
// CTAs per tile.  Bound by reading A once (few rows) or by latency, so the
// shares fill the SMs, two CTAs each; their integer partial sums meet in
// shared memory, each CTA of the cluster finishing R / cluster rows (exact,
// so the split changes no result).  Same roles as above, warps 2..5 finish.
// One row, 4096 x 4096: 10 us with cold caches, 7.4 with the row's
// quantization where W is in L2; 13 rows, 11008 x 4096: 14 us cold, 3.2 TB/s.
template <bool A_MN_, int R_, int ND_, int STAGES_>
struct SmallCfg {
  static constexpr int KIND = kI8, R = R_, ND = ND_, CG = 1, STAGES = STAGES_;
  static constexpr bool A_MN = A_MN_, B_MN = false;
  static constexpr int kK = 128, kN = ND * R, kBRows = R;
  static constexpr int kATile = kLanes * kRowBytes;
  static constexpr int kBTile = kN * kRowBytes;
  static constexpr int kStage = kATile + kBTile;
  static constexpr int kCols = (kN + 31) / 32 * 32;            // columns drained
  static constexpr int kTmemCols = kCols <= 32 ? 32 : (kCols <= 64 ? 64 : (kCols <= 128 ? 128 : 256));
  static constexpr int kSmem = STAGES * kStage + 1024;
  static_assert(kN % 16 == 0 && kN <= 256 && kBTile % 1024 == 0, "tile shape");
  static_assert(kCols * kLanes * 4 <= STAGES * kStage, "the partial sums reuse the stages");
  static_assert(2 * (kSmem + 1024 + 1024) <= 228 * 1024, "two CTAs per SM");
};

template <class C>
__global__ void __launch_bounds__(kSmallThreads, 2) k_act8_small(const __grid_constant__ GemmArgs g) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t full_bar[C::STAGES], empty_bar[C::STAGES], done_bar;
  __shared__ uint32_t tmem_slot;
  __shared__ __align__(16) float scales[4][32];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int shares = gridDim.y, share = blockIdx.y;           // the cluster lies along y
  const int kb0 = int(int64_t(g.kblocks) * share / shares), kb1 = int(int64_t(g.kblocks) * (share + 1) / shares);
  const int m0 = int(blockIdx.x % unsigned(g.tiles_m)) * kLanes, r0 = int(blockIdx.x / unsigned(g.tiles_m)) * C::R;
  auto load_a = [&](int it, int s) {
    mbar_expect_tx(&full_bar[s], C::kStage);
    load_tile<C, C::A_MN, kLanes, 1>(&g.a, m0, (kb0 + it) * C::kK, smem_u32(smem + s * C::kStage),
                                     smem_u32(&full_bar[s]));
  };
  auto load_b = [&](int it, int s) {
    load_tile<C, false, C::R, C::ND>(&g.b, r0, (kb0 + it) * C::kK, smem_u32(smem + s * C::kStage) + C::kATile,
                                     smem_u32(&full_bar[s]));
  };
  const int n = kb1 - kb0, lead = min(n, C::STAGES);
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    mbar_init(&done_bar, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    for (int it = 0; it < lead; ++it) load_a(it, it);       // under the tensor memory allocation
    if (n > 0) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&g.b)) : "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)),
                 "r"(C::kTmemCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = tmem_slot;

  if (warp == 0) {
    if (lane == 0) {                                        // ---- loads
      bool ok = true;
      wait_previous();
      int it = 0;
      for (; it < lead; ++it) load_b(it, it);
      for (; it < n; ++it) {
        const int s = it % C::STAGES;
        if (!mbar_wait(&empty_bar[s], ((it / C::STAGES) & 1) ^ 1)) { ok = false; break; }
        load_a(it, s);
        load_b(it, s);
      }
      for (int i = max(0, it - C::STAGES); i < it; ++i)     // everything loaded has landed before the CTA leaves
        if (!mbar_wait(&full_bar[i % C::STAGES], (i / C::STAGES) & 1)) ok = false;
      if (!ok && g.flags) atomicOr(g.flags, SHAMPOO4_FLAG_TIMEOUT);
    }
  } else if (warp == 1) {                                   // ---- products (the whole warp, as above)
    constexpr uint32_t id = (2u << 4) | (1u << 7) | (1u << 10) | (uint32_t(C::A_MN) << 15) |
                            (uint32_t(C::kN >> 3) << 17) | (uint32_t(kLanes >> 4) << 24);
    const uint32_t base = smem_u32(smem) >> 4;
    bool ok = true;
    wait_previous();                                        // the limits count from here on
    for (int it = 0; it < kb1 - kb0; ++it) {
      const int s = it % C::STAGES;
      ok = __all_sync(0xffffffffu, mbar_wait(&full_bar[s], (it / C::STAGES) & 1, g.wait_ns));
      if (!ok) break;
      fence_after_sync();
      const uint32_t a0 = base + uint32_t(s) * (C::kStage >> 4), b0 = a0 + (C::kATile >> 4);
      if (elected()) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma<kI8, 1>(tmem, tile_desc<C, C::A_MN, 1>(a0, kk), tile_desc<C, false, 1>(b0, kk), id, (it | kk) != 0);
        mma_commit(&empty_bar[s]);
      }
      __syncwarp();
    }
    if (elected()) mma_commit(&done_bar);
    __syncwarp();
    if (!mbar_wait(&done_bar, 0)) ok = false;
    if (!ok && lane == 0 && g.flags) atomicOr(g.flags, SHAMPOO4_FLAG_TIMEOUT);
  }
  // Every load has landed and every MMA is done (or timed out).
  __syncthreads();
  const int q = warp & 3;
  const bool any = kb1 > kb0;
  if (warp >= 2) {
    wait_previous();
    fence_after_sync();
  }
  if (shares == 1) {                                        // straight from tensor memory
    if (warp >= 2) {
      const int m = m0 + 32 * q + lane;
      const float cs = g.out.col_scale && m < g.M ? __ldg(g.out.col_scale + m) : 1.0f;
      const float bias = g.out.bias && m < g.M ? __ldg(g.out.bias + m) : 0.0f;
#pragma unroll 1
      for (int c = 0; c < C::R && r0 + c < g.R; c += 32) {
        float v[32];
        const uint32_t at = tmem + uint32_t(c) + (uint32_t(32 * q) << 16);
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = 0.0f;
        if (any) {
#pragma unroll
          for (int d = 0; d < C::ND; ++d) {
            uint32_t r[32];
            tmem_ld32(at + uint32_t(d * C::R), r);
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = fmaf(v[j], 256.0f, __int2float_rn(int(r[j])));
          }
        }
        __syncwarp();
        scales[warp - 2][lane] = c + lane < C::R ? row_scale(g.out, g.R, r0 + c + lane) : 1.0f;
        __syncwarp();
        store_any(g.out, min(g.R, r0 + C::R), g.M, r0 + c, m, cs, bias, scales[warp - 2], v);
      }
      fence_before_sync();
    }
  } else {
    // the stages become the partial sums, columns of 128 integers; a warp then
    // finishes a row at a time, four columns per lane
    int32_t* part = reinterpret_cast<int32_t*>(smem);
    if (warp >= 2) {
#pragma unroll 1
      for (int c = 0; c < C::kCols; c += 32) {
        uint32_t r[32];
        tmem_ld32(tmem + uint32_t(c) + (uint32_t(32 * q) << 16), r);
#pragma unroll
        for (int j = 0; j < 32; ++j) part[(c + j) * kLanes + 32 * q + lane] = any ? int32_t(r[j]) : 0;
      }
      fence_before_sync();
    }
    __syncthreads();
    cluster_sync();
    if (warp >= 2) {
      const int per = (C::R + shares - 1) / shares, j_end = min(min((share + 1) * per, C::R), g.R - r0);
      const uint32_t base = smem_u32(part) + uint32_t(lane) * 16u;
      const int m = m0 + 4 * lane;
#pragma unroll 4
      for (int j = share * per + q; j < j_end; j += 4) {
        float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int d = 0; d < C::ND; ++d) {
          int sum[4] = {0, 0, 0, 0};
          const uint32_t at = base + uint32_t((d * C::R + j) * kLanes) * 4u;
#pragma unroll 4
          for (int k = 0; k < shares; ++k) {
            int x[4];
            asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(in_cta(at, uint32_t(k))) : "memory");
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[e] += x[e];
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = fmaf(v[e], 256.0f, __int2float_rn(sum[e]));
        }
        const float rs = row_scale(g.out, g.R, r0 + j);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float cs = g.out.col_scale && m + e < g.M ? __ldg(g.out.col_scale + m + e) : 1.0f;
          const float bias = g.out.bias && m + e < g.M ? __ldg(g.out.bias + m + e) : 0.0f;
          v[e] = fmaf(v[e] * rs, cs, bias);
        }
        if (g.out.dtype == ACT8_FP32) store_row4<float>(g.out, r0 + j, m, g.M, v);
        else if (g.out.dtype == ACT8_BF16) store_row4<__nv_bfloat16>(g.out, r0 + j, m, g.M, v);
        else store_row4<__half>(g.out, r0 + j, m, g.M, v);
      }
    }
  }
  if (shares > 1) cluster_sync();                           // nobody leaves while its sums are read
  else __syncthreads();
  __syncwarp();
  if (warp == 1) {
    fence_after_sync();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kTmemCols) : "memory");
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

// Tensor map of an operand's planes (rows x cols each, row-major), box of
// 128 bytes of a row by box_rows by all planes, 128-byte swizzle, zeros
// outside a plane.
shampoo4_status encode(CUtensorMap* out, int kind, const Act8Operand& x, int64_t rows, int64_t cols, int planes,
                       int box_rows) {
  auto fn = encoder();
  if (!fn) return SHAMPOO4_ERR_CUDA;
  const int64_t esize = kind == kI8 ? 1 : 2;
  if ((x.ld * esize) % 16 != 0 || reinterpret_cast<uintptr_t>(x.p) % 16 != 0) return SHAMPOO4_ERR_INVALID_ARG;
  cuuint64_t dims[3] = {cuuint64_t(cols), cuuint64_t(rows), cuuint64_t(planes)};
  cuuint64_t strides[2] = {cuuint64_t(x.ld * esize), cuuint64_t(planes > 1 ? x.plane * x.ld * esize : x.ld * esize)};
  cuuint32_t box[3] = {cuuint32_t(128 / esize), cuuint32_t(box_rows), cuuint32_t(planes)};
  cuuint32_t estr[3] = {1u, 1u, 1u};
  const CUresult r = fn(out, kind == kI8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                        const_cast<void*>(x.p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? SHAMPOO4_OK : SHAMPOO4_ERR_CUDA;
}

// Per-device facts, looked up once.
constexpr int kMaxDevices = 64;
shampoo4_status device_sms(int* dev, int* sms) {
  static std::atomic<int> known[kMaxDevices];
  S4_CUDA(cudaGetDevice(dev));
  if (*dev < 0 || *dev >= kMaxDevices) return SHAMPOO4_ERR_UNSUPPORTED;
  *sms = known[*dev].load(std::memory_order_relaxed);
  if (*sms == 0) {
    S4_CUDA(cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, *dev));
    known[*dev].store(*sms, std::memory_order_relaxed);
  }
  return SHAMPOO4_OK;
}
template <class C>
shampoo4_status allow_smem(const void* kern, int dev) {
  static std::atomic<bool> done[kMaxDevices];
  if (!done[dev].load(std::memory_order_acquire)) {
    S4_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem));
    done[dev].store(true, std::memory_order_release);
  }
  return SHAMPOO4_OK;
}

template <class C>
shampoo4_status fill_args(GemmArgs& g, const Act8Operand& a, int a_planes, const Act8Operand& b, int b_planes,
                          int64_t M, int64_t R, int64_t K, const Act8Out& out, Act8Watch watch) {
  g.out = out;
  g.flags = watch.flags;
  g.wait_ns = watch.wait_ns == 0 || watch.wait_ns > kWaitNs ? kWaitNs : watch.wait_ns;
  g.M = int32_t(M);
  g.R = int32_t(R);
  g.kblocks = int32_t((K + C::kK - 1) / C::kK);
  if (K > 0) {
    S4_TRY(C::A_MN ? encode(&g.a, C::KIND, a, K, M, a_planes, C::kK) : encode(&g.a, C::KIND, a, M, K, a_planes, kLanes));
    S4_TRY(C::B_MN ? encode(&g.b, C::KIND, b, K, R, b_planes, C::kK)
                   : encode(&g.b, C::KIND, b, R, K, b_planes, C::kBRows));
  }
  const int64_t tm = (M + C::CG * kLanes - 1) / (C::CG * kLanes), tr = (R + C::R - 1) / C::R;
  if (tm * tr > INT_MAX / 16) return SHAMPOO4_ERR_INVALID_ARG;
  g.tiles_m = int32_t(tm);
  g.tiles_r = int32_t(tr);
  g.shares = 1;
  g.share_blocks = g.kblocks;
  return SHAMPOO4_OK;
}

// after_pass: the kernel enqueued just before on this stream is this call's
// own operand pass, so the launch may overlap its end.
template <class K>
shampoo4_status start(K kern, int threads, dim3 grid, dim3 cluster, int smem, bool after_pass, const GemmArgs& g, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = size_t(smem);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster.x;
  attr[0].val.clusterDim.y = cluster.y;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = after_pass ? 2 : 1;
  S4_CUDA(cudaLaunchKernelEx(&cfg, kern, g));
  return SHAMPOO4_OK;
}

// shares > 1: Y receives that many fp32 sums of R x M, one after the other.
template <class C>
shampoo4_status launch(const Act8Operand& a, const Act8Operand& b, int64_t M, int64_t R, int64_t K,
                       const Act8Out& out, bool after_pass, Act8Watch watch, cudaStream_t st, int shares = 1) {
  GemmArgs g{};
  S4_TRY(fill_args<C>(g, a, C::PA, b, C::PB * C::ND, M, R, K, out, watch));
  if (shares > 1) {
    g.share_blocks = (g.kblocks + shares - 1) / shares;
    g.shares = shares;
    g.share_stride = M * R;
  }
  int dev = 0, sms = 0;
  S4_TRY(device_sms(&dev, &sms));
  auto kern = k_act8_gemm<C>;
  S4_TRY(allow_smem<C>(reinterpret_cast<const void*>(kern), dev));
  const int tiles = g.tiles_m * g.tiles_r * g.shares;
  return start(kern, kPairThreads, dim3(unsigned(C::CG * std::min(tiles, sms / C::CG))), dim3(C::CG), C::kSmem, after_pass, g, st);
}

template <class C>
shampoo4_status launch_small(const Act8Operand& a, const Act8Operand& b, int64_t M, int64_t R, int64_t K, int shares,
                             const Act8Out& out, bool after_pass, Act8Watch watch, cudaStream_t st) {
  GemmArgs g{};
  S4_TRY(fill_args<C>(g, a, 1, b, C::ND, M, R, K, out, watch));
  int dev = 0, sms = 0;
  S4_TRY(device_sms(&dev, &sms));
  auto kern = k_act8_small<C>;
  S4_TRY(allow_smem<C>(reinterpret_cast<const void*>(kern), dev));
  return start(kern, kSmallThreads, dim3(unsigned(g.tiles_m * g.tiles_r), unsigned(shares)), dim3(1, unsigned(shares)), C::kSmem,
               after_pass, g, st);
}

// Which form an integer product takes: the estimated time (us) of each,
// fitted to measurements on a B200 (1 to 2048 rows, 768 to 11008 columns, 6 to
// 86 k-blocks; its 148 SMs are in the rule: 74 pairs, two small CTAs per SM).
// The pairs: 8.3 and, per wave of tiles,
// 0.31 (digits 0.25) per k-block or the results' stores.  A small tile of n =
// rows x digits columns: 4.9 + 0.004 n, and 0.15 + 0.0006 n per k-block, half
// as much again or more when two CTAs share an SM; joining a split contraction
// 1 and 0.07 per row and digit a CTA finishes; each further wave starts anew.
Form choose_form(int64_t M, int64_t R, int64_t K, int pair_rows, int digits, const int* tile_rows, int forms) {
  const double kb = double((K + 127) / 128);
  const double pair_tiles = double((M + 255) / 256) * double((R + pair_rows - 1) / pair_rows);
  double best = 8.3 + std::max((digits == 1 ? 0.31 : 0.25) * kb, 1.6) * std::ceil(pair_tiles / 74);
  Form f{0, 1};
  for (int i = 0; i < forms; ++i)
    for (int s = 1; s <= 8 && s <= std::max(kb, 1.0); ++s) {
      const int rows = tile_rows[i];
      const double ctas = double((M + 127) / 128) * double((R + rows - 1) / rows) * s;
      const double n = double(rows) * digits, waves = std::ceil(ctas / 296);
      const double share = ctas <= 148 ? 1.0 : 1.45 + 0.0025 * n;
      const double join = s > 1 ? 1.0 + 0.07 * std::ceil(n / s) : 0.0;
      const double cost = 1.9 + waves * (3.0 + 0.004 * n + share * (0.15 + 0.0006 * n) * std::ceil(kb / s) + join);
      if (cost < best) best = cost, f = Form{rows, s};
    }
  return f;
}

}  // namespace

//                               kind   A_MN   B_MN   R   PA PB ND CG stages chunk
using CodesCfg = Cfg<            kI8,   false, false, 256, 1, 1, 1, 2, 6, 0>;
using DigitsCfg = Cfg<           kI8,   true,  false, 64,  1, 1, kAct8Digits, 2, 8, 1024>;
template <int PB, int STAGES>
using HalvesCfg = Cfg<           kHalf, true,  true,  128, 2, PB, 1, 2, STAGES, 4>;
// One half each.  The sum leaves the tensor core every 1024 k (64 additions,
// each cut off at 2^-22 of the sum at most: 2^-16, far below the bfloat16
// result).  4096 x 4096 x 4096: 105 us, against 99 for one sum per tile.
template <bool B_MN> using HalfCfg = Cfg<kHalf, true, B_MN, 256, 1, 1, 1, 2, 6, 16>;

Form act8_codes_form(int64_t M, int64_t R, int64_t K) {
  const int rows[] = {16, 64, 128};
  return choose_form(M, R, K, CodesCfg::R, 1, rows, 3);
}
Form act8_digits_form(int64_t M, int64_t R, int64_t K) {
  const int rows[] = {16, 32};
  // the small form keeps its integer sums whole
  return K <= kAct8MaxInner ? choose_form(M, R, K, DigitsCfg::R, kAct8Digits, rows, 2) : Form{0, 1};
}

shampoo4_status launch_act8_codes(const Act8Operand& a, const Act8Operand& b, int64_t M, int64_t R, int64_t K,
                                  const Act8Out& out, bool after_pass, Act8Watch watch, cudaStream_t st) {
  const Form f = act8_codes_form(M, R, K);
  if (f.rows == 16) return launch_small<SmallCfg<false, 16, 1, 5>>(a, b, M, R, K, f.shares, out, after_pass, watch, st);
  if (f.rows == 64) return launch_small<SmallCfg<false, 64, 1, 4>>(a, b, M, R, K, f.shares, out, after_pass, watch, st);
  if (f.rows == 128)
    return launch_small<SmallCfg<false, 128, 1, 3>>(a, b, M, R, K, f.shares, out, after_pass, watch, st);
  return launch<CodesCfg>(a, b, M, R, K, out, after_pass, watch, st);
}

shampoo4_status launch_act8_digits(const Act8Operand& a, const Act8Operand& b, int64_t M, int64_t R, int64_t K,
                                   const Act8Out& out, Act8Watch watch, cudaStream_t st) {
  const Form f = act8_digits_form(M, R, K);
  if (f.rows == 16)
    return launch_small<SmallCfg<true, 16, kAct8Digits, 4>>(a, b, M, R, K, f.shares, out, true, watch, st);
  if (f.rows == 32)
    return launch_small<SmallCfg<true, 32, kAct8Digits, 3>>(a, b, M, R, K, f.shares, out, true, watch, st);
  return launch<DigitsCfg>(a, b, M, R, K, out, true, watch, st);
}

// The estimated time (us): 0.5 per k-block and 2 per wave of tiles; the join
// 3 and reading the sums.  Every share gets a k-block.
int act8_halves_shares(int64_t M, int64_t R, int64_t K) {
  const int64_t kb = (K + HalvesCfg<2, 4>::kK - 1) / HalvesCfg<2, 4>::kK;
  const double tiles = double((M + 255) / 256) * double((R + HalvesCfg<2, 4>::R - 1) / HalvesCfg<2, 4>::R);
  int best = 1;
  double least = 0.0;
  for (int64_t s = 1; s <= 32 && s <= kb; ++s) {
    const int64_t per = (kb + s - 1) / s;
    if ((kb + per - 1) / per != s) continue;
    const double cost = std::ceil(tiles * double(s) / 74) * (0.5 * double(per) + 2.0) +
                        (s > 1 ? 3.0 + double(s) * double(M) * double(R) * 1e-6 : 0.0);
    if (s == 1 || cost < least) least = cost, best = int(s);
  }
  return best;
}

shampoo4_status launch_act8_halves(const Act8Operand& a, int a_parts, const Act8Operand& b, int b_parts, int64_t M,
                                   int64_t R, int64_t K, int shares, const Act8Out& out, Act8Watch watch,
                                   cudaStream_t st) {
  if (a_parts == 1) return launch<HalfCfg<true>>(a, b, M, R, K, out, true, watch, st, shares);
  return b_parts == 1 ? launch<HalvesCfg<1, 5>>(a, b, M, R, K, out, true, watch, st, shares)
                      : launch<HalvesCfg<2, 4>>(a, b, M, R, K, out, true, watch, st, shares);
}

shampoo4_status launch_act8_row_halves(const Act8Operand& a, const Act8Operand& b, int64_t M, int64_t R, int64_t K,
                                       const Act8Out& out, Act8Watch watch, cudaStream_t st) {
  return launch<HalfCfg<false>>(a, b, M, R, K, out, true, watch, st);
}

}  // namespace s4

// The matrix products of the Newton-Schulz iteration on the tensor cores
// (tcgen05.mma, fp16 operands, fp32 accumulators in TMEM).
//
// Three products per iteration, each one kernel with its epilogue fused:
//   A  = f^2 X X^T          symmetric: only tiles that touch the lower triangle
//   P  = a I + b A + c A A  symmetric, the polynomial formed in the epilogue
//   X' = f P X              (X P for a tall matrix), or the parameter update
// X keeps the caller's orientation: both majors of it are read straight from
// the row-major copy, so nothing is ever transposed.
//
// One persistent CTA per SM walks 128 x BN output tiles. Warp 0 streams
// 64-deep operand slices into a ring of 128-byte-swizzled shared tiles (TMA),
// warp 1 issues the MMAs, warps 2..5 turn finished accumulators into output
// while the next tile's MMAs run into the other half of TMEM.
//
// Every wait is bounded by the global timer. A wait that runs out sets
// MUA_STATUS_TIMEOUT, the CTA's roles stop, copies and MMAs in flight are
// awaited (bounded again), TMEM is freed and the kernel returns.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "muon.cuh"

namespace mua {
namespace {

constexpr int kBM = 128, kBK = 64;
constexpr int kThreads = 192;
constexpr int kEpilogueWarps = 4;
constexpr uint64_t kDrainNs = 2000000000ull;  // bound on waits for copies and MMAs in flight

template <int BN>
struct Tile {
  static constexpr int a_bytes = kBM * kBK * 2, b_bytes = BN * kBK * 2;
  static constexpr int stages = BN == 256 ? 4 : 6;
  static constexpr int stage_bytes = a_bytes + b_bytes;
  static constexpr int smem = stages * stage_bytes + 1024;  // + alignment
  static constexpr int tmem_cols = 2 * BN;
};

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  return t;
}
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n"
      " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// False when the wait ran out, or another role of the CTA has given up.
// A limit of 0 gives up as soon as it would wait.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, uint64_t limit,
                                          volatile uint32_t* stop) {
  if (mbar_try(bar, parity)) return true;
  const uint64_t t0 = now_ns();
  while (limit == 0 || !mbar_try(bar, parity)) {
    if (*stop) return false;
    if (limit == 0 || now_ns() - t0 > limit) {
      *stop = 1;
      return false;
    }
  }
  return true;
}
// A wait for work in flight that other roles' giving up does not end.
__device__ __forceinline__ void mbar_drain(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = now_ns();
  while (!mbar_try(bar, parity) && now_ns() - t0 <= kDrainNs) {
  }
}
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x,
                                         int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// Shared-memory operand descriptor, 128-byte swizzle. K-major: 8-row groups
// 1024 bytes apart. M/N-major: 64-element chunks 8192 bytes apart, 8-deep
// groups of the contraction index 1024 bytes apart.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, bool mn) {
  const uint64_t lead = mn ? 8192 >> 4 : 1;
  return (uint64_t)((addr & 0x3FFFF) >> 4) | (lead << 16) | ((uint64_t)(1024 >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}
// fp16 operands, fp32 accumulators, M = 128.
template <int BN>
__device__ __forceinline__ constexpr uint32_t instruction_desc(bool a_mn, bool b_mn) {
  return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(BN / 8) << 17) | ((uint32_t)(kBM / 16) << 24);
}
__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                        bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n"
      " setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
      : "memory");
}
__device__ __forceinline__ void tmem_load32(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// Output tile t of a launch: matrix, row tile, column tile. Symmetric products
// walk the tiles that touch the lower triangle, row by row: with BN = 128 row
// tile i has i + 1 of them, with BN = 256 rows 2p and 2p + 1 have p + 1 each.
// Others walk the row tiles of one column tile first, so concurrent tiles
// share the columns of X they read.
template <int BN, bool SYM>
__device__ __forceinline__ void tile_of(const MuonGemm& g, int64_t t, int& z, int& i, int& j) {
  z = (int)(t / g.tiles);
  int r = (int)(t - (int64_t)z * g.tiles);
  if constexpr (SYM) {
    if constexpr (BN == 128) {
      i = (int)((sqrtf(8.0f * (float)r + 1.0f) - 1.0f) * 0.5f);
      while (i * (i + 1) / 2 > r) --i;
      while ((i + 1) * (i + 2) / 2 <= r) ++i;
      j = r - i * (i + 1) / 2;
    } else {
      int p = (int)((sqrtf(4.0f * (float)r + 1.0f) - 1.0f) * 0.5f);
      while (p * (p + 1) > r) --p;
      while ((p + 1) * (p + 2) <= r) ++p;
      r -= p * (p + 1);
      i = 2 * p + (r > p ? 1 : 0);
      j = r > p ? r - (p + 1) : r;
    }
  } else {
    j = r / g.tiles_m;
    i = r - j * g.tiles_m;
  }
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Columns col .. col+31 of one row of the tile, accumulators v.
template <int EPI>
__device__ __forceinline__ void store_row(const MuonGemm& g, int z, int row, int col,
                                          const uint32_t (&v)[32], float alpha) {
  if constexpr (EPI == kGram || EPI == kPoly) {
    // The lower triangle directly, its mirror image by columns: for a column
    // the warp's lanes are consecutive rows, 64 contiguous bytes.
    __half* D = static_cast<__half*>(g.out) + (int64_t)z * g.batch_stride;
    const __half* A = static_cast<const __half*>(g.addend) + (int64_t)z * g.batch_stride;
    if (row >= g.M || col > row) return;
    const int64_t at = (int64_t)row * g.ldo + col;
    if (col + 31 < row) {  // whole run strictly below the diagonal
      uint32_t w[16];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint4 a = make_uint4(0u, 0u, 0u, 0u);
        if constexpr (EPI == kPoly) a = *reinterpret_cast<const uint4*>(A + at + 8 * q);
        const uint32_t aw[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x0 = __uint_as_float(v[8 * q + 2 * e]) * alpha;
          float x1 = __uint_as_float(v[8 * q + 2 * e + 1]) * alpha;
          if constexpr (EPI == kPoly) {
            const __half2 h = *reinterpret_cast<const __half2*>(&aw[e]);
            x0 = fmaf(__low2float(h), g.mid, x0);
            x1 = fmaf(__high2float(h), g.mid, x1);
          }
          w[4 * q + e] = pack_f16(x0, x1);
        }
        *reinterpret_cast<uint4*>(D + at + 8 * q) =
            make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
      }
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        const uint16_t h = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
        reinterpret_cast<uint16_t*>(D)[(int64_t)(col + e) * g.ldo + row] = h;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        const int c = col + e;
        if (c <= row) {
          float x = __uint_as_float(v[e]) * alpha;
          if constexpr (EPI == kPoly) {
            x = fmaf(__half2float(A[at + e]), g.mid, x);
            if (c == row) x += g.diag;
          }
          const __half h = __float2half_rn(x);
          D[at + e] = h;
          if (c < row) D[(int64_t)c * g.ldo + row] = h;
        }
      }
    }
  } else if constexpr (EPI == kUpdate) {
    if (row >= g.M || col >= g.N) return;
    __half* D = static_cast<__half*>(g.out) + (int64_t)z * g.batch_stride + (int64_t)row * g.ldo;
#pragma unroll
    for (int q = 0; q < 4; ++q) {  // ldo is N rounded up to 8: whole groups fit
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] = pack_f16(__uint_as_float(v[8 * q + 2 * e]) * alpha,
                        __uint_as_float(v[8 * q + 2 * e + 1]) * alpha);
      if (col + 8 * q < g.N)
        *reinterpret_cast<uint4*>(D + col + 8 * q) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  } else if constexpr (EPI == kOut) {
    if (row >= g.M || col >= g.N) return;
    uint16_t* D = static_cast<uint16_t*>(g.out) + (int64_t)z * g.batch_stride +
                  (int64_t)row * g.ldo;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] = pack_bf16(__uint_as_float(v[8 * q + 2 * e]) * alpha,
                         __uint_as_float(v[8 * q + 2 * e + 1]) * alpha);
      if (g.out_vec && col + 8 * q + 8 <= g.N) {
        *reinterpret_cast<uint4*>(D + col + 8 * q) = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (col + 8 * q + e < g.N)
            D[col + 8 * q + e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
      }
    }
  } else {
    // p decay - alpha x, formed in fp32 and rounded once to the storage type.
    if (row >= g.M || col >= g.N) return;
    const int64_t at = (int64_t)z * g.batch_stride + (int64_t)row * g.ldo + col;
    if (g.out_type == kF32) {
      float* P = static_cast<float*>(g.out) + at;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        if (g.out_vec && col + 4 * q + 4 <= g.N) {
          float4 p = *reinterpret_cast<const float4*>(P + 4 * q);
          p.x = fmaf(-alpha, __uint_as_float(v[4 * q]), p.x * g.decay);
          p.y = fmaf(-alpha, __uint_as_float(v[4 * q + 1]), p.y * g.decay);
          p.z = fmaf(-alpha, __uint_as_float(v[4 * q + 2]), p.z * g.decay);
          p.w = fmaf(-alpha, __uint_as_float(v[4 * q + 3]), p.w * g.decay);
          *reinterpret_cast<float4*>(P + 4 * q) = p;
        } else {
#pragma unroll
          for (int e = 4 * q; e < 4 * q + 4; ++e)
            if (col + e < g.N) P[e] = fmaf(-alpha, __uint_as_float(v[e]), P[e] * g.decay);
        }
      }
    } else {
      uint16_t* P = static_cast<uint16_t*>(g.out) + at;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (g.out_vec && col + 8 * q + 8 <= g.N) {
          const uint4 p = *reinterpret_cast<const uint4*>(P + 8 * q);
          uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float lo = __uint_as_float(w[e] << 16), hi = __uint_as_float(w[e] & 0xFFFF0000u);
            w[e] = pack_bf16(fmaf(-alpha, __uint_as_float(v[8 * q + 2 * e]), lo * g.decay),
                             fmaf(-alpha, __uint_as_float(v[8 * q + 2 * e + 1]), hi * g.decay));
          }
          *reinterpret_cast<uint4*>(P + 8 * q) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
          for (int e = 8 * q; e < 8 * q + 8; ++e)
            if (col + e < g.N) {
              const float p = __uint_as_float((uint32_t)P[e] << 16);
              P[e] = __bfloat16_as_ushort(
                  __float2bfloat16_rn(fmaf(-alpha, __uint_as_float(v[e]), p * g.decay)));
            }
        }
      }
    }
  }
}

template <int BN, bool A_MN, bool B_MN, int EPI>
__global__ void __launch_bounds__(kThreads, 1)
gemm_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
            const __grid_constant__ MuonGemm g) {
  using T = Tile<BN>;
  constexpr bool SYM = EPI == kGram || EPI == kPoly;
  constexpr int S = T::stages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[S], empty[S], acc_full[2], acc_empty[2], drained;
  __shared__ uint32_t tmem_base_s;
  __shared__ uint32_t stop;
  const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(smem_u32(&acc_full[a]), 1);
      mbar_init(smem_u32(&acc_empty[a]), kEpilogueWarps);
    }
    mbar_init(smem_u32(&drained), 1);
    stop = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    tma_prefetch_map(&map_a);
    tma_prefetch_map(&map_b);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&tmem_base_s)),
                 "r"(T::tmem_cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = tmem_base_s;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int64_t total = (int64_t)g.tiles * g.batch;
  const int kblocks = (g.K + kBK - 1) / kBK;
  volatile uint32_t* stop_v = &stop;

  if (warp == 0) {
    if (lane == 0) {
      int64_t issued = 0;
      bool ok = true;
      for (int64_t t = blockIdx.x; ok && t < total; t += gridDim.x) {
        int z, i, j;
        tile_of<BN, SYM>(g, t, z, i, j);
        for (int kb = 0; kb < kblocks; ++kb, ++issued) {
          const int s = (int)(issued % S);
          const uint32_t phase = (uint32_t)(issued / S) & 1u;
          if (!mbar_wait(smem_u32(&empty[s]), phase ^ 1u, g.wait_ns, stop_v)) {
            ok = false;
            break;
          }
          const uint32_t bar = smem_u32(&full[s]);
          const uint32_t a = ring + s * T::stage_bytes, b = a + T::a_bytes;
          mbar_expect(bar, T::stage_bytes);
          if constexpr (A_MN) {
#pragma unroll
            for (int q = 0; q < kBM / 64; ++q)
              tma_load(a + q * 8192, &map_a, bar, i * kBM + 64 * q, kb * kBK, z);
          } else {
            tma_load(a, &map_a, bar, kb * kBK, i * kBM, z);
          }
          if constexpr (B_MN) {
#pragma unroll
            for (int q = 0; q < BN / 64; ++q)
              tma_load(b + q * 8192, &map_b, bar, j * BN + 64 * q, kb * kBK, z);
          } else {
#pragma unroll
            for (int q = 0; q < BN / 128; ++q)
              tma_load(b + q * 16384, &map_b, bar, kb * kBK, j * BN + 128 * q, z);
          }
        }
      }
      // The last copy into each stage has landed before the CTA goes.
      for (int64_t c = issued > S ? issued - S : 0; c < issued; ++c)
        mbar_drain(smem_u32(&full[c % S]), (uint32_t)(c / S) & 1u);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = instruction_desc<BN>(A_MN, B_MN);
      int64_t used = 0;
      int n = 0;
      bool ok = true;
      for (int64_t t = blockIdx.x; ok && t < total; t += gridDim.x, ++n) {
        const int acc = n & 1;
        if (!mbar_wait(smem_u32(&acc_empty[acc]), (uint32_t)((n >> 1) & 1) ^ 1u, g.wait_ns, stop_v)) break;
        fence_after();
        const uint32_t d = tmem + acc * BN;
        for (int kb = 0; kb < kblocks; ++kb, ++used) {
          const int s = (int)(used % S);
          if (!mbar_wait(smem_u32(&full[s]), (uint32_t)(used / S) & 1u, g.wait_ns, stop_v)) {
            ok = false;
            break;
          }
          fence_after();
          const uint32_t a = ring + s * T::stage_bytes, b = a + T::a_bytes;
#pragma unroll
          for (int k = 0; k < kBK / 16; ++k)
            mma_f16(d, operand_desc(a + k * (A_MN ? 2048 : 32), A_MN),
                    operand_desc(b + k * (B_MN ? 2048 : 32), B_MN), idesc, (kb | k) != 0);
          mma_commit(smem_u32(&empty[s]));
        }
        if (ok) mma_commit(smem_u32(&acc_full[acc]));
      }
      mma_commit(smem_u32(&drained));
      mbar_drain(smem_u32(&drained), 0);
    }
  } else {
    const int quarter = warp & 3;  // the TMEM lanes this warp may read
    int n = 0;
    for (int64_t t = blockIdx.x; t < total; t += gridDim.x, ++n) {
      int z, i, j;
      tile_of<BN, SYM>(g, t, z, i, j);
      const int acc = n & 1;
      const bool ok = mbar_wait(smem_u32(&acc_full[acc]), (uint32_t)((n >> 1) & 1), g.wait_ns, stop_v);
      if (!__all_sync(0xFFFFFFFFu, ok)) break;
      fence_after();
      float alpha = g.alpha;
      if (g.factor) {
        const float f = g.factor[z];
        alpha = EPI == kGram ? alpha * f * f : alpha * f;
      }
      const int row = i * kBM + quarter * 32 + lane;
      const int limit = min(BN, g.N - j * BN);
#pragma unroll 1
      for (int c = 0; c < limit; c += 32) {
        uint32_t v[32];
        __syncwarp();
        tmem_load32(tmem + ((uint32_t)(quarter * 32) << 16) + acc * BN + c, v);
        store_row<EPI>(g, z, row, j * BN + c, v, alpha);
      }
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&acc_empty[acc]));
    }
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(T::tmem_cols));
  if (threadIdx.x == 0 && stop) atomicOr(g.status, kMuonTimeout);
}

// ---------------------------------------------------------------- host
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

cudaError_t encode_fn(EncodeFn* out) {
  static EncodeFn fn = nullptr;  // a process-wide driver entry point
  if (!fn) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                                           cudaEnableDefault, &found);
    if (e != cudaSuccess) return e;
    if (found != cudaDriverEntryPointSuccess || !p) return cudaErrorNotSupported;
    fn = reinterpret_cast<EncodeFn>(p);
  }
  *out = fn;
  return cudaSuccess;
}

// Copies of 64 contiguous elements x `box_rows` rows of a batch of row-major
// matrices; what lies outside a matrix reads as 0.
cudaError_t make_map(const MuonOperand& o, int batch, int box_rows, CUtensorMap* map) {
  EncodeFn encode;
  const cudaError_t e = encode_fn(&encode);
  if (e != cudaSuccess) return e;
  const cuuint64_t dims[3] = {(cuuint64_t)o.cols, (cuuint64_t)o.rows, (cuuint64_t)batch};
  const cuuint64_t strides[2] = {(cuuint64_t)o.ld * 2, (cuuint64_t)o.ld * 2 * o.rows};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1}, step[3] = {1, 1, 1};
  const CUresult r =
      encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, o.p, dims, strides, box, step,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int BN, bool A_MN, bool B_MN, int EPI>
cudaError_t run(const CUtensorMap& ma, const CUtensorMap& mb, const MuonGemm& g, int sms,
                cudaStream_t st) {
  using T = Tile<BN>;
  auto kernel = gemm_kernel<BN, A_MN, B_MN, EPI>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, T::smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min<int64_t>(sms, (int64_t)g.tiles * g.batch));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = T::smem;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, ma, mb, g);
}

template <int BN>
cudaError_t dispatch(const CUtensorMap& ma, bool a_mn, const CUtensorMap& mb, bool b_mn,
                     int epilogue, const MuonGemm& g, int sms, cudaStream_t st) {
  switch (epilogue) {
    case kGram:
      return a_mn ? run<BN, true, true, kGram>(ma, mb, g, sms, st)
                  : run<BN, false, false, kGram>(ma, mb, g, sms, st);
    case kPoly: return run<BN, false, false, kPoly>(ma, mb, g, sms, st);
    case kUpdate:
      return b_mn ? run<BN, false, true, kUpdate>(ma, mb, g, sms, st)
                  : run<BN, false, false, kUpdate>(ma, mb, g, sms, st);
    case kOut:
      return b_mn ? run<BN, false, true, kOut>(ma, mb, g, sms, st)
                  : run<BN, false, false, kOut>(ma, mb, g, sms, st);
    default:
      return b_mn ? run<BN, false, true, kParams>(ma, mb, g, sms, st)
                  : run<BN, false, false, kParams>(ma, mb, g, sms, st);
  }
}

int64_t tile_count(bool sym, int bn, int M, int N) {
  const int64_t tm = (M + kBM - 1) / kBM, tn = (N + bn - 1) / bn;
  if (!sym) return tm * tn;
  if (bn == 128) return tm * (tm + 1) / 2;
  const int64_t pairs = tm / 2;  // rows 2p, 2p + 1 have p + 1 tiles each
  return pairs * (pairs + 1) + (tm & 1 ? pairs + 1 : 0);
}

}  // namespace

int muon_sm_count(cudaError_t* e) {
  int dev = 0, sms = 0;
  *e = cudaGetDevice(&dev);
  if (*e == cudaSuccess) *e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

cudaError_t muon_launch_gemm(const MuonOperand& a, bool a_mn, const MuonOperand& b, bool b_mn,
                             int epilogue, MuonGemm g, cudaStream_t st) {
  cudaError_t e;
  const int sms = muon_sm_count(&e);
  if (e != cudaSuccess) return e;
  const bool sym = epilogue == kGram || epilogue == kPoly;
  // Wide tiles read less per MMA; narrow ones fill the SMs when there are few.
  const bool wide = tile_count(sym, 256, g.M, g.N) * g.batch >= sms;
  const int bn = wide ? 256 : 128;
  g.tiles_m = (g.M + kBM - 1) / kBM;
  g.tiles_n = (g.N + bn - 1) / bn;
  g.tiles = (int32_t)tile_count(sym, bn, g.M, g.N);
  CUtensorMap ma, mb;
  e = make_map(a, g.batch, a_mn ? kBK : kBM, &ma);
  if (e == cudaSuccess) e = make_map(b, g.batch, b_mn ? kBK : 128, &mb);
  if (e != cudaSuccess) return e;
  return wide ? dispatch<256>(ma, a_mn, mb, b_mn, epilogue, g, sms, st)
              : dispatch<128>(ma, a_mn, mb, b_mn, epilogue, g, sms, st);
}

}  // namespace mua

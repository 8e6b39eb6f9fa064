// The Newton-Schulz iteration of a stack of matrices in one launch, on the
// tensor cores (tcgen05.mma, fp16 operands, fp32 accumulators in TMEM).
//
// Three products per step, each with its epilogue fused, every matrix of the
// stack at its own pace (a product starts when the one before it is complete):
//   A  = f^2 X X^T          symmetric: lower block triangle only
//   P  = a I + b A + c A A  likewise, the polynomial formed in the epilogue
//   X' = f P X              (X P for a tall matrix); the last one writes the
//                           result or updates the parameters instead
// X keeps the caller's orientation: an operand is read with its contraction
// index contiguous ("K-major") or with its M / N index contiguous, whichever
// the row-major copy has, so nothing is transposed. A and P hold only the
// blocks on and below the diagonal; a block above it is read as its mirror
// block with the other major, so no product writes a mirror image.
//
// A tile is 256 x 256 on a pair of CTAs (cta_group::2: each SM holds half of
// both operands, 8 KB of shared memory read per 16-deep MMA and SM instead of
// 12) or 128 x 128 on one CTA when the 256-wide tiles would be too few for the
// SMs. Per CTA: warp 0 streams 64-deep operand slices into a ring of 128-byte
// swizzled shared tiles (TMA), warp 1 issues the MMAs, warps 2..9 turn
// finished accumulators into output while the next tile's MMAs run into the
// other half of TMEM.
//
// Every wait is bounded by the global timer. A wait that runs out sets
// MUA_STATUS_TIMEOUT, the CTA's roles stop, copies and MMAs in flight are
// awaited (bounded again), TMEM is freed and the kernel returns.
#include <algorithm>

#include "muon_tc.cuh"

namespace mua {
namespace {

constexpr int kEpilogueWarps = 8;            // two for each quarter of the TMEM lanes
constexpr int kThreads = 64 + 32 * kEpilogueWarps;
constexpr int kStageBytes = 32768;           // 128 rows of A and of B, 64 deep
constexpr int kChunkBytes = 4096;            // 32 rows x 64 fp16 columns of output
template <int BN>
struct Ring {
  static constexpr int chunks = BN / 128;    // an epilogue warp's share of a tile
  static constexpr int stages = BN == 256 ? 5 : 6;
  static constexpr int smem =
      stages * kStageBytes + kEpilogueWarps * chunks * kChunkBytes + 1024;  // + alignment
};
struct Maps {
  CUtensorMap load_x[2], load_a, load_p;     // boxes of 64 x 64
  CUtensorMap store_x[2], store_a, store_p;  // 64 x 32
};

enum Product : int { kGram = 0, kPoly = 1, kUpdate = 2 };

// Tiles of one matrix in a symmetric product (the lower block triangle) and in
// an update.
struct Tiles {
  int sm, um, un;      // blocks of the short side; row and column tiles of X
  int gram, update;    // k-slices of the products (gram: along the long side)
  int sym, upd;        // tiles
};
template <int BN>
__device__ __forceinline__ Tiles tiles_of(const MuonNs& g) {
  const int s = min(g.rows, g.cols), l = max(g.rows, g.cols);
  Tiles t;
  t.sm = (s + BN - 1) / BN;
  t.um = (g.rows + BN - 1) / BN;
  t.un = (g.cols + BN - 1) / BN;
  t.gram = (l + 63) / 64;
  t.update = (s + 63) / 64;
  t.sym = t.sm * (t.sm + 1) / 2;
  t.upd = t.um * t.un;
  return t;
}

// Work item w of the launch, in the order (step, product, matrix, tile): tile
// (i, j) of a product of matrix z, which needs `before` finished tiles of z.
// The triangle is walked row by row; the update walks the short side's tiles
// first, so that tiles in flight share their slice of X.
struct Item {
  int step, kind, z, i, j, kblocks;
  uint32_t before;
  bool last;
};
__device__ __forceinline__ int64_t item_count(const MuonNs& g, const Tiles& T) {
  return (int64_t)(2 * T.sym + T.upd) * g.batch * g.steps;
}
__device__ __forceinline__ Item item_of(const MuonNs& g, const Tiles& T, int64_t w) {
  Item it;
  const int64_t sym = (int64_t)T.sym * g.batch, per = 2 * sym + (int64_t)T.upd * g.batch;
  it.step = (int)(w / per);
  int64_t r = w - it.step * per;
  it.kind = r < sym ? kGram : (r < 2 * sym ? kPoly : kUpdate);
  r -= it.kind * sym;
  const int tiles = it.kind == kUpdate ? T.upd : T.sym;
  it.z = (int)(r / tiles);
  const int t = (int)(r - (int64_t)it.z * tiles);
  it.before = (uint32_t)(it.step * (2 * T.sym + T.upd) + it.kind * T.sym);
  it.kblocks = it.kind == kGram ? T.gram : T.update;
  it.last = it.kind == kUpdate && it.step == g.steps - 1;
  if (it.kind == kUpdate) {
    if (g.rows <= g.cols) {
      it.j = t / T.um;
      it.i = t - it.j * T.um;
    } else {
      it.i = t / T.un;
      it.j = t - it.i * T.un;
    }
  } else {
    it.i = (int)((sqrtf(8.0f * (float)t + 1.0f) - 1.0f) * 0.5f);
    while (it.i * (it.i + 1) / 2 > t) --it.i;
    while ((it.i + 1) * (it.i + 2) / 2 <= t) ++it.i;
    it.j = t - it.i * (it.i + 1) / 2;
  }
  return it;
}
// Whether slice kb of the operand with M / N block `block` is read with its
// M / N index contiguous. X has one major per product; A and P (symmetric)
// are read from below the diagonal.
template <int BN>
__device__ __forceinline__ bool reads_mn(const MuonNs& g, int kind, bool a, int block, int kb) {
  const bool tall = g.rows > g.cols;
  if (kind == kGram) return tall;
  const bool symmetric = kind == kPoly || a != tall;
  if (symmetric) return kb * 64 / BN > block;
  return !tall;  // X: the B operand of a wide update
}

// Waits until matrix z has `tiles` finished tiles (every epilogue warp of a
// tile counts one). Items are taken in order by CTAs that are all resident, and
// need earlier items only, so the wait ends.
__device__ __forceinline__ bool matrix_wait(const MuonNs& g, int z, uint32_t want,
                                            volatile uint32_t* stop) {
  const uint32_t* p = g.counters + z;
  uint64_t t0 = 0;
  for (uint32_t n = 1;; ++n) {
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    if (v >= want) return true;
    if (g.wait_ns != 0 && (n & 63u) != 0) continue;
    if (*stop) return false;
    const uint64_t t = now_ns();
    if (t0 == 0) t0 = t;
    if (g.wait_ns == 0 || t - t0 > g.wait_ns) {
      *stop = 1;
      return false;
    }
  }
}

template <int CG, int BN>
__global__ void __launch_bounds__(kThreads, 1)
ns_kernel(const __grid_constant__ Maps maps, const __grid_constant__ MuonNs g) {
  constexpr int S = Ring<BN>::stages;
  constexpr int kChunks = Ring<BN>::chunks;
  constexpr uint32_t kTmemCols = 2 * BN;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[S], empty[S], acc_full[2], acc_empty[2], drained;
  __shared__ __align__(8) uint64_t addend_full[kEpilogueWarps][kChunks];
  __shared__ uint32_t tmem_base_s, stop, issued_s, peer_issued_s;
  const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? (blockIdx.x & 1u) : 0u;
  const int64_t first = blockIdx.x / CG, stride = gridDim.x / CG;
  const Tiles tiles = tiles_of<BN>(g);
  const int64_t items = item_count(g, tiles);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&full[s]), CG);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(smem_u32(&acc_full[a]), 1);
      mbar_init(smem_u32(&acc_empty[a]), kEpilogueWarps * CG);
    }
    for (int w = 0; w < kEpilogueWarps; ++w)
      for (int c = 0; c < kChunks; ++c) mbar_init(smem_u32(&addend_full[w][c]), 1);
    mbar_init(smem_u32(&drained), 1);
    stop = 0;
    issued_s = peer_issued_s = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    if constexpr (CG == 2) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       smem_u32(&tmem_base_s)),
                   "r"(kTmemCols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       smem_u32(&tmem_base_s)),
                   "r"(kTmemCols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
  }
  fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();
  fence_after();
  const uint32_t tmem = tmem_base_s;
  volatile uint32_t* stop_v = &stop;

  // Warps 0 and 1 run their loops converged; an elected lane issues.
  if (warp == 0) {
    uint32_t issued = 0, s = 0, turn = 1;
    bool ok = true;
    int ready_z = -1;
    uint32_t ready = 0;
    for (int64_t w = first; ok && w < items; w += stride) {
      const Item it = item_of(g, tiles, w);
      if (it.z != ready_z || it.before != ready) {
        ok = matrix_wait(g, it.z, it.before * (CG * kEpilogueWarps), stop_v);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        fence_async_global();
        ready_z = it.z;
        ready = it.before;
      }
      const bool tall = g.rows > g.cols;
      const CUtensorMap* x = &maps.load_x[it.step & 1];
      const CUtensorMap* ma = it.kind == kGram ? x : (it.kind == kPoly ? &maps.load_a
                                                                       : (tall ? x : &maps.load_p));
      const CUtensorMap* mb = it.kind == kGram ? x : (it.kind == kPoly ? &maps.load_a
                                                                       : (tall ? &maps.load_p : x));
      const int a0 = it.i * BN + (int)rank * 128;         // this CTA's rows of A
      const int b0 = it.j * BN + (int)rank * (BN / CG);   // and of B
      for (int kb = 0; kb < it.kblocks; ++kb) {
        ok = mbar_wait(smem_u32(&empty[s]), turn, g.wait_ns, stop_v);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        const uint32_t a = ring + s * kStageBytes, b = a + 16384;
        const bool a_mn = reads_mn<BN>(g, it.kind, true, it.i, kb);
        const bool b_mn = reads_mn<BN>(g, it.kind, false, it.j, kb);
        if (elect_one()) {
          uint32_t bar = smem_u32(&full[s]);
          if (CG == 2 && rank != 0) {
            bar = peer_address(bar, 0);
            mbar_expect_cluster(bar, kStageBytes);
          } else {
            mbar_expect(bar, kStageBytes);
          }
#pragma unroll
          for (int q = 0; q < 2; ++q)
            tma_load<CG>(a + q * 8192, ma, bar, a_mn ? a0 + 64 * q : kb * 64,
                         a_mn ? kb * 64 : a0 + 64 * q, it.z);
#pragma unroll
          for (int q = 0; q < 2; ++q)
            tma_load<CG>(b + q * 8192, mb, bar, b_mn ? b0 + 64 * q : kb * 64,
                         b_mn ? kb * 64 : b0 + 64 * q, it.z);
        }
        __syncwarp();
        ++issued;
        if (++s == S) {
          s = 0;
          turn ^= 1u;
        }
      }
    }
    if (elect_one()) {
      issued_s = issued;
      if (CG == 2 && rank != 0)
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(
                         peer_address(smem_u32(&peer_issued_s), 0)),
                     "r"(issued)
                     : "memory");
    }
  } else if (warp == 1) {
    if (rank == 0) {
      uint32_t n = 0, s = 0, turn = 0;
      bool ok = true;
      for (int64_t w = first; ok && w < items; w += stride, ++n) {
        const Item it = item_of(g, tiles, w);
        const uint32_t acc = n & 1u;
        ok = mbar_wait(smem_u32(&acc_empty[acc]), ((n >> 1) & 1u) ^ 1u, g.wait_ns, stop_v);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        fence_after();
        const uint32_t d = tmem + acc * BN;
        for (int kb = 0; kb < it.kblocks; ++kb) {
          ok = mbar_wait(smem_u32(&full[s]), turn, g.wait_ns, stop_v);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
          fence_after();
          const uint32_t a = ring + s * kStageBytes, b = a + 16384;
          const bool a_mn = reads_mn<BN>(g, it.kind, true, it.i, kb);
          const bool b_mn = reads_mn<BN>(g, it.kind, false, it.j, kb);
          const uint32_t idesc = instruction_desc<CG>(BN, a_mn, b_mn);
          const uint64_t da = operand_desc(a, 8192), db = operand_desc(b, 8192);
          const uint64_t sa = a_mn ? 2048 >> 4 : 32 >> 4, sb = b_mn ? 2048 >> 4 : 32 >> 4;
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_f16<CG>(d, da + k * sa, db + k * sb, idesc, (kb | k) != 0);
            mma_commit<CG>(smem_u32(&empty[s]));
          }
          __syncwarp();
          if (++s == S) {
            s = 0;
            turn ^= 1u;
          }
        }
        if (ok && elect_one()) mma_commit<CG>(smem_u32(&acc_full[acc]));
        __syncwarp();
      }
      // The MMAs in flight end before TMEM and the operands go.
      if (elect_one()) {
        if constexpr (CG == 2)
          asm volatile(
              "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                  smem_u32(&drained))
              : "memory");
        else
          mma_commit<1>(smem_u32(&drained));
        mbar_drain(smem_u32(&drained), 0);
      }
    }
  } else {
    const int quarter = warp & 3;     // the TMEM lanes this warp may read
    const int side = (warp - 2) >> 2;  // its half of the tile's columns
    const uint32_t stage = ring + S * kStageBytes + (warp - 2) * kChunks * kChunkBytes;
    uint32_t n = 0;
    uint32_t asked = 0, parity = 0;  // per chunk: an addend copy in flight, its barrier's phase
    int ready_z = -1;
    uint32_t ready = 0;
    bool ok = true;
    for (int64_t w = first; ok && w < items; w += stride, ++n) {
      const Item it = item_of(g, tiles, w);
      const int M = it.kind == kUpdate ? g.rows : min(g.rows, g.cols);
      const int N = it.kind == kUpdate ? g.cols : M;
      const int row0 = it.i * BN + (int)rank * 128 + quarter * 32;
      const int col0 = it.j * BN + side * (BN / 2);
      const int chunks = row0 < M ? max(0, min(kChunks, (N - col0 + 63) / 64)) : 0;
      const uint32_t acc = n & 1u;
      if (it.kind == kPoly && chunks > 0) {
        // The addend on its way while the MMAs run.
        if (it.z != ready_z || it.before != ready) {
          ok = matrix_wait(g, it.z, it.before * (CG * kEpilogueWarps), stop_v);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
          fence_async_global();
          ready_z = it.z;
          ready = it.before;
        }
        if (lane == 0) {
          for (int c = 0; c < chunks; ++c) {
            const uint32_t bar = smem_u32(&addend_full[warp - 2][c]);
            mbar_expect(bar, kChunkBytes);
            tma_load<1>(stage + c * kChunkBytes, &maps.store_a, bar, col0 + 64 * c, row0, it.z);
          }
        }
        asked = (1u << chunks) - 1u;
      }
      ok = mbar_wait(smem_u32(&acc_full[acc]), (n >> 1) & 1u, g.wait_ns, stop_v);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) break;
      fence_after();
      const uint32_t lanes =
          tmem + ((uint32_t)(quarter * 32) << 16) + acc * BN + side * (BN / 2);
      float f = it.step == 0 && it.kind != kPoly ? g.factor[it.z] : 1.0f;
      if (it.kind == kGram) f *= f;
      const float alpha = f * (it.kind == kGram ? g.gram_alpha[it.step]
                                                : (it.kind == kPoly ? g.poly_alpha[it.step]
                                                                    : g.update_alpha[it.step]));
      if (!it.last) {
        const float mid = g.poly_mid[it.step], diag = g.poly_diag[it.step];
        const CUtensorMap* out = it.kind == kGram
                                     ? &maps.store_a
                                     : (it.kind == kPoly ? &maps.store_p
                                                         : &maps.store_x[(it.step & 1) ^ 1]);
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
          const uint32_t tile = stage + c * kChunkBytes;
          uint32_t v[2][32];
          tmem_load32(lanes + 64 * c, v[0]);
          tmem_load32(lanes + 64 * c + 32, v[1]);
          if (it.kind == kPoly) {
            mbar_drain(smem_u32(&addend_full[warp - 2][c]), (parity >> c) & 1u);
            asked &= ~(1u << c);
            parity ^= 1u << c;
          }
          tmem_load_wait();
          const int diagonal = row0 + lane - (col0 + 64 * c);  // column of the diagonal
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const uint32_t at = chunk_address(tile, lane, q);
            uint32_t h[4];
            if (it.kind == kPoly) {
              const uint4 a = ld_shared(at);
              const uint32_t aw[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&aw[e]));
                float x0 = __uint_as_float(v[q >> 2][(8 * q + 2 * e) & 31]) * alpha;
                float x1 = __uint_as_float(v[q >> 2][(8 * q + 2 * e + 1) & 31]) * alpha;
                x0 = fmaf(y.x, mid, x0);
                x1 = fmaf(y.y, mid, x1);
                if (8 * q + 2 * e == diagonal) x0 += diag;
                if (8 * q + 2 * e + 1 == diagonal) x1 += diag;
                h[e] = pack_f16(x0, x1);
              }
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                h[e] = pack_f16(__uint_as_float(v[q >> 2][(8 * q + 2 * e) & 31]) * alpha,
                                __uint_as_float(v[q >> 2][(8 * q + 2 * e + 1) & 31]) * alpha);
            }
            st_shared(at, h[0], h[1], h[2], h[3]);
          }
          fence_async_shared();
          __syncwarp();
          if (lane == 0) tma_store(out, tile, col0 + 64 * c, row0, it.z);
        }
      } else {
        // 32 x 32 fp32 through shared memory: a lane then holds four columns,
        // eight lanes a row's 128 (64) contiguous bytes.
#pragma unroll 1
        for (int c = 0; c < 2 * chunks; ++c) {
          const int col = col0 + 32 * c + 4 * (lane & 7);
          const int64_t at0 = (int64_t)it.z * g.batch_stride +
                              (int64_t)(row0 + (lane >> 3)) * g.ldo + col;
          float4 old[8];  // all loads before the first store
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            old[q] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (row0 + 4 * q + (lane >> 3) < M && col < N)
              old[q] = read_four(g, at0 + 4 * q * g.ldo, N - col);
          }
          uint32_t v[32];
          tmem_load32(lanes + 32 * c, v);
          tmem_load_wait();
#pragma unroll
          for (int q = 0; q < 8; ++q)
            st_shared(chunk_address(stage, lane, q), v[4 * q], v[4 * q + 1], v[4 * q + 2],
                      v[4 * q + 3]);
          __syncwarp();
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const int r = 4 * q + (lane >> 3);
            const uint4 u = ld_shared(chunk_address(stage, r, lane & 7));
            const uint32_t x[4] = {u.x, u.y, u.z, u.w};
            if (row0 + r < M && col < N)
              write_four(g, at0 + 4 * q * g.ldo, N - col, old[q], x, alpha);
          }
          __syncwarp();
        }
      }
      fence_before();
      __syncwarp();
      if (lane == 0) {
        if (CG == 2 && rank != 0)
          mbar_arrive_cluster(peer_address(smem_u32(&acc_empty[acc]), 0));
        else
          mbar_arrive(smem_u32(&acc_empty[acc]));
        if (!it.last) {
          // This warp's part of the tile is in memory: count it.
          tma_store_wait_all();
          asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(g.counters + it.z)
                       : "memory");
        }
      }
      __syncwarp();
    }
    for (int c = 0; c < kChunks; ++c)
      if (asked >> c & 1u)
        mbar_drain(smem_u32(&addend_full[warp - 2][c]), (parity >> c) & 1u);
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();
  // Operand copies land before their shared memory goes. A pair's copies count
  // on the first CTA's barriers, one arrival from each CTA: where the two gave
  // up at different slices the missing arrivals are made here.
  if (threadIdx.x == 0 && rank == 0) {
    const uint32_t mine = issued_s, other = CG == 2 ? peer_issued_s : mine;
    const uint32_t most = max(mine, other);
    for (uint32_t c = min(mine, other); c < most; ++c) mbar_arrive(smem_u32(&full[c % S]));
    for (uint32_t c = most > S ? most - S : 0; c < most; ++c)
      mbar_drain(smem_u32(&full[c % S]), (c / S) & 1u);
  }
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();
  fence_after();
  if (warp == 1) {
    if constexpr (CG == 2)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                   "r"(kTmemCols));
    else
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                   "r"(kTmemCols));
  }
  if constexpr (CG == 2) cluster_sync();
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

struct Operand {
  void* p;  // fp16 [batch][rows][ld]
  int32_t rows, cols, ld;
};

// Copies of 64 contiguous elements x `box_rows` rows of a batch of row-major
// matrices; what lies outside a matrix reads as 0 and is not written.
cudaError_t make_map(const Operand& o, int batch, int box_rows, CUtensorMap* map) {
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


constexpr int kMaxDevices = 64;

// CTAs of a cooperative launch that the current device holds at once.
template <int CG, int BN>
cudaError_t resident_ctas(int* out) {
  static int known[kMaxDevices];  // 0: not asked yet
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < kMaxDevices && known[dev] > 0) {
    *out = known[dev];
    return cudaSuccess;
  }
  auto kernel = ns_kernel<CG, BN>;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Ring<BN>::smem);
  if (e != cudaSuccess) return e;
  int n = 0;
  if (CG == 2) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Ring<BN>::smem;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
    n *= 2;
  } else {
    int sms = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, kThreads, Ring<BN>::smem);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    n *= sms;
  }
  if (e != cudaSuccess) return e;
  if (n < CG) return cudaErrorLaunchOutOfResources;
  if (dev < kMaxDevices) known[dev] = n;
  *out = n;
  return cudaSuccess;
}

template <int CG, int BN>
cudaError_t run(const Maps& maps, const MuonNs& g, int64_t tiles, cudaStream_t st) {
  int most = 0;
  const cudaError_t e = resident_ctas<CG, BN>(&most);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min<int64_t>(most, tiles * CG));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Ring<BN>::smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CG;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CG == 2 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, ns_kernel<CG, BN>, maps, g);
}

int64_t most_tiles(const MuonNs& g, int side) {
  const int64_t tm = (g.rows + side - 1) / side, tn = (g.cols + side - 1) / side;
  return tm * tn * g.batch;
}

}  // namespace

cudaError_t muon_launch_ns(const MuonStack& m, const MuonNs& g, cudaStream_t st) {
  Maps maps;
  const int s = std::min(g.rows, g.cols);
  for (int store = 0; store < 2; ++store) {
    const int rows = store ? 32 : 64;
    CUtensorMap* x = store ? maps.store_x : maps.load_x;
    for (int k = 0; k < 2; ++k) {
      const cudaError_t e = make_map({m.x[k], g.rows, g.cols, m.ld}, g.batch, rows, &x[k]);
      if (e != cudaSuccess) return e;
    }
    cudaError_t e = make_map({m.a, s, s, m.lds}, g.batch, rows, store ? &maps.store_a : &maps.load_a);
    if (e == cudaSuccess)
      e = make_map({m.p, s, s, m.lds}, g.batch, rows, store ? &maps.store_p : &maps.load_p);
    if (e != cudaSuccess) return e;
  }
  // 256-wide tiles on CTA pairs halve the operand traffic; below one tile per
  // pair the 128-wide ones keep more SMs busy.
  const int64_t wide = most_tiles(g, 256);
  if (wide >= 74) return run<2, 256>(maps, g, wide, st);
  return run<1, 128>(maps, g, most_tiles(g, 128), st);
}

}  // namespace mua

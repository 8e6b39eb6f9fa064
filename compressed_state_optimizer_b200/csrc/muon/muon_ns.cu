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
// SMs. Per CTA: warps 0 and 10 stream 64-deep slices of the operands A and B
// into a ring of 128-byte swizzled shared tiles (TMA), warp 1 issues the MMAs,
// warps 2..9 write finished accumulators out, through shared memory into whole
// lines, while the next tile's MMAs run into the other half of TMEM, and warp 11
// brings the addend of P in and counts finished tiles, so that nothing else
// stands still for those.
//
// A slice takes 512 cycles of MMA on 256 x 256 and 256 on 128 x 128, and in both
// cases 32 KB a SM, 512 cycles at the 64 bytes a cycle that L2 delivers: the
// large tile is bound by both at once, the small one by the copies. The way
// through one slice's instructions (about 400 cycles in a producer, 430 in the
// issuing warp) comes close: hence a warp for each operand, one copy for an
// operand whose rows are contiguous in depth, and majors fixed per item.
// Between two products of one matrix lie some 8000 cycles: a finished tile's
// way to memory, its count and the next one's first copy.
// Measured: 4096 x 4096, five steps, 1.0 ms on the device (1.36e12 operations of
// the halved symmetric products and the updates; at the chip's power limit,
// where cuBLAS keeps 1.39e15 a second); 768 x 768 0.10 ms, 48 of them 0.5 ms.
//
// Every wait is bounded by the global timer. A wait that runs out sets
// MUA_STATUS_TIMEOUT, the CTA's roles stop, copies and MMAs in flight are
// awaited (bounded again), TMEM is freed and the kernel returns.
#include <algorithm>
#include <atomic>

#include "muon_tc.cuh"

namespace mua {
namespace {

constexpr int kEpilogueWarps = 8;            // two for each quarter of the TMEM lanes
constexpr int kThreads = 32 * (4 + kEpilogueWarps);
constexpr int kProducerB = 2 + kEpilogueWarps, kPorter = kProducerB + 1;  // warps
constexpr int kOperandBytes = 16384;         // 128 rows of an operand, 64 deep
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kChunkBytes = 16384;           // 128 rows x 64 fp16 columns of output
template <int BN>
struct Ring {
  static constexpr int chunks = BN / 128;    // of each half of a tile's columns
  static constexpr int stages = BN == 256 ? 5 : 6;
  static constexpr int smem =
      stages * kStageBytes + 2 * chunks * kChunkBytes + 1024;  // + alignment
};
struct Maps {
  // X of even and odd steps, A, P: boxes of 64 columns by 128 rows (an operand's
  // rows) and by 64 rows (an operand's columns).
  CUtensorMap rows[4], cols[4];
};

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

// Work items of the launch, in the order (step, product, matrix, tile): tile
// (i, j) of a product of matrix z over k-slices kb0 .. kb1 - 1, which needs
// `before` finished items of z. The triangle is walked row by row; the update
// walks the short side's tiles first, so that tiles in flight share their slice
// of X. Where A's tiles are too few for the SMs, `split` items share one's
// contraction and leave fp32 partial sums, and `reduce` items add them up, in
// a fixed order, a share of the tile's rows each.
enum Product : int { kGram = 0, kReduce = 1, kPoly = 2, kUpdate = 3 };
struct Item {
  int step, kind, z, tile, share, i, j, kb0, kb1;
  uint32_t before;
  bool last;
};
// n / d by the reciprocal ceil(2^32 / d): at most one too large for n < 2^31.
struct Divisor {
  uint32_t d, r;
  __device__ __forceinline__ explicit Divisor(uint32_t x)
      : d(x), r(x > 1 ? 0xFFFFFFFFu / x + 1u : 0u) {}
  __device__ __forceinline__ uint32_t divide(uint32_t n) const {
    if (d <= 1) return n;
    const uint32_t q = __umulhi(n, r);
    return q * d > n ? q - 1 : q;
  }
};
// This CTA's (or pair's) items, one after another.
template <int BN>
struct Walk {
  const MuonNs& g;
  Tiles T;
  uint32_t per[4], all[4], stride, left;  // items of a matrix, of a product; place in it
  Divisor by_sym, by_upd, by_gram, by_reduce, by_split, by_share, by_short;
  int kind = 0, step = 0;
  __device__ __forceinline__ Walk(const MuonNs& g_, uint32_t first, uint32_t stride_)
      : g(g_), T(tiles_of<BN>(g_)), stride(stride_), left(first), by_sym((uint32_t)T.sym),
        by_upd((uint32_t)T.upd), by_gram((uint32_t)(T.sym * g_.split)),
        by_reduce((uint32_t)(T.sym * g_.reduce)), by_split((uint32_t)g_.split),
        by_share((uint32_t)g_.reduce),
        by_short((uint32_t)(g_.rows <= g_.cols ? T.um : T.un)) {
    per[kGram] = (uint32_t)(T.sym * g.split);
    per[kReduce] = g.split > 1 ? (uint32_t)(T.sym * g.reduce) : 0u;
    per[kPoly] = (uint32_t)T.sym;
    per[kUpdate] = (uint32_t)T.upd;
#pragma unroll
    for (int k = 0; k < 4; ++k) all[k] = per[k] * (uint32_t)g.batch;
    settle();
  }
  __device__ __forceinline__ void settle() {
    while (step < g.steps) {
      const uint32_t n = kind == kGram ? all[0] : (kind == kReduce ? all[1]
                                                                   : (kind == kPoly ? all[2] : all[3]));
      if (left < n) break;
      left -= n;
      if (++kind == 4) {
        kind = 0;
        ++step;
      }
    }
  }
  __device__ __forceinline__ bool more() const { return step < g.steps; }
  __device__ __forceinline__ void advance() {
    left += stride;
    settle();
  }
  __device__ __forceinline__ Item item() const {
    Item it;
    it.step = step;
    it.kind = kind;
    it.before = (uint32_t)step * (per[0] + per[1] + per[2] + per[3]);
    it.share = 0;
    it.kb0 = 0;
    it.kb1 = T.update;
    it.last = false;
    uint32_t z, t;
    if (kind == kUpdate) {
      it.before += per[0] + per[1] + per[2];
      it.last = step == g.steps - 1;
      z = by_upd.divide(left);
      t = left - z * per[3];
      const uint32_t q = by_short.divide(t), r = t - q * by_short.d;
      it.i = (int)(g.rows <= g.cols ? r : q);
      it.j = (int)(g.rows <= g.cols ? q : r);
    } else {
      if (kind == kPoly) {
        it.before += per[0] + per[1];
        z = by_sym.divide(left);
        t = left - z * per[2];
      } else if (kind == kReduce) {
        it.before += per[0];
        z = by_reduce.divide(left);
        t = left - z * per[1];
        const uint32_t q = by_share.divide(t);
        it.share = (int)(t - q * by_share.d);
        t = q;
      } else {
        z = by_gram.divide(left);
        t = left - z * per[0];
        const uint32_t q = by_split.divide(t);
        it.share = (int)(t - q * by_split.d);
        t = q;
        it.kb0 = g.split > 1 ? it.share * T.gram / g.split : 0;
        it.kb1 = g.split > 1 ? (it.share + 1) * T.gram / g.split : T.gram;
      }
      it.i = (int)((sqrtf(8.0f * (float)t + 1.0f) - 1.0f) * 0.5f);
      while (it.i * (it.i + 1) / 2 > (int)t) --it.i;
      while ((it.i + 1) * (it.i + 2) / 2 <= (int)t) ++it.i;
      it.j = (int)t - it.i * (it.i + 1) / 2;
    }
    it.z = (int)z;
    it.tile = (int)t;
    return it;
  }
};
// First k-slice of an item whose operand (A or B) is read with its M / N index
// contiguous. X has one major per product; A and P (symmetric) are read from
// below the diagonal, as rows up to the diagonal block and columns behind it.
template <int BN>
__device__ __forceinline__ int first_mn(const MuonNs& g, const Item& it, bool a) {
  constexpr int never = 1 << 30;
  const bool tall = g.rows > g.cols;
  if (it.kind == kGram) return tall ? 0 : never;
  if (it.kind == kPoly || a != tall) return ((a ? it.i : it.j) + 1) * (BN / 64);
  return tall ? never : 0;
}

__device__ __forceinline__ bool matrix_ready(const MuonNs& g, int z, uint32_t want) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(g.counters + z) : "memory");
  return v >= want;
}
// Waits until matrix z has `want` finished items (every CTA of an item counts
// one). Items are taken in order by CTAs that are all resident, and
// need earlier items only, so the wait ends.
__device__ __forceinline__ bool matrix_wait(const MuonNs& g, int z, uint32_t want,
                                            volatile uint32_t* stop) {
  uint64_t t0 = 0;
  for (uint32_t n = 1; !matrix_ready(g, z, want); ++n) {
    if (g.wait_ns != 0 && (n & 63u) != 0) continue;
    if (*stop) return false;
    const uint64_t t = now_ns();
    if (t0 == 0) t0 = t;
    if (g.wait_ns == 0 || t - t0 > g.wait_ns) {
      *stop = 1;
      return false;
    }
  }
  return true;
}

// This CTA's part of an item is in memory: count it.
__device__ __forceinline__ void count_item(const MuonNs& g, int z) {
  asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(g.counters + z) : "memory");
}

// This warp's rows of a share of a split tile of A: the partial sums in the
// order of the splits, scaled and rounded to fp16. A lane takes 8 columns.
template <int CG, int BN>
__device__ __forceinline__ void reduce_rows(const MuonNs& g, const Tiles& T, const Item& it,
                                            uint32_t rank, int warp, int lane, float alpha) {
  const int s = min(g.rows, g.cols);
  const int share = 128 / g.reduce;  // rows of the tile's 128 of this CTA
  const float* from = g.partials + ((int64_t)it.z * T.sym + it.tile) * g.split * (BN * BN);
  const int group = BN == 256 ? lane : lane & 15;
  const int col = it.j * BN + 8 * group;
  for (int q = warp * (256 / BN) + (BN == 256 ? 0 : lane >> 4); q < share;
       q += kEpilogueWarps * (256 / BN)) {
    const int r = (int)rank * 128 + it.share * share + q, row = it.i * BN + r;
    if (row >= s || col >= s) continue;
    float4 lo = make_float4(0.0f, 0.0f, 0.0f, 0.0f), hi = lo;
#pragma unroll 4
    for (int k = 0; k < g.split; ++k) {
      const float4* p =
          reinterpret_cast<const float4*>(from + (int64_t)k * (BN * BN) + r * BN + 8 * group);
      const float4 a = __ldcg(p), b = __ldcg(p + 1);
      lo.x += a.x; lo.y += a.y; lo.z += a.z; lo.w += a.w;
      hi.x += b.x; hi.y += b.y; hi.z += b.z; hi.w += b.w;
    }
    *reinterpret_cast<uint4*>(static_cast<__half*>(g.a) + ((int64_t)it.z * s + row) * g.lds + col) =
        make_uint4(pack_f16(lo.x * alpha, lo.y * alpha), pack_f16(lo.z * alpha, lo.w * alpha),
                   pack_f16(hi.x * alpha, hi.y * alpha), pack_f16(hi.z * alpha, hi.w * alpha));
  }
}

// 64 columns of a warp's rows of P, in place of A's in the output tile.
template <bool DIAGONAL>
__device__ __forceinline__ void poly_chunk(uint32_t tile, int lane, const uint32_t (&v)[2][32],
                                           float alpha, float mid, float diag, int diagonal) {
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const uint32_t at = chunk_address(tile, lane, q);
    const uint4 a = ld_shared(at);
    const uint32_t aw[4] = {a.x, a.y, a.z, a.w};
    uint32_t h[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&aw[e]));
      float x0 = fmaf(y.x, mid, __uint_as_float(v[q >> 2][(8 * q + 2 * e) & 31]) * alpha);
      float x1 = fmaf(y.y, mid, __uint_as_float(v[q >> 2][(8 * q + 2 * e + 1) & 31]) * alpha);
      if constexpr (DIAGONAL) {
        if (8 * q + 2 * e == diagonal) x0 += diag;
        if (8 * q + 2 * e + 1 == diagonal) x1 += diag;
      }
      h[e] = pack_f16(x0, x1);
    }
    st_shared(at, h[0], h[1], h[2], h[3]);
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
  // An item's output: all warps have written theirs; the next one's may follow;
  // P's addend is in shared memory.
  __shared__ __align__(8) uint64_t staged, room, addend;
  __shared__ uint32_t tmem_base_s, stop;
  __shared__ uint32_t issued_s[4];  // copies of A and of B, of this CTA and the pair's other
  const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? (blockIdx.x & 1u) : 0u;
  const uint32_t first = blockIdx.x / CG, stride = gridDim.x / CG;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&full[s]), 2 * CG);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(smem_u32(&acc_full[a]), 1);
      mbar_init(smem_u32(&acc_empty[a]), kEpilogueWarps * CG);
    }
    mbar_init(smem_u32(&staged), kEpilogueWarps);
    mbar_init(smem_u32(&room), 1);
    mbar_init(smem_u32(&addend), 1);
    mbar_init(smem_u32(&drained), 1);
    stop = 0;
    for (int k = 0; k < 4; ++k) issued_s[k] = 0;
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

  // The producing and issuing warps run their loops converged; an elected lane
  // issues.
  const uint32_t tile_base = ring + S * kStageBytes;
  if (warp == 0 || warp == kProducerB) {
    const bool is_a = warp == 0;
    const uint32_t lead = CG == 2 && rank != 0 ? peer_address(smem_u32(&full[0]), 0) : 0;
    uint32_t issued = 0, s = 0, turn = 1;
    bool ok = true;
    int ready_z = -1;
    uint32_t ready = 0;
    for (Walk<BN> walk(g, first, stride); ok && walk.more(); walk.advance()) {
      if (walk.kind == kReduce) continue;
      const Item it = walk.item();
      const bool tall = g.rows > g.cols;
      const int mn_from = first_mn<BN>(g, it, is_a);
      const int which = it.kind == kGram || (it.kind == kUpdate && is_a == tall)
                            ? (it.step & 1)
                            : (it.kind == kPoly ? 2 : 3);
      const CUtensorMap *rows_map = &maps.rows[which], *cols_map = &maps.cols[which];
      const int m0 = is_a ? it.i * BN + (int)rank * 128          // this CTA's rows of A
                          : it.j * BN + (int)rank * (BN / CG);   // and of B
      if (it.z != ready_z || it.before != ready) {
        ok = matrix_wait(g, it.z, it.before * CG, stop_v);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        fence_async_global();
        ready_z = it.z;
        ready = it.before;
      }
      for (int kb = it.kb0; kb < it.kb1; ++kb) {
        ok = mbar_wait_warp(smem_u32(&empty[s]), turn, g.wait_ns, stop_v);
        if (!ok) break;
        const uint32_t to = ring + s * kStageBytes + (is_a ? 0 : kOperandBytes);
        if (elect_one()) {
          uint32_t bar = smem_u32(&full[s]);
          if (CG == 2 && rank != 0) {
            bar = lead + 8 * s;
            mbar_expect_cluster(bar, kOperandBytes);
          } else {
            mbar_expect(bar, kOperandBytes);
          }
          if (kb >= mn_from) {
            tma_load<CG>(to, cols_map, bar, m0, kb * 64, it.z);
            tma_load<CG>(to + 8192, cols_map, bar, m0 + 64, kb * 64, it.z);
          } else {
            tma_load<CG>(to, rows_map, bar, kb * 64, m0, it.z);
          }
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
      issued_s[is_a ? 0 : 1] = issued;
      if (CG == 2 && rank != 0)
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(
                         peer_address(smem_u32(&issued_s[is_a ? 2 : 3]), 0)),
                     "r"(issued)
                     : "memory");
    }
  } else if (warp == 1) {
    if (rank == 0) {
      uint32_t n = 0, s = 0, turn = 0;
      bool ok = true, ready = false;  // the next slice, of whichever item, has landed
      const bool elected = elect_one();
      for (Walk<BN> walk(g, first, stride); ok && walk.more(); walk.advance()) {
        if (walk.kind == kReduce) continue;
        const Item it = walk.item();
        const uint32_t acc = n & 1u;
        const uint32_t d = tmem + acc * BN;
        const int a_from = first_mn<BN>(g, it, true), b_from = first_mn<BN>(g, it, false);
        ok = mbar_wait_warp(smem_u32(&acc_empty[acc]), ((n >> 1) & 1u) ^ 1u, g.wait_ns, stop_v);
        if (!ok) break;
        fence_after();
        for (int kb = it.kb0; kb < it.kb1; ++kb) {
          const uint32_t a = ring + s * kStageBytes, b = a + kOperandBytes;
          const bool a_mn = kb >= a_from, b_mn = kb >= b_from;
          const uint32_t idesc = instruction_desc<CG>(BN, a_mn, b_mn);
          const uint64_t da = operand_desc(a, 8192), db = operand_desc(b, 8192);
          const uint32_t sa = a_mn ? 2048 >> 4 : 32 >> 4, sb = b_mn ? 2048 >> 4 : 32 >> 4;
          if (!ready) ok = mbar_wait_warp(smem_u32(&full[s]), turn, g.wait_ns, stop_v);
          if (!ok) break;
          fence_after();
          const uint32_t done = smem_u32(&empty[s]);
          if (++s == S) {
            s = 0;
            turn ^= 1u;
          }
          // Asked before the MMAs go out, answered behind them.
          const bool landed = mbar_test(smem_u32(&full[s]), turn);
          if (elected) {
            mma_slice<CG>(d, (uint32_t)da, (uint32_t)db, (uint32_t)(da >> 32), sa, sb, idesc,
                          kb != it.kb0);
            mma_commit<CG>(done);
          }
          ready = __all_sync(0xFFFFFFFFu, landed);
        }
        if (ok && elected) mma_commit<CG>(smem_u32(&acc_full[acc]));
        __syncwarp();
        ++n;
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
  } else if (warp == kPorter) {
    const bool elected = elect_one();
    uint32_t done = 0, addends = 0;  // items, and those with an addend
    bool ok = true;
    // The addend of a P tile: the chunks of 64 columns that hold output.
    auto ask = [&](const Item& it) {
      const int N = min(g.rows, g.cols), row0 = it.i * BN + (int)rank * 128;
      const int chunks = row0 < N ? min(BN / 64, (N - it.j * BN + 63) / 64) : 0;
      if (elected) {
        fence_async_global();
        if (chunks > 0)
          mbar_expect(smem_u32(&addend), (uint32_t)chunks * kChunkBytes);
        else
          mbar_arrive(smem_u32(&addend));
        for (int c = 0; c < chunks; ++c)
          tma_load<1>(tile_base + c * kChunkBytes, &maps.rows[2], smem_u32(&addend),
                      it.j * BN + 64 * c, row0, it.z);
      }
      __syncwarp();
      ++addends;
    };
    Walk<BN> walk(g, first, stride);
    Item it = walk.item();
    while (ok && walk.more() && !it.last) {
      if (it.kind == kPoly) {
        ok = matrix_wait(g, it.z, it.before * CG, stop_v);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        ask(it);
      }
      ok = mbar_wait_warp(smem_u32(&staged), done & 1u, g.wait_ns, stop_v);
      if (!ok) break;
      if (elected) {
        mbar_arrive(smem_u32(&room));
        count_item(g, it.z);
      }
      __syncwarp();
      ++done;
      walk.advance();
      it = walk.item();
    }
    if (addends > 0) mbar_drain(smem_u32(&addend), (addends - 1) & 1u);
  } else {
    const int quarter = warp & 3;      // the TMEM lanes this warp may read
    const int side = (warp - 2) >> 2;  // its half of the tile's columns
    // Its 32 rows of the half's chunks in the output tile.
    const uint32_t stage = tile_base + side * kChunks * kChunkBytes + quarter * 4096;
    uint32_t n = 0, out_items = 0, addends = 0;  // items with MMAs, moved out, with an addend
    int ready_z = -1;
    uint32_t ready = 0;
    bool ok = true;
    for (Walk<BN> walk(g, first, stride); ok && walk.more(); walk.advance()) {
      const Item it = walk.item();
      const int M = it.kind == kUpdate ? g.rows : min(g.rows, g.cols);
      const int N = it.kind == kUpdate ? g.cols : M;
      const int row0 = it.i * BN + (int)rank * 128 + quarter * 32;
      const int col0 = it.j * BN + side * (BN / 2);
      const int chunks = row0 < M ? max(0, min(kChunks, (N - col0 + 63) / 64)) : 0;
      float f = it.step == 0 && it.kind != kPoly ? g.factor[it.z] : 1.0f;
      if (it.kind <= kReduce) f *= f;
      const float alpha = f * (it.kind <= kReduce ? g.gram_alpha[it.step]
                                                  : (it.kind == kPoly ? g.poly_alpha[it.step]
                                                                      : g.update_alpha[it.step]));
      if (it.kind == kReduce) {
        if (it.z != ready_z || it.before != ready) {
          ok = matrix_wait(g, it.z, it.before * CG, stop_v);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
          ready_z = it.z;
          ready = it.before;
        }
        reduce_rows<CG, BN>(g, walk.T, it, rank, warp - 2, lane, alpha);
        __syncwarp();  // the lanes' rows before the arrival that counts them
        // No warp arrives for an item before all have arrived for the last one.
        ok = mbar_wait_warp(smem_u32(&room), (out_items & 1u) ^ 1u, g.wait_ns, stop_v);
        if (!ok) break;
        if (lane == 0) mbar_arrive(smem_u32(&staged));
        __syncwarp();
        ++out_items;
        continue;
      }
      const uint32_t acc = n & 1u;
      ok = mbar_wait_warp(smem_u32(&acc_full[acc]), (n >> 1) & 1u, g.wait_ns, stop_v);
      if (!ok) break;
      fence_after();
      if (it.kind == kPoly) {
        ok = mbar_wait_warp(smem_u32(&addend), addends & 1u, g.wait_ns, stop_v);
        if (!ok) break;
        ++addends;
      }
      const uint32_t lanes =
          tmem + ((uint32_t)(quarter * 32) << 16) + acc * BN + side * (BN / 2);
      const bool partial = it.kind == kGram && g.split > 1;
      if (!it.last && !partial) {
        const float mid = g.poly_mid[it.step], diag = g.poly_diag[it.step];
        // The warp's rows of the fp16 output; whole groups of 8 columns fit its stride.
        const int ldo = it.kind == kUpdate ? g.ld : g.lds;
        __half* out = static_cast<__half*>(
            it.kind == kGram ? g.a : (it.kind == kPoly ? g.p : g.x[(it.step & 1) ^ 1]));
        out += ((int64_t)it.z * M + row0) * ldo + col0;
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
          const uint32_t tile = stage + c * kChunkBytes;
          uint32_t v[2][32];
          tmem_load32(lanes + 64 * c, v[0]);
          tmem_load32(lanes + 64 * c + 32, v[1]);
          tmem_load_wait();
          if (it.kind == kPoly) {
            const int diagonal = row0 + lane - (col0 + 64 * c);  // column of the diagonal
            if (row0 < col0 + 64 * c + 64 && col0 + 64 * c < row0 + 32)
              poly_chunk<true>(tile, lane, v, alpha, mid, diag, diagonal);
            else
              poly_chunk<false>(tile, lane, v, alpha, mid, diag, diagonal);
          } else {
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              uint32_t h[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                h[e] = pack_f16(__uint_as_float(v[q >> 2][(8 * q + 2 * e) & 31]) * alpha,
                                __uint_as_float(v[q >> 2][(8 * q + 2 * e + 1) & 31]) * alpha);
              st_shared(chunk_address(tile, lane, q), h[0], h[1], h[2], h[3]);
            }
          }
          __syncwarp();
          // Eight lanes write a row's 128 contiguous bytes.
          const int col = 64 * c + 8 * (lane & 7);
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const int r = 4 * q + (lane >> 3);
            const uint4 u = ld_shared(chunk_address(tile, r, lane & 7));
            if (row0 + r < M && col0 + col < N)
              *reinterpret_cast<uint4*>(out + (int64_t)r * ldo + col) = u;
          }
        }
      } else if (partial) {
        float* out = g.partials +
                     (((int64_t)it.z * walk.T.sym + it.tile) * g.split + it.share) * (BN * BN) +
                     (int)(rank * 128 + quarter * 32) * BN + side * (BN / 2);
#pragma unroll 1
        for (int c = 0; c < 2 * chunks; ++c) {
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
            *reinterpret_cast<uint4*>(out + r * BN + 32 * c + 4 * (lane & 7)) =
                ld_shared(chunk_address(stage, r, lane & 7));
          }
          __syncwarp();
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
      fence_async_shared();
      __syncwarp();
      if (lane == 0) {
        if (CG == 2 && rank != 0)
          mbar_arrive_cluster(peer_address(smem_u32(&acc_empty[acc]), 0));
        else
          mbar_arrive(smem_u32(&acc_empty[acc]));
      }
      ++n;
      if (it.last) continue;
      // No warp arrives for an item before all have arrived for the last one.
      ok = mbar_wait_warp(smem_u32(&room), (out_items & 1u) ^ 1u, g.wait_ns, stop_v);
      if (!ok) break;
      if (lane == 0) mbar_arrive(smem_u32(&staged));
      __syncwarp();
      ++out_items;
    }
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();
  // Operand copies land before their shared memory goes. A slice's barrier counts
  // an arrival per operand and CTA: where the producers gave up at different
  // slices the missing arrivals are made here.
  if (threadIdx.x == 0 && rank == 0) {
    uint32_t least = issued_s[0], most = issued_s[0];
    for (int k = 1; k < 2 * CG; ++k) {
      least = min(least, issued_s[k]);
      most = max(most, issued_s[k]);
    }
    for (uint32_t c = least; c < most; ++c)
      for (int k = 0; k < 2 * CG; ++k)
        if (issued_s[k] <= c) mbar_arrive(smem_u32(&full[c % S]));
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
  // A process-wide driver entry point; threads that ask at once store the same one.
  static std::atomic<EncodeFn> known{nullptr};
  EncodeFn fn = known.load(std::memory_order_relaxed);
  if (!fn) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                                           cudaEnableDefault, &found);
    if (e != cudaSuccess) return e;
    if (found != cudaDriverEntryPointSuccess || !p) return cudaErrorNotSupported;
    fn = reinterpret_cast<EncodeFn>(p);
    known.store(fn, std::memory_order_relaxed);
  }
  *out = fn;
  return cudaSuccess;
}

struct Operand {
  void* p;  // fp16 [batch][rows][ld]
  int32_t rows, cols, ld;
};

// Copies of 64 contiguous elements x `box_rows` rows of a batch of row-major
// matrices; what lies outside a matrix reads as 0.
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
  static std::atomic<int> known[kMaxDevices];  // 0: not asked yet
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < kMaxDevices && (*out = known[dev].load(std::memory_order_acquire)) > 0)
    return cudaSuccess;
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
  if (dev < kMaxDevices) known[dev].store(n, std::memory_order_release);
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

}  // namespace

cudaError_t muon_launch_ns(const MuonNs& g, int bn, cudaStream_t st) {
  Maps maps;
  const int s = std::min(g.rows, g.cols);
  const Operand operands[4] = {{g.x[0], g.rows, g.cols, g.ld},
                               {g.x[1], g.rows, g.cols, g.ld},
                               {g.a, s, s, g.lds},
                               {g.p, s, s, g.lds}};
  for (int k = 0; k < 4; ++k) {
    cudaError_t e = make_map(operands[k], g.batch, 128, &maps.rows[k]);
    if (e == cudaSuccess) e = make_map(operands[k], g.batch, 64, &maps.cols[k]);
    if (e != cudaSuccess) return e;
  }
  // No CTA is without work in the product that has most items.
  const int64_t sym = (int64_t)((s + bn - 1) / bn) * ((s + bn - 1) / bn + 1) / 2 * g.split;
  const int64_t upd = (int64_t)((g.rows + bn - 1) / bn) * ((g.cols + bn - 1) / bn);
  const int64_t most = std::max(sym, upd) * g.batch;
  return bn == 256 ? run<2, 256>(maps, g, most, st) : run<1, 128>(maps, g, most, st);
}

}  // namespace mua

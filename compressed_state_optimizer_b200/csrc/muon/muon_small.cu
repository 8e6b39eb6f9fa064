// Matrices whose iteration fits one SM: the whole operator in one launch, a CTA
// per matrix. X, A and P stay in shared memory as fp16 tiles in the layout the
// MMAs read (128-byte swizzled rows of 64 elements), accumulators in TMEM;
// global memory is read once or twice at the start and written once at the end.
//
// A and P are held as two fp16 tiles each, a value and what its rounding left
// (P's take A's place): A A is then three products and P X two. That costs
// 64 x 64 20.5 us instead of 16.8, 16 x 768 with a step around it 30.6 instead of
// 28.7, 128 x 512 74 instead of 65; a long matrix comes to 0.5e-3 of the exact
// result instead of 0.9e-3 to 2.9e-3, a square one to 0.8e-3 to 1e-3 instead of
// 1.3e-3 to 1.7e-3.
//
// What fits comes here: the general kernels, with their launches and their way
// through L2 between products, take 51 us for 64 x 64 (here 20.5), 68 for 16 x 768
// (27), 235 for 1000 x 64 x 64 (138). Only the longest that fit lose a little,
// 128 x 512 (68, here 73), and stay for the smaller error.
//
// Each of the 3 products per step is a handful of MMAs, issued by a warp of
// their own, followed by an epilogue of the 16 others, so a step is bound by the
// latency of issue, completion, TMEM read and the hand-over, not by arithmetic.
// The issuing warp runs a loop of its own: where it shared one with the others
// it waited some 300 cycles for instructions at every product.
//
// X lies with its long side along the rows of shared memory whichever way the
// caller has it (s = short, l = long side): s rows of ceil(l / 64) chunks,
// padded with zeros to 16 rows and columns; a tall matrix is transposed as it is
// read and written. An MMA always covers 128 rows; those behind the last are
// whatever shared memory holds there, and only make accumulator rows that
// nothing reads.
#include "muon_quant.cuh"

#include <algorithm>

namespace mua {
namespace {

constexpr int kWorkers = 512;             // warps 0 .. 15; warp 16 issues the MMAs
constexpr int kThreads = kWorkers + 32;
constexpr uint32_t kOverread = 16384;  // 128 rows of a chunk that starts at its last row
constexpr uint32_t kMaxSmem = 230000;  // dynamic: 227 KB less what is static

__host__ __device__ __forceinline__ int round16(int x) { return (x + 15) & ~15; }

struct Plan {
  int s, l, s16, l16;     // short and long side, padded
  bool tall;              // rows > cols
  int ns, chunks;         // 64-wide chunks of the short side; of X
  uint32_t xs;            // bytes of a chunk: s16 rows of 128
  uint32_t hi_off, lo_off, bytes;  // of A's and P's two tiles; all
  uint32_t columns;       // of TMEM
};
__host__ __device__ __forceinline__ Plan plan_of(int rows, int cols) {
  Plan p;
  p.tall = rows > cols;
  p.s = p.tall ? cols : rows;
  p.l = p.tall ? rows : cols;
  p.s16 = round16(p.s);
  p.l16 = round16(p.l);
  p.ns = (p.s + 63) / 64;
  p.chunks = (p.l + 63) / 64;
  p.xs = (uint32_t)p.s16 * 128u;
  p.hi_off = (uint32_t)p.chunks * p.xs;
  p.lo_off = p.hi_off + (uint32_t)p.ns * p.xs;
  p.bytes = p.lo_off + (uint32_t)p.ns * p.xs + kOverread;
  const int update = (p.l + 127) / 128 * p.s16;
  const int need = update > 512 ? 512 : (update > p.s16 ? update : p.s16);
  p.columns = 32;
  while ((int)p.columns < need) p.columns *= 2;
  return p;
}

// Address of the 16-byte group holding (row, col .. col + 7) of a chunked tile.
__device__ __forceinline__ uint32_t group_address(uint32_t tile, uint32_t chunk_bytes, int row,
                                                  int col) {
  return chunk_address(tile + (uint32_t)(col >> 6) * chunk_bytes, row, (col >> 3) & 7);
}

// Value (j, i) of X, j along the short side.
__device__ __forceinline__ uint32_t value_address(uint32_t X, uint32_t xs, int j, int i) {
  return group_address(X, xs, j, i) + 2u * (i & 7);
}
__device__ __forceinline__ void st_half(uint32_t at, uint32_t bits) {
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"((uint16_t)bits) : "memory");
}

// Columns col .. col + 15 of a row, in fp16, and what that rounding left of them.
__device__ __forceinline__ void store_split(uint32_t hi, uint32_t lo, uint32_t xs, int row, int col,
                                            const float (&x)[16]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t a[4], b[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float x0 = x[8 * h + 2 * e], x1 = x[8 * h + 2 * e + 1];
      a[e] = pack_f16(x0, x1);
      const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&a[e]));
      b[e] = pack_f16(x0 - y.x, x1 - y.y);
    }
    st_shared(group_address(hi, xs, row, col + 8 * h), a[0], a[1], a[2], a[3]);
    st_shared(group_address(lo, xs, row, col + 8 * h), b[0], b[1], b[2], b[3]);
  }
}

// The 16 values again, to 22 bits.
__device__ __forceinline__ void load_split(uint32_t hi, uint32_t lo, uint32_t xs, int row, int col,
                                           float (&x)[16]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint4 u = ld_shared(group_address(hi, xs, row, col + 8 * h));
    const uint4 w = ld_shared(group_address(lo, xs, row, col + 8 * h));
    const uint32_t a[4] = {u.x, u.y, u.z, u.w}, b[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&a[e]));
      const float2 z = __half22float2(*reinterpret_cast<const __half2*>(&b[e]));
      x[8 * h + 2 * e] = y.x + z.x;
      x[8 * h + 2 * e + 1] = y.y + z.y;
    }
  }
}

// The last product's 16 values of a lane, `left` of them inside the matrix, in
// one row at `at` (four columns a time) or one column (32 lanes are 32
// neighbouring columns). All loads come before the first store.
__device__ __forceinline__ void finish_columns(const MuonNs& g, uint32_t tmem, int64_t at, int left,
                                               float alpha) {
  float4 old[4];
#pragma unroll
  for (int h = 0; h < 4; ++h) old[h] = read_four(g, at + 4 * h, left - 4 * h);
  uint32_t v[16];
  tmem_load16(tmem, v);
  tmem_load_wait();
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const uint32_t y[4] = {v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
    if (4 * h < left) write_four(g, at + 4 * h, left - 4 * h, old[h], y, alpha);
  }
  __syncwarp();
}
__device__ __forceinline__ void finish_rows(const MuonNs& g, uint32_t tmem, int64_t at, int left,
                                            float alpha) {
  float old[16];
  uint32_t v[16];
  if (g.out_type == kF32) {
    float* p = static_cast<float*>(g.out) + at;
#pragma unroll
    for (int e = 0; e < 16; ++e) old[e] = e < left ? p[e * g.ldo] : 0.0f;
    tmem_load16(tmem, v);
    tmem_load_wait();
#pragma unroll
    for (int e = 0; e < 16; ++e)
      if (e < left) p[e * g.ldo] = new_value(g, old[e], __uint_as_float(v[e]), alpha);
  } else {
    uint16_t* p = static_cast<uint16_t*>(g.out) + at;
#pragma unroll
    for (int e = 0; e < 16; ++e)
      old[e] = g.params && e < left ? __uint_as_float((uint32_t)p[e * g.ldo] << 16) : 0.0f;
    tmem_load16(tmem, v);
    tmem_load_wait();
#pragma unroll
    for (int e = 0; e < 16; ++e)
      if (e < left)
        p[e * g.ldo] = __bfloat16_as_ushort(
            __float2bfloat16_rn(new_value(g, old[e], __uint_as_float(v[e]), alpha)));
  }
  __syncwarp();
}

// SRC: 0 fp32 and 1 bf16 matrices to orthogonalize; 2 + type + 2 (4 bits) a step.
template <int SRC>
__global__ void __launch_bounds__(kThreads, 1)
small_kernel(MuonShape sh, const __grid_constant__ MuonNs g, MuonView x, MuonQuant Q,
             const void* grads, float beta, int nesterov, const __grid_constant__ MuonRandom rnd,
             float eps, int e0) {
  constexpr bool STEP = SRC >= 2;
  constexpr int T = SRC & 1;                       // value type of x or the gradients
  constexpr int BITS = SRC >= 4 ? 4 : 8;
  extern __shared__ uint8_t smem_raw[];
  // MMAs of a product complete; taken over by every worker warp; all complete.
  __shared__ __align__(8) uint64_t done, ready, drained;
  __shared__ uint32_t tmem_base_s, stop;
  __shared__ NormScale scale_s;
  const Plan p = plan_of(sh.rows, sh.cols);
  const uint32_t X = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t hi = X + p.hi_off, lo = X + p.lo_off;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t mat = blockIdx.x;
  const int64_t n = (int64_t)sh.rows * sh.cols;

  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&done), 1);
    mbar_init(smem_u32(&ready), kWorkers / 32);
    mbar_init(smem_u32(&drained), 1);
    stop = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  const bool worker = warp < kWorkers / 32;
  if (!worker) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&tmem_base_s)),
                 "r"(p.columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // Rows and columns that pad a side to 16 hold zeros throughout.
  if (((p.s | p.l) & 15) != 0)
    for (uint32_t o = threadIdx.x * 16; worker && o < p.hi_off; o += kWorkers * 16)
      st_shared(X + o, 0u, 0u, 0u, 0u);

  // The norm, then X_0 = x 2^(e0 - t): see muon_launch_load. bf16 matrices may be
  // the result's own memory.
  if constexpr (!STEP) {
    const int es = T == kBf16 ? 2 : 4;
    const uint8_t* xm = static_cast<const uint8_t*>(x.p) + mat * x.matrix_stride * es;
    const bool vec = aligned16(xm) && (x.row_stride * es) % 16 == 0;
    // Groups of 8 columns: along a row for a wide matrix, down the rows for a tall
    // one, whose neighbouring lanes then write neighbouring columns of X.
    const uint32_t per_row = (uint32_t)(sh.cols + 7) / 8, groups = per_row * (uint32_t)sh.rows;
    const uint32_t line = p.tall ? (uint32_t)sh.rows : per_row;
    auto place = [&](uint32_t q, int& row, int& col) {
      const uint32_t a = q / line, b = q - a * line;
      row = (int)(p.tall ? b : a);
      col = 8 * (int)(p.tall ? a : b);
    };
    double sum = 0.0;
    // Up to kHeld groups of 8 per thread stay in registers between the passes.
    constexpr int kHeld = 2;
    uint64_t held[kHeld][4];
    for (uint32_t q0 = threadIdx.x; worker && q0 < groups; q0 += kHeld * kWorkers) {
#pragma unroll
      for (int k = 0; k < kHeld; ++k) {
        const uint32_t q = q0 + k * kWorkers;
        int row, col;
        place(q, row, col);
        load8<T, T != kBf16>(xm + (int64_t)row * x.row_stride * es, col, q < groups ? sh.cols : 0, vec,
                             held[k]);
      }
#pragma unroll
      for (int k = 0; k < kHeld; ++k) sum += sum_squares(held[k]);
    }
    sum = cta_sum<kThreads>(sum);
    if (threadIdx.x == 0) scale_s = scale_of(sum, eps, e0);
    __syncthreads();
    const NormScale ns = scale_s;
#pragma unroll 1
    for (uint32_t q = threadIdx.x, k = 0; worker && q < groups; q += kWorkers, ++k) {
      int row, col;
      place(q, row, col);
      uint64_t v[4];
      if (groups > kHeld * kWorkers) {
        load8<T, T != kBf16>(xm + (int64_t)row * x.row_stride * es, col, sh.cols, vec, v);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = k == 0 ? held[0][e] : held[1][e];
      }
      const uint4 h = scaled_f16(v, ns.first, ns.second);
      if (!p.tall) {
        st_shared(group_address(X, p.xs, row, col), h.x, h.y, h.z, h.w);
      } else {
        const uint32_t hw[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (col + e < sh.cols)
            st_half(value_address(X, p.xs, col + e, row), hw[e >> 1] >> (16 * (e & 1)));
      }
    }
  } else {
    const int half = threadIdx.x >> 4, sub = threadIdx.x & 15;
    const uint8_t* gm = static_cast<const uint8_t*>(grads) + mat * n * (T == kBf16 ? 2 : 4);
    const bool vec = aligned16(gm);
    const int64_t base = mat * Q.bpm;
    // Chunks of kHeld blocks per half-warp; a matrix of one chunk stays in
    // registers between the passes.
    constexpr int kHeld = 3;
    constexpr int kChunk = kHeld * (kWorkers / 16);
    uint64_t gv[kHeld][4];
    float scale[kHeld];
    uint2 codes[kHeld];
    auto fetch = [&](int64_t b0) {
#pragma unroll
      for (int k = 0; k < kHeld; ++k) {
        const int64_t b = b0 + half + k * (kWorkers / 16);
        codes[k] = make_uint2(0u, 0u);
        scale[k] = 0.0f;
        if (b < Q.bpm) {
          codes[k] = load_codes<BITS>(Q.codes, base + b, sub);
          scale[k] = Q.scales[base + b];
        }
        load8<T>(gm, b * kMuonBlock + 8 * sub, n, vec, gv[k]);
      }
    };
    double sum = 0.0;
    for (int64_t b0 = 0; worker && b0 < Q.bpm; b0 += kChunk) {
      fetch(b0);
#pragma unroll
      for (int k = 0; k < kHeld; ++k) {
        uint64_t q[4], m[4], u[4];
        unpack8<BITS>(codes[k], q);
        new_momentum(q, scale[k], gv[k], beta, nesterov, m, u);
        sum += sum_squares(u);
      }
    }
    sum = cta_sum<kThreads>(sum);
    if (threadIdx.x == 0) scale_s = scale_of(sum, eps, e0);
    __syncthreads();
    const NormScale ns = scale_s;
    bool bad = false;
    for (int64_t b0 = 0; worker && b0 < Q.bpm; b0 += kChunk) {
      if (Q.bpm > kChunk) fetch(b0);
#pragma unroll 1
      for (int k = 0; k < kHeld; ++k) {
        const int64_t b = b0 + half + k * (kWorkers / 16);
        if (b0 + 2 * warp + k * (kWorkers / 16) >= Q.bpm) break;
        const int64_t i = b * kMuonBlock + 8 * sub;
        const int left = left_of(i, n);
        uint64_t q[4], m[4], u[4], now[4];
        float old_scale = 0.0f, new_scale;
        uint2 old_codes = make_uint2(0u, 0u);
#pragma unroll
        for (int h = 0; h < kHeld; ++h)
          if (h == k) {
            old_codes = codes[h];
            old_scale = scale[h];
#pragma unroll
            for (int e = 0; e < 4; ++e) now[e] = gv[h][e];
          }
        unpack8<BITS>(old_codes, q);
        new_momentum(q, old_scale, now, beta, nesterov, m, u);
        uint32_t c[8];
        quantize_block<BITS>(m, left, (uint64_t)(rnd.base + (base + b) * kMuonBlock) / 8 + sub, rnd,
                             new_scale, c, bad);
        if (b < Q.bpm) {
          store_codes<BITS>(Q.codes, base + b, sub, c);
          if (sub == 0) Q.scales[base + b] = new_scale;
          int row = (int)((uint32_t)i / (uint32_t)sh.cols);
          int col = (int)i - row * sh.cols;
          const uint4 h = scaled_f16(u, ns.first, ns.second);
          if (!p.tall && (sh.cols & 7) == 0) {  // eight values of one row
            if (left > 0) st_shared(group_address(X, p.xs, row, col), h.x, h.y, h.z, h.w);
          } else {
            const uint32_t hw[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              if (e < left)
                st_half(value_address(X, p.xs, p.tall ? col : row, p.tall ? row : col),
                        hw[e >> 1] >> (16 * (e & 1)));
              if (++col == sh.cols) {
                col = 0;
                ++row;
              }
            }
          }
        }
      }
    }
    if (bad || (threadIdx.x == 0 && isnan(ns.factor))) atomicOr(Q.status, kMuonNonFinite);
  }
  fence_async_shared();
  fence_before();
  __syncthreads();
  fence_after();

  const uint32_t tmem = tmem_base_s;
  volatile uint32_t* stop_v = &stop;
  const int sunits = p.s16 / 16;
  const int tiles = (p.l + 127) / 128, pass = 512 / p.s16;  // of X', in TMEM at once
  uint32_t stage = 0;  // products begun, counting the update's passes
  bool ok = true;

  if (!worker) {
    const bool lead = elect_one();
    const uint32_t sym = instruction_desc<1>(p.s16, false, false);
    const uint32_t upd = instruction_desc<1>(p.s16, true, false);
    const uint64_t x0 = operand_desc(X, 16), h0 = operand_desc(hi, 16), l0 = operand_desc(lo, 16);
    const uint64_t xt = operand_desc(X, p.xs);  // X by its columns
    const uint32_t chunk = p.xs >> 4;
    // `depth` k-steps of 16 along the rows of two operands.
    auto along = [&](uint64_t a, uint64_t b, int depth, bool more) {
      for (int kk = 0; kk < depth; ++kk) {
        if (lead) mma_f16<1>(tmem, a, b, sym, more || kk != 0);
        const uint32_t step = (kk & 3) == 3 ? chunk - 6 : 2;
        a += step;
        b += step;
      }
    };
    // The others have taken the last product over.
    auto begin = [&]() {
      if (stage > 0) ok = mbar_wait_warp(smem_u32(&ready), (stage - 1) & 1u, g.wait_ns, stop_v);
      fence_after();
      ++stage;
      return ok;
    };
    for (int k = 0; ok && k < g.steps; ++k) {
      if (!begin()) break;
      along(x0, x0, p.l16 / 16, false);  // X X^T
      if (lead) mma_commit<1>(smem_u32(&done));
      if (!begin()) break;
      along(h0, h0, sunits, false);      // A A without its low parts' product
      along(h0, l0, sunits, true);
      along(l0, h0, sunits, true);
      if (lead) mma_commit<1>(smem_u32(&done));
      for (int t0 = 0; t0 < tiles; t0 += pass) {
        if (!begin()) break;
        // X^T P: 128 columns of X (two chunks) a tile, 16 rows a step.
        uint64_t a_tile = xt + (uint32_t)t0 * 2 * chunk;
        const int now = min(pass, tiles - t0);
        for (int t = 0; t < now; ++t, a_tile += 2 * chunk) {
          uint64_t a = a_tile, b = h0, c = l0;
          for (int kk = 0; kk < sunits; ++kk) {
            if (lead) {
              mma_f16<1>(tmem + t * p.s16, a, b, upd, kk != 0);
              mma_f16<1>(tmem + t * p.s16, a, c, upd, true);
            }
            a += 2048 >> 4;
            const uint32_t step = (kk & 3) == 3 ? chunk - 6 : 2;
            b += step;
            c += step;
          }
        }
        if (lead) mma_commit<1>(smem_u32(&done));
      }
    }
    __syncwarp();
  } else {
    const float factor = scale_s.factor;
    const int quarter = warp & 3, part = warp >> 2;  // TMEM lanes; every fourth 16 columns
    const int lane_row = quarter * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
    // The next product's MMAs are complete.
    auto take = [&]() {
      ok = mbar_wait_warp(smem_u32(&done), stage & 1u, g.wait_ns, stop_v);
      fence_after();
      ++stage;
      return ok;
    };
    // This warp has read its part of them and written what the next one reads.
    auto hand_over = [&]() {
      fence_async_shared();
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ready));
    };
    for (int k = 0; k < g.steps; ++k) {
      // A = f^2 X X^T
      if (!take()) break;
      if (quarter * 32 < p.s16) {
        const float alpha = k == 0 ? g.gram_alpha[0] * factor * factor : g.gram_alpha[k];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int u = part + 4 * q;
          if (u < sunits) {
            uint32_t v[16];
            float x[16];
            tmem_load16(lanes + 16 * u, v);
            tmem_load_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = __uint_as_float(v[e]) * alpha;
            if (lane_row < p.s16) store_split(hi, lo, p.xs, lane_row, 16 * u, x);
            __syncwarp();
          }
        }
      }
      hand_over();

      // P = a I + b A + c A A
      if (!take()) break;
      if (quarter * 32 < p.s16) {
        const float alpha = g.poly_alpha[k], mid = g.poly_mid[k], diag = g.poly_diag[k];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int u = part + 4 * q;
          if (u < sunits) {
            uint32_t v[16];
            tmem_load16(lanes + 16 * u, v);
            tmem_load_wait();
            const int diagonal = lane_row < p.s ? lane_row - 16 * u : -1;
            if (lane_row < p.s16) {
              float x[16];
              load_split(hi, lo, p.xs, lane_row, 16 * u, x);  // of A: its own values
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                x[e] = fmaf(x[e], mid, __uint_as_float(v[e]) * alpha);
                if (e == diagonal) x[e] += diag;
              }
              store_split(hi, lo, p.xs, lane_row, 16 * u, x);
            }
            __syncwarp();
          }
        }
      }
      hand_over();

      // X' = f P X, with the long side along the accumulator rows so that all TMEM
      // lanes work: tile t holds its rows 128 t .. in columns s16 t .. of a pass of
      // up to 512 columns. A pass replaces only what no other tile reads.
      const bool last = k == g.steps - 1;
      const float alpha = k == 0 ? g.update_alpha[0] * factor : g.update_alpha[k];
      for (int t0 = 0; t0 < tiles; t0 += pass) {
        const int now = min(pass, tiles - t0);
        if (!take()) break;
        for (int u = part; u < now * sunits; u += 4) {
          const int t = u / sunits, j0 = 16 * (u - t * sunits);  // short side j0 .. j0 + 15
          const int i0 = (t0 + t) * 128 + quarter * 32;          // long side
          if (i0 >= p.l16) continue;
          const int i = i0 + lane;
          if (last) {
            const int64_t at = mat * g.batch_stride + (p.tall ? i * g.ldo + j0 : j0 * g.ldo + i);
            if (p.tall)
              finish_columns(g, lanes + 16 * u, at, i < p.l ? p.s - j0 : 0, alpha);
            else
              finish_rows(g, lanes + 16 * u, at, i < p.l ? p.s - j0 : 0, alpha);
            continue;
          }
          uint32_t v[16];
          tmem_load16(lanes + 16 * u, v);
          tmem_load_wait();
          if (i < p.l16) {
            // A lane's value of 16 rows: 32 lanes write 64 contiguous bytes of each.
            // Rows j0 + e, with j0 a multiple of 16, swizzle by e & 7.
            const uint32_t base = X + (uint32_t)(i >> 6) * p.xs + j0 * 128 + 2 * (i & 7);
            const uint32_t group = (uint32_t)(i & 56) << 1;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const uint32_t w = pack_f16(__uint_as_float(v[2 * e]) * alpha,
                                          __uint_as_float(v[2 * e + 1]) * alpha);
              st_half(base + (2 * e) * 128 + (group ^ ((2 * e & 7) << 4)), w);
              st_half(base + (2 * e + 1) * 128 + (group ^ ((2 * e + 1 & 7) << 4)), w >> 16);
            }
          }
          __syncwarp();
        }
        hand_over();
      }
      if (!ok) break;
    }
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  fence_after();
  // MMAs in flight end before shared memory and TMEM go.
  if (!worker) {
    if (stop_v[0] != 0 && stage > 0) {
      if (elect_one()) mma_commit<1>(smem_u32(&drained));
      mbar_drain(smem_u32(&drained), 0);
    }
    __syncwarp();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(p.columns));
  }
  if (threadIdx.x == 0 && stop) atomicOr(g.status, kMuonTimeout);
}

template <int SRC>
cudaError_t run(const MuonShape& s, const MuonNs& g, const MuonView& x, const MuonQuant& q,
                const void* grads, float beta, int nesterov, const MuonRandom& rnd, float eps,
                int e0, cudaStream_t st) {
  auto kernel = small_kernel<SRC>;
  const uint32_t smem = muon_small_smem(s.rows, s.cols);
  // One attribute for all handles of the process: always the same value, so that no
  // thread's call lowers it before another's launch.
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxSmem);
  if (e != cudaSuccess) return e;
  kernel<<<(unsigned)s.count, kThreads, smem, st>>>(s, g, x, q, grads, beta, nesterov, rnd, eps, e0);
  return cudaGetLastError();
}

}  // namespace

uint32_t muon_small_smem(int32_t rows, int32_t cols) {
  if (std::min(rows, cols) > 128) return 0;
  const uint32_t bytes = plan_of(rows, cols).bytes + 1024;  // + alignment
  return bytes <= kMaxSmem ? bytes : 0;
}

cudaError_t muon_launch_small(const MuonShape& s, const MuonNs& g, const MuonView& x, float eps,
                              int e0, cudaStream_t st) {
  const MuonQuant q = {};
  const MuonRandom r = {};
  return x.type == kBf16 ? run<1>(s, g, x, q, nullptr, 0.0f, 0, r, eps, e0, st)
                         : run<0>(s, g, x, q, nullptr, 0.0f, 0, r, eps, e0, st);
}

cudaError_t muon_launch_small_step(const MuonShape& s, const MuonNs& g, const MuonQuant& q,
                                   const void* grads, int g_type, float beta, int nesterov,
                                   const MuonRandom& rnd, float eps, int e0, cudaStream_t st) {
  const MuonView x = {};
  auto k = q.bits == 8 ? (g_type == kBf16 ? run<3> : run<2>) : (g_type == kBf16 ? run<5> : run<4>);
  return k(s, g, x, q, grads, beta, nesterov, rnd, eps, e0, st);
}

}  // namespace mua

// Matrices whose iteration fits one SM: the whole operator in one launch, a CTA
// per matrix. X, A and P stay in shared memory as fp16 tiles in the layout the
// MMAs read (128-byte swizzled rows of 64 elements), accumulators in TMEM;
// global memory is read once or twice at the start and written once at the end.
//
// Each of the 3 products per step is a handful of MMAs, issued by a warp of
// their own, followed by an epilogue of the 16 others, so a step is bound by the latency of issue, completion,
// TMEM read and CTA barrier, not by arithmetic. X has the caller's orientation
// (s = short, l = long side): a wide one is s rows of ceil(l / 64) chunks, a
// tall one l rows of ceil(s / 64) chunks, rows and contracted columns padded
// with zeros to 16. An MMA always covers 128 rows; those behind the last are
// whatever shared memory holds there, and only make accumulator rows that
// nothing reads.
#include "muon_quant.cuh"

#include <algorithm>

namespace mua {
namespace {

constexpr int kWorkers = 512;             // warps 0 .. 15; warp 16 issues the MMAs
constexpr int kThreads = kWorkers + 32;
constexpr uint32_t kOverread = 16384;  // 128 rows of a chunk that starts at its last row

__host__ __device__ __forceinline__ int round16(int x) { return (x + 15) & ~15; }

struct Plan {
  int s, l, s16, l16;     // short and long side, padded
  bool tall;
  int ns, chunks;         // 64-wide chunks of the short side; of X
  uint32_t xs, ps;        // bytes of a chunk of X, of A and P
  uint32_t a_off, p_off, bytes;
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
  p.chunks = p.tall ? p.ns : (p.l + 63) / 64;
  p.xs = (uint32_t)(p.tall ? p.l16 : p.s16) * 128u;
  p.ps = (uint32_t)p.s16 * 128u;
  p.a_off = (uint32_t)p.chunks * p.xs;
  p.p_off = p.a_off + (uint32_t)p.ns * p.ps;
  p.bytes = p.p_off + (uint32_t)p.ns * p.ps + kOverread;
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
  __shared__ __align__(8) uint64_t done;
  __shared__ uint32_t tmem_base_s, stop;
  __shared__ NormScale scale_s;
  const Plan p = plan_of(sh.rows, sh.cols);
  const uint32_t X = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t A = X + p.a_off, P = X + p.p_off;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t mat = blockIdx.x;
  const int64_t n = (int64_t)sh.rows * sh.cols;

  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&done), 1);
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
    for (uint32_t o = threadIdx.x * 16; worker && o < p.a_off; o += kWorkers * 16)
      st_shared(X + o, 0u, 0u, 0u, 0u);

  // The norm, then X_0 = x 2^(e0 - t): see muon_launch_load.
  if constexpr (!STEP) {
    const int es = T == kBf16 ? 2 : 4;
    const uint8_t* xm = static_cast<const uint8_t*>(x.p) + mat * x.matrix_stride * es;
    const bool vec = aligned16(xm) && (x.row_stride * es) % 16 == 0;
    const uint32_t per_row = (uint32_t)(sh.cols + 7) / 8, groups = per_row * (uint32_t)sh.rows;
    double sum = 0.0;
    // Up to kHeld groups of 8 per thread stay in registers between the passes.
    constexpr int kHeld = 2;
    uint64_t held[kHeld][4];
    for (uint32_t q0 = threadIdx.x; worker && q0 < groups; q0 += kHeld * kWorkers) {
#pragma unroll
      for (int k = 0; k < kHeld; ++k) {
        const uint32_t q = q0 + k * kWorkers;
        const uint32_t row = q / per_row, col = 8 * (q - row * per_row);
        const int64_t end = q < groups ? sh.cols : 0;
        load8<T>(xm + (int64_t)row * x.row_stride * es, col, end, vec, held[k]);
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
      const uint32_t row = q / per_row, col = 8 * (q - row * per_row);
      uint64_t v[4];
      if (groups > kHeld * kWorkers) {
        load8<T>(xm + (int64_t)row * x.row_stride * es, col, sh.cols, vec, v);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = k == 0 ? held[0][e] : held[1][e];
      }
      const uint4 h = scaled_f16(v, ns.first, ns.second);
      st_shared(group_address(X, p.xs, (int)row, (int)col), h.x, h.y, h.z, h.w);
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
          if ((sh.cols & 7) == 0) {  // eight values of one row
            if (left > 0) st_shared(group_address(X, p.xs, row, col), h.x, h.y, h.z, h.w);
          } else {
            const uint32_t hw[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              if (e < left)
                asm volatile("st.shared.u16 [%0], %1;" ::"r"(group_address(X, p.xs, row, col) +
                                                             2u * (col & 7)),
                             "h"((uint16_t)(hw[e >> 1] >> (16 * (e & 1))))
                             : "memory");
              if (++col == sh.cols) {
                col = 0;
                ++row;
              }
            }
          }
        }
      }
    }
    if (bad) atomicOr(Q.status, kMuonNonFinite);
  }
  fence_async_shared();
  fence_before();
  __syncthreads();
  fence_after();

  const uint32_t tmem = tmem_base_s;
  const float factor = scale_s.factor;
  const int quarter = warp & 3, part = warp >> 2;     // TMEM lanes; every fourth 16 columns
  const int lane_row = quarter * 32 + lane;
  const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
  const int sunits = p.s16 / 16;
  volatile uint32_t* stop_v = &stop;
  uint32_t turn = 0;
  bool ok = true;
  // Waits for the MMAs issued. A thread that gives up goes on to the next
  // publish(), where the CTA stops as one; what it reads until then is unused.
  auto finish = [&]() {
    ok = mbar_wait(smem_u32(&done), turn, g.wait_ns, stop_v);
    fence_after();
  };
  // Every thread's tile writes and TMEM reads come before the next MMAs.
  auto publish = [&]() {
    fence_async_shared();
    fence_before();
    ok = __syncthreads_or(!ok) == 0;
    fence_after();
    if (ok) turn ^= 1u;
    return ok;
  };

  // The issuing warp runs converged (descriptors stay in uniform registers).
  const uint32_t sym_idesc = instruction_desc<1>(p.s16, false, false);
  for (int k = 0; ok && k < g.steps; ++k) {
    // A = f^2 X X^T
    if (!worker) {
      const bool lead = elect_one();
      if (p.tall) {
        const uint32_t idesc = instruction_desc<1>(p.s16, true, true);
        // 64 further rows of A behind a single chunk: the chunk again.
        uint64_t d = operand_desc(X, p.ns > 1 ? p.xs : 0);
        for (int kk = 0; kk < p.l16 / 16; ++kk, d += 2048 >> 4)
          if (lead) mma_f16<1>(tmem, d, d, idesc, kk != 0);
      } else {
        uint64_t chunk = operand_desc(X, 16);
        for (int left = p.l16 / 16, first = 1; left > 0; left -= 4, chunk += p.xs >> 4) {
          uint64_t d = chunk;
          for (int kk = 0; kk < min(4, left); ++kk, d += 32 >> 4, first = 0)
            if (lead) mma_f16<1>(tmem, d, d, sym_idesc, first == 0);
        }
      }
      if (lead) mma_commit<1>(smem_u32(&done));
      __syncwarp();
    }
    finish();
    uint32_t held[2][8];  // this thread's part of A, for the next product
    if (worker && quarter * 32 < p.s16) {
      const float alpha = k == 0 ? g.gram_alpha[0] * factor * factor : g.gram_alpha[k];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int u = part + 4 * q;
        if (u < sunits) {
          uint32_t v[16];
          tmem_load16(lanes + 16 * u, v);
          tmem_load_wait();
#pragma unroll
          for (int e = 0; e < 8; ++e)
            held[q][e] = pack_f16(__uint_as_float(v[2 * e]) * alpha,
                                  __uint_as_float(v[2 * e + 1]) * alpha);
          if (lane_row < p.s16) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
              st_shared(group_address(A, p.ps, lane_row, 16 * u + 8 * h), held[q][4 * h],
                        held[q][4 * h + 1], held[q][4 * h + 2], held[q][4 * h + 3]);
          }
          __syncwarp();
        }
      }
    }
    if (!publish()) break;

    // P = a I + b A + c A A
    if (!worker) {
      const bool lead = elect_one();
      uint64_t chunk = operand_desc(A, 16);
      for (int left = sunits, first = 1; left > 0; left -= 4, chunk += p.ps >> 4) {
        uint64_t d = chunk;
        for (int kk = 0; kk < min(4, left); ++kk, d += 32 >> 4, first = 0)
          if (lead) mma_f16<1>(tmem, d, d, sym_idesc, first == 0);
      }
      if (lead) mma_commit<1>(smem_u32(&done));
      __syncwarp();
    }
    finish();
    if (worker && quarter * 32 < p.s16) {
      const float alpha = g.poly_alpha[k], mid = g.poly_mid[k], diag = g.poly_diag[k];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int u = part + 4 * q;
        if (u < sunits) {
          uint32_t v[16];
          tmem_load16(lanes + 16 * u, v);
          tmem_load_wait();
          const int diagonal = lane_row < p.s ? lane_row - 16 * u : -1;
          uint32_t w[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&held[q][e]));
            float x0 = fmaf(y.x, mid, __uint_as_float(v[2 * e]) * alpha);
            float x1 = fmaf(y.y, mid, __uint_as_float(v[2 * e + 1]) * alpha);
            if (2 * e == diagonal) x0 += diag;
            if (2 * e + 1 == diagonal) x1 += diag;
            w[e] = pack_f16(x0, x1);
          }
          if (lane_row < p.s16) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
              st_shared(group_address(P, p.ps, lane_row, 16 * u + 8 * h), w[4 * h], w[4 * h + 1],
                        w[4 * h + 2], w[4 * h + 3]);
          }
          __syncwarp();
        }
      }
    }
    if (!publish()) break;

    // X' = f P X (X P), with the long side along the accumulator rows either
    // way so that all TMEM lanes work: tile t holds its rows 128 t .. in columns
    // s16 t .. of a pass of up to 512 columns. A pass replaces only what no
    // other tile reads.
    const bool last = k == g.steps - 1;
    const float alpha = k == 0 ? g.update_alpha[0] * factor : g.update_alpha[k];
    const int tiles = (p.l + 127) / 128, pass = 512 / p.s16;
    for (int p0 = 0; ok && p0 < tiles; p0 += pass) {
      const int now = min(pass, tiles - p0);
      if (!worker) {
        const bool lead = elect_one();
        const uint32_t idesc = instruction_desc<1>(p.s16, !p.tall, false);
        // Tall: rows of X, 16 columns a step, 64 a chunk. Wide: columns of X (two
        // chunks a tile), 16 rows a step.
        uint64_t tile = p.tall ? operand_desc(X + p0 * 16384, 16)
                               : operand_desc(X + 2 * p0 * p.xs, p.xs);
        const uint64_t tile_step = p.tall ? 16384 >> 4 : (2 * p.xs) >> 4;
        const uint64_t a_step = p.tall ? 32 >> 4 : 2048 >> 4;
        const uint64_t a_chunk = p.tall ? p.xs >> 4 : 4 * (2048 >> 4);
        const uint64_t b0 = operand_desc(P, 16);
        for (int t = 0; t < now; ++t, tile += tile_step) {
          uint64_t a_at = tile, b_at = b0;
          for (int left = sunits, first = 1; left > 0;
               left -= 4, a_at += a_chunk, b_at += p.ps >> 4) {
            uint64_t a = a_at, b = b_at;
            for (int kk = 0; kk < min(4, left); ++kk, a += a_step, b += 32 >> 4, first = 0)
              if (lead) mma_f16<1>(tmem + t * p.s16, a, b, idesc, first == 0);
          }
        }
        if (lead) mma_commit<1>(smem_u32(&done));
        __syncwarp();
      }
      finish();
      for (int u = part; worker && u < now * sunits; u += 4) {
        const int t = u / sunits, j0 = 16 * (u - t * sunits);  // short side j0 .. j0 + 15
        const int i0 = (p0 + t) * 128 + quarter * 32;          // long side
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
        uint32_t v[16], w[8];
        tmem_load16(lanes + 16 * u, v);
        tmem_load_wait();
#pragma unroll
        for (int e = 0; e < 8; ++e)
          w[e] = pack_f16(__uint_as_float(v[2 * e]) * alpha, __uint_as_float(v[2 * e + 1]) * alpha);
        if (p.tall) {
          if (i < p.l16) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
              st_shared(group_address(X, p.xs, i, j0 + 8 * h), w[4 * h], w[4 * h + 1],
                        w[4 * h + 2], w[4 * h + 3]);
          }
        } else if (i < p.l16) {
          // A lane's value of 16 rows: 32 lanes write 64 contiguous bytes of each.
          // Rows j0 + e, with j0 a multiple of 16, swizzle by e & 7.
          const uint32_t base = X + (uint32_t)(i >> 6) * p.xs + j0 * 128 + 2 * (i & 7);
          const uint32_t group = (uint32_t)(i & 56) << 1;
#pragma unroll
          for (int e = 0; e < 16; ++e)
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(base + e * 128 +
                                                         (group ^ ((e & 7) << 4))),
                         "h"((uint16_t)(w[e >> 1] >> (16 * (e & 1))))
                         : "memory");
        }
        __syncwarp();
      }
      if (!publish()) break;
    }
  }
  // MMAs in flight end before shared memory and TMEM go.
  if (!ok) mbar_drain(smem_u32(&done), turn);
  __syncthreads();
  if (!worker)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(p.columns));
  if (threadIdx.x == 0 && stop) atomicOr(g.status, kMuonTimeout);
}

template <int SRC>
cudaError_t run(const MuonShape& s, const MuonNs& g, const MuonView& x, const MuonQuant& q,
                const void* grads, float beta, int nesterov, const MuonRandom& rnd, float eps,
                int e0, cudaStream_t st) {
  auto kernel = small_kernel<SRC>;
  const uint32_t smem = muon_small_smem(s.rows, s.cols);
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  kernel<<<(unsigned)s.count, kThreads, smem, st>>>(s, g, x, q, grads, beta, nesterov, rnd, eps, e0);
  return cudaGetLastError();
}

}  // namespace

uint32_t muon_small_smem(int32_t rows, int32_t cols) {
  if (std::min(rows, cols) > 128 || std::max(rows, cols) > 8192) return 0;
  const uint32_t bytes = plan_of(rows, cols).bytes + 1024;  // + alignment
  return bytes <= 230000 ? bytes : 0;
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

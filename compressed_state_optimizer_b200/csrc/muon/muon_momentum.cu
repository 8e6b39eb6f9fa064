// The quantized momentum of the Muon step and the input of its orthogonalization.
//
// The arithmetic of a block is in muon_quant.cuh.
//
// Half a warp holds a block, 8 values per lane: a 16-byte load of bf16
// gradients (two for fp32), one 8- or 4-byte load of codes, one Philox call
// per lane; the block maximum is four shuffles. Nothing is read twice, and U is
// formed from the unrounded m' in the same pass. Of 6.06 bytes a value (bf16
// gradients and direction, 8 bits) HBM would take 0.34 ms for 8 x 11008 x 4096;
// the update takes 0.55 ms, with 4 bits as with 8, so not HBM but its 36
// instructions a value (a fifth of them Philox, the rest the conversions, the clamp
// and the packing) set the time, at 2.4 of the 4 that an SM can issue a cycle: 43 %
// of the warps are resident and a third of their stalls wait for loads. At full
// issue the same instructions would take some 0.36 ms. Packed fp32 pairs and the
// next run's loads in flight brought it there from 0.96 ms. Reading back runs at
// HBM's rate (0.17 ms).
#include "muon_quant.cuh"

#include <algorithm>

namespace mua {
namespace {

constexpr int kThreads = 256;
constexpr int kNormUnroll = 4, kLoadUnroll = 2;
constexpr int kUnroll = 2;                             // blocks per half-warp
constexpr int kChunkBlocks = kThreads / 16 * kUnroll;  // 32 blocks (4096 values) per CTA

__device__ __forceinline__ void wait_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void release_next() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// ---------------------------------------------------------------- kernels

// Grid: splits x count CTAs; a CTA takes every splits-th run of 16 blocks of one
// matrix, the next run's loads in flight while it works on one.
// OUT: 0 fp32, 1 bf16 (contiguous), 2 fp16 X_0 with row stride ld.
template <int BITS, int G, int OUT>
__global__ void __launch_bounds__(kThreads, 4)
momentum_kernel(MuonShape s, MuonQuant Q, const void* g, float beta, int nesterov,
                const __grid_constant__ MuonRandom rnd, void* out, const double* partials,
                float eps, int e0, void* X, float* factor, uint32_t* counters, int splits) {
  wait_previous();
  release_next();
  constexpr int kRun = kThreads / 16;
  const int mat = blockIdx.x / splits, split = blockIdx.x - mat * splits;
  const int64_t n = (int64_t)s.rows * s.cols;
  const int half = threadIdx.x >> 4, sub = threadIdx.x & 15;
  const void* gm = static_cast<const uint8_t*>(g) + mat * n * (G == kBf16 ? 2 : 4);
  const bool vec = aligned16(gm);
  const int64_t base = mat * Q.bpm;
  constexpr int os = OUT == kBf16 ? 2 : 4;
  uint8_t* om = static_cast<uint8_t*>(out) + mat * n * os;
  const bool out_vec = OUT != 2 && aligned16(om);

  // This lane's place in the run: pointers, which advance by a step, and the
  // index in the matrix (below 2^31).
  const uint32_t blocks = (uint32_t)Q.bpm, step = (uint32_t)splits * kRun;
  uint32_t b = (uint32_t)split * kRun + half;
  uint8_t* codes = Q.codes + ((base + b) * kMuonBlock + 8 * sub) * BITS / 8;
  float* scales = Q.scales + base + b;
  uint64_t next_g[4];
  uint2 next_codes;
  float next_scale;
  auto fetch = [&](uint32_t at, const uint8_t* c, const float* sc) {
    next_codes = make_uint2(0u, 0u);
    next_scale = 0.0f;
    if (at < blocks) {
      next_codes = load_codes<BITS>(c);
      next_scale = *sc;
    }
    load8<G>(gm, (int64_t)at * kMuonBlock + 8 * sub, n, vec, next_g);
  };
  fetch(b, codes, scales);
  uint64_t counter = (uint64_t)(rnd.base + (base + b) * kMuonBlock) / 8 + sub;
  NormScale ns;
  if constexpr (OUT == 2) {
    ns = norm_scale(partials + (int64_t)mat * s.parts, s.parts, eps, e0);
    if (split == 0 && threadIdx.x == 0) {
      factor[mat] = ns.factor;
      counters[mat] = 0;
      if (isnan(ns.factor)) atomicOr(Q.status, kMuonNonFinite);
    }
  }
  bool bad = false;
  for (; b - half < blocks; b += step) {
    uint64_t q[4], m[4], u[4];
    unpack8<BITS>(next_codes, q);
    new_momentum(q, next_scale, next_g, beta, nesterov, m, u);
    uint8_t* codes_now = codes;
    float* scales_now = scales;
    codes += (int64_t)step * (kMuonBlock * BITS / 8);
    scales += step;
    if (b - half + step < blocks) fetch(b + step, codes, scales);
    const int64_t i = (int64_t)b * kMuonBlock + 8 * sub;
    const int left = left_of(i, n);
    float new_scale;
    uint32_t c[8];
    quantize_block<BITS>(m, left, counter, rnd, new_scale, c, bad);
    counter += (uint64_t)step * (kMuonBlock / 8);
    if (b < blocks) {
      store_codes<BITS>(codes_now, c);
      if (sub == 0) *scales_now = new_scale;
      if constexpr (OUT == 2) {
        __half* x = static_cast<__half*>(X) + (int64_t)mat * s.rows * s.ld;
        const uint4 h = scaled_f16(u, ns.first, ns.second);
        const uint32_t row = s.ld == s.cols ? 0 : (uint32_t)i / (uint32_t)s.cols;
        if ((s.cols & 7) == 0) {  // eight values of one row
          if (left > 0) *reinterpret_cast<uint4*>(x + i + (int64_t)row * (s.ld - s.cols)) = h;
        } else {
          const uint32_t hw[4] = {h.x, h.y, h.z, h.w};
          uint32_t col = (uint32_t)i - row * (uint32_t)s.cols;
          uint16_t* at = reinterpret_cast<uint16_t*>(x) + (int64_t)row * s.ld + col;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (e < left) *at = (uint16_t)(hw[e >> 1] >> (16 * (e & 1)));
            ++at;
            if (++col == (uint32_t)s.cols) {
              col = 0;
              at += s.ld - s.cols;
            }
          }
        }
      } else {
        store8<OUT>(om, i, n, out_vec, u);
      }
    }
  }
  if (bad) atomicOr(Q.status, kMuonNonFinite);
}

// Partial sums of U^2: as momentum_kernel, without a write to the state. Four
// blocks in flight at 64 registers spill 64 to 96 bytes a thread; the kernel takes
// 2.5 times what its bytes would (53 us for 4096 x 11008, 8 bits, bf16 gradients).
template <int BITS, int G>
__global__ void __launch_bounds__(kThreads, 4)
direction_norm_kernel(MuonShape s, MuonQuant Q, const void* g, float beta, int nesterov,
                      double* partials) {
  wait_previous();
  release_next();
  const int mat = blockIdx.x / s.parts, part = blockIdx.x - mat * s.parts;
  const int64_t n = (int64_t)s.rows * s.cols;
  const int half = threadIdx.x >> 4, sub = threadIdx.x & 15;
  const void* gm = static_cast<const uint8_t*>(g) + mat * n * (G == kBf16 ? 2 : 4);
  const bool vec = aligned16(gm);
  const int64_t base = mat * Q.bpm;
  double sum = 0.0;
  const int64_t stride = (int64_t)s.parts * (kThreads / 16);
  uint64_t gv[kNormUnroll][4];
  uint2 codes[kNormUnroll];
  float scale[kNormUnroll];
  auto fetch = [&](int k, int64_t b) {
    codes[k] = make_uint2(0u, 0u);
    scale[k] = 0.0f;
    if (b < Q.bpm) {
      codes[k] = load_codes<BITS>(Q.codes, base + b, sub);
      scale[k] = Q.scales[base + b];
    }
    load8<G>(gm, b * kMuonBlock + 8 * sub, n, vec, gv[k]);
  };
  int64_t b = (int64_t)part * (kThreads / 16) + half;
#pragma unroll
  for (int k = 0; k < kNormUnroll; ++k) fetch(k, b + k * stride);
  while (b < Q.bpm) {
#pragma unroll
    for (int k = 0; k < kNormUnroll; ++k) {  // a block, and the loads of one further on
      // Codes behind the last value are 0 and its gradients read as 0.
      uint64_t q[4], m[4], u[4];
      unpack8<BITS>(codes[k], q);
      new_momentum(q, scale[k], gv[k], beta, nesterov, m, u);
      if (b + kNormUnroll * stride < Q.bpm)
        fetch(k, b + kNormUnroll * stride);
      else
        codes[k] = make_uint2(0u, 0u), gv[k][0] = gv[k][1] = gv[k][2] = gv[k][3] = 0;
      sum += sum_squares(u);
      b += stride;
    }
  }
  const double t = cta_sum<kThreads>(sum);
  if (threadIdx.x == 0) partials[blockIdx.x] = t;
}

// Groups of 8 values of one row of a strided stack; a contiguous matrix counts
// as one row of rows * cols values.
template <int T>
__global__ void __launch_bounds__(kThreads, 4)
norm_kernel(MuonShape s, MuonView x, double* partials) {
  wait_previous();
  release_next();
  const int mat = blockIdx.x / s.parts, part = blockIdx.x - mat * s.parts;
  const int es = T == kBf16 ? 2 : 4;
  const uint8_t* xm = static_cast<const uint8_t*>(x.p) + mat * x.matrix_stride * es;
  const bool flat = x.row_stride == s.cols;
  const int64_t cols = flat ? (int64_t)s.rows * s.cols : s.cols;
  const bool vec = aligned16(xm) && (flat || (x.row_stride * es) % 16 == 0);
  const uint32_t per_row = (uint32_t)((cols + 7) / 8);
  const uint32_t groups = per_row * (flat ? 1u : (uint32_t)s.rows);
  double sum = 0.0;
  const uint64_t stride = (uint64_t)s.parts * kThreads;
  uint64_t v[kNormUnroll][4];
  auto fetch = [&](int k, uint64_t q) {
    const uint32_t row = (uint32_t)q / per_row, col = 8 * ((uint32_t)q - row * per_row);
    load8<T>(xm + (int64_t)row * x.row_stride * es, col, q < groups ? cols : 0, vec, v[k]);
  };
  uint64_t q = (uint64_t)part * kThreads + threadIdx.x;
#pragma unroll
  for (int k = 0; k < kNormUnroll; ++k) fetch(k, q + k * stride);
  while (q < groups) {
#pragma unroll
    for (int k = 0; k < kNormUnroll; ++k) {  // a group, and the loads of one further on
      sum += sum_squares(v[k]);
      fetch(k, q + kNormUnroll * stride);
      q += stride;
    }
  }
  const double t = cta_sum<kThreads>(sum);
  if (threadIdx.x == 0) partials[blockIdx.x] = t;
}

template <int T>
__global__ void __launch_bounds__(kThreads)
load_kernel(MuonShape s, MuonView x, const double* partials, float eps, int e0, void* X,
            float* factor, uint32_t* counters, int splits) {
  wait_previous();
  release_next();
  const int mat = blockIdx.x / splits, split = blockIdx.x - mat * splits;
  const int es = T == kBf16 ? 2 : 4;
  const uint8_t* xm = static_cast<const uint8_t*>(x.p) + mat * x.matrix_stride * es;
  const bool vec = aligned16(xm) && (x.row_stride * es) % 16 == 0;
  const uint32_t per_row = (uint32_t)(s.cols + 7) / 8, groups = per_row * (uint32_t)s.rows;
  const NormScale ns = norm_scale(partials + (int64_t)mat * s.parts, s.parts, eps, e0);
  if (split == 0 && threadIdx.x == 0) {
    factor[mat] = ns.factor;
    counters[mat] = 0;
  }
  __half* out = static_cast<__half*>(X) + (int64_t)mat * s.rows * s.ld;
  const uint64_t stride = (uint64_t)splits * kThreads;
  for (uint64_t q0 = (uint64_t)split * kThreads + threadIdx.x; q0 < groups;
       q0 += kLoadUnroll * stride) {
    uint64_t v[kLoadUnroll][4];
    uint4* to[kLoadUnroll];
#pragma unroll
    for (int k = 0; k < kLoadUnroll; ++k) {
      const uint64_t q = q0 + k * stride;
      const uint32_t row = (uint32_t)q / per_row, col = 8 * ((uint32_t)q - row * per_row);
      to[k] = q < groups ? reinterpret_cast<uint4*>(out + (int64_t)row * s.ld + col) : nullptr;
      load8<T>(xm + (int64_t)row * x.row_stride * es, col, q < groups ? s.cols : 0, vec, v[k]);
    }
#pragma unroll
    for (int k = 0; k < kLoadUnroll; ++k)
      if (to[k]) *to[k] = scaled_f16(v[k], ns.first, ns.second);
  }
}

template <int BITS, int T>
__global__ void __launch_bounds__(kThreads)
read_kernel(MuonShape s, MuonQuant Q, void* out, int splits) {
  const int mat = blockIdx.x / splits, split = blockIdx.x - mat * splits;
  const int64_t n = (int64_t)s.rows * s.cols;
  const int half = threadIdx.x >> 4, sub = threadIdx.x & 15;
  uint8_t* om = static_cast<uint8_t*>(out) + mat * n * (T == kBf16 ? 2 : 4);
  const bool vec = aligned16(om);
  const int64_t base = mat * Q.bpm;
  uint2 codes[kUnroll];
  float scale[kUnroll];
#pragma unroll
  for (int k = 0; k < kUnroll; ++k) {
    const int64_t b = (int64_t)split * kChunkBlocks + half + k * (kThreads / 16);
    if (b < Q.bpm) {
      codes[k] = load_codes<BITS>(Q.codes, base + b, sub);
      scale[k] = Q.scales[base + b];
    }
  }
#pragma unroll
  for (int k = 0; k < kUnroll; ++k) {
    const int64_t b = (int64_t)split * kChunkBlocks + half + k * (kThreads / 16);
    if (b < Q.bpm) {
      uint64_t q[4];
      unpack8<BITS>(codes[k], q);
#pragma unroll
      for (int e = 0; e < 4; ++e) q[e] = f2_mul_rn(q[e], f2_splat(scale[k]));
      store8<T>(om, b * kMuonBlock + 8 * sub, n, vec, q);
    }
  }
}

// Codes of given values, each to the nearest level (ties to even). Values read
// from a block that holds level L come back as the same codes.
template <int BITS, int T>
__global__ void __launch_bounds__(kThreads)
write_kernel(MuonShape s, MuonQuant Q, const void* values, int splits) {
  const int mat = blockIdx.x / splits, split = blockIdx.x - mat * splits;
  const int64_t n = (int64_t)s.rows * s.cols;
  const int half = threadIdx.x >> 4, sub = threadIdx.x & 15;
  const uint8_t* vm = static_cast<const uint8_t*>(values) + mat * n * (T == kBf16 ? 2 : 4);
  const bool vec = aligned16(vm);
  const int64_t base = mat * Q.bpm;
  bool bad = false;
#pragma unroll
  for (int k = 0; k < kUnroll; ++k) {
    const int64_t b = (int64_t)split * kChunkBlocks + half + k * (kThreads / 16);
    uint64_t v[4];
    load8<T>(vm, b * kMuonBlock + 8 * sub, n, vec, v);
    float top = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      top = max_magnitude(max_magnitude(top, f2_lo(v[e])), f2_hi(v[e]));
    top = half_warp_max(top);
    float scale, inverse;
    block_scale(top, Level<BITS>::recip, scale, inverse);
    bad = bad || !(top < __uint_as_float(0x7F800000u));
    uint32_t c[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x = (e & 1) ? f2_hi(v[e >> 1]) : f2_lo(v[e >> 1]);
      const float y = fminf(fmaxf(__fmul_rn(x, inverse), -Level<BITS>::value),
                            Level<BITS>::value);
      c[e] = __float_as_uint(__fadd_rn(y, 12582912.0f));
    }
    if (b < Q.bpm) {
      store_codes<BITS>(Q.codes, base + b, sub, c);
      if (sub == 0) Q.scales[base + b] = scale;
    }
  }
  if (bad) atomicOr(Q.status, kMuonNonFinite);
}

template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), int64_t grid, cudaStream_t st, bool overlap, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = overlap ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

// CTAs a matrix is split over: eight for each SM of a B200 in all, and none
// without work. Four run at once; twice as many even out their ends (592 CTAs
// take 0.64 ms for the update of 8 x 11008 x 4096, 1184 0.55 ms, 4736 0.57 ms).
int splits_for(int count, int64_t work, int64_t per_cta) {
  const int64_t most = (work + per_cta - 1) / per_cta;
  return (int)std::max<int64_t>(1, std::min<int64_t>(most, 8 * 148 / count));
}

int64_t chunk_splits(const MuonQuant& q) { return (q.bpm + kChunkBlocks - 1) / kChunkBlocks; }

}  // namespace

cudaError_t muon_launch_norm(const MuonShape& s, const MuonView& x, double* partials,
                             cudaStream_t st) {
  const int64_t grid = (int64_t)s.count * s.parts;
  return x.type == kBf16 ? launch(norm_kernel<kBf16>, grid, st, false, s, x, partials)
                         : launch(norm_kernel<kF32>, grid, st, false, s, x, partials);
}

cudaError_t muon_launch_load(const MuonShape& s, const MuonView& x, const double* partials,
                             float eps, int e0, void* X, float* factor, uint32_t* counters,
                             cudaStream_t st) {
  const int splits = splits_for(s.count, (int64_t)s.rows * ((s.cols + 7) / 8), kLoadUnroll * kThreads);
  const int64_t grid = (int64_t)s.count * splits;
  auto k = x.type == kBf16 ? load_kernel<kBf16> : load_kernel<kF32>;
  return launch(k, grid, st, true, s, x, partials, eps, e0, X, factor, counters, splits);
}

cudaError_t muon_launch_direction_norm(const MuonShape& s, const MuonQuant& q, const void* g,
                                       int g_type, float beta, int nesterov, double* partials,
                                       cudaStream_t st) {
  const int64_t grid = (int64_t)s.count * s.parts;
  auto k = q.bits == 8 ? (g_type == kBf16 ? direction_norm_kernel<8, kBf16>
                                          : direction_norm_kernel<8, kF32>)
                       : (g_type == kBf16 ? direction_norm_kernel<4, kBf16>
                                          : direction_norm_kernel<4, kF32>);
  return launch(k, grid, st, false, s, q, g, beta, nesterov, partials);
}

template <int OUT>
static auto pick_momentum(int bits, int g_type) {
  return bits == 8
             ? (g_type == kBf16 ? momentum_kernel<8, kBf16, OUT> : momentum_kernel<8, kF32, OUT>)
             : (g_type == kBf16 ? momentum_kernel<4, kBf16, OUT> : momentum_kernel<4, kF32, OUT>);
}

cudaError_t muon_launch_momentum(const MuonShape& s, const MuonQuant& q, const void* g, int g_type,
                                 float beta, int nesterov, const MuonRandom& rnd, void* out,
                                 int out_type, const double* partials, float eps, int e0, void* X,
                                 float* factor, uint32_t* counters, cudaStream_t st) {
  const int splits = splits_for(s.count, q.bpm, kThreads / 16);
  auto k = X ? pick_momentum<2>(q.bits, g_type)
             : (out_type == kBf16 ? pick_momentum<1>(q.bits, g_type)
                                  : pick_momentum<0>(q.bits, g_type));
  return launch(k, (int64_t)splits * s.count, st, X != nullptr, s, q, g, beta, nesterov, rnd, out,
                partials, eps, e0, X, factor, counters, splits);
}

cudaError_t muon_launch_read(const MuonShape& s, const MuonQuant& q, void* out, int out_type,
                             cudaStream_t st) {
  const int64_t splits = chunk_splits(q);
  auto k = q.bits == 8 ? (out_type == kBf16 ? read_kernel<8, kBf16> : read_kernel<8, kF32>)
                       : (out_type == kBf16 ? read_kernel<4, kBf16> : read_kernel<4, kF32>);
  return launch(k, splits * s.count, st, false, s, q, out, (int)splits);
}

cudaError_t muon_launch_write(const MuonShape& s, const MuonQuant& q, const void* values, int type,
                              cudaStream_t st) {
  const int64_t splits = chunk_splits(q);
  auto k = q.bits == 8 ? (type == kBf16 ? write_kernel<8, kBf16> : write_kernel<8, kF32>)
                       : (type == kBf16 ? write_kernel<4, kBf16> : write_kernel<4, kF32>);
  return launch(k, splits * s.count, st, false, s, q, values, (int)splits);
}

}  // namespace mua

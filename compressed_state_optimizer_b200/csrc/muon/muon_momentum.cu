// The quantized momentum of the Muon step and the input of its orthogonalization.
//
// State: blocks of 128 consecutive values of one matrix share an fp32 scale s;
// a value is s q with q an 8-bit or 4-bit two's complement level, |q| <= L
// (127 or 7). One update is
//   m = s q,  m' = beta m + g,  U = g + beta m' (or m'),
//   a = max |m'| over the block,  s' = a / L,  q' = floor(m' / s' + u)
// with u = r / 2^16 and r the value's 16-bit half of a Philox4x32-10 word.
// Rounding to nearest would pin small values: with beta = 0.95 a level q <= 10
// decays by less than half a step and never moves; the stochastic rounding is
// unbiased at 2^-16 of a step. All of it is fp32 with one rounding per
// operation (the reciprocal included), so a result is fixed bit for bit.
//
// Half a warp holds a block, 8 values per lane: a 16-byte load of bf16
// gradients (two for fp32), one 8- or 4-byte load of codes, one Philox call
// per lane; the block maximum is four shuffles. Bound by HBM: nothing is
// read twice, and U is formed from the unrounded m' in the same pass.
#include "../mua_kernels.cuh"
#include "muon.cuh"

#include <cuda_fp16.h>

namespace mua {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;                          // blocks per half-warp
constexpr int kChunkBlocks = kThreads / 16 * kUnroll;  // 64 blocks (8192 values) per CTA

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Eight consecutive values of type T from p[i ..], those at or past n as 0.
template <int T>
__device__ __forceinline__ void load8(const void* p, int64_t i, int64_t n, bool vec, float (&v)[8]) {
  if (vec && i + 8 <= n) {
    if constexpr (T == kBf16) {
      const uint4 w = ld_stream_v4(static_cast<const uint16_t*>(p) + i);
      v[0] = bf16_lo(w.x); v[1] = bf16_hi(w.x); v[2] = bf16_lo(w.y); v[3] = bf16_hi(w.y);
      v[4] = bf16_lo(w.z); v[5] = bf16_hi(w.z); v[6] = bf16_lo(w.w); v[7] = bf16_hi(w.w);
    } else {
      const float* f = static_cast<const float*>(p) + i;
      const uint4 a = ld_stream_v4(f), b = ld_stream_v4(f + 4);
      v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y);
      v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
      v[4] = __uint_as_float(b.x); v[5] = __uint_as_float(b.y);
      v[6] = __uint_as_float(b.z); v[7] = __uint_as_float(b.w);
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    v[e] = 0.0f;
    if (i + e < n) {
      if constexpr (T == kBf16)
        v[e] = __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i + e] << 16);
      else
        v[e] = static_cast<const float*>(p)[i + e];
    }
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  return (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(lo)) |
         ((uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(hi)) << 16);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <int T>
__device__ __forceinline__ void store8(void* p, int64_t i, int64_t n, bool vec, const float (&v)[8]) {
  if (vec && i + 8 <= n) {
    if constexpr (T == kBf16) {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) =
          make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                     pack_bf16(v[6], v[7]));
    } else {
      float4* f = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
      f[0] = make_float4(v[0], v[1], v[2], v[3]);
      f[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (i + e < n) {
      if constexpr (T == kBf16)
        static_cast<uint16_t*>(p)[i + e] = __bfloat16_as_ushort(__float2bfloat16_rn(v[e]));
      else
        static_cast<float*>(p)[i + e] = v[e];
    }
}

// Levels of 8 codes as floats: the biased code in the low mantissa bits of
// 2^23 (exact, without the quarter-rate conversion).
template <int BITS>
__device__ __forceinline__ void unpack8(uint2 w, float (&q)[8]) {
  constexpr float bias = 8388608.0f + (BITS == 8 ? 128.0f : 8.0f);
  if constexpr (BITS == 8) {
    const uint32_t a = w.x ^ 0x80808080u, b = w.y ^ 0x80808080u;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      q[e] = __uint_as_float(__byte_perm(a, 0x4B000000u, 0x7650 + e)) - bias;
      q[4 + e] = __uint_as_float(__byte_perm(b, 0x4B000000u, 0x7650 + e)) - bias;
    }
  } else {
    const uint32_t a = w.x ^ 0x88888888u;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      q[e] = __uint_as_float(((a >> (4 * e)) & 15u) | 0x4B000000u) - bias;
  }
}

template <int BITS>
__device__ __forceinline__ uint2 load_codes(const uint8_t* codes, int64_t block, int sub) {
  if constexpr (BITS == 8) {
    return *reinterpret_cast<const uint2*>(codes + block * kMuonBlock + 8 * sub);
  } else {
    return make_uint2(
        *reinterpret_cast<const uint32_t*>(codes + block * (kMuonBlock / 2) + 4 * sub), 0u);
  }
}

template <int BITS>
__device__ __forceinline__ void store_codes(uint8_t* codes, int64_t block, int sub,
                                            const uint32_t (&c)[8]) {
  if constexpr (BITS == 8) {
    const uint32_t a = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040),
                                   0x5410);
    const uint32_t b = __byte_perm(__byte_perm(c[4], c[5], 0x0040), __byte_perm(c[6], c[7], 0x0040),
                                   0x5410);
    *reinterpret_cast<uint2*>(codes + block * kMuonBlock + 8 * sub) = make_uint2(a, b);
  } else {
    uint32_t w = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) w |= (c[e] & 15u) << (4 * e);
    *reinterpret_cast<uint32_t*>(codes + block * (kMuonBlock / 2) + 4 * sub) = w;
  }
}

// Scale and its reciprocal of a block whose largest magnitude has the bit
// pattern top. A block below 2^-100 holds zeros: 1 / scale would overflow.
// NaN and infinity order above every finite value as bits and stay in the scale.
__device__ __forceinline__ void block_scale(uint32_t top, float level_recip, float& scale,
                                            float& inverse) {
  const float a = __uint_as_float(top);
  scale = 0.0f;
  inverse = 0.0f;
  if (!(a < 7.8886090522101181e-31f)) {  // 2^-100
    scale = __fmul_rn(a, level_recip);
    inverse = __frcp_rn(scale);
  }
}

__device__ __forceinline__ uint32_t half_warp_max(uint32_t v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

template <int BITS>
struct Level {
  static constexpr float value = BITS == 8 ? 127.0f : 7.0f;
  static constexpr float recip = 1.0f / value;  // rounded to fp32
};

// m' = beta m + g and U of 8 values.
__device__ __forceinline__ void new_momentum(const float (&q)[8], float scale, const float (&g)[8],
                                             float beta, int nesterov, float (&m)[8],
                                             float (&u)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    m[e] = __fadd_rn(__fmul_rn(beta, __fmul_rn(q[e], scale)), g[e]);
    u[e] = nesterov ? __fadd_rn(__fmul_rn(beta, m[e]), g[e]) : m[e];
  }
}

__device__ __forceinline__ double sum_squares(const float (&v)[8]) {
  double s = 0.0;
#pragma unroll
  for (int e = 0; e < 8; ++e) s = fma((double)v[e], (double)v[e], s);
  return s;
}

// Sum over the CTA in a fixed order; valid in thread 0.
__device__ __forceinline__ double cta_sum(double v) {
  __shared__ double warp_sums[kThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if ((threadIdx.x & 31) == 0) warp_sums[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
  if (threadIdx.x == 0)
    for (int w = 0; w < kThreads / 32; ++w) s += warp_sums[w];
  return s;
}

// 2^(e0 - t) as two factors (each an fp32 power of two) and 2^t / (|x| + eps),
// 2^(t-1) <= |x| + eps < 2^t, from the partial sums; the same in every CTA.
// A norm below 2^-126 makes X_0 = 0; one that is not finite makes it NaN.
struct NormScale {
  float first, second, factor;
};
__device__ __forceinline__ NormScale norm_scale(const double* partials, int parts, float eps,
                                                int e0) {
  __shared__ NormScale shared;
  if (threadIdx.x < 32) {
    double s = 0.0;
    for (int i = threadIdx.x; i < parts; i += 32) s += partials[i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    if (threadIdx.x == 0) {
      const double n = sqrt(s) + (double)eps;
      NormScale r;
      if (!(n <= 1.7e308)) {
        r.first = r.second = r.factor = __uint_as_float(0x7FC00000u);
      } else if (n < 1.1754943508222875e-38) {  // 2^-126
        r.first = r.second = 0.0f;
        r.factor = 1.0f;
      } else {
        const int t = ilogb(n) + 1;
        const int c = max(-126, min(126, -t));
        r.first = (float)scalbn(1.0, c);
        r.second = (float)scalbn(1.0, e0 - t - c);
        r.factor = (float)(scalbn(1.0, t) / n);
      }
      shared = r;
    }
  }
  __syncthreads();
  return shared;
}

__device__ __forceinline__ void wait_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void release_next() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// ---------------------------------------------------------------- kernels

// Grid: splits x count CTAs, a CTA takes 64 consecutive blocks of one matrix.
// OUT: 0 fp32, 1 bf16 (contiguous), 2 fp16 X_0 with row stride ld.
template <int BITS, int G, int OUT>
__global__ void __launch_bounds__(kThreads)
momentum_kernel(MuonShape s, MuonQuant Q, const void* g, float beta, int nesterov,
                const __grid_constant__ MuonRandom rnd, void* out, const double* partials,
                float eps, int e0, void* X, float* factor, uint32_t* counters, int splits) {
  wait_previous();
  release_next();
  const int mat = blockIdx.x / splits, split = blockIdx.x - mat * splits;
  const int64_t n = (int64_t)s.rows * s.cols;
  const int half = threadIdx.x >> 4, sub = threadIdx.x & 15;
  const int es = G == kBf16 ? 2 : 4;
  const void* gm = static_cast<const uint8_t*>(g) + mat * n * es;
  const bool vec = aligned16(gm);
  const int64_t first = (int64_t)split * kChunkBlocks + half;
  const int64_t base = mat * Q.bpm;

  float gv[kUnroll][8];
  uint2 codes[kUnroll];
  float scale[kUnroll];
#pragma unroll
  for (int k = 0; k < kUnroll; ++k) {
    const int64_t b = first + k * (kThreads / 16);
    codes[k] = make_uint2(0u, 0u);
    scale[k] = 0.0f;
    if (b < Q.bpm) {
      codes[k] = load_codes<BITS>(Q.codes, base + b, sub);
      scale[k] = Q.scales[base + b];
    }
    load8<G>(gm, b * kMuonBlock + 8 * sub, n, vec, gv[k]);
  }
  NormScale ns;
  if constexpr (OUT == 2) {
    ns = norm_scale(partials + (int64_t)mat * s.parts, s.parts, eps, e0);
    if (split == 0 && threadIdx.x == 0) {
      factor[mat] = ns.factor;
      counters[mat] = 0;
    }
  }
  bool bad = false;
#pragma unroll
  for (int k = 0; k < kUnroll; ++k) {
    const int64_t b = first + k * (kThreads / 16);
    float q[8], m[8], u[8];
    unpack8<BITS>(codes[k], q);
    new_momentum(q, scale[k], gv[k], beta, nesterov, m, u);
    const int64_t i = b * kMuonBlock + 8 * sub;
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      // Behind the matrix's last value nothing is held (its codes are 0).
      if (i + e >= n) m[e] = 0.0f;
      top = max(top, __float_as_uint(m[e]) & 0x7FFFFFFFu);
    }
    top = half_warp_max(top);
    float ns_scale, inverse;
    block_scale(top, Level<BITS>::recip, ns_scale, inverse);
    bad = bad || top >= 0x7F800000u;
    const uint64_t counter = (uint64_t)(rnd.base + (base + b) * kMuonBlock) / 8 + sub;
    const uint4 w = philox4x32_10((uint32_t)counter, (uint32_t)(counter >> 32), rnd.t_lo, rnd.t_hi,
                                  rnd.keys);
    uint32_t c[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t word = chunk_word(w, e >> 1);
      // 1 + r / 2^16, then floor(y + r / 2^16) by rounding toward -inf: first
      // below any integer it passes, then at unit spacing near 1.5 2^23.
      const uint32_t r = (e & 1) ? (word >> 9) & 0x007FFF80u : (word << 7) & 0x007FFF80u;
      const float y = fminf(fmaxf(__fmul_rn(m[e], inverse), -Level<BITS>::value),
                            Level<BITS>::value);
      const float z = __fadd_rd(y, __uint_as_float(0x3F800000u | r));
      c[e] = __float_as_uint(__fadd_rd(z, 12582911.0f));
      if (i + e >= n) c[e] = 0;
    }
    if (b < Q.bpm) {
      store_codes<BITS>(Q.codes, base + b, sub, c);
      if (sub == 0) Q.scales[base + b] = ns_scale;
      if constexpr (OUT == 2) {
        __half* x = static_cast<__half*>(X) + (int64_t)mat * s.rows * s.ld;
#pragma unroll
        for (int e = 0; e < 8; ++e) u[e] = u[e] * ns.first * ns.second;
        if ((s.cols & 7) == 0) {  // eight values of one row, and ld == cols
          if (i < n)
            *reinterpret_cast<uint4*>(x + i) =
                make_uint4(pack_f16(u[0], u[1]), pack_f16(u[2], u[3]), pack_f16(u[4], u[5]),
                           pack_f16(u[6], u[7]));
        } else {
          uint32_t row = (uint32_t)i / (uint32_t)s.cols;
          uint32_t col = (uint32_t)i - row * (uint32_t)s.cols;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (i + e < n) x[(int64_t)row * s.ld + col] = __float2half_rn(u[e]);
            if (++col == (uint32_t)s.cols) { col = 0; ++row; }
          }
        }
      } else {
        const int os = OUT == kBf16 ? 2 : 4;
        uint8_t* om = static_cast<uint8_t*>(out) + mat * n * os;
        store8<OUT>(om, i, n, aligned16(om), u);
      }
    }
  }
  if (bad) atomicOr(Q.status, kMuonNonFinite);
}

// Partial sums of U^2: as momentum_kernel, without a write to the state.
template <int BITS, int G>
__global__ void __launch_bounds__(kThreads)
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
  for (int64_t b = (int64_t)part * (kThreads / 16) + half; b < Q.bpm;
       b += (int64_t)s.parts * (kThreads / 16)) {
    float q[8], m[8], u[8], gv[8];
    load8<G>(gm, b * kMuonBlock + 8 * sub, n, vec, gv);
    unpack8<BITS>(load_codes<BITS>(Q.codes, base + b, sub), q);
    // Codes behind the last value are 0 and its gradients read as 0.
    new_momentum(q, Q.scales[base + b], gv, beta, nesterov, m, u);
    sum += sum_squares(u);
  }
  const double t = cta_sum(sum);
  if (threadIdx.x == 0) partials[blockIdx.x] = t;
}

// Groups of 8 values of one row of a strided stack; a contiguous matrix counts
// as one row of rows * cols values.
template <int T>
__global__ void __launch_bounds__(kThreads)
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
  for (uint64_t q = (uint64_t)part * kThreads + threadIdx.x; q < groups;
       q += (uint64_t)s.parts * kThreads) {
    const uint32_t row = (uint32_t)q / per_row, col = 8 * ((uint32_t)q - row * per_row);
    float v[8];
    load8<T>(xm + (int64_t)row * x.row_stride * es, col, cols, vec, v);
    sum += sum_squares(v);
  }
  const double t = cta_sum(sum);
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
  const uint32_t per_row = (uint32_t)(s.ld / 8), groups = per_row * (uint32_t)s.rows;
  const NormScale ns = norm_scale(partials + (int64_t)mat * s.parts, s.parts, eps, e0);
  if (split == 0 && threadIdx.x == 0) {
    factor[mat] = ns.factor;
    counters[mat] = 0;
  }
  __half* out = static_cast<__half*>(X) + (int64_t)mat * s.rows * s.ld;
  for (uint64_t q = (uint64_t)split * kThreads + threadIdx.x; q < groups;
       q += (uint64_t)splits * kThreads) {
    const uint32_t row = (uint32_t)q / per_row, col = 8 * ((uint32_t)q - row * per_row);
    float v[8];
    load8<T>(xm + (int64_t)row * x.row_stride * es, col, s.cols, vec, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = v[e] * ns.first * ns.second;
    *reinterpret_cast<uint4*>(out + (int64_t)row * s.ld + col) =
        make_uint4(pack_f16(v[0], v[1]), pack_f16(v[2], v[3]), pack_f16(v[4], v[5]),
                   pack_f16(v[6], v[7]));
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
      float q[8];
      unpack8<BITS>(codes[k], q);
#pragma unroll
      for (int e = 0; e < 8; ++e) q[e] = __fmul_rn(q[e], scale[k]);
      store8<T>(om, b * kMuonBlock + 8 * sub, n, vec, q);
    }
  }
}

// Codes of given values, each to the nearest level (ties to even): values
// read from a state come back as the same codes.
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
    float v[8];
    load8<T>(vm, b * kMuonBlock + 8 * sub, n, vec, v);
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[e]) & 0x7FFFFFFFu);
    top = half_warp_max(top);
    float scale, inverse;
    block_scale(top, Level<BITS>::recip, scale, inverse);
    bad = bad || top >= 0x7F800000u;
    uint32_t c[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float y = fminf(fmaxf(__fmul_rn(v[e], inverse), -Level<BITS>::value),
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
  // Two 16-byte groups per thread.
  const int64_t groups = (int64_t)s.rows * (s.ld / 8);
  const int splits = (int)((groups + 2 * kThreads - 1) / (2 * kThreads));
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
  const int64_t splits = chunk_splits(q);
  auto k = X ? pick_momentum<2>(q.bits, g_type)
             : (out_type == kBf16 ? pick_momentum<1>(q.bits, g_type)
                                  : pick_momentum<0>(q.bits, g_type));
  return launch(k, splits * s.count, st, X != nullptr, s, q, g, beta, nesterov, rnd, out, partials,
                eps, e0, X, factor, counters, (int)splits);
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

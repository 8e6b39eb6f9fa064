// The quantized momentum's arithmetic, and the norm's, shared by the Muon
// kernels (muon_momentum.cu, muon_small.cu).
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
#pragma once

#include "../mua_kernels.cuh"
#include "muon_tc.cuh"

namespace mua {
namespace {

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

// Scale and its reciprocal of a block whose largest magnitude is a. A block
// below 2^-100 holds zeros: 1 / scale would overflow. NaN and infinity stay in
// the scale.
__device__ __forceinline__ void block_scale(float a, float level_recip, float& scale,
                                            float& inverse) {
  scale = 0.0f;
  inverse = 0.0f;
  if (!(a < 7.8886090522101181e-31f)) {  // 2^-100
    scale = __fmul_rn(a, level_recip);
    inverse = __frcp_rn(scale);
  }
}

// The larger magnitude, NaN if either is.
__device__ __forceinline__ float max_magnitude(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}
__device__ __forceinline__ float half_warp_max(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = max_magnitude(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
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

// Scale and codes of a block's new momentum, of which this lane holds 8 values,
// `left` (8 or fewer) of them inside the matrix; all lanes of a warp call it.
template <int BITS>
__device__ __forceinline__ void quantize_block(float (&m)[8], int left, uint64_t counter,
                                               const MuonRandom& rnd, float& scale,
                                               uint32_t (&c)[8], bool& bad) {
  if (left < 8) {  // nothing is held behind the matrix's last value
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e >= left) m[e] = 0.0f;
  }
  float top = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) top = max_magnitude(top, m[e]);
  top = half_warp_max(top);
  float inverse;
  block_scale(top, Level<BITS>::recip, scale, inverse);
  bad = bad || !(top < __uint_as_float(0x7F800000u));
  const uint4 w =
      philox4x32_10((uint32_t)counter, (uint32_t)(counter >> 32), rnd.t_lo, rnd.t_hi, rnd.keys);
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
  }
  if (left < 8) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e >= left) c[e] = 0;
  }
}
// Of n values, those from i on that a group of 8 holds (0 .. 8).
__device__ __forceinline__ int left_of(int64_t i, int64_t n) {
  return (int)(i + 8 <= n ? 8 : (i < n ? n - i : 0));
}

__device__ __forceinline__ double sum_squares(const float (&v)[8]) {
  double s = 0.0;
#pragma unroll
  for (int e = 0; e < 8; ++e) s = fma((double)v[e], (double)v[e], s);
  return s;
}

// Sum over a CTA of T threads in a fixed order; valid in thread 0.
template <int T>
__device__ __forceinline__ double cta_sum(double v) {
  __shared__ double warp_sums[T / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if ((threadIdx.x & 31) == 0) warp_sums[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x < 32) {
    v = threadIdx.x < T / 32 ? warp_sums[threadIdx.x] : 0.0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  }
  return v;
}

// 2^(e0 - t) as two factors (each an fp32 power of two) and 2^t / (|x| + eps),
// 2^(t-1) <= |x| + eps < 2^t, from the partial sums; the same in every CTA.
// A norm below 2^-126 makes X_0 = 0; one that is not finite makes it NaN.
struct NormScale {
  float first, second, factor;
};
__device__ __forceinline__ NormScale scale_of(double sum, float eps, int e0) {
  const double n = sqrt(sum) + (double)eps;
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
  return r;
}
__device__ __forceinline__ NormScale norm_scale(const double* partials, int parts, float eps,
                                                int e0) {
  __shared__ NormScale shared;
  if (threadIdx.x < 32) {
    double s = 0.0;
    for (int i = threadIdx.x; i < parts; i += 32) s += partials[i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    if (threadIdx.x == 0) shared = scale_of(s, eps, e0);
  }
  __syncthreads();
  return shared;
}

}  // namespace
}  // namespace mua

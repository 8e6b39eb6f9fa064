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

// Arithmetic on pairs of fp32 values (packed instructions, each half rounded
// by itself as the scalar one is).
__device__ __forceinline__ uint64_t f2_splat(float x) { return f2_pack(x, x); }
__device__ __forceinline__ uint64_t f2_fma_rn(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// A product that the addition after it may not absorb: a packed multiplication
// and a packed addition, both .rn, come out with one rounding (measured), two
// scalar multiplications and a packed addition with two.
__device__ __forceinline__ uint64_t f2_mul_apart(float a, uint64_t b) {
  return f2_pack(__fmul_rn(a, f2_lo(b)), __fmul_rn(a, f2_hi(b)));
}
__device__ __forceinline__ uint64_t f2_add_rm(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rm.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f2_fma_rm(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rm.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Eight consecutive values of type T from p[i ..], those at or past n as 0.
// CONSTANT: nothing in the launch writes them, so that the read-only path is open.
template <int T, bool CONSTANT = true>
__device__ __forceinline__ void load8(const void* p, int64_t i, int64_t n, bool vec,
                                      uint64_t (&v)[4]) {
  auto load = [](const void* at) {
    if constexpr (CONSTANT) return ld_stream_v4(at);
    uint4 w;
    asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "l"(at) : "memory");
    return w;
  };
  if (vec && i + 8 <= n) {
    if constexpr (T == kBf16) {
      const uint4 w = load(static_cast<const uint16_t*>(p) + i);
      v[0] = f2_pack(bf16_lo(w.x), bf16_hi(w.x));
      v[1] = f2_pack(bf16_lo(w.y), bf16_hi(w.y));
      v[2] = f2_pack(bf16_lo(w.z), bf16_hi(w.z));
      v[3] = f2_pack(bf16_lo(w.w), bf16_hi(w.w));
    } else {
      const float* f = static_cast<const float*>(p) + i;
      const uint4 a = load(f), b = load(f + 4);
      v[0] = f2_pack(__uint_as_float(a.x), __uint_as_float(a.y));
      v[1] = f2_pack(__uint_as_float(a.z), __uint_as_float(a.w));
      v[2] = f2_pack(__uint_as_float(b.x), __uint_as_float(b.y));
      v[3] = f2_pack(__uint_as_float(b.z), __uint_as_float(b.w));
    }
    return;
  }
  float x[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    x[e] = 0.0f;
    if (i + e < n) {
      if constexpr (T == kBf16)
        x[e] = __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i + e] << 16);
      else
        x[e] = static_cast<const float*>(p)[i + e];
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = f2_pack(x[2 * e], x[2 * e + 1]);
}

template <int T>
__device__ __forceinline__ void store8(void* p, int64_t i, int64_t n, bool vec,
                                       const uint64_t (&v)[4]) {
  if (vec && i + 8 <= n) {
    if constexpr (T == kBf16) {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) =
          make_uint4(pack_bf16(f2_lo(v[0]), f2_hi(v[0])), pack_bf16(f2_lo(v[1]), f2_hi(v[1])),
                     pack_bf16(f2_lo(v[2]), f2_hi(v[2])), pack_bf16(f2_lo(v[3]), f2_hi(v[3])));
    } else {
      float4* f = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
      f[0] = make_float4(f2_lo(v[0]), f2_hi(v[0]), f2_lo(v[1]), f2_hi(v[1]));
      f[1] = make_float4(f2_lo(v[2]), f2_hi(v[2]), f2_lo(v[3]), f2_hi(v[3]));
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (i + e < n) {
      const float x = (e & 1) ? f2_hi(v[e >> 1]) : f2_lo(v[e >> 1]);
      if constexpr (T == kBf16)
        static_cast<uint16_t*>(p)[i + e] = __bfloat16_as_ushort(__float2bfloat16_rn(x));
      else
        static_cast<float*>(p)[i + e] = x;
    }
}
// The 8 values in fp16, times two powers of two.
__device__ __forceinline__ uint4 scaled_f16(const uint64_t (&v)[4], float first, float second) {
  const uint64_t a = f2_splat(first), b = f2_splat(second);
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint64_t x = f2_mul_rn(f2_mul_rn(v[e], a), b);
    w[e] = pack_f16(f2_lo(x), f2_hi(x));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Levels of 8 codes as pairs of floats: the biased code in the low mantissa
// bits of 2^23 (exact, without the quarter-rate conversion).
template <int BITS>
__device__ __forceinline__ void unpack8(uint2 w, uint64_t (&q)[4]) {
  const uint64_t bias = f2_splat(-8388608.0f - (BITS == 8 ? 128.0f : 8.0f));
  if constexpr (BITS == 8) {
    const uint32_t v[2] = {w.x ^ 0x80808080u, w.y ^ 0x80808080u};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      q[e] = f2_add_rn(
          f2_pack(__uint_as_float(__byte_perm(v[e >> 1], 0x4B000000u, 0x7650 + 2 * (e & 1))),
                  __uint_as_float(__byte_perm(v[e >> 1], 0x4B000000u, 0x7651 + 2 * (e & 1)))),
          bias);
  } else {
    // Nibbles of the even and odd values, a byte each.
    const uint32_t v = w.x ^ 0x88888888u, even = v & 0x0F0F0F0Fu, odd = (v >> 4) & 0x0F0F0F0Fu;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      q[e] = f2_add_rn(f2_pack(__uint_as_float(__byte_perm(even, 0x4B000000u, 0x7650 + e)),
                               __uint_as_float(__byte_perm(odd, 0x4B000000u, 0x7650 + e))),
                       bias);
  }
}

// A lane's 8 codes at p.
template <int BITS>
__device__ __forceinline__ uint2 load_codes(const uint8_t* p) {
  if constexpr (BITS == 8)
    return *reinterpret_cast<const uint2*>(p);
  else
    return make_uint2(*reinterpret_cast<const uint32_t*>(p), 0u);
}
template <int BITS>
__device__ __forceinline__ uint2 load_codes(const uint8_t* codes, int64_t block, int sub) {
  return load_codes<BITS>(codes + (block * kMuonBlock + 8 * sub) * BITS / 8);
}
template <int BITS>
__device__ __forceinline__ void store_codes(uint8_t* p, const uint32_t (&c)[8]) {
  if constexpr (BITS == 8) {
    const uint32_t a = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040),
                                   0x5410);
    const uint32_t b = __byte_perm(__byte_perm(c[4], c[5], 0x0040), __byte_perm(c[6], c[7], 0x0040),
                                   0x5410);
    *reinterpret_cast<uint2*>(p) = make_uint2(a, b);
  } else {
    // Bytes of the even and of the odd values, merged nibble by nibble.
    const uint32_t even = __byte_perm(__byte_perm(c[0], c[2], 0x0040),
                                      __byte_perm(c[4], c[6], 0x0040), 0x5410);
    const uint32_t odd = __byte_perm(__byte_perm(c[1], c[3], 0x0040),
                                     __byte_perm(c[5], c[7], 0x0040), 0x5410);
    *reinterpret_cast<uint32_t*>(p) = (even & 0x0F0F0F0Fu) | ((odd << 4) & 0xF0F0F0F0u);
  }
}
template <int BITS>
__device__ __forceinline__ void store_codes(uint8_t* codes, int64_t block, int sub,
                                            const uint32_t (&c)[8]) {
  store_codes<BITS>(codes + (block * kMuonBlock + 8 * sub) * BITS / 8, c);
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

// The larger magnitude, NaN if either is; the sign means nothing.
__device__ __forceinline__ float max_magnitude(float a, float b) {
  float r;
  asm("max.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float half_warp_max(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = max_magnitude(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return fabsf(v);
}

// philox4x32_10 of mua_kernels.cuh with each round's two products as one wide
// multiplication each.
__device__ __forceinline__ uint4 philox_wide(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3,
                                             const uint32_t (&keys)[10][2]) {
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t p0 = (uint64_t)0xD2511F53u * c0, p1 = (uint64_t)0xCD9E8D57u * c2;
    c0 = (uint32_t)(p1 >> 32) ^ c1 ^ keys[r][0];
    c1 = (uint32_t)p1;
    c2 = (uint32_t)(p0 >> 32) ^ c3 ^ keys[r][1];
    c3 = (uint32_t)p0;
  }
  return make_uint4(c0, c1, c2, c3);
}

template <int BITS>
struct Level {
  static constexpr float value = BITS == 8 ? 127.0f : 7.0f;
  static constexpr float recip = 1.0f / value;  // rounded to fp32
};

// m' = beta m + g and U of 8 values.
__device__ __forceinline__ void new_momentum(const uint64_t (&q)[4], float scale,
                                             const uint64_t (&g)[4], float beta, int nesterov,
                                             uint64_t (&m)[4], uint64_t (&u)[4]) {
  const uint64_t s2 = f2_splat(scale);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    m[e] = f2_add_rn(f2_mul_apart(beta, f2_mul_rn(q[e], s2)), g[e]);
    u[e] = m[e];
  }
  if (nesterov) {
#pragma unroll
    for (int e = 0; e < 4; ++e) u[e] = f2_add_rn(f2_mul_apart(beta, m[e]), g[e]);
  }
}

// Scale and codes of a block's new momentum, of which this lane holds 8 values,
// `left` (8 or fewer) of them inside the matrix; all lanes of a warp call it.
template <int BITS>
__device__ __forceinline__ void quantize_block(uint64_t (&m)[4], int left, uint64_t counter,
                                               const MuonRandom& rnd, float& scale,
                                               uint32_t (&c)[8], bool& bad) {
  if (left < 8) {  // nothing is held behind the matrix's last value
#pragma unroll
    for (int e = 0; e < 4; ++e)
      m[e] = f2_pack(2 * e < left ? f2_lo(m[e]) : 0.0f, 2 * e + 1 < left ? f2_hi(m[e]) : 0.0f);
  }
  float top = 0.0f;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    top = max_magnitude(max_magnitude(top, f2_lo(m[e])), f2_hi(m[e]));
  top = half_warp_max(top);
  float inverse;
  block_scale(top, Level<BITS>::recip, scale, inverse);
  bad |= !(top < __uint_as_float(0x7F800000u));
  const uint4 w =
      philox_wide((uint32_t)counter, (uint32_t)(counter >> 32), rnd.t_lo, rnd.t_hi, rnd.keys);
  const uint64_t inv2 = f2_splat(inverse), step = f2_splat(1.52587890625e-05f);
  const uint64_t magic = f2_splat(12582784.0f);  // 1.5 2^23 - 128
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t word = chunk_word(w, e);
    const uint64_t y = f2_mul_rn(m[e], inv2);
    const uint64_t clamped =
        f2_pack(fminf(fmaxf(f2_lo(y), -Level<BITS>::value), Level<BITS>::value),
                fminf(fmaxf(f2_hi(y), -Level<BITS>::value), Level<BITS>::value));
    // 2^23 + r for both draws; then floor(y + r / 2^16) by rounding toward -inf:
    // y + 128 + r / 2^16 falls below no integer it passes, then unit spacing.
    const uint64_t r = f2_pack(__uint_as_float(__byte_perm(word, 0x4B000000u, 0x7610)),
                               __uint_as_float(__byte_perm(word, 0x4B000000u, 0x7632)));
    const uint64_t z = f2_add_rm(f2_fma_rm(r, step, clamped), magic);
    c[2 * e] = __float_as_uint(f2_lo(z));
    c[2 * e + 1] = __float_as_uint(f2_hi(z));
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

// Sum of 8 squares: in fp32 (a relative error of 2^-22 at most) where that holds
// it, else in fp64, whose range holds every square.
__device__ __forceinline__ double sum_squares(const uint64_t (&v)[4]) {
  uint64_t t = f2_mul_rn(v[0], v[0]);
#pragma unroll
  for (int e = 1; e < 4; ++e) t = f2_fma_rn(v[e], v[e], t);
  const float f = f2_lo(t) + f2_hi(t);
  if ((f > 1e-20f && f < 1e30f) || (t == 0 && v[0] == 0 && v[1] == 0 && v[2] == 0 && v[3] == 0))
    return (double)f;
  double s = 0.0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    s = fma((double)f2_lo(v[e]), (double)f2_lo(v[e]), s);
    s = fma((double)f2_hi(v[e]), (double)f2_hi(v[e]), s);
  }
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

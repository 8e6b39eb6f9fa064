// Tensor-core, barrier and epilogue pieces shared by the Muon product kernels
// (muon_ns.cu, muon_small.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "muon.cuh"

namespace mua {
namespace {

constexpr uint64_t kDrainNs = 2000000000ull;  // bound on waits for copies and MMAs in flight

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  return t;
}
// One lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(p));
  return p != 0;
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
// Whether the phase is over, without waiting (a try may suspend the thread).
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n"
      " mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// False when the wait ran out, or another role of the CTA has given up. The
// timer is read once in 1024 tries: a read takes longer than most waits. A
// limit of 0 gives up where it would wait.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, uint64_t limit,
                                          volatile uint32_t* stop) {
  if (limit == 0) {
    if (mbar_test(bar, parity)) return true;
    *stop = 1;
    return false;
  }
  uint64_t t0 = 0;
  for (uint32_t n = 1; !mbar_try(bar, parity); ++n) {
    if ((n & 1023u) != 0) continue;
    if (*stop) return false;
    const uint64_t t = now_ns();
    if (t0 == 0) t0 = t;
    if (t - t0 > limit) {
      *stop = 1;
      return false;
    }
  }
  return true;
}
// The same for a converged warp: one answer for all lanes.
__device__ __forceinline__ bool mbar_wait_warp(uint32_t bar, uint32_t parity, uint64_t limit,
                                               volatile uint32_t* stop) {
  if (limit != 0 && __all_sync(0xFFFFFFFFu, mbar_try(bar, parity))) return true;
  const bool ok = mbar_wait(bar, parity, limit, stop);
  return __all_sync(0xFFFFFFFFu, ok);
}
// A wait for work in flight that other roles' giving up does not end.
__device__ __forceinline__ void mbar_drain(uint32_t bar, uint32_t parity) {
  uint64_t t0 = 0;
  for (uint32_t n = 1; !mbar_try(bar, parity); ++n) {
    if ((n & 1023u) != 0) continue;
    const uint64_t t = now_ns();
    if (t0 == 0) t0 = t;
    if (t - t0 > kDrainNs) return;
  }
}
// A 64 x `rows` box into this CTA's shared memory. With CG = 2 the barrier may
// be the pair's other CTA's.
template <int CG>
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x,
                                         int y, int z) {
  if constexpr (CG == 2)
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".cta_group::2 [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}
__device__ __forceinline__ void fence_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
// Orders this thread's acquired view of global memory before its TMA copies.
__device__ __forceinline__ void fence_async_global() {
  asm volatile("fence.proxy.async.global;" ::: "memory");
}
__device__ __forceinline__ uint32_t peer_address(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void mbar_expect_cluster(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(
                   bar),
               "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
               : "memory");
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
// Shared-memory operand descriptor, 128-byte swizzle: 8-row groups of 128-byte
// rows 1024 bytes apart. K-major (rows run along M / N): `lead` is not used.
// M/N-major (rows run along the contraction index, 64 M / N elements each):
// `lead` bytes lie between one 64-element chunk and the next.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, uint32_t lead) {
  return (uint64_t)((addr & 0x3FFFF) >> 4) | ((uint64_t)(lead >> 4) << 16) |
         ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// fp16 operands, fp32 accumulators, M = 128 per CTA.
template <int CG>
__device__ __forceinline__ uint32_t instruction_desc(int n, bool a_mn, bool b_mn) {
  return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(n / 8) << 17) | ((uint32_t)(CG * 128 / 16) << 24);
}
template <int CG>
__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                        bool accumulate) {
  if constexpr (CG == 2)
    asm volatile(
        "{\n .reg .pred p;\n"
        " setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n"
        " setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
}
// The four MMAs of a 64-deep slice: low words of the operands' descriptors, their
// steps, and the high word both share.
template <int CG>
__device__ __forceinline__ void mma_slice(uint32_t d, uint32_t a, uint32_t b, uint32_t high,
                                          uint32_t a_step, uint32_t b_step, uint32_t idesc,
                                          bool accumulate) {
#define MUA_MMA_SLICE(G)                                                                        \
  asm volatile(                                                                                 \
      "{\n .reg .pred p, q;\n .reg .b32 x, y;\n .reg .b64 u, v;\n"                              \
      " setp.ne.b32 p, %7, 0;\n setp.eq.b32 q, 0, 0;\n"                                         \
      " mov.b64 u, {%1, %3};\n mov.b64 v, {%2, %3};\n"                                          \
      " tcgen05.mma.cta_group::" G ".kind::f16 [%0], u, v, %6, p;\n"                            \
      " add.u32 x, %1, %4;\n add.u32 y, %2, %5;\n mov.b64 u, {x, %3};\n mov.b64 v, {y, %3};\n"  \
      " tcgen05.mma.cta_group::" G ".kind::f16 [%0], u, v, %6, q;\n"                            \
      " add.u32 x, x, %4;\n add.u32 y, y, %5;\n mov.b64 u, {x, %3};\n mov.b64 v, {y, %3};\n"    \
      " tcgen05.mma.cta_group::" G ".kind::f16 [%0], u, v, %6, q;\n"                            \
      " add.u32 x, x, %4;\n add.u32 y, y, %5;\n mov.b64 u, {x, %3};\n mov.b64 v, {y, %3};\n"    \
      " tcgen05.mma.cta_group::" G ".kind::f16 [%0], u, v, %6, q;\n}\n" ::"r"(d),               \
      "r"(a), "r"(b), "r"(high), "r"(a_step), "r"(b_step), "r"(idesc), "r"((uint32_t)accumulate) \
      : "memory")
  if constexpr (CG == 2)
    MUA_MMA_SLICE("2");
  else
    MUA_MMA_SLICE("1");
#undef MUA_MMA_SLICE
}
// Arrives on the barrier (of both CTAs of a pair) when the MMAs issued so far are done.
template <int CG>
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  if constexpr (CG == 2)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
        "[%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
  else
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
}
__device__ __forceinline__ void tmem_load16(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_load_wait() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}


__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Output rows of one warp (32, one per lane) x 64 columns from accumulators to
// a swizzled shared tile: the layout of a 128-byte-swizzled TMA store.
__device__ __forceinline__ uint32_t chunk_address(uint32_t tile, int row, int group) {
  return tile + row * 128 + ((group ^ (row & 7)) << 4);
}
__device__ __forceinline__ void st_shared(uint32_t a, uint32_t x, uint32_t y, uint32_t z,
                                          uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}
__device__ __forceinline__ uint4 ld_shared(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

// One value of the last product: the result, or a parameter's update formed in
// fp32 and rounded once.
__device__ __forceinline__ float new_value(const MuonNs& g, float old, float x, float alpha) {
  return g.params ? fmaf(-alpha, x, old * g.decay) : x * alpha;
}
__device__ __forceinline__ float read_one(const MuonNs& g, int64_t at) {
  if (!g.params) return 0.0f;
  if (g.out_type == kF32) return static_cast<const float*>(g.out)[at];
  return __uint_as_float((uint32_t)static_cast<const uint16_t*>(g.out)[at] << 16);
}
__device__ __forceinline__ void write_one(const MuonNs& g, int64_t at, float v) {
  if (g.out_type == kF32)
    static_cast<float*>(g.out)[at] = v;
  else
    static_cast<uint16_t*>(g.out)[at] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
}
// Four consecutive columns of a row, `left` of them inside it.
__device__ __forceinline__ float4 read_four(const MuonNs& g, int64_t at, int left) {
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (!g.params) return v;
  if (g.out_vec && left >= 4) {
    if (g.out_type == kF32) {
      v = *reinterpret_cast<const float4*>(static_cast<const float*>(g.out) + at);
    } else {
      const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(g.out) + at);
      v = make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u),
                      __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u));
    }
    return v;
  }
  if (left > 0) v.x = read_one(g, at);
  if (left > 1) v.y = read_one(g, at + 1);
  if (left > 2) v.z = read_one(g, at + 2);
  if (left > 3) v.w = read_one(g, at + 3);
  return v;
}
__device__ __forceinline__ void write_four(const MuonNs& g, int64_t at, int left, float4 old,
                                           const uint32_t (&x)[4], float alpha) {
  const float v[4] = {new_value(g, old.x, __uint_as_float(x[0]), alpha),
                      new_value(g, old.y, __uint_as_float(x[1]), alpha),
                      new_value(g, old.z, __uint_as_float(x[2]), alpha),
                      new_value(g, old.w, __uint_as_float(x[3]), alpha)};
  if (g.out_vec && left >= 4) {
    if (g.out_type == kF32)
      *reinterpret_cast<float4*>(static_cast<float*>(g.out) + at) =
          make_float4(v[0], v[1], v[2], v[3]);
    else
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(g.out) + at) =
          make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < left) write_one(g, at + e, v[e]);
}

}  // namespace
}  // namespace mua

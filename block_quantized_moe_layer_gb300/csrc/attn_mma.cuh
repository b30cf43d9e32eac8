// attn_mma.cuh -- dequantisation into tensor-core operands, warp-level MMAs and
// bounded waits shared by the attention kernels.
#pragma once
#include "attn.cuh"

namespace moe {
namespace attn {

__device__ __forceinline__ uint32_t h2_fma(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t h2_mul(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t bf2_fma(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t bf2_mul(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Keys as bf16.  A scale byte b in both halves, shifted left by 4, is a bf16
// of value d 2^-112 (the same fraction bits; subnormals included), so one
// product gives d.  A nibble q under the exponent of 128 is 128 + q, and
// (128 + q) d - 136 d = (q - 8) d: one fma, exact (136 d has 8 bits).
struct KeyScale {
  uint32_t d, c;
};
__device__ __forceinline__ KeyScale key_scale(uint32_t bytes /* 0x00bb00bb */) {
  const uint32_t t = bytes << 4;
  return KeyScale{bf2_mul(t, 0x77807780u /* 2^112 */), bf2_mul(t, 0xFB08FB08u /* -136 2^112 */)};
}
// The 8 channels of a word as 4 pairs of neighbours.
__device__ __forceinline__ void key_pairs(uint32_t w, KeyScale s, uint32_t* o) {
  o[0] = bf2_fma((w & 0x000F000Fu) | 0x43004300u, s.d, s.c);
  o[1] = bf2_fma(((w >> 4) & 0x000F000Fu) | 0x43004300u, s.d, s.c);
  o[2] = bf2_fma(((w >> 8) & 0x000F000Fu) | 0x43004300u, s.d, s.c);
  o[3] = bf2_fma(((w >> 12) & 0x000F000Fu) | 0x43004300u, s.d, s.c);
}

// Values over 16 as fp16 (the output is multiplied by 16 at the end): a scale
// byte shifted left by 7 is d, times 2^-4.  A nibble q in bits 0..3 under the
// exponent of 1024 is 1024 + q, in bits 4..7 under that of 64 it is 64 + q;
// 1032 d/16 <= 57792 and has 11 bits, 72 d/16 has 7: every step is exact.
struct ValueScale {
  uint32_t d, c0, c1;
};
__device__ __forceinline__ ValueScale value_scale(uint32_t bytes /* 0x00bb00aa */) {
  const uint32_t d = h2_mul(bytes << 7, 0x2C002C00u /* 2^-4 */);
  return ValueScale{d, h2_mul(d, 0xE408E408u /* -1032 */), h2_mul(d, 0xD480D480u /* -72 */)};
}
// Nibbles 0..3 of both halves of u as four pairs.
__device__ __forceinline__ void value_quads(uint32_t u, ValueScale s, uint32_t& o0, uint32_t& o1, uint32_t& o2, uint32_t& o3) {
  const uint32_t v = u >> 8;
  o0 = h2_fma((u & 0x000F000Fu) | 0x64006400u, s.d, s.c0);
  o1 = h2_fma((u & 0x00F000F0u) | 0x54005400u, s.d, s.c1);
  o2 = h2_fma((v & 0x000F000Fu) | 0x64006400u, s.d, s.c0);
  o3 = h2_fma((v & 0x00F000F0u) | 0x54005400u, s.d, s.c1);
}
constexpr float kValueUnscale = 16.f;

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Channels 4 c .. 4 c + 3 of an output row, and its logarithm.
__device__ __forceinline__ void store_joined(const AttnParams& p, int64_t o, int c, int D, float4 x, float lt, float mx) {
  const float inv = mx > -INFINITY ? kValueUnscale / lt : 0.f;
  const __nv_bfloat162 u = __floats2bfloat162_rn(x.x * inv, x.y * inv), w = __floats2bfloat162_rn(x.z * inv, x.w * inv);
  uint2 r;
  r.x = *reinterpret_cast<const uint32_t*>(&u);
  r.y = *reinterpret_cast<const uint32_t*>(&w);
  *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + o * D + 4 * c) = r;
  if (p.lse && c == 0) p.lse[o] = mx > -INFINITY ? (mx + log2f(lt)) * 0.69314718055994531f : -INFINITY;
}

// A wait on an mbarrier phase that gives up after the call's limit (the
// status word then says where) or once another thread of the block has.
__device__ __forceinline__ bool wait_inline(uint64_t* bar, uint32_t parity, volatile int* abort, int* status, uint64_t limit, int site) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (*abort) return false;
    if (globaltimer_ns() - t0 > limit) {
      *abort = 1;
      if (!(atomicOr(status, kTimeout) & kTimeout)) status[1] = site;
      return false;
    }
  }
  return true;
}
// The same as a call, where many waits share the code (a call keeps few
// registers: not for threads that hold a row of scores).
static __device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile int* abort, int* status, uint64_t limit,
                                       int site) {
  return wait_inline(bar, parity, abort, status, limit, site);
}
// SPINS: tests before the suspending wait, whose sleeper takes a few hundred
// cycles to resume.  For the one thread that issues MMAs, not for the many
// that compute: their spinning takes the issue slots of the others.
template <int SPINS = 0>
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort, int* status, uint64_t limit,
                                         int site) {
  if constexpr (SPINS == 0) {
    if (mbar_try_wait(bar, parity)) return true;
  } else {
#pragma unroll 1
    for (int i = 0; i < SPINS; ++i)
      if (mbar_test_wait(bar, parity)) return true;
  }
  return wait_slow(bar, parity, abort, status, limit, site);
}

}  // namespace attn
}  // namespace moe

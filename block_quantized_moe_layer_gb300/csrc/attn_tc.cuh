// attn_tc.cuh -- what the tcgen05 attention kernels share.
#pragma once
#include "attn_mma.cuh"
#include "tc.cuh"

namespace moe {
namespace attn {

// The softmax's reference moves only when the maximum passes it by more than
// this (log2 units): a weight of 2^8 is harmless in fp16 and fp32.
constexpr float kLazy = 8.f;

// D[tmem] (+)= A[smem] B[smem]^T
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 32 lanes x N columns of 32 bits.
template <int N>
__device__ __forceinline__ void st_cols(uint32_t taddr, const uint32_t (&v)[N]) {
  if constexpr (N == 8) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  } else {
    static_assert(N == 16, "8 or 16 columns");
    tc::st_32x32b_x16(taddr, v);
  }
}

// 16 columns of a row's accumulator, to the output or to a part.
__device__ __forceinline__ void store_out16(const AttnParams& p, const uint32_t (&o)[16], float l, float inv, bool has_row,
                                            int64_t part, int64_t orow, int c, int D) {
  float v[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) v[e] = l > 0.f ? __uint_as_float(o[e]) * inv : 0.f;
  if (!has_row) return;
  if (p.n_split > 1) {
    float4* d = reinterpret_cast<float4*>(p.part_o + part * D + c);
#pragma unroll
    for (int e = 0; e < 4; ++e) d[e] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
  } else {
    uint32_t w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const __nv_bfloat162 h2 = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
      w[e] = *reinterpret_cast<const uint32_t*>(&h2);
    }
    uint4* d = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + orow * D + c);
    d[0] = make_uint4(w[0], w[1], w[2], w[3]);
    d[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

}  // namespace attn
}  // namespace moe

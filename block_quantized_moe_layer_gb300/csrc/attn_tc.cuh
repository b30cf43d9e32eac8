// attn_tc.cuh -- what the tcgen05 attention kernels share.
#pragma once
#include "attn_mma.cuh"
#include "tc.cuh"

#include <type_traits>

namespace moe {
namespace attn {

// The softmax's reference moves only when the maximum passes it by more than
// this (log2 units): a weight of 2^8 is harmless in fp16 and fp32.
constexpr float kLazy = 8.f;

// One thread of a converged warp, the same each time.  MMAs are issued under
// it, in a warp whose number came by a shuffle: the compiler then knows that
// one thread of a uniform warp runs them, and an MMA takes 9 cycles to issue.
// Under `lane == 0` it takes 45, and 70 beside busy warps, which is more than
// the MMA itself.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}
__device__ __forceinline__ int uniform_warp() { return __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0); }

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

// The softmax of a block's tiles: thread (share, row) takes QC keys of each
// tile's NQ QC, reads its scores from tensor memory (columns 0 or 128 on, by
// the tile's parity), and stores the weights as fp16 over them.  m is the
// row's reference (log2 units), the same in its NQ threads, l this thread's
// share of the row's sum.  vis(j, bits): bit c of `bits` tells whether key c of
// the thread's is seen; false where all are.
//   The threads of a row exchange their maxima through shared memory,
// behind a barrier of the row group's NQ warps; a warp whose wait gave up keeps
// coming to that barrier, so that the others never wait for it in vain.
template <int QC>
using KeyBits = std::conditional_t<QC == 64, uint64_t, uint32_t>;

template <int D, int QC, int NQ, class Vis>
__device__ __forceinline__ bool softmax_tiles(const AttnParams& p, int n_tiles, uint32_t tl, int quarter, int row, int rows, float* ex,
                                              uint64_t* sfull, uint64_t* pfull, uint64_t* odone, volatile int* abort, float& m,
                                              float& l, Vis vis) {
  const int lane = threadIdx.x & 31, group = (threadIdx.x >> 5) & 3;
  bool ok = true;
  for (int j = 0; j < n_tiles; ++j) {
    const uint32_t tile = tl + 128 * (j & 1);
    float x[QC];
    if (ok) {
      ok = wait_bar(&sfull[j & 1], (uint32_t)((j >> 1) & 1), abort, p.status, p.timeout_ns, 30);
      ok = __all_sync(0xffffffffu, ok);
    }
    if (ok) {
      tc::fence_after();
      uint32_t sv[QC / 16][16];
#pragma unroll
      for (int c = 0; c < QC / 16; ++c) tc::ld_32x32b_x16(tile + QC * quarter + 16 * c, sv[c]);
      tc::wait_ld();
#pragma unroll
      for (int c = 0; c < QC; ++c) x[c] = __uint_as_float(sv[c >> 4][c & 15]);
      KeyBits<QC> bits;
      if (vis(j, bits)) {
#pragma unroll
        for (int c = 0; c < QC; ++c)
          if (!((bits >> c) & 1)) x[c] = -INFINITY;
      }
      float a = fmaxf(x[0], x[1]), b = fmaxf(x[2], x[3]);
#pragma unroll
      for (int c = 4; c < QC; c += 4) {
        a = fmaxf(a, fmaxf(x[c], x[c + 1]));
        b = fmaxf(b, fmaxf(x[c + 2], x[c + 3]));
      }
      ex[((j & 1) * NQ + quarter) * rows + row] = fmaxf(a, b);
    }
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(NQ * 32) : "memory");
    if (!ok) continue;
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < NQ; ++i) mx = fmaxf(mx, ex[((j & 1) * NQ + i) * rows + row]);
    mx *= p.scale_log2;
    const bool move = mx > m + kLazy;  // (also the first visible keys: m = -inf)
    if (__any_sync(0xffffffffu, move)) {
      const float f = move ? (m == -INFINITY ? 0.f : exp2_approx(m - mx)) : 1.f;
      if (move) m = mx;
      l *= f;
      if (j > 0) {
        ok = wait_bar(&odone[(j - 1) & 1], (uint32_t)(((j - 1) >> 1) & 1), abort, p.status, p.timeout_ns, 32);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) continue;
        tc::fence_after();
#pragma unroll 1
        for (int c = quarter * (D / NQ); c < (quarter + 1) * (D / NQ); c += 16) {
          uint32_t o[16];
          tc::ld_32x32b_x16(tl + 256 + c, o);
          tc::wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
          tc::st_32x32b_x16(tl + 256 + c, o);
        }
      }
    }
    const float ref = m == -INFINITY ? 0.f : m;
    uint32_t pk[QC / 2];
    float l0 = 0.f, l1 = 0.f;
#pragma unroll
    for (int c = 0; c < QC / 2; ++c) {
      const float u = exp2_approx(fmaf(x[2 * c], p.scale_log2, -ref));
      const float v = exp2_approx(fmaf(x[2 * c + 1], p.scale_log2, -ref));
      l0 += u;
      l1 += v;
      pk[c] = pack_h2(u, v);
    }
    l += l0 + l1;
    st_cols<QC / 2>(tile + QC / 2 * quarter, pk);
    tc::wait_st();
    tc::fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&pfull[j & 1]);
  }
  if (ok) {
    ok = wait_bar(&odone[(n_tiles - 1) & 1], (uint32_t)(((n_tiles - 1) >> 1) & 1), abort, p.status, p.timeout_ns, 33);
    ok = __all_sync(0xffffffffu, ok);
    tc::fence_after();
  }
  return ok;
}

// The bits of QC keys from k0 on that lie in [lo, hi).
template <int QC>
__device__ __forceinline__ KeyBits<QC> key_bits(int k0, int lo, int hi) {
  using B = KeyBits<QC>;
  constexpr int kBits = 8 * sizeof(B);
  const int a = lo - k0, e = hi - k0;
  B v = e >= kBits ? ~B(0) : (e <= 0 ? B(0) : (B(1) << e) - 1);
  v &= a <= 0 ? ~B(0) : (a >= kBits ? B(0) : ~((B(1) << a) - 1));
  return v;
}

// The same of a tree node's row: prefix keys [lo, p0), then the nodes of `word`.
template <int QC>
__device__ __forceinline__ KeyBits<QC> tree_bits(int k0, int lo, int p0, uint64_t word) {
  const int a = k0 - p0;  // node of the first key
  const uint64_t nodes = a >= 0 ? (a < 64 ? word >> a : 0) : (a > -QC ? word << -a : 0);
  return key_bits<QC>(k0, lo, p0) | (KeyBits<QC>)nodes;
}

// ---- pairs of blocks (clusters of two)
__device__ __forceinline__ void pair_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ void pair_alloc(uint32_t* slot) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(slot)) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_dealloc(uint32_t taddr) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(taddr) : "memory");
}
// Both blocks' rows times both halves of B, into each block's tensor memory.
__device__ __forceinline__ void pair_mma_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void pair_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrives at the barrier of each block in `blocks` (a bit each) once the MMAs issued so far are complete.
__device__ __forceinline__ void pair_commit(uint64_t* bar, uint16_t blocks) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                   smem_u32(bar)),
               "h"(blocks)
               : "memory");
}
// Arrives at the first block's barrier.  No memory that the other block reads
// or writes by loads and stores stands behind such an arrival: weights in
// tensor memory are complete (wait::st), images have landed, and only MMAs read
// either.  So no cluster-wide release, which waits some 1600 cycles for the
// thread's own loads and stores (382 against 268 us).
__device__ __forceinline__ void arrive_first(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .b32 a;\n\t"
      "mapa.shared::cluster.u32 a, %0, 0;\n\t"
      "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [a];\n\t}" ::"r"(smem_u32(bar))
      : "memory");
}
// The same behind stores to shared memory that the pair's MMAs read: with a release
// (of a thread that has none of its own on their way: tree_kernel 37.3 us without, 37.8 so).
__device__ __forceinline__ void arrive_first_release(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .b32 a;\n\t"
      "mapa.shared::cluster.u32 a, %0, 0;\n\t"
      "mbarrier.arrive.release.cluster.shared::cluster.b64 _, [a];\n\t}" ::"r"(smem_u32(bar))
      : "memory");
}

}  // namespace attn
}  // namespace moe

// attn_check.cu -- attention over the 4-bit paged cache in fp32 (the check
// mode, act_dtype MOE_ACT_F32), on the CUDA cores.
//
//   o = sum_j softmax_j(scale q.k_j) v_j over the visible keys j, in one pass:
// a running maximum m, sum l and accumulator o per warp, rescaled by
// 2^(m_old - m_new) when the maximum grows, joined over the warps at the end.
// Everything is fp32; the cache's values enter exactly.
//
// One block a (query token, query head); its warps take chunks of 32 keys in
// turn.  For the scores a lane owns a key and reads its D/2 bytes (the query
// waits in shared memory, read as broadcasts); for the output a lane owns 8
// channels (a 32-bit word) of every key, or of every 2nd or 4th at 128 and 64
// channels.  It is for verification: it re-reads a
// key/value head for each of its query heads and is bound by the
// dequantisation's instructions, not by HBM.  Measured: 2 sequences of 3
// tokens over 999 keys, 16 heads of 64, in 10.9 us (one block a row, 32 chunks
// of keys: a chain of loads, not a rate).
#include "attn.cuh"

namespace moe {
namespace attn {
namespace {

// Warps of a block: of a tree's, whose rows see few keys more than the prefix, twice
// as many (2 trees of 7 nodes over 999 keys, 16 heads of 64: 19.4 and 13.6 us).
template <bool TREE>
constexpr int kCheckWarps = TREE ? 16 : 8;

template <int D, bool TREE>
__global__ void __launch_bounds__(kCheckWarps<TREE> * 32) check_kernel(const __grid_constant__ AttnParams p) {
  constexpr int kWarps = kCheckWarps<TREE>;
  constexpr int kWords = D / 8;  // words of a row: lanes that own channels
  constexpr int kPar = kWords <= 16 ? 32 / kWords : 1, kBatch = 8;
  __shared__ float sq[D];
  __shared__ float so[kWarps][D];
  __shared__ float sm[kWarps], sl[kWarps];
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x / p.hq, h = blockIdx.x % p.hq, b = blockIdx.y;
  const Seq s = load_seq(p, b);
  if (t >= s.nq) return;
  const int tok = s.start + t;
  for (int i = threadIdx.x; i < D; i += blockDim.x)
    sq[i] = static_cast<const float*>(p.q)[tok * p.q_tok + h * p.q_head + i] * p.scale_log2;
  __syncthreads();
  const int p0 = s.len - s.nq, pos = p0 + t;  // its place in the cache: the last key that it may see
  TreeRow tree{0, 0};
  if constexpr (TREE) {
    const TreeWords w = tree_words(p, s);
    const uint64_t w0 = __shfl_sync(0xffffffffu, w.word[0], t & 31), w1 = __shfl_sync(0xffffffffu, w.word[1], t & 31);
    tree = tree_row(p, p0, t < 32 ? w0 : w1);
  }
  const int lo = TREE ? tree.lo : key_lo(p, pos);
  const int kvh = h / p.g;
  const int word = kPar > 1 ? lane % kWords : lane, sub = kPar > 1 ? lane / kWords : 0;
  float m = -INFINITY, l = 0.f, o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  // chunks of 32 keys, aligned so that a chunk lies in at most two pages (16-token pages)
  for (int c = (lo & ~31) + 32 * warp; c <= pos; c += 32 * kWarps) {
    const int j = c + lane;
    const bool in = TREE ? j <= pos && tree_sees(tree, p0, j) : j >= lo && j <= pos;
    const int pg = in ? load_page(p, b, j >> p.pshift) : -1;
    const uint8_t* base = pg < 0 ? nullptr : p.pages + pg * p.page_bytes + kvh * p.head_bytes;
    const int at = j & (p.P - 1);
    float sc = -INFINITY;
    if (base) {
      const uint32_t* kw = reinterpret_cast<const uint32_t*>(base + at * (D / 2));
      const uint8_t* ks = base + p.P * (D / 2) + at * (D / 16);
      sc = 0.f;
#pragma unroll 8
      for (int w = 0; w < kWords; ++w) {
        const uint32_t u = kw[w];
        float a = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          a = fmaf((float)((int)((u >> (4 * e)) & 15) - 8), sq[8 * w + 2 * e], a);
          a = fmaf((float)((int)((u >> (4 * e + 16)) & 15) - 8), sq[8 * w + 2 * e + 1], a);
        }
        sc = fmaf(a, scale_value(ks[w >> 1]), sc);
      }
    }
    if (!__any_sync(0xffffffffu, base != nullptr)) continue;
    const float mn = fmaxf(m, fmaxf(warp_max(sc), kSeen));
    const float f = exp2f(m - mn);  // 0 at the first keys
    const float pr = exp2f(sc - mn);
    m = mn;
    l = l * f + pr;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] *= f;
    // kPar keys at a time, a lane 8 channels of one; their loads go out together
#pragma unroll
    for (int i0 = 0; i0 < 32; i0 += kPar * kBatch) {
      uint32_t u[kBatch];
      float pd[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int i = i0 + kPar * k + sub;
        const float pi = __shfl_sync(0xffffffffu, pr, i);
        const uint64_t bi = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(base), i);
        u[k] = 0;
        pd[k] = 0.f;
        if (bi && word < kWords) {
          const uint8_t* vb = reinterpret_cast<const uint8_t*>(bi) + p.head_bytes / 2;
          const int ai = (c + i) & (p.P - 1);
          u[k] = *reinterpret_cast<const uint32_t*>(vb + ai * (D / 2) + 4 * word);
          pd[k] = pi * scale_value(vb[p.P * (D / 2) + ai * (D / 16) + (word >> 1)]);
        }
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          o[2 * e] = fmaf((float)((int)((u[k] >> (4 * e)) & 15) - 8), pd[k], o[2 * e]);
          o[2 * e + 1] = fmaf((float)((int)((u[k] >> (4 * e + 16)) & 15) - 8), pd[k], o[2 * e + 1]);
        }
    }
  }
  // the keys of a lane group apart
#pragma unroll
  for (int x = kWords; x < 32 && kPar > 1; x <<= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] += __shfl_xor_sync(0xffffffffu, o[i], x);
#pragma unroll
  for (int x = 16; x; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
  if (lane == 0) sm[warp] = m, sl[warp] = l;
  if (lane < kWords)
#pragma unroll
    for (int i = 0; i < 8; ++i) so[warp][8 * lane + i] = o[i];
  __syncthreads();
  float mx = -INFINITY;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, sm[w]);
  float lt = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) lt += sm[w] == -INFINITY ? 0.f : sl[w] * exp2f(sm[w] - mx);
  for (int i = threadIdx.x; i < D; i += blockDim.x) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += sm[w] == -INFINITY ? 0.f : so[w][i] * exp2f(sm[w] - mx);
    // a row that sees no key is 0
    static_cast<float*>(p.out)[((int64_t)tok * p.hq + h) * D + i] = mx > -INFINITY ? v / lt : 0.f;
  }
  if (p.lse && threadIdx.x == 0)
    p.lse[(int64_t)tok * p.hq + h] = mx > -INFINITY ? (mx + log2f(lt)) * 0.69314718055994531f : -INFINITY;
}

}  // namespace

template <bool TREE>
static cudaError_t check_launch_any(const AttnParams& p, cudaStream_t st) {
  const dim3 grid((unsigned)(p.max_q * p.hq), p.n_seqs);
  switch (p.D) {
    case 64: return launch_pdl(check_kernel<64, TREE>, grid, kCheckWarps<TREE> * 32, 0, st, p);
    case 128: return launch_pdl(check_kernel<128, TREE>, grid, kCheckWarps<TREE> * 32, 0, st, p);
    case 192: return launch_pdl(check_kernel<192, TREE>, grid, kCheckWarps<TREE> * 32, 0, st, p);
    default: return launch_pdl(check_kernel<256, TREE>, grid, kCheckWarps<TREE> * 32, 0, st, p);
  }
}
cudaError_t check_launch(const AttnParams& p, cudaStream_t st) {
  return p.parents ? check_launch_any<true>(p, st) : check_launch_any<false>(p, st);
}

}  // namespace attn
}  // namespace moe

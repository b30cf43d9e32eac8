// attn_verify.cu -- attention of verify batches over the 4-bit paged cache: up
// to 64 rows (query token, query head) of a key/value head a block, on the
// tcgen05 tensor cores, the cache read once and dequantised in the block.
//
// At 4 tokens of 16 query heads a key/value head the cache's bytes and the
// products are nearly in balance (227 flops a byte), so warp-level MMAs
// (attn_small.cu) run out at 0.38 of the memory's rate before anything else;
// and an expansion to 16 bits in memory (attn_prompt.cu) would move 8 times the
// bytes.  Here a block's roles run beside each other, tile by tile of KT keys:
//   warps 0-15   index % 4 < 2: softmax, a quarter of the tile's keys each (the
//                MMA's M is 128, of which 64 rows are used: the tensor memory
//                lanes that these warps read); the others: keys, from the
//                pages by way of registers (a tile ahead) to a bf16 operand
//                image in shared memory (exact);
//   warps 16-23  values to an fp16 image (exact);
//   warp 24      issues S = Q K^T and O += P V.
// Both images are [channels/8][keys][8 channels]: for the keys that is K-major
// (the contraction runs over channels), for the values MN-major, so neither is
// transposed.  There are two of each.  Keys are split over blocks and joined.
//
// Bound: shared memory.  A tile of 128 keys at D = 192 moves 240 KB through it
// (both images in and out, the queries), 1900 cycles at 128 bytes a cycle,
// beside 1540 of MMAs, 1180 of the memory's time and 1500 of instructions.
// Measured on the way, cycles a tile: 4300 with the raw pages copied to shared
// memory first (another 54 KB) and single images, whatever the order of the
// roles; values transposed by hand into cores 144 bytes apart made O += P V
// 1850 instead of 800.  Now 4 tokens of 64/4 heads of 192 over 32765 keys take
// 21.7 us with the join where L2 holds the cache (28 MB; 6.7 times the MMAs'
// time at their peak rate, 5.1 times the cache's from HBM), 26.3 where it does
// not: 7 tiles a block, some 3300 cycles each, about half of it, and its start,
// end and join; the tensor pipe is active 26%; the warps wait for page loads,
// then for each other.
//   For trees of drafted tokens (TREE) a row sees the tokens before the tree and
// the nodes of one word (attn.cuh), by which the last tiles are masked.  32 trees
// of 12 nodes (48 rows) over up to 8192 keys, 32/8 heads of 128: 107 us, 256
// blocks, the longest sequences first; a tile takes some 1900 cycles, of which
// shared memory is busy 1400 and the tensor pipe 840.
#include <cooperative_groups.h>

#include "attn_tc.cuh"

namespace moe {
namespace attn {

cudaError_t join_launch(const AttnParams& p, int rows_per_tile, int n_rt, int whole, cudaStream_t st);

namespace {

constexpr int kRowsV = 64;
constexpr int kJoinV = 8;  // parts that a cluster joins at most
constexpr int kWarpsV = 25;
constexpr int kMmaWarp = 24;
constexpr int kThreadsV = kWarpsV * 32;

template <int D>
struct VerifyPlan {
  static constexpr int KT = D == 256 ? 64 : 128;  // keys of a tile
  static constexpr int kImage = D / 8 * KT * 16;
  // queries [D/8][64 rows][8]: the MMA's rows 64..127 run into the next slab
  // (and past the last one into the keys' image): read, never used
  static constexpr int kQ = 0;
  static constexpr int kK = kQ + D / 8 * kRowsV * 16;
  static constexpr int kV = kK + 2 * kImage;
  static constexpr int kMax = kV + 2 * kImage;                 // float [2][4][64] (the sums and references take as much)
  // [8 tiles][16]: a byte for each 8 keys that exist (written up to 4 tiles before the softmax reads it)
  static constexpr int kHere = kMax + 2 * 4 * kRowsV * 4;
  static constexpr int kBars = kHere + 8 * 16;
  static constexpr int kNumBars = 8 + 2;
  static constexpr int kMisc = kBars + kNumBars * 8;           // tensor memory slot, abort
  static constexpr int kTotal = kMisc + 16 + 128;
  static_assert(kTotal <= 232448, "shared memory plan");
  static constexpr int kPitch = D * 4 + 16;  // of an output row on its way out, over the images
  static_assert(kRowsV * kPitch <= kMax, "the output fits the images' room");
};

template <int D, bool TREE>
__global__ void __launch_bounds__(kThreadsV, 1) verify_kernel(const __grid_constant__ AttnParams p, int n_rt, int chunk) {
  using L = VerifyPlan<D>;
  constexpr int KT = L::KT, QC = KT / 4;  // keys of a softmax thread
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  float* smax = reinterpret_cast<float*>(sm + L::kMax);
  uint8_t* here = sm + L::kHere;
  uint64_t* kfull = reinterpret_cast<uint64_t*>(sm + L::kBars);  // [2] key image written
  uint64_t* sfull = kfull + 2;                                    // [2] scores ready (key image free)
  uint64_t* pvfull = sfull + 2;                                   // [2] value image and weights written
  uint64_t* odone = pvfull + 2;                                   // [2] output product done (value image free)
  uint64_t* qfull = odone + 2;                                    // queries written
  uint64_t* fin = qfull + 1;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + L::kMisc);
  volatile int* abort = reinterpret_cast<volatile int*>(sm + L::kMisc + 4);
  volatile int never = 0;
  const int tid = threadIdx.x, warp = uniform_warp(), lane = tid & 31;
  griddep_launch_dependents();
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&kfull[i], 8 + p.miss);
      mbar_init(&sfull[i], 1);
      mbar_init(&pvfull[i], 16);
      mbar_init(&odone[i], 1);
    }
    mbar_init(qfull, 8);
    mbar_init(fin, 1);
    *abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) tc::alloc_512(tslot);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tbase = *tslot;
  griddep_wait();

  const int split = blockIdx.x, b = TREE && p.by_length ? seq_by_length(p, blockIdx.z) : blockIdx.z;
  const int kvh = blockIdx.y / n_rt, rt = blockIdx.y % n_rt;
  const Seq s = load_seq(p, b);
  const int row0 = rt * kRowsV, n_rows = max(0, min(kRowsV, s.nq * p.g - row0));
  const int p0 = s.len - s.nq;
  // (of a tree all rows see what lies before it, and a node's place in the cache bounds its position)
  const int pos_min = TREE ? p0 - 1 : p0 + row0 / p.g, pos_max = p0 + (row0 + max(n_rows, 1) - 1) / p.g;
  const int lo = key_lo(p, max(0, TREE ? p0 : pos_min)), hi = pos_max + 1, lo_max = key_lo(p, pos_max);
  const int tile_a = lo / KT + split * chunk;
  const int n_tiles = hi > lo && n_rows > 0 ? max(0, min(tile_a + chunk, (hi + KT - 1) / KT) - tile_a) : 0;

  const bool soft = warp < 16 && (warp & 3) < 2;
  const int row = (warp & 1) * 32 + lane, quarter = warp >> 2;  // of the softmax threads
  int tq = 0, hq = 0, hi_r = 0, lo_r = 0;
  const bool has_row = soft && row < n_rows;
  if (has_row) {
    tq = (row0 + row) / p.g;
    hq = kvh * p.g + (row0 + row) % p.g;
    hi_r = TREE ? p0 : p0 + tq + 1;
    lo_r = key_lo(p, p0 + tq);
  }
  uint64_t word = 0;  // a tree row's nodes
  if constexpr (TREE) {
    if (soft && n_rows > 0) {
      const TreeWords w = tree_words(p, s);
      const uint64_t w0 = __shfl_sync(0xffffffffu, w.word[0], tq & 31), w1 = __shfl_sync(0xffffffffu, w.word[1], tq & 31);
      if (has_row) {
        const TreeRow r = tree_row(p, p0, tq < 32 ? w0 : w1);
        word = r.word;
        lo_r = r.lo;
      }
    }
  }

  float m = -INFINITY, l = 0.f;
  bool seen = false;  // this thread's keys: one of them by the row
  if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMAs
    if (n_tiles > 0 && elect_one()) {
      constexpr uint32_t kIdescS = tc::idesc_f16(128, KT) | (1u << 7) | (1u << 10);  // bf16 operands
      constexpr uint32_t kIdescO = tc::idesc_f16(128, D) | (1u << 16);  // fp16, the values MN-major
      const uint64_t qd = tc::smem_desc(smem_u32(sm + L::kQ), kRowsV * 16, 128);
      const uint64_t kd = tc::smem_desc(smem_u32(sm + L::kK), KT * 16, 128);
      // MN-major: 8 keys of a core matrix 128 bytes on, 8 channels a slab on
      const uint64_t vd = tc::smem_desc(smem_u32(sm + L::kV), 128, KT * 16);
      bool ok = true;
      auto scores = [&](int j) {
        const int i = j & 1;
        ok = wait_bar<64>(&kfull[i], (uint32_t)((j >> 1) & 1), abort, p.status, p.timeout_ns, 23);
        if (!ok) return;
        tc::fence_after();
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          mma_ss(tbase + 128 * i, qd + k * (2 * kRowsV * 16 / 16), kd + i * (L::kImage / 16) + k * (2 * KT * 16 / 16), kIdescS,
                 k > 0);
        tc::commit(&sfull[i]);
      };
      ok = wait_bar<64>(qfull, 0, abort, p.status, p.timeout_ns, 34);
      if (ok) scores(0);
      for (int j = 0; j < n_tiles && ok; ++j) {
        const int i = j & 1;
        if (j + 1 < n_tiles) scores(j + 1);
        ok = ok && wait_bar<64>(&pvfull[i], (uint32_t)((j >> 1) & 1), abort, p.status, p.timeout_ns, 24);
        if (!ok) break;
        tc::fence_after();
#pragma unroll
        for (int k = 0; k < KT / 16; ++k)
          tc::mma_ts(tbase + 256, tbase + 128 * i + 8 * k, vd + i * (L::kImage / 16) + k * (2 * 128 / 16), kIdescO, j > 0 || k > 0);
        tc::commit(&odone[i]);
      }
      // all MMAs issued are complete before the block frees anything
      tc::commit(fin);
      wait_bar<64>(fin, 0, &never, p.status, p.timeout_ns, 26);
    }
  } else if (!soft && n_tiles > 0) {
    // ------------------------------------------------------------ dequantisation
    const bool values = warp >= 16;
    const int dw = values ? warp - 16 : (warp >> 2) * 2 + (warp & 1);  // 0..7
    const int codes = p.P * (D / 2);
    uint64_t* image_full = values ? pvfull : kfull;
    uint64_t* image_free = values ? odone : sfull;
    uint8_t* image = sm + (values ? L::kV : L::kK);
    // a warp takes KT/8 neighbouring keys, which lie in one page; a lane a key
    // and every (32 / keys)-th piece of 32 channels (one 16-byte load; 8-byte
    // loads held the load units up for a third of a tile).  Each 8 lanes store
    // 8 keys, so they meet all banks.
    constexpr int kKeys = KT / 8, kStep = 32 / kKeys, kUnits = D / 32 / kStep;
    const int kk = lane % kKeys, piece = lane / kKeys;
    // the next tile's codes and scales are asked for once a tile is written,
    // their page number a tile before that (a second set of registers, to ask
    // a whole tile ahead, was slower: 24.6 against 23 us at 32765 keys)
    uint4 code[kUnits];
    uint32_t scale[kUnits];
    int page = -1;
    auto page_seen = [&](int j) {  // (a page that no row here sees is not looked at: it may have been given back)
      const int key = (tile_a + j) * KT + kKeys * dw;
      return j < n_tiles && key < hi && (key | (p.P - 1)) >= lo;
    };
    auto look_up = [&](int j) { page = page_seen(j) ? page_entry(p, b, ((tile_a + j) * KT + kKeys * dw) >> p.pshift) : -1; };
    auto fetch = [&](int j) {  // this lane's codes and scales of tile j: 0 for a key past the end or on an absent page
      const int key = (tile_a + j) * KT + kKeys * dw, at = (key & (p.P - 1)) + kk, pg = checked_page(p, page, page_seen(j));
      const uint8_t* src = p.pages + pg * p.page_bytes + (int64_t)kvh * p.head_bytes + (values ? p.head_bytes / 2 : 0);
      const bool has = pg >= 0 && key + kk < s.len;
      const uint8_t* sc = src + at * (D / 2) + 16 * piece;
      const uint8_t* ss = src + codes + at * (D / 16) + 2 * piece;
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        code[u] = make_uint4(0, 0, 0, 0);
        scale[u] = 0;
        if (has) {
          code[u] = __ldcg(reinterpret_cast<const uint4*>(sc + 16 * kStep * u));
          scale[u] = __ldcg(reinterpret_cast<const uint16_t*>(ss + 2 * kStep * u));
        }
      }
      if (!values && lane < kKeys / 8 && j < n_tiles) here[(j & 7) * 16 + kKeys / 8 * dw + lane] = pg >= 0;
    };
    look_up(0);
    fetch(0);
    look_up(1);
    // Heads of 128 leave the registers to ask for the next tile before this one is
    // written: 32 trees of 48 rows over up to 8192 keys 134 us and 126 so (64: 66.8
    // and 67.6; of 192 a second set of registers was slower).  Not for the shorter
    // tails of chains: 8 sequences of 32 rows over 8000 keys 48.5 us, and 49.3 so.
    constexpr bool kAhead = TREE && D == 128;
    for (int j = 0; j < n_tiles; ++j) {
      const int i = j & 1;
      uint4 code_j[kUnits];
      uint32_t scale_j[kUnits];
#pragma unroll
      for (int u = 0; u < kUnits; ++u) code_j[u] = code[u], scale_j[u] = scale[u];
      if constexpr (kAhead) {
        fetch(j + 1);
        look_up(j + 2);
      }
      bool ok = true;
      if (j > 1) ok = wait_bar(&image_free[i], (uint32_t)((j >> 1) - 1) & 1, abort, p.status, p.timeout_ns, 28);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      uint4* o = reinterpret_cast<uint4*>(image + i * L::kImage) + 4 * piece * KT + kKeys * dw + kk;
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        const uint32_t w[4] = {code_j[u].x, code_j[u].y, code_j[u].z, code_j[u].w};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t sb = __byte_perm(scale_j[u], 0, h ? 0x4141 : 0x4040);
          uint32_t x[8];
          if (values) {
            const ValueScale d = value_scale(sb);
            value_quads(w[2 * h], d, x[0], x[1], x[2], x[3]);
            value_quads(w[2 * h + 1], d, x[4], x[5], x[6], x[7]);
          } else {
            const KeyScale d = key_scale(sb);
            key_pairs(w[2 * h], d, x);
            key_pairs(w[2 * h + 1], d, x + 4);
          }
          o[(4 * kStep * u + 2 * h) * KT] = make_uint4(x[0], x[1], x[2], x[3]);
          o[(4 * kStep * u + 2 * h + 1) * KT] = make_uint4(x[4], x[5], x[6], x[7]);
        }
      }
      tc::fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&image_full[i]);
      if constexpr (!kAhead) {
        fetch(j + 1);
        look_up(j + 2);
      }
    }
  } else if (soft && n_tiles > 0) {
    // ------------------------------------------------------------ softmax
    {
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + (s.start + tq) * p.q_tok + hq * p.q_head;
#pragma unroll
      for (int c = quarter * (D / 32); c < (quarter + 1) * (D / 32); ++c) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (has_row) v = *reinterpret_cast<const uint4*>(q + 8 * c);
        *reinterpret_cast<uint4*>(sm + L::kQ + (c * kRowsV + row) * 16) = v;
      }
    }
    tc::fence_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(qfull);
    const uint32_t tl = tbase + ((uint32_t)(warp & 3) << 21);  // this warp's 32 lanes
    softmax_tiles<D, QC, 4>(p, n_tiles, tl, quarter, row, kRowsV, smax, sfull, pvfull, odone, abort, m, l, [&](int j, uint32_t& bits) {
      const int c0 = (tile_a + j) * KT;
      // the existing 8-key groups of this quarter, a byte each
      uint32_t mask;
      if constexpr (QC == 32) mask = *reinterpret_cast<const volatile uint32_t*>(here + (j & 7) * 16 + 4 * quarter);
      else mask = *reinterpret_cast<const volatile uint16_t*>(here + (j & 7) * 16 + 2 * quarter);
      if (c0 + KT <= pos_min + 1 && c0 >= lo_max && mask == (0x01010101u >> (32 - QC))) {
        seen = true;
        return false;
      }
      if constexpr (TREE) bits = tree_bits<QC>(c0 + QC * quarter, lo_r, hi_r, word);
      else bits = key_bits<QC>(c0 + QC * quarter, lo_r, hi_r);
      bits &= mask * 0xFFu;  // (bytes of 1 to bytes of 0xFF)
      seen |= bits != 0;
      return true;
    });
  }
  // the quarters' sums; the outputs go through shared memory (the images'
  // room), since a thread's row is D apart from its neighbour's: stored from
  // the accumulator's layout they took 5 us
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (soft) {
    smax[quarter * kRowsV + row] = l;
    smax[(4 + quarter) * kRowsV + row] = seen ? fmaxf(m, kSeen) : m;
  }
  if (soft && n_tiles > 0) {
    const uint32_t tl = tbase + ((uint32_t)(warp & 3) << 21);
#pragma unroll 1
    for (int c = quarter * (D / 4); c < (quarter + 1) * (D / 4); c += 16) {
      uint32_t o[16];
      tc::ld_32x32b_x16(tl + 256 + c, o);
      tc::wait_ld();
      uint4* d = reinterpret_cast<uint4*>(sm + row * L::kPitch + c * 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) d[e] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
    }
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == kMmaWarp) tc::dealloc_512(tbase);
  if constexpr (TREE) {
    if (p.clustered) {
      // the blocks' parts, a share of the outputs each (a part without keys has no output)
      __shared__ float2 block_ml[kRowsV];
      if (tid < kRowsV) {
        float mr = smax[4 * kRowsV + tid], lt = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) mr = fmaxf(mr, smax[(4 + k) * kRowsV + tid]), lt += smax[k * kRowsV + tid];
        block_ml[tid] = make_float2(mr, lt);
      }
      auto cl = cooperative_groups::this_cluster();
      cl.sync();
      for (int i = split * kThreadsV + tid; i < n_rows * (D / 4); i += p.n_split * kThreadsV) {
        const int r = i / (D / 4), c = i % (D / 4);
        float2 a[kJoinV];
        float mr = -INFINITY, lt = 0.f;
#pragma unroll
        for (int k = 0; k < kJoinV; ++k) {
          a[k] = k < p.n_split ? *cl.map_shared_rank(&block_ml[r], k) : make_float2(-INFINITY, 0.f);
          mr = fmaxf(mr, a[k].x);
        }
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kJoinV; ++k) {
          if (a[k].x == -INFINITY) continue;
          const float4 v = *cl.map_shared_rank(reinterpret_cast<float4*>(sm + r * L::kPitch + c * 16), k);
          const float f = exp2_approx(a[k].x - mr);
          lt = fmaf(a[k].y, f, lt);
          x.x = fmaf(v.x, f, x.x);
          x.y = fmaf(v.y, f, x.y);
          x.z = fmaf(v.z, f, x.z);
          x.w = fmaf(v.w, f, x.w);
        }
        store_joined(p, (int64_t)(s.start + (row0 + r) / p.g) * p.hq + kvh * p.g + (row0 + r) % p.g, c, D, x, lt, mr);
      }
      cl.sync();  // (a block stays until the others have read its part)
      return;
    }
  }
  const int64_t part0 = ((int64_t)(b * p.hk * n_rt + blockIdx.y) * p.n_split + split) * kRowsV;
  for (int i = tid; i < n_rows * (D / 4); i += kThreadsV) {
    const int r = i / (D / 4), c = i % (D / 4);
    float lt = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) lt += smax[k * kRowsV + r];
    float mr = smax[4 * kRowsV + r];
#pragma unroll
    for (int k = 5; k < 8; ++k) mr = fmaxf(mr, smax[k * kRowsV + r]);
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (mr > -INFINITY) v = *reinterpret_cast<const float4*>(sm + r * L::kPitch + c * 16);
    if (p.n_split > 1) {
      *reinterpret_cast<float4*>(p.part_o + (part0 + r) * D + 4 * c) = v;
      if (c == 0) p.part_ml[part0 + r] = make_float2(mr, lt);
    } else {
      store_joined(p, (int64_t)(s.start + (row0 + r) / p.g) * p.hq + kvh * p.g + (row0 + r) % p.g, c, D, v, lt, mr);
    }
  }
}

template <int D>
cudaError_t verify_launch_d(AttnParams p, int num_sms, size_t part_rows, cudaStream_t st) {
  constexpr int KT = VerifyPlan<D>::KT;
  const int n_rt = (p.max_q * p.g + kRowsV - 1) / kRowsV;
  const int64_t base = (int64_t)p.hk * n_rt * p.n_seqs;
  int64_t span = std::max(p.max_len, 1);  // keys a row tile can see: the window's, or all
  if (p.window > 0) span = std::min<int64_t>(span, (int64_t)p.window + p.max_q + KT);
  const int tiles = (int)((span + KT - 1) / KT);
  // one block a multiprocessor; at least two tiles a block
  int64_t want = std::max<int64_t>(1, num_sms / base);
  want = std::min<int64_t>(std::min<int64_t>(want, kMaxSplit), std::max<int64_t>(1, (int64_t)(part_rows / kRowsV) / base));
  const int chunk = (int)std::max<int64_t>(std::min(tiles, 2), (tiles + want - 1) / want);
  p.n_split = (tiles + chunk - 1) / chunk;
  // (measured for trees alone, of which 32 of 12 nodes over 4096..8192 tokens take 107 us so, 125 in their order)
  p.by_length = p.parents && base > num_sms && p.n_seqs <= kSortedSeqs && p.window == 0;
  // A tree's few parts are a cluster's blocks where all fit the GPU at once (a block
  // a multiprocessor, and a cluster's in one of its groups): no second
  // launch (48 rows over 640 keys, 32/8 heads of 128, 11.0 us and 10.0 so; 4 sequences
  // 12.8 and 10.2)
  p.clustered = p.parents && p.n_split > 1 && p.n_split <= kJoinV && base * p.n_split <= num_sms * 2 / 3;
  if (p.clustered)
    return launch_pdl_cluster(verify_kernel<D, true>, p.n_split, dim3(p.n_split, (unsigned)(p.hk * n_rt), p.n_seqs), kThreadsV,
                              VerifyPlan<D>::kTotal, st, p, n_rt, chunk);
  cudaError_t e = launch_pdl(p.parents ? verify_kernel<D, true> : verify_kernel<D, false>, dim3(p.n_split, (unsigned)(p.hk * n_rt), p.n_seqs), kThreadsV,
                             VerifyPlan<D>::kTotal, st, p, n_rt, chunk);
  if (e != cudaSuccess || p.n_split == 1) return e;
  return join_launch(p, kRowsV, n_rt, -1, st);
}

template <int D>
cudaError_t verify_configure_d() {
  cudaError_t e = cudaFuncSetAttribute(verify_kernel<D, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, VerifyPlan<D>::kTotal);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(verify_kernel<D, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, VerifyPlan<D>::kTotal);
  return e;
}

}  // namespace

cudaError_t verify_configure(int D) {
  switch (D) {
    case 64: return verify_configure_d<64>();
    case 128: return verify_configure_d<128>();
    case 192: return verify_configure_d<192>();
    default: return verify_configure_d<256>();
  }
}

cudaError_t verify_launch(const AttnParams& p, int num_sms, size_t part_rows, cudaStream_t st) {
  switch (p.D) {
    case 64: return verify_launch_d<64>(p, num_sms, part_rows, st);
    case 128: return verify_launch_d<128>(p, num_sms, part_rows, st);
    case 192: return verify_launch_d<192>(p, num_sms, part_rows, st);
    default: return verify_launch_d<256>(p, num_sms, part_rows, st);
  }
}

}  // namespace attn
}  // namespace moe

// attn_tree.cu -- attention of a tree of drafted tokens with many rows over the
// 4-bit paged cache, on the tcgen05 tensor cores.
//
// A pair of blocks (a cluster on two neighbouring multiprocessors) owns 256 rows
// (tree node, query head of one key/value head), 128 a block, and walks over the
// visible 128-key tiles j:
//   S_j = Q K_j^T   (bf16, M = 256, N = 128, both operands in shared memory)
//   P_j = 2^(scale S_j - m), rounded to fp16 in tensor memory
//   O  += P_j V_j   (fp16, P from tensor memory, N = D)
// The keys and values are dequantised inside the pair, beside the MMAs and the
// softmax: each block makes the images of half a tile (64 keys; D/2 channels of
// the 128 values), which the pair's MMAs read together.  So a tile is dequantised
// once for 256 rows: the kernel of verify batches (attn_verify.cu) does it for
// each 64, and is bound by it; the prompt kernel's expansion in memory writes and
// reads 8 times the cache's bytes, which only many row tiles repay.
//   warps 0-7    softmax, a thread half of a row's 128 scores;
//   warps 8-11   keys, from the pages by way of registers (a tile ahead) to a
//                bf16 image (exact); 12-15 values to an fp16 image (exact);
//   warp 16, 17  issue S and O (the second block's: pass on that its images are written).
// Images are [channels/8][keys][8 channels], two of each: K-major for the keys,
// MN-major for the values, so neither is transposed.
//   A node sees the tokens before the tree, and of the tree its ancestors, the
// bits of one word (attn.cuh): tiles that end before the tree have no mask but
// the window's.
// TMEM columns: S at 0 and 128 (P over it), O at 256.
//
// Measured: 16 nodes of 64/4 heads of 192 over 32765 tokens (256 rows) 38 us with
// the join, 0.68 PFLOP/s; 8 trees of 64 nodes over up to 8000 tokens 151 us, 0.90
// PFLOP/s.  A tile takes 2900 cycles, of which the MMAs need 1540 and the memory
// 130.  Bound: the softmax's chain (scores to registers 600, the row's maximum 500,
// exponentials 1000, weights to tensor memory 250, the next scores 300), beside
// dequantising warps that are busy two thirds of the time.  Not better: two groups
// of softmax warps in turn, which read the scores twice (3100), four threads a row
// (3300), weights beside the output so that the next scores come sooner (2950),
// a quarter of the weights while the row's maximum is exchanged (3150), all of
// them, made again where the reference moves (3080: registers, both).  (18 warps
// leave a thread 96 registers, 52 bytes of them spilled; 16 would leave 128.)
#include "attn_tc.cuh"

namespace moe {
namespace attn {

// Joins the parts of split rows (attn_small.cu).
cudaError_t join_launch(const AttnParams& p, int rows_per_tile, int n_rt, int whole, cudaStream_t st);

namespace {

constexpr int kRowsT = 128;  // of a block
constexpr int kPairRowsT = 2 * kRowsT;
constexpr int kTileT = 128;  // keys
constexpr int kSoftWarpsT = 8, kValueWarp = 12, kScoreWarp = 16, kOutWarp = 17;
constexpr int kThreadsT = 18 * 32;

template <int D>
struct TreePlan {
  static constexpr int kImage = kTileT / 2 * D * 2;  // a block's half of an operand image
  static constexpr int kQ = 0;
  static constexpr int kK = kRowsT * D * 2;
  static constexpr int kV = kK + 2 * kImage;
  static constexpr int kMax = kV + 2 * kImage;        // float [4][128]
  static constexpr int kHere = kMax + 4 * kRowsT * 4;  // [8 tiles][16]: a byte for each 8 keys that exist
  static constexpr int kWords = kHere + 8 * 16;       // the nodes' words of ancestors
  static constexpr int kBars = kWords + kTreeNodes * 8;
  static constexpr int kMisc = kBars + 11 * 8;  // tensor memory slot, abort
  static constexpr int kUsed = kMisc + 16 + 128;
  static constexpr int kPitch = D * 4 + 16;  // of an output row on its way out
  static_assert(kRowsT * kPitch <= kMax, "outputs fit below the maxima");
  // one block a multiprocessor (a pair never waits for tensor memory that another pair holds half of)
  static constexpr int kTotal = kUsed > 117 * 1024 ? kUsed : 117 * 1024;
  static_assert(kTotal <= 232448, "shared memory plan");
};

// Two at once.
__device__ __forceinline__ uint64_t two(uint32_t a, uint32_t b) { return (uint64_t)a | ((uint64_t)b << 32); }
__device__ __forceinline__ uint64_t fma_two(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add_two(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max_of(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// The softmax of the pair's tiles: thread (half, row) takes 64 keys of each, and
// stores their weights as fp16.  m is the row's reference, the same in its two
// threads, l this thread's share of the row's sum.  vis(j, bits): the keys seen,
// false where all are.  The threads of a row exchange their maxima through shared
// memory, behind a barrier of their two warps; a warp whose wait gave up keeps
// coming to it, so that the other never waits in vain.
//   No wait for a product skips a phase of its barrier, which two products apart
// share: S(j) was issued after the end of PV(j - 2).
template <int D, class Vis>
__device__ __forceinline__ void tree_softmax(const AttnParams& p, int n_tiles, uint32_t tl, int half, int row, float* ex, uint64_t* sfull,
                                             uint64_t* pfull, uint64_t* odone, volatile int* abort, float& m, float& l, Vis vis) {
  const int lane = threadIdx.x & 31, group = (threadIdx.x >> 5) & 3;
  bool ok = true;
  for (int j = 0; j < n_tiles; ++j) {
    const uint32_t tile = tl + 128 * (j & 1);
    uint32_t x[4][16];
    if (ok) {
      ok = wait_bar(&sfull[j & 1], (uint32_t)((j >> 1) & 1), abort, p.status, p.timeout_ns, 40);
      ok = __all_sync(0xffffffffu, ok);
    }
    if (ok) {
      tc::fence_after();
#pragma unroll
      for (int c = 0; c < 4; ++c) tc::ld_32x32b_x16(tile + 64 * half + 16 * c, x[c]);
      tc::wait_ld();
      uint64_t bits;
      if (vis(j, bits)) {
#pragma unroll
        for (int c = 0; c < 64; ++c)
          if (!((bits >> c) & 1)) x[c >> 4][c & 15] = 0xFF800000u;  // -inf
      }
      float a[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int c = 0; c < 64; c += 8)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          a[i] = max_of(a[i], __uint_as_float(x[c >> 4][(c & 15) + i]), __uint_as_float(x[c >> 4][(c & 15) + 4 + i]));
      ex[((j & 1) * 2 + half) * kRowsT + row] = fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3]));
    }
    asm volatile("bar.sync %0, 64;" ::"r"(1 + group) : "memory");
    if (!ok) continue;
    const float mx = fmaxf(ex[(j & 1) * 2 * kRowsT + row], ex[((j & 1) * 2 + 1) * kRowsT + row]) * p.scale_log2;
    const bool move = mx > m + kLazy;  // (also the first visible keys: m = -inf)
    if (__any_sync(0xffffffffu, move)) {
      const float f = move ? (m == -INFINITY ? 0.f : exp2_approx(m - mx)) : 1.f;
      if (move) m = mx;
      l *= f;
      if (j > 0) {
        ok = wait_bar(&odone[(j - 1) & 1], (uint32_t)(((j - 1) >> 1) & 1), abort, p.status, p.timeout_ns, 41);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) continue;
        tc::fence_after();
#pragma unroll 1
        for (int c = half * (D / 2); c < (half + 1) * (D / 2); c += 16) {
          uint32_t o[16];
          tc::ld_32x32b_x16(tl + 256 + c, o);
          tc::wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
          tc::st_32x32b_x16(tl + 256 + c, o);
        }
      }
    }
    const uint32_t base = __float_as_uint(m == -INFINITY ? 0.f : -m), scale = __float_as_uint(p.scale_log2);
    const uint32_t weights = tile + 32 * half;
    uint64_t sum[2] = {0, 0};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t pk[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const uint64_t y = fma_two(two(x[2 * h + (e >> 3)][(2 * e) & 15], x[2 * h + (e >> 3)][(2 * e + 1) & 15]), two(scale, scale), two(base, base));
        const float u = exp2_approx(__uint_as_float((uint32_t)y)), v = exp2_approx(__uint_as_float((uint32_t)(y >> 32)));
        sum[e & 1] = add_two(sum[e & 1], two(__float_as_uint(u), __float_as_uint(v)));
        pk[e] = pack_h2(u, v);
      }
      tc::st_32x32b_x16(weights + 16 * h, pk);
    }
    sum[0] = add_two(sum[0], sum[1]);
    l += __uint_as_float((uint32_t)sum[0]) + __uint_as_float((uint32_t)(sum[0] >> 32));
    tc::wait_st();
    tc::fence_before();
    __syncwarp();
    if (lane == 0) arrive_first(&pfull[j & 1]);
  }
  ok = ok && wait_bar(&odone[(n_tiles - 1) & 1], (uint32_t)(((n_tiles - 1) >> 1) & 1), abort, p.status, p.timeout_ns, 42);
}

// Bytes of 0 and 1 to bytes of 0 and 0xFF.
__device__ __forceinline__ uint64_t spread(uint64_t e) { return (e << 8) - e; }

template <int D>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreadsT, 1)
    tree_kernel(const __grid_constant__ AttnParams p, int n_rt, int whole, int chunk) {
  using L = TreePlan<D>;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  float* smax = reinterpret_cast<float*>(sm + L::kMax);
  uint8_t* here = sm + L::kHere;
  uint64_t* words = reinterpret_cast<uint64_t*>(sm + L::kWords);
  uint64_t* kfull = reinterpret_cast<uint64_t*>(sm + L::kBars);  // [2] key images written (the first block's: both blocks')
  uint64_t* vfull = kfull + 2;                                    // [2] value images written
  uint64_t* sfull = vfull + 2;                                    // [2] scores ready (key images free)
  uint64_t* pfull = sfull + 2;                                    // [2] weights stored (the first block's are used)
  uint64_t* odone = pfull + 2;                                    // [2] output product done (value images free)
  uint64_t* fin = odone + 2;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + L::kMisc);
  volatile int* abort = reinterpret_cast<volatile int*>(sm + L::kMisc + 4);
  volatile int never = 0;
  const int tid = threadIdx.x, warp = uniform_warp(), lane = tid & 31;
  const int rank = (int)blockIdx.x & 1, pair = (int)blockIdx.x >> 1;  // (a cluster is two neighbours)
  const bool first_block = rank == 0;
  griddep_launch_dependents();
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&kfull[i], (first_block ? 5 : 4) + p.miss);  // (the first block's: its own warps, and word of the other's)
      mbar_init(&vfull[i], (first_block ? 5 : 4) + p.miss);
      mbar_init(&sfull[i], 1);
      mbar_init(&pfull[i], 2 * 8);
      mbar_init(&odone[i], 1);
    }
    mbar_init(fin, 2);
    *abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  griddep_wait();

  // the first `whole` pairs take a row tile each, those with the most nodes
  // first; the others p.n_split parts of one
  const bool split_tile = pair >= whole;
  const int tile_i = split_tile ? whole + (pair - whole) / p.n_split : pair;
  const int split = split_tile ? (pair - whole) % p.n_split : 0;
  const int rt = n_rt - 1 - tile_i / (p.hk * p.n_seqs), bi = tile_i % (p.hk * p.n_seqs) / p.hk, kvh = tile_i % p.hk;
  const int b = p.by_length ? seq_by_length(p, bi) : bi;
  const bool parts = split_tile && p.n_split > 1;
  const Seq s = load_seq(p, b);
  const int pair_row0 = rt * kPairRowsT, pair_rows = min(kPairRowsT, s.nq * p.g - pair_row0);
  if (pair_rows <= 0) return;
  const int row0 = pair_row0 + rank * kRowsT, n_rows = min(kRowsT, s.nq * p.g - row0);  // (may be none in the second block)
  const int p0 = s.len - s.nq;
  // keys of the pair's rows: all see what lies before the tree, and a node's place in the cache bounds its position
  const int pos_max = p0 + (pair_row0 + pair_rows - 1) / p.g;
  const int lo = key_lo(p, max(0, p0)), hi = pos_max + 1, lo_max = key_lo(p, pos_max);
  const int tile_a = lo / kTileT + split * chunk;
  const int n_tiles = hi > lo ? max(0, min(split_tile ? tile_a + chunk : 0x7fffffff, (hi + kTileT - 1) / kTileT) - tile_a) : 0;

  // ---- the dequantising warps' first loads, on their way before anything else
  const bool values = warp >= kValueWarp;
  const int dw = warp & 3;
  const int codes = p.P * (D / 2);
  uint64_t* image_full = values ? vfull : kfull;
  uint64_t* image_free = values ? odone : sfull;
  uint8_t* image = sm + (values ? L::kV : L::kK);
  // A key warp takes 16 of the block's 64 keys, a lane a key and every other
  // piece of 32 channels; a value warp 32 of the 128 keys, a lane a key and the
  // block's half of the channels: D/64 pieces either way, one 16-byte load each.
  // Each 8 lanes store 8 neighbouring keys, so they meet all banks.
  constexpr int kUnits = D / 64;
  const int slab = values ? kTileT : kTileT / 2;                             // keys of an image
  const int at_key = values ? 32 * dw + lane : 16 * dw + (lane & 15);        // in the image
  const int tile_key = values ? at_key : rank * (kTileT / 2) + at_key;       // in the tile
  const int piece0 = values ? rank * kUnits : lane >> 4, step = values ? 1 : 2;
  const int image_piece0 = values ? 0 : lane >> 4;
  uint4 code[kUnits];
  uint32_t scale[kUnits];
  int page = -1, other = -1;
  auto entry_of = [&](int key, bool seen) { return seen ? page_entry(p, b, key >> p.pshift) : -1; };
  // (a page that no row here sees is not looked at: it may have been given back)
  auto is_seen = [&](int j, int key) { return j < n_tiles && key < hi && (key | (p.P - 1)) >= lo; };
  // the 16 keys whose existence this key warp's lanes 0 and 1 note for the softmax
  const int noted = 32 * dw + 16 * (lane & 1);
  auto look_up = [&](int j) {
    const int c0 = (tile_a + j) * kTileT;
    page = entry_of(c0 + tile_key, is_seen(j, c0 + tile_key));
    if (!values && lane < 2) other = entry_of(c0 + noted, is_seen(j, c0 + noted));
  };
  auto fetch = [&](int j) {  // this lane's codes and scales of tile j: 0 for a key past the end or on an absent page
    const int c0 = (tile_a + j) * kTileT, key = c0 + tile_key, at = key & (p.P - 1);
    const int pg = checked_page(p, page, is_seen(j, key));
    const uint8_t* src = p.pages + pg * p.page_bytes + (int64_t)kvh * p.head_bytes + (values ? p.head_bytes / 2 : 0);
    const bool has = pg >= 0 && key < s.len;
    const uint8_t* sc = src + at * (D / 2) + 16 * piece0;
    const uint8_t* ss = src + codes + at * (D / 16) + 2 * piece0;
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      code[u] = make_uint4(0, 0, 0, 0);
      scale[u] = 0;
      if (has) {
        code[u] = __ldcg(reinterpret_cast<const uint4*>(sc + 16 * step * u));
        scale[u] = __ldcg(reinterpret_cast<const uint16_t*>(ss + 2 * step * u));
      }
    }
    if (!values && lane < 2 && j < n_tiles) {
      const bool there = checked_page(p, other, is_seen(j, c0 + noted)) >= 0;
      *reinterpret_cast<uint16_t*>(here + (j & 7) * 16 + 4 * dw + 2 * lane) = there ? 0x0101 : 0;
    }
  };
  if (warp >= kSoftWarpsT && warp < kScoreWarp && n_tiles > 0) {
    look_up(0);
    fetch(0);
    look_up(1);
  }

  if (warp == kScoreWarp) pair_alloc(tslot);
  if (warp == kOutWarp) {
    const TreeWords w = tree_words(p, s);
    words[lane] = w.word[0];
    words[lane + 32] = w.word[1];
  }
  const int half = warp >> 2, row = (warp & 3) * 32 + lane;  // of the softmax threads
  const bool has_row = warp < kSoftWarpsT && row < n_rows;
  const int tq = has_row ? (row0 + row) / p.g : 0, hq = has_row ? kvh * p.g + (row0 + row) % p.g : 0;
  // queries: a warp takes 8 rows and 4 of their pieces of 8 channels at a time
  if (warp < kSoftWarpsT && n_tiles > 0) {
    constexpr int kSteps = kRowsT / 8 / kSoftWarpsT;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int at = row0 + 8 * (kSteps * warp + i) + (lane & 7);
      const bool has = at < row0 + n_rows;
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q);
      if (has) q += (s.start + at / p.g) * p.q_tok + (kvh * p.g + at % p.g) * p.q_head;
      uint4 v[D / 32];
#pragma unroll
      for (int c = 0; c < D / 32; ++c)
        v[c] = has ? *reinterpret_cast<const uint4*>(q + 32 * c + 8 * (lane >> 3)) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int c = 0; c < D / 32; ++c)
        *reinterpret_cast<uint4*>(sm + L::kQ + ((4 * c + (lane >> 3)) * kRowsT + 8 * (kSteps * warp + i) + (lane & 7)) * 16) = v[c];
    }
    tc::fence_async_smem();
  }
  tc::fence_before();
  pair_sync();  // both blocks' barriers, queries and words are there
  tc::fence_after();
  const uint32_t tbase = *tslot;

  float m = -INFINITY, l = 0.f;
  if (warp < kSoftWarpsT) {
    if (n_tiles > 0) {
      // ------------------------------------------------------------ softmax
      const uint32_t tl = tbase + ((uint32_t)(warp & 3) << 21);  // this warp's 32 lanes
      const TreeRow tr = has_row ? tree_row(p, p0, words[tq]) : TreeRow{0, p0};
      bool seen = false;  // of this thread's keys one by the row
      tree_softmax<D>(p, n_tiles, tl, half, row, smax, sfull, pfull, odone, abort, m, l, [&](int j, uint64_t& bits) {
        const int c0 = (tile_a + j) * kTileT;
        const uint64_t e = *reinterpret_cast<const volatile uint64_t*>(here + (j & 7) * 16 + 8 * half);  // a byte for each 8 keys
        if (c0 + kTileT <= p0 && c0 >= lo_max && e == 0x0101010101010101ull) {
          seen = true;
          return false;
        }
        bits = tree_bits<64>(c0 + 64 * half, tr.lo, p0, tr.word) & spread(e);
        seen |= bits != 0;
        return true;
      });
      if (seen) m = fmaxf(m, kSeen);
    }
  } else if (warp < kScoreWarp) {
    // ------------------------------------------------------------ dequantisation
    if (n_tiles > 0) {
      for (int j = 0; j < n_tiles; ++j) {
        const int i = j & 1;
        bool ok = true;
        if (j > 1) ok = wait_bar(&image_free[i], (uint32_t)((j >> 1) - 1) & 1, abort, p.status, p.timeout_ns, 45);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        uint4* o = reinterpret_cast<uint4*>(image + i * L::kImage) + 4 * image_piece0 * slab + at_key;
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
          const uint32_t w[4] = {code[u].x, code[u].y, code[u].z, code[u].w};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t sb = __byte_perm(scale[u], 0, h ? 0x4141 : 0x4040);
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
            o[(4 * step * u + 2 * h) * slab] = make_uint4(x[0], x[1], x[2], x[3]);
            o[(4 * step * u + 2 * h + 1) * slab] = make_uint4(x[4], x[5], x[6], x[7]);
          }
        }
        tc::fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&image_full[i]);
        fetch(j + 1);
        look_up(j + 2);
      }
    }
  } else if (warp == kScoreWarp || warp == kOutWarp) {
    // ------------------------------------------------------------ MMAs: a thread for the scores, one for the products
    const bool v = warp == kOutWarp;
    uint64_t* full = v ? vfull : kfull;
    if (n_tiles > 0 && !first_block && elect_one()) {  // the other block's: its images are written
      bool ok = true;
      for (int j = 0; j < n_tiles && ok; ++j) {
        ok = wait_bar<64>(&full[j & 1], (uint32_t)((j >> 1) & 1), abort, p.status, p.timeout_ns, 46);
        if (ok) arrive_first_release(&full[j & 1]);
      }
    }
    if (n_tiles > 0 && first_block && elect_one()) {
      constexpr uint32_t kIdescS = tc::idesc_f16(kPairRowsT, kTileT) | (1u << 7) | (1u << 10);  // bf16 operands
      constexpr uint32_t kIdescO = tc::idesc_f16(kPairRowsT, D) | (1u << 16);                   // fp16, the values MN-major
      const uint64_t qd = tc::smem_desc(smem_u32(sm + L::kQ), kRowsT * 16, 128);
      const uint64_t kd = tc::smem_desc(smem_u32(sm + L::kK), kTileT / 2 * 16, 128);
      // MN-major: 8 keys of a core matrix 128 bytes on, 8 channels a slab on
      const uint64_t vd = tc::smem_desc(smem_u32(sm + L::kV), 128, kTileT * 16);
      bool ok = true;
      for (int j = 0; j < n_tiles; ++j) {
        const int i = j & 1;
        ok = wait_bar<64>(&full[i], (uint32_t)((j >> 1) & 1), abort, p.status, p.timeout_ns, 47);
        if (!v) {
          // the scores' columns are free: the weights over them are multiplied
          if (j >= 2) ok = ok && wait_bar<64>(&odone[i], (uint32_t)(((j - 2) >> 1) & 1), abort, p.status, p.timeout_ns, 48);
          if (!ok) break;
          tc::fence_after();
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            pair_mma_ss(tbase + 128 * i, qd + k * (2 * kRowsT * 16 / 16), kd + i * (L::kImage / 16) + k * (2 * (kTileT / 2) * 16 / 16), kIdescS,
                        k > 0);
          pair_commit(&sfull[i], 3);
        } else {
          ok = ok && wait_bar<64>(&pfull[i], (uint32_t)((j >> 1) & 1), abort, p.status, p.timeout_ns, 49);
          if (!ok) break;
          tc::fence_after();
#pragma unroll
          for (int k = 0; k < kTileT / 16; ++k)
            pair_mma_ts(tbase + 256, tbase + 128 * i + 8 * k, vd + i * (L::kImage / 16) + k * (2 * 128 / 16), kIdescO, j > 0 || k > 0);
          pair_commit(&odone[i], 3);
        }
      }
      // all MMAs issued are complete before the pair frees anything
      pair_commit(fin, 1);
      wait_bar<64>(fin, 0, &never, p.status, p.timeout_ns, 50);
    }
  }
  // the halves' sums, once no MMA reads either block
  __syncwarp();
  pair_sync();
  tc::fence_after();
  if (warp < kSoftWarpsT) {
    smax[half * kRowsT + row] = m;
    smax[(2 + half) * kRowsT + row] = l;
  }
  __syncthreads();
  if (warp < kSoftWarpsT) {
    m = fmaxf(m, smax[(half ^ 1) * kRowsT + row]);  // (they differ where one half alone has seen keys, of scores -inf)
    l += smax[(2 + (half ^ 1)) * kRowsT + row];
    const uint32_t tl = tbase + ((uint32_t)(warp & 3) << 21);
    const float inv = parts ? 1.f : kValueUnscale / l;  // (rows that see no key: not used)
    // the outputs go through shared memory, where queries and images were
#pragma unroll 2
    for (int c = half * (D / 2); c < (half + 1) * (D / 2); c += 16) {
      uint32_t o[16];
      __syncwarp();
      if (n_tiles > 0) {
        tc::ld_32x32b_x16(tl + 256 + c, o);
        tc::wait_ld();
      }
      float4* d = reinterpret_cast<float4*>(sm + row * L::kPitch + c * 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float4 v = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]), __uint_as_float(o[4 * e + 2]),
                                     __uint_as_float(o[4 * e + 3]));
        d[e] = m > -INFINITY ? make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
    if (has_row && half == 0) {
      const int64_t orow = parts ? ((int64_t)(tile_i - whole) * p.n_split + split) * kPairRowsT + rank * kRowsT + row
                                 : (int64_t)(s.start + tq) * p.hq + hq;
      *reinterpret_cast<int64_t*>(sm + row * L::kPitch + D * 4) = orow;
      if (parts) p.part_ml[orow] = make_float2(m, l);
      else if (p.lse) p.lse[orow] = m > -INFINITY ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
    }
    tc::fence_before();
  }
  __syncthreads();
#pragma unroll 4
  for (int at = warp; at < n_rows; at += kThreadsT / 32) {
    const int64_t orow = *reinterpret_cast<const int64_t*>(sm + at * L::kPitch + D * 4);
#pragma unroll
    for (int c = 4 * lane; c < D; c += 128) {
      const float4 v = *reinterpret_cast<const float4*>(sm + at * L::kPitch + c * 4);
      if (parts) {
        *reinterpret_cast<float4*>(p.part_o + orow * D + c) = v;
      } else {
        const __nv_bfloat162 h0 = __floats2bfloat162_rn(v.x, v.y), h1 = __floats2bfloat162_rn(v.z, v.w);
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + orow * D + c) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&h0), *reinterpret_cast<const uint32_t*>(&h1));
      }
    }
  }
  pair_sync();
  tc::fence_after();
  if (warp == kScoreWarp) pair_dealloc(tbase);
}

template <int D>
cudaError_t tree_launch_d(AttnParams p, int num_sms, size_t part_rows, cudaStream_t st) {
  const int n_rt = (int)(((int64_t)p.max_q * p.g + kPairRowsT - 1) / kPairRowsT);
  int64_t span = std::max(p.max_len, 1);  // keys that a row tile can see: the window's, or all
  if (p.window > 0) span = std::min<int64_t>(span, (int64_t)p.window + p.max_q + kTileT);
  const int tiles = (int)((span + kTileT - 1) / kTileT), places = std::max(1, num_sms / 2);
  // Row tiles that fill the GPU go whole, the keys of the rest are split into the
  // number of parts that ends first, counting a pair's start and end as 4 tiles.
  const int64_t total = (int64_t)p.hk * n_rt * p.n_seqs, whole = total / places * places, rest = total - whole;
  int64_t best = 0;
  int chunk = tiles;
  p.n_split = 1;
  for (int n = 1; rest > 0 && n <= std::min(kMaxSplit, std::max(1, tiles / 2)); ++n) {
    if (n > 1 && rest * n * kPairRowsT > (int64_t)part_rows) break;
    const int c = (tiles + n - 1) / n;
    const int64_t cost = (rest * n + places - 1) / places * (c + 4) + (n > 1 ? 4 : 0);
    if (n == 1 || cost < best) best = cost, chunk = c, p.n_split = (tiles + c - 1) / c;
  }
  // (the join of split parts knows their sequences by the call's order)
  p.by_length = p.n_split == 1 && total > places && p.n_seqs <= kSortedSeqs && p.window == 0;
  cudaError_t e = launch_pdl(tree_kernel<D>, dim3((unsigned)(2 * (whole + rest * p.n_split))), kThreadsT, TreePlan<D>::kTotal, st, p, n_rt,
                             (int)whole, chunk);
  if (e == cudaSuccess && p.n_split > 1) e = join_launch(p, kPairRowsT, n_rt, (int)whole, st);
  return e;
}

template <int D>
cudaError_t tree_configure_d() {
  return cudaFuncSetAttribute(tree_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, TreePlan<D>::kTotal);
}

}  // namespace

cudaError_t tree_configure(int D) {
  switch (D) {
    case 64: return tree_configure_d<64>();
    case 128: return tree_configure_d<128>();
    case 192: return tree_configure_d<192>();
    default: return tree_configure_d<256>();
  }
}

cudaError_t tree_launch(const AttnParams& p, int num_sms, size_t part_rows, cudaStream_t st) {
  switch (p.D) {
    case 64: return tree_launch_d<64>(p, num_sms, part_rows, st);
    case 128: return tree_launch_d<128>(p, num_sms, part_rows, st);
    case 192: return tree_launch_d<192>(p, num_sms, part_rows, st);
    default: return tree_launch_d<256>(p, num_sms, part_rows, st);
  }
}

}  // namespace attn
}  // namespace moe

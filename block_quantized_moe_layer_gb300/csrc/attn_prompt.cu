// attn_prompt.cu -- attention of many query rows (prompt chunks) over the
// 4-bit paged cache, on the tcgen05 tensor cores.
//
// Two kernels.  expand_kernel dequantises the visible tiles of 128 keys of
// each (sequence, key/value head) once into 16-bit operand images in the
// workspace (exact: see attn_mma.cuh); prompt_kernel reads them with one bulk
// copy a tile.  Dequantising inside prompt_kernel instead would repeat it for
// every 128 query rows (T g / 128 times), and its instructions and
// shared-memory writes would not fit beside the softmax; the extra pass writes
// 4 D bytes a key and head once, some 1% of the time of a prompt chunk.
//
// prompt_kernel: a pair of blocks (a cluster on two neighbouring
// multiprocessors) owns 256 rows (query token, query head of one key/value
// head), 128 a block, and walks over the visible 128-key tiles j:
//   S_j = Q K_j^T   (bf16, M = 256, N = 128, both operands in shared memory)
//   P_j = 2^(scale S_j - m), rounded to fp16 in tensor memory
//   O  += P_j V_j   (fp16, P from tensor memory, N = D)
// Each block copies half of every image; the MMAs of the pair read both halves.
// A block alone copies 96 KB a tile of D = 192, for which L2 has about 53 bytes
// a cycle and multiprocessor: 1850 cycles, where the MMAs take 1540.
//   The first block's MMA threads issue for both: one the scores, one the
// products.  S has two buffers of columns; P lies behind O in columns of its
// own where there are some (D <= 192), so that S_{j+2} can follow as soon as
// S_j has been read, over S_j otherwise.  Two groups of four softmax warps take
// turns (softmax_turns), a thread a whole row of scores.
//   The reference m moves only when the maximum passes it by more than 8 (a
// weight of 2^8 is harmless in fp16 and fp32), which keeps the rescaling of
// the output in tensor memory rare; l and O stay consistent with m either way.
//   TMEM columns: S at 0 and 128, O at 256, P from 256 + D on.
// Bound: MMA issue and execution; 1024 query tokens of 64/4 heads of 192 behind
// 7168 keys take 243 to 247 us (1.59 PFLOP/s, 0.82 of the cuBLAS rate measured): the
// tensor pipe is active 77% of prompt_kernel; the rest are the blocks' starts
// and ends (some 12000 cycles of 120000) and the last wave.
//
// Operand images (no swizzle, K-major, 8x8 core matrices of 128 contiguous
// bytes): rows x channels as [channels/8][rows][8]; values as
// [keys/8][D][8 keys], so that the contraction index is innermost in both.  An
// image is cut in halves by its keys, the values' by their channels.
#include "attn_tc.cuh"

namespace moe {
namespace attn {

// Joins the parts of split rows (attn_small.cu).
cudaError_t join_launch(const AttnParams& p, int rows_per_tile, int n_rt, int whole, cudaStream_t st);

namespace {

constexpr int kRowsP = 128;               // of a block
constexpr int kPairRows = 2 * kRowsP;
constexpr int kTurns = 2;  // softmax groups: one takes the even tiles, one the odd ones
constexpr int kSoftWarps = 4 * kTurns, kCopyWarp = kSoftWarps, kMmaWarp = kSoftWarps + 1, kPvWarp = kSoftWarps + 2;
constexpr int kPromptThreads = (kSoftWarps + 4) * 32;  // (with an idle warp: registers are split by four warps)
constexpr int kMaxRing = 8;
constexpr int kPairSpins = 4096;         // tests before a suspending wait, of the threads that copy and issue (64: 1% more)

template <int D>
struct PromptPlan {
  static constexpr int kImage = kTileTokens * D * 2;  // bytes of one operand image
  static constexpr int kHalf = kImage / 2;            // a block's half of it
  // buffers of weights that fit in tensor memory beside scores and output (0: they lie over the scores)
  static constexpr int kWeights = D <= 128 ? 2 : (D == 192 ? 1 : 0);
  static constexpr int kLead = kWeights ? 2 : 1;  // scores issued ahead of a product
  static constexpr int kRing = D == 64 ? 7 : (D == 128 ? 5 : (D == 192 ? 3 : 2));
  static constexpr int kQ = 0;
  static constexpr int kStages = kRowsP * D * 2;
  static constexpr int kMax = kStages + kRing * kImage;              // float [2][turns][128]
  static constexpr int kBars = kMax + kTurns * 2 * kRowsP * 4;
  static constexpr int kNumBars = 4 * kMaxRing + 8 + 1;
  static constexpr int kMisc = kBars + kNumBars * 8;
  static constexpr int kTotal = kMisc + 16 + 128;
  static constexpr int kPitch = D * 4 + 16;  // of an output row on its way out
  static_assert(kRowsP * kPitch <= kMax, "outputs fit below the maxima");
  static_assert(kTotal <= 232448, "shared memory plan");
  // (a pair never waits for tensor memory that another pair holds half of)
  static_assert(kTotal > 116 * 1024, "one block a multiprocessor");
};

// What the two kernels share about the images of a launch.
struct Images {
  uint8_t* base;    // [sequence][kv head][tile]{keys, values}[half]
  uint4* valid;     // [sequence][tile]: a bit for each key that exists
  int tiles;        // tiles of a sequence
};

// Tiles of a sequence that any of its queries sees: [first, last).
__device__ __forceinline__ void seq_tiles(const AttnParams& p, const Seq& s, int& first, int& last) {
  const int lo = key_lo(p, max(0, s.len - s.nq));
  first = lo / kTileTokens;
  last = s.nq > 0 ? (s.len + kTileTokens - 1) / kTileTokens : first;
}

// Four blocks a tile: the keys and the values of its first and second 64 keys
// (one block a tile waits longer for its loads: 250 against 243 us in all for
// the prompt chunk above).
__global__ void __launch_bounds__(256) expand_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ Images im) {
  griddep_launch_dependents();
  griddep_wait();
  const int b = blockIdx.z, kvh = blockIdx.y, at_tile = blockIdx.x >> 2, k_lo = (blockIdx.x & 1) * (kTileTokens / 2);
  const bool values = blockIdx.x & 2;
  const Seq s = load_seq(p, b);
  int first, last;
  seq_tiles(p, s, first, last);
  const int tile = first + at_tile;
  if (tile >= last) return;
  __shared__ int page[kTileTokens / 16];
  const int ppt = kTileTokens >> p.pshift, tid = threadIdx.x, D = p.D;
  if (tid < ppt) {
    const int i = tile * ppt + tid;
    // (a page that no query sees is not looked at: it may have been given back)
    const bool seen = (i << p.pshift) < s.len && ((i + 1) << p.pshift) > key_lo(p, max(0, s.len - s.nq));
    page[tid] = seen ? load_page(p, b, i) : -1;
  }
  __syncthreads();
  const int n_keys = min(kTileTokens, s.len - tile * kTileTokens);
  if (kvh == 0 && (blockIdx.x & 3) == 0 && tid < 4) {
    uint32_t m = 0;
    for (int i = 0; i < 32; ++i) {
      const int k = 32 * tid + i;
      if (k < n_keys && page[k >> p.pshift] >= 0) m |= 1u << i;
    }
    reinterpret_cast<uint32_t*>(im.valid + (int64_t)b * im.tiles + at_tile)[tid] = m;
  }
  const int64_t image = (int64_t)kTileTokens * D * 2;
  uint8_t* kd = im.base + (((int64_t)b * p.hk + kvh) * im.tiles + at_tile) * 2 * image;
  uint8_t* vd = kd + image;
  const int words = D / 8, code_b = p.P * (D / 2);
  // keys: a thread takes a word of 8 channels; a warp 32 keys of the same word
  for (int u = tid; u < (values ? 0 : kTileTokens / 2 * words); u += 256) {
    const int k = k_lo + (u & (kTileTokens / 2 - 1)), w = u / (kTileTokens / 2);
    const int pg = page[k >> p.pshift];
    uint4 o = make_uint4(0, 0, 0, 0);
    if (k < n_keys && pg >= 0) {
      const uint8_t* base = p.pages + pg * p.page_bytes + kvh * p.head_bytes;
      const int at = k & (p.P - 1);
      const uint32_t sb = base[code_b + at * (D / 16) + (w >> 1)];
      uint32_t x[4];
      key_pairs(*reinterpret_cast<const uint32_t*>(base + at * (D / 2) + 4 * w), key_scale(sb | (sb << 16)), x);
      o = make_uint4(x[0], x[1], x[2], x[3]);
    }
    *reinterpret_cast<uint4*>(kd + (k >= kTileTokens / 2 ? image / 2 : 0) + ((int64_t)w * (kTileTokens / 2) + k % (kTileTokens / 2)) * 16) = o;
  }
  // values: a thread takes 8 keys of a word, and turns them to 8 channels of 8 keys
  for (int u = tid; u < (values ? kTileTokens / 16 * words : 0); u += 256) {
    const int w = u % words, k0 = k_lo + 8 * (u / words);
    const int pg = page[k0 >> p.pshift];
    uint32_t x[4][8];  // [pair of keys][channel]
    const uint8_t* base = p.pages + (pg < 0 ? 0 : pg) * p.page_bytes + kvh * p.head_bytes + p.head_bytes / 2;
    const int at = k0 & (p.P - 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t w0 = 0, w1 = 0, s0 = 0, s1 = 0;
      if (pg >= 0 && k0 + 2 * i < n_keys) {
        w0 = *reinterpret_cast<const uint32_t*>(base + (at + 2 * i) * (D / 2) + 4 * w);
        s0 = base[code_b + (at + 2 * i) * (D / 16) + (w >> 1)];
      }
      if (pg >= 0 && k0 + 2 * i + 1 < n_keys) {
        w1 = *reinterpret_cast<const uint32_t*>(base + (at + 2 * i + 1) * (D / 2) + 4 * w);
        s1 = base[code_b + (at + 2 * i + 1) * (D / 16) + (w >> 1)];
      }
      const ValueScale d = value_scale(s0 | (s1 << 16));
      value_quads(__byte_perm(w0, w1, 0x5410), d, x[i][0], x[i][2], x[i][4], x[i][6]);
      value_quads(__byte_perm(w0, w1, 0x7632), d, x[i][1], x[i][3], x[i][5], x[i][7]);
    }
    const int half = w >= words / 2;
    uint4* o = reinterpret_cast<uint4*>(vd + half * (image / 2) + ((int64_t)(k0 / 8) * (D / 2) + 8 * (w - half * (words / 2))) * 16);
#pragma unroll
    for (int c = 0; c < 8; ++c) o[c] = make_uint4(x[0][c], x[1][c], x[2][c], x[3][c]);
  }
}

// The softmax of one group's tiles: thread (turn, row) takes all 128 scores of
// its row in the tiles turn, turn + 2, ...: two tiles are worked on at once, so
// that one group's waits fall into the other's arithmetic.  The reference m
// goes from tile to tile, and so from group to group, through shared memory
// as soon as a tile's maximum is known; l is the thread's share of the sum,
// relative to its own last m.  vis(j, bits): the keys seen, false where all are.
//   No wait for PV below skips a phase of its barrier, which two products
// apart share: the end of PV(j - 3) is known in tile j, from the buffer's wait
// here or two tiles before, or (weights over the scores) from S(j) itself.
template <int D, class Vis>
__device__ __forceinline__ void softmax_turns(const AttnParams& p, int n_tiles, uint32_t tl, int turn, int row, float* ref,
                                              uint64_t* sfull, uint64_t* sread, uint64_t* pfull, uint64_t* odone,
                                              volatile int* abort, float& m, float& l, Vis vis) {
  constexpr int kWeights = PromptPlan<D>::kWeights;
  const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) & 3;
  const int before = 1 + w + (turn ? 0 : 4), behind = 1 + w + (turn ? 4 : 0);  // named barriers with the other group's warp
  bool ok = true;
  auto product = [&](int j, int site) {  // waits for PV(j)
    ok = ok && wait_inline(&odone[j & 1], (uint32_t)((j >> 1) & 1), abort, p.status, p.timeout_ns, site);
    ok = __all_sync(0xffffffffu, ok);
    if (ok) tc::fence_after();
  };
  for (int j = turn; j < n_tiles; j += 2) {
    const uint32_t tile = tl + 128 * turn;
    float x[128];
    float mx = -INFINITY;
    if (ok) {
      ok = wait_inline(&sfull[turn], (uint32_t)((j >> 1) & 1), abort, p.status, p.timeout_ns, 30);
      ok = __all_sync(0xffffffffu, ok);
    }
    if (ok) {
      tc::fence_after();
      uint32_t sv[8][16];
#pragma unroll
      for (int c = 0; c < 8; ++c) tc::ld_32x32b_x16(tile + 16 * c, sv[c]);
      tc::wait_ld();
      if (kWeights > 0 && j + 2 < n_tiles) {
        tc::fence_before();
        __syncwarp();
        if (lane == 0) arrive_first(&sread[turn]);
      }
#pragma unroll
      for (int c = 0; c < 128; ++c) x[c] = __uint_as_float(sv[c >> 4][c & 15]);
      uint64_t bits[2];
      if (vis(j, bits)) {
#pragma unroll
        for (int c = 0; c < 128; ++c)
          if (!((bits[c >> 6] >> (c & 63)) & 1)) x[c] = -INFINITY;
      }
      float a[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
      for (int c = 4; c < 128; c += 8)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          a[i] = c + 4 + i < 128 ? fmaxf(a[i], fmaxf(x[c + i], x[c + 4 + i])) : fmaxf(a[i], x[c + i]);
      mx = fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3])) * p.scale_log2;
    }
    float m0 = m;  // the reference of the tile before
    if (j > 0) {
      asm volatile("bar.sync %0, 64;" ::"r"(before) : "memory");
      m0 = ref[row];
    }
    const bool move = mx > m0 + kLazy;  // (also the first visible keys: m0 = -inf)
    const float m1 = move ? mx : m0;
    if (j + 1 < n_tiles) {
      ref[row] = m1;
      asm volatile("bar.arrive %0, 64;" ::"r"(behind) : "memory");
    }
    if (!ok) continue;
    if (m1 != m) l *= m == -INFINITY ? 0.f : exp2_approx(m - m1);
    m = m1;
    if (kWeights == 2 && j >= 2) product(j - 2, 35);
    if (!ok) continue;
    if (j > 0 && __any_sync(0xffffffffu, move)) {
      const float f = move ? (m0 == -INFINITY ? 0.f : exp2_approx(m0 - m1)) : 1.f;
      product(j - 1, 32);
      if (!ok) continue;
#pragma unroll 1
      for (int c = 0; c < D; c += 16) {
        uint32_t o[16];
        tc::ld_32x32b_x16(tl + 256 + c, o);
        tc::wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
        tc::st_32x32b_x16(tl + 256 + c, o);
      }
    }
    const float base = m == -INFINITY ? 0.f : m;
    uint32_t pk[4][16];
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int c = 0; c < 64; ++c) {
      const float u = exp2_approx(fmaf(x[2 * c], p.scale_log2, -base));
      const float v = exp2_approx(fmaf(x[2 * c + 1], p.scale_log2, -base));
      s0 += u;
      s1 += v;
      pk[c >> 4][c & 15] = pack_h2(u, v);
    }
    l += s0 + s1;
    uint32_t weights = tile;
    if constexpr (kWeights > 0) {
      weights = tl + 256 + D + (kWeights == 2 ? 64 * turn : 0);
      if (kWeights == 1 && j >= 1) {  // the product that read this buffer's last weights
        product(j - 1, 36);
        if (!ok) continue;
      }
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) tc::st_32x32b_x16(weights + 16 * c, pk[c]);
    tc::wait_st();
    tc::fence_before();
    __syncwarp();
    if (lane == 0) arrive_first(&pfull[turn]);
  }
  if (n_tiles > 1) product(n_tiles - 2, 33);
  product(n_tiles - 1, 34);
}

template <int D>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPromptThreads, 1)
    prompt_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ Images im, int n_rt, int whole, int chunk) {
  using L = PromptPlan<D>;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  float* smax = reinterpret_cast<float*>(sm + L::kMax);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + L::kBars);  // ring of keys, ring of values: copy landed
  uint64_t* empty = full + 2 * kMaxRing;                         // the same: MMAs that read it done
  uint64_t* sfull = empty + 2 * kMaxRing;                            // [2] scores ready
  uint64_t* pfull = sfull + 2;                                   // [2] weights stored (the softmax may be a tile ahead)
  uint64_t* odone = pfull + 2;                                   // [2] output product done
  uint64_t* sread = odone + 2;                                   // [2] scores read
  uint64_t* fin = sread + 2;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + L::kMisc);
  volatile int* abort = reinterpret_cast<volatile int*>(sm + L::kMisc + 4);
  volatile int never = 0;
  const int tid = threadIdx.x, warp = uniform_warp(), lane = tid & 31;
  const int rank = (int)blockIdx.x & 1, pair = (int)blockIdx.x >> 1;  // (a cluster is two neighbours)
  const bool first_block = rank == 0;
  griddep_launch_dependents();
  if (tid == 0) {
    for (int i = 0; i < 2 * kMaxRing; ++i) {
      mbar_init(&full[i], (first_block ? 2 : 1) + p.miss);  // (the first block's: its own copy, and word of the other's)
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sfull[i], 1);
      mbar_init(&pfull[i], 2 * 4);  // (the first block's are used)
      mbar_init(&sread[i], 2 * 4);
      mbar_init(&odone[i], 1);
    }
    mbar_init(fin, 2);
    *abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  griddep_wait();

  // the first `whole` pairs take a row tile each, those with the longest key
  // ranges first; the others p.n_split parts of one
  const bool split_tile = pair >= whole;
  const int tile_i = split_tile ? whole + (pair - whole) / p.n_split : pair;
  const int split = split_tile ? (pair - whole) % p.n_split : 0;
  const int rt = n_rt - 1 - tile_i / (p.hk * p.n_seqs), b = tile_i % (p.hk * p.n_seqs) / p.hk, kvh = tile_i % p.hk;
  const bool parts = split_tile && p.n_split > 1;
  const Seq s = load_seq(p, b);
  const int pair_row0 = rt * kPairRows, pair_rows = min(kPairRows, s.nq * p.g - pair_row0);
  if (pair_rows <= 0) return;
  const int row0 = pair_row0 + rank * kRowsP, n_rows = min(kRowsP, s.nq * p.g - row0);  // (may be none in the second block)
  const int p0 = s.len - s.nq;
  // positions of the pair's keys, and those that all of the block's rows see
  const int pair_min = p0 + pair_row0 / p.g, pair_max = p0 + (pair_row0 + pair_rows - 1) / p.g;
  const int pos_min = p0 + row0 / p.g, pos_max = p0 + (row0 + max(n_rows, 1) - 1) / p.g;
  const int lo = key_lo(p, max(0, pair_min)), hi = pair_max + 1, lo_max = key_lo(p, pos_max);
  int seq_first, seq_last;
  seq_tiles(p, s, seq_first, seq_last);
  const int tile_a = lo / kTileTokens + split * chunk;
  const int n_tiles = hi > lo ? max(0, min(split_tile ? tile_a + chunk : 0x7fffffff, (hi + kTileTokens - 1) / kTileTokens) - tile_a) : 0;
  const uint8_t* images = im.base + (((int64_t)b * p.hk + kvh) * im.tiles + (tile_a - seq_first)) * 2 * (int64_t)L::kImage + rank * L::kHalf;
  const uint4* valid = im.valid + (int64_t)b * im.tiles + (tile_a - seq_first);

  if (warp == kMmaWarp) pair_alloc(tslot);
  const int turn = warp >> 2, row = (warp & 3) * 32 + lane;  // of the softmax threads
  int tq = 0, hq = 0, hi_r = 0, lo_r = 0;
  const bool has_row = warp < kSoftWarps && row < n_rows;
  if (has_row) {
    tq = (row0 + row) / p.g;
    hq = kvh * p.g + (row0 + row) % p.g;
    hi_r = p0 + tq + 1;
    lo_r = key_lo(p, p0 + tq);
  }
  // queries: a warp takes 8 rows and 4 of their pieces of 8 channels at a time,
  // all of them on their way at once (a thread a row took 8000 cycles)
  if (warp < kSoftWarps && n_tiles > 0) {
    constexpr int kSteps = kRowsP / 8 / kSoftWarps;
    uint4 v[kSteps][D / 32];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int at = row0 + 8 * (kSteps * warp + i) + (lane & 7);
      const bool has = at < row0 + n_rows;
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q);
      if (has) q += (s.start + at / p.g) * p.q_tok + (kvh * p.g + at % p.g) * p.q_head;
#pragma unroll
      for (int c = 0; c < D / 32; ++c)
        v[i][c] = has ? *reinterpret_cast<const uint4*>(q + 32 * c + 8 * (lane >> 3)) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < kSteps; ++i)
#pragma unroll
      for (int c = 0; c < D / 32; ++c)
        *reinterpret_cast<uint4*>(sm + L::kQ + ((4 * c + (lane >> 3)) * kRowsP + 8 * (kSteps * warp + i) + (lane & 7)) * 16) = v[i][c];
    tc::fence_async_smem();
  }
  tc::fence_before();
  pair_sync();  // both blocks' barriers and queries are there
  tc::fence_after();
  const uint32_t tbase = *tslot;

  // Registers: 384 threads are launched with 168; the softmax takes 216 of a
  // thread (it holds a row of scores), which leaves 72 for the others.  The
  // block's barriers keep the others from asking for theirs again before the
  // softmax has its share, which it would then wait for without end.
  float m = -INFINITY, l = 0.f;
  if (warp >= kSoftWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    __syncthreads();
    if (warp == kCopyWarp) {
      // ------------------------------------------------------------ copies, in order of use: K(i), V(i - lead)
      if (lane == 0) {
        const int n = n_tiles > 0 ? n_tiles + L::kLead : 0;
        bool ok = true;
        int keys = 0, values = 0;  // copied
        auto copy = [&](int v, int& j) {
          const int st = j % L::kRing;
          if (j >= L::kRing)
            ok = ok && wait_bar<kPairSpins>(&empty[v * kMaxRing + st], (uint32_t)((j / L::kRing - 1) & 1), abort, p.status, p.timeout_ns, 11);
          if (!ok) return;
          mbar_arrive_expect_tx(&full[v * kMaxRing + st], L::kHalf);
          bulk_g2s(sm + L::kStages + st * L::kImage + v * L::kHalf, images + ((int64_t)2 * j + v) * L::kImage, L::kHalf,
                   &full[v * kMaxRing + st]);
          ++j;
        };
        for (int i = 0; i < n && ok; ++i) {
          if (i < n_tiles) copy(0, keys);
          if (i >= L::kLead) copy(1, values);
        }
        // the copies have landed and, unless the block gave up, the MMAs' words
        // about them too: nothing is on its way to a block that ends
        bool there = true;
        for (int v = 0; v < 2; ++v) {
          const int all = v ? values : keys;
          for (int k = max(0, all - L::kRing); k < all; ++k) {
            const int at = v * kMaxRing + k % L::kRing;
            there = there && wait_bar(&full[at], (uint32_t)((k / L::kRing) & 1), &never, p.status, p.timeout_ns, 12);
            ok = ok && wait_bar(&empty[at], (uint32_t)((k / L::kRing) & 1), abort, p.status, p.timeout_ns, 16);
          }
        }
      }
    } else if (warp == kMmaWarp || warp == kPvWarp) {
      // ------------------------------------------------------------ MMAs: a thread for the scores, one for the
      // products (one thread for both spent 1800 cycles on a tile, in waits and
      // commits beside the softmax's instructions; the MMAs take 1540)
      const int v = warp == kPvWarp;
      if (n_tiles > 0 && !first_block && elect_one()) {  // the other block's: its copies' arrival
        bool ok = true;
        for (int j = 0; j < n_tiles && ok; ++j) {
          uint64_t* bar = &full[v * kMaxRing + j % L::kRing];
          ok = wait_bar(bar, (uint32_t)((j / L::kRing) & 1), abort, p.status, p.timeout_ns, 17);
          if (ok) arrive_first(bar);
        }
      }
      if (n_tiles > 0 && first_block && elect_one()) {
        constexpr uint32_t kIdescS = tc::idesc_f16(kPairRows, kTileTokens) | (1u << 7) | (1u << 10);  // bf16 operands
        constexpr uint32_t kIdescO = tc::idesc_f16(kPairRows, D);
        const uint64_t qd = tc::smem_desc(smem_u32(sm + L::kQ), kRowsP * 16, 128);
        // the scores' columns are free: read, or with the weights over them, multiplied
        uint64_t* room = L::kWeights ? sread : odone;
        bool ok = true;
        for (int j = 0; j < n_tiles; ++j) {
          const int st = j % L::kRing, at = v * kMaxRing + st;
          const uint32_t image = smem_u32(sm + L::kStages + st * L::kImage + v * L::kHalf);
          ok = wait_bar<kPairSpins>(&full[at], (uint32_t)((j / L::kRing) & 1), abort, p.status, p.timeout_ns, 13);
          if (!v) {
            if (j >= 2) ok = ok && wait_bar<kPairSpins>(&room[j & 1], (uint32_t)(((j - 2) >> 1) & 1), abort, p.status, p.timeout_ns, 18);
            if (!ok) break;
            tc::fence_after();
            const uint64_t kd = tc::smem_desc(image, kTileTokens / 2 * 16, 128);
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              pair_mma_ss(tbase + 128 * (j & 1), qd + k * (2 * kRowsP * 16 / 16), kd + k * (2 * (kTileTokens / 2) * 16 / 16), kIdescS, k > 0);
            pair_commit(&sfull[j & 1], 3);
          } else {
            ok = ok && wait_bar<kPairSpins>(&pfull[j & 1], (uint32_t)((j >> 1) & 1), abort, p.status, p.timeout_ns, 14);
            if (!ok) break;
            tc::fence_after();
            const uint64_t vd = tc::smem_desc(image, D / 2 * 16, 128);
            const uint32_t weights = tbase + (L::kWeights == 0 ? 128 * (j & 1) : 256 + D + (L::kWeights == 2 ? 64 * (j & 1) : 0));
#pragma unroll
            for (int k = 0; k < kTileTokens / 16; ++k)
              pair_mma_ts(tbase + 256, weights + 8 * k, vd + k * (2 * (D / 2) * 16 / 16), kIdescO, j > 0 || k > 0);
            pair_commit(&odone[j & 1], 3);
          }
          pair_commit(&empty[at], 3);
        }
        // all MMAs issued are complete before the pair frees anything
        pair_commit(fin, 1);
        wait_bar(fin, 0, &never, p.status, p.timeout_ns, 15);
      }
    }
    __syncthreads();
    asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    __syncthreads();
    if (n_tiles > 0) {
      // ------------------------------------------------------------ softmax
      const uint32_t tl = tbase + ((uint32_t)(warp & 3) << 21);  // this warp's 32 lanes
      uint4 ahead = make_uint4(0, 0, 0, 0);  // the keys that exist, read two tiles early: they wait for L2
      if (turn < n_tiles) ahead = __ldcg(valid + turn);
      bool seen = false;
      softmax_turns<D>(p, n_tiles, tl, turn, row, smax, sfull, sread, pfull, odone, abort, m, l, [&](int j, uint64_t (&bits)[2]) {
        const int c0 = (tile_a + j) * kTileTokens;
        const uint64_t e0 = ahead.x | ((uint64_t)ahead.y << 32), e1 = ahead.z | ((uint64_t)ahead.w << 32);
        if (j + 2 < n_tiles) ahead = __ldcg(valid + j + 2);
        if (c0 + kTileTokens <= pos_min + 1 && c0 >= lo_max && (e0 & e1) == ~0ull) {
          seen = true;
          return false;
        }
        bits[0] = key_bits<64>(c0, lo_r, hi_r) & e0;
        bits[1] = key_bits<64>(c0 + 64, lo_r, hi_r) & e1;
        seen |= (bits[0] | bits[1]) != 0;
        return true;
      });
      if (seen) m = fmaxf(m, kSeen);
    }
    __syncwarp();
    asm volatile("setmaxnreg.dec.sync.aligned.u32 168;");
    __syncthreads();
  }
  // the groups' sums, at the later reference, once no MMA reads either block
  pair_sync();
  if (warp < kSoftWarps) {
    smax[turn * kRowsP + row] = m;
    smax[(2 + turn) * kRowsP + row] = l;
  }
  __syncthreads();
  if (warp < kSoftWarps) {
    const float other = smax[(turn ^ 1) * kRowsP + row], mm = fmaxf(m, other);
    l = m == -INFINITY ? 0.f : l * exp2_approx(m - mm);
    l += other == -INFINITY ? 0.f : smax[(2 + (turn ^ 1)) * kRowsP + row] * exp2_approx(other - mm);
    m = mm;
    const uint32_t tl = tbase + ((uint32_t)(warp & 3) << 21);
    const float inv = parts ? 1.f : kValueUnscale / l;  // (rows that see no key: not used)
    // the outputs go through shared memory, where queries and images were: a
    // thread's row is D apart from its neighbour's (stored from here they took
    // 6000 cycles, a part's 11000)
#pragma unroll 2
    for (int c = turn * (D / 2); c < (turn + 1) * (D / 2); c += 16) {
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
    if (has_row && turn == 0) {
      const int64_t orow = parts ? ((int64_t)(tile_i - whole) * p.n_split + split) * kPairRows + rank * kRowsP + row
                                 : (int64_t)(s.start + tq) * p.hq + hq;
      *reinterpret_cast<int64_t*>(sm + row * L::kPitch + D * 4) = orow;
      if (parts) p.part_ml[orow] = make_float2(m, l);
      else if (p.lse) p.lse[orow] = m > -INFINITY ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
    }
    tc::fence_before();
  }
  __syncthreads();
#pragma unroll 4
  for (int at = warp; at < n_rows; at += kPromptThreads / 32) {
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
  if (warp == kMmaWarp) pair_dealloc(tbase);
}

template <int D>
cudaError_t prompt_launch_d(AttnParams p, int num_sms, size_t part_rows, uint8_t* ws, int tile_cap, cudaStream_t st) {
  const int n_rt = (int)(((int64_t)p.max_q * p.g + kPairRows - 1) / kPairRows);
  int64_t span = std::max(p.max_len, 1);
  if (p.window > 0) span = std::min<int64_t>(span, (int64_t)p.window + p.max_q + 2 * kTileTokens);
  Images im;
  im.tiles = (int)((span + kTileTokens - 1) / kTileTokens);
  const int at_once = std::max(1, std::min(p.n_seqs, tile_cap / (p.hk * im.tiles)));
  im.base = ws;
  im.valid = reinterpret_cast<uint4*>(ws + (size_t)tile_cap * 2 * PromptPlan<D>::kImage);
  // tiles of one row tile's keys: its window's, or all
  int64_t rspan = std::max(p.max_len, 1);
  if (p.window > 0) rspan = std::min<int64_t>(rspan, (int64_t)p.window + kPairRows + kTileTokens);
  const int rtiles = (int)((rspan + kTileTokens - 1) / kTileTokens);
  const int all = p.n_seqs, places = std::max(1, num_sms / 2);
  for (int b0 = 0; b0 < all; b0 += at_once) {
    AttnParams g = p;
    g.n_seqs = std::min(at_once, all - b0);
    g.starts += b0;
    g.lens += b0;
    g.table += (int64_t)b0 * p.table_stride;
    // Row tiles that fill the GPU go whole; the keys of the rest are split, so
    // that a last wave takes part of one's time: into the number of parts that
    // ends first, counting a block's start and end as 4 tiles.  (512 row tiles
    // of 60 key tiles on 152 multiprocessors: 4 waves whole, 3.5 so.)
    const int64_t total = (int64_t)p.hk * n_rt * g.n_seqs, whole = total / places * places, rest = total - whole;
    int64_t best = 0;
    int chunk = rtiles;
    g.n_split = 1;
    for (int n = 1; rest > 0 && n <= std::min(kMaxSplit, std::max(1, rtiles / 2)); ++n) {
      if (n > 1 && rest * n * kPairRows > (int64_t)part_rows) break;
      const int c = (rtiles + n - 1) / n;
      const int64_t cost = (rest * n + places - 1) / places * (c + 4) + (n > 1 ? 4 : 0);
      if (n == 1 || cost < best) best = cost, chunk = c, g.n_split = (rtiles + c - 1) / c;
    }
    cudaError_t e = launch_pdl(expand_kernel, dim3(4 * im.tiles, p.hk, g.n_seqs), 256, 0, st, g, im);
    if (e == cudaSuccess)
      e = launch_pdl(prompt_kernel<D>, dim3((unsigned)(2 * (whole + rest * g.n_split))), kPromptThreads, PromptPlan<D>::kTotal, st, g, im,
                     n_rt, (int)whole, chunk);
    if (e == cudaSuccess && g.n_split > 1) e = join_launch(g, kPairRows, n_rt, (int)whole, st);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

size_t prompt_ws_bytes(int D, int tile_cap) {
  return (size_t)tile_cap * ((size_t)2 * kTileTokens * D * 2 + sizeof(uint4));
}

cudaError_t prompt_configure() {
  cudaError_t e = cudaFuncSetAttribute(prompt_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize, PromptPlan<64>::kTotal);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(prompt_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize, PromptPlan<128>::kTotal);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(prompt_kernel<192>, cudaFuncAttributeMaxDynamicSharedMemorySize, PromptPlan<192>::kTotal);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(prompt_kernel<256>, cudaFuncAttributeMaxDynamicSharedMemorySize, PromptPlan<256>::kTotal);
  return e;
}

cudaError_t prompt_launch(const AttnParams& p, int num_sms, size_t part_rows, uint8_t* ws, int tile_cap, cudaStream_t st) {
  switch (p.D) {
    case 64: return prompt_launch_d<64>(p, num_sms, part_rows, ws, tile_cap, st);
    case 128: return prompt_launch_d<128>(p, num_sms, part_rows, ws, tile_cap, st);
    case 192: return prompt_launch_d<192>(p, num_sms, part_rows, ws, tile_cap, st);
    default: return prompt_launch_d<256>(p, num_sms, part_rows, ws, tile_cap, st);
  }
}

}  // namespace attn
}  // namespace moe

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
// prompt_kernel: a block owns 128 rows (query token, query head of one
// key/value head) and walks over the visible 128-key tiles j:
//   S_j = Q K_j^T   (bf16, M = 128, N = 128; Q in tensor memory as far as it fits)
//   P_j = 2^(scale S_j - m), rounded to fp16 into the columns of S_j
//   O  += P_j V_j   (fp16, P from tensor memory, N = D)
// One thread issues all MMAs; S is double-buffered, so S_{j+1} runs while the
// softmax of S_j does.  Eight softmax warps: thread (half, row) takes 64 of a
// row's 128 scores (sixteen warps with 32 each: 283 against 275 us).
// The reference m moves only when the maximum passes it by more than 8 (a
// weight of 2^8 is harmless in fp16 and fp32), which keeps the rescaling of
// the output in tensor memory rare; l and O stay consistent with m either way.
//   TMEM columns: S at 0 and 128, O at 256, then Q (two channels a column).
//
// Operand images (no swizzle, K-major, 8x8 core matrices of 128 contiguous
// bytes): rows x channels as [channels/8][rows][8]; values as
// [keys/8][D][8 keys], so that the contraction index is innermost in both.
#include "attn_tc.cuh"

namespace moe {
namespace attn {

// Joins the parts of split rows (attn_small.cu).
cudaError_t join_launch(const AttnParams& p, int rows_per_tile, int n_rt, int whole, cudaStream_t st);

namespace {

constexpr int kRowsP = 128;
constexpr int kShares = 2;  // threads of a row
constexpr int kShareKeys = kTileTokens / kShares;
constexpr int kSoftWarps = 4 * kShares, kCopyWarp = kSoftWarps, kMmaWarp = kSoftWarps + 1;
constexpr int kPromptThreads = (kSoftWarps + 2) * 32;
constexpr int kMaxRing = 8;

template <int D>
struct PromptPlan {
  static constexpr int kImage = kTileTokens * D * 2;  // bytes of one operand image
  // channels of the queries that fit in tensor memory beside scores and output
  static constexpr int kTmemQ = D <= 128 ? D : (D == 192 ? 128 : 0);
  static constexpr int kRing = D == 64 ? 8 : (D == 128 ? 6 : (D == 192 ? 4 : 2));
  static constexpr int kQ = 0;  // the other channels
  static constexpr int kStages = kRowsP * (D - kTmemQ) * 2;
  static constexpr int kMax = kStages + kRing * kImage;              // float [2][shares][128]
  static constexpr int kBars = kMax + 2 * kShares * kRowsP * 4;
  static constexpr int kNumBars = 2 * kMaxRing + 6 + 1;
  static constexpr int kMisc = kBars + kNumBars * 8;
  static constexpr int kTotal = kMisc + 16 + 128;
  static_assert(kTotal <= 232448, "shared memory plan");
};

// What the two kernels share about the images of a launch.
struct Images {
  uint8_t* base;    // [sequence][kv head][tile]{keys, values}
  uint4* valid;     // [sequence][tile]: a bit for each key that exists
  int tiles;        // tiles of a sequence
};

// Tiles of a sequence that any of its queries sees: [first, last).
__device__ __forceinline__ void seq_tiles(const AttnParams& p, const Seq& s, int& first, int& last) {
  const int lo = key_lo(p, max(0, s.len - s.nq));
  first = lo / kTileTokens;
  last = s.nq > 0 ? (s.len + kTileTokens - 1) / kTileTokens : first;
}

__global__ void __launch_bounds__(256) expand_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ Images im) {
  griddep_launch_dependents();
  griddep_wait();
  const int b = blockIdx.z, kvh = blockIdx.y;
  const Seq s = load_seq(p, b);
  int first, last;
  seq_tiles(p, s, first, last);
  const int tile = first + blockIdx.x;
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
  if (kvh == 0 && tid < 4) {
    uint32_t m = 0;
    for (int i = 0; i < 32; ++i) {
      const int k = 32 * tid + i;
      if (k < n_keys && page[k >> p.pshift] >= 0) m |= 1u << i;
    }
    reinterpret_cast<uint32_t*>(im.valid + (int64_t)b * im.tiles + blockIdx.x)[tid] = m;
  }
  const int64_t image = (int64_t)kTileTokens * D * 2;
  uint8_t* kd = im.base + (((int64_t)b * p.hk + kvh) * im.tiles + blockIdx.x) * 2 * image;
  uint8_t* vd = kd + image;
  const int words = D / 8, code_b = p.P * (D / 2);
  // keys: a thread takes a word of 8 channels; a warp 32 keys of the same word
  for (int u = tid; u < kTileTokens * words; u += 256) {
    const int k = u & (kTileTokens - 1), w = u / kTileTokens;
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
    *reinterpret_cast<uint4*>(kd + ((int64_t)w * kTileTokens + k) * 16) = o;
  }
  // values: a thread takes 8 keys of a word, and turns them to 8 channels of 8 keys
  for (int u = tid; u < (kTileTokens / 8) * words; u += 256) {
    const int w = u % words, k0 = 8 * (u / words);
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
    uint4* o = reinterpret_cast<uint4*>(vd + ((int64_t)(k0 / 8) * D + 8 * w) * 16);
#pragma unroll
    for (int c = 0; c < 8; ++c) o[c] = make_uint4(x[0][c], x[1][c], x[2][c], x[3][c]);
  }
}

template <int D>
__global__ void __launch_bounds__(kPromptThreads, 1)
    prompt_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ Images im, int n_rt, int whole, int chunk) {
  using L = PromptPlan<D>;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  float* smax = reinterpret_cast<float*>(sm + L::kMax);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + L::kBars);  // ring: copy landed
  uint64_t* empty = full + kMaxRing;                             // ring: MMAs that read it done
  uint64_t* sfull = empty + kMaxRing;                            // [2] scores ready
  uint64_t* pfull = sfull + 2;                                   // [2] weights stored (the softmax may be a tile ahead)
  uint64_t* odone = pfull + 2;                                   // [2] output product done
  uint64_t* fin = odone + 2;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + L::kMisc);
  volatile int* abort = reinterpret_cast<volatile int*>(sm + L::kMisc + 4);
  volatile int never = 0;
  const int tid = threadIdx.x, warp = uniform_warp(), lane = tid & 31;
  griddep_launch_dependents();
  if (tid == 0) {
    for (int i = 0; i < L::kRing; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sfull[i], 1);
      mbar_init(&pfull[i], kSoftWarps);
      mbar_init(&odone[i], 1);
    }
    mbar_init(fin, 1);
    *abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  griddep_wait();

  // the first `whole` blocks take a row tile each, those with the longest key
  // ranges first; the others p.n_split parts of one
  const bool split_tile = (int)blockIdx.x >= whole;
  const int tile_i = split_tile ? whole + ((int)blockIdx.x - whole) / p.n_split : (int)blockIdx.x;
  const int split = split_tile ? ((int)blockIdx.x - whole) % p.n_split : 0;
  const int rt = n_rt - 1 - tile_i / (p.hk * p.n_seqs), b = tile_i % (p.hk * p.n_seqs) / p.hk, kvh = tile_i % p.hk;
  const bool parts = split_tile && p.n_split > 1;
  const Seq s = load_seq(p, b);
  const int row0 = rt * kRowsP, n_rows = min(kRowsP, s.nq * p.g - row0);
  if (n_rows <= 0) return;
  const int p0 = s.len - s.nq;
  const int pos_min = p0 + row0 / p.g, pos_max = p0 + (row0 + n_rows - 1) / p.g;
  const int lo = key_lo(p, max(0, pos_min)), hi = pos_max + 1, lo_max = key_lo(p, pos_max);
  int seq_first, seq_last;
  seq_tiles(p, s, seq_first, seq_last);
  const int tile_a = lo / kTileTokens + split * chunk;
  const int n_tiles = hi > lo ? max(0, min(split_tile ? tile_a + chunk : 0x7fffffff, (hi + kTileTokens - 1) / kTileTokens) - tile_a) : 0;
  const uint8_t* images = im.base + (((int64_t)b * p.hk + kvh) * im.tiles + (tile_a - seq_first)) * 2 * (int64_t)L::kImage;
  const uint4* valid = im.valid + (int64_t)b * im.tiles + (tile_a - seq_first);

  if (warp == kMmaWarp) tc::alloc_512(tslot);
  // queries: thread (share, row) lays its share of the row's channels into the image
  const int share = warp >> 2, row = (warp & 3) * 32 + lane;  // of the softmax threads
  int tq = 0, hq = 0, hi_r = 0, lo_r = 0;
  const bool has_row = warp < kSoftWarps && row < n_rows;
  if (has_row) {
    tq = (row0 + row) / p.g;
    hq = kvh * p.g + (row0 + row) % p.g;
    hi_r = p0 + tq + 1;
    lo_r = key_lo(p, p0 + tq);
  }
  constexpr int kChunks = D / 32 / kShares;
  uint32_t qr[kChunks][16];
  if (warp < kSoftWarps && n_tiles > 0) {
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + (s.start + tq) * p.q_tok + hq * p.q_head;
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (has_row) v = *reinterpret_cast<const uint4*>(q + 32 * (share * kChunks + c) + 8 * i);
        qr[c][4 * i] = v.x, qr[c][4 * i + 1] = v.y, qr[c][4 * i + 2] = v.z, qr[c][4 * i + 3] = v.w;
      }
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tbase = *tslot;
  if (warp < kSoftWarps && n_tiles > 0) {
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int ch = 32 * (share * kChunks + c);
      if (ch < L::kTmemQ) {
        tc::st_32x32b_x16(tbase + ((uint32_t)(warp & 3) << 21) + 256 + D + ch / 2, qr[c]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<uint4*>(sm + L::kQ + (((ch - L::kTmemQ) / 8 + i) * kRowsP + row) * 16) =
              make_uint4(qr[c][4 * i], qr[c][4 * i + 1], qr[c][4 * i + 2], qr[c][4 * i + 3]);
      }
    }
    tc::wait_st();
    tc::fence_async_smem();
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();

  float m = -INFINITY, l = 0.f;
  if (warp == kCopyWarp) {
    // ------------------------------------------------------------ copies: K0, then K(j+1), V(j)
    if (lane == 0) {
      const int n = 2 * n_tiles;
      bool ok = true;
      int i = 0;
      for (; i < n; ++i) {
        const int st = i % L::kRing;
        if (i >= L::kRing)
          ok = wait_bar(&empty[st], (uint32_t)((i / L::kRing - 1) & 1), abort, p.status, p.timeout_ns, 11);
        if (!ok) break;
        // order of use: K0, K1, V0, K2, V1, ..., V(n-1)
        const bool key = i == 0 || ((i & 1) && i != n - 1);
        const int j = key ? (i + 1) / 2 : (i - 1) / 2;
        mbar_arrive_expect_tx(&full[st], L::kImage);
        bulk_g2s(sm + L::kStages + st * L::kImage, images + ((int64_t)2 * j + (key ? 0 : 1)) * L::kImage, L::kImage, &full[st]);
      }
      for (int k = max(0, i - L::kRing); k < i; ++k)
        wait_bar(&full[k % L::kRing], (uint32_t)((k / L::kRing) & 1), &never, p.status, p.timeout_ns, 12);
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMAs
    if (n_tiles > 0 && elect_one()) {
      constexpr uint32_t kIdescS = tc::idesc_f16(128, kTileTokens) | (1u << 7) | (1u << 10);  // bf16 operands
      constexpr uint32_t kIdescO = tc::idesc_f16(128, D);
      const uint64_t qd = tc::smem_desc(smem_u32(sm + L::kQ), kRowsP * 16, 128);
      bool ok = true;
      auto landed = [&](int i) {
        ok = ok && wait_bar(&full[i % L::kRing], (uint32_t)((i / L::kRing) & 1), abort, p.status, p.timeout_ns, 13);
      };
      auto stored = [&](int j) {
        ok = ok && wait_bar<64>(&pfull[j & 1], (uint32_t)((j >> 1) & 1), abort, p.status, p.timeout_ns, 14);
      };
      auto scores = [&](int j, int i) {
        const uint64_t kd = tc::smem_desc(smem_u32(sm + L::kStages + i % L::kRing * L::kImage), kTileTokens * 16, 128);
        landed(i);
        if (!ok) return;
        tc::fence_after();
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint64_t kk = kd + k * (2 * kTileTokens * 16 / 16);
          if (16 * k < L::kTmemQ) tc::mma_ts(tbase + 128 * (j & 1), tbase + 256 + D + 8 * k, kk, kIdescS, k > 0);
          else mma_ss(tbase + 128 * (j & 1), qd + (k - L::kTmemQ / 16) * (2 * kRowsP * 16 / 16), kk, kIdescS, k > 0);
        }
        tc::commit(&sfull[j & 1]);
        tc::commit(&empty[i % L::kRing]);
      };
      int i = 0;  // images used
      scores(0, i++);
      for (int j = 0; j < n_tiles && ok; ++j) {
        if (j + 1 < n_tiles) scores(j + 1, i++);
        const uint64_t vd = tc::smem_desc(smem_u32(sm + L::kStages + i % L::kRing * L::kImage), D * 16, 128);
        landed(i);
        stored(j);
        if (!ok) break;
        tc::fence_after();
#pragma unroll
        for (int k = 0; k < kTileTokens / 16; ++k)
          tc::mma_ts(tbase + 256, tbase + 128 * (j & 1) + 8 * k, vd + k * (2 * D * 16 / 16), kIdescO, j > 0 || k > 0);
        tc::commit(&odone[j & 1]);
        tc::commit(&empty[i % L::kRing]);
        ++i;
      }
      // all MMAs issued are complete before the block frees anything
      tc::commit(fin);
      wait_bar(fin, 0, &never, p.status, p.timeout_ns, 15);
    }
  } else if (n_tiles > 0) {
    // ------------------------------------------------------------ softmax
    const uint32_t tl = tbase + ((uint32_t)(warp & 3) << 21);  // this warp's 32 lanes
    using Bits = KeyBits<kShareKeys>;
    const Bits* exist_words = reinterpret_cast<const Bits*>(valid) + share;
    Bits ahead = __ldcg(exist_words);  // read a tile early: it waits for L2
    softmax_tiles<D, kShareKeys, kShares>(
        p, n_tiles, tl, share, row, kRowsP, smax, sfull, pfull, odone, abort, m, l, [&](int j, Bits& bits) {
          const int c0 = (tile_a + j) * kTileTokens;
          const Bits exist = ahead;
          if (j + 1 < n_tiles) ahead = __ldcg(exist_words + (j + 1) * kShares);
          if (c0 + kTileTokens <= pos_min + 1 && c0 >= lo_max && exist == ~Bits(0)) return false;
          bits = key_bits<kShareKeys>(c0 + kShareKeys * share, lo_r, hi_r) & exist;
          return true;
        });
  }
  // the shares' sums
  __syncthreads();
  if (warp < kSoftWarps) smax[share * kRowsP + row] = l;
  __syncthreads();
  if (warp < kSoftWarps) {
    l = 0.f;
#pragma unroll
    for (int i = 0; i < kShares; ++i) l += smax[i * kRowsP + row];
    const uint32_t tl = tbase + ((uint32_t)(warp & 3) << 21);
    const int64_t orow = (int64_t)(s.start + tq) * p.hq + hq;
    const int64_t part = ((int64_t)(tile_i - whole) * p.n_split + split) * kRowsP + row;
    const float inv = parts ? 1.f : (l > 0.f ? kValueUnscale / l : 0.f);
#pragma unroll 1
    for (int c = share * (D / kShares); c < (share + 1) * (D / kShares); c += 16) {
      uint32_t o[16];
      __syncwarp();
      if (n_tiles > 0) {
        tc::ld_32x32b_x16(tl + 256 + c, o);
        tc::wait_ld();
      }
      store_out16(p, parts, o, l, inv, has_row, part, orow, c, D);
    }
    if (has_row && share == 0) {
      if (parts) p.part_ml[part] = make_float2(m, l);
      else if (p.lse) p.lse[orow] = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
    }
    tc::fence_before();
  }
  __syncthreads();
  tc::fence_after();
  if (warp == kMmaWarp) tc::dealloc_512(tbase);
}

template <int D>
cudaError_t prompt_launch_d(AttnParams p, int num_sms, size_t part_rows, uint8_t* ws, int tile_cap, cudaStream_t st) {
  const int n_rt = (int)(((int64_t)p.max_q * p.g + kRowsP - 1) / kRowsP);
  int64_t span = p.max_len;
  if (p.window > 0) span = std::min<int64_t>(span, (int64_t)p.window + p.max_q + 2 * kTileTokens);
  Images im;
  im.tiles = (int)((span + kTileTokens - 1) / kTileTokens);
  const int at_once = std::max(1, std::min(p.n_seqs, tile_cap / (p.hk * im.tiles)));
  im.base = ws;
  im.valid = reinterpret_cast<uint4*>(ws + (size_t)tile_cap * 2 * PromptPlan<D>::kImage);
  // tiles of one row tile's keys: its window's, or all
  int64_t rspan = p.max_len;
  if (p.window > 0) rspan = std::min<int64_t>(rspan, (int64_t)p.window + kRowsP + kTileTokens);
  const int rtiles = (int)((rspan + kTileTokens - 1) / kTileTokens);
  const int all = p.n_seqs;
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
    const int64_t total = (int64_t)p.hk * n_rt * g.n_seqs, whole = total / num_sms * num_sms, rest = total - whole;
    int64_t best = 0;
    int chunk = rtiles;
    g.n_split = 1;
    for (int n = 1; rest > 0 && n <= std::min(kMaxSplit, std::max(1, rtiles / 2)); ++n) {
      if (n > 1 && rest * n * kRowsP > (int64_t)part_rows) break;
      const int c = (rtiles + n - 1) / n;
      const int64_t cost = (rest * n + num_sms - 1) / num_sms * (c + 4) + (n > 1 ? 4 : 0);
      if (n == 1 || cost < best) best = cost, chunk = c, g.n_split = (rtiles + c - 1) / c;
    }
    cudaError_t e = launch_pdl(expand_kernel, dim3(im.tiles, p.hk, g.n_seqs), 256, 0, st, g, im);
    if (e == cudaSuccess)
      e = launch_pdl(prompt_kernel<D>, dim3((unsigned)(whole + rest * g.n_split)), kPromptThreads, PromptPlan<D>::kTotal, st, g, im,
                     n_rt, (int)whole, chunk);
    if (e == cudaSuccess && g.n_split > 1) e = join_launch(g, kRowsP, n_rt, (int)whole, st);
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

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
// 1850 instead of 800.
#include "attn_tc.cuh"

namespace moe {
namespace attn {

cudaError_t join_launch(const AttnParams& p, int rows_per_tile, int n_rt, cudaStream_t st);

namespace {

constexpr int kRowsV = 64;
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
  static constexpr int kMax = kV + 2 * kImage;                 // float [2][4][64] (the sums and references need 5 x 64)
  // [8 tiles][16]: a byte for each 8 keys that exist (written up to 4 tiles before the softmax reads it)
  static constexpr int kHere = kMax + 2 * 4 * kRowsV * 4;
  static constexpr int kBars = kHere + 8 * 16;
  static constexpr int kNumBars = 8 + 2 + 2 + 2 + 2;
  static constexpr int kMisc = kBars + kNumBars * 8;           // tensor memory slot, abort
  static constexpr int kTotal = kMisc + 16 + 128;
  static_assert(kTotal <= 232448, "shared memory plan");
  static constexpr int kPitch = D * 4 + 16;  // of an output row on its way out, over the images
  static_assert(kRowsV * kPitch <= kMax, "the output fits the images' room");
};

template <int D>
__global__ void __launch_bounds__(kThreadsV, 1) verify_kernel(const __grid_constant__ AttnParams p, int n_rt, int chunk) {
  using L = VerifyPlan<D>;
  constexpr int KT = L::KT, QC = KT / 4;  // keys of a softmax thread
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  float* smax = reinterpret_cast<float*>(sm + L::kMax);
  uint8_t* here = sm + L::kHere;
  uint64_t* kfull = reinterpret_cast<uint64_t*>(sm + L::kBars);  // [2] key image written
  uint64_t* kfree = kfull + 2;                                    // [2] scores' products from it done
  uint64_t* vfull = kfree + 2;                                    // [2] value image written
  uint64_t* vfree = vfull + 2;                                    // [2] output products from it done
  uint64_t* sfull = vfree + 2;                                    // [2] scores ready
  uint64_t* pfull = sfull + 2;                                    // [2] weights stored (the softmax may be a tile ahead)
  uint64_t* xbar = pfull + 2;                                     // [2] maxima exchanged
  uint64_t* qfull = xbar + 2;                                     // queries written
  uint64_t* fin = qfull + 1;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + L::kMisc);
  volatile int* abort = reinterpret_cast<volatile int*>(sm + L::kMisc + 4);
  volatile int never = 0;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  griddep_launch_dependents();
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&kfull[i], 8);
      mbar_init(&kfree[i], 1);
      mbar_init(&vfull[i], 8);
      mbar_init(&vfree[i], 1);
      mbar_init(&sfull[i], 1);
      mbar_init(&pfull[i], 8);
      mbar_init(&xbar[i], 8);
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

  const int split = blockIdx.x, b = blockIdx.z;
  const int kvh = blockIdx.y / n_rt, rt = blockIdx.y % n_rt;
  const Seq s = load_seq(p, b);
  const int row0 = rt * kRowsV, n_rows = max(0, min(kRowsV, s.nq * p.g - row0));
  const int p0 = s.len - s.nq;
  const int pos_min = p0 + row0 / p.g, pos_max = p0 + (row0 + max(n_rows, 1) - 1) / p.g;
  const int lo = key_lo(p, max(0, pos_min)), hi = pos_max + 1, lo_max = key_lo(p, pos_max);
  const int tile_a = lo / KT + split * chunk;
  const int n_tiles = hi > lo && n_rows > 0 ? max(0, min(tile_a + chunk, (hi + KT - 1) / KT) - tile_a) : 0;

  const bool soft = warp < 16 && (warp & 3) < 2;
  const int row = (warp & 1) * 32 + lane, quarter = warp >> 2;  // of the softmax threads
  int tq = 0, hq = 0, hi_r = 0, lo_r = 0;
  const bool has_row = soft && row < n_rows;
  if (has_row) {
    tq = (row0 + row) / p.g;
    hq = kvh * p.g + (row0 + row) % p.g;
    hi_r = p0 + tq + 1;
    lo_r = key_lo(p, p0 + tq);
  }

  float m = -INFINITY, l = 0.f;
  if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMAs
    if (lane == 0 && n_tiles > 0) {
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
        tc::commit(&kfree[i]);
        tc::commit(&sfull[i]);
      };
      ok = wait_bar<64>(qfull, 0, abort, p.status, p.timeout_ns, 34);
      if (ok) scores(0);
      for (int j = 0; j < n_tiles && ok; ++j) {
        const int i = j & 1;
        if (j + 1 < n_tiles) scores(j + 1);
        ok = ok && wait_bar<64>(&vfull[i], (uint32_t)((j >> 1) & 1), abort, p.status, p.timeout_ns, 24);
        ok = ok && wait_bar<64>(&pfull[i], (uint32_t)((j >> 1) & 1), abort, p.status, p.timeout_ns, 25);
        if (!ok) break;
        tc::fence_after();
#pragma unroll
        for (int k = 0; k < KT / 16; ++k)
          tc::mma_ts(tbase + 256, tbase + 128 * i + 8 * k, vd + i * (L::kImage / 16) + k * (2 * 128 / 16), kIdescO, j > 0 || k > 0);
        tc::commit(&vfree[i]);
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
    uint64_t* image_full = values ? vfull : kfull;
    uint64_t* image_free = values ? vfree : kfree;
    uint8_t* image = sm + (values ? L::kV : L::kK);
    // a warp takes the key groups dw, dw + 8 (of 8 keys), of 64 channels at a
    // time: each 8 lanes 8 keys, so that their stores meet all banks
    const int k8 = lane & 7, c4 = lane >> 3;
    constexpr int kGroups = KT / 64, kUnits = kGroups * (D / 64);
    uint2 code[kUnits];
    uint32_t scale[kUnits];
    auto fetch = [&](int j) {  // this lane's codes and scales of tile j: 0 for a key past the end or on an absent page
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        const int g8 = dw + 8 * g, key = (tile_a + j) * KT + 8 * g8;
        // (a page that no row here sees is not looked at: it may have been given back)
        const int pg = j < n_tiles && key < hi && (key | (p.P - 1)) >= lo ? load_page(p, b, key >> p.pshift) : -1;
        const int at = (key & (p.P - 1)) + k8;
        const uint8_t* src = p.pages + pg * p.page_bytes + (int64_t)kvh * p.head_bytes + (values ? p.head_bytes / 2 : 0);
        const bool has = pg >= 0 && key + k8 < s.len;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          code[g * (D / 64) + c] = make_uint2(0, 0);
          scale[g * (D / 64) + c] = 0;
          if (has) {
            code[g * (D / 64) + c] = __ldcg(reinterpret_cast<const uint2*>(src + at * (D / 2) + 32 * c + 8 * c4));
            scale[g * (D / 64) + c] = __ldcg(src + codes + at * (D / 16) + 4 * c + c4);
          }
        }
        if (!values && lane == 0) here[(j & 7) * 16 + g8] = pg >= 0;
      }
    };
    fetch(0);
    for (int j = 0; j < n_tiles; ++j) {
      const int i = j & 1;
      bool ok = true;
      if (j > 1) ok = wait_bar(&image_free[i], (uint32_t)((j >> 1) - 1) & 1, abort, p.status, p.timeout_ns, 28);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      uint4* o = reinterpret_cast<uint4*>(image + i * L::kImage);
#pragma unroll
      for (int g = 0; g < kGroups; ++g)
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          const uint2 w = code[g * (D / 64) + c];
          const uint32_t sb = scale[g * (D / 64) + c] * 0x00010001u;
          uint32_t x[8];
          if (values) {
            const ValueScale d = value_scale(sb);
            value_quads(w.x, d, x[0], x[1], x[2], x[3]);
            value_quads(w.y, d, x[4], x[5], x[6], x[7]);
          } else {
            const KeyScale d = key_scale(sb);
            key_pairs(w.x, d, x);
            key_pairs(w.y, d, x + 4);
          }
          uint4* r = o + (8 * c + 2 * c4) * KT + 8 * (dw + 8 * g) + k8;
          r[0] = make_uint4(x[0], x[1], x[2], x[3]);
          r[KT] = make_uint4(x[4], x[5], x[6], x[7]);
        }
      tc::fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&image_full[i]);
      if (j + 1 < n_tiles) fetch(j + 1);
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
    bool ok = true;
    for (int j = 0; j < n_tiles; ++j) {
      ok = wait_bar(&sfull[j & 1], (uint32_t)((j >> 1) & 1), abort, p.status, p.timeout_ns, 30);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc::fence_after();
      uint32_t sv[QC / 16][16];
#pragma unroll
      for (int c = 0; c < QC / 16; ++c) tc::ld_32x32b_x16(tl + 128 * (j & 1) + QC * quarter + 16 * c, sv[c]);
      tc::wait_ld();
      float x[QC];
#pragma unroll
      for (int c = 0; c < QC; ++c) x[c] = __uint_as_float(sv[c >> 4][c & 15]);
      const int c0 = (tile_a + j) * KT;
      // the existing 8-key groups of this quarter, a byte each
      uint32_t mask;
      if constexpr (QC == 32) mask = *reinterpret_cast<const volatile uint32_t*>(here + (j & 7) * 16 + 4 * quarter);
      else mask = *reinterpret_cast<const volatile uint16_t*>(here + (j & 7) * 16 + 2 * quarter);
      if (c0 + KT > pos_min + 1 || c0 < lo_max || mask != (0x01010101u >> (32 - QC))) {
        // bit c: key c0 + QC quarter + c is visible to this row
        const int k0 = c0 + QC * quarter;
        uint32_t vis = 0xffffffffu;
        const int a = lo_r - k0, e = hi_r - k0;
        vis &= e >= 32 ? ~0u : (e <= 0 ? 0u : (1u << e) - 1);
        vis &= a <= 0 ? ~0u : (a >= 32 ? 0u : ~((1u << a) - 1));
#pragma unroll
        for (int c = 0; c < QC; ++c) {
          const bool page = (mask >> (c & ~7)) & 1;
          if (!((vis >> c) & 1) || !page) x[c] = -INFINITY;
        }
      }
      float mx = x[0];
#pragma unroll
      for (int c = 1; c < QC; ++c) mx = fmaxf(mx, x[c]);
      // the row's other quarters
      float* ex = smax + (j & 1) * 4 * kRowsV;
      ex[quarter * kRowsV + row] = mx;
      __syncwarp();
      if (lane == 0) mbar_arrive(&xbar[j & 1]);
      ok = wait_bar(&xbar[j & 1], (uint32_t)((j >> 1) & 1), abort, p.status, p.timeout_ns, 31);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
#pragma unroll
      for (int i = 0; i < 4; ++i) mx = fmaxf(mx, ex[i * kRowsV + row]);
      mx *= p.scale_log2;
      const bool move = mx > m + kLazy;  // (also the first visible keys: m = -inf)
      if (__any_sync(0xffffffffu, move)) {
        const float f = move ? (m == -INFINITY ? 0.f : exp2_approx(m - mx)) : 1.f;
        if (move) m = mx;
        l *= f;
        if (j > 0) {
          ok = wait_bar(&vfree[(j - 1) & 1], (uint32_t)(((j - 1) >> 1) & 1), abort, p.status, p.timeout_ns, 32);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc::fence_after();
#pragma unroll 1
          for (int c = quarter * (D / 4); c < (quarter + 1) * (D / 4); c += 16) {
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
      st_cols<QC / 2>(tl + 128 * (j & 1) + QC / 2 * quarter, pk);
      tc::wait_st();
      tc::fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&pfull[j & 1]);
    }
    if (ok) {
      ok = wait_bar(&vfree[(n_tiles - 1) & 1], (uint32_t)(((n_tiles - 1) >> 1) & 1), abort, p.status, p.timeout_ns, 33);
      ok = __all_sync(0xffffffffu, ok);
      tc::fence_after();
    }
  }
  // the quarters' sums; the outputs go through shared memory (the images'
  // room), since a thread's row is D apart from its neighbour's: stored from
  // the accumulator's layout they took 5 us
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (soft) smax[quarter * kRowsV + row] = l;
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
    if (quarter == 0) smax[4 * kRowsV + row] = m;
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == kMmaWarp) tc::dealloc_512(tbase);
  const int64_t part0 = ((int64_t)(b * p.hk * n_rt + blockIdx.y) * p.n_split + split) * kRowsV;
  for (int i = tid; i < n_rows * (D / 4); i += kThreadsV) {
    const int r = i / (D / 4), c = i % (D / 4);
    float lt = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) lt += smax[k * kRowsV + r];
    const float mr = n_tiles > 0 ? smax[4 * kRowsV + r] : -INFINITY;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (lt > 0.f) v = *reinterpret_cast<const float4*>(sm + r * L::kPitch + c * 16);
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
  int64_t span = p.max_len;  // keys a row tile can see: the window's, or all
  if (p.window > 0) span = std::min<int64_t>(span, (int64_t)p.window + p.max_q + KT);
  const int tiles = (int)((span + KT - 1) / KT);
  // one block a multiprocessor; at least two tiles a block
  int64_t want = std::max<int64_t>(1, num_sms / base);
  want = std::min<int64_t>(std::min<int64_t>(want, kMaxSplit), std::max<int64_t>(1, (int64_t)(part_rows / kRowsV) / base));
  const int chunk = (int)std::max<int64_t>(std::min(tiles, 2), (tiles + want - 1) / want);
  p.n_split = (tiles + chunk - 1) / chunk;
  cudaError_t e = launch_pdl(verify_kernel<D>, dim3(p.n_split, (unsigned)(p.hk * n_rt), p.n_seqs), kThreadsV,
                             VerifyPlan<D>::kTotal, st, p, n_rt, chunk);
  if (e != cudaSuccess || p.n_split == 1) return e;
  return join_launch(p, kRowsV, n_rt, st);
}

}  // namespace

cudaError_t verify_configure(int D) {
  const auto set = [](const void* f, int bytes) { return cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes); };
  switch (D) {
    case 64: return set((const void*)verify_kernel<64>, VerifyPlan<64>::kTotal);
    case 128: return set((const void*)verify_kernel<128>, VerifyPlan<128>::kTotal);
    case 192: return set((const void*)verify_kernel<192>, VerifyPlan<192>::kTotal);
    default: return set((const void*)verify_kernel<256>, VerifyPlan<256>::kTotal);
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

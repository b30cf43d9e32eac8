// attn_small.cu -- attention of few query rows (single tokens, small verify
// batches) over the 4-bit paged cache: at most 16 rows (query token, query
// head) of a key/value head a block, bound by reading the cache once.
//
//   o = sum_j 2^(s_j - m) v_j / sum_j 2^(s_j - m),  s_j = log2(e) scale q.k_j,
// in one pass over the keys with a running maximum m, sum l and output, split
// over blocks along the keys and over the 4 compute warps inside a block (32
// keys of each 128-key tile a warp); the parts are joined by their m and l.
//
// Whole (page, head) blocks (codes and scales of keys and values lie
// together, one bulk copy each) are copied into a ring of 128-key stages.
// The warps dequantise straight into the operand registers of m16n8k16 MMAs
// (no shared-memory round trip for 16-bit values), exactly:
//   scores: A = 16 query rows (held in registers), B = keys.  The channel
//     order inside an MMA's k is free as long as both operands agree: lane
//     (n, t) of the 8x4 grid takes channels 64 j + 16 t .. + 15 of key n,
//     two words that share one scale.
//   output: A = weights (the score accumulators as they lie, rounded to
//     fp16), B = values; lane (n, t) takes word n of 64 channels of the keys
//     at k = 2t, 2t+1, 2t+8, 2t+9, and two words interleave to pairs of keys
//     before dequantisation.
// Slot n of 8 keys is key kKey(n) = 0,6,1,7,2,4,3,5: then both access patterns
// meet all banks at 192 and 64 channels.
//
// Per 128 keys of D = 192 a block issues ~3900 instructions and 768 MMAs,
// against 27.6 KB of HBM: both near the memory's time.
#include "attn_mma.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kSmallWarps = 4;
constexpr int kSmallThreads = kSmallWarps * 32;
constexpr int kSmallRows = 16;
constexpr int kSmallTile = 128;
constexpr int kSmallMaxStages = 8;

template <int D>
struct SmallPlan {
  static constexpr int kStage = kSmallTile * D * 9 / 8;
  static constexpr int kStages = D == 64 ? 8 : (D == 128 ? 5 : 3);
  static constexpr int kBars = kStages * kStage;
  static constexpr int kTotal = kBars + 2 * kSmallMaxStages * 8 + kSmallMaxStages * 4 + 16 + kSmallWarps * kSmallRows * 8;
  static_assert(kSmallWarps * kSmallRows * D * 4 <= kBars, "the warps' outputs reuse the ring");
};

template <int D>
__global__ void __launch_bounds__(kSmallThreads, 2) small_kernel(const __grid_constant__ AttnParams p, int n_rt, int chunk) {
  using L = SmallPlan<D>;
  constexpr int kJ = D / 64;
  extern __shared__ __align__(128) uint8_t smem[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBars);
  uint64_t* empty = full + kSmallMaxStages;
  volatile uint32_t* pmask = reinterpret_cast<uint32_t*>(empty + kSmallMaxStages);  // pages present of a stage
  volatile int* abort = reinterpret_cast<int*>(smem + L::kBars + 2 * kSmallMaxStages * 8 + kSmallMaxStages * 4);
  float2* ml = reinterpret_cast<float2*>(smem + L::kBars + 2 * kSmallMaxStages * 8 + kSmallMaxStages * 4 + 16);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int never = 0;
  griddep_launch_dependents();
  if (tid == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kSmallWarps);
    }
    *abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  griddep_wait();

  const int split = blockIdx.x, b = blockIdx.z;
  const int kvh = blockIdx.y / n_rt, rt = blockIdx.y % n_rt;
  const Seq s = load_seq(p, b);
  const int row0 = rt * kSmallRows, n_rows = min(kSmallRows, s.nq * p.g - row0);
  if (n_rows <= 0) return;  // (the whole block; every thread has passed its dependency wait)
  // keys that some row sees, and this block's tiles of them
  const int p0 = s.len - s.nq;  // position of the first query
  const int pos_min = p0 + row0 / p.g, pos_max = p0 + (row0 + n_rows - 1) / p.g;
  const int lo = key_lo(p, pos_min), hi = pos_max + 1;
  const int tile_a = lo / kSmallTile + split * chunk;
  const int tile_b = min(tile_a + chunk, (max(hi, 0) + kSmallTile - 1) / kSmallTile);
  const int n_tiles = hi > lo ? max(0, tile_b - tile_a) : 0;
  const int ppt = kSmallTile >> p.pshift;  // pages of a tile

  // Warp 0 issues the copies too (a fifth warp would cost the compute warps a
  // third of their registers): lane i takes page i of a tile.
  const uint64_t pol = l2_evict_first_policy();
  auto page_of = [&](int i) {  // -1 where nothing of the page is seen
    const int pi = (tile_a + i) * ppt + lane, j0 = pi << p.pshift;
    return lane < ppt && i < n_tiles && j0 < hi && j0 + p.P > lo ? load_page(p, b, pi) : -1;
  };
  auto issue = [&](int i, int pg) {
    const int st = i % L::kStages;
    const uint32_t mask = __ballot_sync(0xffffffffu, pg >= 0);
    if (lane == 0) {
      pmask[st] = mask;
      mbar_arrive_expect_tx(&full[st], (uint32_t)(__popc(mask) * p.head_bytes));
    }
    __syncwarp();
    if (pg >= 0)
      bulk_g2s_hint(smem + st * L::kStage + lane * p.head_bytes, p.pages + pg * p.page_bytes + kvh * p.head_bytes,
                    (uint32_t)p.head_bytes, &full[st], pol);
  };
  int issued = 0, next_pg = -1;
  if (warp == 0) {
    int pg[L::kStages - 1];
#pragma unroll
    for (int i = 0; i < L::kStages - 1; ++i) pg[i] = page_of(i);
    next_pg = page_of(L::kStages - 1);
#pragma unroll
    for (int i = 0; i < L::kStages - 1; ++i)
      if (i < n_tiles) issue(i, pg[i]), ++issued;
  }
  {
    // ------------------------------------------------------------ compute
    const int n = lane >> 2, t = lane & 3;
    const int key_n = (n >> 1) + ((n & 1) ? (((n >> 1) + 2) & 3) + 4 - (n >> 1) : 0);  // kKey(n)
    const int key_e = t, key_o = 4 + ((t + 2) & 3);                                     // kKey(2t), kKey(2t + 1)
    // query rows n and n + 8, channels 64 j + 16 t .. + 15
    uint32_t aq[4 * kJ][4];
    int hi_r[2], lo_r[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = row0 + n + 8 * r;
      const bool valid = n + 8 * r < n_rows;
      const int tq = valid ? row / p.g : 0, h = kvh * p.g + (valid ? row % p.g : 0);
      hi_r[r] = valid ? p0 + tq + 1 : 0;
      lo_r[r] = valid ? key_lo(p, p0 + tq) : 0;
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + (s.start + tq) * p.q_tok + h * p.q_head;
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
        uint4 x = make_uint4(0, 0, 0, 0), y = x;
        if (valid) {
          x = *reinterpret_cast<const uint4*>(q + 64 * j + 16 * t);
          y = *reinterpret_cast<const uint4*>(q + 64 * j + 16 * t + 8);
        }
        aq[4 * j][r] = x.x; aq[4 * j][2 + r] = x.y;
        aq[4 * j + 1][r] = x.z; aq[4 * j + 1][2 + r] = x.w;
        aq[4 * j + 2][r] = y.x; aq[4 * j + 2][2 + r] = y.y;
        aq[4 * j + 3][r] = y.z; aq[4 * j + 3][2 + r] = y.w;
      }
    }
    const int lo_max = key_lo(p, pos_max);
    float o[8 * kJ][4];
#pragma unroll
    for (int i = 0; i < 8 * kJ; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    const int code_b = p.P * (D / 2), half_b = (int)(p.head_bytes / 2);

    for (int i = 0; i < n_tiles; ++i) {
      const int st = i % L::kStages;
      bool ok = true;
      if (warp == 0 && issued < n_tiles) {  // the stage of tile i - 1 is free once every warp is past it
        const int pg = next_pg;
        next_pg = page_of(issued + 1);
        if (issued >= L::kStages)
          ok = wait_bar(&empty[issued % L::kStages], (uint32_t)((issued / L::kStages - 1) & 1), abort, p.status,
                        p.timeout_ns, 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        issue(issued, pg);
        ++issued;
      }
      ok = wait_bar(&full[st], (uint32_t)((i / L::kStages) & 1), abort, p.status, p.timeout_ns, 2);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const uint32_t mask = pmask[st];
      const int c0 = (tile_a + i) * kSmallTile + warp * 32;  // this warp's first key
      if (c0 < hi && c0 + 32 > lo) {
        const uint8_t* ring = smem + st * L::kStage;
        // the 8-key group at key k of the tile lies in one page
        auto group = [&](int k, int& at) {
          at = k & (p.P - 1);
          return ring + (k >> p.pshift) * p.head_bytes;
        };
        float sc[4][4];
#pragma unroll
        for (int a = 0; a < 4; ++a) {
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[a][e] = 0.f;
          int at;
          const uint8_t* base = group(warp * 32 + 8 * a, at);
          const uint8_t* kc = base + (at + key_n) * (D / 2) + 8 * t;
          const uint8_t* ks = base + code_b + (at + key_n) * (D / 16);
#pragma unroll
          for (int j = 0; j < kJ; ++j) {
            const uint2 w = *reinterpret_cast<const uint2*>(kc + 32 * j);
            const uint32_t sw = *reinterpret_cast<const uint32_t*>(ks + 4 * j);
            const KeyScale d = key_scale(__byte_perm(sw, 0, 0x4040 + t * 0x0101));
            uint32_t k[8];
            key_pairs(w.x, d, k);
            key_pairs(w.y, d, k + 4);
#pragma unroll
            for (int c = 0; c < 4; ++c) mma_bf16(sc[a], aq[4 * j + c], k[2 * c], k[2 * c + 1]);
          }
        }
        // masks: past the last or before the first visible key, on absent pages
        const uint32_t need = ppt == 32 ? 0xffffffffu : (1u << ppt) - 1u;
        const bool partial = c0 + 32 > pos_min + 1 || c0 < lo_max || mask != need;
        if (partial) {
#pragma unroll
          for (int a = 0; a < 4; ++a) {
            const bool page = (mask >> ((warp * 32 + 8 * a) >> p.pshift)) & 1;
            const int j0 = c0 + 8 * a + key_e, j1 = c0 + 8 * a + key_o;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              if (!page || j0 >= hi_r[r] || j0 < lo_r[r]) sc[a][2 * r] = -INFINITY;
              if (!page || j1 >= hi_r[r] || j1 < lo_r[r]) sc[a][2 * r + 1] = -INFINITY;
            }
          }
        }
        float mn[2];
        bool grows = false;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float x = fmaxf(sc[0][2 * r], sc[0][2 * r + 1]);
#pragma unroll
          for (int a = 1; a < 4; ++a) x = fmaxf(x, fmaxf(sc[a][2 * r], sc[a][2 * r + 1]));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
          mn[r] = fmaxf(m[r], x * p.scale_log2);
          grows |= mn[r] > m[r];
        }
        if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float f = m[r] == -INFINITY ? 0.f : exp2_approx(m[r] - mn[r]);
            m[r] = mn[r];
            l[r] *= f;
#pragma unroll
            for (int k = 0; k < 8 * kJ; ++k) {
              o[k][2 * r] *= f;
              o[k][2 * r + 1] *= f;
            }
          }
        }
        uint32_t pr[4][2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float ref = m[r] == -INFINITY ? 0.f : m[r];  // a row that has seen nothing: all weights 0
#pragma unroll
          for (int a = 0; a < 4; ++a) {
            const float x = exp2_approx(fmaf(sc[a][2 * r], p.scale_log2, -ref));
            const float y = exp2_approx(fmaf(sc[a][2 * r + 1], p.scale_log2, -ref));
            l[r] += x + y;
            pr[a][r] = pack_h2(x, y);
          }
        }
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
          const uint32_t ap[4] = {pr[2 * kk][0], pr[2 * kk][1], pr[2 * kk + 1][0], pr[2 * kk + 1][1]};
          int at;
          const uint8_t* base = group(warp * 32 + 16 * kk, at) + half_b;  // 16 keys lie in one page
          const uint8_t* vc = base + at * (D / 2) + 4 * n;
          const uint8_t* vs = base + code_b + at * (D / 16);
          // scales of keys past the end or on absent pages are 0: whatever lies there stays finite
          bool z[4] = {false, false, false, false};
          if (partial) {
            const bool page = (mask >> ((warp * 32 + 16 * kk) >> p.pshift)) & 1;
            const int j = c0 + 16 * kk;
            z[0] = !page || j + key_e >= s.len;
            z[1] = !page || j + key_o >= s.len;
            z[2] = !page || j + 8 + key_e >= s.len;
            z[3] = !page || j + 8 + key_o >= s.len;
          }
#pragma unroll
          for (int j = 0; j < kJ; ++j) {
            uint32_t bb[2][8];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const int ke = 8 * u + key_e, ko = 8 * u + key_o;
              const uint32_t w0 = *reinterpret_cast<const uint32_t*>(vc + ke * (D / 2) + 32 * j);
              const uint32_t w1 = *reinterpret_cast<const uint32_t*>(vc + ko * (D / 2) + 32 * j);
              uint32_t s0 = *reinterpret_cast<const uint32_t*>(vs + ke * (D / 16) + 4 * j);
              uint32_t s1 = *reinterpret_cast<const uint32_t*>(vs + ko * (D / 16) + 4 * j);
              if (z[2 * u]) s0 = 0;
              if (z[2 * u + 1]) s1 = 0;
              const uint32_t h = n >> 1;
              const ValueScale d = value_scale(__byte_perm(s0, s1, h | ((4 + h) << 8)) & 0x00FF00FFu);
              value_quads(__byte_perm(w0, w1, 0x5410), d, bb[u][0], bb[u][2], bb[u][4], bb[u][6]);
              value_quads(__byte_perm(w0, w1, 0x7632), d, bb[u][1], bb[u][3], bb[u][5], bb[u][7]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) mma_f16(o[8 * j + e], ap, bb[0][e], bb[1][e]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
    }
    // this warp's part
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      if (t == 0) ml[warp * kSmallRows + n + 8 * r] = make_float2(m[r], l[r]);
    }
    // every copy issued has landed before the ring is reused (they all have, unless a wait gave up)
    if (warp == 0)
      for (int j = max(0, issued - L::kStages); j < issued; ++j)
        wait_bar(&full[j % L::kStages], (uint32_t)((j / L::kStages) & 1), &never, p.status, p.timeout_ns, 3);
    __syncthreads();  // every warp has read its last stage
    float* ob = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
        float* d = ob + (warp * kSmallRows + n + 8 * r) * D + 64 * j + 16 * t;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          d[e] = o[8 * j + e][2 * r];
          d[8 + e] = o[8 * j + e][2 * r + 1];
        }
      }
  }
  __syncthreads();
  // join the warps' parts
  const int64_t part = ((int64_t)(b * p.hk * n_rt + blockIdx.y) * p.n_split + split) * kSmallRows;
  const float* ob = reinterpret_cast<const float*>(smem);
  for (int i = tid; i < n_rows * (D / 4); i += kSmallThreads) {
    const int r = i / (D / 4), c = 4 * (i % (D / 4));
    float mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < kSmallWarps; ++w) mx = fmaxf(mx, ml[w * kSmallRows + r].x);
    float lt = 0.f, x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kSmallWarps; ++w) {
      const float2 a = ml[w * kSmallRows + r];
      const float f = a.x == -INFINITY ? 0.f : exp2_approx(a.x - mx);
      const float4 v = *reinterpret_cast<const float4*>(ob + (w * kSmallRows + r) * D + c);
      lt = fmaf(a.y, f, lt);
      x[0] = fmaf(v.x, f, x[0]);
      x[1] = fmaf(v.y, f, x[1]);
      x[2] = fmaf(v.z, f, x[2]);
      x[3] = fmaf(v.w, f, x[3]);
    }
    if (p.n_split == 1) {
      const float inv = lt > 0.f ? kValueUnscale / lt : 0.f;
      const int row = row0 + r, tok = s.start + row / p.g, h = kvh * p.g + row % p.g;
      const __nv_bfloat162 u = __floats2bfloat162_rn(x[0] * inv, x[1] * inv), v = __floats2bfloat162_rn(x[2] * inv, x[3] * inv);
      uint2 w;
      w.x = *reinterpret_cast<const uint32_t*>(&u);
      w.y = *reinterpret_cast<const uint32_t*>(&v);
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + ((int64_t)tok * p.hq + h) * D + c) = w;
      if (p.lse && c == 0)
        p.lse[(int64_t)tok * p.hq + h] = lt > 0.f ? (mx + log2f(lt)) * 0.69314718055994531f : -INFINITY;
    } else {
      if (c == 0) p.part_ml[part + r] = make_float2(mx, lt);
      *reinterpret_cast<float4*>(p.part_o + (part + r) * D + c) = make_float4(x[0], x[1], x[2], x[3]);
    }
  }
}

// Joins the parts of a row's keys: one block a (query token, query head).
template <int D>
__global__ void __launch_bounds__(D) join_kernel(const __grid_constant__ AttnParams p, int rows_per_tile, int n_rt) {
  griddep_launch_dependents();
  griddep_wait();
  const int t = blockIdx.x / p.hq, h = blockIdx.x % p.hq, b = blockIdx.y;
  const Seq s = load_seq(p, b);
  if (t >= s.nq) return;
  const int kvh = h / p.g, row = t * p.g + h % p.g;
  const int64_t tile = (int64_t)(b * p.hk + kvh) * n_rt + row / rows_per_tile;
  const int64_t first = tile * p.n_split * rows_per_tile + row % rows_per_tile;
  float mx = -INFINITY;
  for (int i = 0; i < p.n_split; ++i) mx = fmaxf(mx, p.part_ml[first + (int64_t)i * rows_per_tile].x);
  float lt = 0.f, x = 0.f;
#pragma unroll 4
  for (int i = 0; i < p.n_split; ++i) {
    const float2 a = p.part_ml[first + (int64_t)i * rows_per_tile];
    const float v = p.part_o[(first + (int64_t)i * rows_per_tile) * D + threadIdx.x];
    const float f = a.x == -INFINITY ? 0.f : exp2_approx(a.x - mx);
    lt = fmaf(a.y, f, lt);
    x = fmaf(v, f, x);
  }
  const int64_t o = (int64_t)(s.start + t) * p.hq + h;
  static_cast<__nv_bfloat16*>(p.out)[o * D + threadIdx.x] = __float2bfloat16_rn(lt > 0.f ? x * kValueUnscale / lt : 0.f);
  if (p.lse && threadIdx.x == 0) p.lse[o] = lt > 0.f ? (mx + log2f(lt)) * 0.69314718055994531f : -INFINITY;
}

}  // namespace

cudaError_t join_launch(const AttnParams& p, int rows_per_tile, int n_rt, cudaStream_t st) {
  const dim3 grid((unsigned)(p.max_q * p.hq), p.n_seqs);
  switch (p.D) {
    case 64: return launch_pdl(join_kernel<64>, grid, 64, 0, st, p, rows_per_tile, n_rt);
    case 128: return launch_pdl(join_kernel<128>, grid, 128, 0, st, p, rows_per_tile, n_rt);
    case 192: return launch_pdl(join_kernel<192>, grid, 192, 0, st, p, rows_per_tile, n_rt);
    default: return launch_pdl(join_kernel<256>, grid, 256, 0, st, p, rows_per_tile, n_rt);
  }
}

namespace {

template <int D>
cudaError_t small_launch_d(AttnParams p, int num_sms, size_t part_rows, cudaStream_t st) {
  const int n_rt = (p.max_q * p.g + kSmallRows - 1) / kSmallRows;
  const int64_t base = (int64_t)p.hk * n_rt * p.n_seqs;
  // tiles that a row can see: the window's, or all
  int64_t span = p.max_len;
  if (p.window > 0) span = std::min<int64_t>(span, (int64_t)p.window + p.max_q + kSmallTile);
  const int tiles = (int)((span + kSmallTile - 1) / kSmallTile);
  // keys are split until there are four blocks for each place on the GPU (two
  // a multiprocessor), so that ragged lengths even out
  const int64_t want = std::max<int64_t>(1, 8LL * num_sms / base);
  int chunk = (int)std::max<int64_t>(1, (tiles + want - 1) / want);
  const int64_t fit = std::max<int64_t>(1, (int64_t)(part_rows / kSmallRows) / base);
  chunk = std::max<int>(chunk, (int)((tiles + fit - 1) / fit));
  p.n_split = (tiles + chunk - 1) / chunk;
  cudaError_t e = launch_pdl(small_kernel<D>, dim3(p.n_split, (unsigned)(p.hk * n_rt), p.n_seqs), kSmallThreads,
                             SmallPlan<D>::kTotal, st, p, n_rt, chunk);
  if (e != cudaSuccess || p.n_split == 1) return e;
  return join_launch(p, kSmallRows, n_rt, st);
}

}  // namespace

cudaError_t small_configure() {
  cudaError_t e = cudaFuncSetAttribute(small_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize, SmallPlan<64>::kTotal);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(small_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize, SmallPlan<128>::kTotal);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(small_kernel<192>, cudaFuncAttributeMaxDynamicSharedMemorySize, SmallPlan<192>::kTotal);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(small_kernel<256>, cudaFuncAttributeMaxDynamicSharedMemorySize, SmallPlan<256>::kTotal);
  return e;
}

cudaError_t small_launch(const AttnParams& p, int num_sms, size_t part_rows, cudaStream_t st) {
  switch (p.D) {
    case 64: return small_launch_d<64>(p, num_sms, part_rows, st);
    case 128: return small_launch_d<128>(p, num_sms, part_rows, st);
    case 192: return small_launch_d<192>(p, num_sms, part_rows, st);
    default: return small_launch_d<256>(p, num_sms, part_rows, st);
  }
}

}  // namespace attn
}  // namespace moe

// attn_small.cu -- attention of few query rows (single tokens, small verify
// batches) over the 4-bit paged cache: at most 16 rows (query token, query
// head) of a key/value head a block, bound by reading the cache once.
//
//   o = sum_j 2^(s_j - m) v_j / sum_j 2^(s_j - m),  s_j = log2(e) scale q.k_j,
// in one pass over the keys with a running maximum m, sum l and output, split
// over blocks along the keys and over the 4 warps of a block (32 keys of each
// 128-key tile a warp); the parts are joined by their m and l.
//
// Whole (page, head) blocks (codes and scales of keys and values lie
// together, one bulk copy each) are copied into a ring of 128-key stages.
// The warps dequantise straight into the operand registers of m16n8k16 MMAs
// (no shared-memory round trip for 16-bit values), exactly.  Keys and values
// are the wide operand (M = 16), the query rows the narrow one (N = 8, or two
// of them): with the rows as M a single token of 4 query heads would waste
// three quarters of the products, the weights and the accumulators' registers.
//   scores: A = 16 keys, B = query rows (in registers).  The channel order
//     inside an MMA's k is free as long as both operands agree: lane (n, t) of
//     the 8x4 grid takes channels 64 j + 16 t .. + 15 of key n, two words that
//     share one scale.
//   output: A = 16 channels of 16 keys' values, B = weights, rounded to fp16
//     and transposed in registers.  Lane (n, t) takes word n of 64 channels of
//     the keys at k = 2t, 2t+1, 2t+8, 2t+9; two words interleave to pairs of
//     keys before dequantisation.
// Measured: 32 sequences of up to 8192 keys, 32/8 heads of 128, in 75 us, 3.0
// TB/s: issue slots are 61% busy (a 32-bit word of codes takes some 10
// instructions to 8 operands, twice for each row tile), the tensor pipe 16%;
// of up to 8000 keys, 64/4 heads of 192 (16 rows), in 76.5 us (the bytes take 24).
// One token over 257 keys takes 8.0 us: two launches and one chain of loads.
// Slot n of 8 keys is key kKey(n) = 0,6,1,7,2,4,3,5: then both access patterns
// meet all banks at 192 and 64 channels.
#include "attn_mma.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kSmallWarps = 4;
constexpr int kSmallThreads = kSmallWarps * 32;
constexpr int kSmallTile = 128;
constexpr int kSmallMaxStages = 8;

// NT: 8-row groups of a block.  Blocks a multiprocessor by the registers that
// the accumulators and queries take (24 D NT / 64 of them); stages by what
// those blocks leave of the shared memory.
template <int D, int NT>
struct SmallPlan {
  static constexpr int kBlocks = D * NT <= 128 ? 4 : (D * NT <= 256 ? 3 : 2);
  static constexpr int kStage = kSmallTile * D * 9 / 8;
  static constexpr int kFit = (227 * 1024 / kBlocks - 2048) / kStage;
  static constexpr int kStages = kFit > kSmallMaxStages ? kSmallMaxStages : kFit;
  static_assert(kStages >= 2, "a stage in flight while one is worked on");
  static constexpr int kRows = 8 * NT;
  static constexpr int kBars = kStages * kStage;
  static constexpr int kTotal = kBars + 2 * kSmallMaxStages * 8 + kSmallMaxStages * 4 + 16 + kSmallWarps * kRows * 8;
  static_assert(kSmallWarps * kRows * D * 4 <= kBars, "the warps' outputs reuse the ring");
};

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {  // an 8x8 fragment of 16-bit elements
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <int D, int NT>
__global__ void __launch_bounds__(kSmallThreads, SmallPlan<D, NT>::kBlocks)
    small_kernel(const __grid_constant__ AttnParams p, int n_rt, int chunk) {
  using L = SmallPlan<D, NT>;
  constexpr int kJ = D / 64, kRows = L::kRows;
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
      mbar_init(&full[s], 1 + p.miss);
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
  const int row0 = rt * kRows, n_rows = min(kRows, s.nq * p.g - row0);
  if (n_rows <= 0) return;  // (the whole block; every thread has passed its dependency wait)
  // keys that some row sees, and this block's tiles of them
  const int p0 = s.len - s.nq;  // position of the first query
  const int pos_min = p0 + row0 / p.g, pos_max = p0 + (row0 + n_rows - 1) / p.g;
  const int lo = key_lo(p, pos_min), hi = pos_max + 1;
  const int tile_a = lo / kSmallTile + split * chunk;
  const int tile_b = min(tile_a + chunk, (max(hi, 0) + kSmallTile - 1) / kSmallTile);
  const int n_tiles = hi > lo ? max(0, tile_b - tile_a) : 0;
  const int ppt = kSmallTile >> p.pshift;  // pages of a tile
  const int head_bytes = (int)p.head_bytes;

  // Warp 0 issues the copies too (a fifth warp would cost the compute warps a
  // third of their registers): lane i takes page i of a tile.
  const uint64_t pol = l2_evict_first_policy();
  auto page_seen = [&](int i) {  // something of this lane's page is seen
    const int j0 = ((tile_a + i) * ppt + lane) << p.pshift;
    return lane < ppt && i < n_tiles && j0 < hi && j0 + p.P > lo;
  };
  auto page_of = [&](int i) { return page_seen(i) ? page_entry(p, b, (tile_a + i) * ppt + lane) : -1; };
  auto issue = [&](int i, int entry) {
    const int st = i % L::kStages;
    const bool has = entry >= 0 && entry < p.n_pages;
    const uint32_t mask = __ballot_sync(0xffffffffu, has);
    if (mask != (1u << ppt) - 1u) checked_page(p, entry, page_seen(i));
    if (lane == 0) {
      pmask[st] = mask;
      mbar_arrive_expect_tx(&full[st], (uint32_t)(__popc(mask) * head_bytes));
    }
    __syncwarp();
    if (has)
      bulk_g2s_hint(smem + st * L::kStage + lane * head_bytes, p.pages + entry * p.page_bytes + (int64_t)kvh * head_bytes,
                    (uint32_t)head_bytes, &full[st], pol);
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

  const int n = lane >> 2, t = lane & 3;
  const int key_n = (n & 1) ? 4 + (((n >> 1) + 2) & 3) : n >> 1;  // kKey(n)
  const int key_e = t, key_o = 4 + ((t + 2) & 3);                  // kKey(2t), kKey(2t + 1)
  // query rows 8 i + n as B operands (channels 64 j + 16 t .. + 15), and what
  // the rows 8 i + 2t, 8 i + 2t + 1 of the accumulators see
  uint32_t bq[NT][8 * kJ];
  int hi_r[2 * NT], lo_r[2 * NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int r = 8 * i + n, tq = (row0 + r) / p.g, h = kvh * p.g + (row0 + r) % p.g;
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + (s.start + tq) * p.q_tok + h * p.q_head;
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
      uint4 x = make_uint4(0, 0, 0, 0), y = x;
      if (r < n_rows) {
        x = *reinterpret_cast<const uint4*>(q + 64 * j + 16 * t);
        y = *reinterpret_cast<const uint4*>(q + 64 * j + 16 * t + 8);
      }
      bq[i][8 * j] = x.x; bq[i][8 * j + 1] = x.y; bq[i][8 * j + 2] = x.z; bq[i][8 * j + 3] = x.w;
      bq[i][8 * j + 4] = y.x; bq[i][8 * j + 5] = y.y; bq[i][8 * j + 6] = y.z; bq[i][8 * j + 7] = y.w;
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int rr = 8 * i + 2 * t + e, pos = p0 + (row0 + rr) / p.g;
      hi_r[2 * i + e] = rr < n_rows ? pos + 1 : 0;
      lo_r[2 * i + e] = key_lo(p, pos);
    }
  }
  const int lo_max = key_lo(p, pos_max);
  float o[NT][4 * kJ][4];  // [.][4 j + e]: channels 64 j + 8 n + 2 e (+1), rows 8 i + 2 t (+1)
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int k = 0; k < 4 * kJ; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][k][e] = 0.f;
  float m[2 * NT], l[2 * NT];
#pragma unroll
  for (int i = 0; i < 2 * NT; ++i) m[i] = -INFINITY, l[i] = 0.f;
  uint32_t seen = 0;  // bit r: row r of m and l has seen a key
  const int code_b = p.P * (D / 2), half_b = head_bytes / 2;

  for (int i = 0; i < n_tiles; ++i) {
    const int st = i % L::kStages;
    bool ok = true;
    if (warp == 0 && issued < n_tiles) {  // the stage of tile i - 1 is free once every warp is past it
      const int pg = next_pg;
      next_pg = page_of(issued + 1);
      if (issued >= L::kStages)
        ok = wait_bar(&empty[issued % L::kStages], (uint32_t)((issued / L::kStages - 1) & 1), abort, p.status, p.timeout_ns, 1);
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
      // 16 keys lie in one page
      const uint8_t* base[2];
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        const int k = warp * 32 + 16 * a;
        base[a] = smem + st * L::kStage + (k >> p.pshift) * head_bytes + (k & (p.P - 1)) * (D / 2);
      }
      // from a key's codes to its scales: (P - at) rows of codes on, then at rows of scales
      float sc[NT][2][4];
#pragma unroll
      for (int a = 0; a < 2; ++a) {
#pragma unroll
        for (int u = 0; u < NT; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[u][a][e] = 0.f;
        const int at = (warp * 32 + 16 * a) & (p.P - 1);
        const uint8_t* kc = base[a] + key_n * (D / 2) + 8 * t;
        const uint8_t* ks = base[a] - at * (D / 2) + code_b + (at + key_n) * (D / 16);
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
          uint32_t k0[8], k1[8];  // keys n and n + 8
          const uint2 w0 = *reinterpret_cast<const uint2*>(kc + 32 * j);
          const uint2 w1 = *reinterpret_cast<const uint2*>(kc + 8 * (D / 2) + 32 * j);
          const uint32_t s0 = *reinterpret_cast<const uint32_t*>(ks + 4 * j);
          const uint32_t s1 = *reinterpret_cast<const uint32_t*>(ks + 8 * (D / 16) + 4 * j);
          const KeyScale d0 = key_scale(__byte_perm(s0, 0, 0x4040 + t * 0x0101));
          const KeyScale d1 = key_scale(__byte_perm(s1, 0, 0x4040 + t * 0x0101));
          key_pairs(w0.x, d0, k0);
          key_pairs(w0.y, d0, k0 + 4);
          key_pairs(w1.x, d1, k1);
          key_pairs(w1.y, d1, k1 + 4);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint32_t ak[4] = {k0[2 * c], k1[2 * c], k0[2 * c + 1], k1[2 * c + 1]};
#pragma unroll
            for (int u = 0; u < NT; ++u) mma_bf16(sc[u][a], ak, bq[u][8 * j + 2 * c], bq[u][8 * j + 2 * c + 1]);
          }
        }
      }
      // masks: past the last or before the first visible key, on absent pages
      const bool partial = c0 + 32 > pos_min + 1 || c0 < lo_max || mask != (1u << ppt) - 1u;
      if (!partial) seen = ~0u;
      else {
        // the values' scales of keys past the end or on absent pages become 0:
        // whatever lies there stays finite (only this warp reads its keys)
        const int k = warp * 32 + lane;
        if (!((mask >> (k >> p.pshift)) & 1) || c0 + lane >= s.len) {
          uint32_t* z = reinterpret_cast<uint32_t*>(smem + st * L::kStage + (k >> p.pshift) * head_bytes + half_b + code_b +
                                                    (k & (p.P - 1)) * (D / 16));
#pragma unroll
          for (int i = 0; i < D / 64; ++i) z[i] = 0;
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before the next copy into this stage
        __syncwarp();
#pragma unroll
        for (int a = 0; a < 2; ++a) {
          const bool page = (mask >> ((warp * 32 + 16 * a) >> p.pshift)) & 1;
          const int j0 = c0 + 16 * a + key_n, j1 = j0 + 8;
#pragma unroll
          for (int u = 0; u < NT; ++u)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const bool s0 = page && j0 < hi_r[2 * u + e] && j0 >= lo_r[2 * u + e];
              const bool s1 = page && j1 < hi_r[2 * u + e] && j1 >= lo_r[2 * u + e];
              if (!s0) sc[u][a][e] = -INFINITY;
              if (!s1) sc[u][a][2 + e] = -INFINITY;
              seen |= s0 || s1 ? 1u << (2 * u + e) : 0u;
            }
        }
      }
      float mn[2 * NT];
      bool grows = false;
#pragma unroll
      for (int r = 0; r < 2 * NT; ++r) {
        const int u = r >> 1, e = r & 1;
        float x = fmaxf(fmaxf(sc[u][0][e], sc[u][0][2 + e]), fmaxf(sc[u][1][e], sc[u][1][2 + e]));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
        mn[r] = fmaxf(m[r], x * p.scale_log2);
        grows |= mn[r] > m[r];
      }
      if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
        for (int r = 0; r < 2 * NT; ++r) {
          const float f = m[r] == -INFINITY ? 0.f : exp2_approx(m[r] - mn[r]);
          m[r] = mn[r];
          l[r] *= f;
#pragma unroll
          for (int k = 0; k < 4 * kJ; ++k) {
            o[r >> 1][k][r & 1] *= f;
            o[r >> 1][k][2 + (r & 1)] *= f;
          }
        }
      }
      uint32_t bp[NT][2][2];  // weights as B operands
#pragma unroll
      for (int u = 0; u < NT; ++u) {
        // a row that has seen nothing: all weights 0
        const float r0 = m[2 * u] == -INFINITY ? 0.f : m[2 * u], r1 = m[2 * u + 1] == -INFINITY ? 0.f : m[2 * u + 1];
#pragma unroll
        for (int a = 0; a < 2; ++a) {
          float w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = exp2_approx(fmaf(sc[u][a][e], p.scale_log2, (e & 1) ? -r1 : -r0));
          l[2 * u] += w[0] + w[2];
          l[2 * u + 1] += w[1] + w[3];
          bp[u][a][0] = transpose8(pack_h2(w[0], w[1]));
          bp[u][a][1] = transpose8(pack_h2(w[2], w[3]));
        }
      }
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        const int at = (warp * 32 + 16 * a) & (p.P - 1);
        const uint8_t* vc = base[a] + half_b + 4 * n;
        const uint8_t* vs = base[a] - at * (D / 2) + half_b + code_b + at * (D / 16);
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
          uint32_t bb[2][8];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int ke = 8 * u + key_e, ko = 8 * u + key_o;
            const uint32_t w0 = *reinterpret_cast<const uint32_t*>(vc + ke * (D / 2) + 32 * j);
            const uint32_t w1 = *reinterpret_cast<const uint32_t*>(vc + ko * (D / 2) + 32 * j);
            const uint32_t s0 = *reinterpret_cast<const uint32_t*>(vs + ke * (D / 16) + 4 * j);
            const uint32_t s1 = *reinterpret_cast<const uint32_t*>(vs + ko * (D / 16) + 4 * j);
            const uint32_t h = n >> 1;
            const ValueScale d = value_scale(__byte_perm(s0, s1, h | ((4 + h) << 8)) & 0x00FF00FFu);
            value_quads(__byte_perm(w0, w1, 0x5410), d, bb[u][0], bb[u][2], bb[u][4], bb[u][6]);
            value_quads(__byte_perm(w0, w1, 0x7632), d, bb[u][1], bb[u][3], bb[u][5], bb[u][7]);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t av[4] = {bb[0][2 * e], bb[0][2 * e + 1], bb[1][2 * e], bb[1][2 * e + 1]};
#pragma unroll
            for (int u = 0; u < NT; ++u) mma_f16(o[u][4 * j + e], av, bp[u][a][0], bp[u][a][1]);
          }
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[st]);
  }
  // this warp's part
#pragma unroll
  for (int x = 4; x < 32; x <<= 1) seen |= __shfl_xor_sync(0xffffffffu, seen, x);
#pragma unroll
  for (int r = 0; r < 2 * NT; ++r) {
    if ((seen >> r) & 1) m[r] = fmaxf(m[r], kSeen);
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 4);
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 8);
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 16);
    if (n == 0) ml[warp * kRows + 8 * (r >> 1) + 2 * t + (r & 1)] = make_float2(m[r], l[r]);
  }
  // every copy issued has landed before the ring is reused (they all have, unless a wait gave up)
  if (warp == 0)
    for (int j = max(0, issued - L::kStages); j < issued; ++j)
      wait_bar(&full[j % L::kStages], (uint32_t)((j / L::kStages) & 1), &never, p.status, p.timeout_ns, 3);
  __syncthreads();  // every warp has read its last stage
  float* ob = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int u = 0; u < NT; ++u)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float* d = ob + (warp * kRows + 8 * u + 2 * t + e) * D + 8 * n;
#pragma unroll
      for (int k = 0; k < 4 * kJ; ++k)
        *reinterpret_cast<float2*>(d + 64 * (k >> 2) + 2 * (k & 3)) = make_float2(o[u][k][e], o[u][k][2 + e]);
    }
  __syncthreads();
  // join the warps' parts
  const int64_t part = ((int64_t)(b * p.hk * n_rt + blockIdx.y) * p.n_split + split) * kRows;
  for (int i = tid; i < n_rows * (D / 4); i += kSmallThreads) {
    const int r = i / (D / 4), c = 4 * (i % (D / 4));
    float mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < kSmallWarps; ++w) mx = fmaxf(mx, ml[w * kRows + r].x);
    float lt = 0.f, x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kSmallWarps; ++w) {
      const float2 a = ml[w * kRows + r];
      const float f = a.x == -INFINITY ? 0.f : exp2_approx(a.x - mx);
      const float4 v = *reinterpret_cast<const float4*>(ob + (w * kRows + r) * D + c);
      lt = fmaf(a.y, f, lt);
      x[0] = fmaf(v.x, f, x[0]);
      x[1] = fmaf(v.y, f, x[1]);
      x[2] = fmaf(v.z, f, x[2]);
      x[3] = fmaf(v.w, f, x[3]);
    }
    if (p.n_split == 1) {
      const float inv = mx > -INFINITY ? kValueUnscale / lt : 0.f;
      const int row = row0 + r, tok = s.start + row / p.g, h = kvh * p.g + row % p.g;
      const __nv_bfloat162 u = __floats2bfloat162_rn(x[0] * inv, x[1] * inv), v = __floats2bfloat162_rn(x[2] * inv, x[3] * inv);
      uint2 w;
      w.x = *reinterpret_cast<const uint32_t*>(&u);
      w.y = *reinterpret_cast<const uint32_t*>(&v);
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + ((int64_t)tok * p.hq + h) * D + c) = w;
      if (p.lse && c == 0)
        p.lse[(int64_t)tok * p.hq + h] = mx > -INFINITY ? (mx + log2f(lt)) * 0.69314718055994531f : -INFINITY;
    } else {
      if (c == 0) p.part_ml[part + r] = make_float2(mx, lt);
      *reinterpret_cast<float4*>(p.part_o + (part + r) * D + c) = make_float4(x[0], x[1], x[2], x[3]);
    }
  }
}

// Joins up to kJoinFew parts of a row's keys: a thread 4 channels of a row,
// all its loads at once.
constexpr int kJoinFew = 8;
// The tile's place among the split ones (-1: it was not split).  whole < 0: all
// were, in the order sequence, head, row tile; else the prompt kernel's order,
// whose first `whole` went whole.
__device__ __forceinline__ int64_t part_tile(const AttnParams& p, int b, int kvh, int rt, int n_rt, int whole) {
  if (whole < 0) return (int64_t)(b * p.hk + kvh) * n_rt + rt;
  const int64_t i = (int64_t)(n_rt - 1 - rt) * p.hk * p.n_seqs + b * p.hk + kvh - whole;
  return i < 0 ? -1 : i;
}

template <int D>
__global__ void __launch_bounds__(256) join_few_kernel(const __grid_constant__ AttnParams p, int rows_per_tile, int n_rt, int whole) {
  griddep_launch_dependents();
  griddep_wait();
  const int b = blockIdx.y;
  const Seq s = load_seq(p, b);
  const int i = blockIdx.x * 256 + threadIdx.x, c = i % (D / 4), th = i / (D / 4);
  const int t = th / p.hq, h = th % p.hq;
  if (t >= s.nq) return;
  const int kvh = h / p.g, row = t * p.g + h % p.g;
  const int64_t tile = part_tile(p, b, kvh, row / rows_per_tile, n_rt, whole);
  if (tile < 0) return;
  const int64_t first = tile * p.n_split * rows_per_tile + row % rows_per_tile;
  const float4* po = reinterpret_cast<const float4*>(p.part_o) + first * (D / 4) + c;
  float2 ml[kJoinFew];
  float4 v[kJoinFew];
#pragma unroll
  for (int k = 0; k < kJoinFew; ++k) {
    const bool has = k < p.n_split;
    ml[k] = has ? p.part_ml[first + (int64_t)k * rows_per_tile] : make_float2(-INFINITY, 0.f);
    v[k] = has ? po[(int64_t)k * rows_per_tile * (D / 4)] : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  float mx = -INFINITY, lt = 0.f;
#pragma unroll
  for (int k = 0; k < kJoinFew; ++k) mx = fmaxf(mx, ml[k].x);
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int k = 0; k < kJoinFew; ++k) {
    const float f = ml[k].x == -INFINITY ? 0.f : exp2_approx(ml[k].x - mx);
    lt = fmaf(ml[k].y, f, lt);
    x.x = fmaf(v[k].x, f, x.x);
    x.y = fmaf(v[k].y, f, x.y);
    x.z = fmaf(v[k].z, f, x.z);
    x.w = fmaf(v[k].w, f, x.w);
  }
  store_joined(p, (int64_t)(s.start + t) * p.hq + h, c, D, x, lt, mx);
}

// Joins the parts of a row's keys: one block a (query token, query head), a
// group of D/4 threads every kJoinGroups-th part.  (A thread a channel walking
// over all parts took 21 us for 37 of them: a chain of loads each.)
constexpr int kJoinGroups = 8;
template <int D>
__global__ void __launch_bounds__(kJoinGroups * D / 4) join_kernel(const __grid_constant__ AttnParams p, int rows_per_tile, int n_rt, int whole) {
  __shared__ float wt[1024];                 // a part's weight 2^(m - max)
  __shared__ float4 sum[kJoinGroups][D / 4];
  __shared__ float2 red[32];
  griddep_launch_dependents();
  const int t = blockIdx.x / p.hq, h = blockIdx.x % p.hq, b = blockIdx.y;
  constexpr int kThreads = kJoinGroups * D / 4, kWarps = kThreads / 32;
  const int tid = threadIdx.x, g = tid / (D / 4), c = tid % (D / 4);
  griddep_wait();
  const Seq s = load_seq(p, b);
  if (t >= s.nq) return;
  const int kvh = h / p.g, row = t * p.g + h % p.g;
  const int64_t tile = part_tile(p, b, kvh, row / rows_per_tile, n_rt, whole);
  if (tile < 0) return;
  const int64_t first = tile * p.n_split * rows_per_tile + row % rows_per_tile;
  const float4* po = reinterpret_cast<const float4*>(p.part_o) + first * (D / 4) + c;
  const int64_t step = (int64_t)rows_per_tile * (D / 4);
  // the first parts are on their way while the weights are found
  constexpr int kBatch = 4;
  float4 v[kBatch];
#pragma unroll
  for (int k = 0; k < kBatch; ++k) {
    const int i = g + k * kJoinGroups;
    v[k] = i < p.n_split ? po[i * step] : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  float mx = -INFINITY;
  for (int i = tid; i < p.n_split; i += kThreads) mx = fmaxf(mx, p.part_ml[first + (int64_t)i * rows_per_tile].x);
  mx = warp_max(mx);
  if ((tid & 31) == 0) red[tid >> 5].x = mx;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, red[w].x);
  float lt = 0.f;
  for (int i = tid; i < p.n_split; i += kThreads) {
    const float2 a = p.part_ml[first + (int64_t)i * rows_per_tile];
    const float f = a.x == -INFINITY ? 0.f : exp2_approx(a.x - mx);
    wt[i] = f;
    lt = fmaf(a.y, f, lt);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) lt += __shfl_xor_sync(0xffffffffu, lt, o);
  if ((tid & 31) == 0) red[tid >> 5].y = lt;
  __syncthreads();
  lt = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) lt += red[w].y;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = g; i0 < p.n_split; i0 += kBatch * kJoinGroups) {
    if (i0 != g) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int i = i0 + k * kJoinGroups;
        v[k] = i < p.n_split ? po[i * step] : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + k * kJoinGroups;
      const float f = i < p.n_split ? wt[i] : 0.f;
      x.x = fmaf(v[k].x, f, x.x);
      x.y = fmaf(v[k].y, f, x.y);
      x.z = fmaf(v[k].z, f, x.z);
      x.w = fmaf(v[k].w, f, x.w);
    }
  }
  sum[g][c] = x;
  __syncthreads();
  const int64_t o = (int64_t)(s.start + t) * p.hq + h;
  if (g == 0) {
    x = sum[0][c];
#pragma unroll
    for (int k = 1; k < kJoinGroups; ++k) {
      const float4 y = sum[k][c];
      x.x += y.x;
      x.y += y.y;
      x.z += y.z;
      x.w += y.w;
    }
    store_joined(p, o, c, D, x, lt, mx);
  }
}

}  // namespace

template <int D>
static cudaError_t join_launch_d(const AttnParams& p, int rows_per_tile, int n_rt, int whole, cudaStream_t st) {
  // query tokens that may lie in a split tile
  int64_t tokens = p.max_q;
  if (whole >= 0) tokens = std::min<int64_t>(tokens, ((int64_t)(n_rt - whole / (p.hk * p.n_seqs)) * rows_per_tile + p.g - 1) / p.g);
  const unsigned rows = (unsigned)(tokens * p.hq);
  if (p.n_split <= kJoinFew)
    return launch_pdl(join_few_kernel<D>, dim3((unsigned)(((int64_t)rows * (D / 4) + 255) / 256), p.n_seqs), 256, 0, st, p,
                      rows_per_tile, n_rt, whole);
  return launch_pdl(join_kernel<D>, dim3(rows, p.n_seqs), kJoinGroups * D / 4, 0, st, p, rows_per_tile, n_rt, whole);
}

cudaError_t join_launch(const AttnParams& p, int rows_per_tile, int n_rt, int whole, cudaStream_t st) {
  switch (p.D) {
    case 64: return join_launch_d<64>(p, rows_per_tile, n_rt, whole, st);
    case 128: return join_launch_d<128>(p, rows_per_tile, n_rt, whole, st);
    case 192: return join_launch_d<192>(p, rows_per_tile, n_rt, whole, st);
    default: return join_launch_d<256>(p, rows_per_tile, n_rt, whole, st);
  }
}

namespace {

template <int D, int NT>
cudaError_t small_launch_d(AttnParams p, int num_sms, size_t part_rows, cudaStream_t st) {
  using L = SmallPlan<D, NT>;
  const int n_rt = (p.max_q * p.g + L::kRows - 1) / L::kRows;
  const int64_t base = (int64_t)p.hk * n_rt * p.n_seqs;
  // tiles that a row can see: the window's, or all
  int64_t span = std::max(p.max_len, 1);
  if (p.window > 0) span = std::min<int64_t>(span, (int64_t)p.window + p.max_q + kSmallTile);
  const int tiles = (int)((span + kSmallTile - 1) / kSmallTile);
  // keys are split until there are four blocks for each place on the GPU, so
  // that ragged lengths even out (32 sequences of 4096 to 8192 keys, 32/8 heads
  // of 128: 104, 88, 78 and 78 us with 2, 4, 8 and 10 parts), but not into a
  // few more parts than the quick join takes
  const int64_t want = std::max<int64_t>(1, 4LL * L::kBlocks * num_sms / base);
  int chunk = (int)std::max<int64_t>(1, (tiles + want - 1) / want);
  const int few = (tiles + kJoinFew - 1) / kJoinFew;
  if (few > chunk && few <= 2 * chunk) chunk = few;
  const int64_t fit = std::min<int64_t>(kMaxSplit, std::max<int64_t>(1, (int64_t)(part_rows / L::kRows) / base));
  chunk = std::max<int>(chunk, (int)((tiles + fit - 1) / fit));
  p.n_split = (tiles + chunk - 1) / chunk;
  cudaError_t e = launch_pdl(small_kernel<D, NT>, dim3(p.n_split, (unsigned)(p.hk * n_rt), p.n_seqs), kSmallThreads, L::kTotal,
                             st, p, n_rt, chunk);
  if (e != cudaSuccess || p.n_split == 1) return e;
  return join_launch(p, L::kRows, n_rt, -1, st);
}

template <int D>
cudaError_t small_configure_d() {
  cudaError_t e = cudaFuncSetAttribute(small_kernel<D, 1>, cudaFuncAttributeMaxDynamicSharedMemorySize, SmallPlan<D, 1>::kTotal);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(small_kernel<D, 2>, cudaFuncAttributeMaxDynamicSharedMemorySize, SmallPlan<D, 2>::kTotal);
}

template <int D>
cudaError_t small_launch_nt(const AttnParams& p, int num_sms, size_t part_rows, cudaStream_t st) {
  return p.max_q * p.g <= 8 ? small_launch_d<D, 1>(p, num_sms, part_rows, st) : small_launch_d<D, 2>(p, num_sms, part_rows, st);
}

}  // namespace

cudaError_t small_configure(int D) {
  switch (D) {
    case 64: return small_configure_d<64>();
    case 128: return small_configure_d<128>();
    case 192: return small_configure_d<192>();
    default: return small_configure_d<256>();
  }
}

cudaError_t small_launch(const AttnParams& p, int num_sms, size_t part_rows, cudaStream_t st) {
  switch (p.D) {
    case 64: return small_launch_nt<64>(p, num_sms, part_rows, st);
    case 128: return small_launch_nt<128>(p, num_sms, part_rows, st);
    case 192: return small_launch_nt<192>(p, num_sms, part_rows, st);
    default: return small_launch_nt<256>(p, num_sms, part_rows, st);
  }
}

}  // namespace attn
}  // namespace moe

// verify_sample.cu -- verification of drafted tokens, a tree of them for each
// sequence, against the target's probabilities from given random numbers, and
// the draw of the next token.
//
// At a node with the target's weights e_v = 2^(c (l_v - l_max)), c = log2(e) / T,
// Z = sum e, the children are tried in order.  Drafts chosen without chance:
//   child x with number u is accepted if u Z < e_x; else e_x leaves Z.
// Drafts drawn from f_v / F, the draft head's weights: with r = e at first, s = 1,
//   accepted if u Z f_x < s F r_x; else
//   k += Z / (s F),  r_v = (e_v - k f_v)+,  Z = sum r,  s -= f_x / F (drawn without replacement),
// since the positive part of (e - k f)+ - d f is (e - (k + d) f)+: one number k
// says what all the rejected children leave, whatever their number.
// Where no child is left, the next token is the first whose cumulative r passes
// u_root Z.
//
// A cluster of blocks owns a sequence and walks down its tree: only the rows of
// the accepted path are read, not those of the nodes that are not reached.
// Each block takes a slice of the vocabulary, each warp a range of the slice;
// the parts are exchanged through distributed shared memory, and every block
// comes to the same decisions from the same numbers.  One launch, no workspace.
//
// Precision.  A draw that falls within d of a border of two tokens can go
// either way, and with 150000 tokens there are that many borders: fp32 sums
// (2^-22) would miss the right token in several draws of a hundred.  So weights
// are pairs of fp32 numbers, right to some 2^-33, and their sums carry the
// rounding errors along (two-sum).  2^y of y = round(256 y) / 256 + g: a table
// of 256 entries, and 1 + g (L + g (L^2/2 + g L^3/6)), L = ln 2, of its series
// (|g| <= 2^-9).
#include <cooperative_groups.h>

#include <cmath>

#include "common.cuh"
#include "layer.cuh"

namespace moe {
namespace {

constexpr int kVsThreads = 512;
constexpr int kVsWarps = kVsThreads / 32;
constexpr int kVsNodes = 64;
constexpr int kVsMaxCluster = 8;

struct VsParams {
  const void* logits;
  int64_t stride;  // elements
  const void* draft;
  int64_t draft_stride;
  int V, n_seqs, n_nodes, max_nodes, replacement, C;
  const int32_t *tokens, *parents, *starts;
  const float *uniforms, *temperature;
  int32_t *path, *n_accepted, *next;
};

// 2^(i/256) as two fp32 numbers, from its series.
struct ExpTable {
  float hi[256], lo[256];
};
constexpr ExpTable make_exp_table() {
  ExpTable t{};
  for (int i = 0; i < 256; ++i) {
    const double x = 0.69314718055994530942 * i / 256.0;
    double term = 1.0, sum = 1.0;
    for (int k = 1; k < 24; ++k) {
      term *= x / k;
      sum += term;
    }
    t.hi[i] = (float)sum;
    t.lo[i] = (float)(sum - (double)t.hi[i]);
  }
  return t;
}
__device__ constexpr ExpTable kExpTable = make_exp_table();

struct Pair {  // h + l
  float h, l;
};
// a + b with the error of the high parts' sum in the low one.
__device__ __forceinline__ void accumulate(Pair& a, Pair b) {
  const float t = __fadd_rn(a.h, b.h), z = __fsub_rn(t, a.h);
  const float e = __fadd_rn(__fsub_rn(a.h, __fsub_rn(t, z)), __fsub_rn(b.h, z));
  a.h = t;
  a.l = __fadd_rn(a.l, __fadd_rn(e, b.l));
}
__device__ __forceinline__ Pair shuffled(Pair a, int o) {
  return Pair{__shfl_xor_sync(0xffffffffu, a.h, o), __shfl_xor_sync(0xffffffffu, a.l, o)};
}
__device__ __forceinline__ double value(Pair a) { return (double)a.h + (double)a.l; }

// A row's exponential: weight(l) = 2^(c (l - ref)) in units of 2^top.  ref is 0
// where |c l_max| < 2^10, else l_max: then the difference is exact for every
// logit that counts.  Below 2^-100 of the largest a weight is 0 (a masked
// logit's is exactly 0).
struct RowExp {
  float ref, floor, cut, ch, cl;
  uint32_t scale0;
};
__device__ __forceinline__ RowExp row_exp(float most, float ch, float cl) {
  RowExp r;
  const float y = most * ch;
  r.ref = fabsf(y) < 1024.f ? 0.f : most;
  const float top = rintf((most - r.ref) * ch);
  r.floor = (top - 120.f) / ch;
  r.cut = top - 100.f;
  r.ch = ch;
  r.cl = cl;
  r.scale0 = (uint32_t)(127 - (int)top) << 23;
  return r;
}
constexpr float kMagic = 49152.f;  // 1.5 2^15: its sum with y has steps of 2^-8
__device__ __forceinline__ Pair weight(float logit, const RowExp& r, const float2* table) {
  constexpr float L1 = 0.693147180559945f, L2 = 0.240226506959101f, L3 = 0.0555041086648216f;
  const float x = fmaxf(__fsub_rn(logit, r.ref), r.floor);
  const float y = __fmul_rn(x, r.ch);
  const float yl = fmaf(x, r.cl, fmaf(x, r.ch, -y));
  const float k = __fadd_rn(y, kMagic);
  const float g = __fsub_rn(y, __fsub_rn(k, kMagic));
  const uint32_t bits = __float_as_uint(k);
  const float2 t = table[bits & 255];
  const float p = fmaf(g, fmaf(g, fmaf(g, L3, L2), L1), yl * L1);
  // (bits >> 8) - (kMagic's bits >> 8) is the whole part of y
  const uint32_t scale = ((bits >> 8) << 23) - ((__float_as_uint(kMagic) >> 8) << 23) + r.scale0;
  const float s = y > r.cut ? __uint_as_float(scale) : 0.f;
  return Pair{__fmul_rn(t.x, s), __fmul_rn(fmaf(t.x, p, t.y), s)};
}
// (e - k f)+
__device__ __forceinline__ Pair residual(Pair e, Pair f, Pair k) {
  const float t = __fmul_rn(k.h, f.h);
  const float tl = fmaf(k.h, f.l, fmaf(k.l, f.h, fmaf(k.h, f.h, -t)));
  const float d = __fsub_rn(e.h, t), z = __fsub_rn(d, e.h);
  const float err = __fsub_rn(__fsub_rn(e.h, __fsub_rn(d, z)), __fadd_rn(t, z));
  const Pair r{d, __fadd_rn(err, __fsub_rn(e.l, tl))};
  return r.h + r.l > 0.f ? r : Pair{0.f, 0.f};
}

template <typename In>
struct Load;
template <>
struct Load<float> {
  static constexpr int kN = 4;
  __device__ static void vec(const float* p, float (&x)[4]) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(p));
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
  }
  __device__ static float one(const float* p) { return __ldg(p); }
};
template <>
struct Load<__nv_bfloat16> {
  static constexpr int kN = 8;
  __device__ static void vec(const __nv_bfloat16* p, float (&x)[8]) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  __device__ static float one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
};

// One row of logits, cut into vectors that start on 16-byte boundaries of the
// target's row: vector j holds the elements from j N - skew on (those before 0
// or from V on count as -inf).
template <typename In>
struct Row {
  const In* p;
  int V, skew;
  bool aligned;  // its vectors start on 16-byte boundaries too
  __device__ void load(int j, float (&x)[Load<In>::kN]) const {
    constexpr int N = Load<In>::kN;
    const int e = j * N - skew;
    if (aligned && e >= 0 && e + N <= V) {
      Load<In>::vec(p + e, x);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = e + i >= 0 && e + i < V ? Load<In>::one(p + e + i) : -INFINITY;
    }
  }
};
template <typename In>
__device__ __forceinline__ int skew_of(const In* p) {
  return (int)((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(In));
}

__device__ __forceinline__ float max_nan(float a, float b) {  // a NaN stays
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// Orders by value, then by the lower id.
__device__ __forceinline__ uint64_t order_key(float x, int id) {
  const uint32_t b = __float_as_uint(x + 0.f);  // -0 and 0 are equal
  const uint32_t o = b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
  return ((uint64_t)o << 32) | (uint32_t)~id;
}

// What a block tells the others of its cluster.
struct Part {
  float most, most_f;
  uint64_t best;
  double sum, sum_f;
};

enum : int { kGoOn, kReject, kDraw };

struct Walk {  // one block's shared memory
  float2 table[256];
  int parent[kVsNodes], token[kVsNodes], path[kVsNodes];
  float u[kVsNodes];
  Part part[2];
  float wmost[kVsWarps], wmost_f[kVsWarps];
  uint64_t wbest[kVsWarps];
  double wsum[kVsWarps], wsum_f[kVsWarps];  // of the warps' ranges: what is left of the target's weights, the draft's
  int child[kVsNodes], n_children;
  double child_e[kVsNodes], child_f[kVsNodes];
  bool gone[kVsNodes];  // of the children: rejected, its token's weight taken out
  double scan[kVsThreads];
  // written by one thread for all
  float most, most_f;
  uint64_t best;
  double Z, F;       // the sums of the cluster
  double kappa, left;  // the draft's part taken out; of its probability what is not rejected
  int act, at, cursor;
  double threshold;
  int owner, range, winner;
};

// The first of the warp's values (one a lane, in order) whose cumulative sum
// passes t, or the last above 0 where rounding leaves none; before: the sum
// ahead of it.  -1 if there is none.
__device__ __forceinline__ int pick(double q, double t, int lane, double& before) {
  double incl = q;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double up = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += up;
  }
  const uint32_t some = __ballot_sync(0xffffffffu, q > 0.0), past = __ballot_sync(0xffffffffu, q > 0.0 && incl > t);
  const int at = past ? __ffs(past) - 1 : (some ? 31 - __clz(some) : -1);
  before = __shfl_sync(0xffffffffu, incl - q, max(at, 0));
  return at;
}

template <typename In>
__global__ void __launch_bounds__(kVsThreads) verify_sample_kernel(const __grid_constant__ VsParams p) {
  namespace cg = cooperative_groups;
  constexpr int N = Load<In>::kN;
  __shared__ Walk w;
  griddep_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.x / p.C, rank = blockIdx.x % p.C;
  if (tid < 256) w.table[tid] = make_float2(kExpTable.hi[tid], kExpTable.lo[tid]);
  griddep_wait();
  cg::cluster_group cl = cg::this_cluster();

  const int start = p.starts[b], end = p.starts[b + 1];
  const bool empty = start < 0 || end > p.n_nodes || end <= start;
  if (empty) {  // (the whole cluster)
    if (rank == 0) {
      for (int i = tid; i < p.max_nodes; i += kVsThreads) p.path[(int64_t)b * p.max_nodes + i] = -1;
      if (tid == 0) p.n_accepted[b] = -1, p.next[b] = -1;
    }
    return;
  }
  const int m = min(end - start, p.max_nodes);
  const float T = p.temperature ? p.temperature[b] : 1.f;
  const bool valid_T = T >= 0.f && T <= 1e6f;
  const bool greedy = T < 1e-6f;
  const double c = 1.4426950408889634074 / (double)(greedy || !valid_T ? 1.f : T);
  const float ch = (float)c, c_lo = (float)(c - (double)ch);
  const bool drawn = p.draft && !greedy;
  if (tid < kVsNodes) {
    w.path[tid] = tid == 0 ? 0 : -1;
    w.parent[tid] = -2;
    if (tid < m) {
      w.parent[tid] = p.parents ? p.parents[start + tid] : tid - 1;
      w.token[tid] = p.tokens[start + tid];
      w.u[tid] = p.uniforms[start + tid];
    }
  }
  __syncthreads();

  int node = 0, length = 1, turn = 0;
  int next = -1;
  bool mine_to_write = rank == 0 && tid == 0;  // the thread that stores the next token
  // Ranges of whole vectors: warp w of block r takes the vectors [(16 r + w) per, ...).
  while (valid_T) {
    const In* pe = static_cast<const In*>(p.logits) + (int64_t)(start + node) * p.stride;
    const In* pf = drawn ? static_cast<const In*>(p.draft) + (int64_t)(start + node) * p.draft_stride : pe;
    const int skew = skew_of(pe);
    const Row<In> re{pe, p.V, skew, true}, rf{pf, p.V, skew, skew_of(pf) == skew};
    const int n_vec = (p.V + skew + N - 1) / N;
    const int per = (n_vec + p.C * kVsWarps - 1) / (p.C * kVsWarps);
    const int range = rank * kVsWarps + warp;
    const int j0 = min(n_vec, range * per), j1 = min(n_vec, j0 + per);

    // ---- the largest logits, and the children
    float most = -INFINITY, most_f = -INFINITY;
    uint64_t best = 0;
    for (int j = j0 + lane; j < j1; j += 32) {
      float x[N];
      re.load(j, x);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (greedy && x[i] > most) best = order_key(x[i], j * N - skew + i);
        most = max_nan(most, x[i]);
      }
      if (drawn) {
        rf.load(j, x);
#pragma unroll
        for (int i = 0; i < N; ++i) most_f = max_nan(most_f, x[i]);
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      most = max_nan(most, __shfl_xor_sync(0xffffffffu, most, o));
      most_f = max_nan(most_f, __shfl_xor_sync(0xffffffffu, most_f, o));
      const uint64_t other = __shfl_xor_sync(0xffffffffu, best, o);
      best = other > best ? other : best;
    }
    if (lane == 0) w.wmost[warp] = most, w.wmost_f[warp] = most_f, w.wbest[warp] = best;
    if (warp == 0) {
      int n = 0;
#pragma unroll
      for (int k = 0; k < kVsNodes; k += 32) {
        const bool is = k + lane > node && w.parent[k + lane] == node;
        const uint32_t set = __ballot_sync(0xffffffffu, is);
        if (is) w.child[n + __popc(set & ((1u << lane) - 1))] = k + lane;
        n += __popc(set);
      }
      if (lane == 0) w.n_children = n;
    }
    __syncthreads();
    if (warp == 0) {
      float a = w.wmost[lane % kVsWarps], d = w.wmost_f[lane % kVsWarps];
      uint64_t k = w.wbest[lane % kVsWarps];
#pragma unroll
      for (int o = kVsWarps / 2; o; o >>= 1) {
        a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, o));
        d = max_nan(d, __shfl_xor_sync(0xffffffffu, d, o));
        const uint64_t other = __shfl_xor_sync(0xffffffffu, k, o);
        k = other > k ? other : k;
      }
      if (lane == 0) w.part[turn].most = a, w.part[turn].most_f = d, w.part[turn].best = k;
    }
    cl.sync();
    if (warp == 0) {
      const Part* q = cl.map_shared_rank(&w.part[turn], lane % p.C);
      float a = q->most, d = q->most_f;
      uint64_t k = q->best;
#pragma unroll
      for (int o = kVsMaxCluster / 2; o; o >>= 1) {
        a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, o));
        d = max_nan(d, __shfl_xor_sync(0xffffffffu, d, o));
        const uint64_t other = __shfl_xor_sync(0xffffffffu, k, o);
        k = other > k ? other : k;
      }
      if (lane == 0) w.most = a, w.most_f = d, w.best = k;
    }
    turn ^= 1;
    __syncthreads();
    most = w.most;
    most_f = w.most_f;
    if (!(most > -INFINITY && most < INFINITY)) break;  // no distribution (NaN, +inf, or nothing left)
    const int n_children = w.n_children;
    if (greedy) {
      const int top = (int)~(uint32_t)w.best;
      int to = -1;
      for (int i = 0; i < n_children && to < 0; ++i)
        if (w.token[w.child[i]] == top) to = w.child[i];
      if (to < 0) {
        next = top;
        break;
      }
      if (tid == 0) w.path[length] = to;
      ++length;
      node = to;
      __syncthreads();
      continue;
    }
    const bool judged = drawn && most_f > -INFINITY && most_f < INFINITY;  // the draft's row is a distribution
    const RowExp ee = row_exp(most, ch, c_lo), ef = row_exp(judged ? most_f : 0.f, ch, c_lo);

    // ---- the sums
    double kappa = 0.0;
    Pair kp{0.f, 0.f};
    auto left_of = [&](const float (&xe)[N], const float (&xf)[N], Pair (&r)[N]) {  // what is left of a vector's weights
#pragma unroll
      for (int k = 0; k < N; ++k) {
        r[k] = weight(xe[k], ee, w.table);
        if (kappa > 0.0) r[k] = residual(r[k], weight(xf[k], ef, w.table), kp);
      }
    };
    auto sums = [&](bool draft) {  // this warp's range: what is left of the target's weights, and the draft's
      Pair a{0.f, 0.f}, d{0.f, 0.f};
      for (int j = j0 + lane; j < j1; j += 32) {
        float xe[N], xf[N];
        Pair r[N];
        re.load(j, xe);
        if (draft || kappa > 0.0) rf.load(j, xf);
        left_of(xe, xf, r);
#pragma unroll
        for (int k = 0; k < N; ++k) accumulate(a, r[k]);
        if (draft) {
#pragma unroll
          for (int k = 0; k < N; ++k) accumulate(d, weight(xf[k], ef, w.table));
        }
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        accumulate(a, shuffled(a, o));
        if (draft) accumulate(d, shuffled(d, o));
      }
      if (lane == 0) {
        w.wsum[warp] = value(a);
        if (draft) w.wsum_f[warp] = value(d);
      }
    };
    auto exchange = [&](bool draft) {  // their sums over the cluster, to warp 0 (and in part[turn ^ 1].sum a block's own)
      __syncthreads();
      if (warp == 0) {
        double a = lane < kVsWarps ? w.wsum[lane] : 0.0, d = draft && lane < kVsWarps ? w.wsum_f[lane] : 0.0;
#pragma unroll
        for (int o = kVsWarps / 2; o; o >>= 1) {
          a += __shfl_xor_sync(0xffffffffu, a, o);
          if (draft) d += __shfl_xor_sync(0xffffffffu, d, o);
        }
        if (lane == 0) w.part[turn].sum = a, w.part[turn].sum_f = d;
      }
      cl.sync();
      if (warp == 0) {
        const Part* q = cl.map_shared_rank(&w.part[turn], lane % p.C);
        double a = lane < p.C ? q->sum : 0.0, d = draft && lane < p.C ? q->sum_f : 0.0;
#pragma unroll
        for (int o = kVsMaxCluster / 2; o; o >>= 1) {
          a += __shfl_xor_sync(0xffffffffu, a, o);
          if (draft) d += __shfl_xor_sync(0xffffffffu, d, o);
        }
        if (lane == 0) {
          w.Z = a;
          if (draft) w.F = d;
        }
      }
      turn ^= 1;
    };
    sums(judged);
    if (tid < n_children) {
      const int x = w.token[w.child[tid]];
      const bool is = x >= 0 && x < p.V;
      w.child_e[tid] = is ? value(weight(Load<In>::one(pe + x), ee, w.table)) : -1.0;
      w.child_f[tid] = is && judged ? value(weight(Load<In>::one(pf + x), ef, w.table)) : 0.0;
      w.gone[tid] = false;
    }
    if (tid == 0) w.kappa = 0.0, w.left = 1.0, w.cursor = 0;
    exchange(judged);

    // ---- the children in order (one thread of each block decides, all of them the same)
    while (true) {
      if (tid == 0) {
        int act = kDraw;
        for (int i = w.cursor; i < n_children; ++i) {
          const int x = w.token[w.child[i]];
          const double e = w.child_e[i], f = w.child_f[i], u = (double)w.u[w.child[i]];
          if (e < 0.0 || (drawn && !judged)) continue;  // no such token, or nothing to judge it by: passed over
          if (!judged || !p.replacement) {
            bool again = false;  // an earlier sibling's token
            for (int k = 0; k < i; ++k) again |= w.token[w.child[k]] == x;
            if (again) continue;
          }
          const double r = judged ? e - w.kappa * f : e;
          if (judged ? u * w.Z * f < w.left * w.F * r : u * w.Z < r) {
            act = kGoOn;
            w.at = w.child[i];
            break;
          }
          if (!judged) {
            w.Z -= e;
            w.gone[i] = true;
          } else if (w.left > 0.0 && w.Z > 0.0) {
            w.kappa += w.Z / (w.left * w.F);
            if (!p.replacement) w.left -= f / w.F;
            w.cursor = i + 1;
            act = kReject;
            break;
          }
        }
        w.act = act;
      }
      __syncthreads();
      if (w.act != kReject) break;
      kappa = w.kappa;
      kp.h = (float)kappa;
      kp.l = (float)(kappa - (double)kp.h);
      sums(false);
      exchange(false);
    }
    if (w.act == kGoOn) {
      node = w.at;
      if (tid == 0) w.path[length] = node;
      ++length;
      __syncthreads();
      continue;
    }

    // ---- the next token
    if (!judged && n_children > 0) {  // what the rejected drafts that were chosen leave of the ranges' sums
      if (tid == 0) {
        for (int i = 0; i < n_children; ++i) {
          if (!w.gone[i]) continue;
          const int at = (w.token[w.child[i]] + skew) / N / per;
          if (at / kVsWarps != rank) continue;
          double& q = w.wsum[at % kVsWarps];
          const double rest = q - w.child_e[i];
          q = rest > q * 0x1p-40 ? rest : 0.0;  // (all of it: no rounding stays)
        }
      }
      exchange(false);
      __syncthreads();
    }
    bool out = !judged;  // the rejected tokens' own weights are out
    if (!(w.Z > 0.0)) {  // nothing is left: the target's own weights
      kappa = 0.0;
      out = false;
      __syncthreads();
      sums(false);
      exchange(false);
    }
    if (warp == 0) {
      // the block, its warp's range, and what the threshold is there
      double before;
      const Part* q = cl.map_shared_rank(&w.part[turn ^ 1], lane % p.C);
      const double t = (double)w.u[0] * w.Z;
      const int owner = pick(lane < p.C ? q->sum : 0.0, t, lane, before);
      double inside;
      const int at = pick(lane < kVsWarps ? w.wsum[lane] : 0.0, t - before, lane, inside);
      if (lane == 0) w.owner = owner, w.range = rank * kVsWarps + max(at, 0), w.threshold = t - before - inside;
    }
    __syncthreads();
    mine_to_write = false;
    if (rank != w.owner) break;
    const int k0 = min(n_vec, w.range * per), k1 = min(n_vec, k0 + per), each = (per + kVsThreads - 1) / kVsThreads;
    const int a0 = min(k1, k0 + tid * each), a1 = min(k1, a0 + each);
    auto left_at = [&](int j, Pair (&r)[N]) {
      float xe[N], xf[N];
      re.load(j, xe);
      if (kappa > 0.0) rf.load(j, xf);
      left_of(xe, xf, r);
      if (out) {
        for (int i = 0; i < n_children; ++i) {
          const int k = w.token[w.child[i]] - (j * N - skew);
          if (!w.gone[i] || k < 0 || k >= N) continue;
#pragma unroll
          for (int e = 0; e < N; ++e)
            if (e == k) r[e] = Pair{0.f, 0.f};
        }
      }
    };
    Pair a{0.f, 0.f};
    for (int j = a0; j < a1; ++j) {
      Pair r[N];
      left_at(j, r);
#pragma unroll
      for (int k = 0; k < N; ++k) accumulate(a, r[k]);
    }
    w.scan[tid] = value(a);
    __syncthreads();
    if (warp == 0) {  // the thread whose vectors hold the threshold: 16 threads a lane, then those
      constexpr int kPer = kVsThreads / 32;
      double sum = 0.0, before, inside;
      for (int k = 0; k < kPer; ++k) sum += w.scan[lane * kPer + k];
      const int some = max(pick(sum, w.threshold, lane, before), 0);
      const int at = max(pick(lane < kPer ? w.scan[some * kPer + lane] : 0.0, w.threshold - before, lane, inside), 0);
      if (lane == 0) w.winner = some * kPer + at, w.threshold -= before + inside;
    }
    __syncthreads();
    if (tid == w.winner) {
      mine_to_write = true;
      double run = 0.0;
      bool found = false;
      for (int j = a0; j < a1 && !found; ++j) {
        Pair r[N];
        left_at(j, r);
#pragma unroll
        for (int k = 0; k < N; ++k) {
          const double q = value(r[k]);
          if (found || !(q > 0.0)) continue;
          next = j * N - skew + k;  // (the last with any where rounding leaves none that passes)
          run += q;
          found = run > w.threshold;
        }
      }
    }
    break;
  }
  if (mine_to_write) p.next[b] = next;
  __syncthreads();
  if (rank == 0) {
    for (int i = tid; i < p.max_nodes; i += kVsThreads) p.path[(int64_t)b * p.max_nodes + i] = i < m ? w.path[i] : -1;
    if (tid == 0) p.n_accepted[b] = length - 1;
  }
  cl.sync();  // nobody reads a block's shared memory after its end
}

template <typename In>
cudaError_t verify_sample_launch(const VsParams& p, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.n_seqs * p.C));
  cfg.blockDim = dim3(kVsThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)p.C;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, verify_sample_kernel<In>, p);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int mtp_verify_sample(const void* logits, int32_t dtype, int64_t row_stride, const void* draft_logits,
                                 int64_t draft_stride, int32_t V, const int32_t* tokens, const int32_t* parents,
                                 const int32_t* starts, int32_t n_seqs, int32_t n_nodes, int32_t max_nodes,
                                 const float* uniforms, const float* temperature, int32_t replacement, int32_t* path,
                                 int32_t* out_n_accepted, int32_t* out_next_token, void* stream) {
  const char* who = "mtp_verify_sample";
  if (dtype != MOE_ACT_BF16 && dtype != MOE_ACT_F32) return set_error(MOE_EINVAL, "%s: dtype=%d", who, dtype);
  if (V < 1 || V > (1 << 24)) return set_error(MOE_EINVAL, "%s: V=%d outside 1..2^24", who, V);
  if (n_seqs < 0 || n_seqs > (1 << 20)) return set_error(MOE_EINVAL, "%s: n_seqs=%d outside 0..2^20", who, n_seqs);
  if (n_nodes < 0 || n_nodes > (1 << 24)) return set_error(MOE_EINVAL, "%s: n_nodes=%d outside 0..2^24", who, n_nodes);
  if (max_nodes < 1 || max_nodes > kVsNodes)
    return set_error(MOE_EINVAL, "%s: max_nodes=%d outside 1..%d", who, max_nodes, kVsNodes);
  if (replacement != 0 && replacement != 1) return set_error(MOE_EINVAL, "%s: replacement=%d", who, replacement);
  if (n_nodes > 1 && (row_stride < V || (draft_logits && draft_stride < V)))
    return set_error(MOE_EINVAL, "%s: row strides %lld and %lld, V=%d", who, (long long)row_stride, (long long)draft_stride, V);
  if (n_seqs == 0) return MOE_OK;
  if (!starts || !path || !out_n_accepted || !out_next_token ||
      (n_nodes > 0 && (!logits || !tokens || !uniforms)))
    return set_error(MOE_EINVAL, "%s: NULL argument", who);
  const uintptr_t rows = reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(draft_logits);
  if (rows % (dtype == MOE_ACT_BF16 ? 2 : 4)) return set_error(MOE_EINVAL, "%s: logits misaligned", who);
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) {
    cudaGetLastError();  // reported here: the next launch of the process is not to find it
    return set_error(MOE_ECUDA, "%s: %s", who, cudaGetErrorString(e));
  }
  VsParams p{logits, row_stride, draft_logits, draft_stride, V, n_seqs, n_nodes, max_nodes, replacement, 1,
             tokens, parents, starts, uniforms, temperature, path, out_n_accepted, out_next_token};
  while (p.C < kVsMaxCluster && 2LL * n_seqs * p.C <= 5LL * sms / 4 && V / (2 * p.C) >= 1024) p.C *= 2;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  e = dtype == MOE_ACT_F32 ? verify_sample_launch<float>(p, st) : verify_sample_launch<__nv_bfloat16>(p, st);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return set_error(MOE_ECUDA, "%s launch: %s", who, cudaGetErrorString(e));
  }
  return MOE_OK;
}

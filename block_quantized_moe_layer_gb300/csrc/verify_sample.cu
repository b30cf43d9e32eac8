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
// A step is decided by fp32 sums (exp2 of the hardware, one pass over the rows)
// where a child is accepted by more than their error, as it mostly is.  Only the
// last row of a walk, and the few steps that are close, need more bits:
// a draw that falls within d of a border of two tokens can go either way, and
// with 150000 tokens there are that many borders; fp32 sums would miss the right
// token in several draws of a hundred.  There a weight is a pair of fp32 numbers,
// right to some 2^-33, sums carry their rounding errors along, and the ranges'
// sums are whole numbers, exact in any order.  2^y of y = round(256 y) / 256 + g:
// a table and a short series (Tang's table-driven exponential), 1 + g (L + g
// (L^2/2 + g L^3/6)), L = ln 2, |g| <= 2^-9.
//
//   Drafts drawn without replacement are judged by shares of what the rejected ones
// leave of f.  Where that is little it is no difference of sums (of a peaked draft
// row nothing but rounding is left of one): it is summed again without them, in
// units of the largest weight that is left: two passes over the draft's row, an
// exchange each.  A sibling is never judged by a share of nothing: it is passed
// over, which leaves the tokens' distribution as it is.
//
//   A drawn draft that is surely rejected takes one pass over both rows for their
// sums and for what is left, at the k that the fp32 sums give, and a correction
// (see there); the others, and a node's second rejection, a pass each.
//
// Measured (three calls' inputs in turn): a chain of 4 nodes, 32768 fp32 logits,
// 11.8 us (2.4 us a step: the pass 0.7, a cluster barrier 0.9, the decision 0.8);
// 4 trees of 64 nodes 15.3; 64 chains of 4 with drawn drafts, 151936 bf16 logits,
// 63 us (the rows read take 20: a step 9 us, 5.7 of them HBM's while all walk; a
// rejected drawn draft 20 to 30, all of it instructions, and 2 for the decision;
// the next token's place in its range 5; 166 where the draft's rows are aligned
// otherwise than the target's); 32 trees of 12 nodes, 151936 fp32, 37 us (inputs in
// L2: 29; the longest walk's five rows: 5 us a step, the last 4, then the place).
// Blocks a sequence: 4, 8 and 16 take 54, 37 and 49 us there, 63, 71 and 115 for the
// 64 chains (two blocks a multiprocessor are on the GPU at once).  Asking L2 for the
// next row ahead of the walk cost 1 us, and 7 of the 64 chains' 67 at the time.
#include <cooperative_groups.h>

#include <cmath>

#include "common.cuh"
#include "layer.cuh"

namespace moe {
namespace {

constexpr int kVsThreads = 256;
constexpr int kVsWarps = kVsThreads / 32, kVsLogWarps = 3;
static_assert(kVsWarps == 1 << kVsLogWarps, "a power of two");
constexpr int kVsNodes = 64;
constexpr int kVsMaxCluster = 16, kVsBlocks = 2;  // blocks a sequence at most; a multiprocessor
constexpr int kVsRanges = kVsMaxCluster * kVsWarps;  // most ranges of a row
constexpr int kVsBands = 4;
constexpr int kVsBatch = 4;  // 16-byte loads in flight a thread

struct VsParams {
  const void* logits;
  int64_t stride;  // elements
  const void* draft;
  int64_t draft_stride;
  int V, n_seqs, n_nodes, max_nodes, replacement, log_c;
  const int32_t *tokens, *parents, *starts;
  const float *uniforms, *temperature;
  int32_t *path, *n_accepted, *next;
};

// 2^(i/256) / (1 + i/256) as two fp32 numbers, from its series.
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
    sum /= 1.0 + i / 256.0;
    t.hi[i] = (float)sum;
    t.lo[i] = (float)(sum - (double)t.hi[i]);
  }
  return t;
}
__device__ constexpr ExpTable kExpTable = make_exp_table();

// Two fp32 numbers in a register pair, an instruction for both.
__device__ __forceinline__ uint64_t f2(float a, float b) {
  return (uint64_t)__float_as_uint(a) | ((uint64_t)__float_as_uint(b) << 32);
}
__device__ __forceinline__ float f2_lo(uint64_t a) { return __uint_as_float((uint32_t)a); }
__device__ __forceinline__ float f2_hi(uint64_t a) { return __uint_as_float((uint32_t)(a >> 32)); }
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f2_sub(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

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
// In whole steps of 1 / scale (a power of two): sums of these are exact, in any order.
__device__ __forceinline__ int64_t fixed(float h, float l, float scale) { return __float2ll_rn(h * scale) + __float2ll_rn(l * scale); }

// 1 / x to some 2^-46 (a division in fp64 takes a step of its own here).
__device__ __forceinline__ double reciprocal(double x) {
  const double y = (double)__frcp_rn((float)x);
  return fma(y, fma(-x, y, 1.0), y);
}

// A row's exponential: weight(l) = k 2^(c (l - ref)) in units of 2^top, k = 1
// unless scaled() says more.  ref is 0 where |c l_max| < 2^10, else l_max: then
// the difference is exact for every logit that counts.  Below 2^-126 of the unit
// a weight is 0: the exponent of what is clamped there is that of 0 (a masked
// logit's weight is exactly 0).
struct RowExp {
  float ref, floor, ceil, top, ch, cl;
  float magic, rest;  // log2(k) in steps of 2^-8, and what is left of it
  uint32_t scale0;
};
constexpr float kMagic = 49152.f;  // 1.5 2^15: its sum with y has steps of 2^-8
__device__ __forceinline__ RowExp row_exp(float ref, float most, float ch, float cl) {  // of logits up to `most`
  RowExp r;
  r.ref = ref;
  const float top = rintf((most - ref) * ch);
  r.top = top;
  r.floor = (top - 127.f) / ch;
  r.ceil = INFINITY;
  r.ch = ch;
  r.cl = cl;
  r.magic = kMagic;
  r.rest = 0.f;
  r.scale0 = ((uint32_t)(127 - (int)top) << 23) - (__float_as_uint(kMagic) << 15);
  return r;
}
__device__ __forceinline__ RowExp row_exp(float most, float ch, float cl) {
  return row_exp(fabsf(most * ch) < 1024.f ? 0.f : most, most, ch, cl);
}
// The same times k > 0 (both weights of a logit are compared); held below 8
// units, which is above every weight of the other row.  log2(k) = e + i/256 +
// log2(1 + d), 1 + d what the table leaves of k's mantissa, by its series.
__device__ __forceinline__ RowExp scaled(RowExp r, double k, const float2* table) {
  const int high = __double2hiint(k);
  int e = ((high >> 20) & 0x7FF) - 1023;
  const double m = __hiloint2double((high & 0xFFFFF) | 0x3FF00000, __double2loint(k));  // 1..2
  float mh = (float)m, ml = (float)(m - (double)mh);
  int i = __float2int_rn(256.f * __log2f(mh));
  if (i > 255) i = 0, ++e, mh *= 0.5f, ml *= 0.5f;
  const float2 t = table[max(i, 0)];
  const float step = 1.f + (float)max(i, 0) * 0.00390625f;
  const float d = __fdiv_rn(fmaf(-t.x, step, mh) + fmaf(-t.y, step, ml), t.x * step);
  const float steps = (float)e + (float)max(i, 0) * 0.00390625f;
  r.magic = kMagic + steps;
  r.rest = d * fmaf(d, fmaf(d, 0.48089835f, -0.72134752f), 1.44269504f);
  r.floor = (r.top - steps - 127.f) / r.ch;
  r.ceil = (r.top - steps + 3.f) / r.ch;
  return r;
}
// 2^y = (h + l) s of two logits: y = c x = (steps of 2^-8) + g; the steps' bits are
// the exponent of s and the eight first ones of its mantissa, by whose value the
// table's entries are divided.
struct Raw {
  uint64_t h, l, s;
};
template <bool SCALED = false>
__device__ __forceinline__ Raw weight(float x0, float x1, const RowExp& r, const float2* table) {
  constexpr float L1 = 0.693147180559945f, L2 = 0.240226506959101f, L3 = 0.0555041086648216f;
  const uint64_t ch = f2(r.ch, r.ch), magic = f2(r.magic, r.magic);
  uint64_t x = f2_sub(f2(x0, x1), f2(r.ref, r.ref));
  x0 = fmaxf(f2_lo(x), r.floor);
  x1 = fmaxf(f2_hi(x), r.floor);
  if (SCALED) x0 = fminf(x0, r.ceil), x1 = fminf(x1, r.ceil);
  x = f2(x0, x1);
  const uint64_t k = f2_fma(x, ch, magic);
  const uint32_t k0 = (uint32_t)k, k1 = (uint32_t)(k >> 32);
  const float2 t0 = table[k0 & 255], t1 = table[k1 & 255];
  uint64_t g = f2_fma(x, f2(r.cl, r.cl), f2_fma(x, ch, f2_sub(magic, k)));
  if (SCALED) g = f2_add(g, f2(r.rest, r.rest));
  const uint64_t p = f2_mul(g, f2_fma(g, f2_fma(g, f2(L3, L3), f2(L2, L2)), f2(L1, L1)));
  Raw w;
  w.h = f2(t0.x, t1.x);
  w.l = f2_fma(w.h, p, f2(t0.y, t1.y));
  w.s = (uint64_t)((k0 << 15) + r.scale0) | ((uint64_t)((k1 << 15) + r.scale0) << 32);
  return w;
}
// Two weights, each in two parts: what it has in steps of 2^-17 of the unit, so
// that a sum of them is exact below 2^6, and the rest.
struct Parts {
  uint64_t hi, lo;
};
__device__ __forceinline__ Parts parts(const Raw& r) {
  const uint64_t grid = f2(96.f, 96.f);  // 1.5 2^6
  const uint64_t l = f2_mul(r.l, r.s), top = f2_sub(f2_add(f2_fma(r.h, r.s, l), grid), grid);
  return Parts{top, f2_add(f2_fma(r.h, r.s, f2_sub(0, top)), l)};
}
// (a - b)+
__device__ __forceinline__ Parts residual(const Parts& a, const Parts& b) {
  Parts r{f2_sub(a.hi, b.hi), f2_sub(a.lo, b.lo)};
  const uint64_t sum = f2_add(r.hi, r.lo);
  if (!(f2_lo(sum) > 0.f)) r.hi &= 0xFFFFFFFF00000000ull, r.lo &= 0xFFFFFFFF00000000ull;
  if (!(f2_hi(sum) > 0.f)) r.hi &= 0xFFFFFFFFull, r.lo &= 0xFFFFFFFFull;
  return r;
}

__device__ __forceinline__ float max_nan(float a, float b) {  // a NaN stays
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

template <typename In>
struct Load;
template <>
struct Load<float> {
  static constexpr int kN = 4;
  __device__ static void unpack(uint4 v, float (&x)[4]) {
    x[0] = __uint_as_float(v.x); x[1] = __uint_as_float(v.y); x[2] = __uint_as_float(v.z); x[3] = __uint_as_float(v.w);
  }
  template <int B>
  __device__ static float most(const uint4 (&v)[B]) {
    float m = -INFINITY;
#pragma unroll
    for (int b = 0; b < B; ++b) {
      m = max_nan(m, __uint_as_float(v[b].x), __uint_as_float(v[b].y));
      m = max_nan(m, __uint_as_float(v[b].z), __uint_as_float(v[b].w));
    }
    return m;
  }
  __device__ static float one(const float* p) { return __ldg(p); }
};
template <>
struct Load<__nv_bfloat16> {
  static constexpr int kN = 8;
  __device__ static void unpack(uint4 v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  template <int B>
  __device__ static float most(const uint4 (&v)[B]) {
    uint32_t m = 0xFF80FF80u;  // -inf twice
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const uint32_t w[4] = {v[b].x, v[b].y, v[b].z, v[b].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i]));
    }
    return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
  }
  __device__ static float one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
};

// One row of logits, cut into vectors that start on 16-byte boundaries of the
// target's row: vector j holds the elements from j N - skew on (those before 0
// or from V on count as -inf).
template <typename In>
struct Row {
  static constexpr int N = Load<In>::kN;
  const In* p;
  int V, skew;
  bool aligned;  // its vectors start on 16-byte boundaries too
  __device__ bool whole(int j) const { return aligned && j * N >= skew && j * N - skew + N <= V; }
  __device__ uint4 raw(int j) const { return __ldg(reinterpret_cast<const uint4*>(p + (j * N - skew))); }
  __device__ uint4 raw_or_none(int j, int j1) const {
    const uint32_t none = sizeof(In) == 4 ? 0xFF800000u : 0xFF80FF80u;  // -inf
    return j < j1 ? raw(j) : make_uint4(none, none, none, none);
  }
  __device__ void load(int j, float (&x)[N]) const {
    if (whole(j)) {
      Load<In>::unpack(raw(j), x);
    } else {
      const int e = j * N - skew;
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = e + i >= 0 && e + i < V ? Load<In>::one(p + e + i) : -INFINITY;
    }
  }
  // A warp's vectors [j0, j1), a lane every 32nd, kBatch at once and the next ones
  // on their way: batch(words, n, vector) of n rounds where those of all lanes
  // are whole (-inf past j1), else one(x, first element) each.
  template <int kBatch, class B, class F>
  __device__ void each(int j0, int j1, B batch, F one) const {
    const int lane = threadIdx.x & 31;
    const bool all = j0 < j1 && whole(j0) && whole(j1 - 1);
    if (!all) {
#pragma unroll 1
      for (int j = j0 + lane; j < j1; j += 32) {
        float x[N];
        load(j, x);
        one(x, j * N - skew);
      }
      return;
    }
    uint4 v[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) v[b] = raw_or_none(j0 + lane + 32 * b, j1);
#pragma unroll 1
    for (int j = j0; j < j1; j += 32 * kBatch) {
      uint4 u[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) u[b] = v[b];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) v[b] = raw_or_none(j + lane + 32 * (kBatch + b), j1);
      batch(u, min(kBatch, (j1 - j + 31) >> 5), j + lane);
    }
  }
};
template <typename In>
__device__ __forceinline__ int skew_of(const In* p) {
  return (int)((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(In));
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Largest logit and sum of 2^(c (l - m)), in fp32.
struct Soft {
  float m, s;
};
__device__ __forceinline__ void raise(Soft& a, float m, float ch) {
  const float mn = max_nan(a.m, m);
  if (mn != a.m) {  // (or NaN)
    a.s = a.m == -INFINITY ? 0.f : a.s * exp2_fast((a.m - mn) * ch);
    a.m = mn;
  }
}
// The joined parts of a warp's lanes, or of each half's.
__device__ __forceinline__ Soft warp_soft(Soft a, float ch, bool halves = false) {
  float m = a.m;
#pragma unroll
  for (int o = 8; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (!halves) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 16));
  raise(a, m, ch);
#pragma unroll
  for (int o = 8; o; o >>= 1) a.s += __shfl_xor_sync(0xffffffffu, a.s, o);
  if (!halves) a.s += __shfl_xor_sync(0xffffffffu, a.s, 16);
  return a;
}
__device__ __forceinline__ Pair warp_pair(Pair a) {
#pragma unroll
  for (int o = 16; o; o >>= 1) accumulate(a, Pair{__shfl_xor_sync(0xffffffffu, a.h, o), __shfl_xor_sync(0xffffffffu, a.l, o)});
  return a;
}
__device__ __forceinline__ uint64_t warp_best(uint64_t k) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const uint64_t other = __shfl_xor_sync(0xffffffffu, k, o);
    k = other > k ? other : k;
  }
  return k;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// The relative widths 2^-13, 2^-15, 2^-17, 2^-19.
__device__ __forceinline__ constexpr float band(int k) { return k == 0 ? 0x1p-13f : k == 1 ? 0x1p-15f : k == 2 ? 0x1p-17f : 0x1p-19f; }
// Orders by value, then by the lower id.
__device__ __forceinline__ uint64_t order_key(float x, int id) {
  const uint32_t b = __float_as_uint(x + 0.f);  // -0 and 0 are equal
  const uint32_t o = b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
  return ((uint64_t)o << 32) | (uint32_t)~id;
}

enum : int { kGoOn, kReject, kDraw, kSureReject, kRest };

// Drafts drawn without replacement: less than this of the draft's probability is
// left, and the sum of what is left is made anew (sum_again).  By subtraction it
// is right to 2^-32 of the whole, so to 2^-30 of itself above this.
constexpr double kFewLeft = 0.25;
// The largest weight left is below 2^-this of the row's largest: nothing is left.
// (Above it, differences from a reference of 2^10 / c are exact down to 2^-44 of the
// largest that is left, half a step of the sums at most.)
constexpr float kNothingLeft = 400.f;

struct Walk {  // one block's shared memory
  float2 table[256];
  int parent[kVsNodes], token[kVsNodes], path[kVsNodes], child[kVsNodes];
  float u[kVsNodes];
  // all warps of the cluster write theirs to every block; two sets, used in turn
  Soft soft[2][kVsRanges];
  union {
    uint64_t best[2][kVsRanges];
    int64_t sum[2][kVsRanges];  // of the ranges: what is left of the target's weights
  };
  int64_t sum_f[2][kVsRanges];  // the draft's
  int64_t whole_e[kVsRanges], whole_f[kVsRanges];  // the same of both rows, beside what is left of one
  float near[kVsBands][kVsRanges];
  int64_t child_e[kVsNodes], child_f[kVsNodes];
  int child_at[kVsNodes];  // their ranges
  bool gone[kVsNodes];  // of the children: rejected, its token's weight taken out (drawn without replacement: out of the draft's)
  int64_t part[kVsWarps];
  // written by the first warp for the block
  float most, most_f;
  int act, at, range, winner, up, found;
  double kappa;
  RowExp kf;
  int64_t threshold;
};

// The first of the warp's values (one a lane, in order) whose cumulative sum
// passes t, or the last above 0 where rounding leaves none; before: the sum
// ahead of it.  -1 if there is none.
__device__ __forceinline__ int pick(int64_t q, int64_t t, int lane, int64_t& before) {
  int64_t incl = q;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += up;
  }
  const uint32_t some = __ballot_sync(0xffffffffu, q > 0), past = __ballot_sync(0xffffffffu, q > 0 && incl > t);
  const int at = past ? __ffs(past) - 1 : (some ? 31 - __clz(some) : -1);
  before = __shfl_sync(0xffffffffu, incl - q, max(at, 0));
  return at;
}
__device__ __forceinline__ int64_t warp_total(int64_t v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// DRAFT: the drafts may be drawn.  Calls without a draft's row have an instance of
// their own, which is shorter (a chain of 4 chosen drafts 13.9 us in the common one, 12.6 in its own).
template <typename In, bool DRAFT>
__global__ void __launch_bounds__(kVsThreads, kVsBlocks) verify_sample_kernel(const __grid_constant__ VsParams p) {
  namespace cg = cooperative_groups;
  constexpr int N = Load<In>::kN;
  constexpr int kGroup = kVsMaxCluster * kVsWarps / 32;  // most ranges of a lane of the first warp
  __shared__ Walk w;
  griddep_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.x >> p.log_c, rank = blockIdx.x & ((1 << p.log_c) - 1);
  if (tid < 256) w.table[tid] = make_float2(kExpTable.hi[tid], kExpTable.lo[tid]);
  cg::cluster_group cl = cg::this_cluster();
  cl.barrier_arrive();  // (waited for before the first write to another block's memory)
  griddep_wait();

  const int start = p.starts[b], end = p.starts[b + 1];
  const float T = p.temperature ? p.temperature[b] : 1.f;
  const bool empty = start < 0 || end > p.n_nodes || end <= start;
  if (empty) {  // (the whole cluster)
    cl.barrier_wait();
    if (rank == 0) {
      for (int i = tid; i < p.max_nodes; i += kVsThreads) p.path[(int64_t)b * p.max_nodes + i] = -1;
      if (tid == 0) p.n_accepted[b] = -1, p.next[b] = -1;
    }
    return;
  }
  const int m = min(end - start, p.max_nodes);
  const bool valid_T = T >= 0.f && T <= 1e6f;
  const bool greedy = T <= 1e-6f;  // (the fp32 number 1e-6 is below 1e-6)
  const bool drawn = DRAFT && p.draft && !greedy;
  // log2(e) / T in two parts
  const float div = greedy || !valid_T ? 1.f : T;
  const float ch = __fdiv_rn(1.44269502f, div), c_lo = __fdiv_rn(fmaf(-ch, div, 1.44269502f) + 1.92596299e-8f, div);
  // steps of the whole sums: below 2^62 for V weights of at most 2^0.5 each
  const float scale = __uint_as_float((uint32_t)(127 + 61 - (32 - __clz(p.V))) << 23);
  if (tid < kVsNodes) {
    w.path[tid] = tid == 0 ? 0 : -1;
    w.parent[tid] = -2;
    if (tid < m) {
      w.parent[tid] = p.parents ? p.parents[start + tid] : tid - 1;
      w.token[tid] = p.tokens[start + tid];
      w.u[tid] = p.uniforms[start + tid];
    }
  }
  cl.barrier_wait();
  __syncthreads();

  int node = 0, length = 1, turn = 0;
  int next = -1;
  bool writes = rank == 0 && tid == 0;  // the thread that stores the next token
  while (valid_T) {
    const In* pe = static_cast<const In*>(p.logits) + (int64_t)(start + node) * p.stride;
    const In* pf = drawn ? static_cast<const In*>(p.draft) + (int64_t)(start + node) * p.draft_stride : pe;
    const int skew = skew_of(pe);
    const Row<In> re{pe, p.V, skew, true}, rf{pf, p.V, skew, skew_of(pf) == skew};
    const int n_vec = (p.V + skew + N - 1) / N;
    // ranges of whole vectors, a warp each: warp w of block r has the range 8 r + w
    const int n_ranges = kVsWarps << p.log_c, per = (n_vec + n_ranges - 1) >> (kVsLogWarps + p.log_c);
    const int j0 = min(n_vec, (rank * kVsWarps + warp) * per), j1 = min(n_vec, j0 + per);

    // ---- the children; the first warp asks for their logits (a lane a child)
    const bool kid0 = lane > node && w.parent[lane] == node, kid1 = lane + 32 > node && w.parent[lane + 32] == node;
    const uint32_t set0 = __ballot_sync(0xffffffffu, kid0), set1 = __ballot_sync(0xffffffffu, kid1);
    const int n_children = __popc(set0) + __popc(set1);
    const bool both = drawn && n_children > 0;  // the draft's row matters
    const bool kid[2] = {kid0, kid1};
    int my_token[2] = {-1, -1};
    float my_x[2] = {0.f, 0.f}, my_y[2] = {0.f, 0.f};
    if (warp == 0) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (!kid[k]) continue;
        my_token[k] = w.token[lane + 32 * k];
        if (my_token[k] >= 0 && my_token[k] < p.V) {
          my_x[k] = Load<In>::one(pe + my_token[k]);
          if (both) my_y[k] = Load<In>::one(pf + my_token[k]);
        }
      }
    }

    // ---- the largest logits and, for children, their sums in fp32: half of the warps a row
    const int log_t = both ? kVsLogWarps - 1 : kVsLogWarps, team_warps = 1 << log_t, team = warp >> log_t;
    const int per_t = (n_vec + (team_warps << p.log_c) - 1) >> (log_t + p.log_c);
    {
      const Row<In>& row = team ? rf : re;
      const int a0 = min(n_vec, (rank * team_warps + (warp & (team_warps - 1))) * per_t), a1 = min(n_vec, a0 + per_t);
      Soft a{-INFINITY, 0.f};
      uint64_t best = 0;
      auto one = [&](const float (&x)[N], int e) {
        float mx = x[0];
#pragma unroll
        for (int i = 1; i < N; ++i) mx = max_nan(mx, x[i]);
        if (greedy) {
#pragma unroll
          for (int i = 0; i < N; ++i)
            if (x[i] > a.m) best = order_key(x[i], e + i), a.m = x[i];
        }
        if (greedy || n_children == 0) {
          a.m = max_nan(a.m, mx);
          return;
        }
        raise(a, mx, ch);
        const float base = a.m == -INFINITY ? 0.f : -a.m * ch;
#pragma unroll
        for (int i = 0; i < N; ++i) a.s += exp2_fast(fmaf(x[i], ch, base));
      };
      row.template each<kVsBatch>(a0, a1, [&](const uint4 (&v)[kVsBatch], int n, int j) {
        const float mx = Load<In>::most(v);
        if (greedy && mx > a.m) {
#pragma unroll
          for (int k = 0; k < kVsBatch; ++k) {
            float x[N];
            Load<In>::unpack(v[k], x);
#pragma unroll
            for (int i = 0; i < N; ++i)
              if (x[i] > a.m) best = order_key(x[i], (j + 32 * k) * N - skew + i), a.m = x[i];
          }
        }
        if (greedy || n_children == 0) {
          a.m = max_nan(a.m, mx);
          return;
        }
        raise(a, mx, ch);
        const float base = a.m == -INFINITY ? 0.f : -a.m * ch;
        uint64_t s[2] = {0, 0};
#pragma unroll
        for (int k = 0; k < kVsBatch; ++k) {
          if (k >= n) break;
          float x[N];
          Load<In>::unpack(v[k], x);
#pragma unroll
          for (int i = 0; i < N; i += 2) {
            const uint64_t y = f2_fma(f2(x[i], x[i + 1]), f2(ch, ch), f2(base, base));
            s[(i >> 1) & 1] = f2_add(s[(i >> 1) & 1], f2(exp2_fast(f2_lo(y)), exp2_fast(f2_hi(y))));
          }
        }
        s[0] = f2_add(s[0], s[1]);
        a.s += f2_lo(s[0]) + f2_hi(s[0]);
      }, one);
      a = warp_soft(a, ch);
      if (greedy) best = warp_best(best);
      if (lane < 1 << p.log_c) {  // a lane a block
        Walk* q = cl.map_shared_rank(&w, lane);
        const int at = ((team * team_warps) << p.log_c) + rank * team_warps + (warp & (team_warps - 1));
        q->soft[turn][at] = a;
        if (greedy) q->best[turn][at] = best;
      }
    }
    cl.sync();
    if (warp == 0) {
      // a lane's parts; where the draft's row is read, half a warp a row
      Soft s[kGroup], a{-INFINITY, 0.f};
      uint64_t best = 0;
      const int parts = both ? n_ranges >> 1 : n_ranges, step = both ? 16 : 32, first = lane & (step - 1);
      const int row_at = both && lane >= 16 ? parts : 0;
#pragma unroll
      for (int g = 0; g < kGroup; ++g) {
        const int i = first + step * g;
        s[g] = Soft{-INFINITY, 0.f};
        if (i < parts) {
          s[g] = w.soft[turn][row_at + i];
          if (greedy) best = w.best[turn][i] > best ? w.best[turn][i] : best;
        }
        a.m = max_nan(a.m, s[g].m);
      }
#pragma unroll
      for (int g = 0; g < kGroup; ++g) a.s += s[g].m == -INFINITY ? 0.f : s[g].s * exp2_fast((s[g].m - a.m) * ch);
      a = warp_soft(a, ch, both);
      const Soft e{__shfl_sync(0xffffffffu, a.m, 0), __shfl_sync(0xffffffffu, a.s, 0)};
      const Soft f{__shfl_sync(0xffffffffu, a.m, 16), __shfl_sync(0xffffffffu, a.s, 16)};
      int act = kDraw, at = 0;
      if (!(e.m > -INFINITY && e.m < INFINITY)) {
        at = -1;  // no distribution (NaN, +inf, or nothing left)
      } else if (greedy) {
        at = (int)~(uint32_t)warp_best(best);
        const uint32_t hit0 = __ballot_sync(0xffffffffu, my_token[0] == at), hit1 = __ballot_sync(0xffffffffu, my_token[1] == at);
        if (hit0 | hit1) act = kGoOn, at = hit0 ? __ffs(hit0) - 1 : 31 + __ffs(hit1);
      } else if (n_children > 0 && (!drawn || (f.m > -INFINITY && f.m < INFINITY))) {
        // a child that is accepted by a margin above the fp32 sums' error: the most
        // likely end of a step.  (Errors, relative: 2^-22 of an exponential and of
        // each time a sum is rescaled, 2^-24 an addition; of an argument y = c l - c m
        // 2^-24 (|y| + |c m|) ln 2, where the weights 2^y bring |y| to log2(V) at most.)
        const float slack = 1e-5f + 3e-7f * (float)(per_t * N / 32 + 1) + 1.2e-7f * fmaxf(fabsf(e.m * ch), both ? fabsf(f.m * ch) : 0.f);
        float left = e.s;
        bool sure = true;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const bool is = kid[k] && my_token[k] >= 0 && my_token[k] < p.V;
          const float we = exp2_fast((my_x[k] - e.m) * ch), wf = both ? exp2_fast((my_y[k] - f.m) * ch) : 0.f, u = w.u[lane + 32 * k];
          uint32_t set = __ballot_sync(0xffffffffu, is);
          if (k == 1 && set && !both) {  // (without those whose token an earlier child had)
            uint32_t again = 0;
            for (uint32_t s = set0; s; s &= s - 1) again |= __ballot_sync(0xffffffffu, my_token[1] == __shfl_sync(0xffffffffu, my_token[0], __ffs(s) - 1));
            set &= ~again;
          }
          while (set && sure) {
            const int i = __ffs(set) - 1;
            const float ui = __shfl_sync(0xffffffffu, u, i), ei = __shfl_sync(0xffffffffu, we, i), fi = __shfl_sync(0xffffffffu, wf, i);
            const float r = both ? f.s * ei : ei, x = both ? ui * e.s * fi : ui * left;
            const float near = both ? 2.f * slack * (x + r) : slack * (ui * e.s + r);
            if (r - x > near) act = kGoOn, at = i + 32 * k;
            if (both && x - r > near) act = kSureReject, at = i + 32 * k;
            sure = !both && x - r > near;  // (of drawn drafts the first alone; not sure to be rejected)
            left -= ei;
            set &= ~__ballot_sync(0xffffffffu, my_token[k] == __shfl_sync(0xffffffffu, my_token[k], i));  // (and its like)
          }
        }
      }
      if (act == kSureReject) {
        // k as it is about (units: see row_exp); above 4 the draft's weights would leave theirs
        const RowExp x = row_exp(e.m, ch, c_lo), y = row_exp(f.m, ch, c_lo);
        const float k0 = e.s * exp2_fast((e.m - x.ref) * ch - x.top) / (f.s * exp2_fast((f.m - y.ref) * ch - y.top));
        if (!(k0 <= 4.f)) act = kDraw;
        if (lane == 0) w.kf = scaled(y, (double)k0, w.table), w.kappa = (double)k0;
      }
      if (lane == 0) w.act = act, w.at = at, w.most = e.m, w.most_f = both ? f.m : -INFINITY;
    }
    turn ^= 1;
    __syncthreads();
    if (w.act == kGoOn) {
      node = w.at;
      if (tid == 0) w.path[length] = node;
      ++length;
      __syncthreads();
      continue;
    }
    if (greedy || w.at < 0) {
      next = w.at;
      break;
    }
    const float most = w.most, most_f = w.most_f;
    const bool judged = both && most_f > -INFINITY && most_f < INFINITY;  // the draft's row is a distribution
    const RowExp ee = row_exp(most, ch, c_lo);
    RowExp ef = row_exp(judged ? most_f : 0.f, ch, c_lo);
    RowExp kf = ef;  // the draft's times kappa

    // ---- else the sums in more bits
    auto whole_weight = [&](float x, const RowExp& x_of) {
      const Parts r = parts(weight(x, x, x_of, w.table));
      return fixed(f2_lo(r.hi), f2_lo(r.lo), scale);
    };
    if (warp == 0) {  // the children in order, and their weights
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (!kid[k]) continue;
        const int i = (k ? __popc(set0) : 0) + __popc((k ? set1 : set0) & ((1u << lane) - 1));
        const bool is = my_token[k] >= 0 && my_token[k] < p.V;
        w.child[i] = lane + 32 * k;
        w.child_e[i] = is ? whole_weight(my_x[k], ee) : -1;
        w.child_f[i] = is && judged ? whole_weight(my_y[k], ef) : 0;
        w.child_at[i] = is ? (my_token[k] + skew) / N / per : 0;
        w.gone[i] = false;
      }
    }
    double kappa = 0.0;
    // Sums of parts: to a pair every 32 elements, while the high ones' sum is exact.
    struct Sum {
      Pair a{0.f, 0.f};
      uint64_t hi = 0, lo = 0;
      __device__ void add(const Parts& r) {
        hi = f2_add(hi, r.hi);
        lo = f2_add(lo, r.lo);
      }
      __device__ void flush() {
        accumulate(a, Pair{__fadd_rn(f2_lo(hi), f2_hi(hi)), __fadd_rn(f2_lo(lo), f2_hi(lo))});
        hi = lo = 0;
      }
    };
    auto total = [&](const Row<In>& row, const RowExp& x_of) {  // this warp's range of a row
      Sum sum;
      auto one = [&](const float (&x)[N], int) {
#pragma unroll
        for (int k = 0; k < N; k += 2) sum.add(parts(weight(x[k], x[k + 1], x_of, w.table)));
        sum.flush();
      };
      row.template each<kVsBatch>(j0, j1, [&](const uint4 (&v)[kVsBatch], int n, int) {
#pragma unroll
        for (int k = 0; k < kVsBatch; ++k) {
          if (k >= n) break;
          float x[N];
          Load<In>::unpack(v[k], x);
#pragma unroll
          for (int i = 0; i < N; i += 2) sum.add(parts(weight(x[i], x[i + 1], x_of, w.table)));
        }
        sum.flush();
      }, one);
      const Pair a = warp_pair(sum.a);
      return fixed(a.h, a.l, scale);
    };
    // This warp's range of both rows, the next vectors on their way; flush() behind
    // every 32 tokens of a lane (16 of each half of the sums: below 2^7, exact).
    auto for_both = [&](auto add, auto flush) {
      int round = 0;
      if (j0 < j1 && re.whole(j0) && re.whole(j1 - 1) && rf.aligned) {
        uint4 ve = re.raw_or_none(j0 + lane, j1), vf = rf.raw_or_none(j0 + lane, j1);
#pragma unroll 1
        for (int j = j0 + lane; j < j1; j += 32) {
          float xe[N], xf[N];
          Load<In>::unpack(ve, xe);
          Load<In>::unpack(vf, xf);
          ve = re.raw_or_none(j + 32, j1);
          vf = rf.raw_or_none(j + 32, j1);
          add(xe, xf);
          if ((++round & (32 / N - 1)) == 0) flush();
        }
      } else {
#pragma unroll 1
        for (int j = j0 + lane; j < j1; j += 32) {
          float xe[N], xf[N];
          re.load(j, xe);
          rf.load(j, xf);
          add(xe, xf);
          if ((++round & (32 / N - 1)) == 0) flush();
        }
      }
      flush();
    };
    auto total_left = [&]() {  // of what is left, with the draft's part taken out
      Sum sum;
      for_both([&](const float (&xe)[N], const float (&xf)[N]) {
#pragma unroll
        for (int i = 0; i < N; i += 2)
          sum.add(residual(parts(weight(xe[i], xe[i + 1], ee, w.table)), parts(weight<true>(xf[i], xf[i + 1], kf, w.table))));
      }, [&]() { sum.flush(); });
      const Pair a = warp_pair(sum.a);
      return fixed(a.h, a.l, scale);
    };
    auto sums = [&](bool draft) {  // this warp's range: what is left of the target's weights, and the draft's, to all blocks
      const int64_t e = kappa > 0.0 ? total_left() : total(re, ee), f = draft ? total(rf, ef) : 0;
      if (lane < 1 << p.log_c) {
        Walk* q = cl.map_shared_rank(&w, lane);
        q->sum[turn][rank * kVsWarps + warp] = e;
        if (draft) q->sum_f[turn][rank * kVsWarps + warp] = f;
      }
    };
    // of the first warp's lanes, in order: the ranges group * lane on
    const int group = max(n_ranges >> 5, 1);
    int64_t mine[kGroup], Z = 0, F = 0;
    auto gather = [&](bool draft) {  // the sums of all ranges, to the first warp
      cl.sync();
      if (warp == 0) {
        int64_t s = 0, d = 0;
#pragma unroll
        for (int g = 0; g < kGroup; ++g) {
          const int i = lane * group + g;
          mine[g] = 0;
          if (g < group && i < n_ranges) {
            mine[g] = w.sum[turn][i];
            if (draft) d += w.sum_f[turn][i];
          }
          s += mine[g];
        }
        Z = warp_total(s);
        if (draft) F = warp_total(d);
      }
      turn ^= 1;
    };
    // (the first warp's)
    double left = 1.0;   // of the draft's weights, F in all, what is not rejected
    bool spent = false;  // nothing is
    int cursor = 0;
    // vector j without the rejected tokens
    auto drop = [&](int j, float (&x)[N]) {
      for (int i = 0; i < n_children; ++i) {
        const int k = w.token[w.child[i]] - (j * N - skew);
        if (!w.gone[i] || k < 0 || k >= N) continue;
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (e == k) x[e] = -INFINITY;
      }
    };
    // What the rejected tokens leave of the draft's row: F its sum, and its weights,
    // in units of the largest that is left.
    auto sum_again = [&]() {
      const int here = rank * kVsWarps + warp;
      bool any = false;  // of the rejected tokens one lies in this warp's range
      for (int i = 0; i < n_children; ++i) any |= w.gone[i] && w.child_at[i] == here;
      auto each_left = [&](auto one) {
#pragma unroll 1
        for (int j = j0 + lane; j < j1; j += 32) {
          float x[N];
          rf.load(j, x);
          if (any) drop(j, x);
          one(x);
        }
      };
      float m = -INFINITY;
      each_left([&](const float (&x)[N]) {
#pragma unroll
        for (int i = 0; i < N; ++i) m = fmaxf(m, x[i]);
      });
#pragma unroll
      for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (lane < 1 << p.log_c) cl.map_shared_rank(&w, lane)->soft[turn][here] = Soft{m, 0.f};
      cl.sync();
      for (int i = lane; i < n_ranges; i += 32) m = fmaxf(m, w.soft[turn][i].m);
#pragma unroll
      for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      turn ^= 1;
      if (!((most_f - m) * ch <= kNothingLeft)) {  // (all threads of the cluster)
        spent = true;
        return;
      }
      // (the reference stays: differences from it are as exact as before)
      const RowExp now = row_exp(ef.ref, m, ch, c_lo);
      kappa *= __hiloint2double((1023 + (int)(now.top - ef.top)) << 20, 0);
      ef = now;
      Sum sum;
      each_left([&](const float (&x)[N]) {
#pragma unroll
        for (int i = 0; i < N; i += 2) sum.add(parts(weight(x[i], x[i + 1], ef, w.table)));
        sum.flush();
      });
      const Pair a = warp_pair(sum.a);
      const int64_t f = fixed(a.h, a.l, scale);
      if (lane < 1 << p.log_c) cl.map_shared_rank(&w, lane)->sum_f[turn][here] = f;
      cl.sync();
      if (warp == 0) {
        int64_t d = 0;
        for (int i = lane; i < n_ranges; i += 32) d += w.sum_f[turn][i];
        F = warp_total(d);
        left = 1.0;
        for (int i = lane; i < n_children; i += 32)
          if (w.child_e[i] >= 0 && !w.gone[i]) w.child_f[i] = whole_weight(Load<In>::one(pf + w.token[w.child[i]]), ef);
        __syncwarp();
      }
      turn ^= 1;
    };
    if (w.act != kSureReject) {
      sums(judged);
      gather(judged);
    } else {
      // The first draft is surely rejected.  Both rows' sums and what is left in one
      // pass, with k as the fp32 sums have it, k0: of what is left R(k0) = sum over
      // {e > k0 f} of e - k0 f, R(k0 (1 + d)) = R(k0) - d sum over the same of k0 f,
      // but for the tokens that change sides, which have |e - k0 f| <= d k0 f and
      // change it by d of their k0 f at most.  So the k0 f of those within 2^-13, 2^-15,
      // 2^-17 and 2^-19 are summed too: d, which is known afterwards, is mostly 2^-20.
      const double k0 = w.kappa;
      const int first_child = w.at;
      kf = w.kf;
      Sum all_e, all_f, rest, taken;
      float near[kVsBands] = {};
      auto note = [&](float d, float b) {
#pragma unroll
        for (int k = 0; k < kVsBands; ++k)
          if (fabsf(d) <= band(k) * b) near[k] += b;
      };
      // (few tokens are near, so they are told by one branch for all of a vector's)
      auto add = [&](const float (&xe)[N], const float (&xf)[N]) {
        float d1[N], b1[N];
        bool close = false;
#pragma unroll
        for (int i = 0; i < N; i += 2) {
          const Parts a = parts(weight(xe[i], xe[i + 1], ee, w.table)), b = parts(weight<true>(xf[i], xf[i + 1], kf, w.table));
          Parts r{f2_sub(a.hi, b.hi), f2_sub(a.lo, b.lo)}, c = b;
          const uint64_t d = f2_add(r.hi, r.lo);
          if (!(f2_lo(d) > 0.f)) r.hi &= 0xFFFFFFFF00000000ull, r.lo &= 0xFFFFFFFF00000000ull, c.hi &= 0xFFFFFFFF00000000ull, c.lo &= 0xFFFFFFFF00000000ull;
          if (!(f2_hi(d) > 0.f)) r.hi &= 0xFFFFFFFFull, r.lo &= 0xFFFFFFFFull, c.hi &= 0xFFFFFFFFull, c.lo &= 0xFFFFFFFFull;
          const uint64_t whole = f2_add(b.hi, b.lo);
          d1[i] = f2_lo(d), d1[i + 1] = f2_hi(d);
          b1[i] = f2_lo(whole), b1[i + 1] = f2_hi(whole);
          close |= (fabsf(d1[i]) <= band(0) * b1[i]) | (fabsf(d1[i + 1]) <= band(0) * b1[i + 1]);
          all_e.add(a);
          all_f.add(b);
          rest.add(r);
          taken.add(c);
        }
        if (close) {
#pragma unroll
          for (int i = 0; i < N; ++i) note(d1[i], b1[i]);
        }
      };
      for_both(add, [&]() {
        all_e.flush();
        all_f.flush();
        rest.flush();
        taken.flush();
      });
      auto fixed_of = [&](const Sum& s) {
        const Pair a = warp_pair(s.a);
        return fixed(a.h, a.l, scale);
      };
      const int64_t v[4] = {fixed_of(rest), fixed_of(taken), fixed_of(all_e), fixed_of(all_f)};
#pragma unroll
      for (int k = 0; k < kVsBands; ++k) near[k] = warp_sum(near[k]);
      if (lane < 1 << p.log_c) {
        Walk* q = cl.map_shared_rank(&w, lane);
        const int i = rank * kVsWarps + warp;
        q->sum[turn][i] = v[0];
        q->sum_f[turn][i] = v[1];
        q->whole_e[i] = v[2];
        q->whole_f[i] = v[3];
#pragma unroll
        for (int k = 0; k < kVsBands; ++k) q->near[k][i] = near[k];
      }
      gather(true);
      if (warp == 0) {
        int64_t te = 0, tf = 0;
        for (int i = lane; i < n_ranges; i += 32) te += w.whole_e[i], tf += w.whole_f[i];
        te = warp_total(te);
        tf = warp_total(tf);
        const float d = __fdiv_rn((float)(te - tf), (float)tf);
        const int64_t f_all = __double2ll_rn((double)tf * reciprocal(k0));
        int within = -1;  // the narrowest band that holds all that change sides
#pragma unroll
        for (int k = 0; k < kVsBands; ++k)
          if (fabsf(d) < 0.9f * band(k)) within = k;
        float tn = 0.f;
        if (within >= 0)
          for (int i = lane; i < n_ranges; i += 32) tn += w.near[within][i];
        tn = warp_sum(tn);
        const bool good = within >= 0 && fabsf(d) * tn * scale <= 0x1p-33f * (float)Z;
        if (good) {
          int64_t s = 0;
#pragma unroll
          for (int g = 0; g < kGroup; ++g) {
            const int i = lane * group + g;
            if (g < group && i < n_ranges) mine[g] -= __float2ll_rn(d * (float)w.sum_f[turn ^ 1][i]);
            if (mine[g] < 0) mine[g] = 0;
            s += mine[g];
          }
          Z = warp_total(s);
          kappa = fma(k0, (double)d, k0);
          kf = scaled(ef, kappa, w.table);
          for (int i = 0; i < n_children; ++i)
            if (w.child[i] == first_child) {
              cursor = i + 1;
              if (!p.replacement) {
                left = 1.0 - (double)w.child_f[i] * reciprocal((double)f_all);
                if (lane == 0) w.gone[i] = true;
              }
            }
        } else {
          Z = te;
        }
        F = f_all;
        if (lane == 0) w.kappa = good ? kappa : 0.0, w.kf = kf;
      }
      __syncthreads();
      kappa = w.kappa;
      kf = w.kf;
      __syncthreads();
    }

    // ---- the children in order (each block's first warp decides, all of them the same)
    while (true) {
      if (warp == 0) {
        int act = kDraw, at = 0;
        for (int i = cursor; i < n_children; ++i) {
          const int x = w.token[w.child[i]];
          const int64_t e = w.child_e[i], f = w.child_f[i];
          if (e < 0 || (drawn && !judged) || spent) continue;  // no such token, or nothing to judge it by: passed over
          if (!judged || !p.replacement) {
            bool again = false;  // an earlier sibling's token
            for (int k = 0; k < i; ++k) again |= w.token[w.child[k]] == x;
            if (again) continue;
          }
          if (judged && left < kFewLeft) {
            cursor = i;
            act = kRest;
            break;
          }
          const double side = (double)w.u[w.child[i]] * (double)Z;
          if (judged ? side * (double)f < left * (double)F * ((double)e - kappa * (double)f) : side < (double)e) {
            act = kGoOn;
            at = w.child[i];
            break;
          }
          if (!judged) {
            Z -= e;
            if (lane == 0) w.gone[i] = true;
          } else if (Z > 0) {
            kappa += (double)Z * reciprocal(left * (double)F);
            if (!p.replacement) {
              left -= (double)f * reciprocal((double)F);
              if (lane == 0) w.gone[i] = true;
            }
            cursor = i + 1;
            act = kReject;
            break;
          }
        }
        if (act == kReject) kf = scaled(ef, kappa, w.table);
        if (lane == 0) w.act = act, w.at = at, w.kappa = kappa, w.kf = kf;
      }
      __syncthreads();
      if constexpr (DRAFT) {
        if (w.act == kRest) {
          sum_again();
          continue;
        }
      }
      if (w.act != kReject) break;
      kappa = w.kappa;
      kf = w.kf;
      sums(false);
      gather(false);
    }
    if (w.act == kGoOn) {
      node = w.at;
      if (tid == 0) w.path[length] = node;
      ++length;
      __syncthreads();
      continue;
    }

    // ---- the next token: the range that holds the number's place, a thread's vectors of it, the token
    if (warp == 0) {
      if (!judged) {  // what the rejected drafts that were chosen leave of the ranges' sums
        for (int i = 0; i < n_children; ++i) {
          if (!w.gone[i]) continue;
          const int at = w.child_at[i];
#pragma unroll
          for (int g = 0; g < kGroup; ++g)
            if (at == lane * group + g) {
              const int64_t rest = mine[g] - w.child_e[i];
              mine[g] = rest > (mine[g] >> 36) + 16 ? rest : 0;  // (all of it: no rounding stays)
            }
        }
        int64_t s = 0;
#pragma unroll
        for (int g = 0; g < kGroup; ++g) s += mine[g];
        Z = warp_total(s);
      }
      if (lane == 0) w.at = Z > 0;
    }
    __syncthreads();
    bool out = !judged && w.at;        // the rejected tokens' own weights are out
    if (!w.at) {                       // nothing is left: the target's own weights
      kappa = 0.0;
      sums(false);
      gather(false);
    }
    if (warp == 0) {
      int64_t s = 0, before;
#pragma unroll
      for (int g = 0; g < kGroup; ++g) s += mine[g];
      const int64_t t = __double2ll_rd((double)w.u[0] * (double)Z);  // (a whole sum passes the number where it passes this)
      const int from = max(pick(s, t, lane, before), 0);
      if (lane == from) {
        int64_t run = before, mass = 1;
        int at = 0;
        bool found = false;
#pragma unroll
        for (int g = 0; g < kGroup; ++g) {
          if (found || mine[g] <= 0) continue;
          at = g;
          mass = mine[g];
          before = run;
          run += mass;
          found = run > t;
        }
        // In the range the steps are finer, its mass 2^49 of them at least: in a long
        // row, or behind rejected drafts, a token may have less than one of the row's,
        // and many roundings of half a step would add up.
        const int up = max(__clzll(mass) - 14, 0);
        w.range = lane * group + at;
        w.up = up;
        const int64_t place = t - before;
        w.threshold = place < 0 ? -1 : (place < mass ? place : mass) << up;
        w.found = -1;
      }
    }
    __syncthreads();
    writes = false;
    if (rank != w.range / kVsWarps) break;
    const int k0 = min(n_vec, w.range * per), k1 = min(n_vec, k0 + per), each = (per + kVsThreads - 1) / kVsThreads;
    const int a0 = min(k1, k0 + tid * each), a1 = min(k1, a0 + each);
    auto load = [&](int j, float (&xe)[N], float (&xf)[N]) {  // vector j, without the tokens that are out
      re.load(j, xe);
      if (kappa > 0.0) rf.load(j, xf);
      if (out) drop(j, xe);
    };
    auto left_of = [&](const float (&xe)[N], const float (&xf)[N], int k) {  // what is left of two weights
      const Parts a = parts(weight(xe[k], xe[k + 1], ee, w.table));
      return kappa > 0.0 ? residual(a, parts(weight<true>(xf[k], xf[k + 1], kf, w.table))) : a;
    };
    // in the finer steps; h and l may be large and of opposite signs beside their sum
    // (held where the range's sum, corrected or short of a rejected draft, says less
    // than its tokens have: sums of these stay below 2^63)
    const float fine = scale * __uint_as_float((uint32_t)(127 + w.up) << 23), most_fine = w.up > 0 ? 0x1p51f : INFINITY;
    auto finer = [&](float h, float l) {
      const float t = __fadd_rn(h, l), z = __fsub_rn(t, h);
      const float e = __fadd_rn(__fsub_rn(h, __fsub_rn(t, z)), __fsub_rn(l, z));
      return __float2ll_rn(fminf(t * fine, most_fine)) + __float2ll_rn(e * fine);
    };
    auto whole_left = [&](const float (&xe)[N], const float (&xf)[N], int64_t (&r)[N]) {
#pragma unroll
      for (int k = 0; k < N; k += 2) {
        const Parts a = left_of(xe, xf, k);
        r[k] = finer(f2_lo(a.hi), f2_lo(a.lo));
        r[k + 1] = finer(f2_hi(a.hi), f2_hi(a.lo));
      }
    };
    float xe[N], xf[N];
    int64_t r[N], own = 0;  // (one vector a thread: the next step has its r still)
    if (a0 < a1) load(a0, xe, xf);
    if (each > 1) {
      Sum sum;
#pragma unroll 1
      for (int j = a0; j < a1; ++j) {
        float ye[N], yf[N];
        if (j + 1 < a1) load(j + 1, ye, yf);
#pragma unroll
        for (int k = 0; k < N; k += 2) sum.add(left_of(xe, xf, k));
        sum.flush();
#pragma unroll
        for (int k = 0; k < N; ++k) xe[k] = ye[k], xf[k] = yf[k];
      }
      own = finer(sum.a.h, sum.a.l);
    } else if (a0 < a1) {
      whole_left(xe, xf, r);
#pragma unroll
      for (int k = 0; k < N; ++k) own += r[k];
    }
    const int64_t of_warp = warp_total(own);
    if (lane == 0) w.part[warp] = of_warp;
    __syncthreads();
    if (warp == 0) {
      int64_t before;
      const int at = pick(lane < kVsWarps ? w.part[lane] : 0, w.threshold, lane, before);  // (-1: see below)
      if (lane == 0) w.winner = at, w.threshold -= before;
    }
    __syncthreads();
    if (warp == w.winner) {  // a lane a vector of the thread's that has the place
      int64_t before;
      const int at = max(pick(own, w.threshold, lane, before), 0);
      const int b0 = __shfl_sync(0xffffffffu, a0, at), b1 = __shfl_sync(0xffffffffu, a1, at);
      int64_t t = w.threshold - before;
      bool passed = false;
#pragma unroll 1
      for (int j0 = b0; j0 < b1 && !passed; j0 += 32) {
        int j = a0, by = at;
        int64_t all = 0;
        before = 0;
        if (each > 1) {
          j = j0 + lane;
          if (j < b1) {
            load(j, xe, xf);
            whole_left(xe, xf, r);
#pragma unroll
            for (int k = 0; k < N; ++k) all += r[k];
          }
          by = pick(all, t, lane, before);
        }
        int token = -1;
        if (lane == by) {
          int64_t run = before;
          bool found = false;
#pragma unroll
          for (int k = 0; k < N; ++k) {
            if (found || r[k] <= 0) continue;
            token = j * N - skew + k;  // (the last with any where rounding leaves none that passes)
            run += r[k];
            found = run > t;
          }
        }
        token = __shfl_sync(0xffffffffu, token, max(by, 0));
        if (token >= 0) next = token;
        if (each > 1) t -= warp_total(all);
        passed = t < 0;
      }
      writes = lane == 0;
      if (writes) w.found = next;
    }
    __syncthreads();
    if (w.found < 0) {
      // Rounding alone had put the place into this range: the first token from its
      // start on, and round the row's end, that has anything left; else that has any.
      constexpr int kRound = 1 << 26;
      const int from = k0 * N - skew;
#pragma unroll 1
      for (int all = 0; all < 2; ++all) {
        if (all) kappa = 0.0, out = false;
        if (tid == 0) w.at = 2 * kRound;
        __syncthreads();
        int first = 2 * kRound;
#pragma unroll 1
        for (int j = tid; j < n_vec; j += kVsThreads) {
          load(j, xe, xf);
#pragma unroll
          for (int k = 0; k < N; k += 2) {
            const Parts a = left_of(xe, xf, k);
            const uint64_t any = f2_add(a.hi, a.lo);
            const int id = j * N - skew + k - from;
            if (f2_hi(any) > 0.f) first = min(first, id + 1 >= 0 ? id + 1 : id + 1 + kRound);
            if (f2_lo(any) > 0.f) first = min(first, id >= 0 ? id : id + kRound);
          }
        }
        atomicMin(&w.at, first);
        __syncthreads();
        first = w.at;
        __syncthreads();
        if (first == 2 * kRound) continue;
        next = from + (first < kRound ? first : first - kRound);
        break;
      }
      writes = tid == 0;
    }
    break;
  }
  if (writes) p.next[b] = next;
  __syncthreads();
  if (rank == 0) {
    for (int i = tid; i < p.max_nodes; i += kVsThreads) p.path[(int64_t)b * p.max_nodes + i] = i < m ? w.path[i] : -1;
    if (tid == 0) p.n_accepted[b] = length - 1;
  }
  // (nothing is written to another block's memory after the last exchange)
}

template <typename In>
cudaError_t verify_sample_launch(const VsParams& p, cudaStream_t st) {
  const auto kernel = p.draft ? verify_sample_kernel<In, true> : verify_sample_kernel<In, false>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.n_seqs << p.log_c);
  cfg.blockDim = dim3(kVsThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1u << p.log_c;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (p.log_c > 3) {  // above the portable size
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  return cudaLaunchKernelEx(&cfg, kernel, p);
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
  VsParams p{logits, row_stride, draft_logits, draft_stride, V, n_seqs, n_nodes, max_nodes, replacement, 0,
             tokens, parents, starts, uniforms, temperature, path, out_n_accepted, out_next_token};
  while ((2 << p.log_c) <= kVsMaxCluster && ((int64_t)n_seqs << (p.log_c + 1)) <= (int64_t)kVsBlocks * sms && (V >> (p.log_c + 1)) >= 1024) ++p.log_c;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  e = dtype == MOE_ACT_F32 ? verify_sample_launch<float>(p, st) : verify_sample_launch<__nv_bfloat16>(p, st);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return set_error(MOE_ECUDA, "%s launch: %s", who, cudaGetErrorString(e));
  }
  return MOE_OK;
}

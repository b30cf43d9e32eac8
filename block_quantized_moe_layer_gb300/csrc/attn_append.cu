// attn_append.cu -- the step before attention: norms of the query and key
// heads, rotation, and the keys' and values' 4-bit rows in the paged cache.
//
// For a token at position p and a head x of D channels:
//   y_i = x_i / sqrt(mean(x^2) + eps) * w_i             (queries and keys, where the handle has weights)
//   y'_a = y_a cos(p f) - y_b sin(p f), y'_b = y_b cos(p f) + y_a sin(p f)   for the rotated pairs (a, b)
// Queries are rounded once to the output type.  Keys y' and values x are
// stored as codes: d = the scale nearest to amax / 7 of 16 channels (ties to
// the even fraction), c = 8 + round-half-even(y / d), clamped to 0..15; NaN is
// stored as 0 and larger values saturate.
//
// Work: one row (token, head) is D/16 lanes of 16 channels, which is a scale's
// block, two 16-byte loads a lane (four for fp32); the sum of squares (and the
// partners of a key's rotation) travel by shuffles, so a row is read once and
// written once.  With 16 channels a lane rather than 8, a warp's fixed costs
// (sums, roots, addresses, the search for a scale) serve twice the rows.  The
// bound is HBM: D (2 + 2) bytes of a query row, D (2 + 9/16) of a key or value
// row.  A group of lanes takes up to 2 query heads of one token, which share
// the angles' cosines and sines (from the handle's fp32 table, computed in
// fp64: far positions lose nothing).
//
// Codes are those of the exact result.  fp32 leaves each y' within
// 2^-19 (|y_a cos| + |y_b sin|) of it, 32 units of 2^-24: the sum of squares
// is off by 20 of them (16 products added in turn, 4 shuffles), its mean with
// eps by 2 more, of which the root halves all; the reciprocal root by 4; the
// weight's, the row's and the angle's product, the angle itself and the sum by
// one each: 20.  A row in which that error could change a scale or a code (about
// one in 500) has just those channels computed again in fp64.
// Values are exact already: their codes are decided by exact fp32 residuals.
//
// Measured: 4096 tokens of 64/4 heads of 192 in 59.8 us, and read back in 6.6
// (issue slots 60% busy, 20 warps a multiprocessor: the chains of a row's sum,
// its rotation and the search for its scale are what is waited for, and at 192
// channels 4 of a query row's 16 lanes hold none); 4 tokens in 2.7 us, of which
// a launch is 2, and read back in 1.7.  A row at a border adds its chain of
// fp64: 128 tokens of 32/8 heads of 128, which nearly always have one, take 5.7
// us (without norms and rotation, where there is none, 3.1), 4 tokens with one 5.4.
#include "attn.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kAppendThreads = 128;
constexpr int kAppendBlocks = 5;  // resident on a multiprocessor: 96 registers a thread (6 of them, with 80, cost a tenth)

struct AppendParams {
  const void *q, *k, *v;
  int64_t q_tok, q_head, k_tok, k_head, v_tok, v_head;  // elements
  const int32_t* positions;
  const int64_t* slots;
  uint8_t* pages;
  void* q_out;  // [T][hq][D]
  int T, hq, hk, P, pshift, n_pages, rot, interleaved, max_pos;
  bool q_norm, k_norm;
  float eps, inv_d;
  const float* rope;
  const float* rope_lo;
  const float* norm_w;
  int64_t head_bytes, page_bytes;
  int* status;
};

// The scale byte nearest to amax / 7, ties to the even byte: the exact amax is
// compared with 7 times the midpoints of neighbouring scales (8 bits, exact).
template <typename T>
__device__ __forceinline__ int scale_byte(T amax) {
  const float a = fminf((float)amax, 60000.f);
  int b = __half_as_ushort(__float2half_rz(a * (1.f / 7.f))) >> 7;
  b = min(max(b - 1, 0), kKvMaxScale);
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const float mid = 3.5f * (scale_value(b) + scale_value(b + 1));
    if constexpr (sizeof(T) == 4) {
      // at an odd b a tie goes up: an fp32 amax is at the midpoint or above if it is above the fp32 number before it
      b += amax > __int_as_float(__float_as_int(mid) - (b & 1)) ? 1 : 0;
    } else {
      b += ((b & 1) ? amax >= (T)mid : amax > (T)mid) ? 1 : 0;
    }
  }
  return min(b, kKvMaxScale);
}

// The code of x for scale d (rd = 1/d rounded), plus 8388608 * 1.5 as a float:
// its low bits are the code.  Round half even of the exact x / d, clamped: x
// times rd picks a candidate q at most one off; the residual x - q d does not
// round (both are multiples of the smaller unit and it is below 1.5 d), so
// comparing it with d/2 settles q.  unsure gets the bit where an x off by err
// could have another code (err < 0: x is exact).  Branch-free: the branches of an if form took
// 1100 instructions a row, this takes about 300.
constexpr float kRound = 12582912.f;  // 1.5 2^23: adding it rounds to an integer
__device__ __forceinline__ uint32_t code_bits(float x, float d, float rd, float err, uint32_t bit, uint32_t& unsure) {
  const float u = fminf(fmaxf(x * rd, -9.f), 8.f) + kRound;
  float q = u - kRound;
  const float r = fmaf(-q, d, x), h = 0.5f * d;
  const float edge = __int_as_float(__float_as_int(h) - (__float_as_int(u) & 1));  // an odd q gives way on a tie
  q += r > edge ? 1.f : 0.f;
  q -= r < -edge ? 1.f : 0.f;
  unsure |= fabsf(fabsf(r) - h) <= err ? bit : 0u;
  return __float_as_uint(fminf(fmaxf(q, -8.f), 7.f) + (kRound + 8.f));
}
// The same for an fp64 x.
__device__ __forceinline__ uint32_t code_bits(double x, float d, float rd) {
  const float u = fminf(fmaxf((float)x * rd, -9.f), 8.f) + kRound;
  float q = u - kRound;
  const double r = fma(-(double)q, (double)d, x), h = 0.5 * d;
  const bool odd = __float_as_int(u) & 1;
  q += (odd ? r >= h : r > h) ? 1.f : 0.f;
  q -= (odd ? r <= -h : r < -h) ? 1.f : 0.f;
  return __float_as_uint(fminf(fmaxf(q, -8.f), 7.f) + (kRound + 8.f));
}
// A word of 8 codes: channel e is nibble e/2 + 4 (e%2).
__device__ __forceinline__ uint32_t pack_codes(const uint32_t* c) {
  uint32_t w = 0, k = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int s = 4 * ((e >> 1) + 4 * (e & 1));
    w += c[e] << s;
    k += 0x4B400000u << s;
  }
  return w - k;  // without the float's exponent bits
}

// The partners of a rotation in halves (i, i + rot/2): a lane's channels 8 b
// .. 8 b + 7 (b = 0, 1) have theirs in lane src[b], in its half b ^ odd.
struct Partner {
  int src[2];
  bool rotated[2], first[2], odd;
};
__device__ __forceinline__ Partner partner_of(int L, int rot) {
  Partner a;
  const int lane = threadIdx.x & 31;
  a.odd = (rot >> 4) & 1;
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const int c = 16 * L + 8 * b;
    a.rotated[b] = c < rot;
    a.first[b] = c < (rot >> 1);
    const int q = a.rotated[b] ? (a.first[b] ? c + (rot >> 1) : c - (rot >> 1)) : c;
    a.src[b] = lane - L + (q >> 4);
  }
  return a;
}

// The angle index of a lane's channel i (of the first half, or its partner's).
__device__ __forceinline__ int angle_of(int L, int i, int rot, bool interleaved) {
  const int c = 16 * L + i;
  return interleaved ? c >> 1 : (c < (rot >> 1) ? c : c - (rot >> 1));
}

// Two floats in a register pair: the packed fp32 instructions halve the
// arithmetic of a row, which is what bounds it after HBM.
__device__ __forceinline__ uint64_t f2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void f2_get(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
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

__device__ __forceinline__ void copy16(void* smem, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(smem)), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A thread's 16-byte pieces of the rows it works on: kAhead tokens are on
// their way in shared memory while one is worked on.  Each thread reads only
// what it copied itself; a warp shares its token's angles.
// (One token ahead, in 5 blocks a multiprocessor, measures as two and better
// than three in 4 blocks: 57.7, 58.8 and 64.6 us for 4096 tokens of 64 / 4
// heads of 192.)
constexpr int kAhead = 1;
constexpr int kRing = kAhead + 1;

// Eight channels from a thread's pieces, as four pairs.
__device__ __forceinline__ void pairs8(const uint4* s, uint64_t* a, __nv_bfloat16*) {
  const uint4 u = *s;
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] = f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}
__device__ __forceinline__ void pairs8(const uint4* s, uint64_t* a, float*) {
  const uint4 u = s[0], v = s[kAppendThreads];
  a[0] = f2(__uint_as_float(u.x), __uint_as_float(u.y));
  a[1] = f2(__uint_as_float(u.z), __uint_as_float(u.w));
  a[2] = f2(__uint_as_float(v.x), __uint_as_float(v.y));
  a[3] = f2(__uint_as_float(v.z), __uint_as_float(v.w));
}
template <typename In>
__device__ __forceinline__ void copy8(uint4* s, const In* p) {
  copy16(s, p);
  if (sizeof(In) == 4) copy16(s + kAppendThreads, p + 4);
}
// A warp's copy of the angles of a position: cos [rot/2], sin [rot/2].
__device__ __forceinline__ void copy_angles(float* s, const AppendParams& p, int pos) {
  if (pos < 0 || pos >= p.max_pos) return;
  const float* r = p.rope + (int64_t)pos * p.rot;
  for (int i = 4 * (threadIdx.x & 31); i < p.rot; i += 128) copy16(s + i, r + i);
}

// A row whose mean square (with eps) v lies outside 2^-60 .. 2^100 is normalised
// at another scale, a power of two, so that its squares neither overflow nor
// vanish (|x| from 2^-149 to 2^128 at D <= 256).  Rare: without this a row above
// 2^64 would become zeros, and without eps one below 2^-75 infinities.
__device__ __forceinline__ bool norm_range(float v) {  // (not a NaN, nor 0)
  constexpr uint32_t kLow = (127 - 60) << 23, kHigh = (127 + 100) << 23;
  return __float_as_uint(v) - kLow <= kHigh - kLow;
}
__device__ __forceinline__ float norm_scale(float v) { return norm_range(v) ? 1.f : (v < 1.f ? 0x1p88f : 0x1p-70f); }

// x_hi + x_lo: the sum of squares of a lane's channels, each step's rounding
// error kept (two-sum; the square's own by an fma).
__device__ __forceinline__ double square_sum(const float (&x)[16]) {
  float hi = 0.f, lo = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float sq = x[i] * x[i], e = fmaf(x[i], x[i], -sq);
    const float s = hi + sq, b = s - hi;
    lo += ((hi - (s - b)) + (sq - b)) + e;
    hi = s;
  }
  return (double)hi + (double)lo;
}

// Channel i of a thread's row, from its pieces in a ring slot.
template <typename In>
__device__ __forceinline__ float ring_channel(const uint4* slot, int thread, int i) {
  constexpr int kPer = 16 / (int)sizeof(In);  // channels of a piece
  const In* piece = reinterpret_cast<const In*>(slot + (i / kPer) * kAppendThreads + thread);
  if constexpr (sizeof(In) == 2) return __bfloat162float(piece[i % kPer]);
  else return piece[i % kPer];
}

// The scale of a thread's row by its mean square v, and the mean square at that
// scale (the whole warp calls it).  A call, so that the rows of every day keep their registers.
template <int G, typename In>
__device__ __noinline__ float2 wide_norm(const uint4* slot, bool holds, float v, float inv_d, float eps) {
  const float scale = norm_scale(v);
  float ss = 0.f;
#pragma unroll 4
  for (int i = 0; i < 16; ++i) {
    const float x = holds ? ring_channel<In>(slot, threadIdx.x, i) * scale : 0.f;
    ss = fmaf(x, x, ss);
  }
#pragma unroll
  for (int o = G / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  return make_float2(scale, fmaf(ss, inv_d, eps * scale * scale));
}

// Settles in fp64 what fp32 left open in a warp's key rows (the whole warp
// calls it): the scales of lanes with `border`, then the codes of `unsure`.
// One channel a turn, with its partner and the row's sum: a row with one
// channel at a border pays some 25 dependent fp64 instructions.  (Whole rows in
// fp64 cost 400 and 10 to 14 us, with sincos instead of the two tables more:
// most of a small call, and the tail of a large one.)  The angles' cosines and
// sines are the sums of two fp32 tables, 2^-49 off.
template <int G, typename In>
__device__ __noinline__ void settle_rows(const uint4* slot, bool holds, const float (&y)[16], const float* w, double eps,
                                         int D, int L, int rot, bool interleaved, const float* hi, const float* lo, bool border,
                                         float amax, float emax, uint32_t unsure, int& sb, uint2& words) {
  const int lane = threadIdx.x & 31;
  double inv = 1.0;
  if (w) {
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = holds ? ring_channel<In>(slot, threadIdx.x, i) : 0.f;
    auto mean_square = [&]() {
      double ss = square_sum(x);
#pragma unroll
      for (int o = G / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      return ss * (1.0 / D);
    };
    double v = mean_square() + eps;
    const float scale = norm_scale((float)v);
    if (__any_sync(0xffffffffu, scale != 1.f)) {
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] *= scale;
      v = mean_square() + eps * scale * scale;
    }
    // a reciprocal square root by two Newton steps from the fp32 one (2^-22, 2^-43, 2^-53)
    inv = (double)rsqrtf((float)v);
#pragma unroll
    for (int i = 0; i < 2; ++i) inv = fma(inv * 0.5, fma(-v * inv, inv, 1.0), inv);
    inv *= scale;
  }
  // channel i of lane `who`, in fp64
  auto channel = [&](int who, int i) {
    const int Lw = who & (G - 1), c = 16 * Lw + i;
    const bool rotated = c < rot;
    const bool first = interleaved ? !(c & 1) : c < (rot >> 1);
    const int q = !rotated ? c : (interleaved ? c ^ 1 : (first ? c + (rot >> 1) : c - (rot >> 1)));
    const int row = (threadIdx.x & ~31) + who - Lw;  // the row's first thread
    double u = ring_channel<In>(slot, row + Lw, i), v = ring_channel<In>(slot, row + (q >> 4), q & 15);
    const double iw = __shfl_sync(0xffffffffu, inv, who);
    if (w) {
      u = u * iw * (double)w[c];
      v = v * iw * (double)w[q];
    }
    if (rotated) {
      const int f = interleaved ? c >> 1 : (first ? c : q), g = (rot >> 1) + f;
      const double cs = (double)hi[f] + lo[f], sn = (double)hi[g] + lo[g];
      u = first ? u * cs - v * sn : u * cs + v * sn;
    }
    return u;
  };
  // scales: the channels that may be the largest
  uint32_t large = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) large |= border && fabsf(y[i]) >= amax - 2.f * emax ? 1u << i : 0u;
  double most = 0.0;
  for (uint32_t any; (any = __ballot_sync(0xffffffffu, large != 0)) != 0;) {
    const int who = __ffs(any) - 1, i = __shfl_sync(0xffffffffu, __ffs(large) - 1, who);
    const double u = channel(who, i);
    if (lane == who) {
      most = fmax(most, fabs(u));
      large &= large - 1;
    }
  }
  if (border) {
    sb = scale_byte<double>(most);
    const float d = scale_value(sb), rd = 1.f / fmaxf(d, 0x1p-17f);
    uint32_t c[16];
    unsure = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) c[i] = code_bits(y[i], d, rd, emax, 1u << i, unsure);  // (the block's largest error for each)
    words = d > 0.f ? make_uint2(pack_codes(c), pack_codes(c + 8)) : make_uint2(0x88888888u, 0x88888888u);
    if (!(d > 0.f)) unsure = 0;
  }
  const float d = scale_value(sb);
  for (uint32_t any; (any = __ballot_sync(0xffffffffu, unsure != 0)) != 0;) {
    const int who = __ffs(any) - 1, i = __shfl_sync(0xffffffffu, __ffs(unsure) - 1, who);
    const double u = channel(who, i);
    if (lane == who) {
      const uint32_t code = code_bits(u, d, 1.f / d) & 15u;
      const int e = i & 7, s = 4 * ((e >> 1) + 4 * (e & 1));
      uint32_t& word = i < 8 ? words.x : words.y;
      word = (word & ~(15u << s)) | (code << s);
      unsure &= unsure - 1;
    }
  }
}

__device__ __forceinline__ void store8(__nv_bfloat16* p, const uint64_t* a) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float x, y;
    f2_get(a[i], x, y);
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float* p, const uint64_t* a) {
  float x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) f2_get(a[i], x[2 * i], x[2 * i + 1]);
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

// The query heads [h0, h0 + NB) of tokens t, t + step, ..., by the G lanes of
// a group.  Of the rotated channels a lane takes 8 and their 8 partners, so
// that a rotation needs no exchange; of the others 16 neighbours.
template <int G, int NB, typename In, typename Out>
__device__ __forceinline__ void query_heads(const AppendParams& p, int D, int t, int step, int h0, int L, const float* w_sm,
                                            uint4* ring, float* rope_sm) {
  const int rows = min(NB, p.hq - h0);
  const bool holds = 16 * L < D && rows > 0, rotated = 16 * L < p.rot, pairs = rotated && !p.interleaved;
  const int c0 = pairs ? 8 * L : 16 * L, c1 = pairs ? (p.rot >> 1) + 8 * L : 16 * L + 8;
  constexpr int kPieces = NB * 2 * (sizeof(In) / 2);
  const In* q = static_cast<const In*>(p.q) + t * p.q_tok + h0 * p.q_head;
  Out* out = static_cast<Out*>(p.q_out) + ((int64_t)t * p.hq + h0) * D;
  const int64_t q_step = step * p.q_tok, o_step = (int64_t)step * p.hq * D;
  uint4* mine = ring + threadIdx.x;
  auto issue = [&](int slot, int at, int pos) {  // token `at` into a slot
    if (at < p.T) {
      if (holds) {
#pragma unroll
        for (int i = 0; i < NB; ++i)
          if (i < rows) {
            uint4* s = mine + (slot * kPieces + i * (kPieces / NB)) * kAppendThreads;
            copy8(s, q + i * p.q_head + c0);
            copy8(s + kPieces / NB / 2 * kAppendThreads, q + i * p.q_head + c1);
          }
      }
      copy_angles(rope_sm + slot * p.rot, p, pos);
    }
    copies_commit();
    q += q_step;
  };
  auto position = [&](int at) { return at < p.T ? p.positions[at] : -1; };
  int pq[kRing];  // positions of tokens t, t + step, ...
#pragma unroll
  for (int i = 0; i < kRing; ++i) pq[i] = position(t + i * step);
#pragma unroll
  for (int i = 0; i < kAhead; ++i) issue(i, t + i * step, pq[i]);
  for (int slot = 0; t < p.T; t += step, slot = slot + 1 == kRing ? 0 : slot + 1) {
    const int after = position(t + kRing * step);
    issue(slot == 0 ? kRing - 1 : slot - 1, t + kAhead * step, pq[kAhead]);
    copies_wait<kAhead>();
    __syncwarp();
    const bool pos_ok = pq[0] >= 0 && pq[0] < p.max_pos;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) pq[i] = pq[i + 1];
    pq[kAhead] = after;
    uint64_t x[NB][8];
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const uint4* s = mine + (slot * kPieces + i * (kPieces / NB)) * kAppendThreads;
      pairs8(s, x[i], (In*)nullptr);
      pairs8(s + kPieces / NB / 2 * kAppendThreads, x[i] + 4, (In*)nullptr);
      if (!holds || i >= rows) {  // lanes past the channels add nothing to the sum
#pragma unroll
        for (int k = 0; k < 8; ++k) x[i][k] = 0;
      }
    }
    uint64_t cs[4], sn[4];
    if (rotated) {
      const ulonglong2* c2 = reinterpret_cast<const ulonglong2*>(rope_sm + slot * p.rot + 8 * L);
      const ulonglong2* s2 = reinterpret_cast<const ulonglong2*>(rope_sm + slot * p.rot + (p.rot >> 1) + 8 * L);
      cs[0] = c2[0].x; cs[1] = c2[0].y; cs[2] = c2[1].x; cs[3] = c2[1].y;
      sn[0] = s2[0].x; sn[1] = s2[0].y; sn[2] = s2[1].x; sn[3] = s2[1].y;
    }
    __syncwarp();  // the warp has its angles before the slot is filled again
    if (p.q_norm) {
      float ss[NB];
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        uint64_t s2 = f2_mul(x[i][0], x[i][0]);
#pragma unroll
        for (int k = 1; k < 8; ++k) s2 = f2_fma(x[i][k], x[i][k], s2);
        float s1;
        f2_get(s2, ss[i], s1);
        ss[i] += s1;
      }
#pragma unroll
      for (int o = G / 2; o; o >>= 1)
#pragma unroll
        for (int i = 0; i < NB; ++i) ss[i] += __shfl_xor_sync(0xffffffffu, ss[i], o);
      bool wide = false;
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        ss[i] = fmaf(ss[i], p.inv_d, p.eps);
        wide |= !norm_range(ss[i]);
      }
      if (__any_sync(0xffffffffu, wide)) {
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const float2 r = wide_norm<G, In>(ring + (slot * kPieces + i * (kPieces / NB)) * kAppendThreads, holds && i < rows, ss[i],
                                            p.inv_d, p.eps);
          ss[i] = r.y;
#pragma unroll
          for (int k = 0; k < 8; ++k) x[i][k] = f2_mul(x[i][k], f2(r.x, r.x));
        }
      }
      uint64_t i2[NB];
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const float inv = rsqrtf(ss[i]);
        i2[i] = f2(inv, inv);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float4 v = *reinterpret_cast<const float4*>(w_sm + (k < 2 ? c0 + 4 * k : c1 + 4 * (k - 2)));
        const uint64_t w0 = f2(v.x, v.y), w1 = f2(v.z, v.w);
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          x[i][2 * k] = f2_mul(x[i][2 * k], f2_mul(i2[i], w0));
          x[i][2 * k + 1] = f2_mul(x[i][2 * k + 1], f2_mul(i2[i], w1));
        }
      }
    }
    if (rotated) {
      if (p.interleaved) {
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) {  // pairs 2k, 2k + 1: (x0 x1) (x2 x3) -> (x0 x2) (x1 x3)
            float a, b, c, d;
            f2_get(x[i][2 * k], a, b);
            f2_get(x[i][2 * k + 1], c, d);
            const uint64_t u = f2(a, c), v = f2(b, d);
            const uint64_t nv = f2(-b, -d);
            f2_get(f2_fma(nv, sn[k], f2_mul(u, cs[k])), a, c);
            f2_get(f2_fma(u, sn[k], f2_mul(v, cs[k])), b, d);
            x[i][2 * k] = f2(a, b);
            x[i][2 * k + 1] = f2(c, d);
          }
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float s0, s1;
          f2_get(sn[k], s0, s1);
          const uint64_t ns = f2(-s0, -s1);
#pragma unroll
          for (int i = 0; i < NB; ++i) {
            const uint64_t u = x[i][k], v = x[i][4 + k];
            x[i][k] = f2_fma(v, ns, f2_mul(u, cs[k]));
            x[i][4 + k] = f2_fma(u, sn[k], f2_mul(v, cs[k]));
          }
        }
      }
    }
    if (!pos_ok) {  // a position outside the table: zeros
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) x[i][k] = 0;
    }
    if (holds) {
#pragma unroll
      for (int i = 0; i < NB; ++i)
        if (i < rows) {
          store8(out + i * D + c0, x[i]);
          store8(out + i * D + c1, x[i] + 4);
        }
    }
    out += o_step;
  }
}

// The key head h < hk or value head h - hk of tokens t, t + step, ..., a lane
// a scale's 16 channels.
template <int G, typename In>
__device__ __forceinline__ void cache_heads(const AppendParams& p, int D, int t, int step, int h, int L, const float* w_sm,
                                            uint4* ring, float* rope_sm) {
  const bool key = h < p.hk, valid = h < 2 * p.hk, holds = valid && 16 * L < D;
  const In* src = key ? static_cast<const In*>(p.k) + t * p.k_tok + h * p.k_head
                      : static_cast<const In*>(p.v) + t * p.v_tok + (h - p.hk) * p.v_head;
  const int64_t src_step = step * (key ? p.k_tok : p.v_tok);
  const bool keys = __any_sync(0xffffffffu, key);
  const int64_t head = (key ? h : h - p.hk) * p.head_bytes + (key ? 0 : p.head_bytes / 2);
  constexpr int kPieces = 2 * (sizeof(In) / 2);
  uint4* mine = ring + threadIdx.x;
  auto issue = [&](int slot, int at, int pos) {
    if (at < p.T) {
      if (holds) {
        copy8(mine + slot * kPieces * kAppendThreads, src + 16 * L);
        copy8(mine + (slot * kPieces + kPieces / 2) * kAppendThreads, src + 16 * L + 8);
      }
      if (keys) copy_angles(rope_sm + slot * p.rot, p, pos);
    }
    copies_commit();
    src += src_step;
  };
  auto position = [&](int at) { return at < p.T ? p.positions[at] : -1; };
  int pq[kRing];  // positions of tokens t, t + step, ...
#pragma unroll
  for (int i = 0; i < kRing; ++i) pq[i] = position(t + i * step);
  int64_t slot_n = p.slots[t];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) issue(i, t + i * step, pq[i]);
  for (int at = 0; t < p.T; t += step, at = at + 1 == kRing ? 0 : at + 1) {
    const int after = position(t + kRing * step);
    issue(at == 0 ? kRing - 1 : at - 1, t + kAhead * step, pq[kAhead]);
    const int64_t my_slot = slot_n;
    if (t + step < p.T) slot_n = p.slots[t + step];
    copies_wait<kAhead>();
    __syncwarp();
    const int my_pos = pq[0];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) pq[i] = pq[i + 1];
    pq[kAhead] = after;
    float x[16], y[16], err[16];
    {
      uint64_t u[8];
      pairs8(mine + at * kPieces * kAppendThreads, u, (In*)nullptr);
      pairs8(mine + (at * kPieces + kPieces / 2) * kAppendThreads, u + 4, (In*)nullptr);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        f2_get(u[i], x[2 * i], x[2 * i + 1]);
        x[2 * i] = holds ? x[2 * i] : 0.f;
        x[2 * i + 1] = holds ? x[2 * i + 1] : 0.f;
      }
    }
    const float* rope = rope_sm + at * p.rot;
    const bool pos_ok = my_pos >= 0 && my_pos < p.max_pos;
    const bool slot_ok = my_slot >= 0 && my_slot < ((int64_t)p.n_pages << p.pshift);
    if (h == 0 && L == 0) {
      if (!pos_ok) atomicOr(p.status, kBadPosition);
      if (my_slot >= 0 && !slot_ok) atomicOr(p.status, kBadSlot);
    }
    if (!slot_ok || !pos_ok) {  // (all lanes)
      __syncwarp();
      continue;
    }
    float emax = -1.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = x[i], err[i] = -1.f;
    if (keys) {
      float mag[16];
      const bool norm = p.k_norm && holds;
      if (p.k_norm) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) ss = fmaf(y[i], y[i], ss);
#pragma unroll
        for (int o = G / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        float v = fmaf(ss, p.inv_d, p.eps);
        if (__any_sync(0xffffffffu, key && !norm_range(v))) {
          const float2 r = wide_norm<G, In>(ring + at * kPieces * kAppendThreads, holds, v, p.inv_d, p.eps);
          v = r.y;
#pragma unroll
          for (int i = 0; i < 16; ++i) y[i] *= r.x;
        }
        const float inv = rsqrtf(v);
        if (norm) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float4 w = *reinterpret_cast<const float4*>(w_sm + 16 * L + 4 * k);
            y[4 * k] *= inv * w.x;
            y[4 * k + 1] *= inv * w.y;
            y[4 * k + 2] *= inv * w.z;
            y[4 * k + 3] *= inv * w.w;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) mag[i] = norm ? fabsf(y[i]) : 0.f;
      if (p.interleaved) {
        if (16 * L < p.rot) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float c = rope[8 * L + i], s = rope[(p.rot >> 1) + 8 * L + i];
            const float a = y[2 * i], b = y[2 * i + 1];
            y[2 * i] = a * c - b * s;
            y[2 * i + 1] = b * c + a * s;
            mag[2 * i] = fabsf(a * c) + fabsf(b * s);
            mag[2 * i + 1] = fabsf(b * c) + fabsf(a * s);
          }
        }
      } else if (p.rot) {
        const Partner pa = partner_of(L, p.rot);
        float o[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = __shfl_sync(0xffffffffu, pa.odd ? y[i ^ 8] : y[i], pa.src[i >> 3]);
#pragma unroll
        for (int b = 0; b < 2; ++b)
          if (pa.rotated[b]) {
            const float4* cr = reinterpret_cast<const float4*>(rope + angle_of(L, 8 * b, p.rot, false));
            const float4* sr = reinterpret_cast<const float4*>(rope + (p.rot >> 1) + angle_of(L, 8 * b, p.rot, false));
            const float4 c4[2] = {cr[0], cr[1]}, s4[2] = {sr[0], sr[1]};
            const float c[8] = {c4[0].x, c4[0].y, c4[0].z, c4[0].w, c4[1].x, c4[1].y, c4[1].z, c4[1].w};
            const float s[8] = {s4[0].x, s4[0].y, s4[0].z, s4[0].w, s4[1].x, s4[1].y, s4[1].z, s4[1].w};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float u = y[8 * b + i] * c[i], v = o[8 * b + i] * s[i];
              y[8 * b + i] = pa.first[b] ? u - v : u + v;
              mag[8 * b + i] = fabsf(u) + fabsf(v);
            }
          }
      }
      // exact: values, zeros, and without a norm what position 0 turns by nothing
      const bool inexact = key && (norm || my_pos != 0);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        y[i] = key ? y[i] : x[i];
        err[i] = inexact && mag[i] > 0.f ? mag[i] * 0x1p-19f : -1.f;
        emax = fmaxf(emax, err[i]);
      }
    }
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      y[i] = y[i] == y[i] ? y[i] : 0.f;
      amax = fmaxf(amax, fabsf(y[i]));
    }
    int sb = scale_byte<float>(amax);
    const float d = scale_value(sb);
    bool border = fabsf(amax - 3.5f * (d + scale_value(sb + 1))) <= emax;
    border |= fabsf(amax - 3.5f * (d + scale_value(max(sb - 1, 0)))) <= emax;
    border &= emax > 0.f && key && holds;  // (a row of zeros is exact)
    const float rd = 1.f / fmaxf(d, 0x1p-17f);
    uint32_t c[16], unsure = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) c[i] = code_bits(y[i], d, rd, err[i], 1u << i, unsure);
    uint2 words = d > 0.f ? make_uint2(pack_codes(c), pack_codes(c + 8)) : make_uint2(0x88888888u, 0x88888888u);
    if (!(d > 0.f) || border) unsure = 0;
    if (keys && __any_sync(0xffffffffu, border || unsure)) {
      const float* hi = p.rope + (int64_t)my_pos * p.rot;
      const float* lo = p.rope_lo + (int64_t)my_pos * p.rot;
      const float* w = p.k_norm ? w_sm : nullptr;
      settle_rows<G, In>(ring + at * kPieces * kAppendThreads, holds, y, w, (double)p.eps, D, L, p.rot, p.interleaved != 0, hi, lo, border, amax, emax, unsure, sb, words);
    }
    __syncwarp();  // the warp has its angles before the slot is filled again
    if (holds) {
      const int64_t pg = my_slot >> p.pshift;
      const int at = (int)(my_slot & (p.P - 1));
      uint8_t* base = p.pages + pg * p.page_bytes + head;
      *reinterpret_cast<uint2*>(base + at * (D / 2) + 8 * L) = words;
      base[p.P * (D / 2) + at * (D / 16) + L] = (uint8_t)sb;
    }
  }
}

template <int NB, typename In>
__host__ __device__ constexpr int append_pieces() {
  return NB * 2 * (int)(sizeof(In) / 2);
}

// G lanes a row: 4 (D = 64), 8 (128) or 16 (192: 12 of them hold channels;
// 256).  A block takes one part of the heads (NB query heads a group, or a key
// or value head a group) of every step-th token: its next rows
// and angles are on their way while it works on a token (a block a token and part
// instead spent 3 us on each, waiting for its position, then its angles).
template <int G, int NB, typename In, typename Out>
__global__ void __launch_bounds__(kAppendThreads, kAppendBlocks) append_kernel(const __grid_constant__ AppendParams p, int D, int q_parts, int q_tokens,
                                                                int kv_parts, int kv_tokens) {
  extern __shared__ __align__(16) uint4 ring[];  // [slot][piece][thread], then the warps' angles [warp][slot][rot]
  __shared__ __align__(16) float w_sm[256];
  griddep_launch_dependents();
  constexpr int kRows = kAppendThreads / G;  // groups of the block
  const int L = threadIdx.x & (G - 1), group = threadIdx.x / G;
  // blocks of keys and values come first: theirs is the longer work
  const int b = (int)blockIdx.x - kv_parts * kv_tokens;
  const bool queries = b >= 0;
  const int part = queries ? b % q_parts : (int)blockIdx.x % kv_parts;
  const int t = queries ? b / q_parts : (int)blockIdx.x / kv_parts, step = queries ? q_tokens : kv_tokens;
  if (queries ? p.q_norm : p.k_norm)
    for (int i = threadIdx.x; i < D; i += kAppendThreads) w_sm[i] = p.norm_w[(queries ? 0 : D) + i];
  __syncthreads();
  griddep_wait();  // the projections and positions may come from the previous kernel
  float* rope_sm = reinterpret_cast<float*>(ring + kRing * append_pieces<NB, In>() * kAppendThreads) +
                   (threadIdx.x >> 5) * kRing * p.rot;
  if (queries) query_heads<G, NB, In, Out>(p, D, t, step, (part * kRows + group) * NB, L, w_sm, ring, rope_sm);
  else cache_heads<G, In>(p, D, t, step, part * kRows + group, L, w_sm, ring, rope_sm);
}

// Rows of the cache as bf16 values: one thread a word of 8 channels.
__global__ void __launch_bounds__(256) read_kernel(const uint8_t* __restrict__ pages, const int64_t* __restrict__ slots,
                                                   int64_t n_words, int hk, int D, int P, int pshift, int n_pages,
                                                   int64_t head_bytes, int64_t page_bytes, __nv_bfloat16* k_out,
                                                   __nv_bfloat16* v_out, int* status) {
  griddep_launch_dependents();
  griddep_wait();
  const int wd = D / 8;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n_words; i += (int64_t)gridDim.x * blockDim.x) {
    const int w = (int)(i % wd);
    const int64_t r = i / wd;  // (row, head, key or value)
    const int which = (int)(r & 1), h = (int)((r >> 1) % hk);
    const int64_t row = (r >> 1) / hk;
    __nv_bfloat16* out = which ? v_out : k_out;
    if (!out) continue;
    const int64_t slot = slots[row];
    uint4 o = make_uint4(0, 0, 0, 0);
    if (slot >= 0 && slot < ((int64_t)n_pages << pshift)) {
      const int64_t pg = slot >> pshift, at = slot & (P - 1);
      const uint8_t* base = pages + pg * page_bytes + h * head_bytes + (which ? head_bytes / 2 : 0);
      const uint32_t word = *reinterpret_cast<const uint32_t*>(base + at * (D / 2) + 4 * w);
      const float d = scale_value(base[P * (D / 2) + at * (D / 16) + (w >> 1)]);
      uint32_t u[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float a = ((int)((word >> (4 * e)) & 15) - 8) * d, b = ((int)((word >> (4 * e + 16)) & 15) - 8) * d;
        const __nv_bfloat162 v2 = __floats2bfloat162_rn(a, b);
        u[e] = *reinterpret_cast<const uint32_t*>(&v2);
      }
      o = make_uint4(u[0], u[1], u[2], u[3]);
    } else if (slot >= 0) {
      atomicOr(status, kBadSlot);
    }
    *reinterpret_cast<uint4*>(out + (row * hk + h) * D + 8 * w) = o;
  }
}

// cos and sin of position times frequency, in fp64: rounded to fp32, and the
// rest (for the rows that are decided in fp64).
__global__ void rope_kernel(const double* __restrict__ freq, int half, int n, float* __restrict__ hi, float* __restrict__ lo) {
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < (int64_t)n * half;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t at = i / half * 2 * half + i % half;
    double s, c;
    sincos((double)(i / half) * freq[i % half], &s, &c);
    hi[at] = (float)c;
    lo[at] = (float)(c - (double)(float)c);
    hi[at + half] = (float)s;
    lo[at + half] = (float)(s - (double)(float)s);
  }
}

template <int NB, typename In>
size_t append_smem(int rot) {
  return (size_t)kRing * append_pieces<NB, In>() * kAppendThreads * 16 + (size_t)(kAppendThreads / 32) * kRing * rot * sizeof(float);
}
template <int G, typename In, typename Out>
cudaError_t append_rows(const AppendParams* p, int D, int num_sms, cudaStream_t st) {
  if (!p) {  // configure
    cudaError_t e = cudaFuncSetAttribute(append_kernel<G, 2, In, Out>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)append_smem<2, In>(256));
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(append_kernel<G, 1, In, Out>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)append_smem<1, In>(256));
  }
  constexpr int kRows = kAppendThreads / G;
  const int kv_parts = (2 * p->hk + kRows - 1) / kRows;
  const int q_two = (p->hq + 2 * kRows - 1) / (2 * kRows), q_one = (p->hq + kRows - 1) / kRows;
  // two query rows a group once their blocks still fill those places
  // twice the resident blocks: uneven tokens are levelled out by the second
  // half (36.9, 32.9 and 33.4 us with one, two and four times as many for 4096
  // tokens of 32 / 8 heads of 128)
  const int64_t places = 2LL * kAppendBlocks * num_sms;
  const bool two = (int64_t)p->T * (q_two + kv_parts) >= places;
  const int q_parts = two ? q_two : q_one;
  // tokens worked on at once: a token of keys and values takes a block about
  // twice the time of two query rows a group (3.5 against 1.6 us, both bound by
  // their instructions' latency), so they get twice the blocks
  const int64_t q_tokens = std::min<int64_t>(p->T, std::max<int64_t>(1, places / (q_parts + 2 * kv_parts)));
  const int64_t kv_tokens = std::min<int64_t>(p->T, std::max<int64_t>(1, (places - q_parts * q_tokens) / kv_parts));
  const dim3 grid((unsigned)(q_tokens * q_parts + kv_tokens * kv_parts));
  if (two)
    return launch_pdl(append_kernel<G, 2, In, Out>, grid, kAppendThreads, append_smem<2, In>(p->rot), st, *p, D, q_parts,
                      (int)q_tokens, kv_parts, (int)kv_tokens);
  return launch_pdl(append_kernel<G, 1, In, Out>, grid, kAppendThreads, append_smem<1, In>(p->rot), st, *p, D, q_parts,
                    (int)q_tokens, kv_parts, (int)kv_tokens);
}
template <int G>
cudaError_t append_types(const AppendParams* p, int D, bool in_f32, bool out_f32, int num_sms, cudaStream_t st) {
  if (in_f32)
    return out_f32 ? append_rows<G, float, float>(p, D, num_sms, st) : append_rows<G, float, __nv_bfloat16>(p, D, num_sms, st);
  return out_f32 ? append_rows<G, __nv_bfloat16, float>(p, D, num_sms, st)
                 : append_rows<G, __nv_bfloat16, __nv_bfloat16>(p, D, num_sms, st);
}
cudaError_t append_any(const AppendParams* p, int D, bool in_f32, bool out_f32, int num_sms, cudaStream_t st) {
  if (D == 64) return append_types<4>(p, D, in_f32, out_f32, num_sms, st);
  if (D == 128) return append_types<8>(p, D, in_f32, out_f32, num_sms, st);
  return append_types<16>(p, D, in_f32, out_f32, num_sms, st);
}

}  // namespace

cudaError_t append_launch(const moe_attn* h, const void* q, const void* k, const void* v, bool in_f32,
                          const int64_t* strides, const int32_t* positions, const int64_t* slots, int T, void* pages,
                          void* q_out, cudaStream_t st) {
  AppendParams p{};
  p.q = q; p.k = k; p.v = v;
  p.q_tok = strides[0]; p.q_head = strides[1];
  p.k_tok = strides[2]; p.k_head = strides[3];
  p.v_tok = strides[4]; p.v_head = strides[5];
  p.positions = positions; p.slots = slots;
  p.pages = static_cast<uint8_t*>(pages);
  p.q_out = q_out;
  p.T = T; p.hq = h->hq; p.hk = h->hk; p.P = h->P; p.n_pages = h->n_pages;
  p.pshift = 31 - __builtin_clz((unsigned)h->P);
  p.rot = h->rot; p.interleaved = h->interleaved; p.max_pos = h->len_max;
  p.q_norm = h->q_norm; p.k_norm = h->k_norm; p.eps = h->eps;
  p.inv_d = 1.f / (float)h->D;
  p.rope = h->rope; p.rope_lo = h->rope + (int64_t)h->len_max * h->rot; p.norm_w = h->norm_w;
  p.head_bytes = h->head_bytes; p.page_bytes = h->page_bytes;
  p.status = h->status;
  return append_any(&p, h->D, in_f32, h->act == MOE_ACT_F32, h->num_sms, st);
}

// Lets the kernels of a handle use their shared memory.
cudaError_t append_configure(const moe_attn* h) {
  const cudaError_t e = append_any(nullptr, h->D, false, h->act == MOE_ACT_F32, 0, nullptr);
  return e != cudaSuccess ? e : append_any(nullptr, h->D, true, h->act == MOE_ACT_F32, 0, nullptr);
}

cudaError_t read_launch(const moe_attn* h, const void* pages, const int64_t* slots, int n, void* k_out, void* v_out,
                        cudaStream_t st) {
  const int64_t words = (int64_t)n * h->hk * 2 * (h->D / 8);
  const int64_t blocks = std::min<int64_t>((words + 255) / 256, 16LL * h->num_sms);
  return launch_pdl(read_kernel, dim3((unsigned)blocks), 256, 0, st, static_cast<const uint8_t*>(pages), slots, words,
                    h->hk, h->D, h->P, 31 - __builtin_clz((unsigned)h->P), h->n_pages, h->head_bytes, h->page_bytes,
                    static_cast<__nv_bfloat16*>(k_out), static_cast<__nv_bfloat16*>(v_out), h->status);
}

cudaError_t rope_launch(const moe_attn* h, cudaStream_t st) {
  if (!h->rot) return cudaSuccess;
  rope_kernel<<<(unsigned)std::min<int64_t>(((int64_t)h->len_max * h->rot / 2 + 255) / 256, 4096), 256, 0, st>>>(
      h->freq, h->rot / 2, h->len_max, h->rope, h->rope + (int64_t)h->len_max * h->rot);
  return cudaGetLastError();
}

}  // namespace attn
}  // namespace moe

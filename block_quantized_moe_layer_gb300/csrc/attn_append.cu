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
// Work: one row (token, head) is D/8 lanes of 8 channels, one 16-byte load a
// lane (two for fp32); the sum of squares and the partner channels of a
// rotation travel by shuffles, so a row is read once and written once.  The
// bound is HBM: D (2 + 2) bytes of a query row, D (2 + 9/16) of a key or value
// row.  The angles' cosines and sines come from the handle's table (fp32,
// computed in fp64: far positions lose nothing), kept in registers while a
// warp walks over heads of one token.
//
// Codes are those of the exact result.  fp32 leaves each y' within
// 2^-19 (|y_a cos| + |y_b sin|) of it (a sum of squares in at most 13
// additions, one division and square root, four products and a sum, each
// within 2^-24); a row in which that error could change a scale or a code
// (about one in 500) is computed again in fp64.  Values are exact already:
// their codes are decided by exact fp32 residuals.
#include "attn.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kAppendThreads = 256;

struct AppendParams {
  const void *q, *k, *v;
  int64_t q_tok, q_head, k_tok, k_head, v_tok, v_head;  // elements
  const int32_t* positions;
  const int64_t* slots;
  uint8_t* pages;
  void* q_out;  // [T][hq][D]
  int T, hq, hk, P, pshift, n_pages, rot, interleaved, max_pos, passes;
  bool q_norm, k_norm;
  float eps;
  const float* rope;
  const double* freq;
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
    const T mid = (T)(3.5f * (scale_value(b) + scale_value(b + 1)));
    b += (amax > mid || (amax == mid && (b & 1))) ? 1 : 0;
  }
  return min(b, kKvMaxScale);
}

// The code of x for scale d: round half even of the exact x / d, clamped.  The
// quotient rounds; the residual x - q d does not (both are multiples of the
// smaller unit and |x - q d| <= |x|), so comparing it with d/2 settles q.
__device__ __forceinline__ int code_of(float x, float d) {
  if (!(d > 0.f) || x != x) return 8;
  float q = rintf(fminf(fmaxf(x / d, -9.f), 8.f));
  const float r = fmaf(-q, d, x);
  if (r > d * 0.5f) q += 1.f;
  else if (r < d * -0.5f) q -= 1.f;
  return (int)fminf(fmaxf(q, -8.f), 7.f) + 8;
}
__device__ __forceinline__ int code_of(double x, double d) {
  if (!(d > 0.0) || x != x) return 8;
  return (int)rint(fmin(fmax(x / d, -8.0), 7.0)) + 8;
}

// Nibble of channel e of eight.
__device__ __forceinline__ uint32_t nibble(int c, int e) { return (uint32_t)c << (4 * ((e >> 1) + 4 * (e & 1))); }

template <typename In>
__device__ __forceinline__ void load8(const In* p, float (&x)[8]) {
  if constexpr (sizeof(In) == 2) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
}

template <typename Out>
__device__ __forceinline__ void store8(Out* p, const float (&x)[8]) {
  if constexpr (sizeof(Out) == 2) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
}

// A key row in fp64 (the whole warp calls it): this lane's word of codes and
// its block's scale byte.
template <int G>
__device__ __noinline__ uint32_t key_codes_f64(const float (&x)[8], const float* w, bool norm, double eps, int D, int L,
                                               int rot, bool interleaved, const double* freq, int pos, int& sbyte) {
  double y[8];
  double ss = 0.0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    y[i] = x[i];
    ss = fma(y[i], y[i], ss);
  }
#pragma unroll
  for (int o = G / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if (norm) {
    const double inv = 1.0 / sqrt(ss / D + eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = y[i] * inv * (double)w[i];
  }
  const int half = rot >> 4;  // lanes of half the rotated channels
  if (interleaved) {
    if (8 * L < rot) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        double s, c;
        sincos(pos * freq[4 * L + i], &s, &c);
        const double a = y[2 * i], b = y[2 * i + 1];
        y[2 * i] = a * c - b * s;
        y[2 * i + 1] = b * c + a * s;
      }
    }
  } else {
    const int lane = threadIdx.x & 31;
    const bool first = L < half;
    const int src = (8 * L < rot) ? lane + (first ? half : -half) : lane;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const double o = __shfl_sync(0xffffffffu, y[i], src);
      if (8 * L < rot) {
        double s, c;
        sincos(pos * freq[8 * (first ? L : L - half) + i], &s, &c);
        y[i] = first ? y[i] * c - o * s : y[i] * c + o * s;
      }
    }
  }
  double amax = 0.0;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmax(amax, fabs(y[i]));
  amax = fmax(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  sbyte = scale_byte<double>(amax);
  const double d = (double)scale_value(sbyte);
  uint32_t word = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) word |= nibble(code_of(y[i], d), i);
  return word;
}

// G lanes a row: 8 (D = 64), 16 (128) or 32 (192: 24 of them hold channels; 256).
template <int G, typename In, typename Out>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const __grid_constant__ AppendParams p, int D) {
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int L = lane & (G - 1);  // lane of the row
  const int t = blockIdx.x;
  constexpr int kRows = kAppendThreads / G;  // rows of a pass
  const bool holds = 8 * L < D;
  const int half = p.rot >> 4;
  const bool rotated = 8 * L < p.rot;
  const bool first = L < half;
  griddep_wait();  // the projections and positions may come from the previous kernel
  const int pos = p.positions[t];
  const int64_t slot = p.slots[t];
  const bool pos_ok = pos >= 0 && pos < p.max_pos;
  const bool slot_ok = slot >= 0 && slot < ((int64_t)p.n_pages << p.pshift);
  if (threadIdx.x == 0 && blockIdx.y == 0) {
    if (!pos_ok) atomicOr(p.status, kBadPosition);
    if (slot >= 0 && !slot_ok) atomicOr(p.status, kBadSlot);
  }
  float cs[8], sn[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) cs[i] = 1.f, sn[i] = 0.f;
  if (rotated && pos_ok) {
    const float* r = p.rope + (int64_t)pos * p.rot;
    if (p.interleaved) {  // four angles
      const float4 c4 = *reinterpret_cast<const float4*>(r + 4 * L);
      const float4 s4 = *reinterpret_cast<const float4*>(r + (p.rot >> 1) + 4 * L);
      cs[0] = c4.x; cs[1] = c4.y; cs[2] = c4.z; cs[3] = c4.w;
      sn[0] = s4.x; sn[1] = s4.y; sn[2] = s4.z; sn[3] = s4.w;
    } else {
      const int f = 8 * (first ? L : L - half);
      load8<float>(r + f, cs);
      load8<float>(r + (p.rot >> 1) + f, sn);
    }
  }
  const int heads = p.hq + 2 * p.hk;
  for (int pass = 0; pass < p.passes; ++pass) {
    const int h = (blockIdx.y * p.passes + pass) * kRows + threadIdx.x / G;
    if (((blockIdx.y * p.passes + pass) * kRows + (threadIdx.x & ~31) / G) >= heads) break;  // the whole warp is past the heads
    const bool valid = h < heads;
    const int kind = h < p.hq ? 0 : (h < p.hq + p.hk ? 1 : 2);
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (valid && holds) {
      const In* src;
      if (kind == 0) src = static_cast<const In*>(p.q) + t * p.q_tok + h * p.q_head;
      else if (kind == 1) src = static_cast<const In*>(p.k) + t * p.k_tok + (h - p.hq) * p.k_head;
      else src = static_cast<const In*>(p.v) + t * p.v_tok + (h - p.hq - p.hk) * p.v_head;
      load8<In>(src + 8 * L, x);
    }
    const bool norm = kind == 0 ? p.q_norm : (kind == 1 ? p.k_norm : false);
    float w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 1.f;
    if (norm && holds) load8<float>(p.norm_w + (kind == 1 ? D : 0) + 8 * L, w);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int o = G / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    float y[8];
    const float inv = norm ? 1.f / sqrtf(ss / (float)D + p.eps) : 1.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = norm ? x[i] * inv * w[i] : x[i];
    // rotation (values stay): err bounds what fp32 lost of each channel
    float z[8], mag[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = y[i], mag[i] = norm ? fabsf(y[i]) : 0.f;
    if (p.interleaved) {
      if (rotated && kind != 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = y[2 * i], b = y[2 * i + 1];
          z[2 * i] = a * cs[i] - b * sn[i];
          z[2 * i + 1] = b * cs[i] + a * sn[i];
          mag[2 * i] = fabsf(a * cs[i]) + fabsf(b * sn[i]);
          mag[2 * i + 1] = fabsf(b * cs[i]) + fabsf(a * sn[i]);
        }
      }
    } else {
      const int src = rotated ? lane + (first ? half : -half) : lane;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float o = __shfl_sync(0xffffffffu, y[i], src);
        if (rotated && kind != 2) {
          z[i] = first ? y[i] * cs[i] - o * sn[i] : y[i] * cs[i] + o * sn[i];
          mag[i] = fabsf(y[i] * cs[i]) + fabsf(o * sn[i]);
        }
      }
    }
    if (kind == 0) {
      if (valid && holds) {
        if (!pos_ok) {
#pragma unroll
          for (int i = 0; i < 8; ++i) z[i] = 0.f;
        }
        store8<Out>(static_cast<Out*>(p.q_out) + ((int64_t)t * p.hq + h) * D + 8 * L, z);
      }
    }
    const bool stores = valid && kind != 0 && slot_ok && pos_ok;
    if (!__any_sync(0xffffffffu, stores)) continue;
    float amax = 0.f, emax = 0.f;
    // position 0 turns nothing, and a row without a norm is exact there
    const bool inexact = norm || pos != 0;
    float err[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      err[i] = inexact ? mag[i] * 0x1p-19f : 0.f;
      amax = fmaxf(amax, fabsf(z[i]));
      emax = fmaxf(emax, err[i]);
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    emax = fmaxf(emax, __shfl_xor_sync(0xffffffffu, emax, 1));
    int sb = scale_byte<float>(amax);
    bool unsure = false;
    if (emax > 0.f) unsure = scale_byte<float>(amax - emax) != sb || scale_byte<float>(amax + emax) != sb;
    const float d = scale_value(sb);
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = code_of(z[i], d);
      if (err[i] > 0.f) unsure |= code_of(z[i] - err[i], d) != c || code_of(z[i] + err[i], d) != c;
      word |= nibble(c, i);
    }
    unsure = unsure && kind == 1 && stores;
    if (__any_sync(0xffffffffu, unsure)) {
      int sb2;
      const uint32_t word2 = key_codes_f64<G>(x, w, norm, (double)p.eps, D, L, p.rot, p.interleaved != 0, p.freq, pos, sb2);
      if (kind == 1) word = word2, sb = sb2;
    }
    if (stores && holds) {
      const int pg = (int)(slot >> p.pshift), at = (int)(slot & (p.P - 1));
      const int hh = kind == 1 ? h - p.hq : h - p.hq - p.hk;
      uint8_t* base = p.pages + pg * p.page_bytes + hh * p.head_bytes + (kind == 2 ? p.head_bytes / 2 : 0);
      *reinterpret_cast<uint32_t*>(base + at * (D / 2) + 4 * L) = word;
      if (!(L & 1)) base[p.P * (D / 2) + at * (D / 16) + (L >> 1)] = (uint8_t)sb;
    }
  }
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

// cos and sin of position times frequency, in fp64, rounded once to fp32.
__global__ void rope_kernel(const double* __restrict__ freq, int half, int n, float* __restrict__ rope) {
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < (int64_t)n * half;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t pos = i / half;
    const int f = (int)(i % half);
    double s, c;
    sincos((double)pos * freq[f], &s, &c);
    rope[pos * 2 * half + f] = (float)c;
    rope[pos * 2 * half + half + f] = (float)s;
  }
}

template <int G, typename In>
cudaError_t append_out(const AppendParams& p, int D, bool out_f32, dim3 grid, cudaStream_t st) {
  if (out_f32) return launch_pdl(append_kernel<G, In, float>, grid, kAppendThreads, 0, st, p, D);
  return launch_pdl(append_kernel<G, In, __nv_bfloat16>, grid, kAppendThreads, 0, st, p, D);
}
template <int G>
cudaError_t append_in(const AppendParams& p, int D, bool in_f32, bool out_f32, dim3 grid, cudaStream_t st) {
  return in_f32 ? append_out<G, float>(p, D, out_f32, grid, st) : append_out<G, __nv_bfloat16>(p, D, out_f32, grid, st);
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
  p.rope = h->rope; p.freq = h->freq; p.norm_w = h->norm_w;
  p.head_bytes = h->head_bytes; p.page_bytes = h->page_bytes;
  p.status = h->status;
  const int G = h->D == 64 ? 8 : (h->D == 128 ? 16 : 32);
  const int rows = kAppendThreads / G, heads = h->hq + 2 * h->hk;
  const int all = (heads + rows - 1) / rows;
  // passes of a block over a token's heads: one while the blocks do not fill
  // the GPU, more where that keeps the angles in registers
  p.passes = 1;
  while (p.passes < all && (int64_t)T * ((all + 2 * p.passes - 1) / (2 * p.passes)) >= 16LL * h->num_sms) p.passes *= 2;
  const dim3 grid(T, (all + p.passes - 1) / p.passes);
  const bool out_f32 = h->act == MOE_ACT_F32;
  if (G == 8) return append_in<8>(p, h->D, in_f32, out_f32, grid, st);
  if (G == 16) return append_in<16>(p, h->D, in_f32, out_f32, grid, st);
  return append_in<32>(p, h->D, in_f32, out_f32, grid, st);
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
      h->freq, h->rot / 2, h->len_max, h->rope);
  return cudaGetLastError();
}

}  // namespace attn
}  // namespace moe

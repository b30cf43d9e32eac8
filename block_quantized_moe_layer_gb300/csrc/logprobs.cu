// logprobs.cu -- log probabilities of given tokens, the entropy of each row
// and its n_top most probable tokens, in one pass over the logits.
//
// For a row x of V logits: with M = max x, z = x - M, S = sum e^z, U = sum z e^z,
//   log p_v = z_v - ln S,   H = -sum p ln p = ln S - U / S.
// A thread keeps its own running maximum m, s and u: when the maximum grows by
// -delta, s <- f s and u <- f (u + delta s) with f = e^delta; the parts are
// joined by the same formula.  All of it is fp32; e^z is 2^(z log2 e) of the
// exact difference z.
//
// The alternatives cost nothing in that pass: each thread's maximum is known
// at its end, and the n_top-th largest of a block's thread maxima bounds the
// row's n_top-th best from below.  So only the threads whose maximum reaches
// that bound (n_top of them when no two are equal) can hold one of the best;
// their elements are read again (from L2) by whole warps, and those that
// reach the bound are inserted into a sorted list kept across the lanes.
// Ties go to the lower token id: the lists order 64-bit keys (value, ~id).
//   Where many logits are equal (a mask leaves a few, or few values occur) all
// of them reach the bound.  They are looked at in the order of their ids, and
// once the list is full only a lower id than its last one's gets in, so a warp
// inserts a few dozen: 64 rows of 151936 fp32, top 20, take 22 us, with 3
// logits left of each 42, all equal 17 (offered one by one: 940).
//
// Rows are read with 16-byte loads, four in flight a thread, and bound by HBM;
// where there are few rows a cluster of up to 8 blocks shares one and joins
// its parts through distributed shared memory (no workspace, one launch).
// Measured: 1023 rows of 32768 fp32 in 28.4 us, 4.7 TB/s of 6.8 (a row is a
// block of 256 threads, so its join and its best tokens are not covered by its
// own loads, only by the other blocks'); 33 rows of 151936 bf16, top 20, in
// 12.8 us; 4 rows of 32768 in 7.4 us.
#include <cooperative_groups.h>

#include "common.cuh"
#include "layer.cuh"

namespace moe {
namespace {

constexpr int kLpThreads = 256;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kLpMaxTop = 32;
constexpr int kLpMaxCluster = 8;
constexpr int kLpBatch = 4;  // 16-byte loads in flight
constexpr float kLog2e = 1.44269504088896341f;

struct LpParams {
  const void* logits;
  int64_t stride;  // elements
  int n, V, n_top, C;
  const int32_t* tokens;
  float *logprob, *entropy;
  int32_t* top_ids;
  float* top_logprobs;
};

__device__ __forceinline__ float max_nan(float a, float b) {  // a NaN stays
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Running maximum, sum of e^(x - m) and of (x - m) e^(x - m).
struct Soft {
  float m, s, u;
};
__device__ __forceinline__ void raise(Soft& a, float m) {
  if (m > a.m) {
    if (a.m == -INFINITY) {
      a.s = a.s == a.s ? 0.f : a.s;  // nothing yet (a NaN stays)
      a.u = a.u == a.u ? 0.f : a.u;
    } else {
      const float d = a.m - m, f = exp2f(d * kLog2e);
      a.u = f == 0.f ? a.u * f : f * fmaf(d, a.s, a.u);  // f = 0: d may be infinite
      a.s *= f;
    }
    a.m = m;
  }
}
// One more logit, not above a.m (or NaN).  Where all are -inf so far z is -inf.
__device__ __forceinline__ void add(Soft& a, float ref, float x) {
  const float z = max_nan(x - ref, -1000.f);  // e^-1000 is 0; 0 * z stays 0
  const float e = exp2f(z * kLog2e);
  a.s += e;
  a.u = fmaf(z, e, a.u);
}
__device__ __forceinline__ Soft join(Soft a, Soft b) {
  const float m = fmaxf(a.m, b.m);
  raise(a, m);
  raise(b, m);
  return Soft{m, a.s + b.s, a.u + b.u};
}

__device__ __forceinline__ uint64_t top_key(float x, int id) {
  const uint32_t b = __float_as_uint(x + 0.f);  // -0 and 0 are equal
  const uint32_t o = b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
  return ((uint64_t)o << 32) | (uint32_t)~id;
}
__device__ __forceinline__ float key_value(uint64_t k) {
  const uint32_t o = (uint32_t)(k >> 32);
  return __uint_as_float((o >> 31) ? o ^ 0x80000000u : ~o);
}

// Descending bitonic merge of a warp's 32 bitonic values.
template <typename T>
__device__ __forceinline__ T merge_down(T v, int lane, int from) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    if (o > from) continue;
    const T w = __shfl_xor_sync(0xffffffffu, v, o);
    v = ((lane & o) == 0) == (w > v) ? w : v;
  }
  return v;
}
__device__ __forceinline__ float sort_down(float v, int lane) {
#pragma unroll
  for (int k = 2; k <= 32; k <<= 1) {
#pragma unroll
    for (int o = k >> 1; o; o >>= 1) {
      const float w = __shfl_xor_sync(0xffffffffu, v, o);
      const bool keep_max = ((lane & o) == 0) == ((lane & k) == 0 || k == 32);
      v = keep_max ? fmaxf(v, w) : fminf(v, w);
    }
  }
  return v;
}
// The 32 largest of two descending lists, descending.
template <typename T>
__device__ __forceinline__ T merge_lists(T a, T b_reversed, int lane) {
  return merge_down(b_reversed > a ? b_reversed : a, lane, 16);
}

template <typename In>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int kN = 4;
  __device__ static void load(const float* p, float (&x)[4]) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(p));
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
  }
  __device__ static float one(const float* p) { return *p; }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int kN = 8;
  __device__ static void load(const __nv_bfloat16* p, float (&x)[8]) {
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

template <typename In>
__global__ void __launch_bounds__(kLpThreads) logprob_kernel(const __grid_constant__ LpParams p) {
  namespace cg = cooperative_groups;
  constexpr int N = Vec<In>::kN;
  __shared__ Soft soft[kLpWarps];
  __shared__ Soft mine;                       // this block's part, read by the cluster's first block
  __shared__ float tmax[kLpWarps][32];
  __shared__ uint64_t lists[kLpWarps][32];
  __shared__ float bound;
  __shared__ uint8_t reachers[kLpWarps][32];  // the warp's threads that reach the bound
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int row = blockIdx.x / p.C, rank = blockIdx.x % p.C;
  const In* x = static_cast<const In*>(p.logits) + (int64_t)row * p.stride;
  // elements before the first 16-byte boundary, whole vectors, the rest
  const int head = min(p.V, (int)(((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / sizeof(In)));
  const int nv = (p.V - head) / N;
  const int tail0 = head + nv * N;
  const int per = (nv + p.C - 1) / p.C;
  const int v0 = min(nv, rank * per), v1 = min(nv, v0 + per);
  const In* xv = x + head;
  const bool has_head = rank == 0 && tid < head;
  const bool has_tail = rank == p.C - 1 && tid < p.V - tail0;

  Soft a{-INFINITY, 0.f, 0.f};
  if (has_head) {
    const float v = Vec<In>::one(x + tid);
    raise(a, v);
    add(a, a.m == -INFINITY ? 0.f : a.m, v);
  }
  if (has_tail) {
    const float v = Vec<In>::one(x + tail0 + tid);
    raise(a, v);
    add(a, a.m == -INFINITY ? 0.f : a.m, v);
  }
  int i = v0 + tid;
  for (; i + (kLpBatch - 1) * kLpThreads < v1; i += kLpBatch * kLpThreads) {
    float v[kLpBatch][N];
#pragma unroll
    for (int b = 0; b < kLpBatch; ++b) Vec<In>::load(xv + (int64_t)(i + b * kLpThreads) * N, v[b]);
    float mx = v[0][0];
#pragma unroll
    for (int b = 0; b < kLpBatch; ++b)
#pragma unroll
      for (int e = 0; e < N; ++e) mx = fmaxf(mx, v[b][e]);
    raise(a, mx);
    const float ref = a.m == -INFINITY ? 0.f : a.m;
#pragma unroll
    for (int b = 0; b < kLpBatch; ++b)
#pragma unroll
      for (int e = 0; e < N; ++e) add(a, ref, v[b][e]);
  }
  for (; i < v1; i += kLpThreads) {
    float v[N];
    Vec<In>::load(xv + (int64_t)i * N, v);
    float mx = v[0];
#pragma unroll
    for (int e = 1; e < N; ++e) mx = fmaxf(mx, v[e]);
    raise(a, mx);
    const float ref = a.m == -INFINITY ? 0.f : a.m;
#pragma unroll
    for (int e = 0; e < N; ++e) add(a, ref, v[e]);
  }
  const float my_max = a.m;

  // this block's part
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    Soft b{__shfl_xor_sync(0xffffffffu, a.m, o), __shfl_xor_sync(0xffffffffu, a.s, o),
           __shfl_xor_sync(0xffffffffu, a.u, o)};
    a = join(a, b);
  }
  if (lane == 0) soft[warp] = a;
  if (p.n_top > 0) tmax[warp][lane] = sort_down(my_max, lane);
  __syncthreads();
  if (warp == 0) {
    Soft b = lane < kLpWarps ? soft[lane] : Soft{-INFINITY, 0.f, 0.f};
#pragma unroll
    for (int o = kLpWarps / 2; o; o >>= 1) {
      Soft c{__shfl_xor_sync(0xffffffffu, b.m, o), __shfl_xor_sync(0xffffffffu, b.s, o),
             __shfl_xor_sync(0xffffffffu, b.u, o)};
      b = join(b, c);
    }
    if (lane == 0) mine = b;
  }
  if (p.n_top > 0) {
    // the n_top-th largest thread maximum
    for (int w = kLpWarps / 2; w; w >>= 1) {
      if (warp < w) tmax[warp][lane] = merge_lists(tmax[warp][lane], tmax[warp + w][31 - lane], lane);
      __syncthreads();
    }
    if (tid == 0) bound = tmax[0][p.n_top - 1];
    __syncthreads();
    // A candidate is above thr, or equal to it with an id below tie.  Both follow
    // the n_top-th of this warp's list once there is one: of many equal logits
    // (masked ones among them) only those with low enough ids are looked at.
    float thr = bound;
    int tie = 0x7fffffff;
    uint64_t best = 0;  // lane r: the r-th best key of this warp so far, 0 for none
    int found = 0;      // keys that were put into it
    auto fits = [&](const float (&v)[N], int id, uint32_t mask) {
      uint32_t m = 0;
#pragma unroll
      for (int e = 0; e < N; ++e) m |= v[e] >= thr ? 1u << e : 0u;
      if (found >= p.n_top) {
#pragma unroll
        for (int e = 0; e < N; ++e) m &= v[e] == thr && id + e >= tie ? ~(1u << e) : ~0u;
      }
      return m & mask;
    };
    // the elements of `mask`: bit e of a lane's stands for its v[e], of id + e
    auto offer = [&](const float (&v)[N], int id, uint32_t mask) {
      mask = fits(v, id, mask);
      uint32_t set = __ballot_sync(0xffffffffu, mask != 0);
      while (set) {
        const int from = __ffs(set) - 1, e = __ffs(mask) - 1;
        float x = v[0];
#pragma unroll
        for (int i = 1; i < N; ++i) x = e == i ? v[i] : x;
        const uint64_t c = __shfl_sync(0xffffffffu, top_key(x, id + e), from);
        if (lane == from) mask &= mask - 1;
        const int at = __popc(__ballot_sync(0xffffffffu, best > c));
        const uint64_t up = __shfl_up_sync(0xffffffffu, best, 1);
        best = lane < at ? best : (lane == at ? c : up);
        set = __ballot_sync(0xffffffffu, mask != 0);
        if (++found < p.n_top || (set && found % 8)) continue;
        const uint64_t kth = __shfl_sync(0xffffffffu, best, p.n_top - 1);
        if (key_value(kth) >= thr) {
          thr = key_value(kth);
          tie = (int)~(uint32_t)kth;
          mask = fits(v, id, mask);
          set = __ballot_sync(0xffffffffu, mask != 0);
        }
      }
    };
    // the vectors of the warp's threads that reach the bound, spread over its
    // lanes in the order of their ids
    const bool mine_too = my_max >= thr;
    const uint32_t reach = __ballot_sync(0xffffffffu, mine_too);
    const float most = warp_max(my_max);
    if (mine_too) reachers[warp][__popc(reach & ((1u << lane) - 1))] = lane;
    __syncwarp();
    if (reach) {  // (the same in all lanes)
      float v[N] = {};
      if (has_head) v[0] = Vec<In>::one(x + tid);
      offer(v, tid, has_head && mine_too ? 1u : 0u);
      if (has_tail) v[0] = Vec<In>::one(x + tail0 + tid);
      offer(v, tail0 + tid, has_tail && mine_too ? 1u : 0u);
    }
    const int n_r = max(__popc(reach), 1), items = __popc(reach) * ((v1 - v0 + kLpThreads - 1) / kLpThreads);
    auto vector_of = [&](int i) { return v0 + warp * 32 + reachers[warp][i % n_r] + i / n_r * kLpThreads; };
    for (int i0 = 0; i0 < items; i0 += 32) {
      // (equal logits alone, and their ids too high: nothing of what is left fits)
      if (most <= thr && head + vector_of(i0) * N >= tie) break;
      const int i = i0 + lane, u = i < items ? vector_of(i) : v1;
      float v[N] = {};
      if (u < v1) Vec<In>::load(xv + (int64_t)u * N, v);
      offer(v, head + u * N, u < v1 ? (1u << N) - 1u : 0u);
    }
    lists[warp][lane] = best;
    __syncthreads();
    for (int w = kLpWarps / 2; w; w >>= 1) {
      if (warp < w) lists[warp][lane] = merge_lists(lists[warp][lane], lists[warp + w][31 - lane], lane);
      __syncthreads();
    }
  } else {
    __syncthreads();
  }

  // the cluster's parts
  if (p.C > 1) {
    cg::cluster_group cl = cg::this_cluster();
    cl.sync();
    if (rank == 0) {
      if (warp == 0) {
        Soft b = Soft{-INFINITY, 0.f, 0.f};
        if (lane < p.C) b = *cl.map_shared_rank(&mine, lane);
#pragma unroll
        for (int o = kLpMaxCluster / 2; o; o >>= 1) {
          Soft c{__shfl_xor_sync(0xffffffffu, b.m, o), __shfl_xor_sync(0xffffffffu, b.s, o),
                 __shfl_xor_sync(0xffffffffu, b.u, o)};
          b = join(b, c);
        }
        if (lane == 0) soft[0] = b;
      }
      if (p.n_top > 0 && warp < p.C && warp > 0) lists[warp][lane] = *(cl.map_shared_rank(&lists[0][0], warp) + lane);
    }
    cl.sync();  // the others' shared memory has been read
    if (rank != 0) return;
    if (p.n_top > 0) {
      for (int w = p.C / 2; w; w >>= 1) {
        if (warp < w) lists[warp][lane] = merge_lists(lists[warp][lane], lists[warp + w][31 - lane], lane);
        __syncthreads();
      }
    }
  } else if (tid == 0) {
    soft[0] = mine;
  }
  __syncthreads();
  if (warp != 0) return;
  const Soft r = soft[0];
  const bool none = r.m == -INFINITY && r.s == 0.f;  // no logit above -inf: no distribution
  const float ls = logf(r.s);
  if (lane == 0) {
    if (p.logprob) {
      const int t = p.tokens[row];
      float lp = __uint_as_float(0x7FC00000u);  // no such token
      if (t >= 0 && t < p.V) {
        const float v = Vec<In>::one(x + t);
        lp = none ? -INFINITY : (v - r.m) - ls;
      }
      p.logprob[row] = lp;
    }
    if (p.entropy) p.entropy[row] = none ? 0.f : ls - r.u / r.s;
  }
  if (lane < p.n_top) {
    const uint64_t k = lists[0][lane];
    p.top_ids[(int64_t)row * p.n_top + lane] = k ? (int32_t)~(uint32_t)k : -1;
    const float v = key_value(k);
    p.top_logprobs[(int64_t)row * p.n_top + lane] =
        !k ? __uint_as_float(0x7FC00000u) : (none ? -INFINITY : (v - r.m) - ls);
  }
}

template <typename In>
cudaError_t logprob_launch(const LpParams& p, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.n * p.C));
  cfg.blockDim = dim3(kLpThreads);
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
  return cudaLaunchKernelEx(&cfg, logprob_kernel<In>, p);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_token_logprobs(const void* logits, int32_t dtype, int64_t row_stride, int32_t n, int32_t V,
                                  const int32_t* tokens, int32_t n_top, float* logprob, float* entropy,
                                  int32_t* top_ids, float* top_logprobs, void* stream) {
  const char* who = "moe_token_logprobs";
  if (dtype != MOE_ACT_BF16 && dtype != MOE_ACT_F32) return set_error(MOE_EINVAL, "%s: dtype=%d", who, dtype);
  if (n < 0 || n > (1 << 24)) return set_error(MOE_EINVAL, "%s: n=%d outside 0..2^24", who, n);
  if (V < 1 || V > (1 << 24)) return set_error(MOE_EINVAL, "%s: V=%d outside 1..2^24", who, V);
  if (n_top < 0 || n_top > std::min(kLpMaxTop, V))
    return set_error(MOE_EINVAL, "%s: n_top=%d outside 0..%d", who, n_top, std::min(kLpMaxTop, V));
  if (n > 1 && row_stride < V) return set_error(MOE_EINVAL, "%s: row_stride %lld below V=%d", who, (long long)row_stride, V);
  if (n == 0) return MOE_OK;
  if (!logits || (logprob && !tokens) || (n_top > 0 && (!top_ids || !top_logprobs)))
    return set_error(MOE_EINVAL, "%s: NULL argument", who);
  if (reinterpret_cast<uintptr_t>(logits) % (dtype == MOE_ACT_BF16 ? 2 : 4))
    return set_error(MOE_EINVAL, "%s: logits misaligned", who);
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) {
    cudaGetLastError();  // reported here: the next launch of the process is not to find it
    return set_error(MOE_ECUDA, "%s: %s", who, cudaGetErrorString(e));
  }
  LpParams p{logits, row_stride, n, V, n_top, 1, tokens, logprob, entropy, top_ids, top_logprobs};
  // blocks a row: more while they stay within 5/4 of the multiprocessors and a
  // block keeps 1024 logits (33 rows of 151936 bf16 logits: 15.3, 10.9, 8.7 and
  // 9.9 us with 1, 2, 4 and 8 blocks a row; 64 of 32768 fp32: 6.9, 6.2, 6.5, 7.5;
  // 1023 of 32768: 25, 29, 34, 47)
  while (p.C < kLpMaxCluster && 2LL * n * p.C <= 5LL * sms / 4 && V / (2 * p.C) >= 1024) p.C *= 2;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  e = dtype == MOE_ACT_F32 ? logprob_launch<float>(p, st) : logprob_launch<__nv_bfloat16>(p, st);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return set_error(MOE_ECUDA, "%s launch: %s", who, cudaGetErrorString(e));
  }
  return MOE_OK;
}

// attn_commit.cu -- the cache rows of a tree's accepted nodes move to the places
// behind the prefix, and the sequences get their new lengths.
//
// Sequence b's nodes are its last m = starts[b+1] - starts[b] cached tokens,
// p0 = lens[b] - m; path[b] lists the accepted ones, ascending, so that node
// path[b][k] >= k: row p0 + k <- row p0 + path[b][k] for all k, codes and scales
// byte for byte (a key keeps the rotation of its position, which is p0 + k on
// the path).
//
// A row may be the source of one move and the target of another, so a block
// owns all rows of a (sequence, key/value head): it loads them into registers,
// at most 64 rows of 24 pieces, and stores them behind a barrier.  Bound: one
// chain of dependent loads (lengths and path, table, rows) and a launch.  Measured
// with the read of the rows after it: one tree of 12 nodes, 64/4 heads of 192, 4.0
// us; 128 trees of 64 nodes, 32/8 heads of 128, 15.7 us (13 of them the read).
#include "attn.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kCommitThreads = 256;

template <int D>
__global__ void __launch_bounds__(kCommitThreads) commit_kernel(const __grid_constant__ CommitParams p) {
  constexpr int kCodes = D / 16;   // 16-byte pieces of a row's codes (keys, then values)
  constexpr int kScales = D / 32;  // 4-byte pieces of its scales
  constexpr int kCodeSteps = kTreeNodes * kCodes / kCommitThreads, kScaleSteps = (kTreeNodes * kScales + kCommitThreads - 1) / kCommitThreads;
  __shared__ int64_t src[kTreeNodes], dst[kTreeNodes];  // a row's place (its key codes), -1: it does not move
  __shared__ int wrong[2];
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x, h = blockIdx.x, b = blockIdx.y;
  const int len = p.lens[b], m = p.starts[b + 1] - p.starts[b], p0 = len - m;
  // a sequence that is not as the call said stays as it is
  const bool ok = len >= 0 && len <= p.max_len && m >= 0 && m <= kTreeNodes && p0 >= 0;
  if (!ok) {
    if (h == 0 && tid == 0) {
      atomicOr(p.status, kBadLength);
      p.new_lens[b] = len;
    }
    return;
  }
  // the first entry that ends the path
  const int at = tid < p.width ? p.path[(int64_t)b * p.width + tid] : -1;
  if (tid < kTreeNodes) {
    const int before = tid > 0 && tid - 1 < p.width ? p.path[(int64_t)b * p.width + tid - 1] : -1;
    const bool good = at >= 0 && at < m && at > before;
    const uint32_t bad = __ballot_sync(0xffffffffu, !good);
    if ((tid & 31) == 0) wrong[tid >> 5] = bad ? __ffs(bad) - 1 : 32;
  }
  __syncthreads();
  const int n = wrong[0] < 32 ? wrong[0] : 32 + wrong[1];
  if (tid == n && tid < p.width && at != -1 && h == 0) atomicOr(p.status, kBadPath);
  if (tid < kTreeNodes) {
    int64_t s = -1, d = -1;
    if (tid < n && at != tid) {
      const int js = p0 + at, jd = p0 + tid;
      const int* row = p.table + (int64_t)b * p.table_stride;
      const int ps = row[js >> p.pshift], pd = row[jd >> p.pshift];
      if (ps >= 0 && ps < p.n_pages && pd >= 0 && pd < p.n_pages) {
        s = ps * p.page_bytes + h * p.head_bytes;
        d = pd * p.page_bytes + h * p.head_bytes;
        s = s << 8 | (js & (p.P - 1));  // (the place in the page beside the page: below 128)
        d = d << 8 | (jd & (p.P - 1));
      } else {
        atomicOr(p.status, kBadPage);
      }
    }
    src[tid] = s;
    dst[tid] = d;
  }
  __syncthreads();
  if (h == 0 && tid == 0) p.new_lens[b] = p0 + n;
  const int half = (int)(p.head_bytes / 2), codes = p.P * (D / 2);
  auto code_at = [&](int64_t where, int c) {
    const int v = c / (kCodes / 2), i = c % (kCodes / 2);
    return reinterpret_cast<uint4*>(p.pages + (where >> 8) + v * half + (where & 255) * (D / 2) + 16 * i);
  };
  auto scale_at = [&](int64_t where, int c) {
    const int v = c / (kScales / 2), i = c % (kScales / 2);
    return reinterpret_cast<uint32_t*>(p.pages + (where >> 8) + v * half + codes + (where & 255) * (D / 16) + 4 * i);
  };
  uint4 code[kCodeSteps];
  uint32_t scale[kScaleSteps];
#pragma unroll
  for (int i = 0; i < kCodeSteps; ++i) {
    const int u = tid + i * kCommitThreads, r = u / kCodes;
    if (r < n && src[r] >= 0) code[i] = *code_at(src[r], u % kCodes);
  }
#pragma unroll
  for (int i = 0; i < kScaleSteps; ++i) {
    const int u = tid + i * kCommitThreads, r = u / kScales;
    if (r < n && src[r] >= 0) scale[i] = *scale_at(src[r], u % kScales);
  }
  __syncthreads();  // every row is read before one is written
#pragma unroll
  for (int i = 0; i < kCodeSteps; ++i) {
    const int u = tid + i * kCommitThreads, r = u / kCodes;
    if (r < n && src[r] >= 0) *code_at(dst[r], u % kCodes) = code[i];
  }
#pragma unroll
  for (int i = 0; i < kScaleSteps; ++i) {
    const int u = tid + i * kCommitThreads, r = u / kScales;
    if (r < n && src[r] >= 0) *scale_at(dst[r], u % kScales) = scale[i];
  }
}

}  // namespace

cudaError_t commit_launch(const CommitParams& p, int n_seqs, cudaStream_t st) {
  const dim3 grid(p.hk, n_seqs);
  switch (p.D) {
    case 64: return launch_pdl(commit_kernel<64>, grid, kCommitThreads, 0, st, p);
    case 128: return launch_pdl(commit_kernel<128>, grid, kCommitThreads, 0, st, p);
    case 192: return launch_pdl(commit_kernel<192>, grid, kCommitThreads, 0, st, p);
    default: return launch_pdl(commit_kernel<256>, grid, kCommitThreads, 0, st, p);
  }
}

}  // namespace attn
}  // namespace moe

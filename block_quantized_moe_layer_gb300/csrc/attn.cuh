// attn.cuh -- the attention handle, the 4-bit page format and the parameter
// blocks of the attention kernels.
//
// Page format.  A page holds P tokens (P = 16, 32, 64 or 128).  For each
// key/value head in turn it holds four arrays:
//   key codes [P][D/2], key scales [P][D/16], value codes [P][D/2], value scales [P][D/16].
// 16 consecutive channels share one scale byte b: the top eight bits below
// the sign of a half-precision number, d = fp16(b << 7) (5 exponent bits, 3
// fraction bits), b <= kKvMaxScale.  A channel is (c - 8) d with c its 4-bit
// code.  Channel e of each eight consecutive ones is nibble e/2 + 4 (e%2) of
// their 32-bit word, so that masking a shifted word with 0x000F000F gives two
// neighbouring channels in the halves of a register.
//   Why these: a 4-bit uniform code with a scale for 16 channels has a smaller
// mean square error on normal data than a 4-bit floating code (0.0075 against
// 0.011 of the variance), and a 4-bit code times a scale of 4 significant bits
// is exact in bf16 and in fp16: nothing is rounded between the cache and the
// tensor core.  4.5 bits a channel.
#pragma once
#include "common.cuh"

namespace moe {
namespace attn {

constexpr int kMaxHeads = 1024;
constexpr int kKvMaxScale = 198;  // d <= 896: 72 d, the dequantisation's offset, stays finite in fp16

// Bits of the status word (kinds of bad input that a kernel met).
enum : int {
  kBadSlot = 1,      // a slot outside the page pool
  kBadPosition = 2,  // a position outside the rotation table
  kBadPage = 4,      // a block-table entry outside the page pool
  kBadLength = 8,    // sequence lengths or query starts outside what the call said
  kTimeout = 16,     // a bounded wait gave up
  kBadParent = 32,   // a tree node's parent that is no earlier node of its sequence
  kBadPath = 64,     // an accepted path that is no ascending list of the sequence's nodes
};

constexpr int kTreeNodes = 64;  // most nodes of a sequence's tree: a node's ancestors are the bits of one word

// Dequantised key/value tiles of one pass of the prompt path.
constexpr int kTileTokens = 128;
constexpr int kMaxSplit = 1024;  // most parts of a row's keys

struct AttnParams {
  int hq, hk, g, D, P, pshift, n_pages, window;
  int T, n_seqs, max_q, max_len, table_stride;
  int n_split;         // parts of the key axis
  float scale_log2;    // softmax scale times log2(e)
  const void* q;       // [T][hq][D], strides in elements
  int64_t q_tok, q_head;
  const uint8_t* pages;
  int64_t head_bytes, page_bytes;
  const int32_t *starts, *lens, *table;
  const int32_t* parents;  // [T] of a tree call, else null
  int by_length;       // 1: a tree call's blocks take the longest sequences first
  int clustered;       // 1: a tree call's parts of a row tile are a cluster, which joins them
  void* out;           // [T][hq][D]
  float* lse;          // [T][hq] or null
  float* part_o;       // [tile][split][rows][D]
  float2* part_ml;     // [tile][split][rows]: running maximum (log2 units) and sum
  int* status;
  uint64_t timeout_ns;
  int miss;            // 1 under moe_attn_inject_timeout: an arrival that the barriers of the first operands wait for in vain
};

struct CommitParams {
  uint8_t* pages;
  const int32_t *starts, *lens, *table, *path;
  int32_t* new_lens;
  int table_stride, width, max_len, hk, D, P, pshift, n_pages;
  int64_t head_bytes, page_bytes;
  int* status;
};

// One sequence of the call, clamped to what the call said (a value outside is
// flagged, never followed).
struct Seq {
  int start, nq, len;
};
__device__ __forceinline__ Seq load_seq(const AttnParams& p, int b) {
  Seq s;
  const int a = p.starts[b], e = p.starts[b + 1], n = p.lens[b];
  s.start = min(max(a, 0), p.T);
  s.nq = min(max(e, s.start), p.T) - s.start;
  s.nq = min(s.nq, p.max_q);
  s.len = min(max(n, 0), p.max_len);
  if ((s.start != a || s.start + s.nq != e || s.len != n) && threadIdx.x == 0) atomicOr(p.status, kBadLength);
  return s;
}

// The sequence with the i-th most cached tokens (the lower one first of two
// equal ones), for a block of all its threads.  Where a call has more blocks than
// the GPU holds at once, those that start last are then the shortest, and end with
// the others.  A length is compared with all others, so a call has few sequences.
constexpr int kSortedSeqs = 128;
__device__ __forceinline__ int seq_by_length(const AttnParams& p, int i) {
  __shared__ int found;
  for (int t = threadIdx.x; t < p.n_seqs; t += blockDim.x) {
    const int n = p.lens[t];
    int before = 0;
#pragma unroll 8
    for (int u = 0; u < p.n_seqs; ++u) {
      const int o = p.lens[u];
      before += o > n || (o == n && u < t);
    }
    if (before == i) found = t;
  }
  __syncthreads();
  return found;
}

// The page of the tokens [i P, (i + 1) P) of sequence b, or -1 for an entry
// outside the pool, which is reported; in two steps where the load is to be on
// its way meanwhile (its result is not touched before the second one; seen:
// the entry was loaded, else pg is -1).
__device__ __forceinline__ int page_entry(const AttnParams& p, int b, int i) { return p.table[(int64_t)b * p.table_stride + i]; }
__device__ __forceinline__ int checked_page(const AttnParams& p, int pg, bool seen) {
  if (pg >= 0 && pg < p.n_pages) return pg;
  if (seen) atomicOr(p.status, kBadPage);
  return -1;
}
__device__ __forceinline__ int load_page(const AttnParams& p, int b, int i) { return checked_page(p, page_entry(p, b, i), true); }

// Keys visible to a query at position pos: [key_lo(pos), pos].
__device__ __forceinline__ int key_lo(const AttnParams& p, int pos) {
  return p.window > 0 ? max(0, pos - p.window + 1) : 0;
}

// The ancestors of a sequence's tree nodes, themselves among them: bit a of a
// node's word stands for node a.  One warp; lane i takes the nodes i and
// i + 32.  Each round doubles how far up a word reaches, so a chain of 64 nodes
// takes 6 rounds, the usual tree 2 or 3.  A parent that is no earlier node is
// reported and taken as -1 (the node follows the prefix).
struct TreeWords {
  uint64_t word[2];
};
__device__ __forceinline__ TreeWords tree_words(const AttnParams& p, const Seq& s) {
  const int lane = threadIdx.x & 31;
  int up[2];
  TreeWords t;
  bool bad = false;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = lane + 32 * k;
    up[k] = -1;
    t.word[k] = 0;
    if (i < s.nq) {
      const int u = p.parents[s.start + i];
      up[k] = u >= 0 && u < i ? u : -1;
      bad |= u != up[k];
      t.word[k] = 1ull << i;
    }
  }
  if (bad) atomicOr(p.status, kBadParent);
#pragma unroll 1
  for (int round = 0; round < 6; ++round) {
    if (!__any_sync(0xffffffffu, up[0] >= 0 || up[1] >= 0)) break;
    uint64_t w[2];
    int n[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int from = up[k] & 31;
      const uint64_t w0 = __shfl_sync(0xffffffffu, t.word[0], from), w1 = __shfl_sync(0xffffffffu, t.word[1], from);
      const int n0 = __shfl_sync(0xffffffffu, up[0], from), n1 = __shfl_sync(0xffffffffu, up[1], from);
      w[k] = up[k] < 0 ? 0 : (up[k] < 32 ? w0 : w1);
      n[k] = up[k] < 0 ? -1 : (up[k] < 32 ? n0 : n1);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      t.word[k] |= w[k];
      up[k] = n[k];
    }
  }
  return t;
}
// What a tree node sees: the tokens [lo, p0) before the tree and the nodes of
// `word`.  A node stands at position p0 + its depth; within a window it sees
// the nearest of its ancestors, which are the highest bits.
struct TreeRow {
  uint64_t word;
  int lo;
};
__device__ __forceinline__ TreeRow tree_row(const AttnParams& p, int p0, uint64_t word) {
  const int n = __popcll(word);
  TreeRow r{word, key_lo(p, p0 + n - 1)};
  if (p.window > 0)
    for (int k = p.window; k < n; ++k) r.word &= r.word - 1;
  return r;
}
__device__ __forceinline__ bool tree_sees(const TreeRow& r, int p0, int j) {
  const int a = j - p0;
  return a < 0 ? j >= r.lo : a < kTreeNodes && ((r.word >> a) & 1);
}

// A row's softmax reference once it has seen a key, whatever the key's score:
// -inf stands for no key (the row is 0), so that a row whose scores are NaN, or
// all -inf, becomes NaN.
constexpr float kSeen = -3.402823466e+38f;

__device__ __forceinline__ float scale_value(int b) { return __half2float(__ushort_as_half((unsigned short)(b << 7))); }

}  // namespace attn
}  // namespace moe

struct moe_attn {
  int dev = 0, num_sms = 0;
  int hq = 0, hk = 0, D = 0, P = 0, n_pages = 0, rot = 0, interleaved = 0, window = 0, act = 0;
  int T_max = 0, S_max = 0, len_max = 0;
  float eps = 0.f, scale = 0.f;
  int inject_us = 0;           // one-shot wait-timeout test hook (moe_attn_inject_timeout)
  float* rope = nullptr;       // [2: rounded, rest][len_max][2: cos, sin][rot/2]
  double* freq = nullptr;      // [rot/2]
  float* norm_w = nullptr;     // [2][D]: query and key weights (ones where there are none)
  bool q_norm = false, k_norm = false;
  int* status = nullptr;       // [4]
  uint8_t* ws = nullptr;       // parts of split rows, dequantised tiles
  size_t part_rows = 0;        // rows of parts that fit
  size_t ws_bytes = 0;
  size_t tile_off = 0;         // dequantised tiles in ws
  int tile_cap = 0;            // 128-token tiles (of all kv heads) that fit
  int64_t head_bytes = 0, page_bytes = 0;
};

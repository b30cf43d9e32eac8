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
};

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
  void* out;           // [T][hq][D]
  float* lse;          // [T][hq] or null
  float* part_o;       // [tile][split][rows][D]
  float2* part_ml;     // [tile][split][rows]: running maximum (log2 units) and sum
  int* status;
  uint64_t timeout_ns;
  int miss;            // 1 under moe_attn_inject_timeout: an arrival that the barriers of the first operands wait for in vain
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

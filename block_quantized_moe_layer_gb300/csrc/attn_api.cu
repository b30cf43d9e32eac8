// attn_api.cu -- the extern "C" entry points of the attention operators
// (include/moe_layer.h): the handle, append, read, forward.
#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "attn.cuh"
#include "layer.cuh"

namespace moe {
namespace attn {
cudaError_t append_launch(const moe_attn* h, const void* q, const void* k, const void* v, bool in_f32,
                          const int64_t* strides, const int32_t* positions, const int64_t* slots, int T, void* pages,
                          void* q_out, cudaStream_t st);
cudaError_t read_launch(const moe_attn* h, const void* pages, const int64_t* slots, int n, void* k_out, void* v_out,
                        cudaStream_t st);
cudaError_t rope_launch(const moe_attn* h, cudaStream_t st);
cudaError_t append_configure(const moe_attn* h);
cudaError_t check_launch(const AttnParams& p, cudaStream_t st);
cudaError_t small_configure(int D);
cudaError_t small_launch(const AttnParams& p, int num_sms, size_t part_rows, cudaStream_t st);
cudaError_t verify_configure(int D);
cudaError_t verify_launch(const AttnParams& p, int num_sms, size_t part_rows, cudaStream_t st);
size_t prompt_ws_bytes(int D, int tile_cap);
cudaError_t prompt_configure();
cudaError_t prompt_launch(const AttnParams& p, int num_sms, size_t part_rows, uint8_t* ws, int tile_cap, cudaStream_t st);
cudaError_t tree_configure(int D);
cudaError_t tree_launch(const AttnParams& p, int num_sms, size_t part_rows, cudaStream_t st);
cudaError_t commit_launch(const CommitParams& p, int n_seqs, cudaStream_t st);
}  // namespace attn
}  // namespace moe

using namespace moe;

namespace {

int cuda_fail(cudaError_t e, const char* what) {
  cudaGetLastError();  // reported here: the next launch of the process is not to find it
  return set_error(e == cudaErrorMemoryAllocation ? MOE_ENOMEM : MOE_ECUDA, "%s: %s", what, cudaGetErrorString(e));
}
int launch_fail(cudaError_t e, const char* who, const char* kernel) {
  cudaGetLastError();
  return set_error(MOE_ECUDA, "%s launch%s: %s", who, kernel, cudaGetErrorString(e));
}
#define CKA(call, what)                              \
  do {                                               \
    cudaError_t e_ = (call);                         \
    if (e_ != cudaSuccess) return cuda_fail(e_, what); \
  } while (0)

// Rows (query tokens times query heads of a key/value head) of a sequence up
// to which a call runs on the small-row kernel, and on the verify kernel.  That
// one reads the cache again for each 64 rows, but needs no expansion: verify
// and prompt kernel take, for one sequence of 8000 keys, 20.5 and 30.6 us at 144
// rows (heads of 192), 27 and 36 at 256 (128), 22 and 33 (256); for 8 sequences
// 93 and 111, 145 and 144, 92 and 90.  Heads of 64, whose products are short
// beside their softmax, 30 and 39 us at 141 rows, 41 and 39 at 256; for 8
// sequences 200 and 219, 265 and 221.
constexpr int kSmallCallRows = 16;
constexpr int verify_call_rows(int D) { return D == 64 ? 192 : 256; }
// The same of a tree, above which it runs on pairs of blocks that share their keys:
// one sequence of 32000 tokens, heads of 192, 33 us (verify) and 34 (pairs) at 128
// rows, 44 and 35 at 192, 56 and 37 at 256; 8 sequences of up to 8000 56 and 55, 90
// and 56, 90 and 57; heads of 128 72 and 79, 97 and 79, 116 and 79; heads of 64 68
// and 73, 90 and 73, 106 and 73.  Heads of 256, whose products are the most beside
// the dequantisation, 36 and 49 at 64 rows, 53 and 41 at 96.  (Expanded in memory
// first, as a prompt's, 1024 rows of 8 sequences of 8000 tokens took 171, pairs 152.)
constexpr int tree_verify_rows(int D) { return D == 256 ? 64 : 128; }

bool head_dim_ok(int D) { return D == 64 || D == 128 || D == 192 || D == 256; }
bool page_ok(int P) { return P == 16 || P == 32 || P == 64 || P == 128; }
uintptr_t addr(const void* p) { return reinterpret_cast<uintptr_t>(p); }

void free_attn(moe_attn* h) {
  if (!h) return;
  cudaFree(h->rope);
  cudaFree(h->freq);
  cudaFree(h->norm_w);
  cudaFree(h->status);
  cudaFree(h->ws);
  delete h;
}

// Rows of [heads][D] read with the given strides (elements of esz bytes):
// every 8-channel piece has to start on a 16-byte boundary.
int check_rows(const char* who, const char* name, const void* p, int64_t tok, int64_t head, int D, int heads, size_t esz) {
  if (!p) return set_error(MOE_EINVAL, "%s: NULL %s", who, name);
  if (addr(p) & 15) return set_error(MOE_EINVAL, "%s: %s must be 16-byte aligned", who, name);
  if (head < 0 || tok < 0 || (head * (int64_t)esz) % 16 || (tok * (int64_t)esz) % 16)
    return set_error(MOE_EINVAL, "%s: %s's strides (%lld, %lld elements) must be multiples of 16 bytes", who, name,
                     (long long)tok, (long long)head);
  if (heads > 1 && head < D)
    return set_error(MOE_EINVAL, "%s: %s's head stride %lld is below the head's %d channels", who, name, (long long)head, D);
  return MOE_OK;
}

// moe_attn_forward, and with parents moe_attn_forward_tree.
int forward(const char* who, moe_attn* h, const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* pages,
            const int32_t* starts, const int32_t* lens, const int32_t* table, int32_t table_stride, const int32_t* parents,
            int32_t n_seqs, int32_t T, int32_t max_q, int32_t max_len, void* out, float* lse, void* stream) {
  if (!h) return set_error(MOE_EINVAL, "%s: NULL handle", who);
  if (T < 0 || T > h->T_max) return set_error(MOE_EINVAL, "%s: T=%d outside 0..%d", who, T, h->T_max);
  if (n_seqs < 0 || n_seqs > h->S_max) return set_error(MOE_EINVAL, "%s: n_seqs=%d outside 0..%d", who, n_seqs, h->S_max);
  if (max_q < 0 || max_q > T) return set_error(MOE_EINVAL, "%s: max_q=%d outside 0..T=%d", who, max_q, T);
  if (max_len < 0 || max_len > h->len_max)
    return set_error(MOE_EINVAL, "%s: max_len=%d outside 0..%d", who, max_len, h->len_max);
  if (T == 0 || n_seqs == 0 || max_q == 0) return MOE_OK;
  if (!pages || !starts || !lens || (!table && max_len > 0) || !out) return set_error(MOE_EINVAL, "%s: NULL argument", who);
  if ((int64_t)table_stride * h->P < max_len)
    return set_error(MOE_EINVAL, "%s: %d table entries a sequence hold %lld tokens, max_len is %d", who, table_stride,
                     (long long)table_stride * h->P, max_len);
  const size_t esz = h->act == MOE_ACT_BF16 ? 2 : 4;
  int rc;
  if ((rc = check_rows(who, "q", q, q_token_stride, q_head_stride, h->D, h->hq, esz))) return rc;
  if ((addr(pages) | addr(out)) & 15) return set_error(MOE_EINVAL, "%s: pages and out must be 16-byte aligned", who);
  if ((addr(starts) | addr(lens) | addr(table) | addr(lse) | addr(parents)) & 3)
    return set_error(MOE_EINVAL, "%s: starts, lens, table, parents and lse must be 4-byte aligned", who);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  attn::AttnParams p{};
  p.hq = h->hq; p.hk = h->hk; p.g = h->hq / h->hk; p.D = h->D; p.P = h->P;
  p.pshift = 31 - __builtin_clz((unsigned)h->P);
  p.n_pages = h->n_pages; p.window = h->window;
  p.T = T; p.n_seqs = n_seqs; p.max_q = max_q; p.max_len = max_len; p.table_stride = table_stride;
  p.n_split = 1;
  p.scale_log2 = h->scale * 1.44269504088896341f;
  p.q = q; p.q_tok = q_token_stride; p.q_head = q_head_stride;
  p.pages = static_cast<const uint8_t*>(pages);
  p.head_bytes = h->head_bytes; p.page_bytes = h->page_bytes;
  p.starts = starts; p.lens = lens; p.table = table; p.parents = parents;
  p.out = out; p.lse = lse;
  p.status = h->status;
  p.timeout_ns = 2000000000ull;
  if (h->act == MOE_ACT_F32) {
    const cudaError_t e = attn::check_launch(p, st);
    return e == cudaSuccess ? MOE_OK : launch_fail(e, who, " (fp32)");
  }
  if (h->inject_us > 0) {  // one launch
    p.timeout_ns = 1000ull * h->inject_us;
    p.miss = 1;
    h->inject_us = 0;
  }
  p.part_o = reinterpret_cast<float*>(h->ws);
  p.part_ml = reinterpret_cast<float2*>(h->ws + h->part_rows * h->D * sizeof(float));
  const int64_t rows = (int64_t)max_q * p.g;
  const char* kernel = "";
  cudaError_t e;
  if (rows <= kSmallCallRows) {
    e = attn::small_launch(p, h->num_sms, h->part_rows, st);
  } else if (parents && rows > tree_verify_rows(h->D)) {
    kernel = " (tree)";
    e = attn::tree_launch(p, h->num_sms, h->part_rows, st);
  } else if (rows <= verify_call_rows(h->D)) {
    kernel = " (verify)";
    e = attn::verify_launch(p, h->num_sms, h->part_rows, st);
  } else {
    kernel = " (prompt)";
    e = attn::prompt_launch(p, h->num_sms, h->part_rows, h->ws + h->tile_off, h->tile_cap, st);
  }
  return e == cudaSuccess ? MOE_OK : launch_fail(e, who, kernel);
}

}  // namespace

extern "C" {

size_t moe_attn_page_bytes(int32_t n_kv_heads, int32_t head_dim, int32_t page_tokens) {
  if (n_kv_heads < 1 || n_kv_heads > attn::kMaxHeads || !head_dim_ok(head_dim) || !page_ok(page_tokens)) return 0;
  return (size_t)n_kv_heads * page_tokens * head_dim * 9 / 8;
}

int moe_attn_create(const moe_attn_desc* d, void* stream, moe_attn** out) {
  if (!d || !out) return set_error(MOE_EINVAL, "moe_attn_create: NULL argument");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (d->n_kv_heads < 1 || d->n_q_heads < 1 || d->n_q_heads > attn::kMaxHeads || d->n_q_heads % d->n_kv_heads)
    return set_error(MOE_EINVAL, "moe_attn_create: %d query heads and %d key/value heads (1..%d, a multiple)",
                     d->n_q_heads, d->n_kv_heads, attn::kMaxHeads);
  if (!head_dim_ok(d->head_dim))
    return set_error(MOE_EINVAL, "moe_attn_create: head_dim=%d (64, 128, 192 or 256)", d->head_dim);
  if (!page_ok(d->page_tokens))
    return set_error(MOE_EINVAL, "moe_attn_create: page_tokens=%d (16, 32, 64 or 128)", d->page_tokens);
  if (d->n_pages < 1) return set_error(MOE_EINVAL, "moe_attn_create: n_pages=%d", d->n_pages);
  if (d->rot_dim < 0 || d->rot_dim > d->head_dim || d->rot_dim % 16)
    return set_error(MOE_EINVAL, "moe_attn_create: rot_dim=%d must be a multiple of 16 in 0..head_dim", d->rot_dim);
  if (d->interleaved != 0 && d->interleaved != 1)
    return set_error(MOE_EINVAL, "moe_attn_create: interleaved=%d", d->interleaved);
  if (d->window < 0) return set_error(MOE_EINVAL, "moe_attn_create: window=%d", d->window);
  if (d->act_dtype != MOE_ACT_BF16 && d->act_dtype != MOE_ACT_F32)
    return set_error(MOE_EINVAL, "moe_attn_create: act_dtype=%d", d->act_dtype);
  if (d->T_max < 1 || d->T_max > (1 << 20)) return set_error(MOE_EINVAL, "moe_attn_create: T_max=%d outside 1..2^20", d->T_max);
  if (d->S_max < 1 || d->S_max > 65535) return set_error(MOE_EINVAL, "moe_attn_create: S_max=%d outside 1..65535", d->S_max);
  if (d->len_max < 1 || d->len_max > (1 << 27))
    return set_error(MOE_EINVAL, "moe_attn_create: len_max=%d outside 1..2^27", d->len_max);
  if (!(d->eps >= 0.f) || d->eps > 1e30f) return set_error(MOE_EINVAL, "moe_attn_create: eps must be finite and >= 0");
  if (!(d->scale >= 0.f) || d->scale > 1e30f)
    return set_error(MOE_EINVAL, "moe_attn_create: scale must be finite and >= 0 (0: 1/sqrt(head_dim))");
  if (!(d->rope_base >= 0.0) || d->rope_base > 1e30)
    return set_error(MOE_EINVAL, "moe_attn_create: rope_base must be finite and >= 0 (0: 10000)");

  double f[128];  // angles a token (rot_dim <= 256), alive until the stream has copied them
  moe_attn* h = new (std::nothrow) moe_attn();
  if (!h) return set_error(MOE_ENOMEM, "moe_attn_create: host allocation");
  struct Guard {
    moe_attn* h;
    bool keep = false;
    ~Guard() {
      if (!keep) free_attn(h);
    }
  } guard{h};
  h->hq = d->n_q_heads; h->hk = d->n_kv_heads; h->D = d->head_dim; h->P = d->page_tokens;
  h->n_pages = d->n_pages; h->rot = d->rot_dim; h->interleaved = d->interleaved;
  // A window that holds every sequence is none.  So position - window, with
  // positions down to -T_max, stays within 32 bits.
  h->window = d->window < d->len_max ? d->window : 0;
  h->act = d->act_dtype; h->T_max = d->T_max; h->S_max = d->S_max; h->len_max = d->len_max;
  h->eps = d->eps;
  h->scale = d->scale > 0.f ? d->scale : (float)(1.0 / std::sqrt((double)d->head_dim));
  h->head_bytes = (int64_t)h->P * h->D * 9 / 8;
  h->page_bytes = h->head_bytes * h->hk;
  h->q_norm = d->q_norm != nullptr;
  h->k_norm = d->k_norm != nullptr;

  CKA(cudaGetDevice(&h->dev), "cudaGetDevice");
  CKA(cudaDeviceGetAttribute(&h->num_sms, cudaDevAttrMultiProcessorCount, h->dev), "SM count");
  CKA(cudaMalloc(&h->status, 16), "alloc status");
  CKA(cudaMemsetAsync(h->status, 0, 16, st), "zero status");
  if (h->rot) {
    const int half = h->rot / 2;
    for (int i = 0; i < half; ++i) {
      f[i] = d->freq ? d->freq[i] : std::pow(d->rope_base > 0.0 ? d->rope_base : 10000.0, -2.0 * i / h->rot);
      if (!(std::fabs(f[i]) <= 1e30)) return set_error(MOE_EINVAL, "moe_attn_create: freq[%d] is not finite", i);
    }
    CKA(cudaMalloc(&h->freq, half * sizeof(double)), "alloc frequencies");
    CKA(cudaMalloc(&h->rope, (size_t)2 * h->len_max * h->rot * sizeof(float)), "alloc rotation table");
    // (on the table's own stream: the default stream's copies are not ordered with it)
    CKA(cudaMemcpyAsync(h->freq, f, half * sizeof(double), cudaMemcpyHostToDevice, st), "copy frequencies");
    CKA(attn::rope_launch(h, st), "rotation table");
  }
  if (h->q_norm || h->k_norm) {
    CKA(cudaMalloc(&h->norm_w, (size_t)2 * h->D * sizeof(float)), "alloc norm weights");
    if (h->q_norm)
      CKA(cudaMemcpyAsync(h->norm_w, d->q_norm, h->D * sizeof(float), cudaMemcpyDefault, st), "copy query norm");
    if (h->k_norm)
      CKA(cudaMemcpyAsync(h->norm_w + h->D, d->k_norm, h->D * sizeof(float), cudaMemcpyDefault, st), "copy key norm");
  }
  CKA(attn::append_configure(h), "configure the append kernels");
  if (h->act == MOE_ACT_BF16) {
    h->part_rows = (size_t)128 * h->num_sms;
    h->ws_bytes = h->part_rows * (h->D * sizeof(float) + sizeof(float2));
    const int64_t most_rows = (int64_t)h->T_max * (h->hq / h->hk);
    if (most_rows > kSmallCallRows) CKA(attn::verify_configure(h->D), "configure the verify kernel");
    if (most_rows > tree_verify_rows(h->D)) CKA(attn::tree_configure(h->D), "configure the tree kernel");
    if (most_rows > verify_call_rows(h->D)) {
      // dequantised tiles of one longest sequence at least (of what its window
      // and a call's queries reach), of more while they stay within 256 MB
      int64_t reach = h->len_max;
      if (h->window > 0) reach = std::min<int64_t>(reach, (int64_t)h->window + h->T_max + 2 * attn::kTileTokens);
      const int64_t one = h->hk * ((reach + attn::kTileTokens - 1) / attn::kTileTokens);
      const int64_t room = (256LL << 20) / (4LL * attn::kTileTokens * h->D);
      const int64_t cap = one * std::max<int64_t>(1, std::min<int64_t>(h->S_max, room / one));
      if (cap > (1 << 28)) return set_error(MOE_EINVAL, "moe_attn_create: len_max=%d with %d heads is too long", h->len_max, h->hk);
      h->tile_cap = (int)cap;
      h->tile_off = (h->ws_bytes + 255) / 256 * 256;
      h->ws_bytes = h->tile_off + attn::prompt_ws_bytes(h->D, h->tile_cap);
      CKA(attn::prompt_configure(), "configure the prompt kernel");
    }
    CKA(cudaMalloc(&h->ws, h->ws_bytes), "alloc workspace");
    CKA(attn::small_configure(h->D), "configure the attention kernels");
  }
  CKA(cudaStreamSynchronize(st), "create sync");
  guard.keep = true;
  *out = h;
  set_error(MOE_OK, "no error");
  return MOE_OK;
}

int moe_attn_append(moe_attn* h, const void* q, const void* k, const void* v, int32_t in_dtype, const int64_t* strides,
                    const int32_t* positions, const int64_t* slots, int32_t T, void* pages, void* q_out, void* stream) {
  const char* who = "moe_attn_append";
  if (!h) return set_error(MOE_EINVAL, "%s: NULL handle", who);
  if (T < 0 || T > h->T_max) return set_error(MOE_EINVAL, "%s: T=%d outside 0..%d", who, T, h->T_max);
  if (in_dtype != MOE_ACT_BF16 && in_dtype != MOE_ACT_F32) return set_error(MOE_EINVAL, "%s: in_dtype=%d", who, in_dtype);
  if (T == 0) return MOE_OK;
  if (!strides || !positions || !slots || !pages || !q_out) return set_error(MOE_EINVAL, "%s: NULL argument", who);
  const size_t esz = in_dtype == MOE_ACT_BF16 ? 2 : 4;
  int rc;
  if ((rc = check_rows(who, "q", q, strides[0], strides[1], h->D, h->hq, esz))) return rc;
  if ((rc = check_rows(who, "k", k, strides[2], strides[3], h->D, h->hk, esz))) return rc;
  if ((rc = check_rows(who, "v", v, strides[4], strides[5], h->D, h->hk, esz))) return rc;
  if ((addr(pages) | addr(q_out)) & 15) return set_error(MOE_EINVAL, "%s: pages and q_out must be 16-byte aligned", who);
  if ((addr(positions) & 3) || (addr(slots) & 7)) return set_error(MOE_EINVAL, "%s: positions or slots misaligned", who);
  CKA(attn::append_launch(h, q, k, v, in_dtype == MOE_ACT_F32, strides, positions, slots, T, pages, q_out,
                          static_cast<cudaStream_t>(stream)),
      "moe_attn_append launch");
  return MOE_OK;
}

int moe_attn_read(moe_attn* h, const void* pages, const int64_t* slots, int32_t n, void* k_out, void* v_out, void* stream) {
  const char* who = "moe_attn_read";
  if (!h) return set_error(MOE_EINVAL, "%s: NULL handle", who);
  if (n < 0) return set_error(MOE_EINVAL, "%s: n=%d", who, n);
  if (n == 0 || (!k_out && !v_out)) return MOE_OK;
  if (!pages || !slots) return set_error(MOE_EINVAL, "%s: NULL argument", who);
  if ((addr(pages) | addr(k_out) | addr(v_out)) & 15)
    return set_error(MOE_EINVAL, "%s: pages, k_out and v_out must be 16-byte aligned", who);
  if (addr(slots) & 7) return set_error(MOE_EINVAL, "%s: slots misaligned", who);
  CKA(attn::read_launch(h, pages, slots, n, k_out, v_out, static_cast<cudaStream_t>(stream)), "moe_attn_read launch");
  return MOE_OK;
}

int moe_attn_forward(moe_attn* h, const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* pages,
                     const int32_t* starts, const int32_t* lens, const int32_t* table, int32_t table_stride,
                     int32_t n_seqs, int32_t T, int32_t max_q, int32_t max_len, void* out, float* lse, void* stream) {
  return forward("moe_attn_forward", h, q, q_token_stride, q_head_stride, pages, starts, lens, table, table_stride, nullptr, n_seqs,
                 T, max_q, max_len, out, lse, stream);
}

int moe_attn_forward_tree(moe_attn* h, const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* pages,
                          const int32_t* starts, const int32_t* lens, const int32_t* table, int32_t table_stride,
                          const int32_t* parents, int32_t n_seqs, int32_t T, int32_t max_q, int32_t max_len, void* out,
                          float* lse, void* stream) {
  const char* who = "moe_attn_forward_tree";
  if (max_q > attn::kTreeNodes)
    return set_error(MOE_EINVAL, "%s: max_q=%d, a tree has at most %d nodes", who, max_q, attn::kTreeNodes);
  if (!parents && T > 0) return set_error(MOE_EINVAL, "%s: NULL parents", who);
  return forward(who, h, q, q_token_stride, q_head_stride, pages, starts, lens, table, table_stride, parents, n_seqs, T, max_q,
                 max_len, out, lse, stream);
}

int moe_attn_commit(moe_attn* h, void* pages, const int32_t* starts, const int32_t* lens, const int32_t* table,
                    int32_t table_stride, const int32_t* path, int32_t path_width, int32_t n_seqs, int32_t max_len,
                    int32_t* new_lens, void* stream) {
  const char* who = "moe_attn_commit";
  if (!h) return set_error(MOE_EINVAL, "%s: NULL handle", who);
  if (n_seqs < 0 || n_seqs > h->S_max) return set_error(MOE_EINVAL, "%s: n_seqs=%d outside 0..%d", who, n_seqs, h->S_max);
  if (path_width < 0 || path_width > attn::kTreeNodes)
    return set_error(MOE_EINVAL, "%s: path_width=%d outside 0..%d", who, path_width, attn::kTreeNodes);
  if (max_len < 0 || max_len > h->len_max)
    return set_error(MOE_EINVAL, "%s: max_len=%d outside 0..%d", who, max_len, h->len_max);
  if (n_seqs == 0) return MOE_OK;
  if (!pages || !starts || !lens || (!table && max_len > 0) || (!path && path_width > 0) || !new_lens)
    return set_error(MOE_EINVAL, "%s: NULL argument", who);
  if ((int64_t)table_stride * h->P < max_len)
    return set_error(MOE_EINVAL, "%s: %d table entries a sequence hold %lld tokens, max_len is %d", who, table_stride,
                     (long long)table_stride * h->P, max_len);
  if (addr(pages) & 15) return set_error(MOE_EINVAL, "%s: pages must be 16-byte aligned", who);
  if ((addr(starts) | addr(lens) | addr(table) | addr(path) | addr(new_lens)) & 3)
    return set_error(MOE_EINVAL, "%s: starts, lens, table, path and new_lens must be 4-byte aligned", who);
  // (lens is read by other blocks than the one that writes a sequence's new length)
  if (addr(new_lens) < addr(lens) + 4 * (size_t)n_seqs && addr(lens) < addr(new_lens) + 4 * (size_t)n_seqs)
    return set_error(MOE_EINVAL, "%s: new_lens must not overlap lens", who);
  attn::CommitParams p{};
  p.pages = static_cast<uint8_t*>(pages);
  p.starts = starts; p.lens = lens; p.table = table; p.path = path; p.new_lens = new_lens;
  p.table_stride = table_stride; p.width = path_width; p.max_len = max_len;
  p.hk = h->hk; p.D = h->D; p.P = h->P; p.pshift = 31 - __builtin_clz((unsigned)h->P);
  p.n_pages = h->n_pages; p.head_bytes = h->head_bytes; p.page_bytes = h->page_bytes;
  p.status = h->status;
  CKA(attn::commit_launch(p, n_seqs, static_cast<cudaStream_t>(stream)), "moe_attn_commit launch");
  return MOE_OK;
}

int moe_attn_status(moe_attn* h, void* stream) {
  if (!h) return set_error(MOE_EINVAL, "moe_attn_status: NULL handle");
  CKA(cudaStreamSynchronize(static_cast<cudaStream_t>(stream)), "status sync");
  int w[4] = {0, 0, 0, 0};
  CKA(cudaMemcpy(w, h->status, 16, cudaMemcpyDeviceToHost), "status read");
  if (!w[0]) return MOE_OK;
  CKA(cudaMemset(h->status, 0, 16), "status reset");
  CKA(cudaDeviceSynchronize(), "status reset sync");
  if (w[0] & attn::kTimeout) return set_error(MOE_ETIMEOUT, "a device-side wait timed out (site %d)", w[1]);
  return set_error(MOE_EINVAL, "an earlier call met%s%s%s%s%s%s", w[0] & attn::kBadSlot ? " a slot outside the pages;" : "",
                   w[0] & attn::kBadPosition ? " a position outside 0..len_max-1;" : "",
                   w[0] & attn::kBadPage ? " a block-table entry outside the pages;" : "",
                   w[0] & attn::kBadLength ? " lengths or query starts outside the call's T, max_q or max_len;" : "",
                   w[0] & attn::kBadParent ? " a tree node's parent that is no earlier node;" : "",
                   w[0] & attn::kBadPath ? " a path that is no ascending list of a sequence's nodes;" : "");
}

int moe_attn_inject_timeout(moe_attn* h, int32_t wait_limit_us) {
  if (!h) return set_error(MOE_EINVAL, "moe_attn_inject_timeout: NULL handle");
  if (h->act == MOE_ACT_F32) return set_error(MOE_EINVAL, "moe_attn_inject_timeout: the fp32 kernel has no waits");
  if (wait_limit_us < 1 || wait_limit_us > 1000000)
    return set_error(MOE_EINVAL, "moe_attn_inject_timeout: wait_limit_us=%d outside 1..10^6", wait_limit_us);
  h->inject_us = wait_limit_us;
  return MOE_OK;
}

size_t moe_attn_workspace_bytes(const moe_attn* h) { return h ? h->ws_bytes : 0; }

void moe_attn_destroy(moe_attn* h) { free_attn(h); }

}  // extern "C"

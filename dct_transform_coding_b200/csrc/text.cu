// C ABI of the text cache (host side): argument checks, workspace, launches.
#include <climits>

#include "text.cuh"

namespace tactkv {
namespace text {
namespace {

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

tactkv_status check_cache(const tactkv_text_cache* c, Cache& out) {
  if (!c || c->format < TACTKV_TEXT_BF16 || c->format > TACTKV_TEXT_MXFP4 || c->heads < 1 || c->head_dim < 1 ||
      c->page_tokens < 1 || c->n_pages < 1)
    return TACTKV_INVALID_ARG;
  if (c->head_dim % kGroup || c->head_dim > kMaxHeadDim || c->heads > 65536 / c->head_dim || c->page_tokens < 16 ||
      c->page_tokens > 1024 || (c->page_tokens & (c->page_tokens - 1)) || c->n_pages > INT_MAX)
    return TACTKV_UNSUPPORTED_SHAPE;
  out.pages[0] = static_cast<unsigned char*>(c->k_pages);
  out.pages[1] = static_cast<unsigned char*>(c->v_pages);
  out.scales[0] = static_cast<unsigned char*>(c->k_scales);
  out.scales[1] = static_cast<unsigned char*>(c->v_scales);
  out.n_pages = c->n_pages;
  out.heads = c->heads;
  out.head_dim = c->head_dim;
  out.page_log2 = 0;
  while ((1 << out.page_log2) < c->page_tokens) ++out.page_log2;
  return TACTKV_OK;
}

// The cache with its pools, and the batch.
tactkv_status check(const tactkv_text_cache* c, const tactkv_text_batch* b, uint32_t flags, Cache& cache, Batch& batch) {
  const tactkv_status st = check_cache(c, cache);
  if (st != TACTKV_OK) return st;
  if (!b || b->n_seqs < 0 || b->n_rows < 0 || b->max_pages < 0 || (flags & ~TACTKV_FP32_IO)) return TACTKV_INVALID_ARG;
  const bool coded = c->format != TACTKV_TEXT_BF16;
  if (!c->k_pages || !c->v_pages || (coded && (!c->k_scales || !c->v_scales))) return TACTKV_INVALID_ARG;
  if (!aligned(c->k_pages, 16) || !aligned(c->v_pages, 16) ||
      (coded && (!aligned(c->k_scales, 16) || !aligned(c->v_scales, 16))))
    return TACTKV_ALIGNMENT;
  if (b->n_seqs > 0 && b->n_rows > 0) {
    if (!b->kv_lens || !b->row_starts || (b->max_pages > 0 && !b->page_table)) return TACTKV_INVALID_ARG;
    if (!aligned(b->kv_lens, 4) || !aligned(b->row_starts, 4) || !aligned(b->page_table, 4)) return TACTKV_ALIGNMENT;
  }
  batch.table = b->page_table;
  batch.kv_lens = b->kv_lens;
  batch.row_starts = b->row_starts;
  batch.n_seqs = b->n_seqs;
  batch.n_rows = b->n_rows;
  batch.max_pages = b->max_pages;
  return TACTKV_OK;
}

tactkv_status check_workspace(void* workspace, size_t have, size_t need) {
  return !workspace || !aligned(workspace, 256) || have < need ? TACTKV_WORKSPACE : TACTKV_OK;
}

tactkv_status check_rows(const void* k, const void* v, int64_t token_stride, int64_t head_stride, uint32_t flags) {
  if (!k || !v || token_stride <= 0) return TACTKV_INVALID_ARG;
  const size_t n = flags & TACTKV_FP32_IO ? 8 : 4;
  if (!aligned(k, n) || !aligned(v, n) || token_stride % 2 || head_stride % 2) return TACTKV_ALIGNMENT;
  return TACTKV_OK;
}

// Rows whose launch would not fit a grid's x dimension.
bool too_many(const Batch& b, long long per_row) { return (long long)b.n_rows * per_row > INT_MAX; }

// Whether (row, head) places of head_dim elements can be written without one meeting another: the outer of the two
// strides passes all that the inner one spans.
bool disjoint(const Cache& c, const Batch& b, int64_t token_stride, int64_t head_stride) {
  const int64_t rows = b.n_rows, heads = c.heads, by_head = head_stride < 0 ? -head_stride : head_stride;
  if (rows == 1 || heads == 1) return (rows == 1 || token_stride >= c.head_dim) && (heads == 1 || by_head >= c.head_dim);
  const bool token_major = by_head < token_stride;
  const int64_t inner = token_major ? by_head : token_stride, outer = token_major ? token_stride : by_head;
  const int64_t n = token_major ? heads : rows;
  return inner >= c.head_dim && inner <= (INT64_MAX - c.head_dim) / n && outer >= (n - 1) * inner + c.head_dim;
}

}  // namespace
}  // namespace text
}  // namespace tactkv

using namespace tactkv;
using namespace tactkv::text;

extern "C" {

size_t tactkv_text_workspace_bytes(const tactkv_text_cache* cache, int n_seqs, int n_rows, int q_heads, int max_rows,
                                   int max_kv_len) {
  Cache c;
  if (check_cache(cache, c) != TACTKV_OK || n_seqs < 0 || n_rows < 0 || q_heads < 0 || max_rows < 0 || max_kv_len < 0)
    return 0;
  return kStatusBytes + (q_heads ? attention_workspace(c.head_dim) : 0);
}

tactkv_status tactkv_text_append(const tactkv_text_cache* cache, const tactkv_text_batch* batch, const void* k,
                                 const void* v, int64_t token_stride, int64_t head_stride, void* k_values,
                                 void* v_values, uint32_t flags, void* workspace, size_t workspace_bytes,
                                 struct CUstream_st* stream) {
  Cache c;
  Batch b;
  tactkv_status st = check(cache, batch, flags, c, b);
  if (st == TACTKV_OK) st = check_workspace(workspace, workspace_bytes, kStatusBytes);
  if (st != TACTKV_OK || !b.n_seqs || !b.n_rows) return st;
  st = check_rows(k, v, token_stride, head_stride, flags);
  if (st != TACTKV_OK) return st;
  if (!k_values != !v_values) return TACTKV_INVALID_ARG;
  if (!aligned(k_values, 16) || !aligned(v_values, 16)) return TACTKV_ALIGNMENT;
  if (too_many(b, (c.heads * c.head_dim + 255) / 256)) return TACTKV_UNSUPPORTED_SHAPE;
  return launch_append(cache->format, flags & TACTKV_FP32_IO, c, b, k, v, token_stride, head_stride, k_values, v_values,
                       static_cast<unsigned int*>(workspace), stream) == cudaSuccess ? TACTKV_OK : TACTKV_CUDA;
}

tactkv_status tactkv_text_read(const tactkv_text_cache* cache, const tactkv_text_batch* batch, void* k, void* v,
                               int64_t token_stride, int64_t head_stride, uint32_t flags, void* workspace,
                               size_t workspace_bytes, struct CUstream_st* stream) {
  Cache c;
  Batch b;
  tactkv_status st = check(cache, batch, flags, c, b);
  if (st == TACTKV_OK) st = check_workspace(workspace, workspace_bytes, kStatusBytes);
  if (st != TACTKV_OK || !b.n_seqs || !b.n_rows) return st;
  st = check_rows(k, v, token_stride, head_stride, flags);
  if (st != TACTKV_OK) return st;
  if (too_many(b, (c.heads * c.head_dim + 255) / 256)) return TACTKV_UNSUPPORTED_SHAPE;
  if (!disjoint(c, b, token_stride, head_stride)) return TACTKV_INVALID_ARG;
  return launch_read(cache->format, flags & TACTKV_FP32_IO, c, b, k, v, token_stride, head_stride,
                     static_cast<unsigned int*>(workspace), stream) == cudaSuccess ? TACTKV_OK : TACTKV_CUDA;
}

tactkv_status tactkv_text_attention(const tactkv_text_cache* cache, const tactkv_text_batch* batch, int q_heads,
                                    int max_rows, int max_kv_len, const void* q, int64_t q_token_stride,
                                    int64_t q_head_stride, const uint64_t* tree, const float* prior_out,
                                    const float* prior_m, const float* prior_l, void* out, float* m, float* l,
                                    uint32_t flags, void* workspace, size_t workspace_bytes,
                                    struct CUstream_st* stream) {
  AttnArgs a;
  tactkv_status st = check(cache, batch, flags, a.c, a.b);
  if (st != TACTKV_OK) return st;
  if (q_heads < 1 || max_rows < 1 || max_kv_len < 0) return TACTKV_INVALID_ARG;
  if (max_rows > kMaxRows || max_kv_len > kMaxLen || a.b.n_seqs > 65535 || q_heads % a.c.heads || q_heads / a.c.heads > kMaxGroup)
    return TACTKV_UNSUPPORTED_SHAPE;
  // TMA's coordinates are 32-bit (such a pool would be larger than the GPU's memory)
  if (cache->format == TACTKV_TEXT_BF16 && ((long long)a.c.n_pages * a.c.heads << a.c.page_log2) > INT_MAX)
    return TACTKV_UNSUPPORTED_SHAPE;
  st = check_workspace(workspace, workspace_bytes,
                       tactkv_text_workspace_bytes(cache, a.b.n_seqs, a.b.n_rows, q_heads, max_rows, max_kv_len));
  if (st != TACTKV_OK || !a.b.n_seqs || !a.b.n_rows) return st;
  if (!q || !out || !m || !l || !prior_out != !prior_m || !prior_out != !prior_l) return TACTKV_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(m, 4) || !aligned(l, 4) || !aligned(tree, 8) ||
      !aligned(prior_out, 16) || !aligned(prior_m, 4) || !aligned(prior_l, 4) || q_token_stride % 8 || q_head_stride % 8)
    return TACTKV_ALIGNMENT;
  if (too_many(a.b, q_heads) || a.c.heads > 65535 / kMaxRows) return TACTKV_UNSUPPORTED_SHAPE;
  a.q_heads = q_heads;
  a.max_rows = max_rows;
  a.max_len = max_kv_len;
  a.q = q;
  a.q_token = q_token_stride;
  a.q_head = q_head_stride;
  a.tree = reinterpret_cast<const unsigned long long*>(tree);
  a.prior_out = prior_out;
  a.prior_m = prior_m;
  a.prior_l = prior_l;
  a.out = out;
  a.m = m;
  a.l = l;
  a.status = static_cast<unsigned int*>(workspace);
  return launch_attention(cache->format, flags & TACTKV_FP32_IO, a, static_cast<unsigned char*>(workspace) + kStatusBytes,
                          stream) == cudaSuccess ? TACTKV_OK : TACTKV_CUDA;
}

}  // extern "C"

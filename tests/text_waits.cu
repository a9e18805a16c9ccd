// The text attention's tcgen05 kernel with a limit of its own for the waits that may give up, for test_gpu_text_waits.py.
// The waits that keep a block alive until its copies and products have ended are as they always are.
#include <cstdint>

__device__ uint32_t text_waits_polls = 1u << 16;
#define TACTKV_TEXT_POLLS text_waits_polls
#include "text_tc.cu"

using namespace tactkv::text;

#define NAME_(x, y) x##y
#define NAME(x, y) NAME_(x, y)

// One call on sequences that are not split (1 if they would be); q, out [rows][q_heads][head_dim] bfloat16.
extern "C" int text_waits_run(uint32_t polls, const tactkv_text_cache* c, const tactkv_text_batch* b, int q_heads, int max_rows,
                              int max_len, const void* q, void* out, float* m, float* l, unsigned int* status) {
  if (cudaError_t e = cudaMemcpyToSymbol(text_waits_polls, &polls, sizeof(polls))) return 100 + e;
  AttnArgs a = {};
  a.c.pages[0] = static_cast<unsigned char*>(c->k_pages);
  a.c.pages[1] = static_cast<unsigned char*>(c->v_pages);
  a.c.scales[0] = static_cast<unsigned char*>(c->k_scales);
  a.c.scales[1] = static_cast<unsigned char*>(c->v_scales);
  a.c.n_pages = c->n_pages;
  a.c.heads = c->heads;
  a.c.head_dim = c->head_dim;
  while ((1 << a.c.page_log2) < c->page_tokens) ++a.c.page_log2;
  a.b = {b->page_table, b->kv_lens, b->row_starts, b->n_seqs, b->n_rows, b->max_pages};
  a.q_heads = q_heads, a.max_rows = max_rows, a.max_len = max_len;
  a.q = q, a.q_token = (long long)q_heads * c->head_dim, a.q_head = c->head_dim;
  a.out = out, a.m = m, a.l = l, a.status = status;
  Parts p = {};
  const int rows = max_rows * (q_heads / c->heads), tile = rows <= 16 ? 16 : (rows <= 32 || c->head_dim > kWideDim ? 32 : 64);
  plan(a, tile, 2 * kSms, 256, p);
  if (p.count != 1) return 1;
  if (cudaError_t e = NAME(tactkv::text::launch_tc_, TACTKV_TEXT_D)(c->format, a, p, 0)) return 100 + e;
  return cudaDeviceSynchronize() == cudaSuccess ? 0 : 2;
}

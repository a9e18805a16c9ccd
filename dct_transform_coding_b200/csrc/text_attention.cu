// Attention of a sequence's newest rows over its text cache (include/tactkv.h, tactkv_text_attention):
//   s_t = q . K[t] / sqrt(D) for the tokens t that the row sees,  m = max s_t,  l = sum exp(s_t - m),
//   out = (sum exp(s_t - m) V[t]) / l,  in one pass over the tokens with a running maximum and sum.
#include <climits>

#include "text.cuh"

namespace tactkv {
namespace text {
namespace {

constexpr int kWarps = 4;

// One warp per (row, query head); a lane has head_dim / 32 of the values, eight neighbouring ones of a lane's
// at a time.
template <int FMT, bool F32>
__global__ void __launch_bounds__(kWarps * 32) attention_kernel(const AttnArgs a) {
  const int D = a.c.head_dim, lane = threadIdx.x & 31;
  const long long item = (long long)blockIdx.x * kWarps + threadIdx.x / 32;
  const int row = (int)(item / a.q_heads), j = (int)(item % a.q_heads);
  if (row >= a.b.n_rows) return;
  const int s = find_seq(a.b, row);
  if (s >= a.b.n_seqs) return;
  const Span p = span_of(a.b, a.c.page_log2, s, a.max_len, a.max_rows);
  const int me = row - p.first;
  const bool ok = p.ok && me >= 0 && me < p.rows;
  if (!ok && lane == 0) report(a.status);
  const int head = j / (a.q_heads / a.c.heads);
  const bool mine = lane * 8 < D;
  const int d = mine ? lane * 8 : 0;
  float q[8], o[8] = {};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const long long at = row * a.q_token + j * a.q_head + d + i;
    q[i] = !mine ? 0.f
           : F32 ? static_cast<const float*>(a.q)[at]
                 : __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[at]);
  }
  float m = -INFINITY, l = 0.f;
  const unsigned long long word = ok && a.tree ? a.tree[row] : (me >= 63 ? ~0ull : (2ull << me) - 1);
  const float scale = rsqrtf((float)D);
  const int before = p.len - p.rows;
  for (int t = 0; ok && t < p.len; ++t) {
    if (t >= before && !(word >> (t - before) & 1)) continue;
    const int page = __ldg(a.b.table + (long long)s * a.b.max_pages + (t >> a.c.page_log2));
    if (page < 0 || page >= a.c.n_pages) {
      if (lane == 0) report(a.status);
      continue;
    }
    const long long at = (((long long)page * a.c.heads + head) << a.c.page_log2) + (t & ((1 << a.c.page_log2) - 1));
    float x[2][8];
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      uint32_t w[4] = {}, sc = 0;
      const unsigned char* src = a.c.pages[kv] + (at * D + d) * code_bits(FMT) / 8;
#pragma unroll
      for (int i = 0; i < code_bits(FMT) / 4; ++i) w[i] = reinterpret_cast<const uint32_t*>(src)[i];
      if constexpr (FMT != kBf16) sc = a.c.scales[kv][at * (D / kGroup) + d / kGroup];
      decode8<FMT>(w, sc, x[kv]);
    }
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) z = mine ? fmaf(q[i], x[0][i], z) : 0.f;
#pragma unroll
    for (int i = 16; i; i >>= 1) z += __shfl_xor_sync(~0u, z, i);
    z *= scale;
    const float top = fmaxf(m, z);
    const float keep = top == -INFINITY ? 1.f : __expf(m - top), w = top == -INFINITY ? 0.f : __expf(z - top);
    l = l * keep + w;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = o[i] * keep + w * x[1][i];
    m = top;
  }
  const long long at = (long long)row * a.q_heads + j;
  if (a.prior_out) {
    const float pm = a.prior_m[at], pl = a.prior_l[at], top = fmaxf(m, pm);
    const float x = m == -INFINITY ? 0.f : __expf(m - top), y = pm == -INFINITY ? 0.f : __expf(pm - top) * pl;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = o[i] * x + (y != 0.f ? a.prior_out[at * D + d + i] * y : 0.f);
    l = l * x + y;
    m = top;
  }
  if (mine) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float y = l == 0.f ? 0.f : o[i] / l;
      if constexpr (F32) static_cast<float*>(a.out)[at * D + d + i] = y;
      else static_cast<__nv_bfloat16*>(a.out)[at * D + d + i] = __float2bfloat16_rn(y);
    }
  }
  if (lane == 0) a.m[at] = m, a.l[at] = l;
}

}  // namespace

cudaError_t launch_attention(int fmt, bool f32, const AttnArgs& a, cudaStream_t st) {
  const unsigned blocks = (unsigned)(((long long)a.b.n_rows * a.q_heads + kWarps - 1) / kWarps);
  if (fmt == kBf16) f32 ? attention_kernel<kBf16, true><<<blocks, kWarps * 32, 0, st>>>(a)
                        : attention_kernel<kBf16, false><<<blocks, kWarps * 32, 0, st>>>(a);
  else if (fmt == kFp8) f32 ? attention_kernel<kFp8, true><<<blocks, kWarps * 32, 0, st>>>(a)
                            : attention_kernel<kFp8, false><<<blocks, kWarps * 32, 0, st>>>(a);
  else f32 ? attention_kernel<kFp4, true><<<blocks, kWarps * 32, 0, st>>>(a)
           : attention_kernel<kFp4, false><<<blocks, kWarps * 32, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace text
}  // namespace tactkv

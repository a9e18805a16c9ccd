// Attention over the text cache: the launch plan, and the sum over a sequence's parts.
#include "text_attention.cuh"

namespace tactkv {
namespace text {

#define TACTKV_FOR_D(X) X(32) X(64) X(96) X(128) X(160) X(192) X(224) X(256)
#define TACTKV_DECL(D) cudaError_t launch_parts_##D(int, bool, const AttnArgs&, const Parts&, cudaStream_t);
TACTKV_FOR_D(TACTKV_DECL)
#undef TACTKV_DECL
#define TACTKV_DECL(D) cudaError_t launch_tc_##D(int, const AttnArgs&, Parts&, cudaStream_t);
TACTKV_DECL(64) TACTKV_DECL(128) TACTKV_DECL(192) TACTKV_DECL(256)
#undef TACTKV_DECL

namespace {

constexpr int kThreads = 128;

// out, m and l of one (row, query head): its parts' sums, each to the largest maximum, in the parts' order.
//   m = max m_i,  l = sum l_i 2^(m_i - m),  out = sum o_i 2^(m_i - m - kBase) / l
// A block takes one row; its threads take four columns each and every n-th part.  A read of the workspace, which is still in
// the L2, bound by its latency: about 2 us of a call.  Its launch overlaps the end of the parts' kernel (1000 tokens, 4 heads
// x 128, 8 bits: 12.0 against 12.6 us).
template <bool F32>
__global__ void __launch_bounds__(kThreads) combine_kernel(const AttnArgs a, const Parts p) {
  __shared__ float4 sum[kThreads];
  __shared__ float part_l[kThreads];
  wait_for_previous();
  const int D = a.c.head_dim, G = a.q_heads / a.c.heads;
  const int unit = blockIdx.y, tile = unit % p.tiles, head = unit / p.tiles % a.c.heads, seq = unit / p.tiles / a.c.heads;
  const Span sp = span_of(a.b, a.c.page_log2, seq, a.max_len, a.max_rows);
  const int row = tile * p.tile_rows + blockIdx.x;
  if (!sp.ok || row >= sp.rows * G) return;
  const int n = max(1, (sp.len + p.tokens - 1) / p.tokens);
  const long long stride = (long long)gridDim.y * p.tile_rows, at = (long long)unit * p.tile_rows + blockIdx.x;
  const int cols = D / 4, groups = kThreads / cols, g = threadIdx.x / cols, d = threadIdx.x % cols * 4;
  float m = -INFINITY;
  for (int i = threadIdx.x & 31; i < n; i += 32) m = max_nan(m, p.ml[i * stride + at].x);
#pragma unroll
  for (int x = 16; x; x >>= 1) m = max_nan(m, __shfl_xor_sync(~0u, m, x));
  const float safe = m == -INFINITY ? 0.f : m;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f;
  if (g < groups) {
#pragma unroll 4
    for (int i = g; i < n; i += groups) {
      const float2 ml = p.ml[i * stride + at];
      const float4 x = *reinterpret_cast<const float4*>(p.o + (i * stride + at) * D + d);
      const float f = exp2f(ml.x - safe);
      l += ml.y * f;
      v.x += x.x * f, v.y += x.y * f, v.z += x.z * f, v.w += x.w * f;
    }
  }
  sum[threadIdx.x] = v;
  part_l[threadIdx.x] = l;
  __syncthreads();
  if (g) return;
  for (int i = 1; i < groups; ++i) {
    const float4 x = sum[i * cols + threadIdx.x];
    l += part_l[i * cols + threadIdx.x];
    v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
  }
  finish4<F32>(a, (long long)(sp.first + row / G) * a.q_heads + head * G + row % G, d, v, m, l);
}

}  // namespace

size_t attention_workspace(int head_dim) {
  return (size_t)kMaxParts * kPartRows(head_dim) * (head_dim * sizeof(float) + sizeof(float2));
}

cudaError_t launch_attention(int fmt, bool f32, const AttnArgs& a, void* workspace, cudaStream_t st) {
  const int D = a.c.head_dim, rows = a.max_rows * (a.q_heads / a.c.heads);
  Parts p;
  p.o = static_cast<float*>(workspace);
  p.ml = reinterpret_cast<float2*>(p.o + (size_t)kMaxParts * kPartRows(D) * D);
  cudaError_t e = cudaErrorInvalidValue;
  if (!f32 && D % 64 == 0 && a.max_len > kOneTile) {
    switch (D) {
#define TACTKV_CASE(D) case D: e = launch_tc_##D(fmt, a, p, st); break;
      TACTKV_CASE(64) TACTKV_CASE(128) TACTKV_CASE(192) TACTKV_CASE(256)
#undef TACTKV_CASE
    }
  } else {
    // 16 sequences x 4 heads x 128 x 6000 tokens, float32 queries: 4 rows take 66 us in tiles of 8, 79 of 16 and 106 of 32
    // (8 bits: 42, 73, 92); 12 rows 115 in two of 8, 79 in one of 16 (8 bits: 75, 74).
    plan(a, rows <= 8 ? 8 : (rows <= 16 || !wide_tiles(fmt, f32, D) ? 16 : 32), kMaxParts, kShortPart, p);
    switch (D) {
#define TACTKV_CASE(D) case D: e = launch_parts_##D(fmt, f32, a, p, st); break;
      TACTKV_FOR_D(TACTKV_CASE)
#undef TACTKV_CASE
    }
  }
  if (e != cudaSuccess || p.count == 1) return e;
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.tile_rows, a.b.n_seqs * a.c.heads * p.tiles);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return f32 ? cudaLaunchKernelEx(&cfg, combine_kernel<true>, a, p) : cudaLaunchKernelEx(&cfg, combine_kernel<false>, a, p);
}

}  // namespace text
}  // namespace tactkv

// Attention over the text cache: the launch plan, and the sum over a sequence's parts.
#include <cstdlib>

#include "text_attention.cuh"

namespace tactkv {
namespace text {

#define TACTKV_FOR_D(X) X(32) X(64) X(96) X(128) X(160) X(192) X(224) X(256)
#define TACTKV_DECL(D) cudaError_t launch_parts_##D(int, bool, const AttnArgs&, const Parts&, cudaStream_t);
TACTKV_FOR_D(TACTKV_DECL)
#undef TACTKV_DECL
#define TACTKV_DECL(D) cudaError_t launch_tc_##D(int, const AttnArgs&, const Flat&, int, cudaStream_t);
TACTKV_DECL(64) TACTKV_DECL(128) TACTKV_DECL(192) TACTKV_DECL(256)
#undef TACTKV_DECL

namespace {

constexpr int kThreads = 128;

// out, m and l of (row, query head) number `at`: the sums of n parts, each to the largest maximum, in the parts' order.
// part(i): the place of part i.
template <bool F32, class F>
__device__ __forceinline__ void sum_parts(const AttnArgs& a, const float* o, const float2* ml, int n, long long at, F part) {
  __shared__ float4 sum[kThreads];
  __shared__ float part_l[kThreads];
  const int D = a.c.head_dim, cols = D / 4, groups = kThreads / cols, g = threadIdx.x / cols, d = threadIdx.x % cols * 4;
  float m = -INFINITY;
  for (int i = threadIdx.x & 31; i < n; i += 32) m = fmaxf(m, ml[part(i)].x);
#pragma unroll
  for (int x = 16; x; x >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, x));
  const float safe = m == -INFINITY ? 0.f : m;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f;
  if (g < groups) {
#pragma unroll 4
    for (int i = g; i < n; i += groups) {
      const float2 x = ml[part(i)];
      const float4 y = *reinterpret_cast<const float4*>(o + part(i) * D + d);
      const float f = exp2f(x.x - safe);
      l += x.y * f;
      v.x += y.x * f, v.y += y.y * f, v.z += y.z * f, v.w += y.w * f;
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
  finish4<F32>(a, at, d, v, m, l);
}

template <bool F32>
__global__ void __launch_bounds__(kThreads) combine_kernel(const AttnArgs a, const Parts p) {
  const int G = a.q_heads / a.c.heads;
  const int unit = blockIdx.y, tile = unit % p.tiles, head = unit / p.tiles % a.c.heads, seq = unit / p.tiles / a.c.heads;
  const Span sp = span_of(a.b, a.c.page_log2, seq, a.max_len, a.max_rows);
  const int row = tile * p.tile_rows + blockIdx.x;
  if (!sp.ok || row >= sp.rows * G) return;
  const int n = max(1, (sp.len + p.tokens - 1) / p.tokens);
  const long long stride = (long long)gridDim.y * p.tile_rows, at = (long long)unit * p.tile_rows + blockIdx.x;
  sum_parts<F32>(a, p.o, p.ml, n, (long long)(sp.first + row / G) * a.q_heads + head * G + row % G,
                 [&](int i) { return i * stride + at; });
}

// Block (x, y): the unit across the border between blocks x and x + 1 of the list of work, if that is the unit's first
// border; its row y.
__global__ void __launch_bounds__(kThreads) flat_combine_kernel(const AttnArgs a, const Flat f) {
  const int blocks = gridDim.x + 1, G = a.q_heads / a.c.heads;
  Piece piece;
  const long long entries = find_entry(a, f.rows, false, -1, &piece);
  const long long share = max((entries + blocks - 1) / blocks, (long long)kLeastShare), border = (blockIdx.x + 1) * share;
  if (border >= entries) return;
  find_entry(a, f.rows, false, border, &piece);
  const long long from = border - piece.first, to = from + piece.of;
  if (piece.first == 0 || from < border - share) return;
  const int row = piece.tile * f.rows + blockIdx.y;
  if (row >= piece.sp.rows * G) return;
  const int n = (int)((to - 1) / share) - blockIdx.x + 1;
  // the unit is the first piece of every block but the one it begins in, unless it begins with that block
  const long long begin = 2 * blockIdx.x + (from > border - share);
  sum_parts<false>(a, f.o, f.ml, n, (long long)(piece.sp.first + row / G) * a.q_heads + piece.head * G + row % G,
                   [&](int i) { return (i ? 2ll * (blockIdx.x + i) : begin) * f.rows + blockIdx.y; });
}

}  // namespace

cudaError_t launch_flat_combine(const AttnArgs& a, const Flat& f, int blocks, cudaStream_t st) {
  flat_combine_kernel<<<dim3(blocks - 1, f.rows), kThreads, 0, st>>>(a, f);
  return cudaGetLastError();
}

size_t attention_workspace(int head_dim) {
  return (size_t)kMaxParts * kPartRows(head_dim) * (head_dim * sizeof(float) + sizeof(float2));
}

cudaError_t launch_attention(int fmt, bool f32, const AttnArgs& a, void* workspace, cudaStream_t st) {
  const int D = a.c.head_dim, rows = a.max_rows * (a.q_heads / a.c.heads);
  float* o = static_cast<float*>(workspace);
  float2* ml = reinterpret_cast<float2*>(o + (size_t)kMaxParts * kPartRows(D) * D);
  cudaError_t e = cudaErrorInvalidValue;
  if (!f32 && D % 64 == 0 && !getenv("NOTC")) {
    const Flat f = {0, false, o, ml};
    switch (D) {
#define TACTKV_CASE(D) case D: e = launch_tc_##D(fmt, a, f, rows, st); break;
      TACTKV_CASE(64) TACTKV_CASE(128) TACTKV_CASE(192) TACTKV_CASE(256)
#undef TACTKV_CASE
    }
    return e;
  }
  Parts p;
  p.tile_rows = rows <= 8 ? 8 : (rows <= 16 || D > kWideDim ? 16 : 32);
  p.tiles = (rows + p.tile_rows - 1) / p.tile_rows;
  const long long units = (long long)a.b.n_seqs * a.c.heads * p.tiles;
  const long long most = (a.max_len + kLeastPart - 1) / kLeastPart;
  p.count = (int)std::max(1ll, std::min(most, kMaxParts / units));
  p.tokens = std::max(kLeastPart, ((a.max_len + p.count - 1) / p.count + 63) / 64 * 64);
  p.count = std::max(1, (a.max_len + p.tokens - 1) / p.tokens);
  p.o = o;
  p.ml = ml;
  switch (D) {
#define TACTKV_CASE(D) case D: e = launch_parts_##D(fmt, f32, a, p, st); break;
    TACTKV_FOR_D(TACTKV_CASE)
#undef TACTKV_CASE
  }
  if (e != cudaSuccess || p.count == 1) return e;
  const dim3 grid(p.tile_rows, (unsigned)units);
  if (f32) combine_kernel<true><<<grid, kThreads, 0, st>>>(a, p);
  else combine_kernel<false><<<grid, kThreads, 0, st>>>(a, p);
  return cudaGetLastError();
}

}  // namespace text
}  // namespace tactkv

// Attention over the text cache: what its kernels share (internal header).
//
// A launch splits every sequence into parts of Parts::tokens tokens (one part when the rows alone fill the GPU: 32 sequences x
// 8 heads and 4 x 8 x 8 tiles of 64 rows both took longer in two parts than in one);
// a part's (m, l, sum) goes to the workspace and the parts are summed by combine_kernel in their order,
// so results do not depend on timing.  Scores are held as log2: z = s * log2(e).
#pragma once

#include <algorithm>
#include <climits>

#include "text.cuh"

namespace tactkv {
namespace text {

constexpr int kSms = 148;
constexpr int kMaxParts = 4 * kSms;              // units times parts, where there is more than one part
constexpr int kLeastPart = 256, kShortPart = 128, kFewParts = 16;   // tokens of a part; see plan()
constexpr int kWideDim = 128;      // up to this head_dim a unit may have twice the rows (registers, columns for their sums)

constexpr int kPartRows(int D) { return D <= kWideDim ? 64 : 32; }

// Whether text_attention.cu has tiles of 32 rows.  16 sequences x 4 heads x 6000 tokens, 32 rows in two tiles of 16 against
// one of 32: float32 queries, head_dim 128 148 against 111 us (bfloat16 cache), 140 against 97 (8 bits); bfloat16 queries on
// coded caches, head_dim 32 42 against 28, but 96 75 against 79 (4 bits), and 128 rows 133 against 142.
__host__ __device__ constexpr bool wide_tiles(int fmt, bool f32, int D) {
  return D <= kWideDim && (f32 || fmt == kBf16 || D == 32);
}

// Up to one tile of text_tc.cu's the kernel of text_attention.cu is used: its start is shorter (100 tokens, 4 heads x 128, 8
// bits: 7.8 against 9.6 us, bfloat16 6.8 against 7.6).  At 256 tokens 8 bits take 10.0 and 9.9, bfloat16 9.2 and 8.2,
// and with more rows or tokens it falls behind (32 sequences x 8 heads x 6001 tokens, 24 rows, 4 bits: 269 against 116).
constexpr int kOneTile = 128;

// A unit is (sequence, K/V head, tile of tile_rows rows), numbered in that order.
struct Parts {
  int tile_rows;       // 8, 16, 32 or 64
  int tiles;           // for max_rows * G rows
  int tokens;          // per part, a multiple of 128
  int count;           // parts of the longest sequence
  float* o;            // [count][unit][tile_rows][D] sums of exp2(z - m) V, times 2^kBase
  float2* ml;          // [count][unit][tile_rows] m (log2), l
};

// Probabilities are held times 2^kBase until a row's end, relative to a maximum that may be kSlack below the true one, so as
// at most 2^-8: float32 sums of any 256 tokens stay finite for all that bfloat16 holds, of 2^16 tokens for |V| up to 2^120,
// of 2^30 up to 2^106.  (At 2^6 one dominant token's V of 2^114 reached infinity.)  The price is at the other end: products
// below 2^-126 lose bits, so those of |V| below 2^-102 and p below 2^-8.
constexpr float kBase = -16.f, kSlack = 8.f;
constexpr float kUnbase = 65536.f;   // 2^-kBase

constexpr double root(double x) {                // by Newton's iteration, at compile time
  double y = x;
  for (int i = 0; i < 40; ++i) y = 0.5 * (y + x / y);
  return y;
}
// log2(e) / sqrt(D), rounded once
constexpr float to_log2(int d) { return (float)(1.4426950408889634074 / root(d)); }

__device__ __forceinline__ float exp2_fast(float x) {   // 2 ulp; 0 for -inf
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {   // NaN if either is
  float y;
  asm("max.NaN.f32 %0, %1, %2;\n" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
// Rounded towards zero: never an infinity, and three such terms hold every bit of a float32.
__device__ __forceinline__ uint32_t pack_bf16x2_rz(float a, float b) {
  uint32_t y;
  asm("cvt.rz.bf16x2.f32 %0, %1, %2;\n" : "=r"(y) : "f"(b), "f"(a));
  return y;
}
// A pair of E4M3 codes (bits 0-15, or 16-31) as half precision, exactly.
__device__ __forceinline__ void unpack_e4m3x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n.reg .b16 a, b;\nmov.b32 {a, b}, %2;\ncvt.rn.f16x2.e4m3x2 %0, a;\ncvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
// Two half-precision values (codes) times their scales, as bfloat16: exact in its range.
__device__ __forceinline__ uint32_t scaled_bf16x2(uint32_t h, float f, float g) {
  const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return pack_bf16x2(v.x * f, v.y * g);
}
// Any infinity or NaN among two packed bfloat16 values.
__device__ __forceinline__ bool odd2(uint32_t v) { return (v & 0x7F80u) == 0x7F80u || (v >> 16 & 0x7F80u) == 0x7F80u; }

constexpr float kLn2 = 0.69314718055994531f;

// A row's end: out = a * (the text tokens' sum, times 2^kBase) + b * prior_out.
struct RowEnd {
  float a, b;
};
// Of (row, head) number `at`, from the text tokens' maximum m2 (log2) and l, merged with the prior; write: m and l, too.
// A row that sees nothing has l = 0: out = 0, m = -inf.  One with a score of +inf or NaN has that as m2, and l and out are NaN.
__device__ __forceinline__ RowEnd end_row(const AttnArgs& a, long long at, float m2, float l, bool write) {
  float m = m2 * kLn2, x = 1.f, y = 0.f;
  if (a.prior_out) {
    const float pm = a.prior_m[at], pl = a.prior_l[at];
    const float top = max_nan(m, pm), safe = top == -INFINITY ? 0.f : top;
    x = expf(m - safe), y = expf(pm - safe) * pl;
    l = l * x + y;
    m = top;
  }
  if (write) a.m[at] = m, a.l[at] = l;
  return l == 0.f ? RowEnd{0.f, 0.f} : RowEnd{x / l * kUnbase, y == 0.f ? 0.f : y / l};   // b = 0 without a prior, l a NaN or not
}
// Columns d .. d+3 of a row with the sum o.
template <bool F32>
__device__ __forceinline__ void finish4(const AttnArgs& a, long long at, int d, float4 o, RowEnd e) {
  const int D = a.c.head_dim;
  o.x *= e.a, o.y *= e.a, o.z *= e.a, o.w *= e.a;
  if (e.b != 0.f) {   // what a prior of weight 0 holds does not matter
    const float4 p = *reinterpret_cast<const float4*>(a.prior_out + at * D + d);
    o.x += p.x * e.b, o.y += p.y * e.b, o.z += p.z * e.b, o.w += p.w * e.b;
  }
  if constexpr (F32)
    *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at * D + d) = o;
  else
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + at * D + d) =
        make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
}
template <bool F32>
__device__ __forceinline__ void finish4(const AttnArgs& a, long long at, int d, float4 o, float m2, float l) {
  finish4<F32>(a, at, d, o, end_row(a, at, m2, l, d == 0));
}

// The rows of a sequence whose numbers do not fit together see no text token.
template <bool F32, int D>
__device__ __forceinline__ void finish_misfit(const AttnArgs& a, const Span& sp, int seq, int head, int G) {
  if (threadIdx.x == 0) report(a.status);
  const int end = __ldg(a.b.row_starts + seq + 1);
  if (sp.first < 0 || end > a.b.n_rows) return;
  for (int row = sp.first; row < end; ++row)
    for (int i = threadIdx.x; i < G * (D / 4); i += blockDim.x)
      finish4<F32>(a, (long long)row * a.q_heads + head * G + i / (D / 4), i % (D / 4) * 4, make_float4(0.f, 0.f, 0.f, 0.f),
                   -INFINITY, 0.f);
}

// The combining kernel may start, and wait for this one, while this block ends.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }

// The split of a launch into at most `blocks` blocks, and each sequence into parts, which have at least kLeastPart tokens:
// with half of that the sum over more parts costs more than it gains (4000 tokens x 4 heads x 128, tcgen05: bfloat16 12.3
// against 11.7 us, 8 bits 14.0 against 13.5; on the other kernel, head_dim 96, it gains: 12.3 against 14.4).  kShortPart is
// used where it makes few parts (kFewParts) and no SM gets two: 1000 tokens 9.5 against 10.1 us, 8 bits 12.0 against 12.6
// and, on the other kernel, 10.4 against 13.2 (head_dim 96) and 16.3 against 24.5 (float32, head_dim 256, 700 tokens).  Sequences
// of up to `whole` tokens are not split.
inline void plan(const AttnArgs& a, int tile_rows, int blocks, int whole, Parts& p) {
  p.tile_rows = tile_rows;
  p.tiles = (a.max_rows * (a.q_heads / a.c.heads) + tile_rows - 1) / tile_rows;
  const long long units = (long long)a.b.n_seqs * a.c.heads * p.tiles, most = (a.max_len + kShortPart - 1) / kShortPart;
  const bool shorts = a.max_len > whole && most <= kFewParts && units * most <= kSms;
  const int least = shorts ? kShortPart : kLeastPart;
  p.count = (int)std::max(1ll, std::min<long long>((a.max_len + least - 1) / least, blocks / units));
  p.tokens = std::max(least, ((a.max_len + p.count - 1) / p.count + 127) / 128 * 128);
  p.count = std::max(1, (a.max_len + p.tokens - 1) / p.tokens);
}

}  // namespace text
}  // namespace tactkv

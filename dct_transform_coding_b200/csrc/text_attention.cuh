// Attention over the text cache: what its kernels share (internal header).
//
// A launch splits every sequence into parts of `part` tokens (one part when the rows alone fill the GPU);
// a part's (m, l, sum) goes to the workspace and the parts are summed by combine_kernel in their order,
// so results do not depend on timing.  Scores are held as log2: z = s * log2(e).
#pragma once

#include <algorithm>
#include <climits>

#include "text.cuh"

namespace tactkv {
namespace text {

constexpr int kMaxParts = 4 * 148; // units times parts, where there is more than one part
constexpr int kLeastPart = 256;    // tokens
constexpr int kWideDim = 128;      // up to this head_dim a unit may have 32 rows (registers for their sums)

// A unit is (sequence, K/V head, tile of tile_rows rows), numbered in that order.
struct Parts {
  int tile_rows;       // 8, 16 or 32
  int tiles;           // for max_rows * G rows
  int tokens;          // per part, a multiple of 64
  int count;           // parts of the longest sequence
  float* o;            // [count][unit][tile_rows][D] sums of exp2(z - m) V
  float2* ml;          // [count][unit][tile_rows] m (log2), l
};

constexpr float kLn2 = 0.69314718055994531f;

// out, m, l of (row, head) number `at` from the text tokens' sum o of columns d .. d+3, their maximum m2 (log2)
// and l, merged with the prior.  A row that sees nothing has l = 0: out = 0, m = -inf.
template <bool F32>
__device__ __forceinline__ void finish4(const AttnArgs& a, long long at, int d, float4 o, float m2, float l) {
  const int D = a.c.head_dim;
  float m = l == l ? m2 * kLn2 : l;
  if (a.prior_out) {
    const float pm = a.prior_m[at], pl = a.prior_l[at];
    const float4 p = *reinterpret_cast<const float4*>(a.prior_out + at * D + d);
    const float top = fmaxf(m, pm), safe = top == -INFINITY ? 0.f : top;
    const float x = expf(m - safe), y = expf(pm - safe) * pl;
    o.x *= x, o.y *= x, o.z *= x, o.w *= x;
    if (pl != 0.f) o.x += p.x * y, o.y += p.y * y, o.z += p.z * y, o.w += p.w * y;
    l = l * x + y;
    m = l == l ? top : l;
  }
  const float f = l == 0.f ? 0.f : 1.f / l;
  if (l == 0.f) o = make_float4(0.f, 0.f, 0.f, 0.f);
  if constexpr (F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at * D + d) = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
  } else {
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + at * D + d) =
        make_uint2(pack_bf16x2(o.x * f, o.y * f), pack_bf16x2(o.z * f, o.w * f));
  }
  if (d == 0) a.m[at] = m, a.l[at] = l;
}

}  // namespace text
}  // namespace tactkv

// Attention of a sequence's newest rows over its text cache (include/tactkv.h, tactkv_text_attention),
// for one head_dim (TACTKV_TEXT_D, compiled once for each):
//   s_t = q . K[t] / sqrt(D) over the tokens t that the row sees,  m = max s_t,  l = sum exp(s_t - m),
//   out = (sum exp(s_t - m) V[t]) / l,  in one pass over the tokens with a running maximum and sum.
//
// A CTA has 16 rows (query heads of one K/V head, row = node * G + head within the group) of one sequence
// and one part of its tokens.  Its warps take 16 tokens at a time each and never wait for one another: a
// warp's two m16n8k16 products QK^T and PV take K and V as B fragments, and because the order of the
// summed index is free, the fragment a lane needs is a piece of a row as it lies in the cache.  So each lane
// copies its own pieces (cp.async, 16 bytes where head_dim allows) into a ring in shared memory and reads
// back only those: no transposition and no barrier but the warp's own.
//
// Codes become half precision exactly, scaled by 2^(s - smax) with smax the token's largest scale: in
// K, 2^smax multiplies the token's score; in V it multiplies the token's probability, relative to the largest
// smax so far (ref).  A group whose scale is more than 2^15 below its token's largest loses bits that
// are 2^-24 of the largest.  bfloat16 caches go in as they are.  Queries: bfloat16 ones are exact in
// either type (scaled by a power of two for each row); float32 ones are split into two half-precision or
// three bfloat16 terms, and so are the probabilities then.
#include <atomic>

#include "text_attention.cuh"

#ifndef TACTKV_TEXT_D
#define TACTKV_TEXT_D 128
#endif

namespace tactkv {
namespace text {
namespace {

constexpr int D = TACTKV_TEXT_D;
constexpr int kWarps = 4;
constexpr int kStep = 16;            // tokens a warp takes at a time: never more than a page's
constexpr float kBase = 6.f;         // probabilities are held times 2^6 ..
constexpr float kSlack = 8.f;        // .. relative to a maximum that may be 8 below the true one: at most 2^14

constexpr double root(double x) {                // by Newton's iteration, at compile time
  double y = x;
  for (int i = 0; i < 40; ++i) y = 0.5 * (y + x / y);
  return y;
}
constexpr float kToLog2 = (float)(1.4426950408889634074 / root(D));   // log2(e) / sqrt(D), rounded once

constexpr int vec_bytes(int bytes, int most) {   // the widest power of two that divides a lane's share
  int v = most;
  while (bytes % v) v /= 2;
  return v;
}

template <int FMT, bool F32>
struct Shape {
  static constexpr bool kCoded = FMT != kBf16;
  static constexpr int kRow = D * code_bits(FMT) / 8;
  static constexpr int kKVec = vec_bytes(kRow / 4, 16), kKVecs = kRow / 4 / kKVec;    // a lane's pieces of a K row
  static constexpr int kVVec = vec_bytes(kRow / 8, 16), kVVecs = kRow / 8 / kVVec;    // and of a V row
  static constexpr int kVCopy = kVVec < 4 ? 4 : kVVec;   // two lanes copy the same 4 bytes where a piece is 2
  static constexpr int kKElems = kKVec * 8 / code_bits(FMT), kVElems = kVVec * 8 / code_bits(FMT);
  static constexpr int kKBytes = 2 * kKVecs * 32 * kKVec, kVBytes = 4 * kVVecs * 32 * kVCopy;
  static constexpr int kScaleBytes = kCoded ? D / 2 : 0;                               // of 16 tokens
  static constexpr int kStage = kKBytes + kVBytes + 2 * kScaleBytes;
  static constexpr int kStagesFit = 17920 / kStage;
  static constexpr int kStages = kStagesFit < 3 ? 3 : (kStagesFit > 8 ? 8 : kStagesFit);
  static constexpr int kLimbs = !F32 ? 1 : (kCoded ? 2 : 3);
  static constexpr int kQBytes = kLimbs * (D / 16) * 32 * 16;
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kSum = kWarps * 16 * (D + 4) * 4;          // the warps' sums, over the ring when it is done
  static constexpr int kBody = kRing > kSum ? kRing : kSum;
  static constexpr int kSmem = kQBytes + kBody + kWarps * 16 * 8;
};

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
template <int N>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool there) {
  const int n = there ? N : 0;   // the rest is zeros
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;\n" ::"r"(dst), "l"(src), "n"(N), "r"(n) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory"); }

template <int N>
__device__ __forceinline__ void load_words(const unsigned char* p, uint32_t (&w)[4]) {
  if constexpr (N == 16) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else if constexpr (N == 8) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

template <bool HALF>
__device__ __forceinline__ void mma(float (&c)[4], const uint4& a, uint32_t b0, uint32_t b1) {
  if constexpr (HALF)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float exp2_fast(float x) {   // 2 ulp; 0 for -inf
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
template <bool HALF>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (HALF) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    return pack_bf16x2(a, b);
  }
}
template <bool HALF>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
  if constexpr (HALF) return __half22float2(*reinterpret_cast<const __half2*>(&v));
  else return unpack_bf16x2(v);
}
__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b) {
  uint32_t y;
  asm("mul.rn.f16x2 %0, %1, %2;\n" : "=r"(y) : "r"(a), "r"(b));
  return y;
}
// A pair of E4M3 codes (bits 0-15, or 16-31) as half precision, exactly.
__device__ __forceinline__ void unpack_e4m3x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n.reg .b16 a, b;\nmov.b32 {a, b}, %2;\ncvt.rn.f16x2.e4m3x2 %0, a;\ncvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
// 2^(s - top) in half precision (s <= top), NaN for the NaN scale.
__device__ __forceinline__ uint32_t half_factor(uint32_t s, uint32_t top) {
  const int e = 127 + (int)s - (int)top;
  const float f = s == 255u ? NAN : __uint_as_float((uint32_t)max(e, 0) << 23);
  const __half h = __float2half_rn(f);
  return *reinterpret_cast<const unsigned short*>(&h);
}

// Any infinity or NaN among two packed half-precision or bfloat16 values.
template <bool HALF>
__device__ __forceinline__ bool odd2(uint32_t v) {
  constexpr uint32_t e = HALF ? 0x7C00u : 0x7F80u;
  return (v & e) == e || (v >> 16 & e) == e;
}

template <int FMT, bool F32>
__global__ void __launch_bounds__(kWarps * 32) parts_kernel(const AttnArgs a, const Parts parts) {
  using Sh = Shape<FMT, F32>;
  constexpr bool kHalf = Sh::kCoded;
  constexpr int NT = D / 8;                       // column tiles of the output
  extern __shared__ __align__(16) unsigned char smem[];
  uint4* q_frag = reinterpret_cast<uint4*>(smem);                                 // [limb][D / 16][lane]
  unsigned char* body = smem + Sh::kQBytes;
  float2* sums = reinterpret_cast<float2*>(body + Sh::kBody);                     // [warp][16] (m, l)

  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, r = lane / 4, c = lane & 3;
  const int G = a.q_heads / a.c.heads;
  const int part = blockIdx.x, seq = blockIdx.z, tiles = gridDim.y / a.c.heads;
  const int head = blockIdx.y / tiles, tile = blockIdx.y % tiles;
  const Span sp = span_of(a.b, a.c.page_log2, seq, a.max_len, a.max_rows);
  if (!sp.ok) {                                   // the sequence's rows see no text token
    if (part == 0 && tile == 0) {
      if (threadIdx.x == 0) report(a.status);
      const int end = __ldg(a.b.row_starts + seq + 1);
      if (sp.first < 0 || end > a.b.n_rows) return;
      for (int row = sp.first; row < end; ++row)
        for (int i = threadIdx.x; i < G * (D / 4); i += kWarps * 32)
          finish4<F32>(a, (long long)row * a.q_heads + head * G + i / (D / 4), i % (D / 4) * 4,
                       make_float4(0.f, 0.f, 0.f, 0.f), -INFINITY, 0.f);
    }
    return;
  }
  const int M = sp.rows * G, row0 = tile * kTileRows, before = sp.len - sp.rows;
  const int t0 = part * parts.tokens, t1 = t0 + min(sp.len - t0, parts.tokens);
  if (row0 >= M || (part > 0 && t0 >= sp.len)) return;

  // ---- the queries' A fragments ----
  // Lane (r, c) of K's step k holds elements idx = 4k .. 4k+3 of its share of row r: d = (idx / kKElems * 4
  // + c) * kKElems + idx % kKElems.  Rows are scaled so that their largest element is in [2^14, 2^15).
  float row_factor[2] = {1.f, 1.f};
  {
    const long long base = (long long)sp.first * a.q_token + (long long)head * G * a.q_head;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = row0 + r + 8 * h;
      const bool in = row < M;
      const long long at = base + (in ? (long long)(row / G) * a.q_token + (long long)(row % G) * a.q_head : 0);
      float f = 1.f;
      if constexpr (kHalf) {
        uint32_t top = 0;
        for (int i = c; i < D / 2; i += 4) {
          float2 v;
          if constexpr (F32) v = *reinterpret_cast<const float2*>(static_cast<const float*>(a.q) + at + 2 * i);
          else v = unpack_bf16x2(*reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(a.q) + at + 2 * i));
          top = max(top, max(__float_as_uint(v.x) & 0x7FFFFFFFu, __float_as_uint(v.y) & 0x7FFFFFFFu));
        }
        top = max(top, __shfl_xor_sync(~0u, top, 1));
        top = max(top, __shfl_xor_sync(~0u, top, 2));
        const int E = (int)(top >> 23);                       // biased; f = 2^(14 + 127 - E) within float32's range
        const int e = E == 255 || top == 0 ? 0 : max(-126, min(126, 141 - E));
        f = __uint_as_float((uint32_t)(127 + e) << 23);
        row_factor[h] = __uint_as_float((uint32_t)(127 - e) << 23);
      }
      for (int k = warp; k < D / 16; k += kWarps) {
        float x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int idx = 4 * k + i, d = (idx / Sh::kKElems * 4 + c) * Sh::kKElems + idx % Sh::kKElems;
          x[i] = !in ? 0.f
                 : F32 ? static_cast<const float*>(a.q)[at + d]
                       : __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[at + d]);
          if constexpr (kHalf) x[i] *= f;
        }
#pragma unroll
        for (int n = 0; n < Sh::kLimbs; ++n) {
          const uint32_t lo = pack2<kHalf>(x[0], x[1]), hi = pack2<kHalf>(x[2], x[3]);
          uint32_t* to = reinterpret_cast<uint32_t*>(q_frag + (n * (D / 16) + k) * 32 + lane);
          to[h] = lo, to[2 + h] = hi;
          const float2 u = unpack2<kHalf>(lo), v = unpack2<kHalf>(hi);
          x[0] -= u.x, x[1] -= u.y, x[2] -= v.x, x[3] -= v.y;
        }
      }
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) row_factor[h] *= kToLog2;
  // Which of the sequence's own rows each of the lane's two rows sees.
  unsigned long long word[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int node = min((row0 + r + 8 * h) / G, sp.rows - 1);
    word[h] = a.tree ? a.tree[sp.first + node] : (node >= 63 ? ~0ull : (2ull << node) - 1);
  }
  __syncthreads();

  // ---- the ring ----
  unsigned char* ring = body + warp * (Sh::kStages * Sh::kStage);
  const int first = t0 / kStep + warp, last = (t1 + kStep - 1) / kStep;      // the warp's steps: first, first + kWarps ..
  const int steps = first < last ? (last - first + kWarps - 1) / kWarps : 0;
  // Lane i keeps the page of the warp's step (32 * n + i); -1 where it is out of range.
  auto page_of = [&](int i) {
    int page = -1;
    if (i < steps) {
      page = __ldg(a.b.table + (long long)seq * a.b.max_pages + ((first + i * kWarps) * kStep >> a.c.page_log2));
      if (page < 0 || page >= a.c.n_pages) {
        page = -1;
        report(a.status);
      }
    }
    return page;
  };
  int pages = page_of(lane), pages_next = page_of(32 + lane);
  auto issue = [&](int i, int page) {
    if (i < steps && page >= 0) {
      const int t = (first + i * kWarps) * kStep;
      const long long at = (((long long)page * a.c.heads + head) << a.c.page_log2) + (t & ((1 << a.c.page_log2) - 1));
      const int held = sp.len - t;                                            // tokens of the step that are there
      const uint32_t to = smem_addr(ring + i % Sh::kStages * Sh::kStage);
      const unsigned char* ks = a.c.pages[0] + at * Sh::kRow;
      const unsigned char* vs = a.c.pages[1] + at * Sh::kRow;
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const bool there = 8 * n + r < held;
#pragma unroll
        for (int j = 0; j < Sh::kKVecs; ++j)
          copy_async<Sh::kKVec>(to + ((n * Sh::kKVecs + j) * 32 + lane) * Sh::kKVec,
                                ks + (8 * n + r) * Sh::kRow + (j * 4 + c) * Sh::kKVec, there);
      }
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const int tok = 2 * c + (n & 1) + 8 * (n >> 1);
        const bool there = tok < held;
#pragma unroll
        for (int j = 0; j < Sh::kVVecs; ++j)
          copy_async<Sh::kVCopy>(to + Sh::kKBytes + ((n * Sh::kVVecs + j) * 32 + lane) * Sh::kVCopy,
                                 vs + tok * Sh::kRow + (j * 8 + (Sh::kVVec < 4 ? r & ~1 : r)) * Sh::kVVec, there);
      }
      if constexpr (Sh::kCoded) {
        // 16 tokens' scales are D / 2 neighbouring bytes: lanes 0 .. copy K's, the next ones V's, 16 at a time
        if (lane < D / 16) {
          const int kv = lane >= D / 32, i16 = lane - kv * (D / 32);
          copy_async<16>(to + Sh::kKBytes + Sh::kVBytes + kv * Sh::kScaleBytes + 16 * i16,
                         a.c.scales[kv] + at * (D / kGroup) + 16 * i16, true);
        }
      }
    }
    copy_commit();
  };
#pragma unroll
  for (int i = 0; i < Sh::kStages - 1; ++i) issue(i, __shfl_sync(~0u, pages, i));

  float o[NT][4] = {};
  float m_ref[2] = {-INFINITY, -INFINITY}, m_true[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  int ref = 0;                                   // the largest V scale so far (coded caches)

  for (int i = 0; i < steps; ++i) {
    if (i && i % 32 == 0) pages = pages_next, pages_next = page_of(i + 32 + lane);
    copy_wait<Sh::kStages - 2>();
    __syncwarp();
    {
      const int n = i + Sh::kStages - 1;         // its slot is the one of step i - 1, which every lane has left
      const int pa = __shfl_sync(~0u, pages, n & 31), pb = __shfl_sync(~0u, pages_next, n & 31);
      issue(n, n / 32 == i / 32 ? pa : pb);
    }
    const int page = __shfl_sync(~0u, pages, i & 31);
    if (page < 0) continue;
    const unsigned char* stage = ring + i % Sh::kStages * Sh::kStage;
    const unsigned char* k_scales = stage + Sh::kKBytes + Sh::kVBytes;
    const unsigned char* v_scales = k_scales + Sh::kScaleBytes;
    const int t = (first + i * kWarps) * kStep;

    // Lane x < 16 finds the largest scale of token x in V, lane 16 + x in K (the NaN scale aside).
    uint32_t top = 0;
    if constexpr (Sh::kCoded) {
      const unsigned char* src = (lane < 16 ? v_scales : k_scales) + (lane & 15) * (D / kGroup);
#pragma unroll
      for (int g = 0; g < D / kGroup; ++g) {
        const uint32_t s = src[g];
        top = max(top, s == 255u ? 0u : s);
      }
      if ((lane & 15) >= sp.len - t) top = 0;     // what the page holds behind the last token
    }

    // ---- scores ----
    float z[2][4] = {};
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      float low[4] = {};                         // the queries' lower terms are summed apart: their rounding stays small
      const uint32_t k_top = Sh::kCoded ? __shfl_sync(~0u, top, 16 + 8 * n + r) : 0u;
#pragma unroll
      for (int j = 0; j < Sh::kKVecs; ++j) {
        uint32_t w[4];
        load_words<Sh::kKVec>(stage + ((n * Sh::kKVecs + j) * 32 + lane) * Sh::kKVec, w);
        uint32_t f = 0;
        if constexpr (Sh::kCoded) {
          f = half_factor(k_scales[(8 * n + r) * (D / kGroup) + (j * 4 + c) * Sh::kKElems / kGroup], k_top);
          f |= f << 16;
        }
#pragma unroll
        for (int k = 0; k < Sh::kKElems / 4; ++k) {
          uint32_t b[2];
          if constexpr (FMT == kBf16) {
            b[0] = w[2 * k], b[1] = w[2 * k + 1];
          } else if constexpr (FMT == kFp8) {
            unpack_e4m3x4(w[k], b[0], b[1]);
          } else {
            uint32_t h[4];
            unpack_e2m1x8(w[k / 2], h);
            b[0] = h[k % 2 * 2], b[1] = h[k % 2 * 2 + 1];
          }
          if constexpr (Sh::kCoded) b[0] = mul_half2(b[0], f), b[1] = mul_half2(b[1], f);
#pragma unroll
          for (int x = 0; x < Sh::kLimbs; ++x)
            mma<kHalf>(x ? low : z[n], q_frag[(x * (D / 16) + j * (Sh::kKElems / 4) + k) * 32 + lane], b[0], b[1]);
        }
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) z[n][x] += low[x];
    }
    // z[n][0, 1]: row r, tokens 8n + 2c, 8n + 2c + 1;  z[n][2, 3]: row r + 8
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float f = Sh::kCoded ? scale_value(__shfl_sync(~0u, top, 16 + 8 * n + 2 * c + x)) : 1.f;
        z[n][x] *= f * row_factor[0], z[n][2 + x] *= f * row_factor[1];
      }
    const bool tail = t + kStep > before;
    if (tail) {
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int node = t + 8 * n + 2 * c + x - before;
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (node >= 0 && (node >= sp.rows || !(word[h] >> node & 1))) z[n][2 * h + x] = -INFINITY;
        }
    }

    // ---- running maximum ----
    bool over = false;
    float high[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      high[h] = fmaxf(fmaxf(z[0][2 * h], z[0][2 * h + 1]), fmaxf(z[1][2 * h], z[1][2 * h + 1]));
      m_true[h] = fmaxf(m_true[h], high[h]);
      over |= high[h] > m_ref[h] + kSlack;
    }
    uint32_t new_ref = ref;
    if constexpr (Sh::kCoded) new_ref = max((uint32_t)ref, __reduce_max_sync(~0u, lane < 16 ? top : 0u));
    if (__any_sync(~0u, over) || new_ref != ref) {
      const float down = Sh::kCoded ? __uint_as_float((uint32_t)max(127 + ref - (int)new_ref, 0) << 23) : 1.f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float v = fmaxf(high[h], __shfl_xor_sync(~0u, high[h], 1));
        v = fmaxf(v, __shfl_xor_sync(~0u, v, 2));
        const float next = v > m_ref[h] + kSlack ? v : m_ref[h];
        const float keep = next == -INFINITY ? 1.f : exp2_fast(m_ref[h] - next);
        m_ref[h] = next;
        l[h] *= keep;
#pragma unroll
        for (int n = 0; n < NT; ++n) o[n][2 * h] *= keep * down, o[n][2 * h + 1] *= keep * down;
      }
      ref = new_ref;
    }

    // ---- probabilities: the lane's tokens 2c, 2c + 1, 8 + 2c, 8 + 2c + 1 of rows r and r + 8 ----
    float p[2][4];                                // [h][token]
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float shift = kBase - (m_ref[h] == -INFINITY ? 0.f : m_ref[h]);
#pragma unroll
      for (int n = 0; n < 4; ++n) p[h][n] = exp2_fast(z[n / 2][2 * h + n % 2] + shift);
      l[h] += (p[h][0] + p[h][1]) + (p[h][2] + p[h][3]);
    }
    uint32_t v_top[4];
    if constexpr (Sh::kCoded) {
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        v_top[n] = __shfl_sync(~0u, top, 2 * c + (n & 1) + 8 * (n >> 1));
        const float f = __uint_as_float((uint32_t)max(127 + (int)v_top[n] - ref, 0) << 23);
        p[0][n] *= f, p[1][n] *= f;
      }
    }
    uint4 pa[Sh::kLimbs];
    {
      float x[2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int n = 0; n < 4; ++n) x[h][n] = p[h][n];
#pragma unroll
      for (int n = 0; n < Sh::kLimbs; ++n) {
        pa[n] = make_uint4(pack2<kHalf>(x[0][0], x[0][1]), pack2<kHalf>(x[1][0], x[1][1]),
                           pack2<kHalf>(x[0][2], x[0][3]), pack2<kHalf>(x[1][2], x[1][3]));
        if (n + 1 < Sh::kLimbs) {
          const float2 u0 = unpack2<kHalf>(pa[n].x), u1 = unpack2<kHalf>(pa[n].y), u2 = unpack2<kHalf>(pa[n].z),
                       u3 = unpack2<kHalf>(pa[n].w);
          x[0][0] -= u0.x, x[0][1] -= u0.y, x[1][0] -= u1.x, x[1][1] -= u1.y;
          x[0][2] -= u2.x, x[0][3] -= u2.y, x[1][2] -= u3.x, x[1][3] -= u3.y;
        }
      }
    }

    // ---- sums: column r of tile (j, e) is d = (j * 8 + r) * kVElems + e ----
#pragma unroll
    for (int j = 0; j < Sh::kVVecs; ++j) {
      uint32_t w[4][4], f01 = 0, f23 = 0;
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        load_words<Sh::kVCopy>(stage + Sh::kKBytes + ((n * Sh::kVVecs + j) * 32 + lane) * Sh::kVCopy, w[n]);
        if constexpr (Sh::kVVec < 4) w[n][0] >>= 16 * (r & 1);
      }
      if constexpr (Sh::kCoded) {
        uint32_t f[4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const int tok = 2 * c + (n & 1) + 8 * (n >> 1);
          const uint32_t s = v_scales[tok * (D / kGroup) + (j * 8 + r) * Sh::kVElems / kGroup];
          f[n] = half_factor(tok < sp.len - t ? s : 0u, tok < sp.len - t ? v_top[n] : 0u);
        }
        f01 = f[0] | f[1] << 16, f23 = f[2] | f[3] << 16;
      }
#pragma unroll
      for (int e0 = 0; e0 < Sh::kVElems; e0 += 4) {
        uint32_t b[4][2];                          // [column e0 + i][token pair]
#pragma unroll
        for (int side = 0; side < 2; ++side) {
          const uint32_t* x = w[2 * side];
          const uint32_t* y = w[2 * side + 1];
          if constexpr (FMT == kBf16) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              b[2 * i][side] = __byte_perm(x[e0 / 2 + i], y[e0 / 2 + i], 0x5410);
              b[2 * i + 1][side] = __byte_perm(x[e0 / 2 + i], y[e0 / 2 + i], 0x7632);
            }
          } else if constexpr (FMT == kFp8) {
            const uint32_t u = __byte_perm(x[e0 / 4], y[e0 / 4], 0x5140), v = __byte_perm(x[e0 / 4], y[e0 / 4], 0x7362);
            unpack_e4m3x4(u, b[0][side], b[1][side]);
            unpack_e4m3x4(v, b[2][side], b[3][side]);
          } else {
            // four columns are 16 bits of each token: half bytes x0 x1 x2 x3 and y0 .. become x0 y0 x1 y1 ..
            const uint32_t xs = x[e0 / 8] >> (e0 % 8 * 4) & 0xFFFFu, ys = y[e0 / 8] >> (e0 % 8 * 4) & 0xFFFFu;
            const uint32_t even = (xs & 0x0F0Fu) | (ys & 0x0F0Fu) << 4, odd = (xs >> 4 & 0x0F0Fu) | (ys & 0xF0F0u);
            uint32_t h[4];
            unpack_e2m1x8(even | odd << 16, h);     // bytes: columns 0, 2, 1, 3
            b[0][side] = h[0], b[2][side] = h[1], b[1][side] = h[2], b[3][side] = h[3];
          }
          if constexpr (Sh::kCoded) {
#pragma unroll
            for (int i = 0; i < 4; ++i) b[i][side] = mul_half2(b[i][side], side ? f23 : f01);
          }
        }
        bool odd = false;
        if (tail) {
#pragma unroll
          for (int i = 0; i < 4; ++i) odd |= odd2<kHalf>(b[i][0]) || odd2<kHalf>(b[i][1]);
          odd = __any_sync(~0u, odd);
        }
        if (!odd) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int n = 0; n < Sh::kLimbs; ++n) mma<kHalf>(o[j * Sh::kVElems + e0 + i], pa[n], b[i][0], b[i][1]);
        } else {
          // An infinity or NaN among the drafted tokens' values: only the rows that see it may get it, so
          // the products are summed one by one.  Token (cc, n) of row r, r + 8 is lane (r, cc)'s p[h][n]; its
          // value in column 2c (+ 1) is lane (2c (+ 1), cc)'s.
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll 1
            for (int cc = 0; cc < 4; ++cc)
#pragma unroll
              for (int n = 0; n < 4; ++n) {
                const int tok = 2 * cc + (n & 1) + 8 * (n >> 1), node = t + tok - before;
                const uint32_t u = __shfl_sync(~0u, b[i][n >> 1], 8 * c + cc),
                               v = __shfl_sync(~0u, b[i][n >> 1], 8 * c + 4 + cc);
                const float2 x = unpack2<kHalf>(u), y = unpack2<kHalf>(v);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const float pr = __shfl_sync(~0u, p[h][n], 4 * r + cc);
                  const bool seen = node < 0 || (node < sp.rows && (word[h] >> node & 1));
                  if (seen) {
                    o[j * Sh::kVElems + e0 + i][2 * h] += pr * (n & 1 ? x.y : x.x);
                    o[j * Sh::kVElems + e0 + i][2 * h + 1] += pr * (n & 1 ? y.y : y.x);
                  }
                }
              }
        }
      }
    }
  }
  copy_wait<0>();

  // ---- the warps' sums, to the rows' true maxima ----
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int x = 1; x <= 2; x *= 2) {
      m_true[h] = fmaxf(m_true[h], __shfl_xor_sync(~0u, m_true[h], x));
      l[h] += __shfl_xor_sync(~0u, l[h], x);
    }
  }
  __syncthreads();                                 // the ring is done: its place takes the sums
  float* mine = reinterpret_cast<float*>(body) + warp * 16 * (D + 4);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float to = m_true[h] == -INFINITY ? 0.f : exp2f(m_ref[h] - m_true[h] - kBase);
    const float unit = Sh::kCoded ? scale_value((uint32_t)ref) : 1.f;
    if (c == 0) sums[warp * 16 + r + 8 * h] = make_float2(m_true[h], l[h] * to);
#pragma unroll
    for (int j = 0; j < Sh::kVVecs; ++j)
#pragma unroll
      for (int e = 0; e < Sh::kVElems; ++e)
#pragma unroll
        for (int x = 0; x < 2; ++x)
          mine[(r + 8 * h) * (D + 4) + (j * 8 + 2 * c + x) * Sh::kVElems + e] =
              o[j * Sh::kVElems + e][2 * h + x] * to * unit;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * (D / 4); i += kWarps * 32) {
    const int lr = i / (D / 4), d = i % (D / 4) * 4, row = row0 + lr;
    if (row >= M) break;
    float m = -INFINITY, lsum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sums[w * 16 + lr].x);
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 s = sums[w * 16 + lr];
      const float f = exp2f(s.x - (m == -INFINITY ? 0.f : m));
      const float4 x = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(body) + (w * 16 + lr) * (D + 4) + d);
      lsum += s.y * f;
      v.x += x.x * f, v.y += x.y * f, v.z += x.z * f, v.w += x.w * f;
    }
    const long long at = (long long)(sp.first + row / G) * a.q_heads + head * G + row % G;
    if (parts.count == 1) {
      finish4<F32>(a, at, d, v, m, lsum);
    } else {
      const long long to = ((long long)part * gridDim.z * gridDim.y + seq * gridDim.y + blockIdx.y) * kTileRows + lr;
      *reinterpret_cast<float4*>(parts.o + to * D + d) = v;
      if (d == 0) parts.ml[to] = make_float2(m, lsum);
    }
  }
}

template <int FMT, bool F32>
cudaError_t launch(const AttnArgs& a, const Parts& p, cudaStream_t st) {
  using Sh = Shape<FMT, F32>;
  // the kernel's shared memory is set once for each device (twice by two threads at once does no harm)
  static std::atomic<unsigned long long> set{0};
  int dev = 0;
  if (cudaError_t e = cudaGetDevice(&dev)) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(set.load(std::memory_order_relaxed) & bit)) {
    if (cudaError_t e = cudaFuncSetAttribute(parts_kernel<FMT, F32>, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem))
      return e;
    set.fetch_or(bit, std::memory_order_relaxed);
  }
  const int tiles = (a.max_rows * (a.q_heads / a.c.heads) + kTileRows - 1) / kTileRows;
  parts_kernel<FMT, F32><<<dim3(p.count, a.c.heads * tiles, a.b.n_seqs), kWarps * 32, Sh::kSmem, st>>>(a, p);
  return cudaGetLastError();
}

}  // namespace

#define TACTKV_CAT_(x, y) x##y
#define TACTKV_CAT(x, y) TACTKV_CAT_(x, y)
cudaError_t TACTKV_CAT(launch_parts_, TACTKV_TEXT_D)(int fmt, bool f32, const AttnArgs& a, const Parts& p, cudaStream_t st) {
  if (fmt == kBf16) return f32 ? launch<kBf16, true>(a, p, st) : launch<kBf16, false>(a, p, st);
  if (fmt == kFp8) return f32 ? launch<kFp8, true>(a, p, st) : launch<kFp8, false>(a, p, st);
  return f32 ? launch<kFp4, true>(a, p, st) : launch<kFp4, false>(a, p, st);
}

}  // namespace text
}  // namespace tactkv

// Attention of a sequence's newest rows over its text cache (include/tactkv.h, tactkv_text_attention),
// for one head_dim (TACTKV_TEXT_D, compiled once for each):
//   s_t = q . K[t] / sqrt(D) over the tokens t that the row sees,  m = max s_t,  l = sum exp(s_t - m),
//   out = (sum exp(s_t - m) V[t]) / l,  in one pass over the tokens with a running maximum and sum.
//
// A CTA has a unit (sequence, K/V head and a tile of 8 NR rows; row = node * G + query head within the group)
// and a part of the sequence's tokens.  Its warps take 16 tokens at a time each and never wait for one another.
// The products are taken with the tokens, or the output's columns, as the m16n8k16 instruction's 16 and the
// rows as its 8: S^T = K Q^T and O^T = V^T P^T.  A decode step's few rows then fill the instruction, K and
// V are decoded once for all rows of the tile, and because the order of a summed index is free, the pieces of K
// and V that a lane needs are pieces of rows as they lie in the cache.  So each lane copies its own
// pieces (cp.async, 16 bytes where head_dim allows) into a ring in shared memory and reads back only those: no
// barrier but the warp's own.  S^T's accumulators become P^T's fragments by one 8 x 8 transposition (movmatrix).
//
// What bounds it: instructions (decoding, splitting into terms, the softmax, for 16 tokens and 8 rows at a time), and
// the latency of a warp's steps where there are few.  16 sequences x 4 heads x 128 x 3000 to 6000 tokens, 4 rows, float32
// queries: bfloat16 cache 66 us, 2.3 TB/s; 8 bits 42 us, 1.8 TB/s; one tile of 100 tokens 8 us.
//
// A coded value, code * 2^e, is a bfloat16 exactly (what bfloat16 drops below 2^-126 aside), and so it goes into the products:
// no value needs another's scale, and magnitudes may differ by all that bfloat16 holds, within a token and between tokens,
// seen or not.  (Half precision relative to the largest scale so far took a product fewer for P and fewer terms for float32
// queries: 35 us for the 42 above, 30 for 36 at head_dim 96.  But a large V in a token that a row does not see took that row's
// probabilities below half precision's range.)
// Queries: bfloat16 ones go in as they are, float32 ones as three bfloat16 terms.  The probabilities are one term for bfloat16
// caches, two for coded ones, whose values have 4 bits or 2 themselves, and three for float32 queries.
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

constexpr float kToLog2 = to_log2(D);

constexpr int vec_bytes(int bytes, int most) {   // the widest power of two that divides a lane's share
  int v = most;
  while (bytes % v) v /= 2;
  return v;
}

template <int FMT, bool F32, int NR>
struct Shape {
  static constexpr bool kCoded = FMT != kBf16;
  static constexpr int kRows = 8 * NR;
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
  static constexpr int kLimbs = F32 ? 3 : 1, kPLimbs = F32 ? 3 : (kCoded ? 2 : 1);      // bfloat16 terms of q and of P
  static constexpr bool kQInRegs = 2 * NR * kLimbs * (D / 16) <= 32;
  static constexpr int kQBytes = NR * kLimbs * (D / 16) * 32 * 8;
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kSum = kWarps * kRows * (D + 4) * 4;       // the warps' sums, over the ring when it is done
  static constexpr int kBody = kRing > kSum ? kRing : kSum;
  static constexpr int kSmem = kQBytes + kBody + kRows * 8 + kWarps * kRows * 8;
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

__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint2 b) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b.x), "r"(b.y));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {   // an 8 x 8 matrix of 16-bit values across the warp
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(v));
  return y;
}

template <int FMT, bool F32, int NR>
__global__ void __launch_bounds__(kWarps * 32) parts_kernel(const AttnArgs a, const Parts parts) {
  using Sh = Shape<FMT, F32, NR>;
  constexpr int MT = D / 16;                      // 16-column tiles of the output
  constexpr int KS = D / 16;                      // K's steps
  extern __shared__ __align__(16) unsigned char smem[];
  uint2* q_frag = reinterpret_cast<uint2*>(smem);                                 // [limb][step][tile][lane]
  unsigned char* body = smem + Sh::kQBytes;
  unsigned long long* words = reinterpret_cast<unsigned long long*>(body + Sh::kBody);   // [row] what it sees
  float2* sums = reinterpret_cast<float2*>(words + Sh::kRows);                    // [warp][row] (m, l)

  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, r = lane / 4, c = lane & 3;
  const int G = a.q_heads / a.c.heads;
  const int part = blockIdx.x, seq = blockIdx.z, tiles = gridDim.y / a.c.heads;
  const int head = blockIdx.y / tiles, tile = blockIdx.y % tiles;
  const Span sp = span_of(a.b, a.c.page_log2, seq, a.max_len, a.max_rows);
  if (!sp.ok) {                                   // the sequence's rows see no text token
    if (part == 0 && tile == 0) finish_misfit<F32, D>(a, sp, seq, head, G);
    return;
  }
  const int M = sp.rows * G, row0 = tile * Sh::kRows, before = sp.len - sp.rows;
  const int t0 = part * parts.tokens, t1 = t0 + min(sp.len - t0, parts.tokens);
  if (row0 >= M || (part > 0 && t0 >= sp.len)) return;

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
        // 16 tokens' scales are D / 2 neighbouring bytes: the first lanes copy K's, the next ones V's, 16 at a time
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

  // ---- the queries' B fragments ----
  // Lane (r, c) of K's step k holds elements idx = 4k .. 4k+3 of its share of row 8n + r: d = (idx / kKElems * 4
  // + c) * kKElems + idx % kKElems.
  for (int n = warp; n < NR; n += kWarps) {
    const int row = row0 + 8 * n + r;
    const bool in = row < M;
    const int node = in ? row / G : 0;
    const long long at = (long long)(sp.first + node) * a.q_token + (long long)(head * G + (in ? row % G : 0)) * a.q_head;
    float x[KS][4];
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      const int d = (4 * k / Sh::kKElems * 4 + c) * Sh::kKElems + 4 * k % Sh::kKElems;
      if constexpr (F32) {
        const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + at + d);
        x[k][0] = v.x, x[k][1] = v.y, x[k][2] = v.z, x[k][3] = v.w;
      } else {
        const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(a.q) + at + d);
        const float2 lo = unpack_bf16x2(v.x), hi = unpack_bf16x2(v.y);
        x[k][0] = lo.x, x[k][1] = lo.y, x[k][2] = hi.x, x[k][3] = hi.y;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (!in) x[k][i] = 0.f;
    }
    if (c == 0) words[8 * n + r] = a.tree ? a.tree[sp.first + node] : (node >= 63 ? ~0ull : (2ull << node) - 1);
#pragma unroll
    for (int k = 0; k < KS; ++k) {
#pragma unroll
      for (int y = 0; y < Sh::kLimbs; ++y) {
        const uint2 w = make_uint2(pack_bf16x2_rz(x[k][0], x[k][1]), pack_bf16x2_rz(x[k][2], x[k][3]));
        q_frag[((y * KS + k) * NR + n) * 32 + lane] = w;
        const float2 u = unpack_bf16x2(w.x), v = unpack_bf16x2(w.y);
        const float held[4] = {u.x, u.y, v.x, v.y};
#pragma unroll
        for (int i = 0; i < 4; ++i) x[k][i] = x[k][i] == held[i] ? 0.f : x[k][i] - held[i];   // nothing is left of an infinity
      }
    }
  }
  __syncthreads();
  uint2 q_reg[Sh::kQInRegs ? Sh::kLimbs * KS * NR : 1];
  if constexpr (Sh::kQInRegs) {
#pragma unroll
    for (int i = 0; i < Sh::kLimbs * KS * NR; ++i) q_reg[i] = q_frag[i * 32 + lane];
  }
  float o[MT][NR][4] = {};                        // columns r (0, 1) and r + 8 (2, 3) of a tile; rows 2c, 2c + 1
  float m_ref[NR][2], m_true[NR][2], l[NR][2] = {};
#pragma unroll
  for (int n = 0; n < NR; ++n)
#pragma unroll
    for (int x = 0; x < 2; ++x) m_ref[n][x] = m_true[n][x] = -INFINITY;

  for (int i = 0; i < steps; ++i) {
    if (i && i % 32 == 0) pages = pages_next, pages_next = page_of(i + 32 + lane);
    copy_wait<Sh::kStages - 2>();
    __syncwarp();
    {
      const int n = i + Sh::kStages - 1;          // its slot is the one of step i - 1, which every lane has left
      const int pa = __shfl_sync(~0u, pages, n & 31), pb = __shfl_sync(~0u, pages_next, n & 31);
      issue(n, n / 32 == i / 32 ? pa : pb);
    }
    const int page = __shfl_sync(~0u, pages, i & 31);
    if (page < 0) continue;
    const unsigned char* stage = ring + i % Sh::kStages * Sh::kStage;
    const unsigned char* k_scales = stage + Sh::kKBytes + Sh::kVBytes;
    const unsigned char* v_scales = k_scales + Sh::kScaleBytes;
    const int t = (first + i * kWarps) * kStep;
    const int held = sp.len - t;

    // ---- scores: z[n][0, 1]: token r, rows 8n + 2c, + 1;  z[n][2, 3]: token r + 8 ----
    float z[NR][4] = {};
    {
      float low[NR][4] = {};                      // the queries' lower terms are summed apart: their rounding stays small
      uint32_t w[2][Sh::kKVecs][4];
      float f[2][Sh::kKVecs];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < Sh::kKVecs; ++j) {
          load_words<Sh::kKVec>(stage + ((h * Sh::kKVecs + j) * 32 + lane) * Sh::kKVec, w[h][j]);
          if constexpr (Sh::kCoded) f[h][j] = scale_value(k_scales[(8 * h + r) * (D / kGroup) + (j * 4 + c) * Sh::kKElems / kGroup]);
        }
#pragma unroll
      for (int j = 0; j < Sh::kKVecs; ++j)
#pragma unroll
        for (int k = 0; k < Sh::kKElems / 4; ++k) {
          uint32_t b[4];                          // A fragment: token r, r + 8 (elements 0, 1), token r, r + 8 (2, 3)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if constexpr (FMT == kBf16) {
              b[h] = w[h][j][2 * k], b[2 + h] = w[h][j][2 * k + 1];
            } else if constexpr (FMT == kFp8) {
              unpack_e4m3x4(w[h][j][k], b[h], b[2 + h]);
            } else {
              uint32_t u[4];
              unpack_e2m1x8(w[h][j][k / 2], u);
              b[h] = u[k % 2 * 2], b[2 + h] = u[k % 2 * 2 + 1];
            }
            if constexpr (Sh::kCoded) b[h] = scaled_bf16x2(b[h], f[h][j], f[h][j]), b[2 + h] = scaled_bf16x2(b[2 + h], f[h][j], f[h][j]);
          }
          const int step = j * (Sh::kKElems / 4) + k;
#pragma unroll
          for (int y = 0; y < Sh::kLimbs; ++y)
#pragma unroll
            for (int n = 0; n < NR; ++n) {
              const int at = (y * KS + step) * NR + n;
              uint2 q;
              if constexpr (Sh::kQInRegs) q = q_reg[at];
              else q = q_frag[at * 32 + lane];
              // odd steps go into the second sum (without lower terms): two chains of dependent products
              mma(y || (Sh::kLimbs == 1 && step % 2) ? low[n] : z[n], b, q);
            }
        }
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          z[n][x] += low[n][x];
          z[n][x] *= kToLog2;
        }
    }
    const bool tail = t + kStep > before;
    if (tail) {
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int node = t + r + 8 * (x / 2) - before;
          if (node >= 0 && (node >= sp.rows || !(words[8 * n + 2 * c + x % 2] >> node & 1))) z[n][x] = -INFINITY;
        }
    }

    // ---- running maximum: moved only when a score is 2^kSlack above it ----
    bool over = false;
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float high = fmaxf(z[n][x], z[n][2 + x]);
        m_true[n][x] = max_nan(m_true[n][x], max_nan(z[n][x], z[n][2 + x]));
        over |= high > m_ref[n][x] + kSlack;
      }
    if (__any_sync(~0u, over)) {
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float v = fmaxf(z[n][x], z[n][2 + x]);
#pragma unroll
          for (int y = 4; y <= 16; y *= 2) v = fmaxf(v, __shfl_xor_sync(~0u, v, y));
          const float next = v > m_ref[n][x] + kSlack ? v : m_ref[n][x];
          const float keep = next == -INFINITY ? 1.f : exp2_fast(m_ref[n][x] - next);
          m_ref[n][x] = next;
          l[n][x] *= keep;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) o[mt][n][x] *= keep, o[mt][n][2 + x] *= keep;
        }
    }

    // ---- probabilities, and their B fragments: tokens 2c, 2c + 1 (x) and 2c + 8, 2c + 9 (y) of row 8n + r ----
    float p[NR][4];
    uint2 pb[Sh::kPLimbs][NR];
    {
#pragma unroll
      for (int n = 0; n < NR; ++n) {
#pragma unroll
        for (int x = 0; x < 4; ++x)
          p[n][x] = exp2_fast(z[n][x] + (kBase - (m_ref[n][x % 2] == -INFINITY ? 0.f : m_ref[n][x % 2])));
#pragma unroll
        for (int x = 0; x < 2; ++x) l[n][x] += p[n][x] + p[n][2 + x];
        float u[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) u[x] = p[n][x];
#pragma unroll
        for (int y = 0; y < Sh::kPLimbs; ++y) {
          const uint32_t lo = pack_bf16x2(u[0], u[1]), hi = pack_bf16x2(u[2], u[3]);
          pb[y][n] = make_uint2(transpose8(lo), transpose8(hi));
          const float2 v = unpack_bf16x2(lo), w = unpack_bf16x2(hi);
          u[0] -= v.x, u[1] -= v.y, u[2] -= w.x, u[3] -= w.y;
        }
      }
    }

    // ---- sums: column r of half tile (j, e) is d = (j * 8 + r) * kVElems + e ----
#pragma unroll
    for (int j = 0; j < Sh::kVVecs; ++j) {
      uint32_t w[4][4];
      float f[4];                                  // of the tokens, 0 for what the page holds behind the last one
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        load_words<Sh::kVCopy>(stage + Sh::kKBytes + ((n * Sh::kVVecs + j) * 32 + lane) * Sh::kVCopy, w[n]);
        if constexpr (Sh::kVVec < 4) w[n][0] >>= 16 * (r & 1);
      }
      if constexpr (Sh::kCoded) {
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const int tok = 2 * c + (n & 1) + 8 * (n >> 1);
          f[n] = tok < held ? scale_value(v_scales[tok * (D / kGroup) + (j * 8 + r) * Sh::kVElems / kGroup]) : 0.f;
        }
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
            for (int i = 0; i < 4; ++i) b[i][side] = scaled_bf16x2(b[i][side], f[2 * side], f[2 * side + 1]);
          }
        }
        bool odd = false;
        if (tail) {
#pragma unroll
          for (int i = 0; i < 4; ++i) odd |= odd2(b[i][0]) || odd2(b[i][1]);
          odd = __any_sync(~0u, odd);
        }
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          float (&sum)[NR][4] = o[(j * Sh::kVElems + e0 + i) / 2];
          if (!odd) {
            const uint32_t av[4] = {b[i][0], b[i + 1][0], b[i][1], b[i + 1][1]};
#pragma unroll
            for (int y = 0; y < Sh::kPLimbs; ++y)
#pragma unroll
              for (int n = 0; n < NR; ++n) mma(sum[n], av, pb[y][n]);
          } else {
            // An infinity or NaN among the drafted tokens' values: only the rows that see it may get it, so
            // the products are summed one by one.  Token 2 cc + x + 8 h of column r is lane (r, cc)'s; its
            // probabilities for rows 2c, 2c + 1 are lane (2 cc + x, c)'s.
#pragma unroll 1
            for (int tok = 0; tok < kStep; ++tok) {
              const int h = tok >> 3, node = t + tok - before;
              const uint32_t u = __shfl_sync(~0u, h ? b[i][1] : b[i][0], 4 * r + (tok & 7) / 2),
                             v = __shfl_sync(~0u, h ? b[i + 1][1] : b[i + 1][0], 4 * r + (tok & 7) / 2);
              const float2 xu = unpack_bf16x2(u), xv = unpack_bf16x2(v);
#pragma unroll
              for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                  const float pr = __shfl_sync(~0u, h ? p[n][2 + x] : p[n][x], 4 * (tok & 7) + c);
                  if (node < 0 || (node < sp.rows && (words[8 * n + 2 * c + x] >> node & 1))) {
                    sum[n][x] += pr * (tok & 1 ? xu.y : xu.x);
                    sum[n][2 + x] += pr * (tok & 1 ? xv.y : xv.x);
                  }
                }
            }
          }
        }
      }
    }
  }
  copy_wait<0>();
  let_next_start();

  // ---- the warps' sums, to the rows' true maxima ----
  __syncthreads();                                 // the ring is done: its place takes the sums
  float* mine = reinterpret_cast<float*>(body) + warp * Sh::kRows * (D + 4);
#pragma unroll
  for (int n = 0; n < NR; ++n)
#pragma unroll
    for (int x = 0; x < 2; ++x) {
#pragma unroll
      for (int y = 4; y <= 16; y *= 2) {
        m_true[n][x] = max_nan(m_true[n][x], __shfl_xor_sync(~0u, m_true[n][x], y));
        l[n][x] += __shfl_xor_sync(~0u, l[n][x], y);
      }
      const int row = 8 * n + 2 * c + x;
      const float to = m_true[n][x] == -INFINITY ? 0.f : exp2f(m_ref[n][x] - m_true[n][x]);
      if (r == 0) sums[warp * Sh::kRows + row] = make_float2(m_true[n][x], l[n][x] * (to * kUnbase));
#pragma unroll
      for (int j = 0; j < Sh::kVVecs; ++j)
#pragma unroll
        for (int e = 0; e < Sh::kVElems; ++e)
          mine[row * (D + 4) + (j * 8 + r) * Sh::kVElems + e] =
              o[(j * Sh::kVElems + e) / 2][n][e % 2 * 2 + x] * to;
    }
  __syncthreads();
  for (int i = threadIdx.x; i < Sh::kRows * (D / 4); i += kWarps * 32) {
    const int lr = i / (D / 4), d = i % (D / 4) * 4, row = row0 + lr;
    if (row >= M) break;
    float m = -INFINITY, lsum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) m = max_nan(m, sums[w * Sh::kRows + lr].x);
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 s = sums[w * Sh::kRows + lr];
      const float f = exp2f(s.x - (m == -INFINITY ? 0.f : m));
      const float4 x = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(body) + (w * Sh::kRows + lr) * (D + 4) + d);
      lsum += s.y * f;
      v.x += x.x * f, v.y += x.y * f, v.z += x.z * f, v.w += x.w * f;
    }
    if (parts.count == 1) {
      finish4<F32>(a, (long long)(sp.first + row / G) * a.q_heads + head * G + row % G, d, v, m, lsum);
    } else {
      const long long to = ((long long)part * gridDim.z * gridDim.y + seq * gridDim.y + blockIdx.y) * Sh::kRows + lr;
      *reinterpret_cast<float4*>(parts.o + to * D + d) = v;
      if (d == 0) parts.ml[to] = make_float2(m, lsum);
    }
  }
}

template <int FMT, bool F32, int NR>
cudaError_t launch(const AttnArgs& a, const Parts& p, cudaStream_t st) {
  using Sh = Shape<FMT, F32, NR>;
  // the kernel's shared memory is set once for each device (twice by two threads at once does no harm)
  static std::atomic<unsigned long long> set{0};
  int dev = 0;
  if (cudaError_t e = cudaGetDevice(&dev)) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(set.load(std::memory_order_relaxed) & bit)) {
    if (cudaError_t e = cudaFuncSetAttribute(parts_kernel<FMT, F32, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem))
      return e;
    set.fetch_or(bit, std::memory_order_relaxed);
  }
  parts_kernel<FMT, F32, NR><<<dim3(p.count, a.c.heads * p.tiles, a.b.n_seqs), kWarps * 32, Sh::kSmem, st>>>(a, p);
  return cudaGetLastError();
}
template <int FMT, bool F32>
cudaError_t launch(const AttnArgs& a, const Parts& p, cudaStream_t st) {
  if (p.tile_rows == 8) return launch<FMT, F32, 1>(a, p, st);
  if (p.tile_rows == 16) return launch<FMT, F32, 2>(a, p, st);
  if constexpr (wide_tiles(FMT, F32, D)) return launch<FMT, F32, 4>(a, p, st);
  return cudaErrorInvalidValue;
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

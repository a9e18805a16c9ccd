// Attention over the text cache on tcgen05, for one head_dim (TACTKV_TEXT_D: 64, 128, 192 or 256) and
// bfloat16 queries; text_attention.cu has the mathematics, and the kernel for the other cases.
//
// Tiles of 128 tokens are the 128 lanes of tensor memory and a unit's N rows its columns:
//   S^T[token][row] = K Q^T        A = K  (K-major), B = Q (K-major)
//   O^T[d][row]    += V^T P^T      A = V^T (the same token rows, MN-major), B = P (K-major)
// so that a decode step's few rows cost the narrowest product, a thread of the softmax owns one token (its mask, its
// K and V scales), and bfloat16 pages are operands as TMA delivers them.  Warps by role:
//   softmax (4 or 8)  S^T from tensor memory -> P in shared memory; running maximum and sum in registers
//   producer (1)      copies pages: TMA tiles into operand slots (bfloat16), bulk copies into raw slots (coded)
//   issuer (1)        all products; the next tile's S^T is issued before this tile's O^T waits for its softmax
//   decoders (8, 4)   coded caches: raw slots -> half-precision operands, once for all rows of the unit
// Every wait is bounded; one that expires records TACTKV_TIMEOUT and ends the block's work.
//
// An infinity or NaN in the V of a drafted token must reach only the rows that see it, so it is taken out of
// the operand, and its rows get it in plain arithmetic at the end.
#include <atomic>
#include <mutex>

#include <cudaTypedefs.h>

#include "tc.cuh"
#include "text_attention.cuh"

#ifndef TACTKV_TEXT_D
#define TACTKV_TEXT_D 128
#endif

namespace tactkv {
namespace text {
namespace {

constexpr int D = TACTKV_TEXT_D;
constexpr int TT = 128;                           // tokens of a tile
constexpr float kToLog2 = to_log2(D);
constexpr uint32_t kPolls = 1u << 20;             // of a wait; each may block for microseconds

template <int FMT, int N>
struct Shape {
  static constexpr bool kCoded = FMT != kBf16;
  static constexpr int kBlocks = D / 64;          // 64 columns, 128 bytes, of 128 tokens: 16 KB, 128-byte swizzle
  static constexpr int kGroups = (D + 127) / 128; // of 128 output columns (the last may be half empty)
  static constexpr int kBlock = TT * 128;
  static constexpr int kOp = kBlocks * kBlock;
  static constexpr int kWGs = N == 64 ? 2 : 1;
  static constexpr int kRowsWG = N / kWGs;
  static constexpr int kDecoders = !kCoded ? 0 : (N == 64 ? 4 : 8);
  static constexpr int kThreads = 32 * (4 * kWGs + 2 + kDecoders);
  static constexpr int kRow = D * code_bits(FMT) / 8;
  static constexpr int kRaw = TT * kRow, kRawScales = TT * (D / kGroup);
  static constexpr int kSlot = kCoded ? kRaw + kRawScales : kOp;
  static constexpr int kQ = kBlocks * N * 128, kP = 2 * N * 128;
  static constexpr int kFactors = kCoded ? TT * (D / kGroup) * 2 : 0;           // of the tile being decoded
  static constexpr int kTops = kCoded ? 4 * TT : 0;                            // [K, V][parity][token]
  static constexpr int kMisc = 2048 + 24 * N + kWGs * 4 * 8 * kRowsWG;
  // With an odd number of blocks the last product reads a block past V's operand: something must be there.
  static constexpr int kPad = kBlocks % 2 ? kBlock : 0;
  static constexpr int kFixed = 1024 + (kCoded ? 2 * kOp : 0) + kQ + kP + kFactors + kTops + kMisc + kPad;
  static constexpr int kFit = (227 * 1024 - kFixed) / kSlot;
  static constexpr int kSlots = kFit > 8 ? 8 : kFit;
  static constexpr int kSmem = kFixed + kSlots * kSlot;
  static constexpr int kCols = (2 + kGroups) * N;
  static constexpr int kTmem = kCols <= 32 ? 32 : (kCols <= 64 ? 64 : (kCols <= 128 ? 128 : 256));
  static_assert(kSlots >= 2 && kCols <= 256, "");
  static_assert(N * (D + 4) * 4 <= kSlots * kSlot + (kCoded ? 2 * kOp : 0), "the sums take the operands' place");
};

struct Bars {
  uint64_t slot_full[8], slot_free[8], op_full[2], op_free[2], s_full[2], p_full, pv_done, drain;
};

// False if the phase did not complete within kPolls, or if another wait of the block expired (dead, where given).
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* dead) {
  const uint32_t a = tc::smem_u32(bar);
  for (uint32_t i = 0; i < kPolls; ++i) {
    uint32_t done;
    asm volatile(
        "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done)
        : "r"(a), "r"(parity)
        : "memory");
    if (done) return true;
    if (dead && (i & 255) == 255 && *dead) return false;
  }
  if (dead) *dead = 1;
  return false;
}
__device__ __forceinline__ void bar_sync(int id) { asm volatile("bar.sync %0, 128;\n" ::"r"(id) : "memory"); }
__device__ __forceinline__ bool bar_or(int id, int threads, bool v) {
  uint32_t y;
  asm volatile(
      "{\n.reg .pred p, q;\nsetp.ne.u32 q, %3, 0;\nbar.red.or.pred p, %1, %2, q;\nselp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(y)
      : "r"(id), "r"(threads), "r"((uint32_t)v)
      : "memory");
  return y;
}

// Element d of K or V at token index `at`, from the cache.
template <int FMT>
__device__ float value_at(const Cache& c, int kv, long long at, int d) {
  const unsigned char* p = c.pages[kv] + at * (D * code_bits(FMT) / 8);
  if constexpr (FMT == kBf16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[d]);
  const float f = scale_value(c.scales[kv][at * (D / kGroup) + d / kGroup]);
  uint32_t h[4];
  if constexpr (FMT == kFp8) unpack_e4m3x4(p[d], h[0], h[1]);
  else unpack_e2m1x8(p[d / 2] >> (d % 2 * 4), h);
  return unpack2<true>(h[0]).x * f;
}

// Sums (or maxima) over the warp of R values a lane: lane i < R gets the i-th (R = 16, 32).
template <int HALF, int R, bool MAX>
__device__ __forceinline__ void reduce_step(float (&v)[R]) {
  const bool upper = threadIdx.x & HALF;
#pragma unroll
  for (int i = 0; i < HALF; ++i) {
    const float mine = upper ? v[HALF + i] : v[i], other = __shfl_xor_sync(~0u, upper ? v[i] : v[HALF + i], HALF);
    v[i] = MAX ? fmaxf(mine, other) : mine + other;
  }
  if constexpr (HALF > 1) reduce_step<HALF / 2, R, MAX>(v);
}
template <int R, bool MAX>
__device__ __forceinline__ float reduce_rows(float (&v)[R]) {
  reduce_step<R / 2, R, MAX>(v);
  if constexpr (R == 16) {
    const float other = __shfl_xor_sync(~0u, v[0], 16);
    return MAX ? fmaxf(v[0], other) : v[0] + other;
  }
  return v[0];
}

template <int FMT, int N>
__global__ void __launch_bounds__(Shape<FMT, N>::kThreads, 1)
    tc_kernel(const AttnArgs a, const Parts parts, const __grid_constant__ CUtensorMap k_map,
              const __grid_constant__ CUtensorMap v_map) {
  using Sh = Shape<FMT, N>;
  constexpr bool kCoded = Sh::kCoded;
  constexpr int R = Sh::kRowsWG;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024 - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
  unsigned char* k_op = smem;                                             // coded: the operands ..
  unsigned char* v_op = k_op + (kCoded ? Sh::kOp : 0);
  unsigned char* q_op = v_op + (kCoded ? Sh::kOp : 0);
  unsigned char* p_op = q_op + Sh::kQ;
  unsigned char* slots = p_op + Sh::kP;                                   // .. and raw slots; bfloat16: operand slots
  unsigned char* factors = slots + Sh::kSlots * Sh::kSlot + Sh::kPad;
  unsigned char* tops = factors + Sh::kFactors;
  unsigned char* misc = tops + Sh::kTops;
  Bars* bars = reinterpret_cast<Bars*>(misc);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc + 512);
  volatile int* dead = reinterpret_cast<volatile int*>(misc + 516);
  uint32_t* odd_nodes = reinterpret_cast<uint32_t*>(misc + 520);          // 2 words
  uint32_t* absent_of = reinterpret_cast<uint32_t*>(misc + 576);          // [tile % 16] 16-token blocks on bad pages
  unsigned long long* words = reinterpret_cast<unsigned long long*>(misc + 2048);
  float* row_factor = reinterpret_cast<float*>(words + N);
  float* m_ref = row_factor + N;
  float2* row_ml = reinterpret_cast<float2*>(m_ref + N);
  float* exchange = reinterpret_cast<float*>(row_ml + N);                 // [WG][warp][2 R]

  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
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
        for (int i = threadIdx.x; i < G * (D / 4); i += Sh::kThreads)
          finish4<false>(a, (long long)row * a.q_heads + head * G + i / (D / 4), i % (D / 4) * 4,
                         make_float4(0.f, 0.f, 0.f, 0.f), -INFINITY, 0.f);
    }
    return;
  }
  const int M = sp.rows * G, row0 = tile * N, before = sp.len - sp.rows;
  const int t0 = part * parts.tokens;
  if (row0 >= M || t0 >= sp.len) return;
  const int n_tiles = (min(sp.len - t0, parts.tokens) + TT - 1) / TT;

  // ---- set up: barriers, tensor memory, the queries' operand ----
  if (threadIdx.x == 0) {
    for (int i = 0; i < Sh::kSlots; ++i) {
      tc::mbar_init(&bars->slot_full[i], 1);
      tc::mbar_init(&bars->slot_free[i], kCoded ? Sh::kDecoders : 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&bars->op_full[i], kCoded ? Sh::kDecoders : 1);
      tc::mbar_init(&bars->op_free[i], 1);
      tc::mbar_init(&bars->s_full[i], 1);
    }
    tc::mbar_init(&bars->p_full, 128 * Sh::kWGs);
    tc::mbar_init(&bars->pv_done, 1);
    tc::mbar_init(&bars->drain, 1);
    tc::fence_mbar_init();
    *dead = 0;
    odd_nodes[0] = odd_nodes[1] = 0;
  }
  if (warp == 4 * Sh::kWGs + 1) tc::tmem_alloc(tmem_slot, Sh::kTmem);
  for (int n = warp; n < N; n += Sh::kThreads / 32) {   // a warp per row: lane i has elements i * D/32 ..
    constexpr int E = D / 32;
    const int row = row0 + n;
    const bool in = row < M;
    const int node = in ? row / G : 0;
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + (long long)(sp.first + node) * a.q_token +
                             (long long)(head * G + (in ? row % G : 0)) * a.q_head + lane * E;
    uint32_t w[E / 2], top = 0;
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      w[i] = in ? reinterpret_cast<const uint32_t*>(q)[i] : 0u;
      top = max(top, max(w[i] << 16 & 0x7FFF0000u, w[i] & 0x7FFF0000u));
    }
    float back = kToLog2;
    if constexpr (kCoded) {                        // largest element into [2^14, 2^15)
      const int E8 = (int)(__reduce_max_sync(~0u, top) >> 23);
      const int e = E8 == 255 || __reduce_max_sync(~0u, top) == 0 ? 0 : max(-126, min(126, 141 - E8));
      const float f = __uint_as_float((uint32_t)(127 + e) << 23);
      back *= __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
      for (int i = 0; i < E / 2; ++i) {
        const float2 v = unpack_bf16x2(w[i]);
        w[i] = pack2<true>(v.x * f, v.y * f);
      }
    }
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      const int d = lane * E + 2 * i;
      *reinterpret_cast<uint32_t*>(q_op + d / 64 * (N * 128) + n * 128 + ((d % 64 / 8) ^ (n & 7)) * 16 + d % 8 * 2) = w[i];
    }
    if (lane == 0) {
      row_factor[n] = back;
      m_ref[n] = -INFINITY;
      words[n] = a.tree ? a.tree[sp.first + node] : (node >= 63 ? ~0ull : (2ull << node) - 1);
    }
  }
  tc::fence_proxy_async();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;

  if (warp == 4 * Sh::kWGs) {
    // ------------------------------------------------------------------------------ producer ---
    const int page_tokens = 1 << a.c.page_log2, run = min(page_tokens, TT), runs = TT / run;
    bool ok = true;
    int issued = 0;
    for (int i = 0; i < n_tiles && ok; ++i) {
      const int t = t0 + i * TT + lane * run;
      const bool there = lane < runs && t < sp.len;
      int page = there ? __ldg(a.b.table + (long long)seq * a.b.max_pages + (t >> a.c.page_log2)) : -1;
      const bool good = there && page >= 0 && page < a.c.n_pages;
      if (there && !good) report(a.status);
      const uint32_t bad = __reduce_or_sync(~0u, there && !good ? ((1u << run / 16) - 1) << (lane * run / 16) : 0u);
      const int copies = __popc(__ballot_sync(~0u, good));
      const long long at = (((long long)page * a.c.heads + head) << a.c.page_log2) + (t & (page_tokens - 1));
      if (lane == 0) absent_of[i & 15] = bad;
      for (int kv = 0; kv < 2 && ok; ++kv) {
        const int s = 2 * i + kv, slot = s % Sh::kSlots, round = s / Sh::kSlots;
        if (round) ok = wait(&bars->slot_free[slot], (round - 1) & 1, dead);
        ok = __all_sync(~0u, ok);
        if (!ok) break;
        if (lane == 0) tc::mbar_expect_tx(&bars->slot_full[slot], copies * run * (Sh::kRow + (kCoded ? D / kGroup : 0)));
        issued = s + 1;
        __syncwarp();
        if (good) {
          unsigned char* to = slots + slot * Sh::kSlot;
          if constexpr (kCoded) {
            tc::bulk_load(to + lane * run * Sh::kRow, a.c.pages[kv] + at * Sh::kRow, run * Sh::kRow, &bars->slot_full[slot]);
            tc::bulk_load(to + Sh::kRaw + lane * run * (D / kGroup), a.c.scales[kv] + at * (D / kGroup), run * (D / kGroup),
                          &bars->slot_full[slot]);
          } else {
#pragma unroll
            for (int b = 0; b < Sh::kBlocks; ++b)
              tc::tma_load_2d(to + b * Sh::kBlock + lane * run * 128, kv ? &v_map : &k_map, &bars->slot_full[slot], 64 * b, (int)at);
          }
        }
      }
    }
    // Copies in flight when a wait expired land before the block ends.
    if (!ok)
      for (int s = max(0, issued - Sh::kSlots); s < issued; ++s) wait(&bars->slot_full[s % Sh::kSlots], s / Sh::kSlots & 1, nullptr);
  } else if (warp == 4 * Sh::kWGs + 1) {
    // -------------------------------------------------------------------------------- issuer ---
    if (lane == 0) {
      constexpr uint32_t kIdS = kCoded ? tc::idesc_f16(128, N, false) : tc::idesc_bf16(128, N, false);
      constexpr uint32_t kIdO = kCoded ? tc::idesc_f16(128, N, true) : tc::idesc_bf16(128, N, true);
      const uint32_t q_addr = tc::smem_u32(q_op), p_addr = tc::smem_u32(p_op);
      auto operand = [&](int s) { return tc::smem_u32(kCoded ? (s & 1 ? v_op : k_op) : slots + s % Sh::kSlots * Sh::kSlot); };
      auto full = [&](int s) {
        return kCoded ? wait(&bars->op_full[s & 1], s / 2 & 1, dead)
                      : wait(&bars->slot_full[s % Sh::kSlots], s / Sh::kSlots & 1, dead);
      };
      auto release = [&](int s) { tc::mma_commit(kCoded ? &bars->op_free[s & 1] : &bars->slot_free[s % Sh::kSlots]); };
      auto scores = [&](int i) {
        if (!full(2 * i)) return false;
        tc::fence_after_sync();
        const uint32_t k_addr = operand(2 * i);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          tc::mma_bf16(tmem + (i & 1) * N, tc::smem_desc(k_addr + k / 4 * Sh::kBlock + k % 4 * 32, 16, 1024, 2),
                       tc::smem_desc(q_addr + k / 4 * (N * 128) + k % 4 * 32, 16, 1024, 2), kIdS, k > 0);
        release(2 * i);
        tc::mma_commit(&bars->s_full[i & 1]);
        return true;
      };
      bool ok = scores(0);
      for (int i = 0; i < n_tiles && ok; ++i) {
        if (i + 1 < n_tiles) ok = scores(i + 1);
        if (ok) ok = full(2 * i + 1);
        if (ok) ok = wait(&bars->p_full, i & 1, dead);
        if (!ok) break;
        tc::fence_after_sync();
        const uint32_t v_addr = operand(2 * i + 1);
#pragma unroll
        for (int g = 0; g < Sh::kGroups; ++g)
#pragma unroll
          for (int k = 0; k < TT / 16; ++k)
            tc::mma_bf16(tmem + (2 + g) * N, tc::smem_desc(v_addr + 2 * g * Sh::kBlock + k * 2048, Sh::kBlock, 1024, 2),
                         tc::smem_desc(p_addr + k / 4 * (N * 128) + k % 4 * 32, 16, 1024, 2), kIdO, i > 0 || k > 0);
        release(2 * i + 1);
        tc::mma_commit(&bars->pv_done);
      }
      if (!ok) {                                   // products in flight end before tensor memory is released
        tc::mma_commit(&bars->drain);
        wait(&bars->drain, 0, nullptr);
      }
    }
    __syncwarp();
  } else if (warp < 4 * Sh::kWGs) {
    // ------------------------------------------------------------------------------- softmax ---
    const int wg = warp / 4, tid = threadIdx.x & 127, bar = 1 + wg, rows0 = wg * R;
    const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);            // lane 32 * (warp % 4) in bits 16 ..
    float l[R] = {}, m_true[R];
#pragma unroll
    for (int n = 0; n < R; ++n) m_true[n] = -INFINITY;
    uint32_t ref = 0;
    bool ok = true;
    for (int i = 0; i < n_tiles; ++i) {
      ok = __all_sync(~0u, wait(&bars->s_full[i & 1], i / 2 & 1, dead));
      ok = !bar_or(bar, 128, !ok);
      if (!ok) break;
      tc::fence_after_sync();
      const int t = t0 + i * TT + tid, node = t - before;
      const bool absent = t >= sp.len || (absent_of[i & 15] >> (tid / 16) & 1);
      const bool tail = t0 + (i + 1) * TT > before;
      uint32_t v_top = 0;
      float k_scale = 1.f;
      if constexpr (kCoded) {
        k_scale = scale_value(tops[(i & 1) * TT + tid]);
      }
      float z[R];
#pragma unroll
      for (int c = 0; c < R; c += 16) {
        float x[16];
        tc::tmem_ld<16>(lanes + (i & 1) * N + rows0 + c, x);
        tc::tmem_ld_wait();
#pragma unroll
        for (int n = 0; n < 16; ++n) z[c + n] = x[n];
      }
#pragma unroll
      for (int n = 0; n < R; ++n) {
        z[n] *= k_scale * row_factor[rows0 + n];
        if (absent) z[n] = -INFINITY;
      }
      if (tail && node >= 0 && !absent) {
#pragma unroll
        for (int n = 0; n < R; ++n)
          if (!(words[rows0 + n] >> node & 1)) z[n] = -INFINITY;
      }
      if constexpr (kCoded) {                      // V's scales are known when its operand is
        ok = wait(&bars->op_full[1], i & 1, dead);
        v_top = tops[(2 + (i & 1)) * TT + tid];
      }
      bool over = v_top > ref;
#pragma unroll
      for (int n = 0; n < R; ++n) {
        m_true[n] = fmaxf(m_true[n], z[n]);
        over |= z[n] > m_ref[rows0 + n] + kSlack;
      }
      if (i) {   // O is whole, and P's place free
        ok &= wait(&bars->pv_done, (i - 1) & 1, dead);
        ok = __all_sync(~0u, ok);
        tc::fence_after_sync();
      }
      if (bar_or(bar, 128, over || !ok)) {
        if (bar_or(bar, 128, !ok)) break;
        // move the references: the largest score of every row, the largest V scale
        float v[R];
#pragma unroll
        for (int n = 0; n < R; ++n) v[n] = z[n];
        const float high = reduce_rows<R, true>(v);
        float* mine = exchange + (wg * 4 + (warp & 3)) * 2 * R;
        if (lane < R) mine[lane] = high;
        const uint32_t top = __reduce_max_sync(~0u, v_top);
        if (lane == 0) mine[R] = __uint_as_float(top);
        bar_sync(bar);
        float keep = 1.f;                          // of row rows0 + tid
        uint32_t new_ref = ref;
#pragma unroll
        for (int w = 0; w < 4; ++w) new_ref = max(new_ref, __float_as_uint(exchange[(wg * 4 + w) * 2 * R + R]));
        if (tid < R) {
          float most = -INFINITY;
#pragma unroll
          for (int w = 0; w < 4; ++w) most = fmaxf(most, exchange[(wg * 4 + w) * 2 * R + tid]);
          const float old = m_ref[rows0 + tid];
          if (most > old + kSlack) {
            m_ref[rows0 + tid] = most;
            keep = exp2_fast(old - most);
          }
        }
        bar_sync(bar);                             // the exchanged maxima are read
        if (tid < R) exchange[wg * 4 * 2 * R + tid] = keep;
        bar_sync(bar);
        const float down = kCoded ? __uint_as_float((uint32_t)max(127 + (int)ref - (int)new_ref, 0) << 23) : 1.f;
        ref = new_ref;
        const float* keeps = exchange + wg * 4 * 2 * R;
#pragma unroll
        for (int n = 0; n < R; ++n) l[n] *= keeps[n];
        if (i) {
#pragma unroll
          for (int g = 0; g < Sh::kGroups; ++g)
#pragma unroll
            for (int c = 0; c < R; c += 16) {
              float o[16];
              const uint32_t at = lanes + (2 + g) * N + rows0 + c;
              tc::tmem_ld<16>(at, o);
              tc::tmem_ld_wait();
#pragma unroll
              for (int n = 0; n < 16; ++n) o[n] *= keeps[c + n] * down;
              tc::tmem_st16(at, o);
            }
          tc::tmem_st_wait();
        }
        bar_sync(bar);                             // before the factors' place is written again
      }
      const float fold = kCoded ? __uint_as_float((uint32_t)max(127 + (int)v_top - (int)ref, 0) << 23) : 1.f;
      unsigned char* p_at = p_op + tid / 64 * (N * 128) + tid % 8 * 2;
      const int chunk = tid % 64 / 8;
#pragma unroll
      for (int n = 0; n < R; ++n) {
        const float r = m_ref[rows0 + n];
        const float p = exp2_fast(z[n] + (kBase - (r == -INFINITY ? 0.f : r)));
        l[n] += p;
        unsigned short h;
        if constexpr (kCoded) {
          const __half x = __float2half_rn(p * fold);
          h = *reinterpret_cast<const unsigned short*>(&x);
        } else {
          const __nv_bfloat16 x = __float2bfloat16_rn(p);
          h = *reinterpret_cast<const unsigned short*>(&x);
        }
        *reinterpret_cast<unsigned short*>(p_at + (rows0 + n) * 128 + ((chunk ^ (n & 7)) << 4)) = h;
      }
      if (!kCoded && tail && wg == 0) {
        // Behind the last token V's operand holds whatever the page holds (decoders write zeros there), and
        // a drafted token's infinities and NaN are for some rows only: zeros take their place.
        ok = __all_sync(~0u, wait(&bars->slot_full[(2 * i + 1) % Sh::kSlots], (2 * i + 1) / Sh::kSlots & 1, dead));
      }
      if (wg == 0 && ok && (absent ? !kCoded : tail && node >= 0)) {
        if (!tail && !kCoded) ok = wait(&bars->slot_full[(2 * i + 1) % Sh::kSlots], (2 * i + 1) / Sh::kSlots & 1, dead);
        unsigned char* v = kCoded ? v_op : slots + (2 * i + 1) % Sh::kSlots * Sh::kSlot;
        bool odd = false;
        for (int b = 0; b < Sh::kBlocks; ++b)
          for (int x = 0; x < 8; ++x) {
            uint4* w = reinterpret_cast<uint4*>(v + b * Sh::kBlock + tid * 128 + x * 16);
            if (absent) {
              *w = make_uint4(0, 0, 0, 0);
            } else {
              uint32_t y[4] = {w->x, w->y, w->z, w->w};
              bool here = false;
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (odd2<kCoded>(y[e])) {
                  here = true;
                  if (odd2<kCoded>(y[e] & 0xFFFFu)) y[e] &= 0xFFFF0000u;
                  if (odd2<kCoded>(y[e] & 0xFFFF0000u)) y[e] &= 0xFFFFu;
                }
              if (here) *w = make_uint4(y[0], y[1], y[2], y[3]);
              odd |= here;
            }
          }
        if (odd) atomicOr(odd_nodes + (node >> 5), 1u << (node & 31));
      }
      tc::fence_proxy_async();
      tc::fence_before_sync();
      tc::mbar_arrive(&bars->p_full);
    }
    if (ok) ok = wait(&bars->pv_done, (n_tiles - 1) & 1, dead);
    if (bar_or(3, 128 * Sh::kWGs, !ok || *dead)) {
      if (tid == 0) atomicCAS(a.status, 0u, (unsigned int)TACTKV_TIMEOUT);
    } else {
      // ---- the rows' true maxima and sums ----
      tc::fence_after_sync();
      const float high = reduce_rows<R, true>(m_true);
      const float total = reduce_rows<R, false>(l);
      if (lane < R) {
        exchange[(wg * 4 + (warp & 3)) * 2 * R + lane] = high;
        exchange[(wg * 4 + (warp & 3)) * 2 * R + R + lane] = total;
      }
      bar_sync(bar);
      if (tid < R) {
        float m = -INFINITY, sum = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          m = fmaxf(m, exchange[(wg * 4 + w) * 2 * R + tid]);
          sum += exchange[(wg * 4 + w) * 2 * R + R + tid];
        }
        const float to = m == -INFINITY ? 0.f : exp2f(m_ref[rows0 + tid] - m - kBase);
        row_ml[rows0 + tid] = make_float2(m, sum * to);
        row_factor[rows0 + tid] = to * (kCoded ? scale_value(ref) : 1.f);   // of the row's sums
      }
      bar_sync(bar);
      float* sums = reinterpret_cast<float*>(smem) + 0;
      if constexpr (!kCoded) sums = reinterpret_cast<float*>(slots);
#pragma unroll
      for (int g = 0; g < Sh::kGroups; ++g)
#pragma unroll
        for (int c = 0; c < R; c += 16) {
          float o[16];
          tc::tmem_ld<16>(lanes + (2 + g) * N + rows0 + c, o);
          tc::tmem_ld_wait();
          if (g * 128 + tid < D) {
#pragma unroll
            for (int n = 0; n < 16; ++n)
              sums[(rows0 + c + n) * (D + 4) + g * 128 + tid] = o[n] * row_factor[rows0 + c + n];
          }
        }
      // Infinities and NaN of drafted tokens, for the rows that see them (rare): p by one thread a row.
      if (Sh::kWGs > 1) asm volatile("bar.sync 3, %0;\n" ::"n"(128 * Sh::kWGs) : "memory");   // both have added theirs
      for (int j = 0; j < sp.rows; ++j) {
        if (!(odd_nodes[j >> 5] >> (j & 31) & 1)) continue;
        const int t = before + j;
        if (t < t0 || t >= t0 + n_tiles * TT) continue;
        const int page = __ldg(a.b.table + (long long)seq * a.b.max_pages + (t >> a.c.page_log2));
        const long long at = (((long long)page * a.c.heads + head) << a.c.page_log2) + (t & ((1 << a.c.page_log2) - 1));
        float* p_row = exchange + wg * 4 * 2 * R;
        bar_sync(bar);
        if (tid < R) {
          const int row = row0 + rows0 + tid;
          float p = -1.f;
          if (row < M && (words[rows0 + tid] >> j & 1)) {
            const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + (long long)(sp.first + row / G) * a.q_token +
                                     (long long)(head * G + row % G) * a.q_head;
            float s = 0.f;
            for (int d = 0; d < D; ++d) s = fmaf(__bfloat162float(q[d]), value_at<FMT>(a.c, 0, at, d), s);
            p = exp2f(s * kToLog2 - row_ml[rows0 + tid].x);
          }
          p_row[tid] = p;
        }
        bar_sync(bar);
        for (int d = tid; d < D; d += 128) {
          const float v = value_at<FMT>(a.c, 1, at, d);
          if (!isfinite(v))
            for (int n = 0; n < R; ++n)
              if (!(p_row[n] < 0.f)) sums[(rows0 + n) * (D + 4) + d] += p_row[n] * v;
        }
      }
      bar_sync(bar);
      for (int i = tid; i < R * (D / 4); i += 128) {
        const int n = rows0 + i / (D / 4), d = i % (D / 4) * 4, row = row0 + n;
        if (row >= M) break;
        const float4 v = *reinterpret_cast<const float4*>(sums + n * (D + 4) + d);
        const float2 ml = row_ml[n];
        if (parts.count == 1) {
          finish4<false>(a, (long long)(sp.first + row / G) * a.q_heads + head * G + row % G, d, v, ml.x, ml.y);
        } else {
          const long long to = ((long long)part * gridDim.z * gridDim.y + seq * gridDim.y + blockIdx.y) * N + n;
          *reinterpret_cast<float4*>(parts.o + to * D + d) = v;
          if (d == 0) parts.ml[to] = ml;
        }
      }
    }
    tc::fence_before_sync();
  } else if constexpr (kCoded) {
    // ------------------------------------------------------------------------------ decoders ---
    constexpr int kTokens = TT / Sh::kDecoders;                            // a warp's tokens of every tile
    constexpr int kPer = 16 * 8 / code_bits(FMT), kPieces = D / kPer;       // values in 16 bytes, pieces of a row
    const int dw = warp - 4 * Sh::kWGs - 2, first = dw * kTokens;
    constexpr int kGroupsRow = D / kGroup;
    bool ok = true;
    for (int s = 0; s < 2 * n_tiles && ok; ++s) {
      const int i = s / 2, kv = s & 1, slot = s % Sh::kSlots;
      ok = wait(&bars->slot_full[slot], s / Sh::kSlots & 1, dead);
      if (ok && i) ok = wait(&bars->op_free[kv], (i - 1) & 1, dead);
      ok = __all_sync(~0u, ok);
      if (!ok) break;
      const unsigned char* raw = slots + slot * Sh::kSlot;
      const int held = sp.len - (t0 + i * TT);
      const uint32_t bad = absent_of[i & 15];
      // a lane takes one token's scales: the largest (the NaN scale aside), and every group's factor to it
      if (lane < kTokens) {
        const int tok = first + lane;
        const bool absent = tok >= held || (bad >> (tok / 16) & 1);
        const unsigned char* sc = raw + Sh::kRaw + tok * kGroupsRow;
        uint32_t b[kGroupsRow], top = 0;
#pragma unroll
        for (int g = 0; g < kGroupsRow; ++g) {
          b[g] = sc[g];
          top = max(top, b[g] == 255u ? 0u : b[g]);
        }
        if (absent) top = 0;
        tops[(2 * kv + (i & 1)) * TT + tok] = (unsigned char)top;
#pragma unroll
        for (int g = 0; g < kGroupsRow; ++g)
          reinterpret_cast<unsigned short*>(factors)[tok * kGroupsRow + g] = absent ? 0 : (unsigned short)half_factor(b[g], top);
      }
      __syncwarp();
      unsigned char* op = kv ? v_op : k_op;
#pragma unroll 2
      for (int x = lane; x < kTokens * kPieces; x += 32) {
        const int tok = first + x / kPieces, piece = x % kPieces, d = piece * kPer;
        uint4 w = *reinterpret_cast<const uint4*>(raw + tok * Sh::kRow + piece * 16);
        if (tok >= held || (bad >> (tok / 16) & 1)) w = make_uint4(0, 0, 0, 0);
        const uint32_t f = reinterpret_cast<const unsigned short*>(factors)[tok * kGroupsRow + d / kGroup] * 0x10001u;
        const uint32_t in[4] = {w.x, w.y, w.z, w.w};
        uint32_t h[kPer / 2];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          if constexpr (FMT == kFp8) unpack_e4m3x4(in[y], h[2 * y], h[2 * y + 1]);
          else {
            uint32_t u[4];
            unpack_e2m1x8(in[y], u);
#pragma unroll
            for (int e = 0; e < 4; ++e) h[4 * y + e] = u[e];
          }
        }
        unsigned char* to = op + d / 64 * Sh::kBlock + tok * 128;
#pragma unroll
        for (int y = 0; y < kPer / 8; ++y)
          *reinterpret_cast<uint4*>(to + ((d % 64 / 8 + y) ^ (tok & 7)) * 16) =
              make_uint4(mul_half2(h[4 * y], f), mul_half2(h[4 * y + 1], f), mul_half2(h[4 * y + 2], f), mul_half2(h[4 * y + 3], f));
      }
      tc::fence_proxy_async();
      __syncwarp();
      if (lane == 0) {
        tc::mbar_arrive(&bars->op_full[kv]);
        tc::mbar_arrive(&bars->slot_free[slot]);
      }
    }
  }
  __syncthreads();
  if (warp == 4 * Sh::kWGs + 1) {
    tc::fence_after_sync();
    tc::tmem_free(tmem, Sh::kTmem);
  }
}

bool make_map(const AttnArgs& a, int kv, CUtensorMap* map) {
  static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  if (!encode) return false;
  const int page = 1 << a.c.page_log2;
  const cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)a.c.n_pages * a.c.heads * page}, strides[1] = {2 * D};
  const cuuint32_t box[2] = {64, (cuuint32_t)(page < TT ? page : TT)}, ones[2] = {1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.c.pages[kv], dims, strides, box, ones,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int FMT, int N>
cudaError_t launch(const AttnArgs& a, const Parts& p, cudaStream_t st) {
  using Sh = Shape<FMT, N>;
  // the kernel's shared memory is set once for each device (twice by two threads at once does no harm)
  static std::atomic<unsigned long long> set{0};
  int dev = 0;
  if (cudaError_t e = cudaGetDevice(&dev)) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(set.load(std::memory_order_relaxed) & bit)) {
    if (cudaError_t e = cudaFuncSetAttribute(tc_kernel<FMT, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem))
      return e;
    set.fetch_or(bit, std::memory_order_relaxed);
  }
  CUtensorMap maps[2] = {};
  if (FMT == kBf16 && !(make_map(a, 0, &maps[0]) && make_map(a, 1, &maps[1]))) return cudaErrorInvalidValue;
  tc_kernel<FMT, N><<<dim3(p.count, a.c.heads * p.tiles, a.b.n_seqs), Sh::kThreads, Sh::kSmem, st>>>(a, p, maps[0], maps[1]);
  return cudaGetLastError();
}
template <int FMT>
cudaError_t launch(const AttnArgs& a, const Parts& p, cudaStream_t st) {
  if (p.tile_rows == 16) return launch<FMT, 16>(a, p, st);
  if (p.tile_rows == 32) return launch<FMT, 32>(a, p, st);
  if constexpr (D <= kWideDim) return launch<FMT, 64>(a, p, st);
  return cudaErrorInvalidValue;
}

}  // namespace

#define TACTKV_CAT_(x, y) x##y
#define TACTKV_CAT(x, y) TACTKV_CAT_(x, y)
cudaError_t TACTKV_CAT(launch_tc_, TACTKV_TEXT_D)(int fmt, const AttnArgs& a, const Parts& p, cudaStream_t st) {
  return fmt == kBf16 ? launch<kBf16>(a, p, st) : (fmt == kFp8 ? launch<kFp8>(a, p, st) : launch<kFp4>(a, p, st));
}

}  // namespace text
}  // namespace tactkv

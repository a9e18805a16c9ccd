// Attention over the text cache on tcgen05, for one head_dim (TACTKV_TEXT_D: 64, 128, 192 or 256) and
// bfloat16 queries; text_attention.cu has the mathematics, and the kernel for the other cases.
//
// Tiles of 128 tokens are the 128 lanes of tensor memory and a unit's N rows its columns:
//   S^T[token][row] = K Q^T        A = K  (K-major), B = Q (K-major)
//   O^T[d][row]    += V^T P^T      A = V^T (the same token rows, MN-major), B = P (K-major)
// so that a decode step's few rows cost the narrowest product, a thread of the softmax owns one token and its mask, and
// bfloat16 pages are operands as TMA delivers them.  Warps by role:
//   softmax (4 to 16)  S^T from tensor memory -> P in shared memory; running maxima and sums in registers
//   producer (1)       copies pages: TMA tiles into operand slots (bfloat16), bulk copies into raw slots (coded)
//   issuer (1)         all products; the next tile's S^T is issued before this tile's O^T waits for its softmax
//   decoders (8 to 16) coded caches, in four groups (K or V, half of the tile): codes -> bfloat16 operands, once for all rows
//                      of the unit
// Every wait is bounded; one that expires records TACTKV_TIMEOUT and ends the block's work.
//
// The running maximum is lazy: a reference that scores may pass by kSlack before it, the sums and O move, so that O stays in
// tensor memory (moved with every higher score: 276 against 189 us, 4 sequences x 8 heads x 504 rows, 8111 tokens).
// Coded caches: a value, code * 2^e, is a bfloat16 exactly, so no value needs another's scale.  (In half precision relative
// to the largest scale so far, a large V that a row does not see took the row's probabilities below that type's range.)
// P is bfloat16: two terms, 16 bits, for coded caches, but one, 8 bits, for bfloat16 ones, where a second would bring bfloat16
// outputs from 2.1e-3 of the exact ones to 1.7e-3 and cost 17 % at 64 rows (112 to 130 us, 4 sequences x 8 heads x 504 rows)
// and 1 to 6 % below.  l is summed in float32 before the rounding.
//
// What bounds it.  bfloat16 caches: HBM (64 sequences x 4 heads x 128, 4000 to 8000 tokens, 16 rows: 122 to 124 us, 6.4 TB/s).
// Coded ones: the roles' own chains of latencies (the same sizes: 139 us at 8 bits and at 4, so 2.9 and 1.5 TB/s).  By
// clock readings in each role a tile costs K's decoders 2500 cycles with 16 rows and 3200 with 64, a third of them waits, and
// the softmax 1400 and 2900.  A block's start and end cost 7 to 12 us.
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
constexpr int kMaxSlots = 12;
constexpr int R = 16;                             // rows of a softmax warpgroup
constexpr float kToLog2 = to_log2(D);
constexpr uint32_t kPolls = 1u << 16;             // of a wait; each suspends the thread for up to kPause ns
// A test's build polls without suspending, and less often where a wait may give up (those with `dead`).
#ifdef TACTKV_TEXT_POLLS
constexpr uint32_t kPause = 0;
#else
#define TACTKV_TEXT_POLLS kPolls
constexpr uint32_t kPause = 20000;
#endif

template <int FMT, int N>
struct Shape {
  static constexpr bool kCoded = FMT != kBf16;
  static constexpr int kBlocks = D / 64;          // 64 columns, 128 bytes, of 128 tokens: 16 KB, 128-byte swizzle
  static constexpr int kGroups = (D + 127) / 128; // of 128 output columns (the last may be half empty)
  static constexpr int kBlock = TT * 128;
  static constexpr int kOp = kBlocks * kBlock;
  static constexpr int kWGs = N / R;              // softmax warpgroups, R rows each
  static constexpr int kRow = D * code_bits(FMT) / 8;
  static constexpr int kParts = kCoded ? 2 : 1, kPart = TT / kParts;            // a slot holds a half or all of K's or V's tile
  static constexpr int kRaw = kPart * kRow, kRawScales = kPart * (D / kGroup);
  static constexpr int kSlot = kCoded ? kRaw + kRawScales : kOp;
  static constexpr int kQ = kBlocks * N * 128;
  static constexpr int kPTerms = kCoded ? 2 : 1, kPTerm = TT * N * 2, kP = kPTerms * kPTerm;     // P's bfloat16 terms
  static constexpr int kMisc = 352 + 12 * N + 144 * kWGs;
  // With an odd number of blocks the last product reads a block past V's operand: something must be there.
  static constexpr int kPad = kBlocks % 2 ? kBlock : 0;
  static constexpr int kFixed = kQ + kMisc + kPad;
  // Two blocks on an SM: one's start, end and waits are the other's time.  bfloat16: 20.9 against 22.8 us where a launch is
  // split into one wave (16 sequences x 4 heads x 128 x 4090 tokens, 7 rows), 122 against 120 in several (64 sequences x
  // 8000).  Coded, 64 sequences x 4 heads x 8000 tokens, 16 rows: head_dim 64 98 against 134 us; 128 fits at 4 bits alone,
  // 127 against 139, but 15.4 against 13.5 for one sequence of 4000 tokens.
  static constexpr int kLeast = kFixed + 2 * kP + (kCoded ? 2 * kOp : 0) + 2 * kParts * kSlot;   // bytes, with two slots each
  static constexpr int kCtas = N <= (kCoded ? 16 : 32) && (!kCoded || D == 64) && kLeast <= 113 * 1024 ? 2 : 1;
  // V operands in turn: two where they leave the raw slots enough (32 sequences x 8 heads, 24 rows: 117 against 123 us)
  static constexpr int kVOps = kCoded && kCtas == 1 && D <= 128 ? 2 : 1;
  static constexpr int kOps = kCoded ? (1 + kVOps) * kOp : 0;
  // head_dim 256, 32 sequences x 4 heads x 8000 tokens: 150 us with 16 warps, 183 with 8; 128, 64 sequences: 148 with 16, 143
  // with 8; 192, of whose three blocks of 64 columns a lane always takes the same one if groups have three warps: 140 with
  // 12, 179 with 16
  static constexpr int kDecoders = !kCoded ? 0 : (D == 192 ? 12 : (D > 128 ? 16 : 8));
  static constexpr int kThreads = 32 * (4 * kWGs + 2 + kDecoders);
  static constexpr int kMost = (kCtas == 2 ? 113 : 227) * 1024;
  // P's places, in turn: two where they leave the raw slots' rings as long as one would, or two slots long (head_dim 128, 64
  // rows, 8 bits: 204 us with two places and rings of one, 189 with one and rings of two)
  static constexpr int ring(int ps) {
    const int n = (kMost - kFixed - ps * kP - kOps) / kSlot / 4;
    return n < 2 ? n : 2;
  }
  static constexpr int kPs = !kCoded || ring(2) == ring(1) ? 2 : 1;
  static constexpr int kFit = (kMost - kFixed - kPs * kP - kOps) / kSlot;
  static constexpr int kSlots = kFit > kMaxSlots ? kMaxSlots : kFit;
  static constexpr int kSmem = kFixed + kPs * kP + kOps + kSlots * kSlot;
  static constexpr int kCols = (2 + kGroups) * N;
  static constexpr int kTmem = kCols <= 32 ? 32 : (kCols <= 64 ? 64 : (kCols <= 128 ? 128 : 256));
  static_assert(kSlots >= 2 * kParts && kCols <= 256, "");
  static_assert(N * (D + 4) * 4 <= kOps + (kCoded ? 0 : kSlots * kSlot), "the sums take the operands' place");
  static_assert(12 * N + kWGs * 4 * 2 * R * 4 <= kP, "and what belongs to the rows' ends P's");
};

struct Bars {
  uint64_t slot_full[kMaxSlots], slot_free[kMaxSlots], op_full[3], op_free[3], s_full[2], p_full[2],
      pv_done[2], drain;
};
static_assert(sizeof(Bars) <= 304, "");
// What the warps of a softmax warpgroup tell one another when references move.
struct Exchange {
  int most[R];                                     // a row's largest score, as order_of() has it
  float shift[R];
  uint32_t moved, unused[3];
};
static_assert(sizeof(Exchange) == 144, "");

// False if the phase did not complete within kPolls, or if another wait of the block expired (dead, where given).
// SLEEP: for waits with time to spare, whose polls would take issue slots from the warps that work.
template <bool SLEEP = false>
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* dead) {
  const uint32_t a = tc::smem_u32(bar), polls = dead ? TACTKV_TEXT_POLLS : kPolls;
  for (uint32_t i = 0; i < polls; ++i) {
    uint32_t done;
    if constexpr (kPause > 0)
      asm volatile(
          "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\nselp.u32 %0, 1, 0, p;\n}\n"
          : "=r"(done)
          : "r"(a), "r"(parity), "r"(kPause)
          : "memory");
    else
      asm volatile("{\n.reg .pred p;\nmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}\n"
                   : "=r"(done)
                   : "r"(a), "r"(parity)
                   : "memory");
    if (done) return true;
    if (dead && (i & 15) == 15 && *dead) return false;
    if constexpr (SLEEP) __nanosleep(50);
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
  return __low2float(*reinterpret_cast<const __half2*>(&h[0])) * f;
}

// Two float32 operations in one instruction.
__device__ __forceinline__ unsigned long long bits2(float2 v) { return *reinterpret_cast<const unsigned long long*>(&v); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  unsigned long long y;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(y) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
  return *reinterpret_cast<const float2*>(&y);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  unsigned long long y;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(y) : "l"(bits2(a)), "l"(bits2(b)));
  return *reinterpret_cast<const float2*>(&y);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  unsigned long long y;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(y) : "l"(bits2(a)), "l"(bits2(b)));
  return *reinterpret_cast<const float2*>(&y);
}
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;\n" : "=f"(y) : "f"(x));
  return y;
}
// A number that orders like x, and back.
__device__ __forceinline__ int order_of(float x) {
  const int b = __float_as_int(x);
  return b < 0 ? b ^ 0x7FFFFFFF : b;
}
__device__ __forceinline__ float of_order(int b) { return __int_as_float(b < 0 ? b ^ 0x7FFFFFFF : b); }
// Two half-precision values (codes) times their group's scale, as bfloat16: exact in its range.
__device__ __forceinline__ uint32_t scaled2(uint32_t h, float2 f) {
  const float2 v = mul2(__half22float2(*reinterpret_cast<const __half2*>(&h)), f);
  return pack_bf16x2(v.x, v.y);
}
// Sums (or maxima) over the warp of R = 16 values a lane: lane i gets the (i % 16)-th.
template <int HALF, bool MAX>
__device__ __forceinline__ void reduce_step(float (&v)[R]) {
  const bool upper = threadIdx.x & HALF;
#pragma unroll
  for (int i = 0; i < HALF; ++i) {
    const float mine = upper ? v[HALF + i] : v[i], other = __shfl_xor_sync(~0u, upper ? v[i] : v[HALF + i], HALF);
    v[i] = MAX ? max_nan(mine, other) : mine + other;
  }
  if constexpr (HALF > 1) reduce_step<HALF / 2, MAX>(v);
}
template <bool MAX>
__device__ __forceinline__ float reduce_rows(float (&v)[R]) {
  reduce_step<R / 2, MAX>(v);
  const float other = __shfl_xor_sync(~0u, v[0], 16);
  return MAX ? max_nan(v[0], other) : v[0] + other;
}

template <int FMT, int N>
__global__ void __launch_bounds__(Shape<FMT, N>::kThreads, Shape<FMT, N>::kCtas)
    tc_kernel(const AttnArgs a, const Parts parts, const __grid_constant__ CUtensorMap k_map,
              const __grid_constant__ CUtensorMap v_map) {
  using Sh = Shape<FMT, N>;
  constexpr bool kCoded = Sh::kCoded;
  extern __shared__ __align__(1024) unsigned char smem[];
  unsigned char* k_op = smem;                                             // coded: the operands ..
  unsigned char* v_op = k_op + (kCoded ? Sh::kOp : 0);
  unsigned char* q_op = smem + Sh::kOps;
  unsigned char* p_op = q_op + Sh::kQ;
  unsigned char* slots = p_op + Sh::kPs * Sh::kP;                                 // .. and raw slots; bfloat16: operand slots
  unsigned char* misc = slots + Sh::kSlots * Sh::kSlot + Sh::kPad;
  Bars* bars = reinterpret_cast<Bars*>(misc);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc + 304);
  volatile int* dead = reinterpret_cast<volatile int*>(misc + 308);
  uint32_t* odd_nodes = reinterpret_cast<uint32_t*>(misc + 312);          // 2 words
  uint32_t* odd_tile = reinterpret_cast<uint32_t*>(misc + 320);           // decoders met an infinity or NaN in a drafted V
  unsigned char* absent_of = misc + 324;                                  // [tile % 16] 16-token blocks on bad pages, a bit each
  unsigned long long* words = reinterpret_cast<unsigned long long*>(misc + 352);
  float* row_r = reinterpret_cast<float*>(words + N);                     // a row's reference's negative
  Exchange* exchanges = reinterpret_cast<Exchange*>(row_r + N);           // [WG]
  float2* row_ml = reinterpret_cast<float2*>(p_op);                       // the rows' ends: P is done
  float* row_f = reinterpret_cast<float*>(row_ml + N);
  float* ends = row_f + N;                                                // [WG][warp][2 R]

  const int warp = __shfl_sync(~0u, threadIdx.x / 32, 0), lane = threadIdx.x & 31;   // (uniform for the compiler, too)
  const int G = a.q_heads / a.c.heads;
  const int part = blockIdx.x, seq = blockIdx.z, tiles = gridDim.y / a.c.heads;
  const int head = blockIdx.y / tiles, tile = blockIdx.y % tiles;
  const Span sp = span_of(a.b, a.c.page_log2, seq, a.max_len, a.max_rows);
  if (!sp.ok) {                                   // the sequence's rows see no text token
    if (part == 0 && tile == 0) finish_misfit<false, D>(a, sp, seq, head, G);
    return;
  }
  const int M = sp.rows * G, row0 = tile * N, before = sp.len - sp.rows;
  const int t0 = part * parts.tokens;
  if (row0 >= M || t0 >= sp.len) return;
  const int n_tiles = (min(sp.len - t0, parts.tokens) + TT - 1) / TT;

  // bfloat16: K's tiles are copied one ahead of V's, K0 K1 V0 K2 V1 .. V(n-1), and slots follow one another in that
  // order.  Coded: raw slots are rings of their own for K and V and for each half (a group of decoders sees every phase
  // of its slots' barriers, and so can tell them apart), and V0 comes before K1.
  constexpr int kRing = kCoded ? Sh::kSlots / 4 : Sh::kSlots;
  auto turn_of = [&](int i, int kv) { return kCoded ? i : (!kv ? max(2 * i - 1, 0) : (i < n_tiles - 1 ? 2 * i + 2 : 2 * n_tiles - 1)); };
  auto slot_of = [&](int i, int kv, int half) { return (kCoded ? (kv * 2 + half) * kRing : 0) + turn_of(i, kv) % kRing; };
  auto round_of = [&](int i, int kv) { return turn_of(i, kv) / kRing; };

  // ---- the producer's copies ----
  // A lane copies a run of tokens, which never leaves its page; K's or V's two slots of a tile are filled at once.  (With
  // quotients in the loop, a slot at a time and the page number read when it was needed, this warp's own chain was the
  // kernel's bound: 3500 cycles a tile.)
  const int page_tokens = 1 << a.c.page_log2, run = min(page_tokens, Sh::kPart), of_part = Sh::kPart / run;
  const int my_half = lane / of_part, my_place = lane % of_part * run;
  const uint32_t of_half = (2u << (of_part - 1)) - 1;
  bool copies_ok = true;
  constexpr int kAtOnce = kRing > 1 ? Sh::kParts : 1;   // a tile's parts copied together (a lone slot's copy does not wait for the other's)
  int last_copy[2][Sh::kParts / kAtOnce];          // of K's and V's tiles
#pragma unroll
  for (int x = 0; x < Sh::kParts / kAtOnce; ++x) last_copy[0][x] = last_copy[1][x] = -1;
  long long at = 0, at_next = 0;                   // the lane's run of this V's and the next K's tile
  uint32_t good = 0, good_next = 0;                // the lanes whose runs are there
  int page_ahead = -1;                             // of the lane's run in the tile after
  auto look = [&](int i) {
    const int t = t0 + i * TT + lane * run;
    page_ahead = my_half < Sh::kParts && t < sp.len ? __ldg(a.b.table + (long long)seq * a.b.max_pages + (t >> a.c.page_log2)) : -1;
  };
  auto find = [&](int i) {
    const int t = t0 + i * TT + lane * run, page = page_ahead;
    const bool there = my_half < Sh::kParts && t < sp.len, in = there && page >= 0 && page < a.c.n_pages;
    if (i + 1 < n_tiles) look(i + 1);
    good_next = __ballot_sync(~0u, in);
    uint32_t bad = __ballot_sync(~0u, there && !in);
    if (bad) {                                     // 16 tokens to a bit
      if (there && !in) report(a.status);
      bad = __reduce_or_sync(~0u, there && !in ? ((1u << run / 16) - 1) << (lane * run / 16) : 0u);
    }
    if (lane == 0) absent_of[i & 15] = (unsigned char)bad;
    at_next = (((long long)page * a.c.heads + head) << a.c.page_log2) + (t & (page_tokens - 1));
    __syncwarp();                                  // absent_of before the lanes' arrivals
  };
  auto copy = [&](int kv, int i) {
    const long long from = kv ? at : at_next;
    const uint32_t mask = kv ? good : good_next;
    const int round = round_of(i, kv);
#pragma unroll
    for (int first = 0; first < Sh::kParts; first += kAtOnce) {
      if (round) copies_ok = wait(&bars->slot_free[slot_of(i, kv, first + lane % kAtOnce)], (round - 1) & 1, dead);
      copies_ok = __all_sync(~0u, copies_ok);
      if (!copies_ok) return;
      if (lane < kAtOnce)
        tc::mbar_expect_tx(&bars->slot_full[slot_of(i, kv, first + lane)],
                           __popc(mask >> ((first + lane) * of_part) & of_half) * run * (Sh::kRow + (kCoded ? D / kGroup : 0)));
      last_copy[kv][first / kAtOnce] = i;
      __syncwarp();
      if ((mask >> lane & 1) && my_half >= first && my_half < first + kAtOnce) {
        const int slot = slot_of(i, kv, my_half);
        unsigned char* to = slots + slot * Sh::kSlot;
        if constexpr (kCoded) {
          tc::bulk_load(to + my_place * Sh::kRow, a.c.pages[kv] + from * Sh::kRow, run * Sh::kRow, &bars->slot_full[slot]);
          tc::bulk_load(to + Sh::kRaw + my_place * (D / kGroup), a.c.scales[kv] + from * (D / kGroup), run * (D / kGroup),
                        &bars->slot_full[slot]);
        } else {
#pragma unroll
          for (int b = 0; b < Sh::kBlocks; ++b)
            tc::tma_load_2d(to + b * Sh::kBlock + my_place * 128, kv ? &v_map : &k_map, &bars->slot_full[slot], 64 * b, (int)from);
        }
      }
    }
  };

  // ---- set up: barriers and the first copy, tensor memory, the queries' operand ----
  constexpr int kProducer = 4 * Sh::kWGs, kIssuer = kProducer + 1;
  if (warp == kProducer) {
    look(0);
    if (lane < Sh::kSlots) {
      tc::mbar_init(&bars->slot_full[lane], 1);
      tc::mbar_init(&bars->slot_free[lane], kCoded ? Sh::kDecoders / 4 : 1);
    }
    if (lane < 3) {                                // K's operand, V's (one or two)
      tc::mbar_init(&bars->op_full[lane], kCoded ? Sh::kDecoders / 2 : 1);
      tc::mbar_init(&bars->op_free[lane], 1);
    }
    if (lane < 2) {
      tc::mbar_init(&bars->s_full[lane], 1);
      tc::mbar_init(&bars->p_full[lane], 4 * Sh::kWGs);
      tc::mbar_init(&bars->pv_done[lane], 1);
      odd_nodes[lane] = 0;
    }
    if (lane == 0) {
      tc::mbar_init(&bars->drain, 1);
      *dead = 0;
      *odd_tile = 0;
    }
    tc::fence_mbar_init();
    __syncwarp();
    find(0);
    copy(0, 0);
    if constexpr (kCoded) {
      at = at_next, good = good_next;
      copy(1, 0);
    }
  } else if (warp == kIssuer) {
    tc::tmem_alloc(tmem_slot, Sh::kTmem);
  } else {
    constexpr int E = D / 32, kStagers = Sh::kThreads / 32 - 2, kMine = (N + kStagers - 1) / kStagers;
    const int stager = warp < kProducer ? warp : warp - 2;
    uint32_t w[kMine][E / 2];                      // a warp per row, lane i with its elements i * E ..; all rows' loads first
    unsigned long long word[kMine];
#pragma unroll
    for (int x = 0; x < kMine; ++x) {
      const int n = stager + x * kStagers, row = row0 + n;
      const bool in = n < N && row < M;
      const int node = in ? row / G : 0;
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + (long long)(sp.first + node) * a.q_token +
                               (long long)(head * G + (in ? row - node * G : 0)) * a.q_head + lane * E;
#pragma unroll
      for (int i = 0; i < E / 2; ++i) w[x][i] = in ? reinterpret_cast<const uint32_t*>(q)[i] : 0u;
      word[x] = a.tree ? a.tree[sp.first + node] : (node >= 63 ? ~0ull : (2ull << node) - 1);
    }
#pragma unroll
    for (int x = 0; x < kMine; ++x) {
      const int n = stager + x * kStagers;
      if (n >= N) break;
#pragma unroll
      for (int i = 0; i < E / 2; ++i) {
        const int d = lane * E + 2 * i;
        *reinterpret_cast<uint32_t*>(q_op + d / 64 * (N * 128) + n * 128 + ((d % 64 / 8) ^ (n & 7)) * 16 + d % 8 * 2) = w[x][i];
      }
      if (lane == 0) {
        row_r[n] = 0.f;
        words[n] = word[x];
      }
    }
  }
  tc::fence_proxy_async();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;

  if (warp == kProducer) {
    // ------------------------------------------------------------------------------ producer ---
    for (int i = 0; i < n_tiles && copies_ok; ++i) {
      at = at_next, good = good_next;
      if (i + 1 < n_tiles) {
        find(i + 1);
        copy(0, i + 1);
      }
      if (copies_ok && !(kCoded && i == 0)) copy(1, i);
    }
    // No copy is in flight when the block ends, not even one whose readers gave up.
    // (A part's own last copy: asked for a phase that its barrier has not reached, the one before's end would pass for it.)
#pragma unroll
    for (int x = 0; x < Sh::kParts / kAtOnce; ++x)
      for (int kv = 0; kv < 2; ++kv) {
        const int last = last_copy[kv][x];
        const int newest = kCoded ? last : max(turn_of(last_copy[0][x], 0), last_copy[1][x] < 0 ? 0 : turn_of(last_copy[1][x], 1));
        for (int i = last; i >= 0 && turn_of(i, kv) + kRing > newest; --i)
          for (int half = x * kAtOnce; half < (x + 1) * kAtOnce; ++half)
            wait<true>(&bars->slot_full[slot_of(i, kv, half)], round_of(i, kv) & 1, nullptr);
      }
  } else if (warp == kIssuer) {
    // -------------------------------------------------------------------------------- issuer ---
    // The whole warp goes along, so that descriptors stay in uniform registers; one lane issues.
    constexpr uint32_t kIdS = tc::idesc_bf16(128, N, false), kIdO = tc::idesc_bf16(128, N, true) | tc::kIdescBMn;
    // P is MN-major: a token's N rows are 32, 64 or 128 bytes with the swizzle of that width
    constexpr uint32_t kSwizzle = N == 16 ? 6 : (N == 32 ? 4 : 2);
    const uint32_t q_addr = tc::smem_u32(q_op), p_addr = tc::smem_u32(p_op);
    auto op = [&](int i, int kv) { return kv ? 1 + i % Sh::kVOps : 0; };
    auto operand = [&](int i, int kv) {
      return tc::smem_u32(kCoded ? k_op + op(i, kv) * Sh::kOp : slots + slot_of(i, kv, 0) * Sh::kSlot);
    };
    auto full = [&](int i, int kv) {
      return __all_sync(~0u, kCoded ? wait(&bars->op_full[op(i, kv)], (kv ? i / Sh::kVOps : i) & 1, dead)
                                    : wait(&bars->slot_full[slot_of(i, kv, 0)], round_of(i, kv) & 1, dead));
    };
    auto release = [&](int i, int kv) {
      tc::mma_commit(kCoded ? &bars->op_free[op(i, kv)] : &bars->slot_free[slot_of(i, kv, 0)]);
    };
    const uint64_t q_desc = tc::smem_desc(q_addr, 16, 1024, 2), p_desc = tc::smem_desc(p_addr, 16, 8 * N * 2, kSwizzle);
    auto scores = [&](int i) {
      if (!full(i, 0)) return false;
      tc::fence_after_sync();
      const uint64_t k_desc = tc::smem_desc(operand(i, 0), 16, 1024, 2);
      if (tc::elect_one()) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k)         // addresses in descriptors count 16 bytes
          tc::mma_bf16(tmem + (i & 1) * N, k_desc + (k / 4 * Sh::kBlock + k % 4 * 32) / 16,
                       q_desc + (k / 4 * (N * 128) + k % 4 * 32) / 16, kIdS, k > 0);
        tc::mma_commit(&bars->s_full[i & 1]);
        release(i, 0);
      }
      __syncwarp();
      return true;
    };
    bool ok = scores(0);
    for (int i = 0; i < n_tiles && ok; ++i) {
      if (i + 1 < n_tiles) ok = scores(i + 1);
      if (ok) ok = full(i, 1);
      if (ok) ok = __all_sync(~0u, wait(&bars->p_full[i & 1], i / 2 & 1, dead));
      if (!ok) break;
      tc::fence_after_sync();
      const uint64_t v_desc = tc::smem_desc(operand(i, 1), Sh::kBlock, 1024, 2);
      if (tc::elect_one()) {
#pragma unroll
        for (int g = 0; g < Sh::kGroups; ++g)
#pragma unroll
          for (int k = 0; k < TT / 16; ++k)
#pragma unroll
            for (int y = 0; y < Sh::kPTerms; ++y)
              tc::mma_bf16(tmem + (2 + g) * N, v_desc + (2 * g * Sh::kBlock + k * 2048) / 16,
                           p_desc + (i % Sh::kPs * Sh::kP + y * Sh::kPTerm + k * (16 * N * 2)) / 16, kIdO, i > 0 || k > 0 || y > 0);
        release(i, 1);
        tc::mma_commit(&bars->pv_done[i & 1]);   // last: whoever sees it knows that every other arrival is in
      }
      __syncwarp();
    }
    if (!ok) {                                   // products in flight end before tensor memory is released
      if (tc::elect_one()) tc::mma_commit(&bars->drain);
      wait(&bars->drain, 0, nullptr);
    }
    __syncwarp();
  } else if (warp < 4 * Sh::kWGs) {
    // ------------------------------------------------------------------------------- softmax ---
    const int wg = warp / 4, tid = threadIdx.x & 127, bar = 1 + wg, rows0 = wg * R;
    const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);            // lane 32 * (warp % 4) in bits 16 ..
    float l[R] = {}, high[R];                      // the thread's tokens' sum, and maximum less the reference
#pragma unroll
    for (int n = 0; n < R; ++n) high[n] = -INFINITY;
    uint32_t unset = (1u << R) - 1;                // rows that have seen no score yet (their reference is 0)
    bool ok = true;
    for (int i = 0; i < n_tiles; ++i) {
      ok = wait<kCoded>(&bars->s_full[i & 1], i / 2 & 1, dead);
      ok = __all_sync(~0u, ok);
      tc::fence_after_sync();
      const int t = t0 + i * TT + tid, node = t - before;
      const uint32_t bad = absent_of[i & 15];
      const bool absent = t >= sp.len || (bad >> (tid / 16) & 1);
      const bool tail = t0 + (i + 1) * TT > before;
      float x[R];
      tc::tmem_ld<R>(lanes + (i & 1) * N + rows0, x);
      tc::tmem_ld_wait();
#pragma unroll
      for (int n = 0; n < R; n += 4) {             // the scores less the references
        const float4 r = *reinterpret_cast<const float4*>(row_r + rows0 + n);
        const float2 f = make_float2(kToLog2, kToLog2);
        const float2 a = fma2(make_float2(x[n], x[n + 1]), f, make_float2(r.x, r.y));
        const float2 b = fma2(make_float2(x[n + 2], x[n + 3]), f, make_float2(r.z, r.w));
        x[n] = a.x, x[n + 1] = a.y, x[n + 2] = b.x, x[n + 3] = b.y;
      }
      if (tail || bad) {
        const uint32_t* half = reinterpret_cast<const uint32_t*>(words + rows0) + (node >> 5 & 1);
        const uint32_t bit = node >= 0 && !absent ? 1u << (node & 31) : 0u;   // 0: every row sees the token, or none
        const uint32_t none = absent ? 0u : ~0u;
#pragma unroll
        for (int n = 0; n < R; ++n) x[n] = (half[2 * n] & bit) == bit && none ? x[n] : -INFINITY;
      }
      float most = -INFINITY;
#pragma unroll
      for (int n = 0; n < R; ++n) most = fmaxf(most, x[n]);
      bool move = most > kSlack || !ok;
      if (unset) {
#pragma unroll
        for (int n = 0; n < R; ++n) move |= (unset >> n & 1) && x[n] > -INFINITY;
      }
      if (bar_or(bar, 128, move)) {
        if (i) ok &= wait(&bars->pv_done[(i - 1) & 1], (i - 1) / 2 & 1, dead);   // O is whole
        tc::fence_after_sync();
        Exchange& ex = exchanges[wg];
        if (tid < R) ex.most[tid] = order_of(-INFINITY);
        if (bar_or(bar, 128, !ok)) break;
        // move the references of the rows with such a score to this tile's largest
        float mine = -INFINITY;                    // lane n: the warp's largest of row n
#pragma unroll
        for (int n = 0; n < R; ++n) {
          const float v = warp_max(x[n]);
          if (lane == n) mine = v;
        }
        if (lane < R) atomicMax(&ex.most[lane], order_of(mine));
        bar_sync(bar);
        if (tid < 32) {
          bool moves = false;
          if (tid < R) {
            const float by = of_order(ex.most[tid]);
            // (not to +inf: the row's sums are then infinities or NaN, and its maximum stays what it is)
            moves = by > (unset >> tid & 1 ? -INFINITY : kSlack) && by < INFINITY;
            ex.shift[tid] = moves ? by : 0.f;
            if (moves) row_r[rows0 + tid] -= by;
          }
          const uint32_t moved = __ballot_sync(~0u, moves);
          if (tid == 0) ex.moved = moved;
        }
        bar_sync(bar);                             // (the next move's first barriers keep it from what is read here)
        const uint32_t moved = ex.moved, first = unset & moved;
        unset &= ~moved;
        auto scale_of = [&](int n) { return first >> n & 1 ? 0.f : exp2_fast(-ex.shift[n]); };
#pragma unroll
        for (int n = 0; n < R; ++n) {
          x[n] -= ex.shift[n];
          l[n] *= scale_of(n);
          if ((moved >> n & 1) && high[n] < INFINITY) high[n] = -INFINITY;   // all before is below this tile's largest
        }
        if (i) {
#pragma unroll 1
          for (int g = 0; g < Sh::kGroups; ++g) {
#pragma unroll 1
            for (int c = 0; c < R; c += 8) {
              const uint32_t at = lanes + (2 + g) * N + rows0 + c;
              float v[8];
              tc::tmem_ld<8>(at, v);
              tc::tmem_ld_wait();
#pragma unroll
              for (int n = 0; n < 8; ++n) v[n] *= scale_of(c + n);
              tc::tmem_st8(at, v);
            }
          }
          tc::tmem_st_wait();
        }
      }
      uint32_t w[Sh::kPTerms][R / 2];
#pragma unroll
      for (int n = 0; n < R; n += 2) {
        float2 p = make_float2(exp2_fast(x[n]), exp2_fast(x[n + 1]));
        high[n] = max_nan(high[n], x[n]), high[n + 1] = max_nan(high[n + 1], x[n + 1]);
        const float2 sum = add2(make_float2(l[n], l[n + 1]), p);
        l[n] = sum.x, l[n + 1] = sum.y;
        // (2^kBase as part of the references would take a bit of 2^-20 from the scores)
        p = mul2(p, make_float2(1.f / kUnbase, 1.f / kUnbase));
#pragma unroll
        for (int y = 0; y < Sh::kPTerms; ++y) {
          w[y][n / 2] = pack_bf16x2(p.x, p.y);
          const float2 u = unpack_bf16x2(w[y][n / 2]);
          p = add2(p, make_float2(-u.x, -u.y));
        }
      }
      if (i >= Sh::kPs) ok = wait(&bars->pv_done[(i - Sh::kPs) & 1], (i - Sh::kPs) / 2 & 1, dead);   // P's place is free
      ok = __all_sync(~0u, ok);
      // the token's rows, 16 bytes at a time; the swizzle xors their place with the address's bits 7 ..
      unsigned char* p_at = p_op + i % Sh::kPs * Sh::kP + tid * (N * 2);
      const int turn = N == 16 ? tid >> 2 & 1 : (N == 32 ? tid >> 1 & 3 : tid & 7);
#pragma unroll
      for (int z = 0; z < Sh::kPTerms; ++z)
#pragma unroll
        for (int y = 0; y < 2; ++y)
          *reinterpret_cast<uint4*>(p_at + z * Sh::kPTerm + (((rows0 / 8 + y) ^ turn) << 4)) =
              make_uint4(w[z][4 * y], w[z][4 * y + 1], w[z][4 * y + 2], w[z][4 * y + 3]);
      // Behind the last token V's operand holds whatever the page holds (decoders write zeros there), and a
      // drafted token's infinities and NaN are for some rows only: zeros take their place.
      if (wg == 0 && (tail || (bad && !kCoded))) {
        // (The operand's barrier is in this tile's phase, or the one before, only when the last tile's is used.)
        if (i) ok &= wait(&bars->pv_done[(i - 1) & 1], (i - 1) / 2 & 1, dead);
        ok &= wait(kCoded ? &bars->op_full[1 + i % Sh::kVOps] : &bars->slot_full[slot_of(i, 1, 0)],
                   (kCoded ? i / Sh::kVOps : round_of(i, 1)) & 1, dead);
        ok = __all_sync(~0u, ok);
        unsigned char* v = kCoded ? v_op + i % Sh::kVOps * Sh::kOp : slots + slot_of(i, 1, 0) * Sh::kSlot;
        const int base = t0 + i * TT, held = min(sp.len - base, TT);
        if (!kCoded) {
          const int from = bad ? 0 : held;
          for (int y = tid; y < (TT - from) * (D / 8); y += 128) {
            const int tok = from + y / (D / 8), c = y % (D / 8);
            if (tok >= held || (bad >> (tok / 16) & 1))
              *reinterpret_cast<uint4*>(v + c / 8 * Sh::kBlock + tok * 128 + c % 8 * 16) = make_uint4(0, 0, 0, 0);
          }
        }
        const int from = max(before - base, 0);
        for (int y = tid; (!kCoded || *odd_tile) && y < (held - from) * (D / 8); y += 128) {
          const int tok = from + y / (D / 8), c = y % (D / 8);
          uint4* at = reinterpret_cast<uint4*>(v + c / 8 * Sh::kBlock + tok * 128 + c % 8 * 16);
          uint32_t u[4] = {at->x, at->y, at->z, at->w};
          if ((bad >> (tok / 16) & 1) || !(odd2(u[0]) || odd2(u[1]) || odd2(u[2]) || odd2(u[3])))
            continue;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (odd2(u[e] & 0xFFFFu)) u[e] &= 0xFFFF0000u;
            if (odd2(u[e] & 0xFFFF0000u)) u[e] &= 0xFFFFu;
          }
          *at = make_uint4(u[0], u[1], u[2], u[3]);
          const int j = base + tok - before;
          atomicOr(odd_nodes + (j >> 5), 1u << (j & 31));
        }
      }
      tc::fence_proxy_async();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&bars->p_full[i & 1]);   // (one arrival a warp: a thread's each took turns)
    }
    let_next_start();
    if (ok) ok = wait(&bars->pv_done[(n_tiles - 1) & 1], (n_tiles - 1) / 2 & 1, dead);
    if (bar_or(5, 128 * Sh::kWGs, !ok || *dead)) {
      if (tid == 0) atomicCAS(a.status, 0u, (unsigned int)TACTKV_TIMEOUT);
    } else {
      // ---- the rows' true maxima and sums ----
      tc::fence_after_sync();
      const float above = reduce_rows<true>(high);
      const float total = reduce_rows<false>(l);
      if (lane < R) {
        ends[(wg * 4 + (warp & 3)) * 2 * R + lane] = above;
        ends[(wg * 4 + (warp & 3)) * 2 * R + R + lane] = total;
      }
      bar_sync(bar);
      if (tid < R) {
        float m = -INFINITY, sum = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          m = max_nan(m, ends[(wg * 4 + w) * 2 * R + tid]);
          sum += ends[(wg * 4 + w) * 2 * R + R + tid];
        }
        const float to = m == -INFINITY ? 0.f : exp2f(-m);
        row_ml[rows0 + tid] = make_float2(m == -INFINITY ? m : m - row_r[rows0 + tid], sum * to);
        row_f[rows0 + tid] = to;                   // of the row's sums, which stay times 2^kBase
      }
      bar_sync(bar);
      float* sums = reinterpret_cast<float*>(kCoded ? smem : slots);
#pragma unroll
      for (int g = 0; g < Sh::kGroups; ++g) {
        float o[R];
        tc::tmem_ld<R>(lanes + (2 + g) * N + rows0, o);
        tc::tmem_ld_wait();
        if (g * 128 + tid < D) {
#pragma unroll
          for (int n = 0; n < R; ++n) sums[(rows0 + n) * (D + 4) + g * 128 + tid] = o[n] * row_f[rows0 + n];
        }
      }
      // Infinities and NaN of drafted tokens, for the rows that see them (rare): p by one thread a row.
      for (int j = 0; (odd_nodes[0] | odd_nodes[1]) && j < sp.rows; ++j) {
        if (!(odd_nodes[j >> 5] >> (j & 31) & 1)) continue;
        const int t = before + j;
        if (t < t0 || t >= t0 + n_tiles * TT) continue;
        const int page = __ldg(a.b.table + (long long)seq * a.b.max_pages + (t >> a.c.page_log2));
        const long long at = (((long long)page * a.c.heads + head) << a.c.page_log2) + (t & ((1 << a.c.page_log2) - 1));
        float* p_row = ends + wg * 4 * 2 * R;
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
      // eight threads to a row
      const int n = rows0 + tid / 8, row = row0 + n;
      if (row < M) {
        const float2 ml = row_ml[n];
        const float* from = sums + n * (D + 4) + tid % 8 * 4;
        if (parts.count == 1) {
          const long long at = (long long)(sp.first + row / G) * a.q_heads + head * G + row % G;
          const RowEnd e = end_row(a, at, ml.x, ml.y, tid % 8 == 0);
#pragma unroll
          for (int k = 0; k < D / 32; ++k)
            finish4<false>(a, at, tid % 8 * 4 + 32 * k, *reinterpret_cast<const float4*>(from + 32 * k), e);
        } else {
          const long long to = ((long long)part * gridDim.z * gridDim.y + seq * gridDim.y + blockIdx.y) * N + n;
#pragma unroll
          for (int k = 0; k < D / 32; ++k)
            *reinterpret_cast<float4*>(parts.o + to * D + tid % 8 * 4 + 32 * k) = *reinterpret_cast<const float4*>(from + 32 * k);
          if (tid % 8 == 0) parts.ml[to] = ml;
        }
      }
    }
    tc::fence_before_sync();
  } else if constexpr (kCoded) {
    // ------------------------------------------------------------------------------ decoders ---
    // A lane takes a group of 32 values at a time.  Eight lanes take four tokens' two groups of a 64-column block, and
    // odd tokens their halves in the other order, so that stores of 16 bytes never meet in a bank.
    // Four groups: for K and for V, for a tile's first 64 tokens and for the rest.
    constexpr int kAll = 8 * Sh::kDecoders, kGroupsRow = D / kGroup;
    constexpr int kItems = Sh::kPart / 4 * Sh::kBlocks;                    // of eight lanes, in a slot
    constexpr int kPasses = kItems / (kAll / 8);
    const int of = threadIdx.x - 32 * (kIssuer + 1), kv = of / kAll / 2, half = of / kAll % 2, me = of % kAll;
    // A lane's block, group and token modulo 8 are the same in every pass, and with them all of its offsets but for constants.
    constexpr int kStep = kAll / 8 / Sh::kBlocks * 4;                      // tokens from pass to pass
    static_assert(kAll / 8 % Sh::kBlocks == 0 && kStep % 8 == 0 && kItems % (kAll / 8) == 0, "");
    struct Place {
      int tok, g, raw, scale, out, chunk[4];
    };
    auto place_of = [&](int item) {
      Place p;
      const int block = item % Sh::kBlocks, sub = me % 2;
      p.tok = item / Sh::kBlocks * 4 + me % 8 / 2;
      p.g = block * 2 + sub;
      p.raw = p.tok * Sh::kRow + p.g * (Sh::kRow / kGroupsRow);
      p.scale = Sh::kRaw + p.tok * kGroupsRow + p.g;
      p.out = block * Sh::kBlock + p.tok * 128;
#pragma unroll
      for (int y = 0; y < 4; ++y) p.chunk[y] = ((sub * 4 + (FMT == kFp8 ? y ^ (p.tok & 1) * 2 : y)) ^ (p.tok & 7)) * 16;
      return p;
    };
    // One group: its codes, scaled, to the operand.  Returns whether it holds an infinity or NaN, if asked to look.
    auto decode = [&](const unsigned char* raw, unsigned char* out, const Place& p, int pass, bool absent, bool look) {
      const float s = absent ? 0.f : scale_value(raw[p.scale + pass * kStep * kGroupsRow]);
      const float2 f = make_float2(s, s);
      const unsigned char* from = raw + p.raw + pass * kStep * Sh::kRow;
      unsigned char* to = out + p.out + pass * kStep * 128;
      bool odd = false;
#pragma unroll
      for (int y = 0; y < (FMT == kFp8 ? 2 : 1); ++y) {   // the half that the lane takes first alternates with its token
        uint4 w = *reinterpret_cast<const uint4*>(from + (FMT == kFp8 ? (y ^ (p.tok & 1)) * 16 : 0));
        if (absent) w = make_uint4(0, 0, 0, 0);
        const uint32_t in[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int c = 0; c < (FMT == kFp8 ? 2 : 4); ++c) {
          uint32_t h[4];
          if constexpr (FMT == kFp8) {
            unpack_e4m3x4(in[2 * c], h[0], h[1]);
            unpack_e4m3x4(in[2 * c + 1], h[2], h[3]);
          } else {
            unpack_e2m1x8(in[c], h);
          }
#pragma unroll
          for (int z = 0; z < 4; ++z) h[z] = scaled2(h[z], f);
          *reinterpret_cast<uint4*>(to + p.chunk[FMT == kFp8 ? 2 * y + c : c]) = make_uint4(h[0], h[1], h[2], h[3]);
          if (look) odd |= odd2(h[0]) || odd2(h[1]) || odd2(h[2]) || odd2(h[3]);
        }
      }
      return odd;
    };
    const Place mine = place_of(me / 8);
    bool ok = true;
    for (int i = 0; i < n_tiles; ++i) {
      const int slot = slot_of(i, kv, half);
      const int op = kv ? 1 + i % Sh::kVOps : 0, turn = kv ? i / Sh::kVOps : i;
      const int t_half = t0 + i * TT + half * Sh::kPart, held = sp.len - t_half;
      ok = wait<true>(&bars->slot_full[slot], round_of(i, kv) & 1, dead);
      if (turn) ok = ok && wait<true>(&bars->op_free[op], (turn - 1) & 1, dead);
      if (!__all_sync(~0u, ok)) break;
      const uint32_t bad = absent_of[i & 15] >> (half * (Sh::kPart / 16)) & ((1u << Sh::kPart / 16) - 1);
      const unsigned char* raw = slots + slot * Sh::kSlot;
      unsigned char* out = k_op + op * Sh::kOp + half * Sh::kPart * 128;
      const bool drafted = kv && t_half + Sh::kPart > before;
      if (held >= Sh::kPart && !bad && !drafted) {
#pragma unroll
        for (int pass = 0; pass < kPasses; ++pass) decode(raw, out, mine, pass, false, false);
      } else {
        bool odd = false;
        for (int pass = 0; pass < kPasses; ++pass) {
          const int item = me / 8 + pass * (kAll / 8);
          const Place p = place_of(item);
          const bool absent = p.tok >= held || (bad >> (p.tok / 16) & 1), look = drafted && t_half + p.tok >= before;
          odd |= decode(raw, out, p, 0, absent, look) && look && !absent;
        }
        if (odd) *odd_tile = 1;
      }
      tc::fence_proxy_async();
      __syncwarp();
      if (lane == 0) {
        tc::mbar_arrive(&bars->op_full[op]);
        tc::mbar_arrive(&bars->slot_free[slot]);
      }
    }
  }
  __syncthreads();
  if (warp == kIssuer) {
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
cudaError_t launch(const AttnArgs& a, Parts& p, cudaStream_t st) {
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
  plan(a, N, kSms * Sh::kCtas, 2 * TT, p);   // (two tiles: 8.3 us whole, 8.8 in parts)
  tc_kernel<FMT, N><<<dim3(p.count, a.c.heads * p.tiles, a.b.n_seqs), Sh::kThreads, Sh::kSmem, st>>>(a, p, maps[0], maps[1]);
  return cudaGetLastError();
}
template <int FMT>
cudaError_t launch(const AttnArgs& a, Parts& p, cudaStream_t st) {
  // The narrowest tile that takes all rows (64 sequences x 4 heads x 8000 tokens, 8 bits): 16 rows in 64 columns take 183
  // us, in 16 columns 143; 64 rows in two tiles of 32, which decode K and V twice, 297, in one 185.
  const int rows = a.max_rows * (a.q_heads / a.c.heads);
  if (rows <= 16) return launch<FMT, 16>(a, p, st);
  if (rows <= 32 || D > kWideDim) return launch<FMT, 32>(a, p, st);
  if constexpr (D <= kWideDim) return launch<FMT, 64>(a, p, st);
  return cudaErrorInvalidValue;
}

}  // namespace

#define TACTKV_CAT_(x, y) x##y
#define TACTKV_CAT(x, y) TACTKV_CAT_(x, y)
cudaError_t TACTKV_CAT(launch_tc_, TACTKV_TEXT_D)(int fmt, const AttnArgs& a, Parts& p, cudaStream_t st) {
  return fmt == kBf16 ? launch<kBf16>(a, p, st) : (fmt == kFp8 ? launch<kFp8>(a, p, st) : launch<kFp4>(a, p, st));
}

}  // namespace text
}  // namespace tactkv

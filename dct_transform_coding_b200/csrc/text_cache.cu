// The text cache's writing and reading kernels (include/tactkv.h, "Text K/V").
//
// append: codes = RNE(x / 2^e), e = min { e : amax <= MAX 2^e } over each 32 values of a row;
// read:   x = code * 2^e.
// Both are copies with a few instructions per value: HBM bound for long prompts (append of 39k rows of 8 x 128, bfloat16
// in, 4-bit codes and the values out: 68 us, 5.3 TB/s; read of 15k rows of 4 x 256 at 8 bits: 22.6 us, 4.8 TB/s),
// and for a decode step bound by the chain row -> sequence -> page -> address of dependent loads.  One warp
// takes 256 values of a row's K and the same 256 of its V: a lane has 8 neighbouring values (one 16-byte load of
// bfloat16), four lanes a group of 32, so a group's largest magnitude takes two shuffles and all stores of a warp
// are whole segments.
#include <climits>

#include "text.cuh"

namespace tactkv {
namespace text {
namespace {

constexpr int kThreads = 256;
constexpr int kItem = 256;   // values of K and of V per warp

// Eight neighbouring values from p, as they lie there: 16-byte loads, or two values at a time where the alignment allows
// no more.
template <bool F32, bool VEC>
__device__ __forceinline__ void load8(const void* p, long long at, uint32_t (&w)[F32 ? 8 : 4]) {
  constexpr int kWords = F32 ? 8 : 4, kBytes = F32 ? 4 : 2;
  const unsigned char* q = static_cast<const unsigned char*>(p) + at * kBytes;
#pragma unroll
  for (int i = 0; i < kWords; i += VEC ? 4 : (F32 ? 2 : 1)) {
    if constexpr (VEC) {
      const uint4 v = *reinterpret_cast<const uint4*>(q + 4 * i);
      w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
    } else if constexpr (F32) {
      const uint2 v = *reinterpret_cast<const uint2*>(q + 4 * i);
      w[i] = v.x, w[i + 1] = v.y;
    } else {
      w[i] = *reinterpret_cast<const uint32_t*>(q + 4 * i);
    }
  }
}
template <bool F32>
__device__ __forceinline__ void values8(const uint32_t (&w)[F32 ? 8 : 4], float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = F32 ? make_float2(__uint_as_float(w[F32 ? 2 * i : 0]), __uint_as_float(w[F32 ? 2 * i + 1 : 0])) : unpack_bf16x2(w[i]);
    x[2 * i] = v.x, x[2 * i + 1] = v.y;
  }
}
// The bits of the largest magnitude of eight values (above all numbers' for an infinity or NaN), as float32's.
template <bool F32>
__device__ __forceinline__ uint32_t amax8(const uint32_t (&w)[F32 ? 8 : 4]) {
  if constexpr (F32) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, w[i] & 0x7FFFFFFFu);
    return m;
  } else {
    const uint32_t m = __vmaxu2(__vmaxu2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu), __vmaxu2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
    return max(m << 16, m & 0xFFFF0000u);
  }
}
template <bool F32, bool VEC>
__device__ __forceinline__ void store8(void* p, long long at, const float (&x)[8]) {
  if constexpr (F32) {
    float* q = static_cast<float*>(p) + at;
#pragma unroll
    for (int i = 0; i < 8; i += VEC ? 4 : 2) {
      if constexpr (VEC) *reinterpret_cast<float4*>(q + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
      else *reinterpret_cast<float2*>(q + i) = make_float2(x[i], x[i + 1]);
    }
  } else {
    __nv_bfloat16* q = static_cast<__nv_bfloat16*>(p) + at;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
    if constexpr (VEC) {
      *reinterpret_cast<uint4*>(q) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) *reinterpret_cast<uint32_t*>(q + 2 * i) = w[i];
    }
  }
}
// The codes of eight neighbouring values: 16, 8 or 4 bytes at p.
template <int FMT>
__device__ __forceinline__ void load_codes(const unsigned char* p, uint32_t (&w)[4]) {
  if constexpr (FMT == kBf16) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else if constexpr (FMT == kFp8) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}
template <int FMT>
__device__ __forceinline__ void store_codes(unsigned char* p, const uint32_t (&w)[4]) {
  if constexpr (FMT == kBf16) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  else if constexpr (FMT == kFp8) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  else *reinterpret_cast<uint32_t*>(p) = w[0];
}

// Where a row's token stands: the index of (page, head 0, token) among all tokens, or -1 (recorded where it is
// an error; a row behind the last sequence is none: *owned is then false).
__device__ __forceinline__ long long place_of(const Cache& c, const Batch& b, int row, unsigned int* status, bool* owned) {
  const int s = find_seq(b, row);
  *owned = s < b.n_seqs;
  if (!*owned) return -1;
  const Span p = span_of(b, c.page_log2, s, INT_MAX, INT_MAX);
  const int i = row - p.first;
  long long at = -1;
  if (p.ok && i >= 0 && i < p.rows) {
    const int t = p.len - p.rows + i;
    const int page = __ldg(b.table + (long long)s * b.max_pages + (t >> c.page_log2));
    if (page >= 0 && page < c.n_pages)
      at = ((long long)page * c.heads << c.page_log2) + (t & ((1 << c.page_log2) - 1));
  }
  if (at < 0 && (threadIdx.x & 31) == 0) report(status);
  return at;
}

// e / head_dim for e < 65536, inverse = ceil(2^32 / head_dim): the product is too large by less than e * 256 / 2^32.
__device__ __forceinline__ int head_of(int e, uint32_t inverse) { return (int)__umulhi((uint32_t)e, inverse); }

// PER items of a row to a warp: 1 where rows are few and every warp counts, more where there are enough, so that a
// row is looked up once for them and their loads are under way together.
template <int FMT, bool F32, bool VEC, int PER>
__global__ void __launch_bounds__(kThreads) append_kernel(const Cache c, const Batch b, const void* k, const void* v,
                                                          long long token_stride, long long head_stride,
                                                          void* k_values, void* v_values, unsigned int* status,
                                                          int items, uint32_t inverse) {
  const long long unit = (long long)blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
  const int row = (int)(unit / items);           // items: of a row, PER at a time
  if (row >= b.n_rows) return;
  const int e0 = (int)(unit % items) * (PER * kItem) + (threadIdx.x & 31) * 8;
  const int width = c.heads * c.head_dim;
  uint32_t in[PER][2][F32 ? 8 : 4];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = e0 + i * kItem;                // whole groups of four lanes are within the row: width is a multiple of 32
    if (e < width) {
      const int head = head_of(e, inverse);
      const long long from = row * token_stride + head * head_stride + (e - head * c.head_dim);
      load8<F32, VEC>(k, from, in[i][0]);
      load8<F32, VEC>(v, from, in[i][1]);
    }
  }
  bool owned;
  const long long first = place_of(c, b, row, status, &owned);
  if (!owned || first < 0) return;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = e0 + i * kItem, head = head_of(e, inverse), d = e - head * c.head_dim;
    const bool mine = e < width;
    const long long at = first + ((long long)head << c.page_log2);
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      uint32_t w[4], s = 0;
      float x[8];
      values8<F32>(in[i][kv], x);
      if constexpr (FMT == kBf16) {
#pragma unroll
        for (int y = 0; y < 4; ++y) w[y] = F32 ? pack_bf16x2(x[2 * y], x[2 * y + 1]) : in[i][kv][y];
      } else {
        uint32_t amax = mine ? amax8<F32>(in[i][kv]) : 0u;
        amax = max(amax, __shfl_xor_sync(~0u, amax, 1));
        amax = max(amax, __shfl_xor_sync(~0u, amax, 2));
        s = scale_byte<FMT>(amax);
        const float f = scale_inverse(s);
#pragma unroll
        for (int y = 0; y < 8; ++y) x[y] *= f;
        if constexpr (FMT == kFp8) {
          w[0] = s == 255u ? 0u : pack_e4m3x4(x[0], x[1], x[2], x[3]);
          w[1] = s == 255u ? 0u : pack_e4m3x4(x[4], x[5], x[6], x[7]);
        } else {
          // The shuffle (of a lane's own word) stands between this packing and the unpacking of the values below: taken
          // together nvcc 12.9 compiles them so that the word's upper bytes are lost, and so are the codes' where the
          // bytes meet in 16-bit halves.  (Values by integer operations instead: 39k rows of 8 x 128 67 against 61 us.)
          w[0] = __shfl_sync(~0u, s == 255u ? 0u : pack_e2m1x8(x), threadIdx.x & 31);
        }
        if (mine && (threadIdx.x & 3) == 0) c.scales[kv][at * (c.head_dim / kGroup) + d / kGroup] = (unsigned char)s;
      }
      if (mine) {
        store_codes<FMT>(c.pages[kv] + (at * c.head_dim + d) * code_bits(FMT) / 8, w);
        void* out = kv ? v_values : k_values;
        if (out) {
          float y[8];
          decode8<FMT>(w, s, y);
          store8<F32, true>(out, (long long)row * width + e, y);
        }
      }
    }
  }
}

template <int FMT, bool F32, bool VEC, int PER>
__global__ void __launch_bounds__(kThreads) read_kernel(const Cache c, const Batch b, void* k, void* v,
                                                        long long token_stride, long long head_stride,
                                                        unsigned int* status, int items, uint32_t inverse) {
  const long long unit = (long long)blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
  const int row = (int)(unit / items);
  if (row >= b.n_rows) return;
  const int e0 = (int)(unit % items) * (PER * kItem) + (threadIdx.x & 31) * 8, width = c.heads * c.head_dim;
  bool owned;
  const long long first = place_of(c, b, row, status, &owned);
  if (!owned) return;
  uint32_t w[PER][2][4] = {}, s[PER][2] = {};
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = e0 + i * kItem, head = head_of(e, inverse), d = e - head * c.head_dim;
    const long long at = first + ((long long)head << c.page_log2);
    if (first >= 0 && e < width) {
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        load_codes<FMT>(c.pages[kv] + (at * c.head_dim + d) * code_bits(FMT) / 8, w[i][kv]);
        if constexpr (FMT != kBf16) s[i][kv] = c.scales[kv][at * (c.head_dim / kGroup) + d / kGroup];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = e0 + i * kItem;
    if (e >= width) break;
    const int head = head_of(e, inverse);
    const long long to = row * token_stride + head * head_stride + (e - head * c.head_dim);
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      float x[8];
      decode8<FMT>(w[i][kv], s[i][kv], x);
      store8<F32, VEC>(kv ? v : k, to, x);
    }
  }
}

bool wide(bool f32, const void* k, const void* v, long long token_stride, long long head_stride) {
  const int per = f32 ? 4 : 8;   // elements in 16 bytes
  return ((uintptr_t)k | (uintptr_t)v) % 16 == 0 && token_stride % per == 0 && head_stride % per == 0;
}

// Warps for all rows, and whether there are enough for several items each.
struct Grid {
  uint32_t inverse;
  int items;
  unsigned blocks;
  bool many;
};
Grid grid_of(const Cache& c, const Batch& b, int many) {
  const int one = (c.heads * c.head_dim + kItem - 1) / kItem;
  Grid g;
  g.inverse = (uint32_t)(((1ull << 32) + c.head_dim - 1) / c.head_dim);
  // One item to a warp up to a GPU full of warps; several from there on: append with two 68 against 82 us (39k rows of 8 x
  // 128), read with four 22.6 against 28.7 (15k rows of 4 x 256).
  g.many = one > 1 && (long long)b.n_rows * one >= 148 * 64;
  g.items = g.many ? (one + many - 1) / many : one;
  g.blocks = (unsigned)(((long long)b.n_rows * g.items + kThreads / 32 - 1) / (kThreads / 32));
  return g;
}

}  // namespace

#define TACTKV_PER(FMT, F32, VEC, MANY) (g.many ? TACTKV_GO(FMT, F32, VEC, MANY) : TACTKV_GO(FMT, F32, VEC, 1))
#define TACTKV_IO(FMT, MANY)                                                       \
  (f32 ? (vec ? TACTKV_PER(FMT, true, true, MANY) : TACTKV_PER(FMT, true, false, MANY))  \
       : (vec ? TACTKV_PER(FMT, false, true, MANY) : TACTKV_PER(FMT, false, false, MANY)))

cudaError_t launch_append(int fmt, bool f32, const Cache& c, const Batch& b, const void* k, const void* v,
                          long long token_stride, long long head_stride, void* k_values, void* v_values,
                          unsigned int* status, cudaStream_t st) {
  const Grid g = grid_of(c, b, 2);
  const bool vec = wide(f32, k, v, token_stride, head_stride);
#define TACTKV_GO(FMT, F32, VEC, PER)                                                                             \
  append_kernel<FMT, F32, VEC, PER><<<g.blocks, kThreads, 0, st>>>(c, b, k, v, token_stride, head_stride, k_values, \
                                                                   v_values, status, g.items, g.inverse)
  if (fmt == kBf16) TACTKV_IO(kBf16, 2);
  else if (fmt == kFp8) TACTKV_IO(kFp8, 2);
  else TACTKV_IO(kFp4, 2);
#undef TACTKV_GO
  return cudaGetLastError();
}

cudaError_t launch_read(int fmt, bool f32, const Cache& c, const Batch& b, void* k, void* v, long long token_stride,
                        long long head_stride, unsigned int* status, cudaStream_t st) {
  const Grid g = grid_of(c, b, 4);
  const bool vec = wide(f32, k, v, token_stride, head_stride);
#define TACTKV_GO(FMT, F32, VEC, PER)                                                                      \
  read_kernel<FMT, F32, VEC, PER><<<g.blocks, kThreads, 0, st>>>(c, b, k, v, token_stride, head_stride,    \
                                                                 status, g.items, g.inverse)
  if (fmt == kBf16) TACTKV_IO(kBf16, 4);
  else if (fmt == kFp8) TACTKV_IO(kFp8, 4);
  else TACTKV_IO(kFp4, 4);
#undef TACTKV_GO
  return cudaGetLastError();
}
#undef TACTKV_IO
#undef TACTKV_PER

}  // namespace text
}  // namespace tactkv

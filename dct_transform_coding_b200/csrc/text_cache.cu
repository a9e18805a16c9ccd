// The text cache's writing and reading kernels (include/tactkv.h, "Text K/V").
//
// append: codes = RNE(x / 2^e), e = min { e : amax <= MAX 2^e } over each 32 values of a row;
// read:   x = code * 2^e.
// Both are copies with a few instructions per value: HBM bound for long prompts, and for a decode step bound
// by the chain row -> sequence -> page -> address of dependent loads.  One warp takes 256 values of a
// row's K and the same 256 of its V: a lane has 8 neighbouring values (one 16-byte load of bfloat16), four
// lanes a group of 32, so a group's largest magnitude takes two shuffles and all stores of a warp are whole
// segments.
#include <climits>

#include "text.cuh"

namespace tactkv {
namespace text {
namespace {

constexpr int kThreads = 256;
constexpr int kItem = 256;   // values of K and of V per warp

// Eight neighbouring values from p: 16-byte loads, or two at a time where the alignment allows no more.
template <bool F32, bool VEC>
__device__ __forceinline__ void load8(const void* p, long long at, float (&x)[8]) {
  if constexpr (F32) {
    const float* q = static_cast<const float*>(p) + at;
#pragma unroll
    for (int i = 0; i < 8; i += VEC ? 4 : 2) {
      if constexpr (VEC) {
        const float4 v = *reinterpret_cast<const float4*>(q + i);
        x[i] = v.x, x[i + 1] = v.y, x[i + 2] = v.z, x[i + 3] = v.w;
      } else {
        const float2 v = *reinterpret_cast<const float2*>(q + i);
        x[i] = v.x, x[i + 1] = v.y;
      }
    }
  } else {
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p) + at;
    uint32_t w[4];
    if constexpr (VEC) {
      const uint4 v = *reinterpret_cast<const uint4*>(q);
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const uint32_t*>(q + 2 * i);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = unpack_bf16x2(w[i]);
      x[2 * i] = v.x, x[2 * i + 1] = v.y;
    }
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

template <int FMT, bool F32, bool VEC>
__global__ void __launch_bounds__(kThreads) append_kernel(const Cache c, const Batch b, const void* k, const void* v,
                                                          long long token_stride, long long head_stride,
                                                          void* k_values, void* v_values, unsigned int* status,
                                                          int items) {
  const long long item = (long long)blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
  const int row = (int)(item / items);
  if (row >= b.n_rows) return;
  const int e = (int)(item % items) * kItem + (threadIdx.x & 31) * 8;
  const int width = c.heads * c.head_dim;
  const bool mine = e < width;                 // whole groups of four lanes: width is a multiple of 32
  const int head = mine ? e / c.head_dim : 0, d = mine ? e % c.head_dim : 0;
  bool owned;
  const long long first = place_of(c, b, row, status, &owned);
  if (!owned || first < 0) return;
  const long long from = row * token_stride + head * head_stride + d;
  float x[2][8];
#pragma unroll
  for (int kv = 0; kv < 2; ++kv)
    if (mine) load8<F32, VEC>(kv ? v : k, from, x[kv]);
  const long long at = first + ((long long)head << c.page_log2);
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    uint32_t w[4], s = 0;
    if constexpr (FMT == kBf16) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(x[kv][2 * i], x[kv][2 * i + 1]);
    } else {
      uint32_t amax = 0;
      if (mine) {
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = max(amax, __float_as_uint(x[kv][i]) & 0x7FFFFFFFu);
      }
      amax = max(amax, __shfl_xor_sync(~0u, amax, 1));
      amax = max(amax, __shfl_xor_sync(~0u, amax, 2));
      s = scale_byte<FMT>(amax);
      const float f = scale_inverse(s);
      float u[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] = s == 255u ? 0.f : x[kv][i] * f;
      if constexpr (FMT == kFp8) {
        w[0] = pack_e4m3x4(u[0], u[1], u[2], u[3]);
        w[1] = pack_e4m3x4(u[4], u[5], u[6], u[7]);
      } else {
        // The shuffle (of a lane's own word) keeps the compiler from folding the unpacking of the values
        // below into this packing: nvcc 12.9 then loses the word's upper bytes.
        w[0] = __shfl_sync(~0u, pack_e2m1x8(u), threadIdx.x & 31);
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

template <int FMT, bool F32, bool VEC>
__global__ void __launch_bounds__(kThreads) read_kernel(const Cache c, const Batch b, void* k, void* v,
                                                        long long token_stride, long long head_stride,
                                                        unsigned int* status, int items) {
  const long long item = (long long)blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
  const int row = (int)(item / items);
  if (row >= b.n_rows) return;
  const int e = (int)(item % items) * kItem + (threadIdx.x & 31) * 8;
  bool owned;
  const long long first = place_of(c, b, row, status, &owned);
  if (!owned || e >= c.heads * c.head_dim) return;
  const int head = e / c.head_dim, d = e % c.head_dim;
  const long long at = first + ((long long)head << c.page_log2);
  uint32_t w[2][4] = {}, s[2] = {};
  if (first >= 0) {
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      load_codes<FMT>(c.pages[kv] + (at * c.head_dim + d) * code_bits(FMT) / 8, w[kv]);
      if constexpr (FMT != kBf16) s[kv] = c.scales[kv][at * (c.head_dim / kGroup) + d / kGroup];
    }
  }
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    float x[8];
    decode8<FMT>(w[kv], s[kv], x);
    store8<F32, VEC>(kv ? v : k, row * token_stride + head * head_stride + d, x);
  }
}

bool wide(bool f32, const void* k, const void* v, long long token_stride, long long head_stride) {
  const int per = f32 ? 4 : 8;   // elements in 16 bytes
  return ((uintptr_t)k | (uintptr_t)v) % 16 == 0 && token_stride % per == 0 && head_stride % per == 0;
}

}  // namespace

cudaError_t launch_append(int fmt, bool f32, const Cache& c, const Batch& b, const void* k, const void* v,
                          long long token_stride, long long head_stride, void* k_values, void* v_values,
                          unsigned int* status, cudaStream_t st) {
  const int items = (c.heads * c.head_dim + kItem - 1) / kItem;
  const long long blocks = ((long long)b.n_rows * items + kThreads / 32 - 1) / (kThreads / 32);
  const bool vec = wide(f32, k, v, token_stride, head_stride);
#define TACTKV_GO(FMT, F32, VEC)                                                                               \
  append_kernel<FMT, F32, VEC><<<(unsigned)blocks, kThreads, 0, st>>>(c, b, k, v, token_stride, head_stride,   \
                                                                      k_values, v_values, status, items)
#define TACTKV_IO(FMT)                                              \
  (f32 ? (vec ? TACTKV_GO(FMT, true, true) : TACTKV_GO(FMT, true, false)) \
       : (vec ? TACTKV_GO(FMT, false, true) : TACTKV_GO(FMT, false, false)))
  if (fmt == kBf16) TACTKV_IO(kBf16);
  else if (fmt == kFp8) TACTKV_IO(kFp8);
  else TACTKV_IO(kFp4);
#undef TACTKV_GO
  return cudaGetLastError();
}

cudaError_t launch_read(int fmt, bool f32, const Cache& c, const Batch& b, void* k, void* v, long long token_stride,
                        long long head_stride, unsigned int* status, cudaStream_t st) {
  const int items = (c.heads * c.head_dim + kItem - 1) / kItem;
  const long long blocks = ((long long)b.n_rows * items + kThreads / 32 - 1) / (kThreads / 32);
  const bool vec = wide(f32, k, v, token_stride, head_stride);
#define TACTKV_GO(FMT, F32, VEC)                                                                             \
  read_kernel<FMT, F32, VEC><<<(unsigned)blocks, kThreads, 0, st>>>(c, b, k, v, token_stride, head_stride,   \
                                                                    status, items)
  if (fmt == kBf16) TACTKV_IO(kBf16);
  else if (fmt == kFp8) TACTKV_IO(kFp8);
  else TACTKV_IO(kFp4);
#undef TACTKV_GO
#undef TACTKV_IO
  return cudaGetLastError();
}

}  // namespace text
}  // namespace tactkv

// Shared device code of the text cache's kernels (internal header): the batch's rows, the pages and the
// codes.  The formats, layouts and calling rules are in include/tactkv.h ("Text K/V").
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace tactkv {
namespace text {

constexpr int kMaxHeadDim = 256;
constexpr int kMaxRows = 64;          // rows of one sequence in an attention call: a tree word's bits
constexpr int kMaxGroup = 16;         // query heads per K/V head
constexpr int kMaxLen = 1 << 30;      // tokens of one sequence in an attention call
constexpr int kGroup = 32;            // values that share a scale

enum Format { kBf16 = TACTKV_TEXT_BF16, kFp8 = TACTKV_TEXT_MXFP8, kFp4 = TACTKV_TEXT_MXFP4 };
__host__ __device__ constexpr int code_bits(int fmt) { return fmt == kBf16 ? 16 : (fmt == kFp8 ? 8 : 4); }

// A cache and a batch as the kernels get them.
struct Cache {
  unsigned char* pages[2];    // K, V
  unsigned char* scales[2];
  long long n_pages;
  int heads, head_dim, page_log2;
};
struct Batch {
  const int* table;
  const int* kv_lens;
  const int* row_starts;
  int n_seqs, n_rows, max_pages;
};

__device__ __forceinline__ void report(unsigned int* status) {
  atomicCAS(status, 0u, (unsigned int)TACTKV_INVALID_ARG);
}

// The sequence that owns row r: how many of row_starts[1 .. n_seqs] are <= r, so n_seqs for the rows
// of a padded batch.  The whole warp calls it; each round compares 32 entries, so 1024 sequences take
// two dependent loads.  Ends, and stays within the array, whatever the entries are.
__device__ __forceinline__ int find_seq(const Batch& b, int r) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = b.n_seqs;
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32;
    const long long i = lo + (lane + 1ll) * step;
    const bool below = i <= hi && __ldg(b.row_starts + i) <= r;
    lo += __popc(__ballot_sync(~0u, below)) * step;
    hi = min(hi, lo + step - 1);
  }
  return lo;
}

// A sequence's rows and length, checked: ok is false (and the error recorded) where they do not fit together.
struct Span {
  int first, rows, len;
  bool ok;
};
__device__ __forceinline__ Span span_of(const Batch& b, int page_log2, int s, long long max_len, int max_rows) {
  Span p;
  p.first = __ldg(b.row_starts + s);
  const int end = __ldg(b.row_starts + s + 1);
  p.len = __ldg(b.kv_lens + s);
  p.rows = end - p.first;
  p.ok = p.first >= 0 && end >= p.first && end <= b.n_rows && p.rows <= max_rows && p.len >= p.rows &&
         p.len <= ((long long)b.max_pages << page_log2) && p.len <= max_len;
  return p;
}

// 2^(s - 127) of a scale byte: exact, 2^-127 a subnormal, NaN for 255.
__device__ __forceinline__ float scale_value(uint32_t s) {
  return __uint_as_float((s << 23) | ((s == 0u || s == 255u) ? 0x400000u : 0u));
}

// The scale byte of a group from the bits of its largest magnitude (the sign bit clear).
//   E4M3: amax <= 448 * 2^e = 1.75 * 2^(e + 8);  E2M1: amax <= 6 * 2^e = 1.5 * 2^(e + 2).
// With amax = 1.f * 2^E the smallest such e is E - 8 + (1.f > 1.75), or E - 2 + (1.f > 1.5); e >= -127,
// which subnormal and zero amax clamp to.
template <int FMT>
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
  if (amax >= 0x7F800000u) return 255u;
  const int E = (int)(amax >> 23) - 127;
  const uint32_t f = amax & 0x7FFFFFu;
  const int e = FMT == kFp8 ? E - 8 + (f > 0x600000u) : E - 2 + (f > 0x400000u);
  return (uint32_t)(max(e, -127) + 127);
}
// 2^(127 - s), the factor that scales by s exactly (0 for the NaN scale, so that its codes are zero).
__device__ __forceinline__ float scale_inverse(uint32_t s) {
  return s == 255u ? 0.f : __uint_as_float((254u - s) << 23 | (s == 254u ? 0x400000u : 0u));
}

__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}
// Eight E2M1 codes, the first in the lowest half byte, to nearest even.
__device__ __forceinline__ uint32_t pack_e2m1x8(const float (&x)[8]) {
  uint32_t w;
  asm("{\n.reg .b8 a, b, c, d;\n"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\ncvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\ncvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      "mov.b32 %0, {a, b, c, d};\n}\n"
      : "=r"(w)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return w;
}
// Eight E2M1 codes as four pairs of half-precision values (exact).
__device__ __forceinline__ void unpack_e2m1x8(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n.reg .b8 a, b, c, d;\nmov.b32 {a, b, c, d}, %4;\n"
      "cvt.rn.f16x2.e2m1x2 %0, a;\ncvt.rn.f16x2.e2m1x2 %1, b;\n"
      "cvt.rn.f16x2.e2m1x2 %2, c;\ncvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
// Two E4M3 codes (16 bits) as float32.
__device__ __forceinline__ float2 unpack_e4m3x2(uint32_t v) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)v, __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ uint32_t pack_bf16x2(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float2 unpack_bf16x2(uint32_t v) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}

// Eight neighbouring values of one token and head from their codes (16, 8 or 4 bytes in w[]).
template <int FMT>
__device__ __forceinline__ void decode8(const uint32_t (&w)[4], uint32_t scale, float (&x)[8]) {
  const float f = FMT == kBf16 ? 1.f : scale_value(scale);
  uint32_t h[4];
  if constexpr (FMT == kFp4) unpack_e2m1x8(w[0], h);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 v;
    if constexpr (FMT == kBf16) v = unpack_bf16x2(w[i]);
    else if constexpr (FMT == kFp8) v = unpack_e4m3x2(w[i / 2] >> (16 * (i & 1)) & 0xFFFFu);
    else v = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    x[2 * i] = FMT == kBf16 ? v.x : v.x * f;
    x[2 * i + 1] = FMT == kBf16 ? v.y : v.y * f;
  }
}

cudaError_t launch_append(int fmt, bool f32, const Cache& c, const Batch& b, const void* k, const void* v,
                          long long token_stride, long long head_stride, void* k_values, void* v_values,
                          unsigned int* status, cudaStream_t st);
cudaError_t launch_read(int fmt, bool f32, const Cache& c, const Batch& b, void* k, void* v, long long token_stride,
                        long long head_stride, unsigned int* status, cudaStream_t st);

struct AttnArgs {
  Cache c;
  Batch b;
  int q_heads, max_rows, max_len;
  const void* q;
  long long q_token, q_head;                   // strides, elements
  const unsigned long long* tree;
  const float *prior_out, *prior_m, *prior_l;
  void* out;
  float *m, *l;
  unsigned int* status;
};
size_t attention_workspace(int head_dim);   // bytes behind the status word
cudaError_t launch_attention(int fmt, bool f32, const AttnArgs& a, void* workspace, cudaStream_t st);

}  // namespace text
}  // namespace tactkv

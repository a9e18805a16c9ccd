/*
 * tactkv.h -- C ABI of the B200 TACT-KV visual-KV transform codec.
 *
 * The operations are those of the TACT-KV summary page ("TACT-KV: Tri-Axis Cosine Transform for
 * Compressing Volumetric KV Caches in Medical VLMs"), section "Methodology in Plain English":
 *   stage 1  the visual K or V of one layer of one sequence is laid out on its (S, H, W) grid;
 *   stage 2  a separable orthonormal 3D DCT-II runs along S, H and W (features untouched);
 *   stage 3  per-bin variances (over all heads x head_dim channels) drive a reverse
 *            water-filling split of the layer's bit budget: b_i = max(0, 1/2 log2(s_i^2/theta)),
 *            theta by bisection, integer rounding, +-1 greedy fix to hit the budget, cap 8 bits;
 *   stage 4  each surviving bin is scaled by its own gain s_i and every coordinate is quantized
 *            with a fixed Lloyd-Max table of a unit Gaussian at the bin's bit width;
 *   decoding reverses the stages (paragraph after stage 4).
 *
 * Terms.  A UNIT is one (sequence, layer, K|V) volume: T = S*H*W tokens by n = heads*head_dim
 * channels.  Token t = (s*H + h)*W + w; channel c = head*head_dim + d.  Frequency bin
 * i = (k_s*H + k_h)*W + k_w, N = T bins.  Nominal budget: bits*N bit slots per channel.
 *
 * Memory.  Every pointer in a unit descriptor and the workspace are DEVICE pointers owned by
 * the caller.  The library allocates nothing.  Its only state is the read-only tables in the CUDA
 * module (constant memory, and 16-byte-aligned copies in global memory that kernels stage into
 * shared memory) and the fixed device scratch array of tactkv_compress_noalloc (below); every other entry
 * point is safe to call from several host threads on different streams provided each call has
 * its own workspace.  Calls are asynchronous on `stream`; a status other than
 * TACTKV_OK means nothing was launched for the failing group of units (earlier groups of the
 * same call may already be queued).  Errors found by the kernels (a corrupt payload) are
 * recorded in the workspace and read back with tactkv_device_status().
 *
 * Payload format (version 1, little-endian), one self-describing blob per unit:
 *   [0, 64)             header: u32 magic 0x31564B54 ("TKV1"), u16 version = 1, u16 flags (the
 *                       unit's flags without TACTKV_FP32_IO),
 *                       i32 layer, kv, S, H, W, heads, head_dim, bits, u32 code_bits (sum b_i,
 *                       or 32*N with TACTKV_NO_QUANT), u32 chan_stride (bytes), u64 total_bytes,
 *                       u32 0, u32 0
 *   [64, +pad16(N))     u8 b[N]          bits of every bin (0..8; 0 = dropped)
 *   then pad16(4N)      f32 sigma[N]     gain of every bin, float32(sqrt(sigma^2)); with
 *                       TACTKV_HEAD_GAIN pad16(4*heads*N) bytes, f32 sigma[heads][N]
 *   then n streams      channel c at offset off_codes + c*chan_stride, chan_stride =
 *                       pad16(ceil(code_bits/8)); stream bit P_i + k is bit k (LSB first) of bin
 *                       i's code, P_i = sum_{j<i} b_j; stream bit q is bit (q&7) of byte q>>3.
 *                       With TACTKV_NO_QUANT a stream holds the N float32 coefficients instead.
 * pad16(x) rounds x up to a multiple of 16.  The gain/rate part is the pages' sum(b_i*d + 32)
 * bits per layer; the b[] bytes are the index the pages add on top of it.
 */
#ifndef TACTKV_H_
#define TACTKV_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

struct CUstream_st; /* cudaStream_t is `struct CUstream_st*`; NULL is the legacy default stream */

typedef enum {
  TACTKV_OK = 0,
  TACTKV_INVALID_ARG = 1,        /* null pointer, n_units < 0, bits outside 1..8, bad flags */
  TACTKV_UNSUPPORTED_SHAPE = 2,  /* an axis length or channel layout the kernels do not cover */
  TACTKV_CAPACITY = 3,           /* payload_capacity below tactkv_payload_bytes() */
  TACTKV_ALIGNMENT = 4,          /* a pointer or stride breaks the alignment rules below */
  TACTKV_CORRUPT_PAYLOAD = 5,    /* (device status) a payload header or allocation is invalid */
  TACTKV_CUDA = 6,               /* a CUDA launch or copy failed */
  TACTKV_WORKSPACE = 7,          /* workspace null or smaller than one unit needs */
  TACTKV_SCRATCH_LIMIT = 8,      /* a unit needs more scratch than tactkv_compress_noalloc has */
  TACTKV_TIMEOUT = 9             /* (device status) a kernel's bounded wait on a tensor-memory copy
                                    or a tensor-core operation expired; its outputs are undefined */
} tactkv_status;

/* flags */
#define TACTKV_NO_QUANT 1u /* transform only: store float32 coefficients (lossless round trip) */
#define TACTKV_FP32_IO  2u /* K/V are float32 instead of bfloat16 */
/* Variants of the summary page's "Main Findings" ablations and of stage 4's shape rotation, all
   recorded in the payload header (decompress must be given the same flags):
     TACTKV_SKIP_S / _H / _W  no DCT along that axis (2-axis, 1-axis and no-DCT transforms);
     TACTKV_UNIFORM_ALLOC     every bin with a nonzero variance gets the nominal bits (no
                              water-filling; the total stays within the budget);
     TACTKV_ROTATE            the fixed shared orthogonal rotation of each bin's shape vector before
                              scalar quantization, undone after dequantization: block-diagonal over
                              the 32-channel groups, H_32 diag(s) / sqrt(32) with H_32 the
                              Sylvester-Hadamard matrix and s_c = -1 exactly when bit 63 of output c
                              of SplitMix64 seeded with 0x544143544B56 is set (ignored with
                              TACTKV_NO_QUANT).  Gains and allocation are unchanged by it;
     TACTKV_HEAD_GAIN         one gain per (bin, head) instead of one per bin: the gain-shape
                              vectors of stage 4 are a bin's head_dim coordinates in one head
                              (the d of stage 4's occupancy sum), each scaled by
                              float32(sqrt(mean over the head's channels of X^2)) and decoded with
                              it (a zero gain scales by 0).  The bit allocation still uses the
                              variance pooled over all channels.  Needs head_dim a multiple of 32;
                              the payload then holds sigma[heads][N] (ignored with TACTKV_NO_QUANT). */
#define TACTKV_SKIP_S        4u
#define TACTKV_SKIP_H        8u
#define TACTKV_SKIP_W       16u
#define TACTKV_UNIFORM_ALLOC 32u
#define TACTKV_ROTATE       64u
#define TACTKV_HEAD_GAIN   128u

typedef struct {
  int32_t layer;          /* recorded in the header, checked by decompress */
  int32_t kv;             /* 0 = K, 1 = V; recorded and checked like layer */
  int32_t S, H, W;        /* token grid; lengths from the supported set below */
  int32_t heads, head_dim;/* n = heads*head_dim channels, n a multiple of 32, head_dim even */
  int32_t bits;           /* nominal bits per element, 1..8 */
  uint32_t flags;         /* TACTKV_NO_QUANT | TACTKV_FP32_IO | the variant flags above */
  const void* kv_in;      /* compress input: element (t, head, d) at
                             kv_in + t*token_stride + head*head_stride + d (elements) */
  void* kv_out;           /* decompress output, same indexing as kv_in */
  int64_t token_stride;   /* in elements; even, > 0 */
  int64_t head_stride;    /* in elements; even */
  void* payload;          /* compress writes, decompress reads; 16-byte aligned */
  size_t payload_capacity;/* bytes available at payload */
} tactkv_unit;

/* Supported shapes: S in {1..16, 20, 24, 28, 32, 40, 48, 56, 64}; H and W in {1..16, 20, 24, 28,
   32} with H*W <= 1024; heads*head_dim a multiple of 32 and at most 65536.  kv_in / kv_out must
   be 4-byte aligned (8-byte with TACTKV_FP32_IO); strides even.  Other shapes return
   TACTKV_UNSUPPORTED_SHAPE. */

/* Worst-case payload size of one unit (every bin budget used): the capacity to provide. */
size_t tactkv_payload_bytes(const tactkv_unit* unit);

/* Workspace bytes that let compress/decompress process the units in as few waves as possible
   (a wave is up to 256 units of one shape).  Any size of at least tactkv_workspace_bytes(units,
   1) works; the units are then processed in more, smaller waves. */
size_t tactkv_workspace_bytes(const tactkv_unit* units, int n_units);

/* Compress every unit: read kv_in, write the payload.  Units with identical shape, bits and
   flags that are adjacent in the array are batched into one set of launches.  Steps: forward
   DCT along S; forward DCT along H and W with per-bin energy sums; per-unit bit allocation and
   gains; quantization of the finished coefficients and bit packing. */
tactkv_status tactkv_compress(const tactkv_unit* units, int n_units, void* workspace,
                              size_t workspace_bytes, struct CUstream_st* stream);

/* Decompress every unit: read the payload, write kv_out (bfloat16, or float32 with
   TACTKV_FP32_IO) with the descriptor's strides.  The payload header must match the
   descriptor (layer, kv, shape, bits, flags); a mismatch or an invalid allocation is recorded
   as TACTKV_CORRUPT_PAYLOAD in the workspace and that unit's output is zero-filled. */
tactkv_status tactkv_decompress(const tactkv_unit* units, int n_units, void* workspace,
                                size_t workspace_bytes, struct CUstream_st* stream);

/* Profiling variants: the same work as tactkv_compress / tactkv_decompress, and, when `events`
   is not NULL, cudaEventRecord(events[k], stream) at the stage boundaries of every wave (so for
   a call that fits in one wave the events bracket each stage).  events[k] are cudaEvent_t
   handles created by the caller; a NULL entry is skipped.
   compress:   0 before the transforms, 1 after the DCTs along S and along H and W (with the
               energy sums) of every unit, 2 after the allocation, 3 after quantization and
               packing.
   decompress: 0 before the payload index, 1 after it, 2 after the inverse DCT along W and H
               (with the decoding), 3 after the inverse DCT along S (with the single-kernel decode
               2 and 3 mark the same point). */
tactkv_status tactkv_compress_profiled(const tactkv_unit* units, int n_units, void* workspace,
                                       size_t workspace_bytes, struct CUstream_st* stream,
                                       void* const* events);
tactkv_status tactkv_decompress_profiled(const tactkv_unit* units, int n_units, void* workspace,
                                         size_t workspace_bytes, struct CUstream_st* stream,
                                         void* const* events);

/* tactkv_compress without a workspace argument, for callers that cannot allocate device memory
   at the point where they compress: code recording a CUDA graph (a cudaMalloc there fails or
   breaks the capture), engines whose device memory is all handed out by their own pool, and
   latency-critical loops where an allocation could synchronize the device.  The TACT-KV pages
   have no counterpart of this call; it only changes where the scratch lives.
   The scratch is a fixed 16 MiB array inside the library's device image, which every GPU that
   loads the library holds until the process exits.  Each unit on its own must fit in it (its
   workspace, tactkv_workspace_bytes of that one unit, at most 16 MiB: e.g. 8x8x8 x 64 channels or
   64x16x16 x 128 channels, not 64x16x16 x 1024); otherwise TACTKV_SCRATCH_LIMIT is returned and
   nothing is launched.  The first call on a device looks the array's address up
   (cudaGetSymbolAddress), so make that first call before any stream capture.  All calls share
   the one array: calls that may overlap on the GPU (different streams, or several host threads)
   race on it and must be serialized by the caller.  Allocates nothing; output is identical to
   tactkv_compress. */
tactkv_status tactkv_compress_noalloc(const tactkv_unit* units, int n_units,
                                      struct CUstream_st* stream);

/* Stage 3 alone ("Methodology in Plain English", stage 3: reverse water-filling of the bit budget
   bits*N over the bins, cap 8 bits): the allocation compress runs, applied to the variances the
   caller gives instead of the ones compress measures.  var: DEVICE array of N = S*H*W doubles,
   var[i] >= 0 the variance of bin i (8-byte aligned; not modified).  Writes into unit->payload
   exactly what compress writes there from its own variances: the header, b[N] (the selection of
   the B = bits*N largest keys var_i * 4^-k, k = 0..7, ties to the lower bin index, every active bin
   at 8 bits when 8*#active <= B; b = 0 where var = 0), sigma[N] = float32(sqrt(var)) and the zero
   padding; the code area is left unspecified.  Only the unit's shape, bits, flags, layer, kv,
   payload and payload_capacity are read.  TACTKV_HEAD_GAIN is refused (TACTKV_INVALID_ARG): its
   gains come from the channels, which this call does not see.  workspace: at least tactkv_workspace_bytes(unit, 1)
   bytes, 256-byte aligned.  Asynchronous on `stream`; one kernel. */
tactkv_status tactkv_allocate(const tactkv_unit* unit, const double* var, void* workspace,
                              size_t workspace_bytes, struct CUstream_st* stream);

/* One decode step of attention over compressed visual K/V (the paragraph after stage 4: decoding
   runs inside the attention computation and the reconstructed cache never exists).  Unit i of
   k_units / v_units is the K / V payload of one (sequence, layer); all 2*n_units descriptors have
   the same shape, bits and flags (quantized, not TACTKV_NO_QUANT), and each unit's kv field must
   match its payload.  Only the payload pointers and the shape fields are read.
     q_heads   query heads, a multiple G of the K/V heads (G <= 16); query head j reads K/V head j/G;
     q         DEVICE float32 [n_units][q_heads][head_dim], the decode step's queries;
     out       DEVICE float32 [n_units][q_heads][head_dim]:
                 out_j = sum_t softmax_t(q_j . K[t] / sqrt(head_dim)) V[t] over the S*H*W visual tokens;
     m, l      DEVICE float32 [n_units][q_heads]: the scores' maximum and sum_t exp(score - m), so
               that a caller can merge these tokens with its bf16 text tokens.
   Limits: n_units <= 128, head_dim a multiple of 32, and shared memory for one slab's stream words
   of a head (head_dim * ((c*H*W + 31)/32 + 3, rounded up to odd) 4-byte words, c = min(8, 2*bits + 2)
   bits per bin; a slab whose codes span more is decoded from the payload directly) and for the
   score volume (S*H*(W rounded up to odd) floats) within 227 KB each; other shapes return
   TACTKV_UNSUPPORTED_SHAPE (every benchmark grid fits).  workspace: at least
   tactkv_attention_workspace_bytes(k_units, n_units, q_heads) bytes, 256-byte aligned.  A corrupt
   payload is recorded as TACTKV_CORRUPT_PAYLOAD (tactkv_device_status) and contributes no
   tokens of its unit: out = 0, m = -inf and l = 0 for that unit's query heads.  Asynchronous on
   `stream`; 5 kernels. */
size_t tactkv_attention_workspace_bytes(const tactkv_unit* k_units, int n_units, int q_heads);
tactkv_status tactkv_attention_decode(const tactkv_unit* k_units, const tactkv_unit* v_units, int n_units,
                                      int q_heads, const float* q, float* out, float* m, float* l,
                                      void* workspace, size_t workspace_bytes,
                                      struct CUstream_st* stream);

/* ------------------------------------------------------------------------------------------------
   Text K/V.  The codec compresses the visual K/V of a finished prefill; the text K/V of the same
   layer grows by the tokens that a decode step adds.  The three calls below keep it in a paged cache
   (as bfloat16, or quantized as it is written), read it back, and attend to it, merging the
   (out, m, l) partial that tactkv_attention_decode returns for the visual tokens.

   Formats.  A token's head_dim values in one K/V head are held as
     TACTKV_TEXT_BF16   bfloat16 (float32 input is rounded to nearest even);
     TACTKV_TEXT_MXFP8  E4M3 codes, one byte each;
     TACTKV_TEXT_MXFP4  E2M1 codes, two to a byte, the even index in the low half;
   the coded formats with one E8M0 scale byte s for each 32 values: a code c stands for
   c * 2^(s - 127).  s is the smallest byte that brings the group's largest magnitude within the
   code's largest value (448; 6), so scaling by it is exact and the one rounding is that to the code's
   grid, to nearest even; no value is clipped.  A group that holds an infinity or a NaN gets s = 255
   and reads back as NaN throughout.

   Pages.  k_pages and v_pages hold n_pages pages of page_tokens tokens:
     code byte i of (page, head, token) at ((page*heads + head)*page_tokens + token)*row_bytes + i,
     row_bytes = head_dim * 16, 8 or 4 / 8;
     scale j at ((page*heads + head)*page_tokens + token)*(head_dim/32) + j of k_scales / v_scales
     (not used with TACTKV_TEXT_BF16).
   heads >= 1, head_dim a multiple of 32 up to 256, page_tokens a power of two, 16 to 1024; every
   pool 16-byte aligned.

   Rows.  A call works on n_rows rows of activations: sequence s owns rows row_starts[s] ..
   row_starts[s+1]-1 (row_starts[0] = 0, not decreasing), n_s of them, which stand for the cache positions
   kv_lens[s] - n_s .. kv_lens[s] - 1: kv_lens counts the sequence's tokens with these rows among
   them.  Position t is token t % page_tokens of page page_table[s*max_pages + t / page_tokens].  Rows
   from row_starts[n_seqs] on (a padded batch) have no effect, and their places in the outputs are left as they
   are.  page_table, kv_lens and
   row_starts are DEVICE arrays of int32, read when the kernels run, so that a captured call can be
   replayed on other lengths and pages.  A page may be shared by sequences that only read it; a
   position that a call appends to must belong to one sequence alone.

   Errors found by the kernels are recorded as TACTKV_INVALID_ARG in the workspace (zeroed by the
   caller before its first use; tactkv_device_status): rows, lengths or tables that do not fit together
   (n_s < 0, kv_lens[s] < n_s, more tokens than max_pages pages hold or, for attention, than
   max_kv_len, more rows than n_rows or max_rows) and page numbers outside 0 .. n_pages-1.  (TACTKV_TIMEOUT
   from tactkv_text_attention: a wait inside the kernel ran out, and its results are not whole.)  Nothing is
   read or written outside the arrays: append skips such rows, read zero-fills them, and attention
   leaves the tokens of such pages, or all tokens of such a sequence, out. */
#define TACTKV_TEXT_BF16  0
#define TACTKV_TEXT_MXFP8 1
#define TACTKV_TEXT_MXFP4 2

typedef struct {
  int32_t format;             /* TACTKV_TEXT_* */
  int32_t heads, head_dim;    /* K/V heads */
  int32_t page_tokens;
  int64_t n_pages;            /* pages in each pool */
  void* k_pages;
  void* v_pages;
  void* k_scales;             /* NULL with TACTKV_TEXT_BF16 */
  void* v_scales;
} tactkv_text_cache;

typedef struct {
  const int32_t* page_table;  /* DEVICE [n_seqs][max_pages] */
  const int32_t* kv_lens;     /* DEVICE [n_seqs] */
  const int32_t* row_starts;  /* DEVICE [n_seqs + 1] */
  int32_t n_seqs, n_rows, max_pages;
} tactkv_text_batch;

/* Workspace of the three calls: a status word for append and read (q_heads = 0), and for attention
   the partial results of the parts that long sequences are split into.  0 if the cache or the numbers
   are not supported. */
size_t tactkv_text_workspace_bytes(const tactkv_text_cache* cache, int n_seqs, int n_rows, int q_heads,
                                   int max_rows, int max_kv_len);

/* Write the rows' K and V into the cache.  Element (row, head, d) is at k + row*token_stride +
   head*head_stride + d (v alike; elements): bfloat16, or float32 with TACTKV_FP32_IO in flags (the only
   flag).  Strides even, k and v 4-byte aligned (8-byte with TACTKV_FP32_IO).  k_values, v_values: NULL
   or DEVICE [n_rows][heads][head_dim] of the same type, 16-byte aligned, which receive the values that the
   cache now holds, rounded to that type.  Asynchronous on `stream`; one kernel. */
tactkv_status tactkv_text_append(const tactkv_text_cache* cache, const tactkv_text_batch* batch, const void* k,
                                 const void* v, int64_t token_stride, int64_t head_stride, void* k_values,
                                 void* v_values, uint32_t flags, void* workspace, size_t workspace_bytes,
                                 struct CUstream_st* stream);

/* Read the rows' K and V from the cache into k and v (indexed and typed as for append).  With n_s =
   kv_lens[s] that is the whole sequence.  Strides with which two (row, head) places would meet are
   TACTKV_INVALID_ARG.  Asynchronous on `stream`; one kernel. */
tactkv_status tactkv_text_read(const tactkv_text_cache* cache, const tactkv_text_batch* batch, void* k, void* v,
                               int64_t token_stride, int64_t head_stride, uint32_t flags, void* workspace,
                               size_t workspace_bytes, struct CUstream_st* stream);

/* Attention of the rows over their sequences' cached tokens: the rows are the last generated token
   (n_s = 1) or a tree of drafted tokens, appended before this call.
     q_heads     query heads, a multiple G of the cache's heads (G <= 16); query head j reads K/V head j/G;
     max_rows    a bound on every n_s, 1 to 64; max_kv_len a bound on every kv_lens[s], up to 2^30 (both size the
                 launch: a closer bound is a faster call); n_seqs up to 65535, heads up to 1023;
     q           (row, head, d) at q + row*q_token_stride + head*q_head_stride + d: bfloat16, or float32
                 with TACTKV_FP32_IO; 16-byte aligned, strides multiples of 8 elements;
     tree        NULL or DEVICE [n_rows]: bit j of row i's word lets it see row j of its own sequence
                 (its ancestors and itself, for a tree).  NULL: rows 0 .. i.  Every row sees all
                 kv_lens[s] - n_s tokens before the rows;
     prior_out, prior_m, prior_l
                 all NULL, or DEVICE float32 [n_rows][q_heads][head_dim], [n_rows][q_heads] (twice): the
                 attention of the same queries over other tokens, as tactkv_attention_decode returns it,
                 to be merged;
     out         [n_rows][q_heads][head_dim], bfloat16 or float32 like q: softmax(q K^T / sqrt(head_dim)) V
                 over the tokens seen (and the prior's), 16-byte aligned;
     m, l        float32 [n_rows][q_heads]: the scores' maximum and sum_t exp(score - m).
   A row that sees nothing gets out = 0, m = -inf, l = 0.  Values at positions that a row does not see
   do not reach it, however large, infinities and NaN among them.  A row with a score of +inf or NaN has that
   as m, and NaN as l and in out.  K and V enter the products as the values that the codes stand for, in
   bfloat16's range.  Scores and sums are float32.  Before they multiply V the probabilities are rounded to 8
   bits (TACTKV_TEXT_BF16) or 16 (the coded formats) with bfloat16 q, to 24 with float32 q; the sums are of
   2^-16 times their products with V, so that V may come near bfloat16's largest value, and products with |V|
   below 2^-102 lose bits.
   No output may overlap an input or another output.  workspace: tactkv_text_workspace_bytes() with the same
   numbers, 256-byte aligned; calls that may overlap in time need workspaces of their own.  Asynchronous on
   `stream`; one kernel, or two where sequences are split. */
tactkv_status tactkv_text_attention(const tactkv_text_cache* cache, const tactkv_text_batch* batch, int q_heads,
                                    int max_rows, int max_kv_len, const void* q, int64_t q_token_stride,
                                    int64_t q_head_stride, const uint64_t* tree, const float* prior_out,
                                    const float* prior_m, const float* prior_l, void* out, float* m, float* l,
                                    uint32_t flags, void* workspace, size_t workspace_bytes,
                                    struct CUstream_st* stream);

/* Synchronizes `stream`, returns the first error the kernels recorded in `workspace` since the
   previous call (TACTKV_OK if none), and clears it. */
tactkv_status tactkv_device_status(void* workspace, size_t workspace_bytes,
                                   struct CUstream_st* stream);

/* Human-readable status name. */
const char* tactkv_status_string(tactkv_status status);

/* The library's own Lloyd-Max codebook for `bits` (1..8): 2^bits levels and 2^bits - 1
   thresholds, increasing, written to the host arrays given.  Returns the number of levels, or
   0 for bits outside 1..8.  Host-only; needs no GPU. */
int tactkv_lloyd_max_table(int bits, double* levels, double* thresholds);

/* Occupancy of one compressed unit ("Methodology in Plain English", stage 4: a layer's cache takes
   sum_i (b_i * d + 32) bits plus a small index).  The sum runs over the gain-shape vectors: one per
   bin with d = n = heads*head_dim, or, with TACTKV_HEAD_GAIN, one per (bin, head) with
   d = head_dim.  The index is the byte b_i of every bin. */
typedef struct {
  uint64_t bins;            /* N */
  uint64_t channels;        /* n */
  uint64_t code_bits;       /* sum_i b_i, the bits of one channel stream */
  uint64_t formula_bits;    /* sum_i (b_i * n + 32 * gains per bin): codes and gains */
  uint64_t index_bits;      /* 8 * N: the bit widths */
  uint64_t payload_bytes;   /* the payload's actual size (header, padding and alignment included) */
  double bits_per_element;  /* 8 * payload_bytes / (N * n) */
  double shrink_vs_bf16;    /* 2 * N * n / payload_bytes: size of the bf16 volume over the payload */
} tactkv_occupancy_t;

/* Reads a HOST copy of a payload (at least its header and b[] array: 64 + N bytes) and fills
   *out.  Returns TACTKV_OK, TACTKV_INVALID_ARG (null pointers) or TACTKV_CORRUPT_PAYLOAD (bad
   magic or version, a bit width above 8, or a code_bits field that disagrees with b[]).
   Host-only; needs no GPU. */
tactkv_status tactkv_occupancy(const void* payload, size_t bytes, tactkv_occupancy_t* out);

/* Largest number of requests whose caches fit: floor((hbm_bytes - fixed_bytes) / per_request_bytes)
   (0 when fixed_bytes >= hbm_bytes, -1 when per_request_bytes is 0).  fixed_bytes: what every
   request shares (weights, activations, runtime reserve); per_request_bytes: one request's cache,
   e.g. the sum of its units' payload_bytes plus its uncompressed text KV.  Host-only. */
int64_t tactkv_max_batch(uint64_t hbm_bytes, uint64_t fixed_bytes, uint64_t per_request_bytes);

/* Version of the payload format this library writes and reads. */
int tactkv_format_version(void);

/* Number of kernels that the calling host thread's most recent tactkv_compress*,
   tactkv_decompress* call launched, over all its waves (0 after a call that failed before
   launching).  A compress wave launches 4 kernels when its grid has a fused three-axis forward
   transform kernel (H x W = 16 x 16, 14 x 14 or 8 x 8 with S = 8, 16, 32 or 64, 24 x 24 with S = 8, 16
   or 32) and 5 otherwise;
   a decompress wave launches 3. */
int tactkv_last_launches(void);

#ifdef __cplusplus
}
#endif

#endif /* TACTKV_H_ */

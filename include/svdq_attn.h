/*
 * svdq_attn.h -- C ABI of the operators that follow the attention projections:
 * head norms with rotary positions (and the per-head Hadamard), a paged
 * key/value cache in the library's NVFP4 format, and attention over it.
 *
 * Conventions are those of svdq.h: device pointers, `stream` a cudaStream_t as
 * void*, asynchronous, an svdq_status returned and nothing thrown.  These calls
 * have no handle and keep nothing between calls; they may run from several host
 * threads and streams at once as long as what they write differs.  They launch
 * on the device that is current, which must be the one the pointers belong to.
 *
 * Tensors of heads, (tokens, heads, head_dim), have head_dim contiguous and
 * token and head strides given in elements: a slice of a packed projection
 * output is passed as it lies.  Pointers 16-byte aligned, strides multiples of
 * 8.  dtype: 0 = bf16, 1 = fp16.
 */
#ifndef SVDQ_ATTN_H_
#define SVDQ_ATTN_H_

#include "svdq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* One tensor of heads. */
typedef struct {
  void* data;
  long long token_stride;     /* elements, multiple of 8 */
  long long head_stride;      /* elements, multiple of 8 */
} svdq_heads;

/*
 * svdq_qk_norm_rope -- for every head of queries and keys, in one pass:
 *   n_d = x_d * rsqrt(mean(x^2) + eps) * weight_d        (weight NULL: n = x)
 *   for pair p < pairs, (a, b) = (n_2p, n_2p+1) if interleaved, else (n_p, n_p+pairs):
 *     phi = positions[token, pair_axis[p]] * inv_freq[p]
 *     (a, b) <- (a cos phi - b sin phi, a sin phi + b cos phi)
 *   y = n H / sqrt(head_dim)                              (if hadamard)
 * Dimensions from 2 * pairs on get no position.  Any split of the pairs over
 * the axes is given by pair_axis (sections, interleaved sections, one axis).
 * H is the Sylvester Hadamard of "Rotate in quantization and its vLLM
 * implementation" (section 3.2, per head_dim block): with it on queries and
 * keys alike q.k stays and keys lose less in 4 bits.
 * fp32 inside (the angle in fp64), one rounding to the storage type; the sum of
 * squares is fp32 too, so norms are for magnitudes below about 2^60.
 *   head_dim   multiple of 8, 8 .. 256; hadamard needs a power of two
 *   pairs      0 .. head_dim / 2; a multiple of 8 unless interleaved
 *   q_out/k_out may be q/k (in place); other overlaps are undefined
 *   strides    below 2^31 elements; tokens below 2^31 - 4096
 * tokens == 0 is a no-op; q_heads or k_heads may be 0.
 */
typedef struct {
  int tokens, q_heads, k_heads, head_dim, dtype;
  svdq_heads q, k, q_out, k_out;
  const void* q_weight;       /* (head_dim) in the storage type, or NULL */
  const void* k_weight;
  float eps;                  /* >= 0 */
  const int* positions;       /* (tokens, axes) int32, row stride position_stride; NULL if pairs == 0 */
  long long position_stride;
  int axes;                   /* >= 1 */
  const float* inv_freq;      /* (pairs) */
  const unsigned char* pair_axis; /* (pairs), values below axes (larger ones count as axes - 1), or NULL: all 0 */
  int pairs, interleaved, hadamard;
} svdq_qk_norm_rope_desc;
SVDQ_API svdq_status svdq_qk_norm_rope(const svdq_qk_norm_rope_desc* desc, void* stream);

/*
 * The paged cache.  Along the head dimension keys and values are NVFP4 as
 * everywhere in the library: E2M1 codes, element 2j in the low nibble of byte
 * j, and one e4m3 scale per 16 elements.  Contiguous, caller-owned:
 *   k_codes, v_codes   (pages, heads, page_size, head_dim / 2)  uint8
 *   k_scales, v_scales (pages, heads, page_size, head_dim / 16) e4m3 bytes
 * head_dim 64 or 128; page_size 16, 32, 64, 128 or 256; 16-byte aligned.
 */
typedef struct {
  void *k_codes, *k_scales, *v_codes, *v_scales;
  long long pages;
  int heads, page_size, head_dim;
} svdq_kv4_cache;

/*
 * svdq_kv4_append -- quantize k, v (tokens, heads, head_dim) into the cache:
 * token t goes to slot slots[t] = page * page_size + offset (int64, device).
 * A slot outside the cache (negative: padding) is skipped.  The slots of one
 * call have to differ; a slot named twice is left with an unspecified mix.  The
 * cache's tensors may not overlap each other, k, v or slots here (attention and
 * svdq_kv4_read may read keys and values from the same ones).
 * scale = e4m3_rne_satfinite(fp32(amax / 6)), code = e2m1_rne_satfinite(fp32(x / scale)),
 * as svdq_quantize_weight.  There is no scale a tensor or head beside these: a
 * block of 16 whose largest magnitude is at most 6 x 2^-10 (0.0059) becomes zeros,
 * below 6 x 2^-6 (0.094) its scale has one to three bits, and magnitudes above
 * 2688 saturate.  Values of another range are scaled by the caller, before the
 * call and on attention's output.
 */
SVDQ_API svdq_status svdq_kv4_append(const svdq_kv4_cache* cache, const svdq_heads* k, const svdq_heads* v,
                                     int tokens, int dtype, const long long* slots, void* stream);

/*
 * svdq_kv4_read -- the inverse: the values that slots hold, code * scale
 * (exact in both storage types), into k_out, v_out (tokens, heads, head_dim).
 * A slot outside the cache reads as zeros.  Slots may repeat.
 */
SVDQ_API svdq_status svdq_kv4_read(const svdq_kv4_cache* cache, const svdq_heads* k_out, const svdq_heads* v_out,
                                   int tokens, int dtype, const long long* slots, void* stream);

/*
 * svdq_kv4_attention -- attention of new query tokens over the cache.
 * Request b has kv_len[b] keys; key j is row j % page_size of page
 * block_table[b, j / page_size].  Its n queries are tokens q_start[b] ..
 * q_start[b+1] (q_start NULL: tokens / requests each); query i stands at
 * position kv_len[b] - n + i, so the new tokens' keys are appended first.
 *   s_j = softmax_scale q.k_j  over keys j < kv_len[b], causal: j <= position
 *   out = sum_j softmax(s)_j v_j,   lse = log sum_j exp(s_j)
 * Query head h reads key head h / (q_heads / heads).
 * A query without a key (kv_len 0, or causal with kv_len < n) gets out 0 and
 * lse -inf; one whose scores are all -inf (an infinite query) counts as such.
 * softmax_scale may be any finite number, 0 and negative ones included; scores
 * past fp32's range give NaN.  Tokens before q_start[0] and from q_start[requests] on are left
 * as they were in out and lse.  Lengths are clamped to the table's capacity;
 * keys in a page outside [0, pages) do not exist.  q_start has to ascend.
 * out and lse must not overlap what is read.  Products are exact in fp32 per term, sums and
 * softmax fp32, softmax weights rounded to fp16 for the product with v (2^-11
 * of themselves, or 2^-32 of the row's largest where that is more).
 * max_kv_len: an upper bound of kv_len for scheduling (0: the table's
 * capacity); a too small one costs time, not correctness.
 * workspace: svdq_kv4_attention_workspace_bytes(desc) bytes, 16-byte aligned,
 * caller-owned, not shared by calls that may overlap; NULL if that is 0.
 */
typedef struct {
  svdq_kv4_cache cache;
  int tokens, requests, q_heads, dtype;
  svdq_heads q, out;
  float* lse;                 /* (tokens, q_heads) fp32, or NULL */
  const int* kv_len;          /* (requests) */
  const int* q_start;         /* (requests + 1), or NULL */
  const int* block_table;     /* (requests, max_pages), row stride table_stride */
  long long table_stride;
  int max_pages, max_kv_len, causal;
  float softmax_scale;        /* finite */
} svdq_kv4_attention_desc;
SVDQ_API size_t svdq_kv4_attention_workspace_bytes(const svdq_kv4_attention_desc* desc);
SVDQ_API svdq_status svdq_kv4_attention(const svdq_kv4_attention_desc* desc, void* workspace, size_t workspace_bytes,
                                        void* stream);

/*
 * svdq_kv4_attention_status -- synchronize the current device and read + clear
 * the error word of svdq_kv4_attention's tensor-core kernel there (nonzero when
 * a bounded wait expired: the kernel then skipped its remaining work).  Returns
 * SVDQ_ERR_DEVICE when it was nonzero.
 */
SVDQ_API svdq_status svdq_kv4_attention_status(int* flags);

#ifdef __cplusplus
}
#endif

#endif /* SVDQ_ATTN_H_ */

// attn_kernels.h -- host-side launch interface of the attention-side kernels
// (internal to the library; the public boundary is include/svdq_attn.h).
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

namespace svdq {

// Text returned by svdq_last_error on this thread (never throws).
void set_last_error(const char* text) noexcept;

// One side (queries or keys) of the head norm / rotary / Hadamard pass.
struct HeadSide {
  const void* x;
  void* y;
  const void* weight;             // (D) in the storage type, or null: no norm
  int xt, xh, yt, yh;             // token and head strides in elements
  int heads;
};
struct QkNormRopeLaunch {
  HeadSide q, k;
  const int* positions;           // (tokens, axes), row stride pos_stride
  const float* inv_freq;          // (pairs)
  const uint8_t* pair_axis;       // (pairs) or null: axis 0
  long long pos_stride;
  int tokens, D, dtype, axes, pairs, num_sms;
  float eps;
  bool interleaved, hadamard;
};
cudaError_t launch_qk_norm_rope(const QkNormRopeLaunch& p, cudaStream_t stream);


// The 4-bit key/value cache: codes (pages, heads, page, D/2), e4m3 scales
// (pages, heads, page, D/16), D = 64 or 128, page = 1 << page_log2 >= 16.
struct Kv4Cache {
  uint8_t *kc, *ks, *vc, *vs;
  long long pages;
  int heads, D, page_log2;
};
struct Kv4RowsLaunch {
  Kv4Cache c;
  const void *k, *v;              // append: inputs
  void *k_out, *v_out;            // read: outputs
  long long kt, kh, vt, vh;       // token and head strides of k / v (or k_out / v_out), elements
  const long long* slots;         // (tokens); page * page_size + offset, outside the cache: skipped / zeros
  int tokens, dtype, num_sms;
};
cudaError_t launch_kv4_append(const Kv4RowsLaunch& p, cudaStream_t stream);
cudaError_t launch_kv4_read(const Kv4RowsLaunch& p, cudaStream_t stream);

// A segment that a CTA began and another one goes on with (rows 0: none).
struct Kv4Cut {
  int token0, row0, rows;         // of the request; of the tile
  int head, last_cta, slot;       // key head; CTA that ends it; the beginner's part
  int pad[2];
};
struct Kv4AttnLaunch {
  Kv4Cache c;
  const void* q;
  void* out;
  float* lse;                     // (tokens, q_heads) or null
  long long qt, qh, ot, oh;       // token and head strides, elements
  const int* kv_len;              // (requests)
  const int* q_start;             // (requests + 1) or null: tokens / requests each
  const int* table;               // (requests, max_pages), row stride table_stride
  long long table_stride;
  int max_pages, requests, tokens, q_heads, dtype, causal;
  float scale;                    // softmax scale
  // Set by kv4_attention_plan:
  int num_sms;
  int tile_rows;                  // rows of a tile: 8, 16, 24, 32 or 256
  int min_rows, max_rows;         // requests with fewer or more rows are left out
  long long segments;             // tiles x heads, at most
  int ctas, join;                 // CTAs that share the work; whether segments may be cut
  float* part_o;                  // join: (ctas, 2, tile_rows, D) fp32
  float2* part_ml;                //       (ctas, 2, tile_rows) {max, sum} in base 2
  Kv4Cut* cuts;                   //       (ctas)
};
// The launches of one call: requests of few rows and of many (kv4_attention_tc.cu).
struct Kv4Plan {
  Kv4AttnLaunch few, many;
  bool use_few, use_many;
};
// `max_kv`: keys a request has at most (for the number of CTAs only).  The
// launch needs kv4_attention_workspace bytes, 16-byte aligned.
Kv4Plan kv4_attention_plan(const Kv4AttnLaunch& base, int max_kv, int num_sms);
size_t kv4_attention_workspace(const Kv4Plan& plan);
cudaError_t launch_kv4_attention(const Kv4Plan& plan, void* workspace, cudaStream_t stream);
cudaError_t launch_kv4_attention_tc(const Kv4AttnLaunch& p, cudaStream_t stream);
// Reads and clears the error word of launch_kv4_attention_tc on the current device (synchronizes it).
cudaError_t kv4_attention_status(unsigned* flags);

}  // namespace svdq

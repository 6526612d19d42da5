// attn_api.cu -- the C entry points of svdq_attn.h: argument checks and
// launches.  Host-side checks answer before any device work.
#include "svdq_attn.h"

#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "attn_kernels.h"

namespace {

constexpr long long kMaxBlocks = 1ll << 30;      // CTAs of one launch, far below the grid's limit

svdq_status fail(svdq_status s, const char* why) {
  svdq::set_last_error(why);
  return s;
}
svdq_status launched(cudaError_t e) { return e == cudaSuccess ? SVDQ_OK : fail(SVDQ_ERR_CUDA, cudaGetErrorString(e)); }

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// SMs of the current device, looked up once per device (a B200's count where
// there is no device to ask: argument errors are answered without one).
int num_sms() {
  static std::atomic<int> known[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return 148;
  }
  int n = dev >= 0 && dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
  if (n > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) {
    cudaGetLastError();
    return 148;
  }
  if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

// A tensor of heads with anything to read or write.
svdq_status check_heads(const svdq_heads& h) {
  if (!h.data) return fail(SVDQ_ERR_INVALID_ARG, "null tensor of heads");
  if (!aligned(h.data, 16)) return fail(SVDQ_ERR_INVALID_ARG, "tensor of heads not 16-byte aligned");
  if (h.token_stride % 8 != 0 || h.head_stride % 8 != 0)
    return fail(SVDQ_ERR_INVALID_ARG, "token and head strides have to be multiples of 8 elements");
  return SVDQ_OK;
}

svdq_status check_cache(const svdq_kv4_cache* c, svdq::Kv4Cache* out) {
  if (!c) return fail(SVDQ_ERR_INVALID_ARG, "null cache");
  if (c->head_dim != 64 && c->head_dim != 128) return fail(SVDQ_ERR_SHAPE, "head_dim of the cache has to be 64 or 128");
  int log2 = 4;
  while (log2 < 8 && (1 << log2) != c->page_size) ++log2;
  if ((1 << log2) != c->page_size) return fail(SVDQ_ERR_SHAPE, "page_size has to be 16, 32, 64, 128 or 256");
  if (c->heads < 1 || c->heads > 65535) return fail(SVDQ_ERR_SHAPE, "heads of the cache out of range");
  if (c->pages < 1 || c->pages > (1ll << 31)) return fail(SVDQ_ERR_SHAPE, "pages of the cache out of range");
  // Rows (page, head, offset) are numbered in 32 bits: 2^32 rows are more than any device holds.
  if (((c->pages * c->heads) << log2) >= 0xFFFFFFFFll) return fail(SVDQ_ERR_SHAPE, "the cache has too many rows");
  const void* ptr[4] = {c->k_codes, c->k_scales, c->v_codes, c->v_scales};
  for (const void* p : ptr)
    if (!p || !aligned(p, 16)) return fail(SVDQ_ERR_INVALID_ARG, "cache tensor null or not 16-byte aligned");
  out->kc = static_cast<uint8_t*>(c->k_codes);
  out->ks = static_cast<uint8_t*>(c->k_scales);
  out->vc = static_cast<uint8_t*>(c->v_codes);
  out->vs = static_cast<uint8_t*>(c->v_scales);
  out->pages = c->pages;
  out->heads = c->heads;
  out->D = c->head_dim;
  out->page_log2 = log2;
  return SVDQ_OK;
}

svdq_status check_rows(const svdq_kv4_cache* cache, const svdq_heads* k, const svdq_heads* v, int tokens, int dtype,
                       const long long* slots, svdq::Kv4RowsLaunch* p) {
  svdq_status s = check_cache(cache, &p->c);
  if (s != SVDQ_OK) return s;
  if (!k || !v || tokens < 0 || (dtype != 0 && dtype != 1)) return fail(SVDQ_ERR_INVALID_ARG, "bad k, v, tokens or dtype");
  if (tokens == 0) return SVDQ_OK;
  if ((s = check_heads(*k)) != SVDQ_OK || (s = check_heads(*v)) != SVDQ_OK) return s;
  if (!slots || !aligned(slots, 8)) return fail(SVDQ_ERR_INVALID_ARG, "slots null or misaligned");
  if ((long long)tokens * p->c.heads > kMaxBlocks / 8) return fail(SVDQ_ERR_SHAPE, "too many tokens");
  p->num_sms = num_sms();
  p->kt = k->token_stride;
  p->kh = k->head_stride;
  p->vt = v->token_stride;
  p->vh = v->head_stride;
  p->slots = slots;
  p->tokens = tokens;
  p->dtype = dtype;
  return SVDQ_OK;
}

svdq_status check_attention(const svdq_kv4_attention_desc* d, svdq::Kv4Plan* plan) {
  svdq::Kv4AttnLaunch launch = {}, *p = &launch;
  plan->use_few = plan->use_many = false;
  if (!d) return fail(SVDQ_ERR_INVALID_ARG, "null description");
  svdq_status s = check_cache(&d->cache, &p->c);
  if (s != SVDQ_OK) return s;
  if (d->tokens < 0 || d->requests < 0 || (d->dtype != 0 && d->dtype != 1) || !std::isfinite(d->softmax_scale))
    return fail(SVDQ_ERR_INVALID_ARG, "bad tokens, requests, dtype or softmax_scale");
  if (d->q_heads < 1 || d->q_heads % p->c.heads != 0)
    return fail(SVDQ_ERR_SHAPE, "q_heads has to be a multiple of the cache's heads");
  if (d->max_pages < 0 || d->max_kv_len < 0 || ((long long)d->max_pages << p->c.page_log2) > 0x7FFFFFFFll - 4096)
    return fail(SVDQ_ERR_SHAPE, "max_pages or max_kv_len out of range");
  if (d->requests > 0 && !d->q_start && d->tokens % d->requests != 0)
    return fail(SVDQ_ERR_SHAPE, "without q_start tokens has to be a multiple of requests");
  if ((long long)d->tokens * d->q_heads > kMaxBlocks || d->requests > (1 << 24))
    return fail(SVDQ_ERR_SHAPE, "too many tokens or requests");
  p->q = d->q.data;
  p->out = d->out.data;
  p->lse = d->lse;
  p->qt = d->q.token_stride;
  p->qh = d->q.head_stride;
  p->ot = d->out.token_stride;
  p->oh = d->out.head_stride;
  p->kv_len = d->kv_len;
  p->q_start = d->q_start;
  p->table = d->block_table;
  p->table_stride = d->table_stride;
  p->max_pages = d->max_pages;
  p->requests = d->requests;
  p->tokens = d->tokens;
  p->q_heads = d->q_heads;
  p->dtype = d->dtype;
  p->causal = d->causal != 0;
  p->scale = d->softmax_scale;
  if (d->tokens > 0 && d->requests > 0) {
    const long long cap = (long long)d->max_pages << p->c.page_log2;
    const long long bound = d->max_kv_len > 0 && d->max_kv_len < cap ? d->max_kv_len : cap;
    *plan = svdq::kv4_attention_plan(launch, (int)bound, num_sms());
  }
  return SVDQ_OK;
}

}  // namespace

extern "C" {

svdq_status svdq_qk_norm_rope(const svdq_qk_norm_rope_desc* d, void* stream) {
  if (!d) return fail(SVDQ_ERR_INVALID_ARG, "null description");
  if (d->tokens < 0 || (d->dtype != 0 && d->dtype != 1) || !(d->eps >= 0.0f))
    return fail(SVDQ_ERR_INVALID_ARG, "bad tokens, dtype or eps");
  if (d->tokens > 0x7FFFFFFF - 4096) return fail(SVDQ_ERR_SHAPE, "too many tokens");     // (a CTA takes up to 4096)
  if (d->head_dim < 8 || d->head_dim > 256 || d->head_dim % 8 != 0)
    return fail(SVDQ_ERR_SHAPE, "head_dim has to be a multiple of 8, 8 .. 256");
  if (d->hadamard && (d->head_dim & (d->head_dim - 1)) != 0)
    return fail(SVDQ_ERR_SHAPE, "the Hadamard rotation needs a head_dim that is a power of two");
  if (d->q_heads < 0 || d->k_heads < 0 || d->q_heads > 65535 || d->k_heads > 65535)
    return fail(SVDQ_ERR_SHAPE, "heads out of range");
  if (d->pairs < 0 || 2 * d->pairs > d->head_dim || (!d->interleaved && d->pairs % 8 != 0))
    return fail(SVDQ_ERR_SHAPE, "pairs has to be at most head_dim / 2, and a multiple of 8 unless interleaved");
  if (d->tokens == 0 || d->q_heads + d->k_heads == 0) return SVDQ_OK;
  svdq_status s;
  if (d->q_heads && ((s = check_heads(d->q)) != SVDQ_OK || (s = check_heads(d->q_out)) != SVDQ_OK)) return s;
  if (d->k_heads && ((s = check_heads(d->k)) != SVDQ_OK || (s = check_heads(d->k_out)) != SVDQ_OK)) return s;
  if (!aligned(d->q_weight, 16) || !aligned(d->k_weight, 16))
    return fail(SVDQ_ERR_INVALID_ARG, "norm weights have to be 16-byte aligned");
  if (d->pairs > 0 && (!d->positions || !d->inv_freq || d->axes < 1 || !aligned(d->positions, 4) || !aligned(d->inv_freq, 4)))
    return fail(SVDQ_ERR_INVALID_ARG, "positions, inv_freq and axes >= 1 are needed with pairs");
  svdq::QkNormRopeLaunch p;
  const svdq_heads* sides[4] = {&d->q, &d->q_out, &d->k, &d->k_out};
  for (int i = 0; i < 4; ++i)
    if (i < 2 ? d->q_heads : d->k_heads)
      if (sides[i]->token_stride != (int)sides[i]->token_stride || sides[i]->head_stride != (int)sides[i]->head_stride)
        return fail(SVDQ_ERR_SHAPE, "strides have to fit 32 bits");
  p.q = {d->q.data, d->q_out.data, d->q_weight, (int)d->q.token_stride, (int)d->q.head_stride,
         (int)d->q_out.token_stride, (int)d->q_out.head_stride, d->q_heads};
  p.k = {d->k.data, d->k_out.data, d->k_weight, (int)d->k.token_stride, (int)d->k.head_stride,
         (int)d->k_out.token_stride, (int)d->k_out.head_stride, d->k_heads};
  p.num_sms = num_sms();
  p.positions = d->positions;
  p.inv_freq = d->inv_freq;
  p.pair_axis = d->pair_axis;
  p.pos_stride = d->position_stride;
  p.tokens = d->tokens;
  p.D = d->head_dim;
  p.dtype = d->dtype;
  p.axes = d->axes;
  p.pairs = d->pairs;
  p.eps = d->eps;
  p.interleaved = d->interleaved != 0;
  p.hadamard = d->hadamard != 0;
  return launched(svdq::launch_qk_norm_rope(p, static_cast<cudaStream_t>(stream)));
}

svdq_status svdq_kv4_append(const svdq_kv4_cache* cache, const svdq_heads* k, const svdq_heads* v, int tokens,
                            int dtype, const long long* slots, void* stream) {
  svdq::Kv4RowsLaunch p = {};
  svdq_status s = check_rows(cache, k, v, tokens, dtype, slots, &p);
  if (s != SVDQ_OK || tokens == 0) return s;
  p.k = k->data;
  p.v = v->data;
  return launched(svdq::launch_kv4_append(p, static_cast<cudaStream_t>(stream)));
}

svdq_status svdq_kv4_read(const svdq_kv4_cache* cache, const svdq_heads* k_out, const svdq_heads* v_out, int tokens,
                          int dtype, const long long* slots, void* stream) {
  svdq::Kv4RowsLaunch p = {};
  svdq_status s = check_rows(cache, k_out, v_out, tokens, dtype, slots, &p);
  if (s != SVDQ_OK || tokens == 0) return s;
  p.k_out = k_out->data;
  p.v_out = v_out->data;
  return launched(svdq::launch_kv4_read(p, static_cast<cudaStream_t>(stream)));
}

size_t svdq_kv4_attention_workspace_bytes(const svdq_kv4_attention_desc* d) {
  svdq::Kv4Plan p;
  if (check_attention(d, &p) != SVDQ_OK) return 0;
  return svdq::kv4_attention_workspace(p);
}

svdq_status svdq_kv4_attention(const svdq_kv4_attention_desc* d, void* workspace, size_t workspace_bytes,
                               void* stream) {
  svdq::Kv4Plan p;
  svdq_status s = check_attention(d, &p);
  if (s != SVDQ_OK || d->tokens == 0 || d->requests == 0) return s;
  if ((s = check_heads(d->q)) != SVDQ_OK || (s = check_heads(d->out)) != SVDQ_OK) return s;
  if (!d->kv_len || (d->max_pages > 0 && !d->block_table)) return fail(SVDQ_ERR_INVALID_ARG, "null kv_len or block_table");
  const void* words[4] = {d->kv_len, d->q_start, d->block_table, d->lse};
  for (const void* w : words)
    if (!aligned(w, 4)) return fail(SVDQ_ERR_INVALID_ARG, "kv_len, q_start, block_table or lse not 4-byte aligned");
  const size_t need = svdq::kv4_attention_workspace(p);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 16)))
    return fail(SVDQ_ERR_WORKSPACE, "workspace null, too small or not 16-byte aligned");
  return launched(svdq::launch_kv4_attention(p, workspace, static_cast<cudaStream_t>(stream)));
}

svdq_status svdq_kv4_attention_status(int* flags) {
  if (!flags) return SVDQ_ERR_INVALID_ARG;
  unsigned word = 0;
  const svdq_status s = launched(svdq::kv4_attention_status(&word));
  *flags = (int)word;
  return s != SVDQ_OK ? s : word ? SVDQ_ERR_DEVICE : SVDQ_OK;
}

}  // extern "C"

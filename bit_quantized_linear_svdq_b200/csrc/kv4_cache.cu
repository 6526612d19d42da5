// kv4_cache.cu -- the paged 4-bit key/value cache: write (quantize) and read
// (dequantize) rows by slot number.
//
// Format: the library's NVFP4 along the head dimension, one e4m3 scale per 16
// values (nvfp4_block.cuh; the rules of the activation and weight quantizers,
// so codes and scales are bit-identical to theirs):
//   scale = e4m3_rne_satfinite(fp32(amax / 6)),  code = e2m1_rne_satfinite(fp32(x / scale))
// A value read back, e2m1 x e4m3, has at most 6 significant bits and lies in
// 2^-10 .. 2688, so it is exact in fp16 and bf16.
//
// Slot s is offset s % page of page s / page; both tensors keep a page's rows
// of one head contiguous, codes (pages, heads, page, D/2) and scales (pages,
// heads, page, D/16), which is the order attention reads them in.
//
// One thread per 16-value block: consecutive threads take a row's blocks, so a
// warp reads 1 KB of keys or values contiguously (heads are adjacent in the
// projection's output) and writes whole rows of codes.  HBM-bound: 2 + 9/16
// bytes a value.
#include <cuda_runtime.h>

#include "attn_kernels.h"
#include "kv4_codes.cuh"
#include "nvfp4_block.cuh"

namespace svdq {
namespace {

constexpr int kThreadsC = 256;

// Block b of the launch: token, which of k / v, head, 16-value block.
struct RowBlock {
  long long code_at, scale_at;                  // byte offsets in the cache tensors, code_at < 0: slot outside
  int token, head, blk;
  bool is_v;
};
__device__ __forceinline__ RowBlock row_block(const Kv4RowsLaunch& p, long long i) {
  RowBlock r;
  const int nb = p.c.D / 16;
  r.blk = (int)(i % nb);
  long long j = i / nb;
  r.head = (int)(j % p.c.heads);
  j /= p.c.heads;
  r.is_v = j & 1;
  r.token = (int)(j >> 1);
  const long long slot = p.slots[r.token];
  r.code_at = r.scale_at = -1;
  if (slot >= 0 && (slot >> p.c.page_log2) < p.c.pages) {
    const long long page = slot >> p.c.page_log2, off = slot & ((1ll << p.c.page_log2) - 1);
    const long long row = ((page * p.c.heads + r.head) << p.c.page_log2) + off;
    r.scale_at = row * nb + r.blk;
    r.code_at = 8 * r.scale_at;
  }
  return r;
}

template <bool BF16>
__global__ void __launch_bounds__(kThreadsC) kv4_append_kernel(const __grid_constant__ Kv4RowsLaunch p) {
  __shared__ float2 srec[128];                  // e4m3 code -> {-s, RN(1/s)}
  if (threadIdx.x < 128) {
    const float s = e4m3_to_f32(threadIdx.x);
    srec[threadIdx.x] = make_float2(-s, threadIdx.x ? __frcp_rn(s) : 0.0f);
  }
  const float y6 = __frcp_rn(6.0f);
  __syncthreads();
  const long long i = (long long)blockIdx.x * kThreadsC + threadIdx.x;
  if (i >= 2ll * p.tokens * p.c.heads * (p.c.D / 16)) return;
  const RowBlock r = row_block(p, i);
  if (r.code_at < 0) return;
  const uint16_t* x = static_cast<const uint16_t*>(r.is_v ? p.v : p.k) + r.token * (r.is_v ? p.vt : p.kt) +
                      r.head * (r.is_v ? p.vh : p.kh) + 16 * r.blk;
  const uint4 a = reinterpret_cast<const uint4*>(x)[0], b = reinterpret_cast<const uint4*>(x)[1];
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint64_t v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (BF16) {
      v[j] = bf16x2_to_f2(w[j]);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
      v[j] = pk2(f.x, f.y);
    }
  }
  uint32_t c0, c1;
  const uint32_t sb = quantize_any(v, srec, y6, c0, c1);
  *reinterpret_cast<uint2*>((r.is_v ? p.c.vc : p.c.kc) + r.code_at) = make_uint2(c0, c1);
  (r.is_v ? p.c.vs : p.c.ks)[r.scale_at] = (uint8_t)sb;
}

template <bool BF16>
__global__ void __launch_bounds__(kThreadsC) kv4_read_kernel(const __grid_constant__ Kv4RowsLaunch p) {
  const long long i = (long long)blockIdx.x * kThreadsC + threadIdx.x;
  if (i >= 2ll * p.tokens * p.c.heads * (p.c.D / 16)) return;
  const RowBlock r = row_block(p, i);
  uint32_t o[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (r.code_at >= 0) {
    const uint2 c = *reinterpret_cast<const uint2*>((r.is_v ? p.c.vc : p.c.kc) + r.code_at);
    const uint32_t sb = (r.is_v ? p.c.vs : p.c.ks)[r.scale_at];
    const __half2 s = e4m3x2_to_half2(sb | (sb << 8));
    uint32_t d[8];
    e2m1x8_to_f16x8(c.x, d);
    e2m1x8_to_f16x8(c.y, d + 4);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const __half2 h = __hmul2(*reinterpret_cast<const __half2*>(&d[j]), s);
      if (BF16) {
        const float2 f = __half22float2(h);
        o[j] = pack_bf16x2(f.x, f.y);
      } else {
        o[j] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
  }
  uint16_t* y = static_cast<uint16_t*>(r.is_v ? p.v_out : p.k_out) + r.token * (r.is_v ? p.vt : p.kt) +
                r.head * (r.is_v ? p.vh : p.kh) + 16 * r.blk;
  reinterpret_cast<uint4*>(y)[0] = make_uint4(o[0], o[1], o[2], o[3]);
  reinterpret_cast<uint4*>(y)[1] = make_uint4(o[4], o[5], o[6], o[7]);
}

unsigned blocks_for(const Kv4RowsLaunch& p) {
  const long long n = 2ll * p.tokens * p.c.heads * (p.c.D / 16);
  return (unsigned)((n + kThreadsC - 1) / kThreadsC);
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4RowsLaunch& p, cudaStream_t stream) {
  if (p.dtype == 0)
    kv4_append_kernel<true><<<blocks_for(p), kThreadsC, 0, stream>>>(p);
  else
    kv4_append_kernel<false><<<blocks_for(p), kThreadsC, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_kv4_read(const Kv4RowsLaunch& p, cudaStream_t stream) {
  if (p.dtype == 0)
    kv4_read_kernel<true><<<blocks_for(p), kThreadsC, 0, stream>>>(p);
  else
    kv4_read_kernel<false><<<blocks_for(p), kThreadsC, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace svdq

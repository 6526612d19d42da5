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
// A thread takes one 16-value block at a time, consecutive threads a row's
// blocks, so a warp reads 1 KB of keys or values contiguously (heads are
// adjacent in the projection's output) and writes whole rows of codes; keys and
// values are the two halves of the grid.  One resident set of CTAs strides over
// the blocks, two in flight a thread (a CTA per 256 blocks spent as much on its
// table of scale reciprocals and on index divisions as on its blocks).
// HBM-bound: 2 + 9/16 bytes a value.
#include <cuda_runtime.h>

#include "attn_kernels.h"
#include "kcommon.cuh"
#include "kv4_codes.cuh"
#include "nvfp4_block.cuh"

namespace svdq {
namespace {

constexpr int kThreadsC = 256, kFlightC = 2;

// Block i of one side: its token, its place in the rows and (as soon as the
// slot is known) in the cache.
struct RowBlock {
  unsigned token, head, blk;
};
__device__ __forceinline__ RowBlock row_block(const Kv4RowsLaunch& p, unsigned i) {
  const unsigned log2nb = p.c.D == 128 ? 3 : 2;
  RowBlock r;
  r.blk = i & ((1u << log2nb) - 1u);
  i >>= log2nb;
  r.token = i / (unsigned)p.c.heads;
  r.head = i - r.token * (unsigned)p.c.heads;
  return r;
}
// The block's number in the cache's scale tensor (its codes lie at 8 times that); -1: the slot is outside.
__device__ __forceinline__ long long cache_block(const Kv4RowsLaunch& p, const RowBlock& r, long long slot) {
  if (slot < 0 || (slot >> p.c.page_log2) >= p.c.pages) return -1;
  const long long page = slot >> p.c.page_log2, off = slot & ((1ll << p.c.page_log2) - 1);
  return (((page * p.c.heads + r.head) << p.c.page_log2) + off) * (p.c.D / 16) + r.blk;
}

template <bool BF16>
__global__ void __launch_bounds__(kThreadsC) kv4_append_kernel(const __grid_constant__ Kv4RowsLaunch p) {
  // e4m3 code -> {s, RN(-1/s)}: -x divided by -s gives x / s with its sign, zeros too (nvfp4_block.cuh).
  __shared__ float2 srec[128];
  if (threadIdx.x < 128) {
    const float s = e4m3_to_f32(threadIdx.x);
    srec[threadIdx.x] = make_float2(s, threadIdx.x ? -__frcp_rn(s) : 0.0f);
  }
  const float y6 = __frcp_rn(6.0f);
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
  const bool is_v = blockIdx.y;
  const uint16_t* x = static_cast<const uint16_t*>(is_v ? p.v : p.k);
  const long long xt = is_v ? p.vt : p.kt, xh = is_v ? p.vh : p.kh;
  uint8_t *codes = is_v ? p.c.vc : p.c.kc, *scales = is_v ? p.c.vs : p.c.ks;
  const unsigned total = (unsigned)p.tokens * (unsigned)p.c.heads * (unsigned)(p.c.D / 16), step = gridDim.x * kThreadsC;
  for (unsigned i0 = blockIdx.x * kThreadsC + threadIdx.x; i0 < total; i0 += kFlightC * step) {
    uint4 w[kFlightC][2];
    long long at[kFlightC];
#pragma unroll
    for (int f = 0; f < kFlightC; ++f) {
      at[f] = -1;
      const unsigned i = i0 + f * step;
      if (i < total) {
        const RowBlock r = row_block(p, i);
        const uint4* src = reinterpret_cast<const uint4*>(x + r.token * xt + r.head * xh + 16 * r.blk);
        w[f][0] = src[0];
        w[f][1] = src[1];
        at[f] = cache_block(p, r, p.slots[r.token]);
      }
    }
#pragma unroll
    for (int f = 0; f < kFlightC; ++f) {
      if (at[f] < 0) continue;
      const uint32_t u[8] = {w[f][0].x, w[f][0].y, w[f][0].z, w[f][0].w, w[f][1].x, w[f][1].y, w[f][1].z, w[f][1].w};
      uint64_t v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t m = u[j] ^ 0x80008000u;              // -x
        if (BF16) {
          v[j] = bf16x2_to_f2(m);
        } else {
          const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&m));
          v[j] = pk2(h.x, h.y);
        }
      }
      const float amax = amax8(v);
      uint32_t c0, c1, sb;
      if (amax < 3.0e38f) {
        sb = quant_block<true>(v, amax, srec, y6, c0, c1);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] ^= 0x8000000080000000ull;
        sb = quant_block_slow(v, c0, c1);
      }
      *reinterpret_cast<uint2*>(codes + 8 * at[f]) = make_uint2(c0, c1);
      scales[at[f]] = (uint8_t)sb;
    }
  }
}

template <bool BF16>
__global__ void __launch_bounds__(kThreadsC) kv4_read_kernel(const __grid_constant__ Kv4RowsLaunch p) {
  griddep_wait();
  griddep_launch_dependents();
  const bool is_v = blockIdx.y;
  uint16_t* y = static_cast<uint16_t*>(is_v ? p.v_out : p.k_out);
  const long long yt = is_v ? p.vt : p.kt, yh = is_v ? p.vh : p.kh;
  const uint8_t *codes = is_v ? p.c.vc : p.c.kc, *scales = is_v ? p.c.vs : p.c.ks;
  const unsigned total = (unsigned)p.tokens * (unsigned)p.c.heads * (unsigned)(p.c.D / 16), step = gridDim.x * kThreadsC;
  for (unsigned i0 = blockIdx.x * kThreadsC + threadIdx.x; i0 < total; i0 += kFlightC * step) {
    uint2 c[kFlightC];
    uint32_t sb[kFlightC];
#pragma unroll
    for (int f = 0; f < kFlightC; ++f) {
      c[f] = make_uint2(0, 0);
      sb[f] = 0;
      const unsigned i = i0 + f * step;
      if (i < total) {
        const RowBlock r = row_block(p, i);
        const long long at = cache_block(p, r, p.slots[r.token]);
        if (at >= 0) {
          c[f] = *reinterpret_cast<const uint2*>(codes + 8 * at);
          sb[f] = scales[at];
        }
      }
    }
#pragma unroll
    for (int f = 0; f < kFlightC; ++f) {
      const unsigned i = i0 + f * step;
      if (i >= total) continue;
      const RowBlock r = row_block(p, i);
      const __half2 s = e4m3x2_to_half2(sb[f] | (sb[f] << 8));
      uint32_t d[8], o[8];
      e2m1x8_to_f16x8(c[f].x, d);
      e2m1x8_to_f16x8(c[f].y, d + 4);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const __half2 h = __hmul2(*reinterpret_cast<const __half2*>(&d[j]), s);
        if (BF16) {
          const float2 v = __half22float2(h);
          o[j] = pack_bf16x2(v.x, v.y);
        } else {
          o[j] = *reinterpret_cast<const uint32_t*>(&h);
        }
      }
      uint4* dst = reinterpret_cast<uint4*>(y + r.token * yt + r.head * yh + 16 * r.blk);
      dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
      dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
  }
}

cudaError_t launch(void (*kernel)(Kv4RowsLaunch), const Kv4RowsLaunch& p, cudaStream_t stream) {
  const long long n = (long long)p.tokens * p.c.heads * (p.c.D / 16), need = (n + kThreadsC - 1) / kThreadsC;
  const long long resident = 4ll * p.num_sms;              // of 8 an SM, for keys and for values each
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(need < resident ? need : resident), 2);
  cfg.blockDim = dim3(kThreadsC);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4RowsLaunch& p, cudaStream_t stream) {
  return launch(p.dtype == 0 ? kv4_append_kernel<true> : kv4_append_kernel<false>, p, stream);
}

cudaError_t launch_kv4_read(const Kv4RowsLaunch& p, cudaStream_t stream) {
  return launch(p.dtype == 0 ? kv4_read_kernel<true> : kv4_read_kernel<false>, p, stream);
}

}  // namespace svdq

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
// the blocks (a CTA per 256 blocks spent as much on its table of scale
// reciprocals and on index divisions as on its blocks), two in flight a thread.
//
// Bound: 2 + 9/16 bytes a value (HBM).  16411 tokens of 8 heads x 128, keys and
// values, of 4 x 8 packed heads: 18.3 us to write (86 MB, 4.7 TB/s; issue slots
// 61%, the largest stall is the wait for loads), 14.8 us to read back (5.8 TB/s).
// 16-byte accesses instead of 32: 22 and 21 us; a grid of twice what is
// resident: 19.2 to write; one block in flight 19.4, four 21.8.
#include <cuda_runtime.h>

#include "attn_kernels.h"
#include "kcommon.cuh"
#include "kv4_codes.cuh"
#include "nvfp4_block.cuh"

namespace svdq {
namespace {

constexpr int kThreadsC = 256, kFlightC = 2, kAppendCtas = 4, kReadCtas = 8;

// A block of one side: its token and its number among the token's.
struct RowBlock {
  unsigned token, at;
};
__device__ __forceinline__ unsigned log2_blocks(const Kv4RowsLaunch& p) { return p.c.D == 128 ? 3 : 2; }
// Blocks i, i + step, i + 2 step, ... of a thread: one division each at the start.
struct RowWalk {
  RowBlock r, by;
  unsigned per;
  __device__ __forceinline__ RowWalk(const Kv4RowsLaunch& p, unsigned i, unsigned step) {
    per = (unsigned)p.c.heads << log2_blocks(p);
    r.token = i / per;
    r.at = i - r.token * per;
    by.token = step / per;
    by.at = step - by.token * per;
  }
  __device__ __forceinline__ void next() {
    r.token += by.token;
    r.at += by.at;
    if (r.at >= per) r.at -= per, ++r.token;
  }
};
__device__ __forceinline__ long long row_offset(const Kv4RowsLaunch& p, const RowBlock& r, long long xt, long long xh) {
  const unsigned log2nb = log2_blocks(p);
  return r.token * xt + (r.at >> log2nb) * xh + 16 * (r.at & ((1u << log2nb) - 1u));
}
// The block's number in the cache's scale tensor (its codes lie at 8 times that); -1: the slot is outside.
__device__ __forceinline__ long long cache_block(const Kv4RowsLaunch& p, const RowBlock& r, long long slot) {
  if (slot < 0 || (slot >> p.c.page_log2) >= p.c.pages) return -1;
  const long long page = slot >> p.c.page_log2, off = slot & ((1ll << p.c.page_log2) - 1);
  const unsigned log2nb = log2_blocks(p), head = r.at >> log2nb, blk = r.at & ((1u << log2nb) - 1u);
  return ((((page * p.c.heads + head) << p.c.page_log2) + off) << log2nb) + blk;
}

// A block's 32 bytes of 16-bit values: one access where they are aligned (two of
// 16 bytes leave each only half of every sector), else two.
__device__ __forceinline__ void load_block(const uint16_t* x, bool wide, uint32_t (&u)[8]) {
  if (wide) {
    asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7])
                 : "l"(x));
  } else {
    const uint4 a = reinterpret_cast<const uint4*>(x)[0], b = reinterpret_cast<const uint4*>(x)[1];
    u[0] = a.x, u[1] = a.y, u[2] = a.z, u[3] = a.w, u[4] = b.x, u[5] = b.y, u[6] = b.z, u[7] = b.w;
  }
}
__device__ __forceinline__ void store_block(uint16_t* y, bool wide, const uint32_t (&u)[8]) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]),
                 "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "l"(y)
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(y)[0] = make_uint4(u[0], u[1], u[2], u[3]);
    reinterpret_cast<uint4*>(y)[1] = make_uint4(u[4], u[5], u[6], u[7]);
  }
}
__device__ __forceinline__ bool is_wide(const void* x, long long xt, long long xh) {
  return ((reinterpret_cast<unsigned long long>(x) | (unsigned long long)(2 * xt) | (unsigned long long)(2 * xh)) & 31) == 0;
}

template <bool BF16>
__global__ void __launch_bounds__(kThreadsC, kAppendCtas) kv4_append_kernel(const __grid_constant__ Kv4RowsLaunch p) {
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
  const bool wide = is_wide(x, xt, xh);
  uint8_t *codes = is_v ? p.c.vc : p.c.kc, *scales = is_v ? p.c.vs : p.c.ks;
  const unsigned tokens = (unsigned)p.tokens;
  for (RowWalk walk(p, blockIdx.x * kThreadsC + threadIdx.x, gridDim.x * kThreadsC); walk.r.token < tokens;) {
    uint32_t u[kFlightC][8];
    long long at[kFlightC];
#pragma unroll
    for (int f = 0; f < kFlightC; ++f) {
      at[f] = -1;
      if (walk.r.token < tokens) {
        load_block(x + row_offset(p, walk.r, xt, xh), wide, u[f]);
        at[f] = cache_block(p, walk.r, p.slots[walk.r.token]);
      }
      walk.next();
    }
#pragma unroll
    for (int f = 0; f < kFlightC; ++f) {
      if (at[f] < 0) continue;
      uint64_t v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t m = u[f][j] ^ 0x80008000u;             // -x
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
__global__ void __launch_bounds__(kThreadsC, kReadCtas) kv4_read_kernel(const __grid_constant__ Kv4RowsLaunch p) {
  griddep_wait();
  griddep_launch_dependents();
  const bool is_v = blockIdx.y;
  uint16_t* y = static_cast<uint16_t*>(is_v ? p.v_out : p.k_out);
  const long long yt = is_v ? p.vt : p.kt, yh = is_v ? p.vh : p.kh;
  const bool wide = is_wide(y, yt, yh);
  const uint8_t *codes = is_v ? p.c.vc : p.c.kc, *scales = is_v ? p.c.vs : p.c.ks;
  const unsigned tokens = (unsigned)p.tokens;
  for (RowWalk walk(p, blockIdx.x * kThreadsC + threadIdx.x, gridDim.x * kThreadsC); walk.r.token < tokens;) {
    uint2 c[kFlightC];
    uint32_t sb[kFlightC];
    RowBlock r[kFlightC];
#pragma unroll
    for (int f = 0; f < kFlightC; ++f) {
      c[f] = make_uint2(0, 0);
      sb[f] = 0;
      r[f] = walk.r;
      if (walk.r.token < tokens) {
        const long long at = cache_block(p, walk.r, p.slots[walk.r.token]);
        if (at >= 0) {
          c[f] = *reinterpret_cast<const uint2*>(codes + 8 * at);
          sb[f] = scales[at];
        }
      }
      walk.next();
    }
#pragma unroll
    for (int f = 0; f < kFlightC; ++f) {
      if (r[f].token >= tokens) continue;
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
      store_block(y + row_offset(p, r[f], yt, yh), wide, o);
    }
  }
}

cudaError_t launch(void (*kernel)(Kv4RowsLaunch), int ctas, const Kv4RowsLaunch& p, cudaStream_t stream) {
  const long long n = (long long)p.tokens * p.c.heads * (p.c.D / 16), need = (n + kThreadsC - 1) / kThreadsC;
  const long long resident = (long long)ctas / 2 * p.num_sms;  // for keys and for values each
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
  return launch(p.dtype == 0 ? kv4_append_kernel<true> : kv4_append_kernel<false>, kAppendCtas, p, stream);
}

cudaError_t launch_kv4_read(const Kv4RowsLaunch& p, cudaStream_t stream) {
  return launch(p.dtype == 0 ? kv4_read_kernel<true> : kv4_read_kernel<false>, kReadCtas, p, stream);
}

}  // namespace svdq

// kv4_common.cuh -- what the attention kernels over the 4-bit cache share:
// arithmetic helpers, the output row, the work description, launches.
#pragma once

#include <cuda_runtime.h>

#include <cfloat>

#include "attn_kernels.h"
#include "kcommon.cuh"
#include "kv4_codes.cuh"
#include "kv4_rows.cuh"
#include "ptx.cuh"

namespace svdq {

constexpr float kLog2e = 1.4426950408889634f;
// Weights are 2^(score - ref), rounded to fp16 for the product with the values.
// A row's reference is first set kRoom below its largest score, so that weights
// begin at 2^7, and set again when one would pass 2^kMost, half of fp16's range:
// what is lost below fp16's range is 2^-32 of the largest weight, not 2^-25 (over
// 131072 keys 2^-15 of a value at most, not 2^-8).
constexpr float kRoom = 7.0f, kMost = 15.0f;        // (log_sum has 2^-kRoom as a number)
constexpr uint32_t kAbsent = 0xFFFFFFFFu;             // no such cache row: past the keys, or in no page of the cache

__device__ __forceinline__ uint32_t hmul2u(uint32_t a, __half2 b) {
  const __half2 h = __hmul2(*reinterpret_cast<const __half2*>(&a), b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t half2u(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 2^(m - to), 0 for a part that saw nothing (m = -inf, whatever `to` is).
__device__ __forceinline__ float ex2_diff(float m, float to) { return m == -INFINITY ? 0.0f : ex2(m - to); }

// Eight stored values -> fp32.
template <bool BF16>
__device__ __forceinline__ void unpack8(uint4 w, float* v) {
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (BF16) {
      v[2 * i] = bf16lo_to_f32(x[i]);
      v[2 * i + 1] = bf16hi_to_f32(x[i]);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&x[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
}

// Exponent e with 2^e * big in [2^14, 2^15), clamped so that 2^e and 2^-e are normal numbers.
__device__ __forceinline__ int row_exponent(float big) {
  return big > 0.0f ? min(max(14 - (int)((__float_as_uint(big) >> 23) & 0xFF) + 127, -126), 126) : 0;
}

// Factor of a row's scores to exponents in base 2: its queries were scaled by 2^e.  Kept finite: a score of zero stays
// zero whatever the scale.  (Scale and log2 e alone may overflow where 2^-e brings their product back.)
__device__ __forceinline__ float row_factor(float scale, int e) {
  const float f = scale * (kLog2e * __uint_as_float((uint32_t)(127 - e) << 23));
  return fminf(fmaxf(f, -FLT_MAX), FLT_MAX);
}

// A row's log sum from its reference and its sum of weights (not 0).  The room is taken out of both first: a log of
// about 7 next to a reference of about -7 would round coarser than their sum.
__device__ __forceinline__ float log_sum(float ref, float total) {
  return (ref + kRoom + log2f(total * 0x1p-7f)) * 0.6931471805599453f;
}

// One 8-element piece of an output row: v / total in the storage type, and the
// row's log sum.  total == 0: the row saw no key (or only scores of -inf).
template <bool BF16>
__device__ __forceinline__ void store_row8(const Kv4AttnLaunch& p, long long token, int head, int d0,
                                           const float (&v)[8], float top, float total) {
  const float inv = total == 0.0f ? 0.0f : 1.0f / total;
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    w[j] = BF16 ? pack_bf16x2(v[2 * j] * inv, v[2 * j + 1] * inv) : half2u(v[2 * j] * inv, v[2 * j + 1] * inv);
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + token * p.ot + head * p.oh + d0) =
      make_uint4(w[0], w[1], w[2], w[3]);
  if (p.lse && d0 == 0)
    p.lse[token * p.q_heads + head] = total == 0.0f ? -INFINITY : log_sum(top, total);
}

__device__ __forceinline__ Kv4Work work_of(const Kv4AttnLaunch& p) {
  Kv4Work w;
  w.q_start = p.q_start;
  w.kv_len = p.kv_len;
  w.requests = p.requests;
  w.tokens = p.tokens;
  w.group = p.q_heads / p.c.heads;
  w.heads = p.c.heads;
  w.tile_rows = p.tile_rows;
  w.causal = p.causal;
  w.min_rows = p.min_rows;
  w.max_rows = p.max_rows;
  w.capacity = (long long)p.max_pages << p.c.page_log2;
  return w;
}

// The note of a segment that a CTA began and did not finish.
__device__ __forceinline__ Kv4Cut cut_of(const RowTile& t, int head, int last_cta, int slot) {
  Kv4Cut c = {};
  c.token0 = t.token0;
  c.row0 = t.row0;
  c.rows = t.rows;
  c.head = head;
  c.last_cta = last_cta;
  c.slot = slot;
  return c;
}

// Programmatic dependent launch: set-up overlaps the previous kernel's end.
template <typename... Args>
inline cudaError_t launch_after(void (*kernel)(Args...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                         const Kv4AttnLaunch& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace svdq

// kv4_attention.cu -- attention of a few query rows over the paged 4-bit cache
// (decoding, drafted tokens, short chunks).
//
// Query i of the n of request b stands at position L - n + i, L = kv_len[b],
// and sees keys j < L (causal: j <= its position); key j is row j % page of
// page table[b, j / page]:
//   s_j = scale q.k_j,  p = softmax(s),  o = sum_j p_j v_j,  lse = log sum_j exp(s_j);
// a query that sees no key gets o = 0 and lse = -inf.
//
// Work split.  The query heads that share a key head, times the request's
// tokens, are the rows of one tile (16 or 32); a CTA takes one tile, one key
// head and one part of the key axis, its four warps alternate 16-key tiles and
// join once at the end.  With several parts a second kernel joins them in
// order (no atomics: results do not depend on timing).
//
// Arithmetic.  Both products run on fp16 tensor-core MMAs (m16n8k16) with fp32
// sums.  A cache value, e2m1 x e4m3, has 6 significant bits and is exact in
// fp16, so dequantizing (cvt.e2m1x2, one packed multiply) rounds nothing.
// Queries are scaled per row by a power of two into fp16's range: bf16's 8 bits
// fit, and what falls below fp16's smallest subnormal is under 2^-38 of the
// row's largest value.  The softmax (base 2) is fp32; its weights, in [0, 1], are
// rounded to fp16 (2^-11 relative) for the second product only.
//
// Layout.  The MMA's contraction and column indexes are free to permute, and
// are chosen so that no dequantized value moves between lanes: lane (g, t) of
// the first product takes 1/4 of key row g's codes (16 bytes for D = 128, one
// shared-memory load), lane (g, t) of the second takes 1/8 of four keys' rows,
// the same four keys t, 4+t, 8+t, 12+t whose scores it holds; two keys' codes
// are interleaved as nibbles (two logic ops per 8 values) so that one convert
// gives the pair of rows an MMA operand wants.
//
// Bound: codes and scales are 9/16 byte a value, read once (HBM) with a ring of
// cp.async copies per warp (no barrier between warps); dequantizing costs
// about 1.2 instructions a value and lane, the same order as the memory time.
//
// Keys past L, pages outside the cache and everything masked for a row
// contribute nothing, NaN included: such rows of the ring are zero-filled, scores
// are selected, not added to, and a NaN value inside a partly masked tile is
// taken out of the product and given to the rows that see it.
#include <cuda_runtime.h>

#include "attn_kernels.h"
#include "kv4_codes.cuh"
#include "kv4_rows.cuh"
#include "kcommon.cuh"
#include "ptx.cuh"

namespace svdq {
namespace {

constexpr int kWarpsA = 4, kThreadsA = 32 * kWarpsA, kTileA = 16, kStagesA = 4;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
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
// a x b where a == 0 wins over any b: a factor exp2(-inf - m) of a part that saw nothing.
__device__ __forceinline__ float ex2_diff(float m, float to) { return m == -INFINITY ? 0.0f : ex2(m - to); }

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
    p.lse[token * p.q_heads + head] = total == 0.0f ? -INFINITY : (top + log2f(total)) * 0.6931471805599453f;
}

template <int D>
struct Tile {
  static constexpr int kCode = kTileA * D / 2, kScale = kTileA * D / 16;      // bytes of 16 keys
  static constexpr int kStage = 2 * kCode + 2 * kScale;
};
template <int D, int MT>
constexpr int smem_bytes() {
  const int ring = kWarpsA * kStagesA * Tile<D>::kStage;
  const int join = kWarpsA * 16 * MT * (D + 4) * 4 + kWarpsA * 16 * MT * 8;
  return ring > join ? ring : join;
}

// D: head dimension (64, 128).  MT: 16-row tiles per warp.  BF16: storage type of q and out.
template <int D, int MT, bool BF16>
__global__ void __launch_bounds__(kThreadsA, MT == 1 ? 3 : 2)
    kv4_attention_kernel(const __grid_constant__ Kv4AttnLaunch p) {
  constexpr int kRows = 16 * MT, kKS = D / 16, kDG = D / 8;       // MMA k-steps; head dims per lane group g
  constexpr int kCode = Tile<D>::kCode, kScale = Tile<D>::kScale, kStage = Tile<D>::kStage;
  extern __shared__ __align__(16) uint8_t smem[];

  const int group = p.q_heads / p.c.heads;
  const RowTile rt = find_row_tile(p.q_start, p.kv_len, p.requests, p.tokens, group, kRows, blockIdx.x,
                                   (long long)p.max_pages << p.c.page_log2, p.causal);
  if (rt.rows <= 0) return;
  const int active = active_parts(rt.last_key, p.splits, p.chunk);
  const int part = blockIdx.y;
  if (part >= active) return;
  const int k_begin = part * p.chunk, k_end = part == active - 1 ? rt.last_key : k_begin + p.chunk;
  const int kvh = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;

  // ---- ring: stage s of this warp holds one 16-key tile {K codes, V codes, K scales, V scales}
  const uint32_t ring = smem_u32(smem) + warp * (kStagesA * kStage);
  const int n_tiles = (k_end - k_begin + kTileA - 1) / kTileA;
  const int my_tiles = n_tiles > warp ? (n_tiles - warp + kWarpsA - 1) / kWarpsA : 0;
  const int* table = p.table + rt.request * p.table_stride;
  int page_ids = -1;                                      // lane i: page of this warp's tile (base + i)
  uint32_t absent = 0;                                    // bit it % 32: tile it lies in no page of the cache
  auto issue = [&](int it) {
    if ((it & 31) == 0) {
      const int k = k_begin + kTileA * (warp + kWarpsA * (it + lane));
      page_ids = it + lane < my_tiles ? table[k >> p.c.page_log2] : -1;
    }
    const int page = __shfl_sync(0xFFFFFFFFu, page_ids, it & 31);
    if (it < my_tiles) {
      const int k0 = k_begin + kTileA * (warp + kWarpsA * it);
      const bool ok = page >= 0 && page < p.c.pages;
      absent = (absent & ~(1u << (it & 31))) | ((ok ? 0u : 1u) << (it & 31));
      const int nv = ok ? min(kTileA, k_end - k0) : 0;    // keys of the tile that exist
      const long long row = ((((long long)(ok ? page : 0)) * p.c.heads + kvh) << p.c.page_log2) +
                            (k0 & ((1 << p.c.page_log2) - 1));
      const uint32_t dst = ring + (it % kStagesA) * kStage;
      constexpr int kChunks = kCode / 16, kPerKey = D / 32;           // 16-byte pieces: of a tile, of a key
#pragma unroll
      for (int i = 0; i < kChunks / 32; ++i) {
        const int c = lane + 32 * i;
        const int bytes = c / kPerKey < nv ? 16 : 0;
        cp_async16(dst + 16 * c, p.c.kc + row * (D / 2) + 16 * c, bytes);
        cp_async16(dst + kCode + 16 * c, p.c.vc + row * (D / 2) + 16 * c, bytes);
      }
      constexpr int kSc = kScale / 16;                                // 16-byte pieces of one tensor's scales
      if (lane < 2 * kSc) {
        const int c = lane % kSc;
        const uint8_t* src = (lane < kSc ? p.c.ks : p.c.vs) + row * (D / 16) + 16 * c;
        cp_async16(dst + 2 * kCode + 16 * lane, src, max(0, min(16, nv * (D / 16) - 16 * c)));
      }
    }
    cp_commit();
  };
#pragma unroll
  for (int s = 0; s < kStagesA - 1; ++s) issue(s);

  // ---- queries: rows g and g + 8 of each 16-row tile, this lane's quarter of the head
  uint32_t qa[MT][kKS][4];
  float qs[MT][2];                                        // row factor: scale * log2e / 2^shift
  int lim[MT][2];                                         // keys the row sees
#pragma unroll
  for (int m = 0; m < MT; ++m) {
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const int r = 16 * m + 8 * hf + g;
      float f[D / 4];
      lim[m][hf] = 0;
#pragma unroll
      for (int i = 0; i < D / 4; ++i) f[i] = 0.0f;
      if (r < rt.rows) {
        const int row = rt.row0 + r, tok = row / group, head = kvh * group + row - tok * group;
        lim[m][hf] = rt.keys_of(tok, p.causal);
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) +
                                                          (long long)(rt.token0 + tok) * p.qt + head * p.qh + t * (D / 4));
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const uint4 w = src[i];
          const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (BF16) {
              f[8 * i + 2 * j] = bf16lo_to_f32(x[j]);
              f[8 * i + 2 * j + 1] = bf16hi_to_f32(x[j]);
            } else {
              const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&x[j]));
              f[8 * i + 2 * j] = v.x;
              f[8 * i + 2 * j + 1] = v.y;
            }
          }
        }
      }
      // Power of two that takes the row's largest finite magnitude to [2^14, 2^15).
      float mx = 0.0f;
#pragma unroll
      for (int i = 0; i < D / 4; ++i) mx = fmaxf(mx, fabsf(f[i]) < INFINITY ? fabsf(f[i]) : 0.0f);
      mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
      // Exponent clamped so that both 2^e and 2^-e are normal numbers.
      const int e = mx > 0.0f ? min(max(14 - (int)((__float_as_uint(mx) >> 23) & 0xFF) + 127, -126), 126) : 0;
      const float up = __uint_as_float((uint32_t)(127 + e) << 23);
      qs[m][hf] = p.scale * kLog2e * __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
      for (int j = 0; j < kKS; ++j) {
        qa[m][j][hf] = half2u(f[4 * j] * up, f[4 * j + 1] * up);
        qa[m][j][2 + hf] = half2u(f[4 * j + 2] * up, f[4 * j + 3] * up);
      }
    }
  }
  // Tiles that end at or before the first row's keys need no mask.
  const int free_end = min(rt.keys_of(rt.row0 / group, p.causal), k_end);

  float o[MT][kDG][4], mx[MT][2], sum[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    mx[m][0] = mx[m][1] = -INFINITY;
    sum[m][0] = sum[m][1] = 0.0f;
#pragma unroll
    for (int i = 0; i < kDG; ++i) o[m][i][0] = o[m][i][1] = o[m][i][2] = o[m][i][3] = 0.0f;
  }

  for (int it = 0; it < my_tiles; ++it) {
    issue(it + kStagesA - 1);
    cp_wait<kStagesA - 1>();
    __syncwarp();
    if ((absent >> (it & 31)) & 1u) continue;
    const uint8_t* st = smem + warp * (kStagesA * kStage) + (it % kStagesA) * kStage;
    const int k0 = k_begin + kTileA * (warp + kWarpsA * it);

    // ---- scores: column n of the MMA is key (n >> 1) + 4 (n & 1) of its 8-key half
    float s[MT][2][4];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
      const int key = 8 * nt + (g >> 1) + 4 * (g & 1);
      uint32_t w[D / 32];
      __half2 sc[2];
      if (D == 128) {
        const uint4 c = *reinterpret_cast<const uint4*>(st + key * 64 + 16 * t);
        w[0] = c.x, w[1] = c.y, w[2 % (D / 32)] = c.z, w[3 % (D / 32)] = c.w;
        const __half2 two = e4m3x2_to_half2(*reinterpret_cast<const uint16_t*>(st + 2 * kCode + key * 8 + 2 * t));
        sc[0] = __low2half2(two);
        sc[1] = __high2half2(two);
      } else {
        const uint2 c = *reinterpret_cast<const uint2*>(st + key * 32 + 8 * t);
        w[0] = c.x, w[1] = c.y;
        const uint32_t b = st[2 * kCode + key * 4 + t];
        sc[0] = sc[1] = e4m3x2_to_half2(b | (b << 8));
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) s[m][nt][0] = s[m][nt][1] = s[m][nt][2] = s[m][nt][3] = 0.0f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        uint32_t d[4];
        e2m1x8_to_f16x8(w[i], d);
        const __half2 f = sc[i / 2];
#pragma unroll
        for (int j = 0; j < 4; ++j) d[j] = hmul2u(d[j], f);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          mma16816(s[m][nt], qa[m][2 * i], d[0], d[1]);
          mma16816(s[m][nt], qa[m][2 * i + 1], d[2], d[3]);
        }
      }
    }

    // ---- softmax weights of keys t, 4+t (nt 0) and 8+t, 12+t (nt 1)
    const bool masked = k0 + kTileA > free_end;
    uint32_t pa[MT][4];
    bool grew = false;
    float to[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          s[m][nt][c] *= qs[m][c >> 1];
          if (masked && k0 + 8 * nt + t + 4 * (c & 1) >= lim[m][c >> 1]) s[m][nt][c] = -INFINITY;
        }
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        float v = fmaxf(fmaxf(s[m][0][2 * hf], s[m][0][2 * hf + 1]), fmaxf(s[m][1][2 * hf], s[m][1][2 * hf + 1]));
        v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 1));
        v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 2));
        to[m][hf] = fmaxf(mx[m][hf], v);
        grew |= to[m][hf] > mx[m][hf];
      }
    }
    if (__any_sync(0xFFFFFFFFu, grew)) {
#pragma unroll
      for (int m = 0; m < MT; ++m) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const float f = ex2_diff(mx[m][hf], to[m][hf]);
          mx[m][hf] = to[m][hf];
          sum[m][hf] *= f;
#pragma unroll
          for (int i = 0; i < kDG; ++i) {
            o[m][i][2 * hf] *= f;
            o[m][i][2 * hf + 1] *= f;
          }
        }
      }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const float base = mx[m][hf] == -INFINITY ? 0.0f : mx[m][hf];
        float e[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          e[c] = ex2(s[m][c >> 1][2 * hf + (c & 1)] - base);
          sum[m][hf] += e[c];
        }
        pa[m][hf] = half2u(e[0], e[1]);
        pa[m][2 + hf] = half2u(e[2], e[3]);
      }
    }

    // ---- values: lane (g, t) takes dims kDG g .. of keys t, 4+t, 8+t, 12+t
    const uint8_t* vs = st + 2 * kCode + kScale + (D == 128 ? g : g >> 1);
    uint32_t sb[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) sb[c] = vs[(t + 4 * c) * (D / 16)];
    if (masked) {
      bool bad = false;
#pragma unroll
      for (int c = 0; c < 4; ++c) bad |= (sb[c] & 0x7Fu) == 0x7Fu;
      if (__any_sync(0xFFFFFFFFu, bad)) {
        // A NaN value that some rows may not see: which (row, 16-dim block)
        // pairs see one, as an MMA of 0/1 operands; then it leaves the product.
        constexpr uint32_t kOne = 0x3C00u;
        uint32_t b[2];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          b[nt] = 0;
#pragma unroll
          for (int c = 0; c < 2; ++c)
            if ((sb[2 * nt + c] & 0x7Fu) == 0x7Fu) {
              b[nt] |= kOne << (16 * c);
              sb[2 * nt + c] = 0;
            }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          uint32_t a[4];
          float hit[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
              a[2 * nt + hf] = (k0 + 8 * nt + t < lim[m][hf] ? kOne : 0u) |
                               (k0 + 8 * nt + 4 + t < lim[m][hf] ? kOne << 16 : 0u);
          mma16816(hit, a, b[0], b[1]);
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (hit[c] > 0.0f) {
#pragma unroll
              for (int i = 0; i < kDG; ++i) o[m][i][c] = __uint_as_float(0x7FC00000u);
            }
        }
      }
    }
    const __half2 s01 = e4m3x2_to_half2(sb[0] | (sb[1] << 8)), s23 = e4m3x2_to_half2(sb[2] | (sb[3] << 8));
    uint32_t vw[4][D / 64];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint8_t* src = st + kCode + (t + 4 * c) * (D / 2) + g * (D / 16);
      if (D == 128) {
        const uint2 w = *reinterpret_cast<const uint2*>(src);
        vw[c][0] = w.x, vw[c][D / 64 - 1] = w.y;
      } else {
        vw[c][0] = *reinterpret_cast<const uint32_t*>(src);
      }
    }
#pragma unroll
    for (int h = 0; h < D / 64; ++h) {
      uint32_t ev[2][4], od[2][4];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        const uint32_t a = vw[2 * nt][h], b = vw[2 * nt + 1][h];
        e2m1x8_to_f16x8((a & 0x0F0F0F0Fu) | ((b << 4) & 0xF0F0F0F0u), ev[nt]);
        e2m1x8_to_f16x8(((a >> 4) & 0x0F0F0F0Fu) | (b & 0xF0F0F0F0u), od[nt]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t e0 = hmul2u(ev[0][j], s01), e1 = hmul2u(ev[1][j], s23);
        const uint32_t d0 = hmul2u(od[0][j], s01), d1 = hmul2u(od[1][j], s23);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          mma16816(o[m][8 * h + 2 * j], pa[m], e0, e1);
          mma16816(o[m][8 * h + 2 * j + 1], pa[m], d0, d1);
        }
      }
    }
    __syncwarp();                                         // the ring slot is free again
  }
  cp_wait<0>();

  // ---- join the four warps: o holds dims kDG * (2t), kDG * (2t+1) onward of rows g, g + 8
  float* jo = reinterpret_cast<float*>(smem);
  float2* jm = reinterpret_cast<float2*>(smem + kWarpsA * kRows * (D + 4) * 4);
  __syncthreads();                                        // every warp has left its ring
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      float v = sum[m][hf];
      v += __shfl_xor_sync(0xFFFFFFFFu, v, 1);
      v += __shfl_xor_sync(0xFFFFFFFFu, v, 2);
      const int r = 16 * m + 8 * hf + g;
      if (t == 0) jm[warp * kRows + r] = make_float2(mx[m][hf], v);
      float* dst = jo + (warp * kRows + r) * (D + 4);
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int i = 0; i < kDG; i += 4)
          *reinterpret_cast<float4*>(dst + kDG * (2 * t + c) + i) =
              make_float4(o[m][i][2 * hf + c], o[m][i + 1][2 * hf + c], o[m][i + 2][2 * hf + c], o[m][i + 3][2 * hf + c]);
    }
  __syncthreads();
  constexpr int kVec = D / 8;
  for (int i = threadIdx.x; i < rt.rows * kVec; i += kThreadsA) {
    const int r = i / kVec, d0 = 8 * (i % kVec);
    float top = -INFINITY, total = 0.0f, v[8];
#pragma unroll
    for (int w = 0; w < kWarpsA; ++w) top = fmaxf(top, jm[w * kRows + r].x);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarpsA; ++w) {
      const float2 ml = jm[w * kRows + r];
      const float f = ex2_diff(ml.x, top);
      total = fmaf(ml.y, f, total);
      const float4* src = reinterpret_cast<const float4*>(jo + (w * kRows + r) * (D + 4) + d0);
      const float4 a = src[0], b = src[1];
      v[0] = fmaf(a.x, f, v[0]), v[1] = fmaf(a.y, f, v[1]), v[2] = fmaf(a.z, f, v[2]), v[3] = fmaf(a.w, f, v[3]);
      v[4] = fmaf(b.x, f, v[4]), v[5] = fmaf(b.y, f, v[5]), v[6] = fmaf(b.z, f, v[6]), v[7] = fmaf(b.w, f, v[7]);
    }
    const int row = rt.row0 + r, tok = row / group, head = kvh * group + row - tok * group;
    const long long token = rt.token0 + tok;
    if (active == 1) {
      store_row8<BF16>(p, token, head, d0, v, top, total);
    } else {
      const long long at = ((long long)part * p.tokens + token) * p.q_heads + head;
      float4* dst = reinterpret_cast<float4*>(p.part_o + at * D + d0);
      dst[0] = make_float4(v[0], v[1], v[2], v[3]);
      dst[1] = make_float4(v[4], v[5], v[6], v[7]);
      if (d0 == 0) p.part_ml[at] = make_float2(top, total);
    }
  }
}

// Joins the parts of the key axis, in order: D/8 threads per (token, head).
template <int D, bool BF16>
__global__ void __launch_bounds__(128) kv4_join_kernel(const __grid_constant__ Kv4AttnLaunch p, int tile_rows) {
  griddep_wait();
  constexpr int kVec = D / 8, kPer = 128 / kVec;
  const int group = p.q_heads / p.c.heads;
  const long long i = (long long)blockIdx.x * kPer + threadIdx.x / kVec;
  if (i >= (long long)p.tokens * p.q_heads) return;
  const int token = (int)(i / p.q_heads), head = (int)(i % p.q_heads), d0 = 8 * (threadIdx.x % kVec);
  const int last_key = find_last_key(p.q_start, p.kv_len, p.requests, p.tokens, token, group, head % group, tile_rows,
                                     (long long)p.max_pages << p.c.page_log2, p.causal);
  if (last_key < 0) return;                               // behind the last sequence
  const int active = active_parts(last_key, p.splits, p.chunk);
  if (active == 1) return;                                // written by the first kernel
  const long long step = (long long)p.tokens * p.q_heads;
  float top = -INFINITY, total = 0.0f, v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  for (int s = 0; s < active; ++s) top = fmaxf(top, p.part_ml[s * step + i].x);
  for (int s = 0; s < active; ++s) {
    const float2 ml = p.part_ml[s * step + i];
    const float f = ex2_diff(ml.x, top);
    total = fmaf(ml.y, f, total);
    const float4* src = reinterpret_cast<const float4*>(p.part_o + (s * step + i) * D + d0);
    const float4 a = src[0], b = src[1];
    v[0] = fmaf(a.x, f, v[0]), v[1] = fmaf(a.y, f, v[1]), v[2] = fmaf(a.z, f, v[2]), v[3] = fmaf(a.w, f, v[3]);
    v[4] = fmaf(b.x, f, v[4]), v[5] = fmaf(b.y, f, v[5]), v[6] = fmaf(b.z, f, v[6]), v[7] = fmaf(b.w, f, v[7]);
  }
  store_row8<BF16>(p, token, head, d0, v, top, total);
}

int tile_rows_for(const Kv4AttnLaunch& p) {
  const int group = p.q_heads / p.c.heads;
  // Rows of an average request; 32-row tiles dequantize each key once for twice the rows.
  return (long long)p.tokens * group > 16ll * p.requests ? 32 : 16;
}
long long row_tiles_for(const Kv4AttnLaunch& p, int rows) {
  return max_row_tiles(p.tokens, p.requests, p.q_heads / p.c.heads, rows, p.q_start != nullptr);
}

template <int D, int MT, bool BF16>
cudaError_t launch_mt(const Kv4AttnLaunch& p, cudaStream_t stream) {
  constexpr int kSmem = smem_bytes<D, MT>();
  cudaError_t e = ensure_smem_limit(kv4_attention_kernel<D, MT, BF16>, kSmem);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)row_tiles_for(p, 16 * MT), (unsigned)p.splits, (unsigned)p.c.heads);
  kv4_attention_kernel<D, MT, BF16><<<grid, kThreadsA, kSmem, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.splits == 1) return e;
  cudaLaunchConfig_t cfg = {};
  constexpr int kPer = 128 / (D / 8);
  cfg.gridDim = dim3((unsigned)(((long long)p.tokens * p.q_heads + kPer - 1) / kPer));
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kv4_join_kernel<D, BF16>, p, 16 * MT);
}

template <int D, bool BF16>
cudaError_t launch_d(const Kv4AttnLaunch& p, cudaStream_t stream) {
  return tile_rows_for(p) == 16 ? launch_mt<D, 1, BF16>(p, stream) : launch_mt<D, 2, BF16>(p, stream);
}

}  // namespace

void kv4_attention_plan(Kv4AttnLaunch& p, int max_kv) {
  // Parts of the key axis: enough CTAs for about three an SM, at least one
  // 16-key tile a warp each.
  const int rows = tile_rows_for(p);
  const long long ctas = row_tiles_for(p, rows) * p.c.heads, want = 3 * 148;
  const int step = kTileA * kWarpsA;
  if (max_kv < 1) max_kv = 1;
  long long parts = (want + ctas - 1) / ctas;
  const long long most = (max_kv + step - 1) / step;
  if (parts > most) parts = most;
  if (parts > 128) parts = 128;
  if (parts < 1) parts = 1;
  p.chunk = (int)(((max_kv + parts - 1) / parts + step - 1) / step * step);
  p.splits = (max_kv + p.chunk - 1) / p.chunk;
}

size_t kv4_attention_workspace(const Kv4AttnLaunch& p) {
  if (p.splits <= 1) return 0;
  return (size_t)p.splits * p.tokens * p.q_heads * ((size_t)p.c.D * 4 + 8);
}

cudaError_t launch_kv4_attention(const Kv4AttnLaunch& p0, void* workspace, cudaStream_t stream) {
  Kv4AttnLaunch p = p0;
  p.part_o = static_cast<float*>(workspace);
  p.part_ml = p.splits > 1 ? reinterpret_cast<float2*>(p.part_o + (size_t)p.splits * p.tokens * p.q_heads * p.c.D)
                           : nullptr;
  if (p.c.D == 128)
    return p.dtype == 0 ? launch_d<128, true>(p, stream) : launch_d<128, false>(p, stream);
  return p.dtype == 0 ? launch_d<64, true>(p, stream) : launch_d<64, false>(p, stream);
}

}  // namespace svdq

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
// tokens, are the rows of one tile (8, 16, 24 or 32).  One resident set of CTAs takes
// equal shares of all keys of all tiles and heads (kv4_rows.cuh), so unequal
// lengths and counts that do not divide leave no SM idle; a share starts and
// ends wherever it falls.  A CTA's four warps alternate 32-key tiles and join
// once per tile; what a share's end cuts is joined by a second kernel, in
// order (no atomics: results do not depend on timing).
//
// Arithmetic.  Both products run on fp16 tensor-core MMAs (m16n8k16) with fp32
// sums.  A cache value, e2m1 x e4m3, has 6 significant bits and is exact in
// fp16, so dequantizing (cvt.e2m1x2, one packed multiply) rounds nothing.
// Queries are scaled per row by a power of two into fp16's range: bf16's 8 bits
// fit, and what falls below fp16's smallest subnormal is under 2^-38 of the
// row's largest value.  The softmax (base 2) is fp32; its weights are rounded to
// fp16 for the second product only: 2^-11 relative, or 2^-32 of the row's largest
// (kv4_common.cuh).
//
// Layout.  Both products are transposed, keys (dims) on the MMA's 16 rows and
// query rows on its 8 columns: at one to eight query rows a key head, the usual
// case of decoding, nothing of the MMA or the softmax is wasted.  The
// contraction and row indexes are free to permute, and are chosen so that no
// dequantized value moves between lanes: lane (g, t) of the first product takes
// a quarter of two key rows (16 bytes each for D = 128, one shared-memory
// load), lane (g, t) of the second an eighth of the rows of keys t, 4+t, 8+t,
// 12+t; two keys' codes are interleaved as nibbles (two logic ops per 8 values)
// so that one convert gives the pair of keys an MMA operand wants.  Only the
// weights change lanes (an 8x8 transpose, movmatrix).
//
// Bound: codes and scales are 9/16 byte a value, read once (HBM), through a ring
// of cp.async copies per warp (no barrier between warps).  64 sequences of up to
// 8192 keys, 32 query and 8 key heads: 102 us, 4.4 TB/s; two of 131059 keys, 4 key
// heads: 40 us, 3.7 TB/s; one of 1021 keys: 8.3 us, set-up and latencies.  No unit
// is full on the first (second): issue slots 62% (59), 2.2 (2.0) instructions a
// clock, the ALU pipe 54% (51), DRAM 53% (46).  About 620 warp instructions per 32
// keys of one head (D = 128, up to 8 rows), 256 of which convert and scale the 8192
// values (cvt.e2m1x2 takes any byte of a register; the same from shifts and logic
// is 2.2 times slower), run on 3.5 warps a scheduler that wait on their own results,
// and 30% of the shared-memory wavefronts are bank conflicts of the code loads
// (keys k and k + 4 of the first product, k and k + 2 of the second).  16-key
// tiles: 128 us on the first case; five CTAs an SM, with spills, 129.
//
// Keys past L, pages outside the cache and everything masked for a row
// contribute nothing, NaN included: such rows of the ring are zero-filled, scores
// are selected, not added to, and a NaN value inside a partly masked tile is
// taken out of the product and given to the rows that see it.
#include <cuda_runtime.h>

#include "kv4_common.cuh"

namespace svdq {
namespace {

constexpr int kWarpsA = 4, kThreadsA = 32 * kWarpsA, kTileA = 32, kStagesA = 2;
// Resident CTAs an SM by head dimension and rows of a tile / 8: what the accumulators leave room for.
__host__ __device__ constexpr int ctas_per_sm(int d, int nt) {
  return d == 64 ? (nt == 1 ? 5 : nt == 2 ? 4 : nt == 3 ? 3 : 2) : (nt == 1 ? 4 : nt == 2 ? 3 : 2);
}
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
// Transposes an 8x8 matrix of 16-bit values held row-wise by the warp.
__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
template <int D>
struct Tile {
  static constexpr int kCode = kTileA * D / 2, kScale = kTileA * D / 16;      // bytes of 32 keys
  static constexpr int kStage = 2 * kCode + 2 * kScale;
};
template <int D, int NT>
constexpr int smem_bytes() {
  const int ring = kWarpsA * kStagesA * Tile<D>::kStage;
  const int join = kWarpsA * 8 * NT * (D + 4) * 4 + kWarpsA * 8 * NT * 8;
  return (ring > join ? ring : join) + NT * (D / 32) * 512 + 8 * NT * 8;
}

// Keys [k_begin, k_end) of one segment: its rows' unnormalized outputs, maxima
// and sums, joined over the CTA's warps, finished (whole) or left as a part.
// D: head dimension (64, 128).  NT: 8-row tiles.  BF16: storage type of q and out.
template <int D, int NT, bool BF16>
__device__ __forceinline__ void attend_segment(const Kv4AttnLaunch& p, const RowTile& rt, int kvh, int k_begin, int k_end,
                                               bool whole, long long part) {
  constexpr int kRows = 8 * NT, kDM = D / 16;                     // rows of the tile; 16-dim tiles of the output
  constexpr int kCode = Tile<D>::kCode, kScale = Tile<D>::kScale, kStage = Tile<D>::kStage;
  extern __shared__ __align__(16) uint8_t smem[];
  const int group = p.q_heads / p.c.heads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;

  // ---- ring: stage s of this warp holds one 32-key tile {K codes, V codes, K scales, V scales}
  const uint32_t ring = smem_u32(smem) + warp * (kStagesA * kStage);
  const int n_tiles = (k_end - k_begin + kTileA - 1) / kTileA;
  const int my_tiles = n_tiles > warp ? (n_tiles - warp + kWarpsA - 1) / kWarpsA : 0;
  const int* table = p.table + rt.request * p.table_stride;
  uint32_t rows16 = kAbsent;                              // lane i: cache row of 16-key half i & 1 of tile base + i / 2
  uint32_t absent = 0;                                    // bits 2 (it % 16) + u: half u of tile it is in no page
  auto issue = [&](int it) {
    if ((it & 15) == 0) {
      const int k = k_begin + kTileA * (warp + kWarpsA * (it + (lane >> 1))) + 16 * (lane & 1);
      rows16 = kAbsent;
      if (it + (lane >> 1) < my_tiles && k < k_end) {
        const int page = table[k >> p.c.page_log2];
        if (page >= 0 && page < p.c.pages)
          rows16 = ((((uint32_t)page * p.c.heads) + kvh) << p.c.page_log2) + (k & ((1 << p.c.page_log2) - 1));
      }
    }
    uint32_t row[2];
    row[0] = __shfl_sync(0xFFFFFFFFu, rows16, 2 * (it & 15));
    row[1] = __shfl_sync(0xFFFFFFFFu, rows16, 2 * (it & 15) + 1);
    if (it < my_tiles) {
      const int k0 = k_begin + kTileA * (warp + kWarpsA * it), sh = 2 * (it & 15);
      absent = (absent & ~(3u << sh)) | ((row[0] == kAbsent ? 1u : 0u) << sh) | ((row[1] == kAbsent ? 2u : 0u) << sh);
      const uint32_t dst = ring + (it % kStagesA) * kStage + 16 * lane;
      constexpr int kPerHalf = D / 64;                    // 16-byte pieces a lane of one half's codes
      constexpr int kSc = D / 16;                         // 16-byte pieces of one half's scales
      const int tensor = lane / (2 * kSc), su = lane / kSc & 1, sp = lane % kSc;
      const uint8_t* scales = (tensor ? p.c.vs : p.c.ks) + 16 * sp;
      if (row[0] != kAbsent && row[1] != kAbsent && k0 + kTileA <= k_end) {
#pragma unroll
        for (int i = 0; i < 2 * kPerHalf; ++i) {
          const size_t at = (size_t)row[i / kPerHalf] * (D / 2) + 16 * (lane + 32 * (i % kPerHalf));
          cp_async16(dst + 512 * i, p.c.kc + at, 16);
          cp_async16(dst + kCode + 512 * i, p.c.vc + at, 16);
        }
        if (lane < 4 * kSc) cp_async16(dst + 2 * kCode, scales + (size_t)row[su] * (D / 16), 16);
      } else {                                            // rows that do not exist become zeros
        int nv[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          nv[u] = row[u] == kAbsent ? 0 : min(16, k_end - k0 - 16 * u);
          if (row[u] == kAbsent) row[u] = 0;
        }
#pragma unroll
        for (int i = 0; i < 2 * kPerHalf; ++i) {
          const int c = lane + 32 * (i % kPerHalf), bytes = c / (D / 32) < nv[i / kPerHalf] ? 16 : 0;
          const size_t at = (size_t)row[i / kPerHalf] * (D / 2) + 16 * c;
          cp_async16(dst + 512 * i, p.c.kc + at, bytes);
          cp_async16(dst + kCode + 512 * i, p.c.vc + at, bytes);
        }
        if (lane < 4 * kSc)
          cp_async16(dst + 2 * kCode, scales + (size_t)row[su] * (D / 16), max(0, min(16, nv[su] * (D / 16) - 16 * sp)));
      }
    }
    cp_commit();
  };
  // The queries' loads first: they are under way while the page numbers come.  Lane (g, t) takes row g of an 8-row tile, a
  // quarter of the head; warp w the tile w (NT <= 4).
  static_assert(NT <= kWarpsA, "one 8-row tile a warp");
  uint4 q_raw[D / 32];
  int q_sees = 0;                                         // keys that this row sees
#pragma unroll
  for (int i = 0; i < D / 32; ++i) q_raw[i] = make_uint4(0, 0, 0, 0);
  if (warp < NT && 8 * warp + g < rt.rows) {
    const int row = rt.row0 + 8 * warp + g, tok = (int)((uint32_t)row / (uint32_t)group);
    const int head = kvh * group + row - tok * group;
    q_sees = rt.keys_of(tok, p.causal);
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) +
                                                      (long long)(rt.token0 + tok) * p.qt + head * p.qh + t * (D / 4));
#pragma unroll
    for (int i = 0; i < D / 32; ++i) q_raw[i] = src[i];
  }
#pragma unroll
  for (int s = 0; s < kStagesA - 1; ++s) issue(s);

  // ---- queries, as the first product's column operand: in shared memory, for every two MMA steps one 16-byte piece a lane
  constexpr int kQ = smem_bytes<D, NT>() - NT * (D / 32) * 512 - kRows * 8;
  uint4* qsm = reinterpret_cast<uint4*>(smem + kQ);                             // [NT][D / 32][32 lanes]
  float* back = reinterpret_cast<float*>(smem + kQ + NT * (D / 32) * 512);      // [rows] scale * log2e / 2^shift
  int* sees = reinterpret_cast<int*>(back + kRows);                             // [rows] keys that the row sees
  if (warp < NT) {
    float f[D / 4];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) unpack8<BF16>(q_raw[i], f + 8 * i);
    // Power of two that takes the row's largest finite magnitude to [2^14, 2^15).
    float big = 0.0f;
#pragma unroll
    for (int i = 0; i < D / 4; ++i) big = fmaxf(big, fabsf(f[i]) < INFINITY ? fabsf(f[i]) : 0.0f);
    big = fmaxf(big, __shfl_xor_sync(0xFFFFFFFFu, big, 1));
    big = fmaxf(big, __shfl_xor_sync(0xFFFFFFFFu, big, 2));
    const int e = row_exponent(big);
    const float up = __uint_as_float((uint32_t)(127 + e) << 23);
    if (t == 0) {
      back[8 * warp + g] = row_factor(p.scale, e);
      sees[8 * warp + g] = q_sees;
    }
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
      qsm[(warp * (D / 32) + i) * 32 + lane] =
          make_uint4(half2u(f[8 * i] * up, f[8 * i + 1] * up), half2u(f[8 * i + 2] * up, f[8 * i + 3] * up),
                     half2u(f[8 * i + 4] * up, f[8 * i + 5] * up), half2u(f[8 * i + 6] * up, f[8 * i + 7] * up));
  }
  __syncthreads();
  float qs[NT][2];                                        // factor of rows 2t, 2t + 1
  int lim[NT][2];                                         // keys that they see
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      qs[n][c] = back[8 * n + 2 * t + c];
      lim[n][c] = sees[8 * n + 2 * t + c];
    }
  // Tiles that end at or before the first row's keys need no mask.
  const int free_end = min(rt.keys_of((int)((uint32_t)rt.row0 / (uint32_t)group), p.causal), k_end);

  // Rows 2t, 2t + 1 of each tile: reference exponent (base 2), sum of weights, outputs.
  float o[NT][kDM][4], ref[NT][2], sum[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    ref[n][0] = ref[n][1] = -INFINITY;
    sum[n][0] = sum[n][1] = 0.0f;
#pragma unroll
    for (int i = 0; i < kDM; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.0f;
  }

  for (int it = 0; it < my_tiles; ++it) {
    issue(it + kStagesA - 1);
    cp_wait<kStagesA - 1>();
    __syncwarp();
    const uint32_t gone = (absent >> (2 * (it & 15))) & 3u;
    if (gone == 3u) continue;
    const uint8_t* st = smem + warp * (kStagesA * kStage) + (it % kStagesA) * kStage;
    const int k0 = k_begin + kTileA * (warp + kWarpsA * it);

    // ---- scores (keys x rows), one MMA row tile per 16-key half u: its row r is key (r >> 1) + 4 (r & 1) (+ 8 for r >= 8)
    float s[2][NT][4];
    uint32_t w[2][2][D / 32];
    __half2 sc[2][2][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int n = 0; n < NT; ++n) s[u][n][0] = s[u][n][1] = s[u][n][2] = s[u][n][3] = 0.0f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = 16 * u + (g >> 1) + 4 * (g & 1) + 8 * h;
        if (D == 128) {
          const uint4 c = *reinterpret_cast<const uint4*>(st + k * 64 + 16 * t);
          w[u][h][0] = c.x, w[u][h][1] = c.y, w[u][h][2 % (D / 32)] = c.z, w[u][h][3 % (D / 32)] = c.w;
          const __half2 two = e4m3x2_to_half2(*reinterpret_cast<const uint16_t*>(st + 2 * kCode + k * 8 + 2 * t));
          sc[u][h][0] = __low2half2(two);
          sc[u][h][1] = __high2half2(two);
        } else {
          const uint2 c = *reinterpret_cast<const uint2*>(st + k * 32 + 8 * t);
          w[u][h][0] = c.x, w[u][h][1] = c.y;
          const uint32_t b = st[2 * kCode + k * 4 + t];
          sc[u][h][0] = sc[u][h][1] = e4m3x2_to_half2(b | (b << 8));
        }
      }
    }
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      uint32_t a[2][2][4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t d[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          e2m1x8_to_f16x8(w[u][h][i], d[h]);
#pragma unroll
          for (int j = 0; j < 4; ++j) a[u][j >> 1][h + 2 * (j & 1)] = hmul2u(d[h][j], sc[u][h][i / 2]);
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint4 q = qsm[(n * (D / 32) + i) * 32 + lane];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          mma16816(s[u][n], a[u][0], q.x, q.y);
          mma16816(s[u][n], a[u][1], q.z, q.w);
        }
      }
    }

    // ---- weights.  s[u][.][0..1]: key kg + 16u, rows 2t and 2t + 1; s[u][.][2..3]: key kg + 16u + 8.  The reference
    // exponent is raised only when a score exceeds it by more than kMost (or at a row's first key).
    const bool masked = gone != 0 || k0 + kTileA > free_end;
    const int kg = k0 + (g >> 1) + 4 * (g & 1);
    float x[2][NT][4];
    auto exponents = [&]() {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float base = ref[n][c & 1] == -INFINITY ? 0.0f : ref[n][c & 1];
            x[u][n][c] = fmaf(s[u][n][c], qs[n][c & 1], -base);
          }
      if (masked) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (((gone >> u) & 1u) || kg + 16 * u + 8 * (c >> 1) >= lim[n][c & 1]) x[u][n][c] = -INFINITY;
      }
    };
    exponents();
    bool over = false;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c)
        over |= fmaxf(fmaxf(x[0][n][c], x[0][n][2 + c]), fmaxf(x[1][n][c], x[1][n][2 + c])) >
                (ref[n][c] == -INFINITY ? -INFINITY : kMost);
    if (__any_sync(0xFFFFFFFFu, over)) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float v = fmaxf(fmaxf(x[0][n][c], x[0][n][2 + c]), fmaxf(x[1][n][c], x[1][n][2 + c]));
          v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 4));
          v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 8));
          v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 16));
          const float to = ref[n][c] == -INFINITY ? v - kRoom : ref[n][c] + fmaxf(v - kRoom, 0.0f);
          const float f = ex2_diff(ref[n][c], to);
          ref[n][c] = to;
          sum[n][c] *= f;
#pragma unroll
          for (int i = 0; i < kDM; ++i) {
            o[n][i][c] *= f;
            o[n][i][2 + c] *= f;
          }
        }
      exponents();
    }
    uint32_t pb[2][NT][2];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          x[u][n][c] = ex2(x[u][n][c]);
          sum[n][c & 1] += x[u][n][c];
        }
        // (key, rows 2t 2t+1) -> (keys 2t 2t+1, row g): the second product's operand.
        pb[u][n][0] = movmatrix(half2u(x[u][n][0], x[u][n][1]));
        pb[u][n][1] = movmatrix(half2u(x[u][n][2], x[u][n][3]));
      }

    // ---- values (dims x keys): lane (g, t) takes D/8 dims from D/8 g on, of keys t, 4+t, 8+t, 12+t of each half
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint8_t* vs = st + 2 * kCode + kScale + u * (kScale / 2) + (D == 128 ? g : g >> 1);
      uint32_t sb[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) sb[c] = vs[(t + 4 * c) * (D / 16)];
      if (masked) {
        bool bad = false;
#pragma unroll
        for (int c = 0; c < 4; ++c) bad |= (sb[c] & 0x7Fu) == 0x7Fu;
        if (__any_sync(0xFFFFFFFFu, bad)) {
          // A NaN value that some rows may not see: which (16-dim block, row)
          // pairs see one, as an MMA of 0/1 operands; then it leaves the product.
          constexpr uint32_t kOne = 0x3C00u;
          uint32_t a[4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t two = 0;
#pragma unroll
            for (int c = 0; c < 2; ++c)
              if ((sb[2 * h + c] & 0x7Fu) == 0x7Fu) {
                two |= kOne << (16 * c);
                sb[2 * h + c] = 0;
              }
            a[2 * h] = a[2 * h + 1] = two;
          }
          const int kt = k0 + 16 * u + t;
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const int see = sees[8 * n + g];
            uint32_t b[2];
            float hit[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int h = 0; h < 2; ++h)
              b[h] = (kt + 8 * h < see ? kOne : 0u) | (kt + 8 * h + 4 < see ? kOne << 16 : 0u);
            mma16816(hit, a, b[0], b[1]);
#pragma unroll
            for (int c = 0; c < 2; ++c)
              if (hit[c] > 0.0f) {
#pragma unroll
                for (int i = 0; i < kDM; ++i) o[n][i][c] = o[n][i][2 + c] = __uint_as_float(0x7FC00000u);
              }
          }
        }
      }
      const __half2 s01 = e4m3x2_to_half2(sb[0] | (sb[1] << 8)), s23 = e4m3x2_to_half2(sb[2] | (sb[3] << 8));
      uint32_t vw[4][D / 64];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint8_t* src = st + kCode + (16 * u + t + 4 * c) * (D / 2) + g * (D / 16);
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
        for (int q = 0; q < 2; ++q) {
          const uint32_t a = vw[2 * q][h], b = vw[2 * q + 1][h];
          e2m1x8_to_f16x8((a & 0x0F0F0F0Fu) | ((b << 4) & 0xF0F0F0F0u), ev[q]);
          e2m1x8_to_f16x8(((a >> 4) & 0x0F0F0F0Fu) | (b & 0xF0F0F0F0u), od[q]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t a[4] = {hmul2u(ev[0][j], s01), hmul2u(od[0][j], s01), hmul2u(ev[1][j], s23),
                                 hmul2u(od[1][j], s23)};
#pragma unroll
          for (int n = 0; n < NT; ++n) mma16816(o[n][4 * h + j], a, pb[u][n][0], pb[u][n][1]);
        }
      }
    }
    __syncwarp();                                         // the ring slot is free again
  }
  cp_wait<0>();

  // ---- join the four warps: o[n][i] holds dims D/8 g + 2i (c 0, 1) and + 2i + 1 (c 2, 3) of rows 2t, 2t + 1
  float* jo = reinterpret_cast<float*>(smem);
  float2* jm = reinterpret_cast<float2*>(smem + kWarpsA * kRows * (D + 4) * 4);
  __syncthreads();                                        // every warp has left its ring
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float v = sum[n][c];
      v += __shfl_xor_sync(0xFFFFFFFFu, v, 4);
      v += __shfl_xor_sync(0xFFFFFFFFu, v, 8);
      v += __shfl_xor_sync(0xFFFFFFFFu, v, 16);
      const int r = 8 * n + 2 * t + c;
      if (g == 0) jm[warp * kRows + r] = make_float2(ref[n][c], v);
      float* dst = jo + (warp * kRows + r) * (D + 4) + (D / 8) * g;
#pragma unroll
      for (int i = 0; i < kDM; i += 2)
        *reinterpret_cast<float4*>(dst + 2 * i) = make_float4(o[n][i][c], o[n][i][2 + c], o[n][i + 1][c], o[n][i + 1][2 + c]);
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
    const int row = rt.row0 + r, tok = (int)((uint32_t)row / (uint32_t)group), head = kvh * group + row - tok * group;
    const long long token = rt.token0 + tok;
    if (whole) {
      store_row8<BF16>(p, token, head, d0, v, top, total);
    } else {
      const long long at = part * kRows + r;
      float4* dst = reinterpret_cast<float4*>(p.part_o + at * D + d0);
      dst[0] = make_float4(v[0], v[1], v[2], v[3]);
      dst[1] = make_float4(v[4], v[5], v[6], v[7]);
      if (d0 == 0) p.part_ml[at] = make_float2(top, total);
    }
  }
}

template <int D, int NT, bool BF16>
__global__ void __launch_bounds__(kThreadsA, ctas_per_sm(D, NT))
    kv4_attention_kernel(const __grid_constant__ Kv4AttnLaunch p) {
  griddep_wait();
  griddep_launch_dependents();
  const Kv4Work w = work_of(p);
  const WarpUnits wu = warp_units(w);
  const long long per = kv4_div(wu.total + gridDim.x - 1, gridDim.x);
  const long long u0 = per * blockIdx.x, u1 = min(u0 + per, wu.total);
  bool noted = false;
  for (long long u = u0; u < u1;) {
    long long first;
    const int b = request_of_unit(w, wu, u, &first);
    const Segment sg = segment_in(w, span_of(w, b), b, u - first);
    const int n = (int)min((long long)(sg.units - sg.unit0), u1 - u);
    const bool whole = n == sg.units;
    attend_segment<D, NT, BF16>(p, sg.tile, sg.head, sg.unit0 * kUnitKeys,
                                min(sg.tile.last_key, (sg.unit0 + n) * kUnitKeys), whole,
                                2ll * blockIdx.x + (u == u0 ? 0 : 1));
    if (!whole && sg.unit0 == 0) {
      if (threadIdx.x == 0) p.cuts[blockIdx.x] = cut_of(sg.tile, sg.head, (int)kv4_div(u + sg.units - 1, per), u == u0 ? 0 : 1);
      noted = true;
    }
    u += n;
    __syncthreads();                                      // shared memory changes hands
  }
  if (p.join && !noted && threadIdx.x == 0) p.cuts[blockIdx.x].rows = 0;
}

// Joins the parts of segments that several CTAs took, row by row: item (c, r)
// is row r of the segment that CTA c began and did not finish (the first kernel
// left a note of it).  WR warps take an item: 1, while a segment has five to
// eight parts (fewer: the kernel below), or all 8, and then a CTA looks at 32
// notes at once for the few that exist.  Warp w of them adds parts w, w + WR,
// ..., eight in flight, and the warps' sums are added in order.
constexpr int kWarpsJ = 8;
template <int D, int WR, bool BF16>
__global__ void __launch_bounds__(32 * kWarpsJ) kv4_join_kernel(const __grid_constant__ Kv4AttnLaunch p) {
  constexpr int kVec = D / 32, kFlight = 8;               // floats a lane, parts in flight
  __shared__ float acc[kWarpsJ][D];
  __shared__ float2 sums[kWarpsJ];
  const int lane = threadIdx.x & 31, warp = WR == 1 ? 0 : threadIdx.x >> 5;
  const int group = p.q_heads / p.c.heads;
  griddep_wait();
  griddep_launch_dependents();
  // WR = 1: warps stride over all items.  WR = 8: block (x, r), row r of the notes 32 x .. 32 x + 31.
  const long long items = (long long)(p.ctas - 1) * p.tile_rows, step = (long long)gridDim.x * kWarpsJ;
  const int note = 32 * blockIdx.x + lane;
  unsigned found = 0;
  if (WR != 1) found = __ballot_sync(0xFFFFFFFFu, note < p.ctas && (int)blockIdx.y < p.cuts[min(note, p.ctas - 1)].rows);
  for (long long i = (long long)blockIdx.x * kWarpsJ + (threadIdx.x >> 5); WR == 1 ? i < items : found != 0; i += step) {
    int c0, r;
    if (WR == 1) {
      c0 = (int)(i / p.tile_rows);
      r = (int)(i - (long long)c0 * p.tile_rows);
    } else {
      c0 = 32 * blockIdx.x + __ffs(found) - 1;
      r = blockIdx.y;
      found &= found - 1;
    }
    const Kv4Cut cut = p.cuts[c0];
    if (r >= cut.rows) continue;
    const int c1 = cut.last_cta;
    auto part_row = [&](int c) { return (2ll * c + (c == c0 ? cut.slot : 0)) * p.tile_rows + r; };
    float top = -INFINITY, total = 0.0f, v[kVec];
#pragma unroll
    for (int j = 0; j < kVec; ++j) v[j] = 0.0f;
    for (int c = c0 + warp; c <= c1; c += WR * kFlight) {
      float2 ml[kFlight];
      float a[kFlight][kVec];
#pragma unroll
      for (int q = 0; q < kFlight; ++q) {
        ml[q] = make_float2(-INFINITY, 0.0f);
        if (c + WR * q <= c1) {
          const long long at = part_row(c + WR * q);
          const float* src = p.part_o + at * D + kVec * lane;
          ml[q] = p.part_ml[at];
          if (kVec == 4) {
            const float4 x = *reinterpret_cast<const float4*>(src);
            a[q][0] = x.x, a[q][1] = x.y, a[q][kVec - 2] = x.z, a[q][kVec - 1] = x.w;
          } else {
            const float2 x = *reinterpret_cast<const float2*>(src);
            a[q][0] = x.x, a[q][1] = x.y;
          }
        }
      }
      float to = top;
#pragma unroll
      for (int q = 0; q < kFlight; ++q) to = fmaxf(to, ml[q].x);
      const float f0 = ex2_diff(top, to);
      top = to;
      total *= f0;
#pragma unroll
      for (int j = 0; j < kVec; ++j) v[j] *= f0;
#pragma unroll
      for (int q = 0; q < kFlight; ++q) {
        if (c + WR * q <= c1) {
          const float f = ex2_diff(ml[q].x, top);
          total = fmaf(ml[q].y, f, total);
#pragma unroll
          for (int j = 0; j < kVec; ++j) v[j] = fmaf(a[q][j], f, v[j]);
        }
      }
    }
    const int row = cut.row0 + r, tok = row / group, head = cut.head * group + row - tok * group;
    const long long token = cut.token0 + tok;
    const int wj = threadIdx.x >> 5;
#pragma unroll
    for (int j = 0; j < kVec; ++j) acc[wj][kVec * lane + j] = v[j];
    if (WR == 1) {
      __syncwarp();
      if (lane < D / 8) {
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = acc[wj][8 * lane + j];
        store_row8<BF16>(p, token, head, 8 * lane, y, top, total);
      }
      __syncwarp();
      continue;
    }
    if (lane == 0) sums[wj] = make_float2(top, total);
    __syncthreads();
    if (threadIdx.x < D / 8) {
      float y[8];
      top = -INFINITY;
#pragma unroll
      for (int k = 0; k < kWarpsJ; ++k) top = fmaxf(top, sums[k].x);
      total = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = 0.0f;
#pragma unroll
      for (int k = 0; k < kWarpsJ; ++k) {
        const float f = ex2_diff(sums[k].x, top);
        total = fmaf(sums[k].y, f, total);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = fmaf(acc[k][8 * threadIdx.x + j], f, y[j]);
      }
      store_row8<BF16>(p, token, head, 8 * threadIdx.x, y, top, total);
    }
    __syncthreads();
  }
}

// The same where a segment has a few parts at most: a warp takes two rows of a
// note, two parts of each in flight.  After the prompt chunks that
// kv4_attention_tc.cu measures (147 notes, about 40 MB of parts) this takes 12
// us, the kernel above 28, four rows a warp 17, one 14; after 16 requests of 32
// rows and 4096 keys 2 us less than the one above, of 64 rows 4.
constexpr int kRowsJ = 2;
template <int D, bool BF16>
__global__ void __launch_bounds__(32 * kWarpsJ) kv4_join_rows_kernel(const __grid_constant__ Kv4AttnLaunch p) {
  constexpr int kVec = D / 32, kFlight = 2;
  __shared__ float acc[kWarpsJ][kRowsJ][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group = p.q_heads / p.c.heads;
  griddep_wait();
  griddep_launch_dependents();
  const int per_cut = p.tile_rows / kRowsJ, items = (p.ctas - 1) * per_cut;
  for (int i = blockIdx.x * kWarpsJ + warp; i < items; i += gridDim.x * kWarpsJ) {
    const int c0 = i / per_cut, r0 = (i - c0 * per_cut) * kRowsJ;
    const Kv4Cut cut = p.cuts[c0];
    const int rows = min(cut.rows - r0, kRowsJ);
    if (rows <= 0) continue;
    float top[kRowsJ], total[kRowsJ], v[kRowsJ][kVec];
#pragma unroll
    for (int r = 0; r < kRowsJ; ++r) {
      top[r] = -INFINITY, total[r] = 0.0f;
#pragma unroll
      for (int j = 0; j < kVec; ++j) v[r][j] = 0.0f;
    }
    for (int c = c0; c <= cut.last_cta; c += kFlight) {
      float2 ml[kFlight][kRowsJ];
      float a[kFlight][kRowsJ][kVec];
#pragma unroll
      for (int q = 0; q < kFlight; ++q)
#pragma unroll
        for (int r = 0; r < kRowsJ; ++r) {
          ml[q][r] = make_float2(-INFINITY, 0.0f);
          if (c + q <= cut.last_cta && r < rows) {
            const long long at = (2ll * (c + q) + (c + q == c0 ? cut.slot : 0)) * p.tile_rows + r0 + r;
            const float* src = p.part_o + at * D + kVec * lane;
            ml[q][r] = p.part_ml[at];
            if (kVec == 4) {
              const float4 x = *reinterpret_cast<const float4*>(src);
              a[q][r][0] = x.x, a[q][r][1] = x.y, a[q][r][kVec - 2] = x.z, a[q][r][kVec - 1] = x.w;
            } else {
              const float2 x = *reinterpret_cast<const float2*>(src);
              a[q][r][0] = x.x, a[q][r][1] = x.y;
            }
          }
        }
#pragma unroll
      for (int r = 0; r < kRowsJ; ++r) {
        const float to = fmaxf(top[r], fmaxf(ml[0][r].x, ml[1][r].x)), f0 = ex2_diff(top[r], to);
        top[r] = to;
        total[r] *= f0;
#pragma unroll
        for (int j = 0; j < kVec; ++j) v[r][j] *= f0;
#pragma unroll
        for (int q = 0; q < kFlight; ++q)
          if (c + q <= cut.last_cta && r < rows) {
            const float f = ex2_diff(ml[q][r].x, to);
            total[r] = fmaf(ml[q][r].y, f, total[r]);
#pragma unroll
            for (int j = 0; j < kVec; ++j) v[r][j] = fmaf(a[q][r][j], f, v[r][j]);
          }
      }
    }
#pragma unroll
    for (int r = 0; r < kRowsJ; ++r)
#pragma unroll
      for (int j = 0; j < kVec; ++j) acc[warp][r][kVec * lane + j] = v[r][j];
    __syncwarp();
#pragma unroll
    for (int r = 0; r < kRowsJ; ++r)
      if (r < rows && lane < D / 8) {
        const int row = cut.row0 + r0 + r, tok = row / group, head = cut.head * group + row - tok * group;
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = acc[warp][r][8 * lane + j];
        store_row8<BF16>(p, cut.token0 + tok, head, 8 * lane, y, top[r], total[r]);
      }
    __syncwarp();
  }
}

// Requests of at most kFewRows rows (query heads of one key head x tokens) go to
// this file's kernel, larger ones to kv4_attention_tc.cu.  Both measured, us at
// 32 / 64 / 96 / 128 rows a request, 8 key heads, D = 128: one request of 4096
// keys 14.9 / 19.6 / 28.9 / 27.7 here, 20.6 / 20.6 / 21.1 / 23.9 there; 16 of
// them 51 / 82 / 119 / 149 and 72 / 73 / 75 / 77 (D = 64: 34 / 54 / 76 / 95 and
// 59 / 60 / 60 / 61).  Where the sizes are on the device split_rows (kv4_rows.cuh)
// goes by their sum.

size_t parts_bytes(const Kv4AttnLaunch& p) {
  return p.join ? (size_t)p.ctas * (2 * p.tile_rows * ((size_t)p.c.D * 4 + 8) + sizeof(Kv4Cut)) : 0;
}

template <int D, int NT, bool BF16>
cudaError_t launch_nt(const Kv4AttnLaunch& p, cudaStream_t stream) {
  constexpr int kSmem = smem_bytes<D, NT>();
  cudaError_t e = ensure_smem_limit(kv4_attention_kernel<D, NT, BF16>, kSmem);
  if (e != cudaSuccess) return e;
  return launch_after(kv4_attention_kernel<D, NT, BF16>, dim3((unsigned)p.ctas), kThreadsA, kSmem, stream, p);
}
template <int D, bool BF16>
cudaError_t launch_few(const Kv4AttnLaunch& p, cudaStream_t stream) {
  if (p.tile_rows == 8) return launch_nt<D, 1, BF16>(p, stream);
  if (p.tile_rows == 16) return launch_nt<D, 2, BF16>(p, stream);
  if (p.tile_rows == 24) return launch_nt<D, 3, BF16>(p, stream);
  return launch_nt<D, 4, BF16>(p, stream);
}
template <int D, bool BF16>
cudaError_t launch_join(const Kv4AttnLaunch& p, cudaStream_t stream) {
  if (p.ctas > 8 * p.segments)
    return launch_after(kv4_join_kernel<D, kWarpsJ, BF16>, dim3((unsigned)(p.ctas + 31) / 32, (unsigned)p.tile_rows),
                        32 * kWarpsJ, 0, stream, p);
  if (p.ctas <= 4 * p.segments) {
    const int items = (p.ctas - 1) * (p.tile_rows / kRowsJ);
    return launch_after(kv4_join_rows_kernel<D, BF16>, dim3((unsigned)(items + kWarpsJ - 1) / kWarpsJ), 32 * kWarpsJ, 0,
                        stream, p);
  }
  const long long blocks = ((long long)(p.ctas - 1) * p.tile_rows + kWarpsJ - 1) / kWarpsJ, most = 16ll * p.num_sms;
  return launch_after(kv4_join_kernel<D, 1, BF16>, dim3((unsigned)(blocks < most ? blocks : most)), 32 * kWarpsJ, 0, stream, p);
}
template <int D, bool BF16>
cudaError_t launch_all(const Kv4Plan& plan, uint8_t* workspace, cudaStream_t stream) {
  const Kv4AttnLaunch* launches[2] = {plan.use_few ? &plan.few : nullptr, plan.use_many ? &plan.many : nullptr};
  for (int i = 0; i < 2; ++i) {
    if (!launches[i]) continue;
    Kv4AttnLaunch p = *launches[i];
    if (p.join) {
      p.part_o = reinterpret_cast<float*>(workspace);
      p.part_ml = reinterpret_cast<float2*>(p.part_o + (size_t)p.ctas * 2 * p.tile_rows * D);
      p.cuts = reinterpret_cast<Kv4Cut*>(p.part_ml + (size_t)p.ctas * 2 * p.tile_rows);
      workspace += parts_bytes(p);
    }
    cudaError_t e = i == 0 ? launch_few<D, BF16>(p, stream) : launch_kv4_attention_tc(p, stream);
    if (e == cudaSuccess && p.join) e = launch_join<D, BF16>(p, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// Fills in the launch for requests of min_rows .. max_rows rows, in tiles of tile_rows.
void plan_launch(Kv4AttnLaunch& p, int tile_rows, int min_rows, int max_rows, long long slots, int max_kv) {
  p.tile_rows = tile_rows;
  p.min_rows = min_rows;
  p.max_rows = max_rows;
  // One resident set of CTAs shares the work evenly, whatever the lengths; no
  // more CTAs than units of work.
  p.segments = max_units(p.tokens, p.requests, p.q_heads / p.c.heads, p.c.heads, tile_rows, p.q_start != nullptr, 0);
  const long long units = p.segments * tile_units(max_kv);
  p.ctas = (int)(units < slots ? (units > 0 ? units : 1) : slots);
  // One CTA, or tables that hold one unit at most: no segment is ever cut.
  p.join = p.ctas > 1 && ((long long)p.max_pages << p.c.page_log2) > kUnitKeys;
}

}  // namespace

Kv4Plan kv4_attention_plan(const Kv4AttnLaunch& base, int max_kv, int num_sms) {
  Kv4Plan plan;
  plan.few = plan.many = base;
  plan.few.num_sms = plan.many.num_sms = num_sms;
  const long long rows = (long long)base.tokens * (base.q_heads / base.c.heads);
  const RowSplit split = split_rows(rows, base.requests, base.q_start != nullptr);
  plan.use_few = split.few;
  plan.use_many = split.many;
  // The smallest tile that holds an average request's rows: a larger one
  // dequantizes each key for more rows at once, a smaller one leaves room for
  // more warps (20 rows, 16 x 3001 keys, 8 heads: tiles of 24 rows 35.1 us, of
  // 32 42.8; D = 64: 26.0 and 29.8).
  // Beside prompts (q_start), single tokens.
  long long each = base.requests > 0 ? (rows + base.requests - 1) / base.requests : 0;
  if (base.q_start && plan.use_many) each = base.q_heads / base.c.heads;
  const int nt = each <= 8 ? 1 : each <= 16 ? 2 : each <= 24 ? 3 : 4;
  plan_launch(plan.few, 8 * nt, 0, split.few_max, (long long)num_sms * ctas_per_sm(base.c.D, nt), max_kv);
  plan_launch(plan.many, 256, split.many_min, 0x7FFFFFFF, num_sms, max_kv);
  return plan;
}

size_t kv4_attention_workspace(const Kv4Plan& plan) {
  return (plan.use_few ? parts_bytes(plan.few) : 0) + (plan.use_many ? parts_bytes(plan.many) : 0);
}

cudaError_t launch_kv4_attention(const Kv4Plan& plan, void* workspace, cudaStream_t stream) {
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const Kv4AttnLaunch& p = plan.few;
  if (p.c.D == 128) return p.dtype == 0 ? launch_all<128, true>(plan, ws, stream) : launch_all<128, false>(plan, ws, stream);
  return p.dtype == 0 ? launch_all<64, true>(plan, ws, stream) : launch_all<64, false>(plan, ws, stream);
}

}  // namespace svdq

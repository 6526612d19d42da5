// kv4_attention_tc.cu -- attention of many query rows over the paged 4-bit
// cache (prompts, chunks, cross attention) on the 5th-generation tensor cores.
//
// Same definition, work split and join as kv4_attention.cu, with tiles of 256
// rows: two 128-row halves share every key tile of 128 keys, so each key and
// value is dequantized once for 256 rows.  At that many rows the products
// bound it (4 D flops a row and key: D = 128, 2048 cycles a tile), and next to
// them the exponentials (one a row and key: as many cycles of the special
// function unit).  Measured about 3900 cycles a tile; with the join 0.88 PFLOP/s
// on chunks of up to 1024 tokens behind 8203 keys (216 us) and 0.97 on 4096
// queries of 32 heads over 4333 keys (300 us), 0.54 and 0.59 of the measured bf16
// rate: a half's chain from scores to weights and back through its two products is
// not hidden altogether by the other half's.
//
// Roles (one CTA per SM; 176, 176, 88 and 72 registers a thread):
//   warps 0-3, 4-7   softmax of half 0 and 1: thread = row = tensor memory lane.
//                    A row's 128 scores come from tensor memory into registers
//                    (with 152 registers and half of them read twice: 266 us
//                    against 231 at the time), weights go back there as fp16
//                    over the scores; the output is rescaled there only when
//                    the reference exponent has to rise (by more than 8).
//   warps 8-11       thread = key of the tile: 4-bit rows -> fp16 rows in shared
//                    memory, K and V in the same layout (128-byte swizzled rows
//                    of 64 dims): K is the first product's K-major operand, V
//                    the second's MN-major one.  The next tile's codes are
//                    loaded into registers before the wait for a free stage.
//   warp 12          issues O_h += P_h V and S_h = Q_h K^T for the halves in
//                    turn, so that one half's softmax runs beside the other's
//                    products; each half's outputs begin with the first 64
//                    weights a row.
// Measured and left out (the prompt chunks above, then 231 us): 64-key sub-tiles
// with scores double-buffered (an MMA of N = 64 takes 48 cycles, not 32: 302 us
// against 284 at the time); two threads a row on 16 warps (284 against 275); an
// eighth to a half of the exponentials as polynomials on the FMA pipe (235 to 280
// us); the halves' exponentials taking turns (287 against 266); the next
// segment's queries fetched before a segment's outputs are written (spills: 247
// us against 216).
// Tensor memory: S_h (128 columns, P over the last 64), O_0 O_1 (D each).
// Shared memory: Q 2 x 128 x D, two stages of K and of V (128 x D each), fp16.
//
// Numerics are those of kv4_attention.cu: cache values exact in fp16, queries
// scaled per row by a power of two (and the sign of the softmax scale), fp32
// sums, weights rounded to fp16 for the second product (2^-11, or 2^-32 of the
// row's largest).  A NaN value in a tile
// that some rows see only in part is written as zero and remembered per row.
//
// Every wait is bounded; one that runs out sets an error word
// (svdq_kv4_attention_status), the CTA's roles leave, and tensor memory is freed.
#include <cuda_runtime.h>

#include <type_traits>

#include "hadamard.cuh"
#include "kv4_common.cuh"

namespace svdq {

__device__ unsigned g_kv4_attention_err;

namespace {

constexpr int kHalf = 128, kKeys = 128;
constexpr int kThreadsT = 32 * 16;                        // warps 13-15 only complete the register split's last group
constexpr int kDequantThreads = 128;
static_assert(kUnitKeys == kKeys, "a unit of work is one key tile");

template <int D>
struct TcSmem {
  static constexpr int kTile = kKeys * D * 2;             // 128 rows of D fp16: Q half, K stage, V stage
  static constexpr int kQ = 0, kK = 2 * kTile, kV = kK + 2 * kTile, kBars = kV + 2 * kTile;
  static constexpr int kNan = kBars + 256;                // [2][128] bytes: NaN blocks of a value row
  static constexpr int kMisc = kNan + 2 * kKeys;          // abort, tensor memory base, per stage: absent bits, NaN flag
  static constexpr int kBytes = kMisc + 64 + 1024;        // + alignment of the base
};
// One of each for the two stages (K, V), for the halves (S, O, Q), for half h and part x of its weights at 2 h + x (P: keys
// 64 x .. 64 x + 63 of the tile).  A parity wait tells a phase only from its neighbours, so no barrier may run two phases
// ahead of who waits on it: scores' next phase needs the waiting half's weights, outputs' (one a segment) its next segment.
enum Bar { kKFull = 0, kKFree = 2, kVFull = 4, kVFree = 6, kSFull = 8, kOFull = 10, kQFull = 12, kPFull = 14, kEnd = 18 };

// The MMA warp stays converged and one elected lane's predicate guards each
// instruction: in a branch that one lane takes, every operand is computed in
// that lane's registers and moved to the uniform ones the instruction reads
// (about 125 cycles an MMA, twice its time; measured).
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e;
}
// D[tmem] (+)= A[tmem] * B[smem], fp16 A (two per 32-bit column), fp32 D.
__device__ __forceinline__ void mma_f16_ts(uint32_t one, uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 e, %5, 0;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(one)
      : "memory");
}
// Both operands in shared memory.
__device__ __forceinline__ void mma_f16_ss(uint32_t one, uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 e, %5, 0;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(one)
      : "memory");
}
__device__ __forceinline__ void commit_one(uint32_t one, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "setp.ne.b32 e, %1, 0;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"(one)
      : "memory");
}
// fp16 A and B, fp32 D; B K-major or MN-major.
constexpr uint32_t idesc_f16(uint32_t m, uint32_t n, bool b_mn) {
  return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | ((n >> 3) << 17) | ((m >> 4) << 24);
}
// MN-major operand, 128-byte swizzle: 8-row (K) groups of 128 bytes (64 MN
// elements) 1024 bytes apart, blocks of 64 MN elements `block` bytes apart.
__device__ __forceinline__ uint64_t sdesc_mnmajor_sw128(uint32_t saddr, uint32_t block) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(block >> 4) << 16) | ((uint64_t)(1024u >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}
// Byte offset of 16-byte piece `c` (8 of the D elements) of row r in a 128-row tile: blocks of 64 elements.
__device__ __forceinline__ uint32_t tile_offset(int r, int c) {
  return (uint32_t)((c >> 3) * (kKeys * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// Registers a thread of this warpgroup: the four shares add up to what the
// launch gave (512 threads x 128).
template <bool INC, int N>
__device__ __forceinline__ void set_registers() {
  if (INC)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
  else
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// Largest of three (NaN: the others).
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

struct Ctl {
  uint32_t bars;
  volatile int* abort;
  unsigned* err;
  __device__ __forceinline__ uint32_t bar(int i) const { return bars + 8 * i; }
  __device__ __forceinline__ bool wait(int i, uint32_t parity) const {
    return wait_bounded(bar(i), parity & 1u, abort, err, 1u);
  }
  // The same for a warp: true if every lane's wait ended.
  __device__ __forceinline__ bool wait_warp(int i, uint32_t parity) const {
    return __all_sync(0xFFFFFFFFu, wait(i, parity));
  }
};

// Scores of 32 columns that do not exist: from column `see` on, and in 16-column halves that `gone` names.
__device__ __forceinline__ void mask32(uint32_t (&v)[32], int see, uint32_t gone) {
#pragma unroll
  for (int i = 0; i < 32; ++i)
    if (i >= see || ((gone >> (i / 16)) & 1u)) v[i] = 0xFF800000u;
}

// One key row, packed and (16 values at a time) scaled.
template <int D>
struct PackedRow {
  uint4 c[D / 32];
  uint32_t s[D / 64];                                     // D / 16 scale bytes
  __device__ __forceinline__ void load(const uint8_t* codes, const uint8_t* scales, uint32_t row) {
    if (row == kAbsent) {
#pragma unroll
      for (int i = 0; i < D / 32; ++i) c[i] = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < D / 64; ++i) s[i] = 0;
      return;
    }
    const uint4* cp = reinterpret_cast<const uint4*>(codes + (size_t)row * (D / 2));
#pragma unroll
    for (int i = 0; i < D / 32; ++i) c[i] = cp[i];
    const uint32_t* sp = reinterpret_cast<const uint32_t*>(scales + (size_t)row * (D / 16));
#pragma unroll
    for (int i = 0; i < D / 64; ++i) s[i] = sp[i];
  }
  // Bit b: block b's scale is NaN; those scales become zero.
  __device__ __forceinline__ uint32_t take_nan() {
    uint32_t bits = 0;
#pragma unroll
    for (int b = 0; b < D / 16; ++b)
      if (((s[b / 4] >> (8 * (b & 3))) & 0x7Fu) == 0x7Fu) {
        bits |= 1u << b;
        s[b / 4] &= ~(0xFFu << (8 * (b & 3)));
      }
    return bits;
  }
  __device__ __forceinline__ void store(uint32_t tile, int r) const {
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {                     // 8 elements each
      const uint32_t w = i % 4 == 0 ? c[i / 4].x : i % 4 == 1 ? c[i / 4].y : i % 4 == 2 ? c[i / 4].z : c[i / 4].w;
      const int b = i / 2;
      const __half2 two = e4m3x2_to_half2((s[b / 4] >> (16 * ((b & 3) >> 1))) & 0xFFFFu);
      const __half2 f = (b & 1) ? __high2half2(two) : __low2half2(two);
      uint32_t d[4];
      e2m1x8_to_f16x8(w, d);
      st_shared_v4(tile + tile_offset(r, i), make_uint4(hmul2u(d[0], f), hmul2u(d[1], f), hmul2u(d[2], f), hmul2u(d[3], f)));
    }
  }
};

// What all roles work out alike for a segment.
struct Job {
  RowTile rt;
  int head, k_begin, k_end, tiles, halves;
  bool whole, begun;                                      // the whole segment; its first unit
  int units, slot;
};
__device__ __forceinline__ Job next_job(const Kv4Work& w, const WarpUnits& wu, long long u, long long u0, long long u1) {
  long long first;
  const int b = request_of_unit(w, wu, u, &first);
  const Segment sg = segment_in(w, span_of(w, b), b, u - first);
  Job j;
  j.rt = sg.tile;
  j.head = sg.head;
  j.tiles = (int)min((long long)(sg.units - sg.unit0), u1 - u);
  j.k_begin = sg.unit0 * kUnitKeys;
  j.k_end = min(sg.tile.last_key, (sg.unit0 + j.tiles) * kUnitKeys);
  j.units = sg.units;
  j.whole = j.tiles == sg.units;
  j.begun = sg.unit0 == 0;
  j.slot = u == u0 ? 0 : 1;
  j.halves = sg.tile.rows > kHalf ? 2 : 1;
  return j;
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreadsT, 1) kv4_attention_tc_kernel(const __grid_constant__ Kv4AttnLaunch p) {
  using SM = TcSmem<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* sm = smem_raw + (base - raw);
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  volatile int* misc = reinterpret_cast<volatile int*>(sm + SM::kMisc);        // [0] abort [1] tmem [2..5] absent [6..7] NaN seen
  Ctl ctl;
  ctl.bars = base + SM::kBars;
  ctl.abort = misc;
  ctl.err = &g_kv4_attention_err;

  if (threadIdx.x == 0) {
    misc[0] = 0;
    misc[6] = misc[7] = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(ctl.bar(kKFull + i), kDequantThreads);
      mbar_init(ctl.bar(kKFree + i), 1);
      mbar_init(ctl.bar(kVFull + i), kDequantThreads);
      mbar_init(ctl.bar(kVFree + i), 1);
      mbar_init(ctl.bar(kSFull + i), 1);
      mbar_init(ctl.bar(kOFull + i), 1);
      mbar_init(ctl.bar(kQFull + i), kHalf);
      mbar_init(ctl.bar(kPFull + 2 * i), kHalf);
      mbar_init(ctl.bar(kPFull + 2 * i + 1), kHalf);
    }
    mbar_init(ctl.bar(kEnd), 1);
    fence_mbar_init();
  }
  if (warp == 12) {
    tmem_alloc(base + SM::kMisc + 4, 512);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = (uint32_t)misc[1];

  griddep_wait();
  griddep_launch_dependents();
  const Kv4Work w = work_of(p);
  const WarpUnits wu = warp_units(w);
  const long long per = kv4_div(wu.total + gridDim.x - 1, gridDim.x);
  const long long u0 = per * blockIdx.x, u1 = min(u0 + per, wu.total);
  const int group = p.q_heads / p.c.heads;

  if (warp < 8) {
    // ------------------------------------------------------------ softmax of half h, row = lane of tensor memory
    set_registers<true, 176>();
    const int h = warp >> 2, r = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;     // lane field (bits 31:16) of this warp's quadrant
    const uint32_t s_tm = tmem + lanes + h * kKeys, o_tm = tmem + lanes + 2 * kKeys + h * D;
    uint32_t n_tile = 0, n_job = 0;                       // tiles and segments this half has had
    long long n_all = 0;                                  // tiles the CTA has had
    bool ok = true;
    for (long long u = u0; ok && u < u1;) {
      const Job job = next_job(w, wu, u, u0, u1);
      u += job.tiles;
      if (h >= job.halves) {
        n_all += job.tiles;
        continue;
      }
      const int row = h * kHalf + r;                      // of the tile
      const bool live = row < job.rt.rows;
      const int abs_row = job.rt.row0 + (live ? row : 0), tok = abs_row / group;
      const int head = job.head * group + abs_row - tok * group;
      const int lim = live ? job.rt.keys_of(tok, p.causal) : 0;
      const int free_end = min(job.rt.keys_of(job.rt.row0 / group, p.causal), job.k_end);
      // ---- queries: scaled by a power of two to [2^14, 2^15) at the row's largest finite magnitude.  A warp loads whole
      // rows of its 32 (D / 8 lanes a row: a load of one row a lane touches 32 lines at once), each lane learns its
      // row's address from the row's owner and leaves it the factor.
      constexpr int kPieces = D / 8, kAtOnce = 32 / kPieces;      // 16-byte pieces of a row, rows a load
      const int mine = lane % kPieces, which = lane / kPieces;
      const uint32_t tile = base + SM::kQ + h * SM::kTile;
      float qs = 0.0f;
      {
        const long long at = (long long)(job.rt.token0 + tok) * p.qt + (long long)head * p.qh;
        uint4 packed[kPieces];
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          const int rr = kAtOnce * i + which;
          const long long from = __shfl_sync(0xFFFFFFFFu, at, rr);
          const bool there = h * kHalf + 32 * (warp & 3) + rr < job.rt.rows;
          packed[i] = there ? *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + from + 8 * mine)
                            : make_uint4(0, 0, 0, 0);
        }
        const float sign = p.scale < 0.0f ? -1.0f : 1.0f;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          const int rr = kAtOnce * i + which;
          float f[8], big = 0.0f;
          unpack8<BF16>(packed[i], f);
#pragma unroll
          for (int j = 0; j < 8; ++j) big = fmaxf(big, fabsf(f[j]) < INFINITY ? fabsf(f[j]) : 0.0f);
#pragma unroll
          for (int o = 1; o < kPieces; o <<= 1) big = fmaxf(big, __shfl_xor_sync(0xFFFFFFFFu, big, o));
          const int e = row_exponent(big);
          const float up = sign * __uint_as_float((uint32_t)(127 + e) << 23);
          st_shared_v4(tile + tile_offset(32 * (warp & 3) + rr, mine),
                       make_uint4(half2u(f[0] * up, f[1] * up), half2u(f[2] * up, f[3] * up), half2u(f[4] * up, f[5] * up),
                                  half2u(f[6] * up, f[7] * up)));
          // (Never zero: the mask writes -inf over scores, and -inf x 0 is no number.  At the smallest normal number what
          // is visible stays below 2^-90, as good as zero.)
          const float down = fmaxf(row_factor(sign * p.scale, e), 0x1p-126f);
          const float theirs = __shfl_sync(0xFFFFFFFFu, down, (lane % kAtOnce) * kPieces);
          if (lane / kAtOnce == i) qs = theirs;             // row kAtOnce * i + lane % kAtOnce is this lane's
        }
        fence_proxy_async_smem();
        mbar_arrive(ctl.bar(kQFull + h));
      }
      float ref = -INFINITY, sum = 0.0f;
      uint32_t poison = 0;                                // 16-dim blocks in which the row has seen a NaN value
      for (int j = 0; ok && j < job.tiles; ++j, ++n_tile, ++n_all) {
        const int k0 = job.k_begin + kKeys * j, stage = (int)(n_all & 1);
        const bool partial = k0 + kKeys > free_end;
        if (!(ok = ctl.wait_warp(kSFull + h, n_tile))) break;
        tc_fence_after_sync();
        const uint32_t absent = (uint32_t)misc[2 + (n_all & 3)];
        const bool masked = partial || absent != 0;
        const int see = lim - k0;                         // columns below it are visible
        // ---- the row's scores, and the maximum of the visible ones
        uint32_t v[4][32];
        float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(s_tm + 32 * c, v[c]);
        tmem_ld_wait();
        if (masked) {
#pragma unroll
          for (int c = 0; c < 4; ++c) mask32(v[c], see - 32 * c, absent >> (8 * c));
        }
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int i = 0; i < 32; i += 2)
            tops[c] = max3(tops[c], __uint_as_float(v[c][i]), __uint_as_float(v[c][i + 1]));
        const float top = fmaxf(max3(tops[0], tops[1], tops[2]), tops[3]);
        // Relative to the reference (kRoom below the first tile's largest, then raised past kMost only).
        const float rel = ref == -INFINITY ? top * qs : fmaf(top, qs, -ref);
        const bool over = ref == -INFINITY ? top > -INFINITY : rel > kMost;
        if (__any_sync(0xFFFFFFFFu, over)) {
          const float to = over ? (ref == -INFINITY ? rel : ref + rel) - kRoom : ref;
          const float f = over ? ex2_diff(ref, to) : 1.0f;
          ref = to;
          sum *= f;
          if (j > 0) {                                    // (these scores were issued after the last outputs: those are done)
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              uint32_t y[16];
              tmem_ld16(o_tm + 16 * c, y);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i) y[i] = __float_as_uint(__uint_as_float(y[i]) * f);
              tmem_st16(o_tm + 16 * c, y);
            }
          }
        }
        // ---- weights, two to a column, over the last 64 columns of the scores: those of columns 64-127 first, whose
        // outputs begin while those of columns 0-63 are formed
        const float minus = ref == -INFINITY ? 0.0f : -ref;
        const uint64_t qs2 = pk2(qs, qs), minus2 = pk2(minus, minus);
        uint64_t part[2] = {0, 0};
        auto weights = [&](const uint32_t (&v)[32], uint32_t to) {
          uint32_t pw[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const uint64_t e = fma2(pk2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), qs2, minus2);
            const float a = ex2(lo2(e)), b = ex2(hi2(e));
            part[i & 1] = add2(part[i & 1], pk2(a, b));
            pw[i] = half2u(a, b);
          }
          tmem_st16(to, pw);
        };
        weights(v[2], s_tm + 96);
        weights(v[3], s_tm + 112);
        tmem_st_wait();
        tc_fence_before_sync();
        mbar_arrive(ctl.bar(kPFull + 2 * h + 1));
        weights(v[0], s_tm + 64);
        weights(v[1], s_tm + 80);
        const uint64_t both = add2(part[0], part[1]);
        sum += lo2(both) + hi2(both);
        if (partial) {                                    // rows see it in part: NaN values were taken out
          if (!(ok = ctl.wait_warp(kVFull + stage, (uint32_t)(n_all >> 1)))) break;
          const volatile uint8_t* bits = sm + SM::kNan + stage * kKeys;
          if (misc[6 + stage])
            for (int k = 0; k < min(see, kKeys); ++k) poison |= bits[k];
        }
        tmem_st_wait();
        tc_fence_before_sync();
        mbar_arrive(ctl.bar(kPFull + 2 * h));
      }
      if (!ok) break;
      // ---- output: through the rows' own places in the query tile (the half's scores are all done), so that a warp
      // writes whole rows of its 32
      if (!(ok = ctl.wait_warp(kOFull + h, n_job))) break;
      ++n_job;
      tc_fence_after_sync();
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      const long long part_row = (2ll * blockIdx.x + job.slot) * p.tile_rows;
      const long long to = job.whole ? (long long)(job.rt.token0 + tok) * p.ot + (long long)head * p.oh : (part_row + row) * D;
      // A pass: D 16-bit or D / 2 fp32 values a row.
      for (int pass = 0; pass < (job.whole ? 1 : 2); ++pass) {
#pragma unroll 1
        for (int c = 0; c < (job.whole ? D / 32 : D / 64); ++c) {
          uint32_t y[32];
          const int c32 = pass * (D / 64) + c;            // 32 columns, two blocks of the cache's format
          tmem_ld32(o_tm + 32 * c32, y);
          tmem_ld_wait();
#pragma unroll
          for (int b = 0; b < 2; ++b)
            if ((poison >> (2 * c32 + b)) & 1u) {
#pragma unroll
              for (int i = 0; i < 16; ++i) y[16 * b + i] = 0x7FC00000u;
            }
          if (job.whole) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t o[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float a = __uint_as_float(y[8 * i + 2 * k]) * inv, b = __uint_as_float(y[8 * i + 2 * k + 1]) * inv;
                o[k] = BF16 ? pack_bf16x2(a, b) : half2u(a, b);
              }
              st_shared_v4(tile + tile_offset(r, 4 * c + i), make_uint4(o[0], o[1], o[2], o[3]));
            }
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              st_shared_v4(tile + tile_offset(r, 8 * c + i),
                           make_uint4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]));
          }
        }
        __syncwarp();
#pragma unroll 4
        for (int i = 0; i < kPieces; ++i) {
          const int rr = kAtOnce * i + which;
          const long long dst = __shfl_sync(0xFFFFFFFFu, to, rr);
          if (h * kHalf + 32 * (warp & 3) + rr < job.rt.rows) {
            const uint4 y = ld_shared_v4(tile + tile_offset(32 * (warp & 3) + rr, mine));
            if (job.whole)
              *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + dst + 8 * mine) = y;
            else
              *reinterpret_cast<uint4*>(p.part_o + dst + pass * (D / 2) + 4 * mine) = y;
          }
        }
        __syncwarp();
      }
      if (live) {
        if (!job.whole)
          p.part_ml[part_row + row] = make_float2(ref, sum);
        else if (p.lse)
          p.lse[(long long)(job.rt.token0 + tok) * p.q_heads + head] =
              sum == 0.0f ? -INFINITY : log_sum(ref, sum);
      }
      tc_fence_before_sync();
    }
  } else if (warp < 12) {
    // ------------------------------------------------------------ dequantize: thread = key of the tile
    set_registers<false, 88>();
    const int key = threadIdx.x - 256;
    long long n_all = 0;
    bool ok = true;
    bool noted = false;
    for (long long u = u0; ok && u < u1;) {
      const Job job = next_job(w, wu, u, u0, u1);
      if (!job.whole && job.begun) {
        if (key == 0) p.cuts[blockIdx.x] = cut_of(job.rt, job.head, (int)kv4_div(u + job.units - 1, per), job.slot);
        noted = true;
      }
      u += job.tiles;
      const int* table = p.table + job.rt.request * p.table_stride;
      const int free_end = min(job.rt.keys_of(job.rt.row0 / group, p.causal), job.k_end);
      auto row_of = [&](int j) {
        const int k = job.k_begin + kKeys * j + key;
        if (j >= job.tiles || k >= job.k_end) return kAbsent;
        const int page = table[k >> p.c.page_log2];
        if (page < 0 || page >= p.c.pages) return kAbsent;
        return ((((uint32_t)page * p.c.heads) + job.head) << p.c.page_log2) + (k & ((1 << p.c.page_log2) - 1));
      };
      PackedRow<D> kr, vr;
      uint32_t row = row_of(0), next = row_of(1);
      kr.load(p.c.kc, p.c.ks, row);
      vr.load(p.c.vc, p.c.vs, row);
      for (int j = 0; j < job.tiles; ++j, ++n_all) {
        const int stage = (int)(n_all & 1), k0 = job.k_begin + kKeys * j;
        const uint32_t round = (uint32_t)(n_all >> 1);
        const bool masked = k0 + kKeys > free_end;
        // (A stage's first use waits for nothing: the phase before the first counts as complete.)
        if (!(ok = ctl.wait_warp(kKFree + stage, round + 1))) break;
        kr.store(base + SM::kK + stage * SM::kTile, key);
        // Halves of 16 keys that are in no page: their scores do not exist.
        const bool gone = row == kAbsent && k0 + key < job.k_end;
        const unsigned votes = __ballot_sync(0xFFFFFFFFu, gone);
        volatile uint8_t* absent = reinterpret_cast<volatile uint8_t*>(const_cast<int*>(misc) + 2 + (n_all & 3));
        if (lane == 0) absent[warp - 8] = (uint8_t)((votes & 0xFFFFu ? 1u : 0u) | (votes >> 16 ? 2u : 0u));
        fence_proxy_async_smem();
        mbar_arrive(ctl.bar(kKFull + stage));
        kr.load(p.c.kc, p.c.ks, next);
        if (!(ok = ctl.wait_warp(kVFree + stage, round + 1))) break;
        if (masked) {
          const uint32_t bits = vr.take_nan();
          sm[SM::kNan + stage * kKeys + key] = (uint8_t)bits;
          if (bits) misc[6 + stage] = 1;
        }
        vr.store(base + SM::kV + stage * SM::kTile, key);
        fence_proxy_async_smem();
        mbar_arrive(ctl.bar(kVFull + stage));
        vr.load(p.c.vc, p.c.vs, next);
        row = next;
        next = row_of(j + 2);
      }
    }
    if (p.join && !noted && key == 0) p.cuts[blockIdx.x].rows = 0;
  } else {
    set_registers<false, 72>();
    if (warp == 12) {
      // ------------------------------------------------------------ MMA
      constexpr uint32_t kIdS = idesc_f16(kHalf, kKeys, false), kIdO = idesc_f16(kHalf, D, true);
      bool ok = true;
      uint32_t n_all = 0, n_tile[2] = {0, 0}, n_job[2] = {0, 0};      // tiles of the CTA, tiles and segments of each half
      // Operand descriptors of half 0, stage 0: an offset only adds to the low word (address / 16).  The loop below is one
      // thread's instruction stream beside MMAs of 64 cycles, so everything that can be is a constant there.
      const uint64_t q_desc = sdesc_kmajor_sw128(base + SM::kQ), k_desc = sdesc_kmajor_sw128(base + SM::kK),
                     v_desc = sdesc_mnmajor_sw128(base + SM::kV, kKeys * 128);
      const uint32_t one = elect_one(), tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
      auto segment = [&](auto halves, int tiles) {
        constexpr int H = decltype(halves)::value;
        auto scores = [&](int h, uint64_t k) {
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            const uint32_t off = ((i / 4) * (kKeys * 128) + (i % 4) * 32) >> 4;
            mma_f16_ss(one, tm + h * kKeys, q_desc + (h * (SM::kTile >> 4) + off), k + off, kIdS, i > 0);
          }
          commit_one(one, ctl.bar(kSFull + h));
        };
        auto outputs = [&](int h, int x, uint64_t v, uint32_t accumulate) {
#pragma unroll
          for (int i = 4 * x; i < 4 * x + 4; ++i)
            mma_f16_ts(one, tm + 2 * kKeys + h * D, tm + h * kKeys + 64 + 8 * i, v + (i * 2048 >> 4), kIdO,
                       i > 4 * x ? 1u : accumulate);
        };
        ok = ctl.wait_warp(kKFull + (n_all & 1), n_all >> 1);
#pragma unroll
        for (int h = 0; h < H; ++h) {
          ok = ok && ctl.wait_warp(kQFull + h, n_job[h]++);
          if (!ok) return;
          tc_fence_after_sync();
          scores(h, k_desc + (n_all & 1) * (SM::kTile >> 4));
        }
        commit_one(one, ctl.bar(kKFree + (n_all & 1)));
        // Tile by tile, for each half in turn: outputs of its two parts as they come, then the next tile's scores in the
        // columns that these weights leave.  The scores' commit stands for the outputs too (MMAs end in order); the last
        // tile's outputs have their own.
        for (int left = tiles; left > 0; --left) {
          const uint32_t so = n_all & 1, ss = so ^ 1u;
          const uint64_t v = v_desc + so * (SM::kTile >> 4), k = k_desc + ss * (SM::kTile >> 4);
          ok = ctl.wait_warp(kVFull + so, n_all >> 1);
          ++n_all;
#pragma unroll
          for (int h = 0; h < H; ++h) {
            ok = ok && ctl.wait_warp(kPFull + 2 * h + 1, n_tile[h]);
            if (!ok) return;
            tc_fence_after_sync();
            outputs(h, 1, v, left < tiles ? 1u : 0u);
            ok = ctl.wait_warp(kPFull + 2 * h, n_tile[h]++);
            if (ok && left > 1 && h == 0) ok = ctl.wait_warp(kKFull + ss, n_all >> 1);
            if (!ok) return;
            tc_fence_after_sync();
            outputs(h, 0, v, 1u);
            if (h == H - 1) commit_one(one, ctl.bar(kVFree + so));
            if (left > 1)
              scores(h, k);
            else
              commit_one(one, ctl.bar(kOFull + h));
          }
          if (left > 1) commit_one(one, ctl.bar(kKFree + ss));
        }
      };
      for (long long u = u0; ok && u < u1;) {
        const Job job = next_job(w, wu, u, u0, u1);
        u += job.tiles;
        const int tiles = __shfl_sync(0xFFFFFFFFu, job.tiles, 0);
        if (__shfl_sync(0xFFFFFFFFu, job.halves, 0) == 2)
          segment(std::integral_constant<int, 2>(), tiles);
        else
          segment(std::integral_constant<int, 1>(), tiles);
      }
      // Whatever ended the roles: the MMAs that were issued end before the memory they use is given up.
      commit_one(one, ctl.bar(kEnd));
      if (one) wait_for(ctl.bar(kEnd), 0, kWaitTimeoutNs);
      __syncwarp();
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 12) tmem_dealloc(tmem, 512);
}

template <int D, bool BF16>
cudaError_t launch_tc(const Kv4AttnLaunch& p, cudaStream_t stream) {
  cudaError_t e = ensure_smem_limit(kv4_attention_tc_kernel<D, BF16>, TcSmem<D>::kBytes);
  if (e != cudaSuccess) return e;
  return launch_after(kv4_attention_tc_kernel<D, BF16>, dim3((unsigned)p.ctas), kThreadsT, TcSmem<D>::kBytes, stream, p);
}

}  // namespace

cudaError_t launch_kv4_attention_tc(const Kv4AttnLaunch& p, cudaStream_t stream) {
  if (p.c.D == 128) return p.dtype == 0 ? launch_tc<128, true>(p, stream) : launch_tc<128, false>(p, stream);
  return p.dtype == 0 ? launch_tc<64, true>(p, stream) : launch_tc<64, false>(p, stream);
}

cudaError_t kv4_attention_status(unsigned* flags) {
  cudaError_t e = cudaDeviceSynchronize();
  if (e != cudaSuccess) return e;
  e = cudaMemcpyFromSymbol(flags, g_kv4_attention_err, sizeof(unsigned));
  const unsigned zero = 0;
  if (e == cudaSuccess && *flags != 0) e = cudaMemcpyToSymbol(g_kv4_attention_err, &zero, sizeof(unsigned));
  return e;
}

}  // namespace svdq

// qk_norm_rope.cu -- per-head RMS norm, rotary positions with several axes and
// the Hadamard rotation of each head, in one pass over queries and keys.
//
// One row is one head of one token, D values (D % 8 == 0, D <= 256):
//   n_d = x_d * rsqrt(mean_d(x_d^2) + eps) * w_d                (if a weight is given)
//   pair p < P: (a, b) = (n_2p, n_2p+1) or (n_p, n_p+P),
//               phi = pos[token, axis_p] * f_p,
//               (a, b) <- (a cos phi - b sin phi, a sin phi + b cos phi)
//   y = n H_D / sqrt(D)                                          (if asked; H_D: Sylvester Hadamard)
// The Hadamard step is "HadamardTransform per head_dim block" of "Rotate in
// quantization and its vLLM implementation" (section 3.2): applied to queries
// and keys alike it leaves their products unchanged and spreads a key's large
// channels over its 4-bit blocks.  fp32 throughout, one rounding to the
// storage type at the end.
//
// The angle is formed in 64 bits: at position 10^5 an fp32 product pos * f is
// off by up to 2^-8 radian.  phi / 2pi is reduced to half a turn in fp64 and
// only then rounded; sincospif needs no further reduction.
//
// Layout: a row is held by LP lanes (a power of two), each with two 8-element
// chunks, chunk numbers lane and lane + LP, so a warp's 16-byte accesses are
// contiguous.  For D = 16 LP the element bits are: three inside a chunk, log2
// LP across lanes, the top bit between the two chunks; so a half-split pair
// over the whole head (P = D/2) lies in one lane, an adjacent pair always
// does, and the Hadamard needs log2 LP shuffle stages (3 for D = 128; with one
// chunk a lane it would be 4).  Arithmetic runs on pairs (f32x2).
//
// One resident set of CTAs shares the tokens.  A CTA computes the cosines and
// sines of its tokens once into shared memory, for all of their heads; a slot's
// next row is on its way while the current one is worked on.
//
// Bound: 4 bytes an element (HBM).  4096 tokens x 64 heads x 128, norms and
// adjacent pairs: 25.4 us, 5.3 TB/s (the loads and stores alone 23.9).  The
// Hadamard is bound by instruction issue (about 400 per four rows of 128, 70% of
// the slots) and the shared-memory pipe (51 wavefronts of shuffles, 32 of
// cosines, sines and weights, 16 of loads and stores, 66%) instead: 9973 tokens x
// 32 heads 43.9 us, 3.7 TB/s (with bank conflicts on the tables 48.7).  29991 tokens x 40 heads x 64, 48 values
// of a head rotated: 58.0 us, 5.3 TB/s.  Three or five CTAs an SM instead of
// four: 29.2 / 46.4 / 64.8 and 30.8 / 50.2 / 66.1 us.  One kernel for every
// pairing, with and without the Hadamard, instead of six: 27.9 / 48.7 / 64.1.
#include <cuda_runtime.h>

#include "attn_kernels.h"
#include "hadamard.cuh"
#include "kcommon.cuh"
#include "ptx.cuh"

namespace svdq {
namespace {

constexpr int kThreadsR = 256;
constexpr int kCtasR = 4;                       // resident CTAs an SM (64 registers)
constexpr int kMaxTable = 4096;                 // cos/sin pairs per CTA (32 KB)

// One 16-byte chunk <-> four packed fp32 pairs.
template <bool BF16>
__device__ __forceinline__ void unpack4(uint4 w, uint64_t (&v)[4]) {
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (BF16) {
      v[i] = pk2(bf16lo_to_f32(x[i]), bf16hi_to_f32(x[i]));
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&x[i]));
      v[i] = pk2(f.x, f.y);
    }
  }
}
template <bool BF16>
__device__ __forceinline__ uint4 pack4(const uint64_t (&v)[4]) {
  uint32_t x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (BF16) {
      x[i] = pack_bf16x2(lo2(v[i]), hi2(v[i]));
    } else {
      const __half2 h = __floats2half2_rn(lo2(v[i]), hi2(v[i]));
      x[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  return make_uint4(x[0], x[1], x[2], x[3]);
}
// Four consecutive floats of shared memory as two pairs.
__device__ __forceinline__ void load2(const float* p, uint64_t& a, uint64_t& b) {
  const float4 f = *reinterpret_cast<const float4*>(p);
  a = pk2(f.x, f.y);
  b = pk2(f.z, f.w);
}

// (a, b) <- (a cos - b sin, a sin + b cos)
__device__ __forceinline__ void turn(uint64_t& v, float cs, float sn) {
  const float a = lo2(v), b = hi2(v);
  v = pk2(fmaf(a, cs, -(b * sn)), fmaf(a, sn, b * cs));
}

struct RowsArgs {
  QkNormRopeLaunch p;
  int tb, hb;                                   // tokens and heads per CTA
};

// Where a pair's halves are: neighbours, this lane's two chunks (half-split pairs over the whole of a head of 16 LP
// values), or two chunks anywhere.
enum Pairs { kAdjacent, kOwnChunks, kAnyChunks };

// BF16: storage type.  LOGLP: log2 of the lanes per row.  HAD: with the Hadamard step.
template <bool BF16, int LOGLP, Pairs PAIRS, bool HAD>
__global__ void __launch_bounds__(kThreadsR, kCtasR) qk_norm_rope_kernel(const __grid_constant__ RowsArgs a) {
  constexpr int LP = 1 << LOGLP, kSlots = kThreadsR / LP;
  // Of each token's pairs: cos and sin, adjacent for adjacent pairs, in two halves of the table otherwise.  A lane reads
  // what belongs to one chunk as two 16-byte pieces; all chunks' first pieces come first, then all second ones, so that
  // neighbours read neighbouring words.
  __shared__ __align__(16) float table[2 * kMaxTable];
  __shared__ __align__(16) float gain[2][16 * LP];        // norm weights of queries and keys, in such pieces too
  const QkNormRopeLaunch& p = a.p;
  const int D = p.D, P = p.pairs, PT = (P + 3) & ~3, chunks = D / 8;
  const int t0 = blockIdx.x * a.tb, nt = min(a.tb, p.tokens - t0);
  const int slot = threadIdx.x / LP, l = threadIdx.x % LP;
  constexpr bool inter = PAIRS == kAdjacent;
  const float inv_d = 1.0f / (float)D;

  griddep_wait();
  griddep_launch_dependents();
  for (int i = threadIdx.x; i < 2 * D; i += kThreadsR) {
    const uint16_t* g = static_cast<const uint16_t*>(i < D ? p.q.weight : p.k.weight);
    if (g) {
      const uint16_t bits = g[i < D ? i : i - D];
      const int d = i < D ? i : i - D;
      gain[i >= D][(d >> 2 & 1) * (8 * LP) + 4 * (d >> 3) + (d & 3)] =
          BF16 ? __uint_as_float((uint32_t)bits << 16) : __half2float(__ushort_as_half(bits));
    }
  }
  bool filled = false;
  for (int side = 0; side < 2; ++side) {                  // the same for the whole CTA
    const HeadSide& s = side ? p.k : p.q;
    const int off = side ? p.q.heads : 0;
    const int first = max((int)blockIdx.y * a.hb - off, 0), nh = min((int)(blockIdx.y + 1) * a.hb - off, s.heads) - first;
    if (nh <= 0) continue;
    // Row r = (token, head) of this side; a slot's next row is kSlots further.
    const int rows = nt * nh, more_t = kSlots / nh, more_h = kSlots % nh;
    int t = slot / nh, h = slot - t * nh, tn = t, hn = h;
    auto advance = [&](int& tt, int& hh) {
      tt += more_t;
      hh += more_h;
      if (hh >= nh) {
        hh -= nh;
        ++tt;
      }
    };
    const uint16_t* x0 = static_cast<const uint16_t*>(s.x) + (long long)t0 * s.xt + (long long)first * s.xh + 8 * l;
    uint16_t* y0 = static_cast<uint16_t*>(s.y) + (long long)t0 * s.yt + (long long)first * s.yh + 8 * l;
    auto load = [&](int tt, int hh, uint4 (&w)[2]) {
      const uint16_t* x = x0 + (long long)tt * s.xt + (long long)hh * s.xh;
      if (tt < nt && l < chunks) w[0] = *reinterpret_cast<const uint4*>(x);
      if (tt < nt && l + LP < chunks) w[1] = *reinterpret_cast<const uint4*>(x + 8 * LP);
    };
    uint4 w[2], wn[2];
    w[0] = w[1] = wn[0] = wn[1] = make_uint4(0, 0, 0, 0);
    load(t, h, w);
    advance(tn, hn);
    if (!filled) {
      filled = true;
      for (int i = threadIdx.x; i < nt * P; i += kThreadsR) {
        const int tt = i / P, j = i - tt * P;
        const int ax = p.pair_axis ? min((int)p.pair_axis[j], p.axes - 1) : 0;
        const int pos = p.positions[(t0 + tt) * p.pos_stride + ax];
        double angle = (double)pos * (double)p.inv_freq[j] * 0.15915494309189535;      // 1 / 2pi
        angle -= rint(angle);
        float sn, cn;
        sincospif(2.0f * (float)angle, &sn, &cn);
        if (inter) {
          float* e = table + 2 * (tt * PT) + (j >> 1 & 1) * PT + 4 * (j >> 2) + 2 * (j & 1);
          e[0] = cn;
          e[1] = sn;
        } else {
          float* e = table + tt * P + (j >> 2 & 1) * (P / 2) + 4 * (j >> 3) + (j & 3);
          e[0] = cn;
          e[kMaxTable] = sn;
        }
      }
      __syncthreads();
    }

  // The loop bound is uniform over the CTA: every lane takes part in the
  // shuffles, lanes of rows beyond the last with what they hold.
  for (int r0 = 0; r0 < rows; r0 += kSlots) {
    load(tn, hn, wn);
    const bool live = t < nt;
    const int tl = live ? t : 0;
    uint64_t v[2][4];
    unpack4<BF16>(w[0], v[0]);
    unpack4<BF16>(w[1], v[1]);

    if (s.weight) {
      uint64_t s2 = 0;
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) s2 = fma2(v[c][i], v[c][i], s2);
      float ss = lo2(s2) + hi2(s2);
#pragma unroll
      for (int o = 1; o < LP; o <<= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
      const float rs = rsqrtf(fmaf(ss, inv_d, p.eps));
      const uint64_t rs2 = pk2(rs, rs);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float* g = gain[side] + 4 * (l + LP * c);   // (16 LP of them: in range for lanes without a chunk too)
        uint64_t g2[4];
        load2(g, g2[0], g2[1]);
        load2(g + 8 * LP, g2[2], g2[3]);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[c][i] = mul2(mul2(v[c][i], rs2), g2[i]);
      }
    }

    if (P > 0) {
      if (inter) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int p0 = 4 * (l + LP * c);
          const float* e = table + 2 * (tl * PT) + p0;
          if (p0 < P) {                                   // cos and sin of two pairs at once
            const float4 e0 = *reinterpret_cast<const float4*>(e), e1 = *reinterpret_cast<const float4*>(e + PT);
            turn(v[c][0], e0.x, e0.y);
            if (p0 + 4 <= P) {
              turn(v[c][1], e0.z, e0.w);
              turn(v[c][2], e1.x, e1.y);
              turn(v[c][3], e1.z, e1.w);
            } else {
              if (p0 + 1 < P) turn(v[c][1], e0.z, e0.w);
              if (p0 + 2 < P) turn(v[c][2], e1.x, e1.y);
            }
          }
        }
      } else if (PAIRS == kOwnChunks) {
        const float* e = table + tl * P + 4 * l;
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          uint64_t cn[2], sn[2];
          load2(e + (i / 2) * (P / 2), cn[0], cn[1]);
          load2(e + kMaxTable + (i / 2) * (P / 2), sn[0], sn[1]);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const uint64_t x0 = v[0][i + q], x1 = v[1][i + q];
            v[0][i + q] = sub2(mul2(x0, cn[q]), mul2(x1, sn[q]));
            v[1][i + q] = fma2(x0, sn[q], mul2(x1, cn[q]));
          }
        }
      } else {                                       // P % 8 == 0: the other half is a whole chunk elsewhere
        const int pc = P / 8;
        uint64_t o[2][4];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int ci = l + LP * c;
          const int other = ci < pc ? ci + pc : (ci < 2 * pc ? ci - pc : ci);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint64_t u0 = __shfl_sync(0xFFFFFFFFu, v[0][i], other & (LP - 1), LP);
            const uint64_t u1 = __shfl_sync(0xFFFFFFFFu, v[1][i], other & (LP - 1), LP);
            o[c][i] = other >= LP ? u1 : u0;
          }
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int ci = l + LP * c;
          if (ci < 2 * pc) {
            const bool first = ci < pc;
            const float* e = table + tl * P + 4 * (first ? ci : ci - pc);
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
              uint64_t cn[2], sn[2];
              load2(e + (i / 2) * (P / 2), cn[0], cn[1]);
              load2(e + kMaxTable + (i / 2) * (P / 2), sn[0], sn[1]);
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                const uint64_t x = v[c][i + q], y = o[c][i + q];
                v[c][i + q] = first ? sub2(mul2(x, cn[q]), mul2(y, sn[q])) : fma2(y, sn[q], mul2(x, cn[q]));
              }
            }
          }
        }
      }
    }

    if (HAD) {                                       // D is a power of two; D = 8 has one chunk (LP = 1)
      const bool two = D >= 16;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        // Neighbours: two pairs give two sums and two differences.
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          const uint64_t x = pk2(lo2(v[c][i]), lo2(v[c][i + 1])), y = pk2(hi2(v[c][i]), hi2(v[c][i + 1]));
          const uint64_t sm = add2(x, y), df = sub2(x, y);
          v[c][i] = pk2(lo2(sm), lo2(df));
          v[c][i + 1] = pk2(hi2(sm), hi2(df));
        }
#pragma unroll
        for (int hp = 1; hp < 4; hp <<= 1)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if ((i & hp) == 0) {
              const uint64_t x = v[c][i], y = v[c][i + hp];
              v[c][i] = add2(x, y);
              v[c][i + hp] = sub2(x, y);
            }
      }
#pragma unroll
      for (int o = 1; o < LP; o <<= 1) {
        const float sg = (l & o) ? -1.0f : 1.0f;
        const uint64_t sg2 = pk2(sg, sg);
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int i = 0; i < 4; ++i) v[c][i] = fma2(sg2, v[c][i], __shfl_xor_sync(0xFFFFFFFFu, v[c][i], o));
      }
      const float scale = rsqrtf((float)D);
      const uint64_t scale2 = pk2(scale, scale);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t x = v[0][i], y = two ? v[1][i] : 0;
        v[0][i] = mul2(add2(x, y), scale2);
        v[1][i] = mul2(sub2(x, y), scale2);
      }
    }

    if (live) {
      uint16_t* y = y0 + (long long)t * s.yt + (long long)h * s.yh;
      if (l < chunks) *reinterpret_cast<uint4*>(y) = pack4<BF16>(v[0]);
      if (l + LP < chunks) *reinterpret_cast<uint4*>(y + 8 * LP) = pack4<BF16>(v[1]);
    }
    w[0] = wn[0];
    w[1] = wn[1];
    t = tn;
    h = hn;
    advance(tn, hn);
  }
  }
}

template <bool BF16, int LOGLP, Pairs PAIRS, bool HAD>
cudaError_t launch(const QkNormRopeLaunch& p, cudaStream_t stream) {
  constexpr int kSlots = kThreadsR >> LOGLP;
  const int heads = p.q.heads + p.k.heads;
  RowsArgs a;
  a.p = p;
  // Few tokens: one row per slot and the heads split over CTAs (latency).
  // Otherwise every resident CTA takes all heads of an equal share of the
  // tokens, in as many rounds as the table of angles asks for.
  const long long resident = (long long)kCtasR * p.num_sms;
  if ((long long)p.tokens * heads <= resident * kSlots) {
    a.tb = heads >= kSlots ? 1 : kSlots / heads;
    a.hb = kSlots < heads ? kSlots : heads;
  } else {
    const int most = p.pairs > 0 ? kMaxTable / ((p.pairs + 3) & ~3) : kMaxTable;
    const long long share = (p.tokens + resident - 1) / resident, rounds = (share + most - 1) / most;
    a.tb = (int)((p.tokens + resident * rounds - 1) / (resident * rounds));
    a.hb = heads;
  }
  if (p.pairs > 0) {                            // at most 128 of them
    const int most = kMaxTable / ((p.pairs + 3) & ~3);
    if (a.tb > most) a.tb = most;
  }
  const dim3 grid((unsigned)((p.tokens + a.tb - 1) / a.tb), (unsigned)((heads + a.hb - 1) / a.hb));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreadsR);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<BF16, LOGLP, PAIRS, HAD>, a);
}

template <bool BF16, int LOGLP>
cudaError_t launch_kind(const QkNormRopeLaunch& p, cudaStream_t stream) {
  const Pairs pairs = p.interleaved ? kAdjacent : p.pairs == (8 << LOGLP) ? kOwnChunks : kAnyChunks;
  if (p.hadamard)
    return pairs == kAdjacent    ? launch<BF16, LOGLP, kAdjacent, true>(p, stream)
           : pairs == kOwnChunks ? launch<BF16, LOGLP, kOwnChunks, true>(p, stream)
                                 : launch<BF16, LOGLP, kAnyChunks, true>(p, stream);
  return pairs == kAdjacent    ? launch<BF16, LOGLP, kAdjacent, false>(p, stream)
         : pairs == kOwnChunks ? launch<BF16, LOGLP, kOwnChunks, false>(p, stream)
                               : launch<BF16, LOGLP, kAnyChunks, false>(p, stream);
}

template <bool BF16>
cudaError_t launch_lp(const QkNormRopeLaunch& p, cudaStream_t stream) {
  if (p.D <= 16) return launch_kind<BF16, 0>(p, stream);
  if (p.D <= 32) return launch_kind<BF16, 1>(p, stream);
  if (p.D <= 64) return launch_kind<BF16, 2>(p, stream);
  if (p.D <= 128) return launch_kind<BF16, 3>(p, stream);
  return launch_kind<BF16, 4>(p, stream);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const QkNormRopeLaunch& p, cudaStream_t stream) {
  return p.dtype == 0 ? launch_lp<true>(p, stream) : launch_lp<false>(p, stream);
}

}  // namespace svdq

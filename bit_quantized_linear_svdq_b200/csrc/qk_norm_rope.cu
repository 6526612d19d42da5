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
// does, and the Hadamard needs log2 LP shuffle stages (3 for D = 128; one
// chunk a lane needed 4, and shuffles are the tightest unit of that stage).
// Cosines and sines are computed once per token and CTA into shared memory
// and used by all of the token's heads; the first rows' loads are in flight
// meanwhile.  HBM-bound: 4 bytes an element.
#include <cuda_runtime.h>

#include "attn_kernels.h"
#include "hadamard.cuh"
#include "ptx.cuh"

namespace svdq {
namespace {

constexpr int kThreadsR = 256;
constexpr int kMaxTable = 2048;                 // cos/sin pairs per CTA (16 KB)

template <bool BF16>
__device__ __forceinline__ void unpack8(uint4 w, float (&v)[8]) {
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
template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  uint32_t x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (BF16) {
      x[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
    } else {
      const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
      x[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  return make_uint4(x[0], x[1], x[2], x[3]);
}

struct RowsArgs {
  QkNormRopeLaunch p;
  int tb, hb;                                   // tokens and heads per CTA
};

// BF16: storage type.  LOGLP: log2 of the lanes per row.
template <bool BF16, int LOGLP>
__global__ void __launch_bounds__(kThreadsR) qk_norm_rope_kernel(const __grid_constant__ RowsArgs a) {
  constexpr int LP = 1 << LOGLP, kSlots = kThreadsR / LP;
  __shared__ float2 cs[kMaxTable];
  const QkNormRopeLaunch& p = a.p;
  const int D = p.D, P = p.pairs, heads = p.q.heads + p.k.heads;
  const int t0 = blockIdx.x * a.tb, nt = min(a.tb, p.tokens - t0);
  const int h0 = blockIdx.y * a.hb, nh = min(a.hb, heads - h0);
  const int slot = threadIdx.x / LP, l = threadIdx.x % LP;
  const int chunks = D / 8, rows = nt * nh;

  // Row r of this CTA: its token, whether it is a key, its first element.
  auto load = [&](int r, uint4 (&w)[2]) {
    w[0] = w[1] = make_uint4(0, 0, 0, 0);
    if (r >= rows) return;
    const int t = t0 + r / nh;
    int h = h0 + r % nh;
    const bool key = h >= p.q.heads;
    const HeadSide& s = key ? p.k : p.q;
    if (key) h -= p.q.heads;
    const uint16_t* x = static_cast<const uint16_t*>(s.x) + t * s.xt + h * s.xh;
#pragma unroll
    for (int c = 0; c < 2; ++c)
      if (l + LP * c < chunks) w[c] = *reinterpret_cast<const uint4*>(x + 8 * (l + LP * c));
  };

  uint4 w[2], wn[2];
  load(slot, w);
  for (int i = threadIdx.x; i < nt * P; i += kThreadsR) {
    const int t = i / P, j = i - t * P;
    const int ax = p.pair_axis ? min((int)p.pair_axis[j], p.axes - 1) : 0;
    const int pos = p.positions[(t0 + t) * p.pos_stride + ax];
    double turn = (double)pos * (double)p.inv_freq[j] * 0.15915494309189535;      // 1 / 2pi
    turn -= rint(turn);
    float sn, cn;
    sincospif(2.0f * (float)turn, &sn, &cn);
    cs[i] = make_float2(cn, sn);
  }
  __syncthreads();

  // The loop bound is uniform over the CTA: every lane takes part in the
  // shuffles, lanes of rows beyond the last with zeros.
  for (int r0 = 0; r0 < rows; r0 += kSlots) {
    const int r = r0 + slot;
    load(r + kSlots, wn);
    const bool live = r < rows;
    const int rr = live ? r : rows - 1;
    const int tl = rr / nh;
    int h = h0 + rr % nh;
    const bool key = h >= p.q.heads;
    const HeadSide& s = key ? p.k : p.q;
    if (key) h -= p.q.heads;
    float v[2][8];
    unpack8<BF16>(w[0], v[0]);
    unpack8<BF16>(w[1], v[1]);

    if (p.q.weight || p.k.weight) {                 // uniform: shuffles inside
      float ss = 0.0f;
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(v[c][i], v[c][i], ss);
#pragma unroll
      for (int o = 1; o < LP; o <<= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
      if (s.weight) {
        const float rs = rsqrtf(ss / (float)D + p.eps);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (l + LP * c < chunks) {
            float g[8];
            unpack8<BF16>(*(reinterpret_cast<const uint4*>(s.weight) + l + LP * c), g);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[c][i] = v[c][i] * rs * g[i];
          }
        }
      }
    }

    if (P > 0) {
      const float2* tab = cs + tl * P;
      if (p.interleaved) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int p0 = 4 * (l + LP * c);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (p0 + i < P) {
              const float2 e = tab[p0 + i];
              const float x0 = v[c][2 * i], x1 = v[c][2 * i + 1];
              v[c][2 * i] = fmaf(x0, e.x, -(x1 * e.y));
              v[c][2 * i + 1] = fmaf(x0, e.y, x1 * e.x);
            }
          }
        }
      } else if (P == 8 * LP) {                      // the pair's halves are this lane's two chunks
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 e = tab[8 * l + i];
          const float x0 = v[0][i], x1 = v[1][i];
          v[0][i] = fmaf(x0, e.x, -(x1 * e.y));
          v[1][i] = fmaf(x0, e.y, x1 * e.x);
        }
      } else {                                       // P % 8 == 0: the other half is a whole chunk elsewhere
        const int pc = P / 8;
        float o[2][8];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int ci = l + LP * c;
          const int other = ci < pc ? ci + pc : (ci < 2 * pc ? ci - pc : ci);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float u0 = __shfl_sync(0xFFFFFFFFu, v[0][i], other & (LP - 1), LP);
            const float u1 = __shfl_sync(0xFFFFFFFFu, v[1][i], other & (LP - 1), LP);
            o[c][i] = other >= LP ? u1 : u0;
          }
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int ci = l + LP * c;
          if (ci < 2 * pc) {
            const bool first = ci < pc;
            const float2* e8 = tab + 8 * (first ? ci : ci - pc);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float2 e = e8[i];
              v[c][i] = first ? fmaf(v[c][i], e.x, -(o[c][i] * e.y)) : fmaf(o[c][i], e.y, v[c][i] * e.x);
            }
          }
        }
      }
    }

    if (p.hadamard) {                                // D is a power of two; D = 8 has one chunk (LP = 1)
      const bool two = D >= 16;
#pragma unroll
      for (int hp = 1; hp < 8; hp <<= 1) {
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if ((i & hp) == 0) {
              const float x0 = v[c][i], x1 = v[c][i + hp];
              v[c][i] = x0 + x1;
              v[c][i + hp] = x0 - x1;
            }
      }
#pragma unroll
      for (int o = 1; o < LP; o <<= 1) {
        const float sg = (l & o) ? -1.0f : 1.0f;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) v[c][i] = fmaf(sg, v[c][i], __shfl_xor_sync(0xFFFFFFFFu, v[c][i], o));
      }
      const float scale = rsqrtf((float)D);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float x0 = v[0][i], x1 = two ? v[1][i] : 0.0f;
        v[0][i] = (x0 + x1) * scale;
        v[1][i] = (x0 - x1) * scale;
      }
    }

    if (live) {
      uint16_t* y = static_cast<uint16_t*>(s.y) + (long long)(t0 + tl) * s.yt + h * s.yh;
#pragma unroll
      for (int c = 0; c < 2; ++c)
        if (l + LP * c < chunks) *reinterpret_cast<uint4*>(y + 8 * (l + LP * c)) = pack8<BF16>(v[c]);
    }
    w[0] = wn[0];
    w[1] = wn[1];
  }
}

template <bool BF16, int LOGLP>
cudaError_t launch(const QkNormRopeLaunch& p, cudaStream_t stream) {
  constexpr int kSlots = kThreadsR >> LOGLP;
  const int heads = p.q.heads + p.k.heads;
  RowsArgs a;
  a.p = p;
  // Few tokens: one row per slot and the heads split over CTAs (latency).
  // Otherwise a CTA takes all heads of enough tokens for four rows per slot,
  // so that the loads of the next rows hide behind the current ones.
  if ((long long)p.tokens * heads <= 4ll * 148 * kSlots) {
    a.tb = heads >= kSlots ? 1 : kSlots / heads;
    a.hb = kSlots < heads ? kSlots : heads;
  } else {
    a.tb = (4 * kSlots + heads - 1) / heads;
    a.hb = heads;
  }
  if (p.pairs > 0 && a.tb * p.pairs > kMaxTable) a.tb = kMaxTable / p.pairs;    // pairs <= 128
  const dim3 grid((unsigned)((p.tokens + a.tb - 1) / a.tb), (unsigned)((heads + a.hb - 1) / a.hb));
  qk_norm_rope_kernel<BF16, LOGLP><<<grid, kThreadsR, 0, stream>>>(a);
  return cudaGetLastError();
}

template <bool BF16>
cudaError_t launch_lp(const QkNormRopeLaunch& p, cudaStream_t stream) {
  if (p.D <= 16) return launch<BF16, 0>(p, stream);
  if (p.D <= 32) return launch<BF16, 1>(p, stream);
  if (p.D <= 64) return launch<BF16, 2>(p, stream);
  if (p.D <= 128) return launch<BF16, 3>(p, stream);
  return launch<BF16, 4>(p, stream);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const QkNormRopeLaunch& p, cudaStream_t stream) {
  return p.dtype == 0 ? launch_lp<true>(p, stream) : launch_lp<false>(p, stream);
}

}  // namespace svdq

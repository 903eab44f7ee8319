// What the scan's forward, step and backward kernels share.
//
//   delta = softplus(dt + dt_bias),  s[n] <- exp(delta A[n]) s[n] + delta x B[n]
//
// The exponent is kept in base two: A2 = A log2 e once per thread, one multiplication and
// one ex2 per state and token.  Four states lie in a lane and LPC lanes (2, 4, 8 or 16) hold
// a channel, so N is padded to 8, 16, 32 or 64; padded states have A = B = C = 0 and stay zero.
#pragma once

#include "block_common.cuh"

namespace mlstm {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// 2^x, relative error about 2^-22, 0 far below zero.
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// log(1 + exp(v)) without overflow.
__device__ __forceinline__ float softplusf(float v) { return fmaxf(v, 0.f) + log1pf(__expf(-fabsf(v))); }

// Sums V values over L lanes that are STRIDE apart (rank: the lane's index among them) and
// spreads the results: with V >= L lane r ends with the sums of values r V / L .. in v[0 ..];
// with V < L the lanes of rank r / (L / V) share value r / (L / V) in v[0].
template <int V, int L, int STRIDE, int M>
__device__ __forceinline__ void scatter_sum(float (&v)[M], int rank) {
  if constexpr (L > 1) {
    constexpr int bit = L / 2;
    if constexpr (V > 1) {
      const bool up = rank & bit;
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        const float keep = up ? v[i + V / 2] : v[i], send = up ? v[i] : v[i + V / 2];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, send, bit * STRIDE);
      }
      scatter_sum<V / 2, L / 2, STRIDE>(v, rank);
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], bit * STRIDE);
      scatter_sum<1, L / 2, STRIDE>(v, rank);
    }
  }
}

// B and C of tokens t0 .. t0 + TT - 1 as fp32 rows [TT][2 NP]; zero past the end and in the padding.
template <typename T, int NP, int TT>
__device__ __forceinline__ void stage_bc(const ScanArgs& a, int b, int g, int t0, float* out, int tid,
                                         int threads) {
  const T* bp = (const T*)a.b.p + b * a.b.sb + g * a.b.sh;
  const T* cp = (const T*)a.c.p + b * a.c.sb + g * a.c.sh;
  if (a.wide_bc && a.N == NP) {  // whole vectors of eight
    for (int e = tid; e < TT * NP / 4; e += threads) {
      const int t = e / (NP / 4), r = e % (NP / 4), n = (r % (NP / 8)) * 8;
      const bool is_c = r >= NP / 8;
      float v[8];
      if (t0 + t < a.T)
        load8<true>(is_c ? cp + (t0 + t) * a.c.st + n : bp + (t0 + t) * a.b.st + n, v, 8);
      else
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.f;
      store8<true>(out + t * 2 * NP + (is_c ? NP : 0) + n, v, 8);
    }
  } else {
    for (int e = tid; e < TT * 2 * NP; e += threads) {
      const int t = e / (2 * NP), r = e % (2 * NP), n = r % NP;
      float v = 0.f;
      if (t0 + t < a.T && n < a.N)
        v = r >= NP ? to_f32(cp[(t0 + t) * a.c.st + n]) : to_f32(bp[(t0 + t) * a.b.st + n]);
      out[e] = v;
    }
  }
}

// Channels of a CTA: tiles do not cross groups.
struct ChannelTile {
  int g, c0, n;  // group, first channel, channels
};
__device__ __forceinline__ ChannelTile channel_tile(const ScanArgs& a, int i, int tiles, int width) {
  const int per = a.D / a.G;
  ChannelTile q;
  q.g = i / tiles;
  const int first = (i % tiles) * width;
  q.c0 = q.g * per + first;
  q.n = min(width, per - first);
  return q;
}

}  // namespace mlstm

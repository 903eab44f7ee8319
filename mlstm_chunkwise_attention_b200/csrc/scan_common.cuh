// What the scan's forward, step and backward kernels share.
//
//   delta = softplus(dt + dt_bias),  s[n] <- exp(delta A[n]) s[n] + delta x B[n]
//
// The exponent is kept in base two: A2 = A log2 e once per thread, one multiplication and
// one ex2 per state and token.  Four states lie in a lane and LPC lanes (2, 4, 8 or 16) hold
// a channel, so N is padded to 8, 16, 32 or 64; padded states have B = C = 0 and stay zero.
#pragma once

#include "block_common.cuh"

namespace mlstm {

// log(1 + exp(v)) = max(v, 0) + log(1 + e), e = exp(-|v|) in (0, 1], of two values.  log(1 + e) / e is
// a polynomial of degree 8, the best one in relative error on [0, 1] (found with Remez' exchange
// algorithm in 50 digits): 1.4e-7 of the value with fp32 arithmetic, for small e as well.  Half
// the instructions of log1pf, on the pipe that the exponentials leave free.
__device__ __forceinline__ float2 softplus_pair(float2 v) {
  const float2 e =
      make_float2(exp2_fast(-fabsf(v.x) * kLog2e), exp2_fast(-fabsf(v.y) * kLog2e));
  constexpr float c[9] = {9.999999699e-01f, -4.999949314e-01f, 3.331909679e-01f,
                          -2.484298211e-01f, 1.910600644e-01f, -1.366324530e-01f,
                          7.822594782e-02f, -2.950523728e-02f, 5.232694110e-03f};
  float2 p = make_float2(c[8], c[8]);
#pragma unroll
  for (int i = 7; i >= 0; --i) p = fma2(e, p, make_float2(c[i], c[i]));
  return fma2(e, p, make_float2(fmaxf(v.x, 0.f), fmaxf(v.y, 0.f)));
}
__device__ __forceinline__ float softplusf(float v) { return softplus_pair(make_float2(v, v)).x; }

// A (or A log2 e) kept finite, NaN for NaN.  A = -inf is a decay of 0, which -FLT_MAX is as well, but the
// tokens behind the end, and empty steps between segments, have a delta of 0, and 0 times infinity would
// be NaN where such a step must leave the state as it is.
__device__ __forceinline__ float finite_rate(float v) {
  asm("max.NaN.f32 %0, %0, 0fFF7FFFFF;" : "+f"(v));
  asm("min.NaN.f32 %0, %0, 0f7F7FFFFF;" : "+f"(v));
  return v;
}

// A2 of padded states and absent channels: negative, so that an infinite delta is a decay of 0 there too
// (with a rate of 0 it made the gradients that earlier tokens get NaN).
constexpr float kPadRate = -1.f;

// A unit is eight channels of one token in shared memory, written by one thread with 16-byte
// stores and read by a warp along the channels.  The padding (16 bytes to a unit) spreads eight
// threads' 16-byte accesses over all 32 banks.
//
// What bounds the inner loops is what shared memory hands to registers, 128 bytes a cycle and SM,
// and a value that several lanes read counts once for each: a thread that holds four states of one
// channel takes 10 bytes for each state and token, two channels 6.  So a thread holds two channels,
// and nothing is stored twice to save a move.
constexpr int kPairUnit = 20;   // floats of a unit of pairs (delta, w)
constexpr int kFloatUnit = 12;  // floats of a unit of floats

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

__device__ __forceinline__ void load_unit(const float* u, float2* v) {
  const float4 a = reinterpret_cast<const float4*>(u)[0], b = reinterpret_cast<const float4*>(u)[1];
  v[0] = make_float2(a.x, a.y); v[1] = make_float2(a.z, a.w);
  v[2] = make_float2(b.x, b.y); v[3] = make_float2(b.z, b.w);
}
__device__ __forceinline__ void store_unit(float* u, const float2* v) {
  reinterpret_cast<float4*>(u)[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
  reinterpret_cast<float4*>(u)[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
}

// delta of eight channels from dt as it lies in memory; zero where there is no token or channel,
// so that such a token leaves every state as it is.
template <typename T>
__device__ __forceinline__ void delta_of(const ScanArgs& a, const Raw<T, 8>& dt, const float* bias, bool in,
                                         int n, float2* delta) {
  expand(dt, delta);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    delta[i] = add2(delta[i], *reinterpret_cast<const float2*>(bias + 2 * i));
    if (a.softplus) delta[i] = softplus_pair(delta[i]);
    if (!in || 2 * i >= n) delta[i].x = 0.f;
    if (!in || 2 * i + 1 >= n) delta[i].y = 0.f;
  }
}
// A unit of pairs (delta, w).
template <typename T>
__device__ __forceinline__ void stage_pairs(const ScanArgs& a, const float2* w, const Raw<T, 8>& dt,
                                            const float* bias, bool in, int n, float* unit) {
  float2 d[4];
  delta_of<T>(a, dt, bias, in, n, d);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    reinterpret_cast<float4*>(unit)[i] = make_float4(d[i].x, w[i].x, d[i].y, w[i].y);
}
// A unit of pairs (delta, delta x).  Absent elements of x were loaded as zero.  LOOK: false if one of them is
// infinite or NaN.
template <typename T, bool LOOK = false>
__device__ __forceinline__ bool stage_delta(const ScanArgs& a, const Raw<T, 8>& x, const Raw<T, 8>& dt,
                                            const float* bias, bool in, int n, float* unit) {
  float2 d[4], v[4];
  expand(x, v);
  delta_of<T>(a, dt, bias, in, n, d);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 w = mul2(d[i], v[i]);
    reinterpret_cast<float4*>(unit)[i] = make_float4(d[i].x, w.x, d[i].y, w.y);
    v[i] = w;
  }
  if (!LOOK) return true;
  // 0 times each product, NaN if one is not finite; and it is not where its delta is not
  float2 s = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) s = fma2(v[i], make_float2(0.f, 0.f), s);
  return s.x + s.y == 0.f;
}

// The states of a lane that do not exist are zero.
__device__ __forceinline__ void clear_padding(float2* h, int nl, int N) {
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    if (nl * 4 + 2 * p >= N) h[p].x = 0.f;
    if (nl * 4 + 2 * p + 1 >= N) h[p].y = 0.f;
  }
}

// Element i becomes element i ^ perm.
__device__ __forceinline__ float4 permuted(float4 v, int perm) {
  if (perm & 2) v = make_float4(v.z, v.w, v.x, v.y);
  if (perm & 1) v = make_float4(v.y, v.x, v.w, v.z);
  return v;
}

// v held to -126 .. 127, the exponents of fp32's normal numbers; NaN for NaN.
__device__ __forceinline__ float held_exponent(float v) {
  asm("max.NaN.f32 %0, %0, 0fC2FC0000;" : "+f"(v));
  asm("min.NaN.f32 %0, %0, 0f42FE0000;" : "+f"(v));
  return v;
}
__device__ __forceinline__ float2 held_exponents(float2 v) {
  return make_float2(held_exponent(v.x), held_exponent(v.y));
}

// The state (or, REVERSE, the state's gradient) that enters segment `seg`, from what enters the
// first (last) one in h and the segments between; A2 and h hold state i ^ perm at i.
template <int NP, bool REVERSE>
__device__ __forceinline__ void enter_segment(const ScanArgs& a, int b, int c, int nl, int seg,
                                              const float2* A2, float2* h, int perm = 0) {
  constexpr int BATCH = 6;  // segments whose loads are in flight together
  const int count = REVERSE ? a.segs - 1 - seg : seg;
  const float2 half = make_float2(0.5f, 0.5f),
               r0 = mul2(make_float2(finite_rate(A2[0].x), finite_rate(A2[0].y)), half),
               r1 = mul2(make_float2(finite_rate(A2[1].x), finite_rate(A2[1].y)), half);
  for (int i0 = 0; i0 < count; i0 += BATCH) {
    float4 s[BATCH];
    float sum[BATCH];
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      s[k] = make_float4(0.f, 0.f, 0.f, 0.f);  // behind the last one: a step of 0, which leaves h
      sum[k] = 0.f;
      if (i0 + k < count) {
        const int i = REVERSE ? a.segs - 1 - i0 - k : i0 + k;
        const long long row = ((long long)i * a.B + b) * a.D + c;
        s[k] = *reinterpret_cast<const float4*>(a.seg_state + row * NP + nl * 4);
        sum[k] = a.seg_sum[row];
      }
    }
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const float4 v = permuted(s[k], perm);
      const float2 by = make_float2(sum[k], sum[k]);
      // The decay in two halves: a whole segment's may leave fp32's range (2^-126 .. 2^128) although the state
      // is inside it before and after; half of it does not.  Held at 2^-252 and 2^254 in all, so that a state
      // of zero stays zero, however far it would have grown, and an infinite one infinite.
      const float2 e0 = exp2_pair(held_exponents(mul2(by, r0))),
                   e1 = exp2_pair(held_exponents(mul2(by, r1)));
      h[0] = fma2(mul2(e0, h[0]), e0, make_float2(v.x, v.y));
      h[1] = fma2(mul2(e1, h[1]), e1, make_float2(v.z, v.w));
    }
  }
}

// B and C of tokens t0 .. t0 + TT - 1 as fp32 rows [TT][2 NP]; zero from token `last` on and in the
// padding.  COPIES > 1: copy p, STRIDE floats behind copy p - 1, holds element n ^ p at n.
template <typename T, int NP, int TT, int COPIES = 1, int STRIDE = 0>
__device__ __forceinline__ void stage_bc(const ScanArgs& a, int b, int g, int t0, int last, float* out,
                                         int tid, int threads) {
  const T* bp = (const T*)a.b.p + b * a.b.sb + g * a.b.sh;
  const T* cp = (const T*)a.c.p + b * a.c.sb + g * a.c.sh;
  if (a.wide_bc && a.N == NP) {  // whole vectors of eight
    for (int e = tid; e < TT * NP / 4; e += threads) {
      const int t = e / (NP / 4), r = e % (NP / 4), n = (r % (NP / 8)) * 8;
      const bool is_c = r >= NP / 8;
      float v[8];
      if (t0 + t < last)
        load8<true>(is_c ? cp + (t0 + t) * a.c.st + n : bp + (t0 + t) * a.b.st + n, v, 8);
      else
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.f;
#pragma unroll
      for (int p = 0; p < COPIES; ++p) {
        float w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = v[i ^ p];
        store8<true>(out + p * STRIDE + t * 2 * NP + (is_c ? NP : 0) + n, w, 8);
      }
    }
  } else {
    // eight loads before their stores, which the compiler must take to be where the loads read
    constexpr int BATCH = 8;
    for (int e0 = tid; e0 < TT * 2 * NP; e0 += BATCH * threads) {
      float v[BATCH];
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        const int e = e0 + i * threads, t = e / (2 * NP), r = e % (2 * NP), n = r % NP;
        v[i] = 0.f;
        if (e < TT * 2 * NP && t0 + t < last && n < a.N)
          v[i] = r >= NP ? to_f32(cp[(t0 + t) * a.c.st + n]) : to_f32(bp[(t0 + t) * a.b.st + n]);
      }
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        const int e = e0 + i * threads;
        if (e < TT * 2 * NP)
#pragma unroll
          for (int p = 0; p < COPIES; ++p) out[p * STRIDE + (e ^ p)] = v[i];
      }
    }
  }
}

// B and C of a tile in whole vectors of eight, loaded ahead of their tile: what stage_bc does for
// a.wide_bc and N == NP, in two steps.  PAIRS 2: B and C, rows of 2 NP; 1: `b` alone, rows of NP.
template <typename T, int NP, int TT, int PAIRS, int THREADS>
struct RowLoads {
  static constexpr int PER = PAIRS * NP / 8, COUNT = (TT * PER + THREADS - 1) / THREADS;
  Raw<T, 8> r[COUNT];
  __device__ __forceinline__ void load(const T* b, long long bst, const T* c, long long cst, int t0, int last,
                                       int tid) {
#pragma unroll
    for (int m = 0; m < COUNT; ++m) {
      const int e = tid + m * THREADS, t = t0 + e / PER, v = e % PER, n = (v % (NP / 8)) * 8;
      zero_raw(r[m]);
      if (e < TT * PER && t < last) load_raw<true>(v >= NP / 8 ? c + t * cst + n : b + t * bst + n, r[m], 8);
    }
  }
  __device__ __forceinline__ void store(float* out, int tid) const {
#pragma unroll
    for (int m = 0; m < COUNT; ++m) {
      const int e = tid + m * THREADS, t = e / PER, v = e % PER;
      if (e < TT * PER) {
        float2 f[4];
        expand(r[m], f);
        store_unit(out + t * PAIRS * NP + v * 8, f);
      }
    }
  }
};

// ---- segments in turn ----
// Work items are (segment, channel tile), all tiles of a segment before the next segment's, and a CTA
// takes the next one from a counter when it is free.  An item waits for its tile's item of the
// segment before, which was taken earlier by a CTA that runs: so some CTA can always go on,
// however many of them are resident, and the wait is bounded as the tensor-core kernels' are.

// The next item, for all threads of the CTA (a barrier inside, which also ends the last item's use of
// shared memory); `only`: the CTA's one item where segments are not taken in turn.
__device__ __forceinline__ int next_item(const ScanArgs& a, int only, bool first, int total, int* box) {
  __syncthreads();
  if (threadIdx.x == 0) *box = a.in_turn ? (int)atomicAdd(a.turn + kTurnNext, 1u) : first ? only : total;
  __syncthreads();
  return *box;
}

// Waits until `tile` has finished `count` segments; false if the wait was given up.  `box` is not
// next_item's: its slow readers may not be through.
__device__ __forceinline__ bool wait_turn(const ScanArgs& a, int tile, unsigned int count,
                                          unsigned int* failures, int* box) {
  if (threadIdx.x == 0)
    *box = wait_at_least(a.turn + kTurnTiles + tile, count, LaunchAbort{a.turn + kTurnAbort, failures}, 200);
  __syncthreads();
  return *box != 0;
}

// Hands the tile on: every thread's stores before this are visible to the CTA that waits for it.
__device__ __forceinline__ void pass_turn(const ScanArgs& a, int tile) {
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0)
    asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(a.turn + kTurnTiles + tile) : "memory");
}

__device__ __forceinline__ void prefetch_l2(const void* gmem) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(gmem));
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

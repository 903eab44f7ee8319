// Selective state space scan, forward and one-token step.
//
// The scan is serial in time, so parallelism comes from batches, channels and states: a
// thread holds four states of two channels in registers and walks the sequence.  Tiles of 32
// tokens go through shared memory: delta and delta x are computed once per (token,
// channel) from 16-byte loads, B and C are shared by all channels, and y is summed over
// the channels' lanes by a transposing reduction (each lane ends with one token of one
// channel), then gated and stored with 16-byte stores.
//
// One ex2 per state, channel and token is the floor (16 a cycle and SM at 1.965 GHz: 461 us at B8 T4096
// D4096 N16, 19 % more with softplus and the gate).  Measured there on one B200, bf16: 903 us, 953 us with
// the states kept for the backward; fp32 1075 with them.  No pipe is full: the exponentials' 0.57, what
// shared memory hands over 0.68, the issue 0.54.  32768 channels are 14 warps an SM, all that 128
// registers a thread leave room for, and they do not cover each other's latencies.  Measured and not kept:
// one channel to a lane (28 warps, but 10 bytes from shared memory for each state and token: 963 us); tiles
// staged by warps of their own (1078 us, 80 registers).
//
// With few rows the sequence is cut into segments that are scanned at once.  A first pass finds
// each segment's state from zero and its sum of delta; segment j then starts from
// sum_i exp(A sum of delta over i + 1 .. j - 1) state_i, which each CTA adds up for itself.
#include "scan_common.cuh"

namespace mlstm {

namespace {

constexpr int kTile = 32;

constexpr int kThreads = 64;
// CTAs of an SM, by registers.  Shared memory holds as many from 9 states on, but 6 of up to 8 states
// (34.5 KB each), for which scan_cut so counts more slots than there are.
constexpr int kCtas = 8;
constexpr int kSlots = 148 * kCtas;
__device__ unsigned int g_scan_fwd_failures = 0;  // launches that gave up a wait

template <int LPC>
struct Shape {
  static constexpr int NP = 4 * LPC, CT = 2 * kThreads / LPC, VECS = CT / 8;
  static constexpr int ITEMS = (kTile * VECS + kThreads - 1) / kThreads;  // units of a thread
};

// A thread's two channels, cl + swap first.  Neighbouring lanes take them in opposite orders, so that
// in the sum over a channel's lanes each sends its second and keeps its first.
template <int LPC>
struct Lanes {
  int nl, cl, ch[2];
  __device__ __forceinline__ Lanes(int tid) {
    const int lane = tid & 31;
    nl = lane % LPC;
    cl = ((tid / 32) * (32 / LPC) + lane / LPC) * 2;
    ch[0] = cl + (nl & 1);
    ch[1] = cl + 1 - (nl & 1);
  }
};

// What a thread loads of one tile: its units of x and dt.
template <typename T, int ITEMS>
struct TileLoads {
  Raw<T, 8> x[ITEMS], dt[ITEMS];
};

// The walk through a tile in which a delta or delta x is not finite, where N < NP: infinity times a B of
// nought would make the padded states NaN, and with them y where the sum over the N states is
// infinite.  So they are cleared after every token; otherwise the operations of scan_fwd_kernel's loop in
// their order.  A function of its own: such tiles are rare, and a second loop in the kernel took 12 % of
// its speed (1075 us instead of 956 at B8 T4096 D4096 N16) by the registers it left to the first.  The
// kernels for N == NP have neither this nor the check of each tile, which costs 4 % (B8 T2048 D4096 N12
// bf16: 695 us instead of 667).
struct Lane {
  float2 A2[2][2], h[2][2];
};
template <int LPC>
__device__ __noinline__ Lane walk_masked(Lane s, int nl, int N, const float* d0, const float* d1, const float* bc,
                                         float* ydst, float* keep0, float* keep1, long long keep_step, int tokens) {
  using S = Shape<LPC>;
  constexpr int AT_ONCE = LPC / 2;
  float* keep[2] = {keep0, keep1};
  const float* dsrc[2] = {d0, d1};
#pragma unroll 1
  for (int tg = 0; tg < kTile; tg += AT_ONCE) {
    float acc[AT_ONCE];
#pragma unroll
    for (int u = 0; u < AT_ONCE; ++u) {
      const int t = tg + u;
      float yv[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (t % kScanEvery == 0 && t < tokens && keep[e] != nullptr)
          *reinterpret_cast<float4*>(keep[e] + t / kScanEvery * keep_step) =
              make_float4(s.h[e][0].x, s.h[e][0].y, s.h[e][1].x, s.h[e][1].y);
        const float2 d = *reinterpret_cast<const float2*>(dsrc[e] + t * S::VECS * kPairUnit);
        const float2 dd = make_float2(d.x, d.x), w = make_float2(d.y, d.y);
        const float4 Bv = *reinterpret_cast<const float4*>(bc + t * 2 * S::NP);
        const float4 Cv = *reinterpret_cast<const float4*>(bc + t * 2 * S::NP + S::NP);
        s.h[e][0] = fma2(exp2_pair(mul2(dd, s.A2[e][0])), s.h[e][0], mul2(w, make_float2(Bv.x, Bv.y)));
        s.h[e][1] = fma2(exp2_pair(mul2(dd, s.A2[e][1])), s.h[e][1], mul2(w, make_float2(Bv.z, Bv.w)));
        clear_padding(s.h[e], nl, N);
        const float2 v = fma2(s.h[e][1], make_float2(Cv.z, Cv.w), mul2(s.h[e][0], make_float2(Cv.x, Cv.y)));
        yv[e] = v.x + v.y;
      }
      acc[u] = yv[0] + __shfl_xor_sync(0xffffffffu, yv[1], 1);
    }
    scatter_sum<AT_ONCE, AT_ONCE, 2>(acc, nl >> 1);
    ydst[tg * S::VECS * kFloatUnit] = acc[0];
  }
  return s;
}

template <typename T, int LPC, bool GATE, bool WIDE, bool PAD>
__global__ void __launch_bounds__(kThreads, kCtas)
    scan_fwd_kernel(ScanArgs a, int tiles) {
  using S = Shape<LPC>;
  constexpr int NP = S::NP, CT = S::CT, VECS = S::VECS, ITEMS = S::ITEMS;
  __shared__ __align__(16) float sd[kTile * VECS * kPairUnit];  // delta, delta x
  __shared__ __align__(16) float sy[kTile * VECS * kFloatUnit];
  __shared__ __align__(16) float sbc[kTile][2 * NP];
  __shared__ __align__(16) float sbias[CT], sskip[CT];
  const int tid = threadIdx.x;
  const Lanes<LPC> l(tid);
  const int nl = l.nl;
  __shared__ int box[2];
  const int per_seg = a.B * a.G * tiles, NC = (a.T + kScanEvery - 1) / kScanEvery;
  for (bool once = true;; once = false) {
  const int work = next_item(a, blockIdx.x, once, per_seg * a.segs, box);
  if (work >= per_seg * a.segs) return;
  const int seg = work / per_seg, bi = work % per_seg;
  const int b = bi / (tiles * a.G);
  const ChannelTile q = channel_tile(a, bi % (tiles * a.G), tiles, CT);
  const int first = seg * a.seg_len, last = min(first + a.seg_len, a.T);
  const bool handed = a.in_turn && seg > 0;  // the segment before hands its state on
  if (handed && !wait_turn(a, bi, seg, &g_scan_fwd_failures, box + 1)) return;
  float2 A2[2][2], h[2][2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    float av[4], hv[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int n = nl * 4 + k;
      const bool on = l.ch[e] < q.n && n < a.N;
      const long long row = q.c0 + l.ch[e];
      av[k] = on ? finite_rate(a.A[row * a.N + n] * kLog2e) : kPadRate;
      hv[k] = on && a.state_in != nullptr ? a.state_in[((long long)b * a.D + row) * a.N + n] : 0.f;
    }
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      A2[e][p] = make_float2(av[2 * p], av[2 * p + 1]);
      h[e][p] = make_float2(hv[2 * p], hv[2 * p + 1]);
    }
    if (l.ch[e] < q.n && handed) {
      const float4 v = __ldcg(reinterpret_cast<const float4*>(
          a.seg_state + ((long long)b * a.D + q.c0 + l.ch[e]) * NP + nl * 4));
      h[e][0] = make_float2(v.x, v.y);
      h[e][1] = make_float2(v.z, v.w);
    } else if (l.ch[e] < q.n && !a.in_turn) {
      enter_segment<NP, false>(a, b, q.c0 + l.ch[e], nl, seg, A2[e], h[e]);
      if (PAD) clear_padding(h[e], nl, a.N);  // which an infinite input in an earlier segment made NaN
    }
  }
  for (int i = tid; i < CT; i += kThreads) {
    sbias[i] = a.dt_bias != nullptr && i < q.n ? a.dt_bias[q.c0 + i] : 0.f;
    sskip[i] = a.skip != nullptr && i < q.n ? a.skip[q.c0 + i] : 0.f;
  }
  const T* xp = (const T*)a.x.p + b * a.x.sb + q.c0;
  const T* dp = (const T*)a.dt.p + b * a.dt.sb + q.c0;
  const T* zp = GATE ? (const T*)a.z.p + b * a.z.sb + q.c0 : nullptr;
  T* yp = (T*)a.y.p + b * a.y.sb + q.c0;
  TileLoads<T, ITEMS> next;
  auto fetch = [&](int t0) {
#pragma unroll
    for (int m = 0; m < ITEMS; ++m) {
      const int item = tid + m * kThreads, t = t0 + item / VECS, cv = (item % VECS) * 8, n = q.n - cv;
      zero_raw(next.x[m]);
      zero_raw(next.dt[m]);
      if (item < kTile * VECS && t < last && n > 0) {
        load_raw<WIDE>(xp + t * a.x.st + cv, next.x[m], n);
        load_raw<WIDE>(dp + t * a.dt.st + cv, next.dt[m], n);
      }
    }
  };
  // B and C come ahead too where they come in whole vectors
  const bool vectors = a.wide_bc && a.N == NP;
  const T* bp = (const T*)a.b.p + b * a.b.sb + q.g * a.b.sh;
  const T* cp = (const T*)a.c.p + b * a.c.sb + q.g * a.c.sh;
  RowLoads<T, NP, kTile, 2, kThreads> bc;
  fetch(first);
  if (vectors) bc.load(bp, a.b.st, cp, a.c.st, first, last, tid);
  __syncthreads();
  for (int t0 = first; t0 < last; t0 += kTile) {
    const TileLoads<T, ITEMS> now = next;
    Raw<T, 8> zr[ITEMS];
    bool finite = true;
#pragma unroll
    for (int m = 0; m < ITEMS; ++m) {
      const int item = tid + m * kThreads, t = item / VECS, cv = (item % VECS) * 8;
      if (item < kTile * VECS)
        finite &= stage_delta<T, PAD>(a, now.x[m], now.dt[m], sbias + cv, t0 + t < last, q.n - cv,
                                      sd + item * kPairUnit);
    }
    if (vectors) {
      bc.store(&sbc[0][0], tid);
      bc.load(bp, a.b.st, cp, a.c.st, t0 + kTile, last, tid);
    } else {
      stage_bc<T, NP, kTile>(a, b, q.g, t0, last, &sbc[0][0], tid, kThreads);
    }
    if (t0 + kTile < last) fetch(t0 + kTile);
    if (GATE) {
#pragma unroll
      for (int m = 0; m < ITEMS; ++m) {
        const int item = tid + m * kThreads, t = t0 + item / VECS, cv = (item % VECS) * 8, n = q.n - cv;
        zero_raw(zr[m]);
        if (item < kTile * VECS && t < last && n > 0) load_raw<WIDE>(zp + t * a.z.st + cv, zr[m], n);
      }
    }
    // whether padded states need care: an infinite delta or delta x, rare
    bool mask = false;
    if (PAD)
      mask = __syncthreads_or(!finite);
    else
      __syncthreads();
    // eight tokens, between two saved states, at a time
    constexpr int AT_ONCE = LPC / 2;  // tokens whose sums are taken together
    const float* dsrc[2] = {sd + (l.cl / 8) * kPairUnit + (l.ch[0] % 8) * 2,
                            sd + (l.cl / 8) * kPairUnit + (l.ch[1] % 8) * 2};
    float* ydst = sy + ((nl >> 1) * VECS + l.cl / 8) * kFloatUnit + l.ch[0] % 8;
    if (PAD && mask) {
      Lane lane = {{{A2[0][0], A2[0][1]}, {A2[1][0], A2[1][1]}}, {{h[0][0], h[0][1]}, {h[1][0], h[1][1]}}};
      float* keep[2];
#pragma unroll
      for (int e = 0; e < 2; ++e)
        keep[e] = a.saved != nullptr && l.ch[e] < q.n
                      ? a.saved + (((long long)b * NC + t0 / kScanEvery) * a.D + q.c0 + l.ch[e]) * NP + nl * 4
                      : nullptr;
      lane = walk_masked<LPC>(lane, nl, a.N, dsrc[0], dsrc[1], &sbc[0][nl * 4], ydst, keep[0], keep[1],
                              (long long)a.D * NP, last - t0);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        h[e][0] = lane.h[e][0];
        h[e][1] = lane.h[e][1];
      }
    }
#pragma unroll 1
    for (int tg = PAD && mask ? kTile : 0; tg < kTile; tg += kScanEvery) {
      if (a.saved != nullptr && t0 + tg < last) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (l.ch[e] < q.n)
            *reinterpret_cast<float4*>(
                a.saved + (((long long)b * NC + (t0 + tg) / kScanEvery) * a.D + q.c0 + l.ch[e]) * NP +
                nl * 4) = make_float4(h[e][0].x, h[e][0].y, h[e][1].x, h[e][1].y);
      }
      // The eight tokens' sums over the lanes come after all of their updates: then eight shuffles
      // are under way at once instead of each token waiting for its own.
      float2 y[kScanEvery], ex[2][2], w[2];
      auto ahead = [&](int t) {  // a token's decays, while the token before it is worked on
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float2 d = *reinterpret_cast<const float2*>(dsrc[e] + t * VECS * kPairUnit);
          const float2 dd = make_float2(d.x, d.x);
          ex[e][0] = exp2_pair(mul2(dd, A2[e][0]));
          ex[e][1] = exp2_pair(mul2(dd, A2[e][1]));
          w[e] = make_float2(d.y, d.y);
        }
      };
      ahead(tg);
#pragma unroll
      for (int u = 0; u < kScanEvery; ++u) {
        const int t = tg + u;
        const float4 Bv = *reinterpret_cast<const float4*>(&sbc[t][nl * 4]);
        const float4 Cv = *reinterpret_cast<const float4*>(&sbc[t][NP + nl * 4]);
        float2 E[2][2], W[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          E[e][0] = ex[e][0];
          E[e][1] = ex[e][1];
          W[e] = w[e];
        }
        if (u + 1 < kScanEvery) ahead(t + 1);
        float yv[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          h[e][0] = fma2(E[e][0], h[e][0], mul2(W[e], make_float2(Bv.x, Bv.y)));
          h[e][1] = fma2(E[e][1], h[e][1], mul2(W[e], make_float2(Bv.z, Bv.w)));
          const float2 v = fma2(h[e][1], make_float2(Cv.z, Cv.w), mul2(h[e][0], make_float2(Cv.x, Cv.y)));
          yv[e] = v.x + v.y;
        }
        y[u] = make_float2(yv[0], yv[1]);
      }
#pragma unroll
      for (int u = 0; u < kScanEvery; ++u) y[u].x += __shfl_xor_sync(0xffffffffu, y[u].y, 1);
#pragma unroll
      for (int ti = 0; ti < kScanEvery; ti += AT_ONCE) {
        float acc[AT_ONCE];
#pragma unroll
        for (int u = 0; u < AT_ONCE; ++u) acc[u] = y[ti + u].x;
        scatter_sum<AT_ONCE, AT_ONCE, 2>(acc, nl >> 1);
        ydst[(tg + ti) * VECS * kFloatUnit] = acc[0];
      }
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < ITEMS; ++m) {
      const int item = tid + m * kThreads, t = t0 + item / VECS, cv = (item % VECS) * 8, n = q.n - cv;
      if (item < kTile * VECS && t < last && n > 0) {
        float2 x[4], o[4], z[4];
        expand(now.x[m], x);
        load_unit(sy + item * kFloatUnit, o);
        if (a.skip != nullptr)  // without one nothing is added, not 0 times an infinite x
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] = fma2(*reinterpret_cast<const float2*>(sskip + cv + 2 * i), x[i], o[i]);
        if (GATE) {
          expand(zr[m], z);
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] = mul2(o[i], act_pair<kActSilu>(z[i]));
        }
        store_pairs<WIDE, 8>(yp + t * a.y.st + cv, o, n);
      }
    }
    // the next tile's sd and sbc were last read before the barrier above; its sy is written
    // after the next one
  }
  if (a.state_out != nullptr && last == a.T) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float hv[4] = {h[e][0].x, h[e][0].y, h[e][1].x, h[e][1].y};
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (l.ch[e] < q.n && nl * 4 + k < a.N)
          a.state_out[((long long)b * a.D + q.c0 + l.ch[e]) * a.N + nl * 4 + k] = hv[k];
    }
  }
  if (a.in_turn && last < a.T) {
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (l.ch[e] < q.n)
        __stcg(reinterpret_cast<float4*>(a.seg_state + ((long long)b * a.D + q.c0 + l.ch[e]) * NP + nl * 4),
               make_float4(h[e][0].x, h[e][0].y, h[e][1].x, h[e][1].y));
    pass_turn(a, bi);
  }
  }
}

// A segment's own state: REVERSE false, the forward state from zero over all segments but the
// last; true, the gradient that all segments but the first hand back, from zero and dy alone.  With
// them the segment's sum of delta, whose exponential carries a state across it.
template <typename T, int LPC, bool REVERSE, bool GATE, bool WIDE>
__global__ void __launch_bounds__(kThreads, kCtas) scan_segment_kernel(ScanArgs a, int tiles) {
  using S = Shape<LPC>;
  constexpr int NP = S::NP, CT = S::CT, VECS = S::VECS, ITEMS = S::ITEMS;
  __shared__ __align__(16) float sd[kTile * VECS * kPairUnit];  // delta and delta x, or delta and dy
  __shared__ __align__(16) float sv[kTile][NP];                 // B, or C
  __shared__ __align__(16) float sbias[CT];
  const int tid = threadIdx.x;
  const Lanes<LPC> l(tid);
  const int nl = l.nl;
  const int per_seg = a.B * a.G * tiles, bi = blockIdx.x % per_seg;
  const int seg = blockIdx.x / per_seg + (REVERSE ? 1 : 0);
  const int b = bi / (tiles * a.G);
  const ChannelTile q = channel_tile(a, bi % (tiles * a.G), tiles, CT);
  const int first = seg * a.seg_len, last = min(first + a.seg_len, a.T);
  float2 A2[2][2], h[2][2] = {};
  float sum[2] = {0.f, 0.f};
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    float av[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      av[k] = l.ch[e] < q.n && nl * 4 + k < a.N
                  ? finite_rate(a.A[(long long)(q.c0 + l.ch[e]) * a.N + nl * 4 + k] * kLog2e)
                  : kPadRate;
    A2[e][0] = make_float2(av[0], av[1]);
    A2[e][1] = make_float2(av[2], av[3]);
  }
  for (int i = tid; i < CT; i += kThreads)
    sbias[i] = a.dt_bias != nullptr && i < q.n ? a.dt_bias[q.c0 + i] : 0.f;
  // the second factor: x, or dy (with its gate)
  const Rows& wr = REVERSE ? a.y : a.x;
  const T* xp = (const T*)wr.p + b * wr.sb + q.c0;
  const T* dp = (const T*)a.dt.p + b * a.dt.sb + q.c0;
  const T* zp = GATE ? (const T*)a.z.p + b * a.z.sb + q.c0 : nullptr;
  const Rows& vr = REVERSE ? a.c : a.b;
  const T* vp = (const T*)vr.p + b * vr.sb + q.g * vr.sh;
  const int count = (last - first + kTile - 1) / kTile;
  TileLoads<T, ITEMS> next;
  auto fetch = [&](int t0) {
#pragma unroll
    for (int m = 0; m < ITEMS; ++m) {
      const int item = tid + m * kThreads, t = t0 + item / VECS, cv = (item % VECS) * 8, n = q.n - cv;
      zero_raw(next.x[m]);
      zero_raw(next.dt[m]);
      if (item < kTile * VECS && t < last && n > 0) {
        load_raw<WIDE>(xp + t * wr.st + cv, next.x[m], n);
        load_raw<WIDE>(dp + t * a.dt.st + cv, next.dt[m], n);
      }
    }
  };
  auto origin = [&](int i) { return first + (REVERSE ? count - 1 - i : i) * kTile; };
  const bool vectors = a.wide_bc && a.N == NP;
  RowLoads<T, NP, kTile, 1, kThreads> rows;
  fetch(origin(0));
  if (vectors) rows.load(vp, vr.st, nullptr, 0, origin(0), last, tid);
  __syncthreads();
  for (int i = 0; i < count; ++i) {
    const int t0 = origin(i);
    const TileLoads<T, ITEMS> now = next;
#pragma unroll
    for (int m = 0; m < ITEMS; ++m) {
      const int item = tid + m * kThreads, t = item / VECS, cv = (item % VECS) * 8, n = q.n - cv;
      if (item < kTile * VECS) {
        if (!REVERSE) {
          stage_delta<T>(a, now.x[m], now.dt[m], sbias + cv, t0 + t < last, n, sd + item * kPairUnit);
        } else {
          float2 g[4], z[4];
          expand(now.x[m], g);
          if (GATE) {
            Raw<T, 8> zr;
            zero_raw(zr);
            if (t0 + t < last && n > 0) load_raw<WIDE>(zp + (t0 + t) * a.z.st + cv, zr, n);
            expand(zr, z);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              g[k] = mul2(g[k], act_pair<kActSilu>(z[k]));
          }
          stage_pairs<T>(a, g, now.dt[m], sbias + cv, t0 + t < last, n, sd + item * kPairUnit);
        }
      }
    }
    if (vectors) {
      rows.store(&sv[0][0], tid);
      if (i + 1 < count) rows.load(vp, vr.st, nullptr, 0, origin(i + 1), last, tid);
    } else {
      for (int e0 = tid; e0 < kTile * NP; e0 += 8 * kThreads) {  // eight loads before their stores
        float v[8];
#pragma unroll
        for (int m = 0; m < 8; ++m) {
          const int e = e0 + m * kThreads, t = t0 + e / NP, n = e % NP;
          v[m] = e < kTile * NP && t < last && n < a.N ? to_f32(vp[t * vr.st + n]) : 0.f;
        }
#pragma unroll
        for (int m = 0; m < 8; ++m) {
          const int e = e0 + m * kThreads;
          if (e < kTile * NP) sv[e / NP][e % NP] = v[m];
        }
      }
    }
    if (i + 1 < count) fetch(origin(i + 1));
    __syncthreads();
    const float* dsrc[2] = {sd + (l.cl / 8) * kPairUnit + (l.ch[0] % 8) * 2,
                            sd + (l.cl / 8) * kPairUnit + (l.ch[1] % 8) * 2};
#pragma unroll 4
    for (int u = 0; u < kTile; ++u) {
      const int t = REVERSE ? kTile - 1 - u : u;
      const float4 V = *reinterpret_cast<const float4*>(&sv[t][nl * 4]);
      const float2 v0 = make_float2(V.x, V.y), v1 = make_float2(V.z, V.w);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float2 d = *reinterpret_cast<const float2*>(dsrc[e] + t * VECS * kPairUnit);
        const float2 dd = make_float2(d.x, d.x), ww = make_float2(d.y, d.y);
        const float2 e0 = exp2_pair(mul2(dd, A2[e][0])), e1 = exp2_pair(mul2(dd, A2[e][1]));
        if (REVERSE) {
          h[e][0] = mul2(e0, fma2(ww, v0, h[e][0]));
          h[e][1] = mul2(e1, fma2(ww, v1, h[e][1]));
        } else {
          h[e][0] = fma2(e0, h[e][0], mul2(ww, v0));
          h[e][1] = fma2(e1, h[e][1], mul2(ww, v1));
        }
        sum[e] += d.x;
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    if (l.ch[e] < q.n) {
      const long long row = ((long long)seg * a.B + b) * a.D + q.c0 + l.ch[e];
      *reinterpret_cast<float4*>(a.seg_state + row * NP + nl * 4) =
          make_float4(h[e][0].x, h[e][0].y, h[e][1].x, h[e][1].y);
      if (nl == 0) a.seg_sum[row] = sum[e];
    }
  }
}

// One token: eight states of one channel to a lane, in fours that are L fours apart, so that a
// channel's lanes read whole sectors.  Bound by the states, read and written once, and close behind
// by the instructions for delta and the gate, which each of a channel's lanes computes (four states
// to a lane, with twice the lanes, took 10.1 us where this takes 8.9: B = 64, D = 4096, N = 16, states
// from HBM, 34 MB in all; a copy of the states alone takes 5.5).  Each lane reads its own states before
// it writes them, so state_out may be state_in.  WIDE: the four states, and their elements of A, B
// and C, exist together and are read in one access each.
template <typename T, int L, bool WIDE>
__global__ void __launch_bounds__(256) scan_step_kernel(ScanArgs a, unsigned per_row,
                                                        unsigned group) {
  constexpr int CPB = 256 / L;
  const int nl = threadIdx.x % L;
  const unsigned b = blockIdx.x / per_row;
  const unsigned c0 = (blockIdx.x - b * per_row) * CPB + threadIdx.x / L;
  const bool live = c0 < (unsigned)a.D;
  const unsigned c = live ? c0 : 0, g = a.G == 1 ? 0 : c / group;
  const long long at = ((long long)b * a.D + c) * a.N;
  const T* bp = (const T*)a.b.p + b * a.b.sb + g * a.b.sh;
  const T* cp = (const T*)a.c.p + b * a.c.sb + g * a.c.sh;
  Raw<float, 4> sr[2], ar[2];
  Raw<T, 4> br[2], cr[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int n = (k * L + nl) * 4, left = live ? a.N - n : 0;
    zero_raw(sr[k]);
    zero_raw(ar[k]);
    zero_raw(br[k]);
    zero_raw(cr[k]);
    if (left > 0) {
      load_raw<WIDE>(a.state_in + at + n, sr[k], left);
      load_raw<WIDE>(a.A + (long long)c * a.N + n, ar[k], left);
      load_raw<WIDE>(bp + n, br[k], left);
      load_raw<WIDE>(cp + n, cr[k], left);
    }
  }
  const float x = to_f32(((const T*)a.x.p)[b * a.x.sb + c]);
  float delta = to_f32(((const T*)a.dt.p)[b * a.dt.sb + c]);
  const float z = a.z.p != nullptr ? to_f32(((const T*)a.z.p)[b * a.z.sb + c]) : 0.f;
  const float skip = a.skip != nullptr ? a.skip[c] : 0.f;
  if (a.dt_bias != nullptr) delta += a.dt_bias[c];
  if (a.softplus) delta = softplusf(delta);
  const float2 dd = make_float2(delta * kLog2e, delta * kLog2e), ww = make_float2(delta * x, delta * x);
  float acc = 0.f;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int n = (k * L + nl) * 4, left = live ? a.N - n : 0;
    float2 h[2], A[2], B[2], C[2];
    expand(sr[k], h);
    expand(ar[k], A);
    expand(br[k], B);
    expand(cr[k], C);
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      A[p] = make_float2(finite_rate(A[p].x), finite_rate(A[p].y));
      h[p] = fma2(exp2_pair(mul2(dd, A[p])), h[p], mul2(ww, B[p]));
      // Past N an infinite delta or x would add the product of infinity and nought.
      if (WIDE ? left > 0 : left > 2 * p) acc = fmaf(h[p].x, C[p].x, acc);
      if (WIDE ? left > 0 : left > 2 * p + 1) acc = fmaf(h[p].y, C[p].y, acc);
    }
    if (left > 0) store_pairs<WIDE, 4>(a.state_out + at + n, h, left);
  }
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  if (live && nl == 0) {
    if (a.skip != nullptr) acc = fmaf(skip, x, acc);
    if (a.z.p != nullptr) acc *= act_pair<kActSilu>(make_float2(z, z)).x;
    ((T*)a.y.p)[b * a.y.sb + c] = from_f32<T>(acc);
  }
}

template <typename T, int LPC, bool REVERSE>
cudaError_t segments(const ScanArgs& a, cudaStream_t s) {
  const int tiles = (a.D / a.G + Shape<LPC>::CT - 1) / Shape<LPC>::CT;
  const unsigned grid = (unsigned)((long long)a.B * a.G * tiles * (a.segs - 1));
  if (REVERSE && a.z.p != nullptr) {
    if (a.wide) scan_segment_kernel<T, LPC, REVERSE, REVERSE, true><<<grid, kThreads, 0, s>>>(a, tiles);
    else scan_segment_kernel<T, LPC, REVERSE, REVERSE, false><<<grid, kThreads, 0, s>>>(a, tiles);
  } else {
    if (a.wide) scan_segment_kernel<T, LPC, REVERSE, false, true><<<grid, kThreads, 0, s>>>(a, tiles);
    else scan_segment_kernel<T, LPC, REVERSE, false, false><<<grid, kThreads, 0, s>>>(a, tiles);
  }
  return cudaGetLastError();
}

template <typename T, int LPC>
cudaError_t fwd(const ScanArgs& a, cudaStream_t s) {
  if (a.segs > 1 && !a.in_turn) {
    const cudaError_t e = segments<T, LPC, false>(a, s);
    if (e != cudaSuccess) return e;
  }
  const int tiles = (a.D / a.G + Shape<LPC>::CT - 1) / Shape<LPC>::CT;
  const long long items = (long long)a.B * a.G * tiles * a.segs;
  const unsigned grid = (unsigned)(a.in_turn && items > kSlots ? kSlots : items);
  auto run = [&](auto* kernel) { kernel<<<grid, kThreads, 0, s>>>(a, tiles); };
  const bool pad = a.N != Shape<LPC>::NP;
  if (a.z.p != nullptr) {
    if (a.wide) run(pad ? scan_fwd_kernel<T, LPC, true, true, true> : scan_fwd_kernel<T, LPC, true, true, false>);
    else run(pad ? scan_fwd_kernel<T, LPC, true, false, true> : scan_fwd_kernel<T, LPC, true, false, false>);
  } else {
    if (a.wide) run(pad ? scan_fwd_kernel<T, LPC, false, true, true> : scan_fwd_kernel<T, LPC, false, true, false>);
    else run(pad ? scan_fwd_kernel<T, LPC, false, false, true> : scan_fwd_kernel<T, LPC, false, false, false>);
  }
  return cudaGetLastError();
}

template <typename T, int LPC>
cudaError_t step(const ScanArgs& a, cudaStream_t s) {
  // Blocks are whole rows of the batch apart: with one row of B D channels each thread divided by D
  // in 64 bits, and a call took 14.3 us instead of 10.1 (B = 64, D = 4096, N = 16).
  constexpr int L = LPC / 2, kPer = 256 / L;
  const unsigned per_row = (unsigned)((a.D + kPer - 1) / kPer), group = (unsigned)(a.D / a.G);
  if (a.N % 4 == 0 && a.wide_bc && ((uintptr_t)a.A & 15) == 0)
    scan_step_kernel<T, L, true><<<per_row * a.B, 256, 0, s>>>(a, per_row, group);
  else
    scan_step_kernel<T, L, false><<<per_row * a.B, 256, 0, s>>>(a, per_row, group);
  return cudaGetLastError();
}

enum Pass { kFwd, kStep, kReverseSegments };

template <Pass P, typename T, int LPC>
cudaError_t run_pass(const ScanArgs& a, cudaStream_t s) {
  if constexpr (P == kFwd) return fwd<T, LPC>(a, s);
  if constexpr (P == kStep) return step<T, LPC>(a, s);
  return segments<T, LPC, true>(a, s);
}
template <Pass P, typename T>
cudaError_t by_states(const ScanArgs& a, cudaStream_t s) {
  switch (scan_pad(a.N)) {
    case 8: return run_pass<P, T, 2>(a, s);
    case 16: return run_pass<P, T, 4>(a, s);
    case 32: return run_pass<P, T, 8>(a, s);
    default: return run_pass<P, T, 16>(a, s);
  }
}
template <Pass P>
cudaError_t by_type(const ScanArgs& a, cudaStream_t s) {
  return a.dtype == 0 ? by_states<P, bf16>(a, s) : by_states<P, float>(a, s);
}

__global__ void selftest_kernel(unsigned int* words) { selftest_wait(words, &g_scan_fwd_failures); }

}  // namespace

ScanSegments scan_cut(int T, int tile, long long ctas, int slots) {
  constexpr int most = 256, unit = 32;  // tokens of a segment in turn, at least; and a divisor of them
  ScanSegments z = {T, 1, false, (int)ctas};
  long long segs = 1;
  if (ctas > slots) {
    // In turn: about eight rounds of items, so that the last, partly empty one is an eighth.
    segs = (8LL * slots + ctas - 1) / ctas;
    if (segs > T / most) segs = T / most;
    z.in_turn = segs > 1;
    tile = unit;
  } else if (2 * ctas <= slots && T > 2 * tile) {
    // At once: as many segments as fill the GPU, down to a tile each; the first pass over them adds
    // about half of the scan's own work.  With two tiles at least to a segment, B2 T577 D201 N12 fp32
    // took 33 us forward and 56 backward instead of 18 and 31.
    segs = slots / (ctas > 0 ? ctas : 1);
  }
  if (segs <= 1) return z;
  const long long tiles = (T + tile - 1) / tile;
  z.len = (int)((tiles + segs - 1) / segs) * tile;
  z.count = (T + z.len - 1) / z.len;
  return z;
}

ScanSegments scan_fwd_segments(int B, int T, int D, int G, int N) {
  const int CT = 2 * kThreads * 4 / scan_pad(N);
  return scan_cut(T, kTile, (long long)B * G * ((D / G + CT - 1) / CT), kSlots);
}

cudaError_t launch_scan_fwd_selftest(unsigned int* words, cudaStream_t s) {
  selftest_kernel<<<1, 1, 0, s>>>(words);
  return cudaGetLastError();
}
cudaError_t scan_fwd_flag(unsigned int** at) { return cudaGetSymbolAddress((void**)at, g_scan_fwd_failures); }

cudaError_t launch_scan_fwd(const ScanArgs& a, cudaStream_t s) { return by_type<kFwd>(a, s); }
cudaError_t launch_scan_step(const ScanArgs& a, cudaStream_t s) { return by_type<kStep>(a, s); }
cudaError_t launch_scan_reverse_segments(const ScanArgs& a, cudaStream_t s) {
  return by_type<kReverseSegments>(a, s);
}

}  // namespace mlstm

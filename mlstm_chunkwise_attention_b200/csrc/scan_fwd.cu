// Selective state space scan, forward and one-token step.
//
// The scan is serial in time, so parallelism comes from batches, channels and states: a
// thread holds four states of one channel in registers and walks the sequence.  Tiles of 32
// tokens go through shared memory: delta and delta x are computed once per (token,
// channel) from 16-byte loads, B and C are shared by all channels, and y is summed over
// the channel's lanes by a transposing reduction (LPC tokens at a time, one result per
// lane), then gated and stored with 16-byte stores.
//
// Bound by the exponentials: one ex2 per state, channel and token.
#include "scan_common.cuh"

namespace mlstm {

namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps, kTile = 32;

template <typename T, int LPC, bool GATE, bool WIDE>
__global__ void __launch_bounds__(kThreads) scan_fwd_kernel(ScanArgs a, int tiles) {
  constexpr int NP = 4 * LPC, CT = kWarps * 32 / LPC, VECS = CT / 8;
  constexpr int ITEMS = (kTile * VECS + kThreads - 1) / kThreads;
  __shared__ __align__(16) float2 sd[kTile][CT];   // delta, delta x
  __shared__ __align__(16) float sy[kTile][CT];
  __shared__ __align__(16) float sbc[kTile][2 * NP];
  const int tid = threadIdx.x, lane = tid & 31, nl = lane % LPC;
  const int cl = (tid / 32) * (32 / LPC) + lane / LPC;  // channel within the tile
  const int b = blockIdx.x / (tiles * a.G);
  const ChannelTile q = channel_tile(a, blockIdx.x % (tiles * a.G), tiles, CT);
  const bool live = cl < q.n;
  const int c = q.c0 + cl, NC = (a.T + kScanEvery - 1) / kScanEvery;
  float A2[4], h[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int n = nl * 4 + k;
    const bool on = live && n < a.N;
    A2[k] = on ? a.A[(long long)c * a.N + n] * kLog2e : 0.f;
    h[k] = on && a.state_in != nullptr ? a.state_in[((long long)b * a.D + c) * a.N + n] : 0.f;
  }
  const T* xp = (const T*)a.x.p + b * a.x.sb + q.c0;
  const T* dp = (const T*)a.dt.p + b * a.dt.sb + q.c0;
  const T* zp = GATE ? (const T*)a.z.p + b * a.z.sb + q.c0 : nullptr;
  T* yp = (T*)a.y.p + b * a.y.sb + q.c0;

  for (int t0 = 0; t0 < a.T; t0 += kTile) {
    float xv[ITEMS][8];
#pragma unroll
    for (int m = 0; m < ITEMS; ++m) {
      const int item = tid + m * kThreads, t = item / VECS, cv = (item % VECS) * 8;
      if (item < kTile * VECS) {
        const int n = min(8, q.n - cv);
        float dv[8];
        const bool in = t0 + t < a.T && n > 0;
        if (in) {
          load8<WIDE>(xp + (t0 + t) * a.x.st + cv, xv[m], n);
          load8<WIDE>(dp + (t0 + t) * a.dt.st + cv, dv, n);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float delta = 0.f, dx = 0.f;
          if (in && i < n) {
            delta = dv[i] + (a.dt_bias != nullptr ? a.dt_bias[q.c0 + cv + i] : 0.f);
            if (a.softplus) delta = softplusf(delta);
            dx = delta * xv[m][i];
          }
          sd[t][cv + i] = make_float2(delta, dx);
        }
      }
    }
    stage_bc<T, NP, kTile>(a, b, q.g, t0, &sbc[0][0], tid, kThreads);
    __syncthreads();
    for (int t = 0; t < kTile; t += LPC) {
      float acc[LPC];
#pragma unroll
      for (int u = 0; u < LPC; ++u) {
        if (a.saved != nullptr && ((t + u) % kScanEvery) == 0 && t0 + t + u < a.T && live)
          *reinterpret_cast<float4*>(a.saved +
                                     (((long long)b * NC + (t0 + t + u) / kScanEvery) * a.D + c) * NP +
                                     nl * 4) = make_float4(h[0], h[1], h[2], h[3]);
        const float2 d = sd[t + u][cl];
        const float4 Bv = *reinterpret_cast<const float4*>(&sbc[t + u][nl * 4]);
        const float4 Cv = *reinterpret_cast<const float4*>(&sbc[t + u][NP + nl * 4]);
        h[0] = fmaf(exp2_fast(d.x * A2[0]), h[0], d.y * Bv.x);
        h[1] = fmaf(exp2_fast(d.x * A2[1]), h[1], d.y * Bv.y);
        h[2] = fmaf(exp2_fast(d.x * A2[2]), h[2], d.y * Bv.z);
        h[3] = fmaf(exp2_fast(d.x * A2[3]), h[3], d.y * Bv.w);
        acc[u] = fmaf(h[0], Cv.x, fmaf(h[1], Cv.y, fmaf(h[2], Cv.z, h[3] * Cv.w)));
      }
      scatter_sum<LPC, LPC, 1>(acc, nl);
      sy[t + nl][cl] = acc[0];
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < ITEMS; ++m) {
      const int item = tid + m * kThreads, t = item / VECS, cv = (item % VECS) * 8;
      const int n = min(8, q.n - cv);
      if (item < kTile * VECS && t0 + t < a.T && n > 0) {
        float z[8], o[8];
        if (GATE) load8<WIDE>(zp + (t0 + t) * a.z.st + cv, z, n);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          o[i] = sy[t][cv + i];
          if (a.skip != nullptr && i < n) o[i] = fmaf(a.skip[q.c0 + cv + i], xv[m][i], o[i]);
          if (GATE) o[i] *= act_value<kActSilu>(z[i]);
        }
        store8<WIDE>(yp + (t0 + t) * a.y.st + cv, o, n);
      }
    }
    // the next tile's sd and sbc were last read before the barrier above; its sy is written
    // after the next one
  }
  if (a.state_out != nullptr && live)
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (nl * 4 + k < a.N) a.state_out[((long long)b * a.D + c) * a.N + nl * 4 + k] = h[k];
}

// One token: four states of one channel to a lane.  Bound by the states, read and written once.
// Each lane reads its own states before it writes them, so state_out may be state_in.
template <typename T, int LPC>
__global__ void __launch_bounds__(256) scan_step_kernel(ScanArgs a) {
  constexpr int CPB = 256 / LPC;
  const int lane = threadIdx.x & 31, nl = lane % LPC;
  const long long row = (long long)blockIdx.x * CPB + threadIdx.x / LPC;  // b D + c
  const bool live = row < (long long)a.B * a.D;
  const int b = live ? (int)(row / a.D) : 0, c = live ? (int)(row % a.D) : 0, g = c / (a.D / a.G);
  const int n0 = nl * 4, left = live ? a.N - n0 : 0;
  const float x = to_f32(((const T*)a.x.p)[b * a.x.sb + c]);
  float delta = to_f32(((const T*)a.dt.p)[b * a.dt.sb + c]);
  if (a.dt_bias != nullptr) delta += a.dt_bias[c];
  if (a.softplus) delta = softplusf(delta);
  const T* bp = (const T*)a.b.p + b * a.b.sb + g * a.b.sh + n0;
  const T* cp = (const T*)a.c.p + b * a.c.sb + g * a.c.sh + n0;
  const float* si = a.state_in + ((long long)b * a.D + c) * a.N + n0;
  float* so = a.state_out + ((long long)b * a.D + c) * a.N + n0;
  const float* A = a.A + (long long)c * a.N + n0;
  float h[4], acc = 0.f;
  const bool whole = a.N % 4 == 0;  // the four states exist together and are 16-byte aligned
  if (whole && left > 0) {
    const float4 v = *reinterpret_cast<const float4*>(si);
    h[0] = v.x; h[1] = v.y; h[2] = v.z; h[3] = v.w;
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) h[k] = k < left ? si[k] : 0.f;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (k < left) {
      h[k] = fmaf(exp2_fast(delta * (A[k] * kLog2e)), h[k], delta * x * to_f32(bp[k]));
      acc = fmaf(h[k], to_f32(cp[k]), acc);
    }
  if (whole && left > 0) {
    *reinterpret_cast<float4*>(so) = make_float4(h[0], h[1], h[2], h[3]);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < left) so[k] = h[k];
  }
#pragma unroll
  for (int o = LPC / 2; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  if (live && nl == 0) {
    if (a.skip != nullptr) acc = fmaf(a.skip[c], x, acc);
    if (a.z.p != nullptr) acc *= act_value<kActSilu>(to_f32(((const T*)a.z.p)[b * a.z.sb + c]));
    ((T*)a.y.p)[b * a.y.sb + c] = from_f32<T>(acc);
  }
}

template <typename T, int LPC>
cudaError_t fwd(const ScanArgs& a, cudaStream_t s) {
  constexpr int CT = kWarps * 32 / LPC;
  const int tiles = (a.D / a.G + CT - 1) / CT;
  const unsigned grid = (unsigned)((long long)a.B * a.G * tiles);
  if (a.z.p != nullptr) {
    if (a.wide) scan_fwd_kernel<T, LPC, true, true><<<grid, kThreads, 0, s>>>(a, tiles);
    else scan_fwd_kernel<T, LPC, true, false><<<grid, kThreads, 0, s>>>(a, tiles);
  } else {
    if (a.wide) scan_fwd_kernel<T, LPC, false, true><<<grid, kThreads, 0, s>>>(a, tiles);
    else scan_fwd_kernel<T, LPC, false, false><<<grid, kThreads, 0, s>>>(a, tiles);
  }
  return cudaGetLastError();
}

template <typename T, int LPC>
cudaError_t step(const ScanArgs& a, cudaStream_t s) {
  const long long rows = (long long)a.B * a.D, per = 256 / LPC;
  scan_step_kernel<T, LPC><<<(unsigned)((rows + per - 1) / per), 256, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T, bool STEP>
cudaError_t by_states(const ScanArgs& a, cudaStream_t s) {
  switch (scan_pad(a.N)) {
    case 8: return STEP ? step<T, 2>(a, s) : fwd<T, 2>(a, s);
    case 16: return STEP ? step<T, 4>(a, s) : fwd<T, 4>(a, s);
    case 32: return STEP ? step<T, 8>(a, s) : fwd<T, 8>(a, s);
    default: return STEP ? step<T, 16>(a, s) : fwd<T, 16>(a, s);
  }
}

}  // namespace

cudaError_t launch_scan_fwd(const ScanArgs& a, cudaStream_t s) {
  return a.dtype == 0 ? by_states<bf16, false>(a, s) : by_states<float, false>(a, s);
}
cudaError_t launch_scan_step(const ScanArgs& a, cudaStream_t s) {
  return a.dtype == 0 ? by_states<bf16, true>(a, s) : by_states<float, true>(a, s);
}

}  // namespace mlstm

// Short causal convolution, one filter of W taps per channel:
//
//   pre[t, c] = bias[c] + sum_{j < W} w[c, j] x[t - (W - 1) + j, c],  y = act(pre)
//
// and its backward, with dp = dy act'(pre):
//
//   dx_t = sum_j w_j dp_{t + W - 1 - j}   dw_j = sum_t dp_t x_{t - W + 1 + j}   dbias = sum_t dp_t
//
// Bound by HBM: about W multiply-adds per element moved.  A thread owns a few
// channels and walks a run of tokens with the last W - 1 inputs in registers,
// so each input is loaded once per run plus W - 1 tokens of the run before it.
// Inputs and outputs are addressed by strides: the convolved half of a wider
// projection is read in place, and y can be written head-major.
#include "block_common.cuh"

namespace mlstm {

namespace {

// Channels c0 .. c0 + 7 of token t, where t < 0 is the carried state (or zero).
template <typename T, int W, bool WIDE>
__device__ __forceinline__ void load_input(const ConvArgs& a, const T* x, const T* st, int t, int c0,
                                           int n, float* v) {
  if (t >= 0) {
    load8<WIDE>(x + (long long)t * a.x.st, v, n);
  } else if (st != nullptr) {
    load8<WIDE>(st + (long long)(t + W - 1) * a.D() + c0, v, n);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.f;
  }
}

// Writes channels c0 .. c0 + n - 1 of a row whose channels lie in heads of d.
template <typename T, bool WIDE>
__device__ __forceinline__ void store_heads(T* row, long long sh, int d, int c0, int n, const float* v) {
  if (WIDE) {  // d is a multiple of 8, so the eight channels share a head
    store8<true>(row + (c0 / d) * sh + c0 % d, v, n);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) row[((c0 + i) / d) * sh + (c0 + i) % d] = from_f32<T>(v[i]);
  }
}

template <typename T, int W, int ACT, bool WIDE>
__global__ void __launch_bounds__(128) conv_fwd_kernel(ConvArgs a, int run, int runs, int vecs) {
  const long long item = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (item >= (long long)vecs * runs * a.B) return;
  const int c0 = (int)(item % vecs) * 8;
  const long long br = item / vecs;
  const int t0 = (int)(br % runs) * run, b = (int)(br / runs);
  const int D = a.D(), n = min(8, D - c0);
  const T* x = (const T*)a.x.p + (long long)b * a.x.sb + c0;
  const T* st = a.state_in ? (const T*)a.state_in + (long long)b * (W - 1) * D : nullptr;
  T* y = (T*)a.y.p + (long long)b * a.y.sb;
  float w[W][8], bias[8], win[W - 1][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    bias[i] = a.bias != nullptr && i < n ? a.bias[c0 + i] : 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) w[j][i] = i < n ? a.w[(long long)(c0 + i) * W + j] : 0.f;
  }
#pragma unroll
  for (int j = 0; j < W - 1; ++j) load_input<T, W, WIDE>(a, x, st, t0 - (W - 1) + j, c0, n, win[j]);
  const int t1 = min(t0 + run, a.T);
  constexpr int U = 4;  // tokens in flight
  for (int tb = t0; tb < t1; tb += U) {
    float v[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (tb + u < t1) load8<WIDE>(x + (long long)(tb + u) * a.x.st, v[u], n);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (tb + u < t1) {
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float p = bias[i];
#pragma unroll
          for (int j = 0; j < W - 1; ++j) p = fmaf(w[j][i], win[j][i], p);
          p = fmaf(w[W - 1][i], v[u][i], p);
          o[i] = act_value<ACT>(p);
#pragma unroll
          for (int j = 0; j + 2 < W; ++j) win[j][i] = win[j + 1][i];
          win[W - 2][i] = v[u][i];
        }
        store_heads<T, WIDE>(y + (long long)(tb + u) * a.y.st, a.y.sh, a.d, c0, n, o);
      }
    }
  }
  if (a.state_out != nullptr && t1 == a.T) {  // the window is the last W - 1 inputs
    T* so = (T*)a.state_out + (long long)b * (W - 1) * D + c0;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) store8<WIDE>(so + (long long)j * D, win[j], n);
  }
}

// One token: each thread reads its channels' carried inputs before it writes them, so
// state_out may be state_in.
template <typename T, int W, int ACT, bool WIDE>
__global__ void __launch_bounds__(128) conv_step_kernel(ConvArgs a, int vecs) {
  const long long item = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (item >= (long long)vecs * a.B) return;
  const int c0 = (int)(item % vecs) * 8, b = (int)(item / vecs);
  const int D = a.D(), n = min(8, D - c0);
  const T* st = (const T*)a.state_in + (long long)b * (W - 1) * D + c0;
  T* so = (T*)a.state_out + (long long)b * (W - 1) * D + c0;
  float v[W][8], o[8];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) load8<WIDE>(st + (long long)j * D, v[j], n);
  load8<WIDE>((const T*)a.x.p + (long long)b * a.x.sb + c0, v[W - 1], n);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float p = a.bias != nullptr && i < n ? a.bias[c0 + i] : 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) p = fmaf(i < n ? a.w[(long long)(c0 + i) * W + j] : 0.f, v[j][i], p);
    o[i] = act_value<ACT>(p);
  }
  store_heads<T, WIDE>((T*)a.y.p + (long long)b * a.y.sb, a.y.sh, a.d, c0, n, o);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) store8<WIDE>(so + (long long)j * D, v[j + 1], n);
}

constexpr int kBwdRun = 64;    // tokens of one thread's run
constexpr int kBwdLanes = 32;  // channel vectors of a CTA
constexpr int kBwdRuns = 4;    // runs of a CTA, joined in shared memory
constexpr int kBwdC = 4;       // channels of a thread: W windows of x and dp stay in registers

template <bool WIDE>
__device__ __forceinline__ void load4(const bf16* p, float* v, int n) {
  if (WIDE) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    v[0] = __uint_as_float(u.x << 16); v[1] = __uint_as_float(u.x & 0xffff0000u);
    v[2] = __uint_as_float(u.y << 16); v[3] = __uint_as_float(u.y & 0xffff0000u);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = i < n ? to_f32(p[i]) : 0.f;
  }
}
template <bool WIDE>
__device__ __forceinline__ void load4(const float* p, float* v, int n) {
  if (WIDE) {
    const float4 u = *reinterpret_cast<const float4*>(p);
    v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = i < n ? p[i] : 0.f;
  }
}
template <bool WIDE>
__device__ __forceinline__ void store4(bf16* p, const float* v, int n) {
  if (WIDE) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    uint2 u;
    u.x = *reinterpret_cast<const uint32_t*>(&a);
    u.y = *reinterpret_cast<const uint32_t*>(&b);
    *reinterpret_cast<uint2*>(p) = u;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = from_f32<bf16>(v[i]);
  }
}
template <bool WIDE>
__device__ __forceinline__ void store4(float* p, const float* v, int n) {
  if (WIDE) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = v[i];
  }
}

// A thread walks tokens t0 .. t0 + run + W - 2 of its channels: it recomputes pre at each,
// forms dp, and W - 1 tokens later emits dx, whose last term is then known.  The first run
// of a sequence also emits the carried state's gradient (tokens -(W - 1) .. -1).  Sums over
// tokens are taken for the run's own tokens only and joined over the CTA's runs, one row
// of partials per CTA.
template <typename T, int W, int ACT, bool WIDE>
__global__ void __launch_bounds__(kBwdLanes * kBwdRuns) conv_bwd_kernel(ConvArgs a, int run, int runs,
                                                                       int vecs, int cblocks) {
  __shared__ float red[kBwdRuns][W + 1][kBwdC][kBwdLanes];
  const int lane = threadIdx.x, rr = threadIdx.y;
  const int vec = (int)(blockIdx.x % cblocks) * kBwdLanes + lane;
  const long long row = blockIdx.x / cblocks;          // partial row of this CTA
  const long long br = row * kBwdRuns + rr;            // run of all batches
  const int D = a.D();
  float dw[W][kBwdC], db[kBwdC];
#pragma unroll
  for (int i = 0; i < kBwdC; ++i) {
    db[i] = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) dw[j][i] = 0.f;
  }
  if (vec < vecs && br < (long long)runs * a.B) {
    const int c0 = vec * kBwdC, n = min(kBwdC, D - c0);
    const int t0 = (int)(br % runs) * run, b = (int)(br / runs);
    const int t1 = min(t0 + run, a.T);
    const T* x = (const T*)a.x.p + (long long)b * a.x.sb + c0;
    const T* st = a.state_in ? (const T*)a.state_in + (long long)b * (W - 1) * D + c0 : nullptr;
    const T* dy = (const T*)a.y.p + (long long)b * a.y.sb;
    long long off[kBwdC];  // of each channel in a row of dy
#pragma unroll
    for (int i = 0; i < kBwdC; ++i) off[i] = i < n ? ((c0 + i) / a.d) * a.y.sh + (c0 + i) % a.d : 0;
    T* dx = (T*)a.dx.p + (long long)b * a.dx.sb + c0;
    float w[W][kBwdC], bias[kBwdC], win[W][kBwdC], dp[W][kBwdC];
#pragma unroll
    for (int i = 0; i < kBwdC; ++i) {
      bias[i] = a.bias != nullptr && i < n ? a.bias[c0 + i] : 0.f;
#pragma unroll
      for (int j = 0; j < W; ++j) {
        w[j][i] = i < n ? a.w[(long long)(c0 + i) * W + j] : 0.f;
        dp[j][i] = 0.f;
      }
    }
    // win[j] = x_{tau - (W - 1) + j}; one step before tau = t0 it holds tokens t0 - W .. t0 - 1,
    // of which the first is shifted out unread
#pragma unroll
    for (int j = 1; j < W; ++j) {
      const int t = t0 - W + j;
      if (t >= 0)
        load4<WIDE>(x + (long long)t * a.x.st, win[j], n);
      else if (st != nullptr)
        load4<WIDE>(st + (long long)(t + W - 1) * D, win[j], n);
      else
#pragma unroll
        for (int i = 0; i < kBwdC; ++i) win[j][i] = 0.f;
    }
    const int emit0 = t0 == 0 ? -(W - 1) : t0;  // first token whose gradient this run writes
    const int end = t1 + W - 1;                 // dx of t1 - 1 is complete at tau = t1 + W - 2
    constexpr int U = 4;
    for (int tb = t0; tb < end; tb += U) {
      float xv[U][kBwdC], gv[U][kBwdC];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = tb + u;
        if (t < end && t < a.T) {
          load4<WIDE>(x + (long long)t * a.x.st, xv[u], n);
          if (WIDE) {
            load4<true>(dy + (long long)t * a.y.st + off[0], gv[u], n);
          } else {
#pragma unroll
            for (int i = 0; i < kBwdC; ++i)
              gv[u][i] = i < n ? to_f32(dy[(long long)t * a.y.st + off[i]]) : 0.f;
          }
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = tb + u;
        if (t < end) {
          const bool in = t < a.T;
#pragma unroll
          for (int i = 0; i < kBwdC; ++i) {
#pragma unroll
            for (int j = 0; j + 1 < W; ++j) {
              win[j][i] = win[j + 1][i];
              dp[j][i] = dp[j + 1][i];
            }
            win[W - 1][i] = in ? xv[u][i] : 0.f;
            float p = bias[i], val, slope;
#pragma unroll
            for (int j = 0; j < W; ++j) p = fmaf(w[j][i], win[j][i], p);
            act_slope<ACT>(p, &val, &slope);
            dp[W - 1][i] = in ? gv[u][i] * slope : 0.f;
            if (t < t1) {
              db[i] += dp[W - 1][i];
#pragma unroll
              for (int j = 0; j < W; ++j) dw[j][i] = fmaf(dp[W - 1][i], win[j][i], dw[j][i]);
            }
          }
          const int e = t - (W - 1);  // the token whose gradient is complete
          if (e >= emit0 && e < t1) {
            float o[kBwdC];
#pragma unroll
            for (int i = 0; i < kBwdC; ++i) {
              o[i] = 0.f;
#pragma unroll
              for (int j = 0; j < W; ++j) o[i] = fmaf(w[j][i], dp[W - 1 - j][i], o[i]);
            }
            const int r = e - a.T + W - 1;  // row of the final state that is token e
            if (a.dstate_out != nullptr && r >= 0) {
              float g[kBwdC];
              load4<WIDE>((const T*)a.dstate_out + ((long long)b * (W - 1) + r) * D + c0, g, n);
#pragma unroll
              for (int i = 0; i < kBwdC; ++i) o[i] += g[i];
            }
            if (e >= 0)
              store4<WIDE>(dx + (long long)e * a.dx.st, o, n);
            else if (a.dstate_in != nullptr)
              store4<WIDE>((T*)a.dstate_in + ((long long)b * (W - 1) + e + W - 1) * D + c0, o, n);
          }
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kBwdC; ++i) {
    red[rr][W][i][lane] = db[i];
#pragma unroll
    for (int j = 0; j < W; ++j) red[rr][j][i][lane] = dw[j][i];
  }
  __syncthreads();
  // [W + 1][channels] sums of this CTA, channels contiguous
  const int tid = rr * kBwdLanes + lane, cbase = (int)(blockIdx.x % cblocks) * kBwdLanes * kBwdC;
  for (int e = tid; e < (W + 1) * kBwdLanes * kBwdC; e += kBwdLanes * kBwdRuns) {
    const int k = e / (kBwdLanes * kBwdC), c = e % (kBwdLanes * kBwdC);
    float s = 0.f;
#pragma unroll
    for (int q = 0; q < kBwdRuns; ++q) s += red[q][k][c % kBwdC][c / kBwdC];
    if (cbase + c < D) a.partial[(row * (W + 1) + k) * D + cbase + c] = s;
  }
}

// Sums over the rows of partials, 8 row shares to a column joined in a fixed order.
__global__ void __launch_bounds__(256) param_sums_kernel(const float* __restrict__ partial,
                                                         float* __restrict__ dw,
                                                         float* __restrict__ dbias, int rows, int D,
                                                         int W) {
  __shared__ float red[8][32];
  const int lane = threadIdx.x & 31, part = threadIdx.x >> 5;
  const long long col = (long long)blockIdx.x * 32 + lane, cols = (long long)(W + 1) * D;
  float s = 0.f;
  if (col < cols)
#pragma unroll 4
    for (int r = part; r < rows; r += 8) s += partial[(long long)r * cols + col];
  red[part][lane] = s;
  __syncthreads();
  if (part == 0 && col < cols) {
    s = 0.f;
#pragma unroll
    for (int q = 0; q < 8; ++q) s += red[q][lane];
    const int j = (int)(col / D);
    const long long c = col % D;
    if (j < W) {
      if (dw != nullptr) dw[c * W + j] = s;
    } else if (dbias != nullptr)
      dbias[c] = s;
  }
}

int bwd_runs(int T) { return (T + kBwdRun - 1) / kBwdRun; }

template <typename T, int W, int ACT, bool WIDE>
cudaError_t fwd(const ConvArgs& a, cudaStream_t s) {
  const int vecs = (a.D() + 7) / 8;
  // Runs of 32 tokens (3 of 35 loads are the halo), shorter while that leaves under two
  // thousand warps: few rows then spread over the GPU.
  int run = 32;
  while (run > 4 && (long long)vecs * a.B * ((a.T + run - 1) / run) < 65536) run /= 2;
  const int runs = (a.T + run - 1) / run;
  const long long items = (long long)vecs * runs * a.B;
  conv_fwd_kernel<T, W, ACT, WIDE><<<(unsigned)((items + 127) / 128), 128, 0, s>>>(a, run, runs, vecs);
  return cudaGetLastError();
}

template <typename T, int W, int ACT, bool WIDE>
cudaError_t step(const ConvArgs& a, cudaStream_t s) {
  const int vecs = (a.D() + 7) / 8;
  const long long items = (long long)vecs * a.B;
  conv_step_kernel<T, W, ACT, WIDE><<<(unsigned)((items + 127) / 128), 128, 0, s>>>(a, vecs);
  return cudaGetLastError();
}

template <typename T, int W, int ACT, bool WIDE>
cudaError_t bwd(const ConvArgs& a, cudaStream_t s) {
  const int D = a.D(), vecs = (D + kBwdC - 1) / kBwdC, cblocks = (vecs + kBwdLanes - 1) / kBwdLanes;
  const int rows = conv_bwd_rows(a.B, a.T, D);
  conv_bwd_kernel<T, W, ACT, WIDE>
      <<<(unsigned)((long long)rows * cblocks), dim3(kBwdLanes, kBwdRuns), 0, s>>>(
          a, kBwdRun, bwd_runs(a.T), vecs, cblocks);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_param_sums(a.partial, rows, D, W, a.dw, a.dbias, s);
}

enum Pass { kFwd, kStep, kBwd };

template <Pass P, typename T, int W, int ACT, bool WIDE>
cudaError_t run_pass(const ConvArgs& a, cudaStream_t s) {
  if constexpr (P == kFwd) return fwd<T, W, ACT, WIDE>(a, s);
  if constexpr (P == kStep) return step<T, W, ACT, WIDE>(a, s);
  return bwd<T, W, ACT, WIDE>(a, s);
}
template <Pass P, typename T, int W>
cudaError_t by_act(const ConvArgs& a, cudaStream_t s) {
  if (a.act == kActSilu)
    return a.wide ? run_pass<P, T, W, kActSilu, true>(a, s) : run_pass<P, T, W, kActSilu, false>(a, s);
  return a.wide ? run_pass<P, T, W, kActNone, true>(a, s) : run_pass<P, T, W, kActNone, false>(a, s);
}
template <Pass P, typename T>
cudaError_t by_taps(const ConvArgs& a, cudaStream_t s) {
  if (a.W == 2) return by_act<P, T, 2>(a, s);
  if (a.W == 3) return by_act<P, T, 3>(a, s);
  return by_act<P, T, 4>(a, s);
}
template <Pass P>
cudaError_t by_type(const ConvArgs& a, cudaStream_t s) {
  return a.dtype == 0 ? by_taps<P, bf16>(a, s) : by_taps<P, float>(a, s);
}

}  // namespace

int conv_bwd_rows(int B, int T, int) {
  return (int)(((long long)B * bwd_runs(T) + kBwdRuns - 1) / kBwdRuns);
}

cudaError_t launch_param_sums(const float* partial, int rows, int D, int W, float* dw, float* dbias,
                              cudaStream_t s) {
  param_sums_kernel<<<(unsigned)(((long long)(W + 1) * D + 31) / 32), 256, 0, s>>>(partial, dw, dbias,
                                                                                   rows, D, W);
  return cudaGetLastError();
}

cudaError_t launch_conv_fwd(const ConvArgs& a, cudaStream_t s) { return by_type<kFwd>(a, s); }
cudaError_t launch_conv_step(const ConvArgs& a, cudaStream_t s) { return by_type<kStep>(a, s); }
cudaError_t launch_conv_bwd(const ConvArgs& a, cudaStream_t s) { return by_type<kBwd>(a, s); }

}  // namespace mlstm

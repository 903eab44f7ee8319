// Short causal convolution, one filter of W taps per channel:
//
//   pre[t, c] = bias[c] + sum_{j < W} w[c, j] x[t - (W - 1) + j, c],  y = act(pre)
//
// and its backward, with dp = dy act'(pre):
//
//   dx_t = sum_j w_j dp_{t + W - 1 - j}   dw_j = sum_t dp_t x_{t - W + 1 + j}   dbias = sum_t dp_t
//
// Bound by HBM: about W multiply-adds per element moved.  A thread owns four
// channels and walks a run of tokens with the last W - 1 inputs in registers,
// so each input is loaded once per run plus W - 1 tokens of the run before it.
// Inputs and outputs are addressed by strides: the convolved half of a wider
// projection is read in place, and y can be written head-major.
//
// Measured on one B200 at B8 T4096 D4096 W4 bf16 with SiLU: forward 103 us, 5.2 TB/s or 0.80 of
// a plain copy; backward with its parameter sums 176 us, 4.6 TB/s or 0.71, where 0.57 of the cycles issue
// and the fp32 pipe stands at 0.47: few warps (126 registers) between memory and the arithmetic.  fp32: 177
// and 260 us, 6.1 and 6.2 TB/s.
#include "block_common.cuh"

namespace mlstm {

namespace {

// A thread's channels: two packed pairs.  With eight the forward took 128 registers, 22 % of the SM's warps
// and 2.2 TB/s; with four it takes 70 and has 37 % of them.  The backward, with windows of x and dp and its
// sums, takes 126 (23 %) with four.
constexpr int kC = 4, kPairs = kC / 2;

// Channels c0 .. c0 + 3 of token t, where t < 0 is the carried state (or zero).
template <typename T, int W, bool WIDE>
__device__ __forceinline__ void load_input(const ConvArgs& a, const T* x, const T* st, int t, int n,
                                           float2* v) {
  Raw<T, kC> r;
  zero_raw(r);
  if (t >= 0)
    load_raw<WIDE>(x + t * a.x.st, r, n);
  else if (st != nullptr)
    load_raw<WIDE>(st + (long long)(t + W - 1) * a.D(), r, n);
  expand(r, v);
}

// The taps of a thread's channels, [W][pairs], and its biases.
template <int W, bool WIDE>
__device__ __forceinline__ void load_taps(const ConvArgs& a, int c0, int n, float2 (*w)[kPairs],
                                          float2* bias) {
  float f[kC * W];
  if (WIDE) {
#pragma unroll
    for (int i = 0; i < W; ++i)
      reinterpret_cast<float4*>(f)[i] = reinterpret_cast<const float4*>(a.w + (long long)c0 * W)[i];
  } else {
#pragma unroll
    for (int i = 0; i < kC * W; ++i) f[i] = i < n * W ? a.w[(long long)c0 * W + i] : 0.f;
  }
#pragma unroll
  for (int p = 0; p < kPairs; ++p) {
#pragma unroll
    for (int j = 0; j < W; ++j) w[j][p] = make_float2(f[2 * p * W + j], f[(2 * p + 1) * W + j]);
    bias[p] = make_float2(a.bias != nullptr && 2 * p < n ? a.bias[c0 + 2 * p] : 0.f,
                          a.bias != nullptr && 2 * p + 1 < n ? a.bias[c0 + 2 * p + 1] : 0.f);
  }
}

// Writes channels c0 .. c0 + n - 1 of a row whose channels lie in heads of d; `off` is c0's place.
template <typename T, bool WIDE>
__device__ __forceinline__ void store_heads(T* row, long long off, long long sh, int d, int c0, int n,
                                            const float2* v) {
  if (WIDE) {  // d is a multiple of 8, so the channels share a head
    store_pairs<true, kC>(row + off, v, n);
  } else {
#pragma unroll
    for (int i = 0; i < kC; ++i)
      if (i < n)
        row[((c0 + i) / d) * sh + (c0 + i) % d] = from_f32<T>(i & 1 ? v[i / 2].y : v[i / 2].x);
  }
}

template <int W, int ACT>
__device__ __forceinline__ void conv_token(const float2 (*w)[kPairs], const float2* bias,
                                           float2 (*win)[kPairs], const float2* x, float2* o) {
#pragma unroll
  for (int p = 0; p < kPairs; ++p) {
    float2 s = bias[p];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) s = fma2(w[j][p], win[j][p], s);
    s = fma2(w[W - 1][p], x[p], s);
    o[p] = act_pair<ACT>(s);
#pragma unroll
    for (int j = 0; j + 2 < W; ++j) win[j][p] = win[j + 1][p];
    win[W - 2][p] = x[p];
  }
}

// Tokens a thread has on their way from memory, in its own slots of shared memory, and how many of
// them it takes at a time.  Loads into registers left the memory idle while a batch was worked on
// (4.0 TB/s at B8 T4096 D4096 bf16); what lies in shared memory does not cost registers.
template <typename T> constexpr int kRing = sizeof(T) == 2 ? 16 : 8;
constexpr int kBatch = 4;

// A batch of tokens into slots that lie `apart` from each other; `left` tokens exist.
template <bool WIDE, typename T>
__device__ __forceinline__ void fetch_batch(Raw<T, kC>* to, int apart, const T* from, long long step, int n,
                                            int left) {
  if (WIDE || sizeof(T) == 4) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (u < left) fetch_raw<WIDE>(to + u * apart, from + u * step, n);
  } else {  // all loads before the first store, which might be to where they read from
    Raw<T, kC> r[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (u < left) load_raw<false>(from + u * step, r[u], n);
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (u < left) to[u * apart] = r[u];
  }
}

template <typename T, int W, int ACT, bool WIDE>
__global__ void __launch_bounds__(128, 7) conv_fwd_kernel(ConvArgs a, int run, int runs, int vecs) {
  constexpr int RING = kRing<T>;
  __shared__ Raw<T, kC> ring[RING][128];
  const long long item = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (item >= (long long)vecs * runs * a.B) return;
  const int c0 = (int)(item % vecs) * kC;
  const long long br = item / vecs;
  const int t0 = (int)(br % runs) * run, b = (int)(br / runs);
  const int D = a.D(), n = min(kC, D - c0);
  const T* x = (const T*)a.x.p + (long long)b * a.x.sb + c0;
  const T* st = a.state_in ? (const T*)a.state_in + (long long)b * (W - 1) * D + c0 : nullptr;
  T* y = (T*)a.y.p + (long long)b * a.y.sb;
  const long long off = (c0 / a.d) * a.y.sh + c0 % a.d;
  const int t1 = min(t0 + run, a.T);
  const T* src = x + t0 * a.x.st;  // of the next token to fetch
  int ahead = t0;
  auto fetch = [&](int slot) {
    fetch_batch<WIDE>(&ring[slot][threadIdx.x], 128, src, a.x.st, n, t1 - ahead);
    src += kBatch * a.x.st;
    ahead += kBatch;
    copies_commit();
  };
#pragma unroll
  for (int i = 0; i < RING; i += kBatch) fetch(i);
  float2 w[W][kPairs], bias[kPairs], win[W - 1][kPairs];
  load_taps<W, WIDE>(a, c0, n, w, bias);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) load_input<T, W, WIDE>(a, x, st, t0 - (W - 1) + j, n, win[j]);
  int slot = 0;
  T* dst = y + t0 * a.y.st;
  for (int tb = t0; tb < t1; tb += kBatch) {
    copies_wait<RING / kBatch - 1>();
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (tb + u < t1) {
        float2 v[kPairs], o[kPairs];
        expand(ring[slot + u][threadIdx.x], v);
        conv_token<W, ACT>(w, bias, win, v, o);
        store_heads<T, WIDE>(dst, off, a.y.sh, a.d, c0, n, o);
      }
      dst += a.y.st;
    }
    fetch(slot);
    slot = slot + kBatch == RING ? 0 : slot + kBatch;
  }
  if (a.state_out != nullptr && t1 == a.T) {  // the window is the last W - 1 inputs
    T* so = (T*)a.state_out + (long long)b * (W - 1) * D + c0;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) store_pairs<WIDE, kC>(so + (long long)j * D, win[j], n);
  }
}

// One token: each thread reads its channels' carried inputs before it writes them, so
// state_out may be state_in.
template <typename T, int W, int ACT, bool WIDE>
__global__ void __launch_bounds__(128) conv_step_kernel(ConvArgs a, int vecs) {
  const long long item = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (item >= (long long)vecs * a.B) return;
  const int c0 = (int)(item % vecs) * kC, b = (int)(item / vecs);
  const int D = a.D(), n = min(kC, D - c0);
  const T* st = (const T*)a.state_in + (long long)b * (W - 1) * D + c0;
  T* so = (T*)a.state_out + (long long)b * (W - 1) * D + c0;
  float2 w[W][kPairs], bias[kPairs], win[W - 1][kPairs], v[kPairs], o[kPairs];
  load_taps<W, WIDE>(a, c0, n, w, bias);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) load_input<T, W, WIDE>(a, nullptr, st, j - (W - 1), n, win[j]);
  load_input<T, W, WIDE>(a, (const T*)a.x.p + (long long)b * a.x.sb + c0, st, 0, n, v);
  conv_token<W, ACT>(w, bias, win, v, o);
  store_heads<T, WIDE>((T*)a.y.p + (long long)b * a.y.sb, (c0 / a.d) * a.y.sh + c0 % a.d, a.y.sh, a.d, c0,
                       n, o);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) store_pairs<WIDE, kC>(so + (long long)j * D, win[j], n);
}

constexpr int kBwdLanes = 32;  // channel vectors of a CTA
constexpr int kBwdRuns = 4;    // runs of a CTA, joined in shared memory

// Tokens of one thread's run: 256 (a run's first and last batches cost twice the others, and the halo
// is read twice), fewer while that leaves under eight CTAs an SM, but 8 at least.
int bwd_run(int B, int T, int D) {
  const long long cblocks = (D + kC * kBwdLanes - 1) / (kC * kBwdLanes);
  int run = 256;
  while (run > 8 && cblocks * (((long long)B * ((T + run - 1) / run) + kBwdRuns - 1) / kBwdRuns) < 8 * 148)
    run /= 2;
  return run;
}

// One thread's walk through its run: windows of W inputs and W values of dp, sums for the taps.
template <typename T, int W, int ACT, bool WIDE>
struct BwdWalk {
  float2 w[W][kPairs], bias[kPairs], win[W][kPairs], dp[W][kPairs], dw[W][kPairs], db[kPairs];

  // Takes a token in (x and dy); `own`: its sums are this run's.
  __device__ __forceinline__ void take(const float2* x, const float2* g, bool own) {
#pragma unroll
    for (int p = 0; p < kPairs; ++p) {
#pragma unroll
      for (int j = 0; j + 1 < W; ++j) {
        win[j][p] = win[j + 1][p];
        dp[j][p] = dp[j + 1][p];
      }
      win[W - 1][p] = x[p];
      float2 s = bias[p], val, slope;
#pragma unroll
      for (int j = 0; j < W; ++j) s = fma2(w[j][p], win[j][p], s);
      slope_pair<ACT>(s, &val, &slope);
      dp[W - 1][p] = mul2(g[p], slope);
      if (own) {
        db[p] = add2(db[p], dp[W - 1][p]);
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][p] = fma2(dp[W - 1][p], win[j][p], dw[j][p]);
      }
    }
  }
  // A token behind the end: nothing comes from it.
  __device__ __forceinline__ void skip() {
#pragma unroll
    for (int p = 0; p < kPairs; ++p) {
#pragma unroll
      for (int j = 0; j + 1 < W; ++j) dp[j][p] = dp[j + 1][p];
      dp[W - 1][p] = make_float2(0.f, 0.f);
    }
  }
  __device__ __forceinline__ void dx(float2* o) const {
#pragma unroll
    for (int p = 0; p < kPairs; ++p) {
      o[p] = mul2(w[0][p], dp[W - 1][p]);
#pragma unroll
      for (int j = 1; j < W; ++j) o[p] = fma2(w[j][p], dp[W - 1 - j][p], o[p]);
    }
  }
};

// A thread walks tokens t0 .. t0 + run + W - 2 of its channels: it recomputes pre at each,
// forms dp, and W - 1 tokens later emits dx, whose last term is then known.  The first run
// of a sequence also emits the carried state's gradient (tokens -(W - 1) .. -1).  Sums over
// tokens are taken for the run's own tokens only and joined over the CTA's runs, one row
// of partials per CTA.
template <typename T, int W, int ACT, bool WIDE>
__global__ void __launch_bounds__(kBwdLanes * kBwdRuns, 4) conv_bwd_kernel(ConvArgs a, int run, int runs,
                                                                          int vecs, int cblocks) {
  constexpr int RING = kRing<T>;
  __shared__ Raw<T, kC> ring[2][RING][kBwdLanes * kBwdRuns];  // x and dy on their way
  static_assert(sizeof(ring) >= kBwdRuns * (W + 1) * kC * kBwdLanes * sizeof(float), "the sums reuse it");
  float(*red)[W + 1][kC][kBwdLanes] = reinterpret_cast<float(*)[W + 1][kC][kBwdLanes]>(ring);
  const int lane = threadIdx.x, rr = threadIdx.y, tid = rr * kBwdLanes + lane;
  const int vec = (int)(blockIdx.x % cblocks) * kBwdLanes + lane;
  const long long row = blockIdx.x / cblocks;          // partial row of this CTA
  const long long br = row * kBwdRuns + rr;            // run of all batches
  const int D = a.D();
  BwdWalk<T, W, ACT, WIDE> k;
#pragma unroll
  for (int p = 0; p < kPairs; ++p) {
    k.db[p] = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < W; ++j) k.dw[j][p] = k.dp[j][p] = make_float2(0.f, 0.f);
  }
  if (vec < vecs && br < (long long)runs * a.B) {
    const int c0 = vec * kC, n = min(kC, D - c0);
    const int t0 = (int)(br % runs) * run, b = (int)(br / runs);
    const int t1 = min(t0 + run, a.T);
    const T* x = (const T*)a.x.p + (long long)b * a.x.sb + c0;
    const T* st = a.state_in ? (const T*)a.state_in + (long long)b * (W - 1) * D + c0 : nullptr;
    const T* dy = (const T*)a.y.p + (long long)b * a.y.sb;
    const long long off = (c0 / a.d) * a.y.sh + c0 % a.d;
    T* dx = (T*)a.dx.p + (long long)b * a.dx.sb + c0;
    load_taps<W, WIDE>(a, c0, n, k.w, k.bias);
    const int end = min(t1 + W - 1, a.T);  // tokens read: dx of t1 - 1 is complete at t1 + W - 2
    const T *sx = x + t0 * a.x.st, *sg = dy + t0 * a.y.st + off;
    long long place[kC];  // of each channel in a row of dy, where they are taken one by one
    if (!WIDE)
#pragma unroll
      for (int i = 0; i < kC; ++i) place[i] = ((c0 + i) / a.d) * a.y.sh + (c0 + i) % a.d;
    int ahead = t0;
    auto fetch = [&](int slot) {
      fetch_batch<WIDE>(&ring[0][slot][tid], kBwdLanes * kBwdRuns, sx, a.x.st, n, end - ahead);
      if (WIDE) {
        fetch_batch<true>(&ring[1][slot][tid], kBwdLanes * kBwdRuns, sg, a.y.st, n, end - ahead);
      } else {  // the channels may lie in several heads
        float2 v[kBatch][kPairs];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          if (ahead + u < end) {
            const T* row = sg - off + u * a.y.st;
#pragma unroll
            for (int p = 0; p < kPairs; ++p) {
              v[u][p].x = 2 * p < n ? to_f32(row[place[2 * p]]) : 0.f;
              v[u][p].y = 2 * p + 1 < n ? to_f32(row[place[2 * p + 1]]) : 0.f;
            }
          }
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u)  // exact: the values come from T
          if (ahead + u < end) store_pairs<true, kC>(reinterpret_cast<T*>(&ring[1][slot + u][tid]), v[u], kC);
      }
      sx += kBatch * a.x.st;
      sg += kBatch * a.y.st;
      ahead += kBatch;
      copies_commit();
    };
#pragma unroll
    for (int i = 0; i < RING; i += kBatch) fetch(i);
    // win[j] = x_{tau - (W - 1) + j}; one step before tau = t0 it holds tokens t0 - W .. t0 - 1,
    // of which the first is shifted out unread
#pragma unroll
    for (int j = 1; j < W; ++j) load_input<T, W, WIDE>(a, x, st, t0 - W + j, n, k.win[j]);
    const int emit0 = t0 == 0 ? -(W - 1) : t0;  // first token whose gradient this run writes
    auto emit = [&](int e) {                    // the token whose gradient is complete
      if (e < emit0) return;
      float2 o[kPairs];
      k.dx(o);
      const int r = e - a.T + W - 1;  // row of the final state that is token e
      if (a.dstate_out != nullptr && r >= 0) {
        Raw<T, kC> q;
        float2 g[kPairs];
        load_raw<WIDE>((const T*)a.dstate_out + ((long long)b * (W - 1) + r) * D + c0, q, n);
        expand(q, g);
#pragma unroll
        for (int p = 0; p < kPairs; ++p) o[p] = add2(o[p], g[p]);
      }
      if (e >= 0)
        store_pairs<WIDE, kC>(dx + e * a.dx.st, o, n);
      else if (a.dstate_in != nullptr)
        store_pairs<WIDE, kC>((T*)a.dstate_in + ((long long)b * (W - 1) + e + W - 1) * D + c0, o, n);
    };
    int slot = 0;
    for (int tb = t0; tb < t1 + W - 1; tb += kBatch) {
      copies_wait<RING / kBatch - 1>();
      if (tb >= t0 + W - 1 && tb + kBatch <= t1) {  // inside the run: every token is read, summed and emitted
        T* out = dx + (tb - (W - 1)) * a.dx.st;
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          float2 v[kPairs], g[kPairs];
          expand(ring[0][slot + u][tid], v);
          expand(ring[1][slot + u][tid], g);
          k.take(v, g, true);
          k.dx(v);
          store_pairs<WIDE, kC>(out, v, n);
          out += a.dx.st;
        }
      } else {
#pragma unroll 1
        for (int u = 0; u < kBatch; ++u) {
          const int t = tb + u;
          if (t < end) {
            float2 v[kPairs], g[kPairs];
            expand(ring[0][slot + u][tid], v);
            expand(ring[1][slot + u][tid], g);
            k.take(v, g, t < t1);
          } else {
            k.skip();
          }
          if (t < t1 + W - 1) emit(t - (W - 1));
        }
      }
      fetch(slot);
      slot = slot + kBatch == RING ? 0 : slot + kBatch;
    }
    copies_wait<0>();  // empty groups by now; the slots are reused below
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kC; ++i) {
    red[rr][W][i][lane] = i & 1 ? k.db[i / 2].y : k.db[i / 2].x;
#pragma unroll
    for (int j = 0; j < W; ++j) red[rr][j][i][lane] = i & 1 ? k.dw[j][i / 2].y : k.dw[j][i / 2].x;
  }
  __syncthreads();
  // [W + 1][channels] sums of this CTA, channels contiguous
  const int cbase = (int)(blockIdx.x % cblocks) * kBwdLanes * kC;
  for (int e = tid; e < (W + 1) * kBwdLanes * kC; e += kBwdLanes * kBwdRuns) {
    const int q = e / (kBwdLanes * kC), c = e % (kBwdLanes * kC);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kBwdRuns; ++i) s += red[i][q][c % kC][c / kC];
    if (cbase + c < D) a.partial[(row * (W + 1) + q) * D + cbase + c] = s;
  }
}

// Sums over the rows of partials, 32 row shares to a column joined in a fixed order.
__global__ void __launch_bounds__(1024) param_sums_kernel(const float* __restrict__ partial,
                                                          float* __restrict__ dw,
                                                          float* __restrict__ dbias, int rows, int D, int W) {
  __shared__ float red[32][33];
  const int lane = threadIdx.x & 31, part = threadIdx.x >> 5;
  const long long first = (long long)blockIdx.x * 32, cols = (long long)(W + 1) * D;
  float s = 0.f;
  if (first + lane < cols)
#pragma unroll 4
    for (int r = part; r < rows; r += 32) s += partial[(long long)r * cols + first + lane];
  red[part][lane] = s;
  __syncthreads();
  const long long col = first + part;  // a warp joins one column
  s = warp_sum(red[lane][part]);
  if (lane == 0 && col < cols) {
    const int j = (int)(col / D);
    const long long c = col % D;
    if (j < W) {
      if (dw != nullptr) dw[c * W + j] = s;
    } else if (dbias != nullptr) {
      dbias[c] = s;
    }
  }
}

template <typename T, int W, int ACT, bool WIDE>
cudaError_t fwd(const ConvArgs& a, cudaStream_t s) {
  const int vecs = (a.D() + kC - 1) / kC;
  // Runs of 256 tokens, shorter while that leaves under eight thousand warps (the GPU holds half of
  // them): few rows then spread over the GPU.
  int run = 256;
  while (run > 4 && (long long)vecs * a.B * ((a.T + run - 1) / run) < 8192 * 32) run /= 2;
  const int runs = (a.T + run - 1) / run;
  const long long items = (long long)vecs * runs * a.B;
  conv_fwd_kernel<T, W, ACT, WIDE><<<(unsigned)((items + 127) / 128), 128, 0, s>>>(a, run, runs, vecs);
  return cudaGetLastError();
}

template <typename T, int W, int ACT, bool WIDE>
cudaError_t step(const ConvArgs& a, cudaStream_t s) {
  const int vecs = (a.D() + kC - 1) / kC;
  const long long items = (long long)vecs * a.B;
  conv_step_kernel<T, W, ACT, WIDE><<<(unsigned)((items + 127) / 128), 128, 0, s>>>(a, vecs);
  return cudaGetLastError();
}

template <typename T, int W, int ACT, bool WIDE>
cudaError_t bwd(const ConvArgs& a, cudaStream_t s) {
  const int D = a.D(), vecs = (D + kC - 1) / kC, cblocks = (vecs + kBwdLanes - 1) / kBwdLanes;
  const int rows = conv_bwd_rows(a.B, a.T, D), run = bwd_run(a.B, a.T, D);
  conv_bwd_kernel<T, W, ACT, WIDE>
      <<<(unsigned)((long long)rows * cblocks), dim3(kBwdLanes, kBwdRuns), 0, s>>>(
          a, run, (a.T + run - 1) / run, vecs, cblocks);
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

int conv_bwd_rows(int B, int T, int D) {
  const int run = bwd_run(B, T, D);
  return (int)(((long long)B * ((T + run - 1) / run) + kBwdRuns - 1) / kBwdRuns);
}

cudaError_t launch_param_sums(const float* partial, int rows, int D, int W, float* dw, float* dbias,
                              cudaStream_t s) {
  param_sums_kernel<<<(unsigned)(((long long)(W + 1) * D + 31) / 32), 1024, 0, s>>>(partial, dw, dbias,
                                                                                   rows, D, W);
  return cudaGetLastError();
}

cudaError_t launch_conv_fwd(const ConvArgs& a, cudaStream_t s) { return by_type<kFwd>(a, s); }
cudaError_t launch_conv_step(const ConvArgs& a, cudaStream_t s) { return by_type<kStep>(a, s); }
cudaError_t launch_conv_bwd(const ConvArgs& a, cudaStream_t s) { return by_type<kBwd>(a, s); }

}  // namespace mlstm

// Group norm of channels-last (or head-major) activations with an activation or
// an output gate, forward and backward.  With n = xhat w + bias over groups of d
// channels, xhat = (x - mean) rstd:
//
//   y = act(n)  or  y = n act(gate)
//   dn = dy act'(n)  or  dn = dy act(gate), dgate = dy n act'(gate)
//   dx = rstd (dn w - mean(dn w) - xhat mean(dn w xhat))   means over what x's mean is over
//   dw = sum dn xhat, dbias = sum dn                        over batches and tokens
//
// Bound by HBM.  Token scope (d <= 512, the widest head of the recurrence): 4 to 32 lanes hold
// one (token, group) row in registers, so every tensor moves once.  Sequence scope: a first
// pass writes each CTA's share of the sums and a second pass joins them and applies the norm.
// Means and variances are joined as (count, mean, sum of squared distances), never as a
// difference of squares.
#include "block_common.cuh"

namespace mlstm {

namespace {

constexpr int kThreads = 256;
constexpr int kSMs = 148;

// The activation of eight channels.  The choice is made once for all eight: a choice for each
// element cost more instructions than the norm itself.
__device__ __forceinline__ void act8(int act, float2* v) {
  if (act == kActSilu) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = act_pair<kActSilu>(v[i]);
  } else if (act == kActSigmoid) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = act_pair<kActSigmoid>(v[i]);
  }
}
// v becomes the value.
__device__ __forceinline__ void slope8(int act, float2* v, float2* slope) {
  if (act == kActSilu) {
#pragma unroll
    for (int i = 0; i < 4; ++i) slope_pair<kActSilu>(v[i], &v[i], &slope[i]);
  } else if (act == kActSigmoid) {
#pragma unroll
    for (int i = 0; i < 4; ++i) slope_pair<kActSigmoid>(v[i], &v[i], &slope[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) slope[i] = make_float2(1.f, 1.f);
  }
}

template <int LANES>
__device__ __forceinline__ float lanes_sum(float x) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Channels c .. c + n - 1 of the weight and bias (1 and 0 where there is none).
template <bool WIDE>
__device__ __forceinline__ void load_affine(const NormArgs& a, int c, int n, float2* w, float2* b) {
  float f[8], g[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    f[i] = 1.f;
    g[i] = 0.f;
  }
  if (a.w != nullptr && n > 0) load8<WIDE>(a.w + c, f, n);
  if (a.bias != nullptr && n > 0) load8<WIDE>(a.bias + c, g, n);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] = make_float2(f[2 * i], f[2 * i + 1]);
    b[i] = make_float2(g[2 * i], g[2 * i + 1]);
  }
}

// ---------------------------------------------------------------------------
// Token scope: LANES lanes to a row, K vectors of eight channels to a lane
// (LANES 8 K >= d).  A CTA stays with one head, so its weights stay in registers, and takes
// every gridDim-th block of tokens; heads are the fastest grid dimension, so CTAs that run
// together write neighbouring parts of the same tokens.
// ---------------------------------------------------------------------------

constexpr int kRowThreads = 128;

// A pointer that walks rows r, r + step, .. of [B, T] in a strided tensor (head and channel of the
// lane already added), dividing only where it leaves a sequence.
template <typename T>
struct RowPtr {
  T* base;
  T* p;
  long long sb, st, jump;
  int t;
  __device__ __forceinline__ RowPtr(const Rows& r, int head, int c, int row, int step, int len) {
    base = (T*)r.p + head * r.sh + c;
    sb = r.sb;
    st = r.st;
    jump = step * r.st;
    t = row % len;
    p = base + (row / len) * sb + t * st;
    b = row / len;
  }
  int b;
  __device__ __forceinline__ void advance(int step, int len) {
    t += step;
    p += jump;
    if (t >= len) {
      b += t / len;
      t %= len;
      p = base + b * sb + t * st;
    }
  }
};

// Rows that a lane has on their way from memory, in its own slots of shared memory (with the rows
// in registers the kernels waited on memory at 3.7 TB/s): as many as 44 KB hold, up to six.
template <typename T, int K, int TENSORS>
constexpr int kRowRing = 45056 / (kRowThreads * (K * TENSORS * 8 * (int)sizeof(T) + 8)) < 6
                             ? 45056 / (kRowThreads * (K * TENSORS * 8 * (int)sizeof(T) + 8))
                             : 6;

template <typename T, int LANES, int K, bool GATED, bool WIDE>
__global__ void __launch_bounds__(kRowThreads) norm_token_fwd_kernel(NormArgs a, int blocks) {
  constexpr int ROWS = kRowThreads / LANES, RING = kRowRing<T, K, 1 + GATED>;
  __shared__ Raw<T, 8> ring[RING][1 + GATED][K][kRowThreads];
  const int head = blockIdx.x % a.NH, lane = threadIdx.x % LANES, tid = threadIdx.x;
  const int tokens = a.B * a.T, d = a.d, step = blocks * ROWS;
  const int first = (blockIdx.x / a.NH) * ROWS, row = first + tid / LANES;
  const int c0 = lane * 8;  // vector k: channels c0 + k LANES 8
  int n[K];
  float2 w[K][4], bias[K][4];
  RowPtr<const T> px(a.x, head, c0, row, step, a.T), pg(a.gate, head, c0, row, step, a.T);
  RowPtr<T> py(a.y, head, c0, row, step, a.T);
  int ahead = row;
  auto fetch = [&](int slot) {
    if (ahead < tokens) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (n[k] > 0) {
          fetch_raw<WIDE>(&ring[slot][0][k][tid], px.p + k * LANES * 8, n[k]);
          if (GATED) fetch_raw<WIDE>(&ring[slot][GATED][k][tid], pg.p + k * LANES * 8, n[k]);
        }
      }
    }
    ahead += step;
    px.advance(step, a.T);
    if (GATED) pg.advance(step, a.T);
    copies_commit();
  };
#pragma unroll
  for (int k = 0; k < K; ++k) {
    n[k] = max(0, min(8, d - c0 - k * LANES * 8));
#pragma unroll
    for (int s = 0; s < RING; ++s)
      if (n[k] <= 0) zero_raw(ring[s][0][k][tid]);  // absent channels add nothing to the sums
  }
#pragma unroll
  for (int s = 0; s < RING; ++s) fetch(s);
#pragma unroll
  for (int k = 0; k < K; ++k)
    load_affine<WIDE>(a, head * d + c0 + k * LANES * 8, n[k], w[k], bias[k]);
  const float inv_d = 1.f / d;
  float2* stats = reinterpret_cast<float2*>(a.stats) + (long long)row * a.NH + head;
  int r = row, slot = 0;
  // whole warps stay in the loop together; rows past the end compute on what they hold, unstored
  for (int r0 = first; r0 < tokens; r0 += step) {
    copies_wait<RING - 1>();
    float2 v[K][4], g[K][4], s = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      expand(ring[slot][0][k][tid], v[k]);
      if (GATED) expand(ring[slot][GATED][k][tid], g[k]);
#pragma unroll
      for (int i = 0; i < 4; ++i) s = add2(s, v[k][i]);
    }
    fetch(slot);
    slot = slot + 1 == RING ? 0 : slot + 1;
    const float mean = lanes_sum<LANES>(s.x + s.y) * inv_d;
    const float2 neg = make_float2(-mean, -mean);
    s = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[k][i] = add2(v[k][i], neg);
        // channels that do not exist do not count
        if (WIDE ? n[k] > 0 : 2 * i + 1 < n[k])
          s = fma2(v[k][i], v[k][i], s);
        else if (2 * i < n[k])
          s.x = fmaf(v[k][i].x, v[k][i].x, s.x);
      }
    const float rstd = rsqrtf(fmaf(lanes_sum<LANES>(s.x + s.y), inv_d, a.eps));
    if (r < tokens) {
      const float2 rs = make_float2(rstd, rstd);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (n[k] > 0) {
#pragma unroll
          for (int i = 0; i < 4; ++i) v[k][i] = fma2(mul2(v[k][i], rs), w[k][i], bias[k][i]);
          if (GATED) {
            act8(a.act, g[k]);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[k][i] = mul2(v[k][i], g[k][i]);
          } else {
            act8(a.act, v[k]);
          }
          store_pairs<WIDE, 8>(py.p + k * LANES * 8, v[k], n[k]);
        }
      }
      if (a.stats != nullptr && lane == 0) *stats = make_float2(mean, rstd);
    }
    r += step;
    stats += (long long)step * a.NH;
    py.advance(step, a.T);
  }
}

// ws: rows of partial sums [blocks, 2, NH d] (dw, then dbias).
template <typename T, int LANES, int K, bool GATED, bool WIDE>
__global__ void __launch_bounds__(kRowThreads, K == 1 ? 4 : 2) norm_token_bwd_kernel(NormArgs a, int blocks) {
  constexpr int ROWS = kRowThreads / LANES, CH = LANES * K * 8, WARPS = kRowThreads / 32;
  constexpr int RING = kRowRing<T, K, 2 + GATED>;
  __shared__ union {
    struct {
      Raw<T, 8> raw[RING][2 + GATED][K][kRowThreads];
      float2 ms[RING][kRowThreads];
    } ring;
    float red[WARPS][2][CH];
  } sm;
  const int head = blockIdx.x % a.NH, block = blockIdx.x / a.NH, tid = threadIdx.x, lane = tid % LANES;
  const int tokens = a.B * a.T, d = a.d, step = blocks * ROWS;
  const int first = block * ROWS, row = first + tid / LANES, c0 = lane * 8;
  int n[K];
  float2 w[K][4], bias[K][4], dw[K][4], db[K][4];
  RowPtr<const T> px(a.x, head, c0, row, step, a.T), py(a.y, head, c0, row, step, a.T);
  RowPtr<const T> pg(a.gate, head, c0, row, step, a.T);
  RowPtr<T> pdx(a.dx, head, c0, row, step, a.T), pdg(a.dgate, head, c0, row, step, a.T);
  const float2* stats = reinterpret_cast<const float2*>(a.stats) + (long long)row * a.NH + head;
  int ahead = row;
  auto fetch = [&](int slot) {
    if (ahead < tokens) {
      copy_async<8>(&sm.ring.ms[slot][tid], stats);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (n[k] > 0) {
          fetch_raw<WIDE>(&sm.ring.raw[slot][0][k][tid], px.p + k * LANES * 8, n[k]);
          fetch_raw<WIDE>(&sm.ring.raw[slot][1][k][tid], py.p + k * LANES * 8, n[k]);
          if (GATED) fetch_raw<WIDE>(&sm.ring.raw[slot][1 + GATED][k][tid], pg.p + k * LANES * 8, n[k]);
        }
      }
    }
    ahead += step;
    stats += (long long)step * a.NH;
    px.advance(step, a.T);
    py.advance(step, a.T);
    if (GATED) pg.advance(step, a.T);
    copies_commit();
  };
#pragma unroll
  for (int k = 0; k < K; ++k) {
    n[k] = max(0, min(8, d - c0 - k * LANES * 8));
#pragma unroll
    for (int i = 0; i < 4; ++i) dw[k][i] = db[k][i] = make_float2(0.f, 0.f);
  }
#pragma unroll
  for (int s = 0; s < RING; ++s) fetch(s);
#pragma unroll
  for (int k = 0; k < K; ++k)
    load_affine<WIDE>(a, head * d + c0 + k * LANES * 8, n[k], w[k], bias[k]);
  const float inv_d = 1.f / d;
  int r = row, slot = 0;
  for (int r0 = first; r0 < tokens; r0 += step) {
    copies_wait<RING - 1>();
    const bool live = r < tokens;
    const float2 ms = sm.ring.ms[slot][tid];
    float2 v[K][4], q[K][4], s1 = make_float2(0.f, 0.f), s2 = s1;
    const float2 neg = make_float2(-ms.x, -ms.x), rs = make_float2(ms.y, ms.y);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float2 f[4], slope[4], nn[4], dg[4];  // f: the activation's argument, then its value
      expand(sm.ring.raw[slot][0][k][tid], v[k]);
      expand(sm.ring.raw[slot][1][k][tid], q[k]);
      if (GATED) expand(sm.ring.raw[slot][1 + GATED][k][tid], f);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[k][i] = mul2(add2(v[k][i], neg), rs);
        nn[i] = fma2(v[k][i], w[k][i], bias[k][i]);
        if (!GATED) f[i] = nn[i];
      }
      slope8(a.act, f, slope);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float2 dn = mul2(q[k][i], GATED ? f[i] : slope[i]);
        if (GATED) dg[i] = mul2(mul2(q[k][i], nn[i]), slope[i]);
        // nothing from rows or channels that do not exist
        if (!live || (WIDE ? n[k] <= 0 : 2 * i >= n[k])) dn.x = 0.f, v[k][i].x = 0.f;
        if (!live || (WIDE ? n[k] <= 0 : 2 * i + 1 >= n[k])) dn.y = 0.f, v[k][i].y = 0.f;
        dw[k][i] = fma2(dn, v[k][i], dw[k][i]);
        db[k][i] = add2(db[k][i], dn);
        q[k][i] = mul2(dn, w[k][i]);
        s1 = add2(s1, q[k][i]);
        s2 = fma2(q[k][i], v[k][i], s2);
      }
      if (GATED && live && n[k] > 0) store_pairs<WIDE, 8>(pdg.p + k * LANES * 8, dg, n[k]);
    }
    fetch(slot);
    slot = slot + 1 == RING ? 0 : slot + 1;
    const float m1 = lanes_sum<LANES>(s1.x + s1.y) * inv_d, m2 = lanes_sum<LANES>(s2.x + s2.y) * inv_d;
    if (live) {
      const float2 n1 = make_float2(-m1, -m1), n2 = make_float2(-m2, -m2);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (n[k] > 0) {
#pragma unroll
          for (int i = 0; i < 4; ++i) q[k][i] = mul2(rs, fma2(v[k][i], n2, add2(q[k][i], n1)));
          store_pairs<WIDE, 8>(pdx.p + k * LANES * 8, q[k], n[k]);
        }
      }
    }
    r += step;
    pdx.advance(step, a.T);
    if (GATED) pdg.advance(step, a.T);
  }
  if (a.dw == nullptr && a.dbias == nullptr) return;
  // the rows of a warp, then the warps, in a fixed order
  copies_wait<0>();
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float sw = i & 1 ? dw[k][i / 2].y : dw[k][i / 2].x, sb = i & 1 ? db[k][i / 2].y : db[k][i / 2].x;
#pragma unroll
      for (int o = LANES; o < 32; o <<= 1) {
        sw += __shfl_xor_sync(0xffffffffu, sw, o);
        sb += __shfl_xor_sync(0xffffffffu, sb, o);
      }
      if ((tid & 31) < LANES) {
        sm.red[tid / 32][0][c0 + k * LANES * 8 + i] = sw;
        sm.red[tid / 32][1][c0 + k * LANES * 8 + i] = sb;
      }
    }
  __syncthreads();
  const int D = a.NH * d;
  for (int e = tid; e < 2 * d; e += kRowThreads) {
    const int p = e / d, ch = e % d;
    float s = 0.f;
#pragma unroll
    for (int q = 0; q < WARPS; ++q) s += sm.red[q][p][ch];
    a.ws[((long long)block * 2 + p) * D + head * d + ch] = s;
  }
}

// ---------------------------------------------------------------------------
// Sequence scope.  A CTA takes one slab of tokens and one block of up to 2048 channels of a
// (batch, group): lanes along the channels, eight to a lane, and the CTA's other threads
// along tokens.
// ---------------------------------------------------------------------------

struct Spread {
  int lanes, rows;         // threads along channels / tokens of a CTA
  int slab, slabs;         // tokens of a CTA, CTAs along a sequence
  int cblocks;             // channel blocks of a group
  __host__ __device__ int parts() const { return slabs * cblocks; }
  long long ctas(int B, int NH) const { return (long long)B * NH * parts(); }
};

struct Cta {
  int b, head, part, slab, c0, n, t0, t1;  // n channels from c0 for this thread (0: idle)
  int row;                                   // thread's first token, relative to t0
};

__device__ __forceinline__ Cta cta_of(const NormArgs& a, const Spread& p) {
  Cta q;
  long long i = blockIdx.x;
  q.head = (int)(i % a.NH); i /= a.NH;
  q.part = (int)(i % p.parts());
  q.b = (int)(i / p.parts());
  q.slab = q.part / p.cblocks;
  q.c0 = (q.part % p.cblocks) * p.lanes * 8 + (threadIdx.x % p.lanes) * 8;
  q.n = max(0, min(8, a.d - q.c0));
  q.t0 = q.slab * p.slab;
  q.t1 = min(q.t0 + p.slab, a.T);
  q.row = threadIdx.x / p.lanes;
  return q;
}

// Offset of the thread's channels of token t in a strided tensor.
__device__ __forceinline__ long long at(const Rows& r, const Cta& q, int t) {
  return q.b * r.sb + t * r.st + q.head * r.sh + q.c0;
}

// Joins (count, mean, m2) pairs: Chan, Golub and LeVeque's pairwise update.
template <typename F>
__device__ __forceinline__ void join(F& n, F& mean, F& m2, F nb, F meanb, F m2b) {
  const F tot = n + nb;
  if (tot == F(0)) return;
  const F d = meanb - mean, f = nb / tot;
  mean += d * f;
  m2 += m2b + d * d * n * f;
  n = tot;
}

// Pass 1 of the forward: each CTA's (count, mean, m2) to ws[batch, head, part].
template <typename T, bool WIDE>
__global__ void __launch_bounds__(kThreads) norm_stats_kernel(NormArgs a, Spread p) {
  const Cta q = cta_of(a, p);
  float cnt = 0.f, mean = 0.f, m2 = 0.f;
  if (q.n > 0 && q.t0 + q.row < q.t1) {
    // A thread sums its distances from the mean of its first vector.  Were that vector far from the
    // rest, its own distances would make m2 as large: m2 loses at most a factor of the thread's
    // tokens in precision, whatever the values.
    const T* x = (const T*)a.x.p;
    Raw<T, 8> r;
    float2 v[4], s = make_float2(0.f, 0.f), e = s;
    load_raw<WIDE>(x + at(a.x, q, q.t0 + q.row), r, q.n);
    expand(r, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) s = add2(s, v[i]);
    const float pivot = (s.x + s.y) / q.n;
    const float2 neg = make_float2(-pivot, -pivot);
    s = e;
    int tokens = 0;
#pragma unroll 4
    for (int t = q.t0 + q.row; t < q.t1; t += p.rows) {
      load_raw<WIDE>(x + at(a.x, q, t), r, q.n);
      expand(r, v);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float2 d = add2(v[i], neg);
        if (!WIDE && 2 * i >= q.n) d.x = 0.f;
        if (!WIDE && 2 * i + 1 >= q.n) d.y = 0.f;
        s = add2(s, d);
        e = fma2(d, d, e);
      }
      ++tokens;
    }
    cnt = (float)tokens * q.n;
    const float off = (s.x + s.y) / cnt;
    mean = pivot + off;
    m2 = fmaxf((e.x + e.y) - off * (s.x + s.y), 0.f);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float nb = __shfl_down_sync(0xffffffffu, cnt, o), mb = __shfl_down_sync(0xffffffffu, mean, o),
                sb = __shfl_down_sync(0xffffffffu, m2, o);
    join(cnt, mean, m2, nb, mb, sb);
  }
  __shared__ float red[kThreads / 32][3];
  if ((threadIdx.x & 31) == 0) {
    red[threadIdx.x / 32][0] = cnt;
    red[threadIdx.x / 32][1] = mean;
    red[threadIdx.x / 32][2] = m2;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kThreads / 32; ++w) join(cnt, mean, m2, red[w][0], red[w][1], red[w][2]);
    float* o = a.ws + (((long long)q.b * a.NH + q.head) * p.parts() + q.part) * 3;
    o[0] = cnt;
    o[1] = mean;
    o[2] = m2;
  }
}

// Pass 2 of the forward: join the parts (every CTA for itself, in fp64), apply.
template <typename T, bool GATED, bool WIDE>
__global__ void __launch_bounds__(kThreads) norm_apply_kernel(NormArgs a, Spread p) {
  const Cta q = cta_of(a, p);
  __shared__ float sh[2];
  const long long group = (long long)q.b * a.NH + q.head;
  if (threadIdx.x < 32) {
    double cnt = 0, mean = 0, m2 = 0;
    const float* w = a.ws + group * p.parts() * 3;
    for (int i = threadIdx.x; i < p.parts(); i += 32)
      join(cnt, mean, m2, (double)w[3 * i], (double)w[3 * i + 1], (double)w[3 * i + 2]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double nb = __shfl_down_sync(0xffffffffu, cnt, o), mb = __shfl_down_sync(0xffffffffu, mean, o),
                   sb = __shfl_down_sync(0xffffffffu, m2, o);
      join(cnt, mean, m2, nb, mb, sb);
    }
    if (threadIdx.x == 0) {
      sh[0] = (float)mean;
      sh[1] = (float)(1.0 / sqrt(m2 / cnt + (double)a.eps));
      if (a.stats != nullptr && q.part == 0)
        reinterpret_cast<float2*>(a.stats)[group] = make_float2(sh[0], sh[1]);
    }
  }
  __syncthreads();
  if (q.n == 0) return;
  const float mean = sh[0], rstd = sh[1];
  float2 w[4], bias[4];
  load_affine<WIDE>(a, q.head * a.d + q.c0, q.n, w, bias);
  const float2 neg = make_float2(-mean, -mean), rs = make_float2(rstd, rstd);
  const T* x = (const T*)a.x.p;
#pragma unroll 4
  for (int t = q.t0 + q.row; t < q.t1; t += p.rows) {
    Raw<T, 8> xr, gr;
    float2 v[4], g[4];
    load_raw<WIDE>(x + at(a.x, q, t), xr, q.n);
    if (GATED) load_raw<WIDE>((const T*)a.gate.p + at(a.gate, q, t), gr, q.n);
    expand(xr, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = fma2(mul2(add2(v[i], neg), rs), w[i], bias[i]);
    if (GATED) {
      expand(gr, g);
      act8(a.act, g);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = mul2(v[i], g[i]);
    } else {
      act8(a.act, v);
    }
    store_pairs<WIDE, 8>((T*)a.y.p + at(a.y, q, t), v, q.n);
  }
}

// What one vector contributes to the backward: dn, xhat into v, dxh = dn w into q, dgate into f.
template <bool GATED>
__device__ __forceinline__ void dxhat8(int act, float2 neg, float2 rs, const float2* w, const float2* bias,
                                       float2* v, float2* q, float2* f, float2* dn) {
  float2 nn[4], slope[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = mul2(add2(v[i], neg), rs);
    nn[i] = fma2(v[i], w[i], bias[i]);
    if (!GATED) f[i] = nn[i];
  }
  slope8(act, f, slope);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    dn[i] = mul2(q[i], GATED ? f[i] : slope[i]);
    if (GATED) f[i] = mul2(mul2(q[i], nn[i]), slope[i]);
    q[i] = mul2(dn[i], w[i]);
  }
}

// Pass 1 of the backward: sums of dxh and dxh xhat to ws[batch, head, part, 2], and each
// channel's sums of dn xhat and dn to the rows [batch slabs, 2, NH d] behind them.
template <typename T, bool GATED, bool WIDE>
__global__ void __launch_bounds__(kThreads) norm_dsums_kernel(NormArgs a, Spread p, float* param) {
  extern __shared__ float cols[];  // [rows][2][lanes][8]
  const Cta q = cta_of(a, p);
  const long long group = (long long)q.b * a.NH + q.head;
  float2 s1 = make_float2(0.f, 0.f), s2 = s1, dw[4], db[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) dw[i] = db[i] = make_float2(0.f, 0.f);
  if (q.n > 0) {
    const float2 ms = reinterpret_cast<const float2*>(a.stats)[group];
    const float2 neg = make_float2(-ms.x, -ms.x), rs = make_float2(ms.y, ms.y);
    float2 w[4], bias[4];
    load_affine<WIDE>(a, q.head * a.d + q.c0, q.n, w, bias);
#pragma unroll 2
    for (int t = q.t0 + q.row; t < q.t1; t += p.rows) {
      Raw<T, 8> xr, yr, gr;
      float2 v[4], r[4], g[4], dn[4];
      load_raw<WIDE>((const T*)a.x.p + at(a.x, q, t), xr, q.n);
      load_raw<WIDE>((const T*)a.y.p + at(a.y, q, t), yr, q.n);
      if (GATED) load_raw<WIDE>((const T*)a.gate.p + at(a.gate, q, t), gr, q.n);
      expand(xr, v);
      expand(yr, r);
      if (GATED) expand(gr, g);
      dxhat8<GATED>(a.act, neg, rs, w, bias, v, r, g, dn);
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // absent channels have dy = 0 and so add nothing
        s1 = add2(s1, r[i]);
        s2 = fma2(r[i], v[i], s2);
        dw[i] = fma2(dn[i], v[i], dw[i]);
        db[i] = add2(db[i], dn[i]);
      }
    }
  }
  const int lane = threadIdx.x % p.lanes;
  if (param != nullptr) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      cols[((q.row * 2 + 0) * p.lanes + lane) * 8 + i] = i & 1 ? dw[i / 2].y : dw[i / 2].x;
      cols[((q.row * 2 + 1) * p.lanes + lane) * 8 + i] = i & 1 ? db[i / 2].y : db[i / 2].x;
    }
  }
  __shared__ float red[kThreads / 32][2];
  const float w1 = warp_sum(s1.x + s1.y), w2 = warp_sum(s2.x + s2.y);
  if ((threadIdx.x & 31) == 0) {
    red[threadIdx.x / 32][0] = w1;
    red[threadIdx.x / 32][1] = w2;
  }
  __syncthreads();
  if (threadIdx.x < 2) {
    float s = 0.f;
    for (int w = 0; w < kThreads / 32; ++w) s += red[w][threadIdx.x];
    a.ws[(group * p.parts() + q.part) * 2 + threadIdx.x] = s;
  }
  if (param != nullptr) {
    const int cb = (q.part % p.cblocks) * p.lanes * 8, width = p.lanes * 8, D = a.NH * a.d;
    float* out = param + ((long long)q.b * p.slabs + q.slab) * 2 * D + q.head * a.d + cb;
    for (int e = threadIdx.x; e < 2 * width; e += kThreads) {
      const int which = e / width, c = e % width;
      if (cb + c < a.d) {
        float s = 0.f;
        for (int r = 0; r < p.rows; ++r) s += cols[(r * 2 + which) * width + c];
        out[(long long)which * D + c] = s;
      }
    }
  }
}

// Pass 2 of the backward.
template <typename T, bool GATED, bool WIDE>
__global__ void __launch_bounds__(kThreads) norm_dx_kernel(NormArgs a, Spread p) {
  const Cta q = cta_of(a, p);
  __shared__ float sh[2];
  const long long group = (long long)q.b * a.NH + q.head;
  if (threadIdx.x < 32) {
    double s1 = 0, s2 = 0;
    const float* w = a.ws + group * p.parts() * 2;
    for (int i = threadIdx.x; i < p.parts(); i += 32) {
      s1 += w[2 * i];
      s2 += w[2 * i + 1];
    }
    s1 = warp_sum(s1);
    s2 = warp_sum(s2);
    if (threadIdx.x == 0) {
      const double inv = 1.0 / ((double)a.T * a.d);
      sh[0] = (float)(s1 * inv);
      sh[1] = (float)(s2 * inv);
    }
  }
  __syncthreads();
  if (q.n == 0) return;
  const float m1 = sh[0], m2 = sh[1];
  const float2 ms = reinterpret_cast<const float2*>(a.stats)[group];
  const float2 neg = make_float2(-ms.x, -ms.x), rs = make_float2(ms.y, ms.y);
  const float2 n1 = make_float2(-m1, -m1), n2 = make_float2(-m2, -m2);
  float2 w[4], bias[4];
  load_affine<WIDE>(a, q.head * a.d + q.c0, q.n, w, bias);
#pragma unroll 2
  for (int t = q.t0 + q.row; t < q.t1; t += p.rows) {
    Raw<T, 8> xr, yr, gr;
    float2 v[4], r[4], g[4], dn[4];
    load_raw<WIDE>((const T*)a.x.p + at(a.x, q, t), xr, q.n);
    load_raw<WIDE>((const T*)a.y.p + at(a.y, q, t), yr, q.n);
    if (GATED) load_raw<WIDE>((const T*)a.gate.p + at(a.gate, q, t), gr, q.n);
    expand(xr, v);
    expand(yr, r);
    if (GATED) expand(gr, g);
    dxhat8<GATED>(a.act, neg, rs, w, bias, v, r, g, dn);
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = mul2(rs, fma2(v[i], n2, add2(r[i], n1)));
    store_pairs<WIDE, 8>((T*)a.dx.p + at(a.dx, q, t), r, q.n);
    if (GATED) store_pairs<WIDE, 8>((T*)a.dgate.p + at(a.dgate, q, t), g, q.n);
  }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------

int lanes_for(int d) {
  const int v = (d + 7) / 8;
  return v <= 4 ? 4 : v <= 8 ? 8 : v <= 16 ? 16 : 32;
}

#ifndef FW
#define FW 16
#define BW 8
#endif
// Token blocks of the token-scope kernels: enough CTAs for `waves` per SM, no more than rows need.
int token_blocks(long long tokens, int NH, int d, int waves) {
  const int rows = kRowThreads / lanes_for(d);
  const long long need = (tokens + rows - 1) / rows;
  const long long want = ((long long)kSMs * waves + NH - 1) / NH;
  return (int)(need < want ? need : want);
}
constexpr int kFwdWaves = FW, kBwdWaves = BW;

Spread spread_for(int B, int T, int NH, int d) {
  Spread p;
  const int v = (d + 7) / 8;
  p.lanes = 1;
  while (p.lanes < v && p.lanes < kThreads) p.lanes *= 2;
  p.rows = kThreads / p.lanes;
  p.cblocks = (v + p.lanes - 1) / p.lanes;
  // Slabs of at least 8 tokens to a thread, more where that already gives 16 CTAs per SM.
  const long long groups = (long long)B * NH * p.cblocks;
  long long slabs = ((long long)kSMs * 16 + groups - 1) / groups;
  const long long most = (T + p.rows * 8 - 1) / (p.rows * 8);
  if (slabs > most) slabs = most;
  if (slabs < 1) slabs = 1;
  p.slab = (int)((T + slabs - 1) / slabs);
  p.slabs = (T + p.slab - 1) / p.slab;
  return p;
}

template <typename T, int LANES, int K>
cudaError_t token_fwd(const NormArgs& a, cudaStream_t s) {
  const int blocks = token_blocks((long long)a.B * a.T, a.NH, a.d, kFwdWaves);
  const unsigned grid = (unsigned)blocks * a.NH;
  if (a.gate.p != nullptr) {
    if (a.wide) norm_token_fwd_kernel<T, LANES, K, true, true><<<grid, kRowThreads, 0, s>>>(a, blocks);
    else norm_token_fwd_kernel<T, LANES, K, true, false><<<grid, kRowThreads, 0, s>>>(a, blocks);
  } else {
    if (a.wide) norm_token_fwd_kernel<T, LANES, K, false, true><<<grid, kRowThreads, 0, s>>>(a, blocks);
    else norm_token_fwd_kernel<T, LANES, K, false, false><<<grid, kRowThreads, 0, s>>>(a, blocks);
  }
  return cudaGetLastError();
}
template <typename T, int LANES, int K>
cudaError_t token_bwd(const NormArgs& a, cudaStream_t s) {
  const int blocks = token_blocks((long long)a.B * a.T, a.NH, a.d, kBwdWaves);
  const unsigned grid = (unsigned)blocks * a.NH;
  if (a.gate.p != nullptr) {
    if (a.wide) norm_token_bwd_kernel<T, LANES, K, true, true><<<grid, kRowThreads, 0, s>>>(a, blocks);
    else norm_token_bwd_kernel<T, LANES, K, true, false><<<grid, kRowThreads, 0, s>>>(a, blocks);
  } else {
    if (a.wide) norm_token_bwd_kernel<T, LANES, K, false, true><<<grid, kRowThreads, 0, s>>>(a, blocks);
    else norm_token_bwd_kernel<T, LANES, K, false, false><<<grid, kRowThreads, 0, s>>>(a, blocks);
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || (a.dw == nullptr && a.dbias == nullptr)) return e;
  return launch_param_sums(a.ws, blocks, a.NH * a.d, 1, a.dw, a.dbias, s);
}
template <typename T, bool BWD>
cudaError_t by_lanes(const NormArgs& a, cudaStream_t s) {
  const int lanes = lanes_for(a.d);
  if (lanes == 4) return BWD ? token_bwd<T, 4, 1>(a, s) : token_fwd<T, 4, 1>(a, s);
  if (lanes == 8) return BWD ? token_bwd<T, 8, 1>(a, s) : token_fwd<T, 8, 1>(a, s);
  if (lanes == 16) return BWD ? token_bwd<T, 16, 1>(a, s) : token_fwd<T, 16, 1>(a, s);
  if (a.d <= 256) return BWD ? token_bwd<T, 32, 1>(a, s) : token_fwd<T, 32, 1>(a, s);
  return BWD ? token_bwd<T, 32, 2>(a, s) : token_fwd<T, 32, 2>(a, s);
}

template <typename T, bool GATED, bool WIDE>
cudaError_t spread_fwd(const NormArgs& a, cudaStream_t s) {
  const Spread p = spread_for(a.B, a.T, a.NH, a.d);
  const unsigned grid = (unsigned)p.ctas(a.B, a.NH);
  norm_stats_kernel<T, WIDE><<<grid, kThreads, 0, s>>>(a, p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  norm_apply_kernel<T, GATED, WIDE><<<grid, kThreads, 0, s>>>(a, p);
  return cudaGetLastError();
}
template <typename T, bool GATED, bool WIDE>
cudaError_t spread_bwd(const NormArgs& a, cudaStream_t s) {
  const Spread p = spread_for(a.B, a.T, a.NH, a.d);
  const unsigned grid = (unsigned)p.ctas(a.B, a.NH);
  const bool params = a.dw != nullptr || a.dbias != nullptr;
  float* rows = params ? a.ws + p.ctas(a.B, a.NH) * 2 : nullptr;
  norm_dsums_kernel<T, GATED, WIDE><<<grid, kThreads, kThreads * 16 * sizeof(float), s>>>(a, p, rows);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  norm_dx_kernel<T, GATED, WIDE><<<grid, kThreads, 0, s>>>(a, p);
  e = cudaGetLastError();
  if (e != cudaSuccess || !params) return e;
  return launch_param_sums(rows, a.B * p.slabs, a.NH * a.d, 1, a.dw, a.dbias, s);
}
template <typename T, bool BWD>
cudaError_t spread_pass(const NormArgs& a, cudaStream_t s) {
  if (a.gate.p != nullptr) {
    if (a.wide) return BWD ? spread_bwd<T, true, true>(a, s) : spread_fwd<T, true, true>(a, s);
    return BWD ? spread_bwd<T, true, false>(a, s) : spread_fwd<T, true, false>(a, s);
  }
  if (a.wide) return BWD ? spread_bwd<T, false, true>(a, s) : spread_fwd<T, false, true>(a, s);
  return BWD ? spread_bwd<T, false, false>(a, s) : spread_fwd<T, false, false>(a, s);
}
template <bool BWD>
cudaError_t norm_pass(const NormArgs& a, cudaStream_t s) {
  if (a.scope == 0)
    return a.dtype == 0 ? by_lanes<bf16, BWD>(a, s) : by_lanes<float, BWD>(a, s);
  return a.dtype == 0 ? spread_pass<bf16, BWD>(a, s) : spread_pass<float, BWD>(a, s);
}

}  // namespace

size_t norm_workspace(int B, int T, int NH, int d, int scope, int, bool backward) {
  const size_t D = (size_t)NH * d;
  if (scope == 0)
    return backward ? (size_t)token_blocks((long long)B * T, NH, d, kBwdWaves) * 2 * D * 4 : 0;
  const Spread p = spread_for(B, T, NH, d);
  if (!backward) return (size_t)p.ctas(B, NH) * 3 * 4;
  return ((size_t)p.ctas(B, NH) * 2 + (size_t)B * p.slabs * 2 * D) * 4;
}

cudaError_t launch_norm_fwd(const NormArgs& a, cudaStream_t s) { return norm_pass<false>(a, s); }
cudaError_t launch_norm_bwd(const NormArgs& a, cudaStream_t s) { return norm_pass<true>(a, s); }

}  // namespace mlstm

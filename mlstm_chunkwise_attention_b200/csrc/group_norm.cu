// Group norm of channels-last (or head-major) activations with an activation or
// an output gate, forward and backward; here the statistics of single tokens, in
// norm_resident.cu and norm_sequence.cu those of whole sequences.  With n = xhat w + bias over groups of d
// channels, xhat = (x - mean) rstd:
//
//   y = act(n)  or  y = n act(gate)
//   dn = dy act'(n)  or  dn = dy act(gate), dgate = dy n act'(gate)
//   dx = rstd (dn w - mean(dn w) - xhat mean(dn w xhat))   means over what x's mean is over
//   dw = sum dn xhat, dbias = sum dn                        over batches and tokens
//
// Bound by HBM.  Token scope (d <= 512, the widest head of the recurrence): 4 to 32 lanes hold
// one (token, group) row in registers, so every tensor moves once.  Measured on one B200 at B8 NH32
// T4096 d128 bf16 with a sigmoid gate: forward 142 us, 5.7 TB/s or 0.87 of a plain copy; backward
// 232 us, 5.8 TB/s or 0.89.
#include "norm_common.cuh"

namespace mlstm {

namespace {

constexpr int kSMs = 148;

template <int LANES>
__device__ __forceinline__ float lanes_sum(float x) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
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
// launches
// ---------------------------------------------------------------------------

int lanes_for(int d) {
  const int v = (d + 7) / 8;
  return v <= 4 ? 4 : v <= 8 ? 8 : v <= 16 ? 16 : 32;
}

// Token blocks of the token-scope kernels: enough CTAs for `waves` per SM, no more than rows need.
int token_blocks(long long tokens, int NH, int d, int waves) {
  const int rows = kRowThreads / lanes_for(d);
  const long long need = (tokens + rows - 1) / rows;
  const long long want = (long long)kSMs * waves > NH ? (long long)kSMs * waves / NH : 1;
  return (int)(need < want ? need : want);
}
constexpr int kFwdWaves = 24, kBwdWaves = 8;

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

template <bool BWD>
cudaError_t norm_pass(const NormArgs& a, cudaStream_t s) {
  if (a.scope == 1) return launch_norm_sequence(a, BWD, s);
  return a.dtype == 0 ? by_lanes<bf16, BWD>(a, s) : by_lanes<float, BWD>(a, s);
}

}  // namespace

size_t norm_workspace(int B, int T, int NH, int d, int scope, int dtype, bool backward) {
  if (scope == 1) return norm_sequence_workspace(B, T, NH, d, dtype, backward);
  return backward ? (size_t)token_blocks((long long)B * T, NH, d, kBwdWaves) * 2 * NH * d * 4 : 0;
}

cudaError_t launch_norm_fwd(const NormArgs& a, cudaStream_t s) { return norm_pass<false>(a, s); }
cudaError_t launch_norm_bwd(const NormArgs& a, cudaStream_t s) { return norm_pass<true>(a, s); }

}  // namespace mlstm

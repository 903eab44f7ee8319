// Backward of the selective state space scan.  With s_t the state after token t, e_t =
// exp(delta_t A), dy_t the gradient of the ungated output and G the gradient that the state
// carries back (dstate_out after the last token):
//
//   g_t = G + dy_t C_t         dC_t = sum_c dy_t s_t         dB_t = sum_c delta_t x_t g_t
//   u_t = g_t e_t s_{t-1}      dA += u_t delta_t             G <- e_t g_t
//   ddelta_t = sum_n u_t A + x_t sum_n g_t B_t               dx_t = delta_t sum_n g_t B_t + skip dy_t
//
// The forward kept the state entering every eighth token, so eight tokens at a time are
// recomputed forwards into registers (e and s, 128 of them) and walked backwards: one ex2 per
// state and token.  A lane holds four states of two channels; sums over a channel's states
// run along LPC lanes, sums over channels along the others, both as transposing reductions,
// then over the CTA's warps in shared memory.  Each CTA writes its share of dB and dC; a
// second kernel adds the shares in a fixed order.
#include "scan_common.cuh"

namespace mlstm {

namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps, kTile = 16;

template <int LPC>
struct Cfg {
  static constexpr int NP = 4 * LPC;
  static constexpr int CL = 32 / LPC;         // channel lanes of a warp
  static constexpr int CT = kWarps * CL * 2;  // channels of a CTA
  static constexpr int VECS = CT / 8;
  static constexpr int ITEMS = (kTile * VECS + kThreads - 1) / kThreads;
  // shared memory, in floats: delta, delta x, dy [tile][CT]; sums over states [3][tile][CT];
  // B and C [tile][2 NP]; dB and dC of each warp [warps][tile][2 NP]; dskip and ddt_bias
  // shares of each thread's channels [16][threads]
  static constexpr int DT = 0, DTX = DT + kTile * CT, DY = DTX + kTile * CT, SUM = DY + kTile * CT,
                       BC = SUM + 3 * kTile * CT, RED = BC + kTile * 2 * NP,
                       ACC = RED + kWarps * kTile * 2 * NP, TOTAL = ACC + 16 * kThreads;
};

template <typename T, int LPC, bool GATE, bool WIDE>
__global__ void __launch_bounds__(kThreads) scan_bwd_kernel(ScanArgs a, int tiles) {
  using C = Cfg<LPC>;
  constexpr int NP = C::NP, CL = C::CL, CT = C::CT, VECS = C::VECS;
  extern __shared__ __align__(16) float sm[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32, nl = lane % LPC, cr = lane / LPC;
  const int cl = (warp * CL + cr) * 2;  // the lane's two channels within the tile
  const int b = blockIdx.x / (tiles * a.G), ti = blockIdx.x % (tiles * a.G);
  const ChannelTile q = channel_tile(a, ti, tiles, CT);
  const int NC = (a.T + kScanEvery - 1) / kScanEvery;
  float A2[2][4], G[2][4], dA[2][4];
#pragma unroll
  for (int e = 0; e < 2; ++e)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int n = nl * 4 + k;
      const bool on = cl + e < q.n && n < a.N;
      A2[e][k] = on ? a.A[(long long)(q.c0 + cl + e) * a.N + n] * kLog2e : 0.f;
      G[e][k] = on && a.dstate_out != nullptr
                    ? a.dstate_out[((long long)b * a.D + q.c0 + cl + e) * a.N + n]
                    : 0.f;
      dA[e][k] = 0.f;
    }
#pragma unroll
  for (int i = 0; i < 16; ++i) sm[C::ACC + i * kThreads + tid] = 0.f;
  const T* xp = (const T*)a.x.p + b * a.x.sb + q.c0;
  const T* dp = (const T*)a.dt.p + b * a.dt.sb + q.c0;
  const T* zp = GATE ? (const T*)a.z.p + b * a.z.sb + q.c0 : nullptr;
  const T* gp = (const T*)a.y.p + b * a.y.sb + q.c0;

  for (int t0 = (a.T - 1) / kTile * kTile; t0 >= 0; t0 -= kTile) {
#pragma unroll
    for (int m = 0; m < C::ITEMS; ++m) {
      const int item = tid + m * kThreads, t = item / VECS, cv = (item % VECS) * 8;
      if (item < kTile * VECS) {
        const int n = min(8, q.n - cv);
        const bool in = t0 + t < a.T && n > 0;
        float x[8], d[8], g[8], z[8];
        if (in) {
          load8<WIDE>(xp + (t0 + t) * a.x.st + cv, x, n);
          load8<WIDE>(dp + (t0 + t) * a.dt.st + cv, d, n);
          load8<WIDE>(gp + (t0 + t) * a.y.st + cv, g, n);
          if (GATE) load8<WIDE>(zp + (t0 + t) * a.z.st + cv, z, n);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float delta = 0.f, dx = 0.f, dy = 0.f;
          if (in && i < n) {
            delta = d[i] + (a.dt_bias != nullptr ? a.dt_bias[q.c0 + cv + i] : 0.f);
            if (a.softplus) delta = softplusf(delta);
            dx = delta * x[i];
            dy = GATE ? g[i] * act_value<kActSilu>(z[i]) : g[i];
          }
          sm[C::DT + t * CT + cv + i] = delta;
          sm[C::DTX + t * CT + cv + i] = dx;
          sm[C::DY + t * CT + cv + i] = dy;
        }
      }
    }
    stage_bc<T, NP, kTile>(a, b, q.g, t0, sm + C::BC, tid, kThreads);
    __syncthreads();
#pragma unroll 1
    for (int sub = kTile - kScanEvery; sub >= 0; sub -= kScanEvery) {
      if (t0 + sub >= a.T) continue;
      float h0[2][4], s[kScanEvery][2][4], ev[kScanEvery][2][4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (cl + e < q.n)
          v = *reinterpret_cast<const float4*>(
              a.saved + (((long long)b * NC + (t0 + sub) / kScanEvery) * a.D + q.c0 + cl + e) * NP + nl * 4);
        h0[e][0] = v.x; h0[e][1] = v.y; h0[e][2] = v.z; h0[e][3] = v.w;
      }
#pragma unroll
      for (int i = 0; i < kScanEvery; ++i) {
        const int t = sub + i;
        const float2 dt = *reinterpret_cast<const float2*>(sm + C::DT + t * CT + cl);
        const float2 dtx = *reinterpret_cast<const float2*>(sm + C::DTX + t * CT + cl);
        const float4 Bq = *reinterpret_cast<const float4*>(sm + C::BC + t * 2 * NP + nl * 4);
        const float Bv[4] = {Bq.x, Bq.y, Bq.z, Bq.w};
        const float dtv[2] = {dt.x, dt.y}, dxv[2] = {dtx.x, dtx.y};
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            ev[i][e][k] = exp2_fast(dtv[e] * A2[e][k]);
            s[i][e][k] = fmaf(ev[i][e][k], i == 0 ? h0[e][k] : s[i - 1][e][k], dxv[e] * Bv[k]);
          }
        if (GATE) {  // the ungated output, for dz
          const float4 Cq = *reinterpret_cast<const float4*>(sm + C::BC + t * 2 * NP + NP + nl * 4);
          float y[2];
#pragma unroll
          for (int e = 0; e < 2; ++e)
            y[e] = fmaf(s[i][e][0], Cq.x, fmaf(s[i][e][1], Cq.y, fmaf(s[i][e][2], Cq.z, s[i][e][3] * Cq.w)));
          scatter_sum<2, LPC, 1>(y, nl);
          if (nl % (LPC / 2) == 0) sm[C::SUM + (2 * kTile + t) * CT + cl + nl / (LPC / 2)] = y[0];
        }
      }
#pragma unroll
      for (int i = kScanEvery - 1; i >= 0; --i) {
        const int t = sub + i;
        const float2 dt = *reinterpret_cast<const float2*>(sm + C::DT + t * CT + cl);
        const float2 dtx = *reinterpret_cast<const float2*>(sm + C::DTX + t * CT + cl);
        const float2 dy = *reinterpret_cast<const float2*>(sm + C::DY + t * CT + cl);
        const float4 Bq = *reinterpret_cast<const float4*>(sm + C::BC + t * 2 * NP + nl * 4);
        const float4 Cq = *reinterpret_cast<const float4*>(sm + C::BC + t * 2 * NP + NP + nl * 4);
        const float Bv[4] = {Bq.x, Bq.y, Bq.z, Bq.w}, Cv[4] = {Cq.x, Cq.y, Cq.z, Cq.w};
        const float dtv[2] = {dt.x, dt.y}, dxv[2] = {dtx.x, dtx.y}, dyv[2] = {dy.x, dy.y};
        float bc[8], st[4] = {0.f, 0.f, 0.f, 0.f};  // dB, dC; sums of g B and of u A per channel
#pragma unroll
        for (int k = 0; k < 8; ++k) bc[k] = 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float g = fmaf(dyv[e], Cv[k], G[e][k]);
            bc[k] = fmaf(dxv[e], g, bc[k]);
            bc[4 + k] = fmaf(dyv[e], s[i][e][k], bc[4 + k]);
            st[e] = fmaf(g, Bv[k], st[e]);
            G[e][k] = ev[i][e][k] * g;
            const float u = G[e][k] * (i == 0 ? h0[e][k] : s[i - 1][e][k]);
            st[2 + e] = fmaf(u, A2[e][k], st[2 + e]);
            dA[e][k] = fmaf(u, dtv[e], dA[e][k]);
          }
        scatter_sum<4, LPC, 1>(st, nl);
        if constexpr (LPC == 2) {  // lane 0: both channels' g B; lane 1: their u A
          sm[C::SUM + (nl * kTile + t) * CT + cl] = st[0];
          sm[C::SUM + (nl * kTile + t) * CT + cl + 1] = st[1];
        } else if (nl % (LPC / 4) == 0) {
          const int v = nl / (LPC / 4);
          sm[C::SUM + ((v >> 1) * kTile + t) * CT + cl + (v & 1)] = st[0];
        }
        scatter_sum<8, CL, LPC>(bc, cr);
        float* red = sm + C::RED + (warp * kTile + t) * 2 * NP + nl * 4;
        if constexpr (CL >= 8) {
          if (cr % (CL / 8) == 0) {
            const int v = cr / (CL / 8);
            red[(v >> 2) * NP + (v & 3)] = bc[0];
          }
        } else {
#pragma unroll
          for (int k = 0; k < 8 / CL; ++k) {
            const int v = cr * (8 / CL) + k;
            red[(v >> 2) * NP + (v & 3)] = bc[k];
          }
        }
      }
    }
    __syncthreads();
    // the CTA's share of dB and dC
    for (int e = tid; e < kTile * 2 * NP; e += kThreads) {
      const int t = e / (2 * NP), r = e % (2 * NP);
      if (t0 + t < a.T) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v += sm[C::RED + (w * kTile + t) * 2 * NP + r];
        a.part_bc[((((long long)(ti % tiles) * a.B + b) * a.T + t0 + t) * a.G + q.g) * 2 * NP + r] = v;
      }
    }
#pragma unroll
    for (int m = 0; m < C::ITEMS; ++m) {
      const int item = tid + m * kThreads, t = item / VECS, cv = (item % VECS) * 8;
      const int n = min(8, q.n - cv);
      if (item < kTile * VECS && t0 + t < a.T && n > 0) {
        float x[8], d[8], g[8], z[8], o[8];
        load8<WIDE>(xp + (t0 + t) * a.x.st + cv, x, n);
        load8<WIDE>(dp + (t0 + t) * a.dt.st + cv, d, n);
        if (GATE) {
          load8<WIDE>(gp + (t0 + t) * a.y.st + cv, g, n);
          load8<WIDE>(zp + (t0 + t) * a.z.st + cv, z, n);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (i < n) {
            const int at = t * CT + cv + i, ch = q.c0 + cv + i;
            const float sgb = sm[C::SUM + at], sua = sm[C::SUM + kTile * CT + at] * kLn2;
            const float dy = sm[C::DY + at], delta = sm[C::DT + at];
            const float skip = a.skip != nullptr ? a.skip[ch] : 0.f;
            if (GATE) {
              const float y = fmaf(skip, x[i], sm[C::SUM + 2 * kTile * CT + at]);
              float val, slope;
              act_slope<kActSilu>(z[i], &val, &slope);
              z[i] = g[i] * y * slope;
            }
            float dd = fmaf(x[i], sgb, sua);
            if (a.softplus) dd *= sigmoidf(d[i] + (a.dt_bias != nullptr ? a.dt_bias[ch] : 0.f));
            sm[C::ACC + i * kThreads + tid] += dy * x[i];
            sm[C::ACC + (8 + i) * kThreads + tid] += dd;
            o[i] = fmaf(delta, sgb, skip * dy);
            d[i] = dd;
          }
        }
        store8<WIDE>((T*)a.dx.p + b * a.dx.sb + (t0 + t) * a.dx.st + q.c0 + cv, o, n);
        store8<WIDE>((T*)a.ddt.p + b * a.ddt.sb + (t0 + t) * a.ddt.st + q.c0 + cv, d, n);
        if (GATE) store8<WIDE>((T*)a.dz.p + b * a.dz.sb + (t0 + t) * a.dz.st + q.c0 + cv, z, n);
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int e = 0; e < 2; ++e)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int n = nl * 4 + k;
      if (cl + e < q.n && n < a.N) {
        const long long at = ((long long)b * a.D + q.c0 + cl + e) * a.N + n;
        a.part_a[at] = dA[e][k];
        if (a.dstate_in != nullptr) a.dstate_in[at] = G[e][k];
      }
    }
  // threads with the same channels: tid % VECS (a thread keeps its vector through all items)
  static_assert(kThreads % VECS == 0, "a thread's channels are the same in every item");
  __syncthreads();
  for (int e = tid; e < 2 * CT; e += kThreads) {
    const int which = e / CT, c = e % CT;
    if (c < q.n) {
      float v = 0.f;
      for (int w = c / 8; w < kThreads; w += VECS) v += sm[C::ACC + (which * 8 + c % 8) * kThreads + w];
      a.part_d[((long long)b * 2 + which) * a.D + q.c0 + c] = v;
    }
  }
}

// dB and dC: the sum of the channel tiles' shares.
template <typename T>
__global__ void __launch_bounds__(256) scan_bc_kernel(ScanArgs a, int tiles, int NP) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  const long long total = (long long)a.B * a.T * a.G * 2 * NP;
  if (i >= total) return;
  const int r = (int)(i % (2 * NP)), n = r % NP;
  if (n >= a.N) return;
  float v = 0.f;
#pragma unroll 8
  for (int k = 0; k < tiles; ++k) v += a.part_bc[k * total + i];
  const long long row = i / (2 * NP);
  const int g = (int)(row % a.G);
  const long long bt = row / a.G;
  const int t = (int)(bt % a.T), b = (int)(bt / a.T);
  const Rows& o = r >= NP ? a.dc : a.db;
  ((T*)o.p)[b * o.sb + t * o.st + g * o.sh + n] = from_f32<T>(v);
}

// dA: the sum of the batches' shares.
__global__ void __launch_bounds__(256) scan_da_kernel(const float* __restrict__ part, float* __restrict__ dA,
                                                      int B, long long count) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= count) return;
  float v = 0.f;
#pragma unroll 8
  for (int b = 0; b < B; ++b) v += part[b * count + i];
  dA[i] = v;
}

template <typename T, int LPC, bool GATE, bool WIDE>
cudaError_t bwd_kernel(const ScanArgs& a, int tiles, cudaStream_t s) {
  constexpr int bytes = Cfg<LPC>::TOTAL * sizeof(float);
  const cudaError_t e = cudaFuncSetAttribute(scan_bwd_kernel<T, LPC, GATE, WIDE>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  scan_bwd_kernel<T, LPC, GATE, WIDE>
      <<<(unsigned)((long long)a.B * a.G * tiles), kThreads, bytes, s>>>(a, tiles);
  return cudaGetLastError();
}

template <typename T, int LPC>
cudaError_t bwd(const ScanArgs& a, cudaStream_t s) {
  const int tiles = (a.D / a.G + Cfg<LPC>::CT - 1) / Cfg<LPC>::CT;
  cudaError_t e;
  if (a.z.p != nullptr)
    e = a.wide ? bwd_kernel<T, LPC, true, true>(a, tiles, s) : bwd_kernel<T, LPC, true, false>(a, tiles, s);
  else
    e = a.wide ? bwd_kernel<T, LPC, false, true>(a, tiles, s) : bwd_kernel<T, LPC, false, false>(a, tiles, s);
  if (e != cudaSuccess) return e;
  const long long total = (long long)a.B * a.T * a.G * 2 * Cfg<LPC>::NP;
  scan_bc_kernel<T><<<(unsigned)((total + 255) / 256), 256, 0, s>>>(a, tiles, Cfg<LPC>::NP);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const long long count = (long long)a.D * a.N;
  scan_da_kernel<<<(unsigned)((count + 255) / 256), 256, 0, s>>>(a.part_a, a.dA, a.B, count);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (a.dskip == nullptr && a.ddt_bias == nullptr) return cudaSuccess;
  return launch_param_sums(a.part_d, a.B, a.D, 1, a.dskip, a.ddt_bias, s);
}

template <typename T>
cudaError_t by_states(const ScanArgs& a, cudaStream_t s) {
  switch (scan_pad(a.N)) {
    case 8: return bwd<T, 2>(a, s);
    case 16: return bwd<T, 4>(a, s);
    case 32: return bwd<T, 8>(a, s);
    default: return bwd<T, 16>(a, s);
  }
}

}  // namespace

ScanBwdSizes scan_bwd_sizes(int B, int T, int D, int G, int N) {
  const int NP = scan_pad(N), CT = kWarps * 2 * 32 * 4 / NP;
  ScanBwdSizes z;
  z.tiles = (D / G + CT - 1) / CT;
  z.part_bc = (size_t)z.tiles * B * T * G * 2 * NP;
  z.part_a = (size_t)B * D * N;
  z.part_d = (size_t)B * 2 * D;
  return z;
}

cudaError_t launch_scan_bwd(const ScanArgs& a, cudaStream_t s) {
  return a.dtype == 0 ? by_states<bf16>(a, s) : by_states<float>(a, s);
}

}  // namespace mlstm

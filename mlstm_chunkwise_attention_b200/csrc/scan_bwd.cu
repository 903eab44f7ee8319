// Backward of the selective state space scan.  With s_t the state after token t, e_t =
// exp(delta_t A), dy_t the gradient of the ungated output and G the gradient that the state
// carries back (dstate_out after the last token):
//
//   g_t = G + dy_t C_t         dC_t = sum_c dy_t s_t         dB_t = sum_c delta_t x_t g_t
//   u_t = g_t e_t s_{t-1}      dA += u_t delta_t             G <- e_t g_t
//   ddelta_t = sum_n u_t A + x_t sum_n g_t B_t               dx_t = delta_t sum_n g_t B_t + skip dy_t
//
// The forward kept the state entering every eighth token, so eight tokens at a time are
// recomputed forwards into registers (s; e is computed again on the way back, since the
// exponentials' pipe has room and 64 registers do not) and walked backwards.  A lane holds four
// states of two channels; sums over a channel's states run along LPC lanes, sums over channels
// along the others, both as transposing reductions, then over the CTA's warps in shared memory.
// Each CTA writes its share of dB, dC and the parameters' gradients; a second kernel adds the shares in
// a fixed order.
//
// Measured on one B200 at B8 T4096 D4096 N16 bf16 with a gate: 2.44 ms, and 0.06 for the sums (268 MB
// of shares of dB and dC; they grow with N, 4.3 GB at N = 64); the exponentials alone would take 0.46.
// Shared memory hands over 0.65 of what it can, 0.51 of the cycles issue, with 12 warps an SM: no pipe is
// full, the warps are too few to cover latencies.  fp32, with two CTAs an SM: 2.99 ms.  With the decays
// kept in registers (two CTAs an SM) 3.43 ms; without segments in turn the 512 CTAs take two waves of 444.
#include "scan_common.cuh"

namespace mlstm {

namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps, kTile = 16;
// CTAs of an SM, by registers.  Shared memory holds three of 9 to 32 states in bf16 and of 17 to 32 in fp32;
// else two (more than 32 states; fp32 from 9 to 16; bf16 up to 8), or one (fp32 up to 8).  scan_cut counts
// three for all: there it makes more segments than run at once.
constexpr int kCtas = 3;
constexpr int kSlots = 148 * kCtas;
__device__ unsigned int g_scan_bwd_failures = 0;  // launches that gave up a wait
static_assert(kTile == 2 * kScanEvery, "two saved states to a tile");

template <typename T, int LPC>
struct Cfg {
  static constexpr int NP = 4 * LPC;
  static constexpr int CL = 32 / LPC;         // channel lanes of a warp
  static constexpr int CT = kWarps * CL * 2;  // channels of a CTA
  static constexpr int VECS = CT / 8, UNITS = kTile * VECS;
  static constexpr int ITEMS = (UNITS + kThreads - 1) / kThreads;  // units of a thread
  // A lane keeps its states in the order k ^ perm, perm from its channel rank, so that each step
  // of the sum over channels sends one half of what it holds and keeps the other without choosing;
  // B and C lie in one copy for each order.
  static constexpr int ORDER = kTile * 2 * NP + 8;  // floats of a copy, with 8 to spread the banks
  // shared memory, in floats: delta and delta x of the tile, dy of the tile; sums over states of g B,
  // u A and C s; B and C; dB and dC of each warp [warps][tile][2 NP]; dskip and ddt_bias shares of
  // each thread's channels [4][threads] of four; dt_bias and skip; the next saved state [2][threads] of
  // four floats; and the tile's x, dt, dy, z as they lie in memory
  static constexpr int DX = 0, DY = DX + UNITS * kPairUnit, SUM = DY + UNITS * kFloatUnit,
                       BC = SUM + 3 * UNITS * kFloatUnit, RED = BC + 4 * ORDER,
                       ACC = RED + kWarps * kTile * 2 * NP, BIAS = ACC + 16 * kThreads, SKIP = BIAS + CT,
                       SAVED = SKIP + CT, RAW = SAVED + 8 * kThreads,
                       TOTAL = RAW + 4 * UNITS * 8 * (int)sizeof(T) / 4;
};

template <typename T, int LPC, bool GATE, bool WIDE>
__global__ void __launch_bounds__(kThreads, kCtas) scan_bwd_kernel(ScanArgs a, int tiles) {
  using C = Cfg<T, LPC>;
  constexpr int NP = C::NP, CL = C::CL, CT = C::CT, VECS = C::VECS, UNITS = C::UNITS;
  extern __shared__ __align__(16) float sm[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32, nl = lane % LPC, cr = lane / LPC;
  const int cl = (warp * CL + cr) * 2;  // the lane's two channels within the tile
  const int swap = nl & 1;              // it takes them in this order: cl + swap, then the other
  const int perm = (cr & 1) * 2 + (CL >= 4 ? (cr >> 1) & 1 : 0);  // and state k ^ perm as its k-th
  const int ch[2] = {cl + swap, cl + 1 - swap};
  __shared__ int box[2];
  const int per_seg = a.B * a.G * tiles, NC = (a.T + kScanEvery - 1) / kScanEvery;
  for (bool once = true;; once = false) {
  const int work = next_item(a, blockIdx.x, once, per_seg * a.segs, box);
  if (work >= per_seg * a.segs) return;
  const int seg = a.segs - 1 - work / per_seg, bi = work % per_seg;
  const int b = bi / (tiles * a.G), ti = bi % (tiles * a.G);
  const ChannelTile q = channel_tile(a, ti, tiles, CT);
  const int first = seg * a.seg_len, last = min(first + a.seg_len, a.T);
  const bool handed = a.in_turn && seg < a.segs - 1;  // the segment behind hands its gradient on
  if (handed && !wait_turn(a, bi, a.segs - 1 - seg, &g_scan_bwd_failures, box + 1)) return;
  float2 A2[2][2], G[2][2], dA[2][2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    float av[4], gv[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int n = nl * 4 + (k ^ perm);
      const bool on = ch[e] < q.n && n < a.N;
      av[k] = on ? a.A[(long long)(q.c0 + ch[e]) * a.N + n] * kLog2e : kPadRate;
      gv[k] = on && a.dstate_out != nullptr
                  ? a.dstate_out[((long long)b * a.D + q.c0 + ch[e]) * a.N + n]
                  : 0.f;
    }
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      A2[e][p] = make_float2(av[2 * p], av[2 * p + 1]);
      G[e][p] = make_float2(gv[2 * p], gv[2 * p + 1]);
      dA[e][p] = make_float2(0.f, 0.f);
    }
    if (ch[e] < q.n && handed) {
      const float4 v = permuted(
          __ldcg(reinterpret_cast<const float4*>(a.seg_state + ((long long)b * a.D + q.c0 + ch[e]) * NP + nl * 4)),
          perm);
      G[e][0] = make_float2(v.x, v.y);
      G[e][1] = make_float2(v.z, v.w);
    } else if (ch[e] < q.n && !a.in_turn) {
      enter_segment<NP, true>(a, b, q.c0 + ch[e], nl, seg, A2[e], G[e], perm);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    reinterpret_cast<float4*>(sm + C::ACC)[i * kThreads + tid] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = tid; i < CT; i += kThreads) {
    sm[C::BIAS + i] = a.dt_bias != nullptr && i < q.n ? a.dt_bias[q.c0 + i] : 0.f;
    sm[C::SKIP + i] = a.skip != nullptr && i < q.n ? a.skip[q.c0 + i] : 0.f;
  }
  const T* in[4] = {(const T*)a.x.p + b * a.x.sb + q.c0, (const T*)a.dt.p + b * a.dt.sb + q.c0,
                    (const T*)a.y.p + b * a.y.sb + q.c0,
                    GATE ? (const T*)a.z.p + b * a.z.sb + q.c0 : nullptr};
  const long long stride[4] = {a.x.st, a.dt.st, a.y.st, a.z.st};
  const long long part_step = (long long)a.G * 2 * NP;
  float* part = a.part_bc + (((long long)(ti % tiles) * a.B + b) * a.T * a.G + q.g) * 2 * NP;
  auto raw = [&](int tensor, int item) {
    return reinterpret_cast<Raw<T, 8>*>(sm + C::RAW) + tensor * UNITS + item;
  };
  // A thread fetches and reads only its own units, so no barrier is needed for them.
  auto fetch = [&](int t0) {
#pragma unroll
    for (int m = 0; m < C::ITEMS; ++m) {
      const int item = tid + m * kThreads, t = t0 + item / VECS, cv = (item % VECS) * 8, n = q.n - cv;
      if (item < UNITS) {
#pragma unroll
        for (int k = 0; k < 3 + GATE; ++k) {
          Raw<T, 8>* to = raw(k, item);
          const T* from = in[k] + t * stride[k] + cv;
          if (t < last && n > 0) {
            fetch_raw<WIDE>(to, from, n);
            // the same units of the next tile, into L2
            if (WIDE && t - kTile >= first) prefetch_l2(from - kTile * stride[k]);
          } else {
            zero_raw(*to);
          }
        }
      }
    }
  };
  // The lane's states entering the eight tokens from t on; each thread reads its own slots.
  auto fetch_saved = [&](int t) {
    if (t < first || t >= last) return;
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (ch[e] < q.n)
        copy_async(sm + C::SAVED + (e * kThreads + tid) * 4,
                     a.saved + (((long long)b * NC + t / kScanEvery) * a.D + q.c0 + ch[e]) * NP + nl * 4);
  };
#pragma unroll
  for (int i = 0; i < 2; ++i)  // channels that do not exist keep a state of zero
    *reinterpret_cast<float4*>(sm + C::SAVED + (i * kThreads + tid) * 4) = make_float4(0.f, 0.f, 0.f, 0.f);
  // Where this is done moves the compiler's registers: for the gated form once before the loop took 2655 us,
  // every eight tokens 2502 (B8 T4096 D4096 N16 bf16); for the ungated 1136 and 1160 (T2048).
  auto finite_rates = [&] {
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int p = 0; p < 2; ++p) A2[e][p] = make_float2(finite_rate(A2[e][p].x), finite_rate(A2[e][p].y));
  };
  if (!GATE) finite_rates();
  const int top = (last - 1 - first) / kTile * kTile + first;
  // the upper eight tokens of the first tile may lie behind the end; then the lower come first
  fetch_saved(top + kScanEvery < last ? top + kScanEvery : top);
  __syncthreads();
  for (int t0 = top; t0 >= first; t0 -= kTile) {
    fetch(t0);
    copies_commit();
    stage_bc<T, NP, kTile, 4, C::ORDER>(a, b, q.g, t0, last, sm + C::BC, tid, kThreads);
    copies_wait<0>();
#pragma unroll
    for (int m = 0; m < C::ITEMS; ++m) {
      const int item = tid + m * kThreads, t = t0 + item / VECS, cv = (item % VECS) * 8, n = q.n - cv;
      if (item < UNITS) {
        stage_delta<T>(a, *raw(0, item), *raw(1, item), sm + C::BIAS + cv, t < last, n,
                       sm + C::DX + item * kPairUnit);
        float2 g[4], z[4];
        expand(*raw(2, item), g);
        if (GATE) {
          expand(*raw(3, item), z);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            g[i] = mul2(g[i], act_pair<kActSilu>(z[i]));
        }
        store_unit(sm + C::DY + item * kFloatUnit, g);
      }
    }
    __syncthreads();
#pragma unroll 1
    for (int sub = kTile - kScanEvery; sub >= 0; sub -= kScanEvery) {
      if (t0 + sub >= last) continue;
      copies_wait<0>();
      float2 h0[2][2], s[kScanEvery][2][2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float4 v = permuted(
            *reinterpret_cast<const float4*>(sm + C::SAVED + (e * kThreads + tid) * 4), perm);
        h0[e][0] = make_float2(v.x, v.y);
        h0[e][1] = make_float2(v.z, v.w);
      }
      fetch_saved(t0 + sub - kScanEvery);
      copies_commit();
      if (GATE) finite_rates();
      const float* bcs = sm + C::BC + perm * C::ORDER + sub * 2 * NP + nl * 4;
      const float* dxs[2] = {sm + C::DX + (sub * VECS + cl / 8) * kPairUnit + (ch[0] % 8) * 2,
                             sm + C::DX + (sub * VECS + cl / 8) * kPairUnit + (ch[1] % 8) * 2};
      const float* dys[2] = {sm + C::DY + (sub * VECS + cl / 8) * kFloatUnit + ch[0] % 8,
                             sm + C::DY + (sub * VECS + cl / 8) * kFloatUnit + ch[1] % 8};
      float* sums = sm + C::SUM + (sub * VECS + cl / 8) * kFloatUnit + ch[0] % 8;
#pragma unroll
      for (int i = 0; i < kScanEvery; ++i) {
        const float4 Bq = *reinterpret_cast<const float4*>(bcs + i * 2 * NP);
        const float2 Bv[2] = {make_float2(Bq.x, Bq.y), make_float2(Bq.z, Bq.w)};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float2 d = *reinterpret_cast<const float2*>(dxs[e] + i * VECS * kPairUnit);
          const float2 dd = make_float2(d.x, d.x), dx = make_float2(d.y, d.y);
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            s[i][e][p] = fma2(exp2_pair(mul2(dd, A2[e][p])), i == 0 ? h0[e][p] : s[i - 1][e][p], mul2(dx, Bv[p]));
          }
        }
      }
#pragma unroll
      for (int i = kScanEvery - 1; i >= 0; --i) {
        const float4 Bq = *reinterpret_cast<const float4*>(bcs + i * 2 * NP);
        const float4 Cq = *reinterpret_cast<const float4*>(bcs + i * 2 * NP + NP);
        const float2 Bv[2] = {make_float2(Bq.x, Bq.y), make_float2(Bq.z, Bq.w)};
        const float2 Cv[2] = {make_float2(Cq.x, Cq.y), make_float2(Cq.z, Cq.w)};
        float2 db[2], dc[2], gb[2], ua[2], cs[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float2 d = *reinterpret_cast<const float2*>(dxs[e] + i * VECS * kPairUnit);
          const float2 dd = make_float2(d.x, d.x), dx = make_float2(d.y, d.y);
          const float dy1 = dys[e][i * VECS * kFloatUnit];
          const float2 dy = make_float2(dy1, dy1);
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const float2 g = fma2(dy, Cv[p], G[e][p]);
            db[p] = e == 0 ? mul2(dx, g) : fma2(dx, g, db[p]);
            dc[p] = e == 0 ? mul2(dy, s[i][e][p]) : fma2(dy, s[i][e][p], dc[p]);
            if (GATE) cs[e] = p == 0 ? mul2(s[i][e][p], Cv[p]) : fma2(s[i][e][p], Cv[p], cs[e]);
            gb[e] = p == 0 ? mul2(g, Bv[p]) : fma2(g, Bv[p], gb[e]);
            G[e][p] = mul2(exp2_pair(mul2(dd, A2[e][p])), g);
            const float2 u = mul2(G[e][p], i == 0 ? h0[e][p] : s[i - 1][e][p]);
            ua[e] = p == 0 ? mul2(u, A2[e][p]) : fma2(u, A2[e][p], ua[e]);
            dA[e][p] = fma2(u, dd, dA[e][p]);
          }
        }
        // over the channel's lanes: the neighbour's first channel is this lane's second
        float sg = gb[0].x + gb[0].y, su = ua[0].x + ua[0].y;
        sg += __shfl_xor_sync(0xffffffffu, gb[1].x + gb[1].y, 1);
        su += __shfl_xor_sync(0xffffffffu, ua[1].x + ua[1].y, 1);
        if (GATE) {  // the ungated output, for dz
          float sy = cs[0].x + cs[0].y;
          sy += __shfl_xor_sync(0xffffffffu, cs[1].x + cs[1].y, 1);
#pragma unroll
          for (int o = 2; o < LPC; o <<= 1) sy += __shfl_xor_sync(0xffffffffu, sy, o);
          if (nl < 2) sums[(2 * UNITS + i * VECS) * kFloatUnit] = sy;
        }
        if constexpr (LPC == 2) {
          sums[i * VECS * kFloatUnit] = sg;
          sums[(UNITS + i * VECS) * kFloatUnit] = su;
        } else {  // lanes 0, 1 of a channel end with g B, lanes 2, 3 with u A
          const bool up = nl & 2;
          float v = (up ? su : sg) + __shfl_xor_sync(0xffffffffu, up ? sg : su, 2);
#pragma unroll
          for (int o = 4; o < LPC; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
          if (nl < 4) sums[((nl >> 1) * UNITS + i * VECS) * kFloatUnit] = v;
        }
        // over the warp's channels: rank bit 0 halves the states by pairs, bit 1 the pair, bit 2
        // chooses between dB and dC; what is sent is the partner's first half
        float2 rb = db[0], rc = dc[0];
        rb.x += __shfl_xor_sync(0xffffffffu, db[1].x, LPC);
        rb.y += __shfl_xor_sync(0xffffffffu, db[1].y, LPC);
        rc.x += __shfl_xor_sync(0xffffffffu, dc[1].x, LPC);
        rc.y += __shfl_xor_sync(0xffffffffu, dc[1].y, LPC);
        float* red = sm + C::RED + (warp * kTile + sub + i) * 2 * NP + nl * 4;
        if constexpr (CL == 2) {
          red[perm] = rb.x;
          red[perm ^ 1] = rb.y;
          red[NP + perm] = rc.x;
          red[NP + (perm ^ 1)] = rc.y;
        } else {
          rb.x += __shfl_xor_sync(0xffffffffu, rb.y, 2 * LPC);
          rc.x += __shfl_xor_sync(0xffffffffu, rc.y, 2 * LPC);
          if constexpr (CL == 4) {
            red[perm] = rb.x;
            red[NP + perm] = rc.x;
          } else {
            const bool up = cr & 4;
            float v = (up ? rc.x : rb.x) + __shfl_xor_sync(0xffffffffu, up ? rb.x : rc.x, 4 * LPC);
            if constexpr (CL == 16) v += __shfl_xor_sync(0xffffffffu, v, 8 * LPC);
            if (cr < 8) red[(up ? NP : 0) + perm] = v;
          }
        }
      }
    }
    __syncthreads();
    // the CTA's share of dB and dC, four states at a time
    for (int e = tid; e < kTile * NP / 2; e += kThreads) {
      const int t = e / (NP / 2), r = (e % (NP / 2)) * 4;
      if (t0 + t < last) {
        const float* red = sm + C::RED + t * 2 * NP + r;
        float2 v[2] = {};
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float4 f = *reinterpret_cast<const float4*>(red + w * kTile * 2 * NP);
          v[0] = add2(v[0], make_float2(f.x, f.y));
          v[1] = add2(v[1], make_float2(f.z, f.w));
        }
        *reinterpret_cast<float4*>(part + (t0 + t) * part_step + r) = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
      }
    }
#pragma unroll
    for (int m = 0; m < C::ITEMS; ++m) {
      const int item = tid + m * kThreads, t = t0 + item / VECS, cv = (item % VECS) * 8, n = q.n - cv;
      if (item < UNITS && t < last && n > 0) {
        float2 x[4], d[4], v[4], sgb[4], dy[4], o[4];
        expand(*raw(0, item), x);
        load_unit(sm + C::SUM + item * kFloatUnit, sgb);
        load_unit(sm + C::DY + item * kFloatUnit, dy);
        if (GATE) {
          float2 g[4], z[4], y[4];
          expand(*raw(2, item), g);
          expand(*raw(3, item), z);
          load_unit(sm + C::SUM + (2 * UNITS + item) * kFloatUnit, y);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float2 val, slope;
            slope_pair<kActSilu>(z[i], &val, &slope);
            if (a.skip != nullptr)
              y[i] = fma2(*reinterpret_cast<const float2*>(sm + C::SKIP + cv + 2 * i), x[i], y[i]);
            o[i] = mul2(mul2(g[i], y[i]), slope);
          }
          store_pairs<WIDE, 8>((T*)a.dz.p + b * a.dz.sb + t * a.dz.st + q.c0 + cv, o, n);
        }
        expand(*raw(1, item), d);
        load_unit(sm + C::SUM + (UNITS + item) * kFloatUnit, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 pair = reinterpret_cast<const float4*>(sm + C::DX + item * kPairUnit)[i];
          v[i] = fma2(v[i], make_float2(kLn2, kLn2), mul2(x[i], sgb[i]));
          if (a.softplus) {
            const float2 rw = add2(d[i], *reinterpret_cast<const float2*>(sm + C::BIAS + cv + 2 * i));
            v[i] = mul2(v[i], sigmoid_pair(rw));
          }
          o[i] = mul2(make_float2(pair.x, pair.z), sgb[i]);
          if (a.skip != nullptr)
            o[i] = fma2(*reinterpret_cast<const float2*>(sm + C::SKIP + cv + 2 * i), dy[i], o[i]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float4* acc = reinterpret_cast<float4*>(sm + C::ACC) + i * kThreads + tid;
          float4 k = acc[0], l = acc[2 * kThreads];
          k.x = fmaf(dy[2 * i].x, x[2 * i].x, k.x);
          k.y = fmaf(dy[2 * i].y, x[2 * i].y, k.y);
          k.z = fmaf(dy[2 * i + 1].x, x[2 * i + 1].x, k.z);
          k.w = fmaf(dy[2 * i + 1].y, x[2 * i + 1].y, k.w);
          l.x += v[2 * i].x;
          l.y += v[2 * i].y;
          l.z += v[2 * i + 1].x;
          l.w += v[2 * i + 1].y;
          acc[0] = k;
          acc[2 * kThreads] = l;
        }
        store_pairs<WIDE, 8>((T*)a.dx.p + b * a.dx.sb + t * a.dx.st + q.c0 + cv, o, n);
        store_pairs<WIDE, 8>((T*)a.ddt.p + b * a.ddt.sb + t * a.ddt.st + q.c0 + cv, v, n);
      }
    }
    __syncthreads();
  }
  const int row = seg * a.B + b;  // of the partial sums
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const float da[4] = {dA[e][0].x, dA[e][0].y, dA[e][1].x, dA[e][1].y};
    const float gs[4] = {G[e][0].x, G[e][0].y, G[e][1].x, G[e][1].y};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int n = nl * 4 + (k ^ perm);
      if (ch[e] < q.n && n < a.N) {
        const long long at = (long long)(q.c0 + ch[e]) * a.N + n, all = (long long)a.D * a.N;
        a.part_a[row * all + at] = da[k];
        if (seg == 0 && a.dstate_in != nullptr) a.dstate_in[b * all + at] = gs[k];
      }
    }
    if (a.in_turn && seg > 0 && ch[e] < q.n)
      __stcg(reinterpret_cast<float4*>(a.seg_state + ((long long)b * a.D + q.c0 + ch[e]) * NP + nl * 4),
             permuted(make_float4(gs[0], gs[1], gs[2], gs[3]), perm));
  }
  if (a.in_turn && seg > 0) pass_turn(a, bi);
  // threads with the same channels: tid % VECS (a thread keeps its vector through all items)
  static_assert(kThreads % VECS == 0, "a thread's channels are the same in every item");
  for (int e = tid; e < 2 * CT; e += kThreads) {
    const int which = e / CT, c = e % CT;
    if (c < q.n) {
      float v = 0.f;
      for (int w = c / 8; w < kThreads; w += VECS) v += sm[C::ACC + ((which * 2 + c % 8 / 4) * kThreads + w) * 4 + c % 4];
      a.part_d[((long long)row * 2 + which) * a.D + q.c0 + c] = v;
    }
  }
  }
}

// The sums of all shares, in a fixed order.  The first `columns` / 32 blocks add those of dA and, behind
// them, dskip and ddt_bias over batches and segments, eight threads to a column (one to a column waited
// for each row of few long sequences in turn); the others those of dB and dC over the channel tiles.
template <typename T>
__global__ void __launch_bounds__(256) scan_sums_kernel(ScanArgs a, int tiles, int NP, int rows, long long columns,
                                                        unsigned int column_blocks) {
  __shared__ float red[8][32];
  if (blockIdx.x < column_blocks) {
    const long long i = (long long)blockIdx.x * 32 + threadIdx.x % 32, all = (long long)a.D * a.N, j = i - all;
    const int part = threadIdx.x / 32;
    const float* from = j < 0 ? a.part_a + i : a.part_d + j;
    const long long step = j < 0 ? all : 2LL * a.D;
    float v = 0.f;
    if (i < columns)
#pragma unroll 8
      for (int r = part; r < rows; r += 8) v += from[r * step];
    red[part][threadIdx.x % 32] = v;
    __syncthreads();
    if (part == 0 && i < columns) {
      float* to = j < 0 ? a.dA + i : j < a.D ? a.dskip : a.ddt_bias;
#pragma unroll
      for (int k = 1; k < 8; ++k) v += red[k][threadIdx.x];
      if (to != nullptr) to[j < 0 ? 0 : j % a.D] = v;
    }
    return;
  }
  const long long i = (long long)(blockIdx.x - column_blocks) * 256 + threadIdx.x;
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

template <typename T, int LPC, bool GATE, bool WIDE>
cudaError_t bwd_kernel(const ScanArgs& a, int tiles, cudaStream_t s) {
  constexpr int bytes = Cfg<T, LPC>::TOTAL * sizeof(float);
  const cudaError_t e = cudaFuncSetAttribute(scan_bwd_kernel<T, LPC, GATE, WIDE>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  const long long items = (long long)a.B * a.G * tiles * a.segs;
  const long long grid = a.in_turn && items > kSlots ? kSlots : items;
  scan_bwd_kernel<T, LPC, GATE, WIDE><<<(unsigned)grid, kThreads, bytes, s>>>(a, tiles);
  return cudaGetLastError();
}

template <typename T, int LPC>
cudaError_t bwd(const ScanArgs& a, cudaStream_t s) {
  const int tiles = (a.D / a.G + Cfg<T, LPC>::CT - 1) / Cfg<T, LPC>::CT;
  cudaError_t e;
  if (a.segs > 1 && !a.in_turn && (e = launch_scan_reverse_segments(a, s)) != cudaSuccess) return e;
  if (a.z.p != nullptr)
    e = a.wide ? bwd_kernel<T, LPC, true, true>(a, tiles, s) : bwd_kernel<T, LPC, true, false>(a, tiles, s);
  else
    e = a.wide ? bwd_kernel<T, LPC, false, true>(a, tiles, s) : bwd_kernel<T, LPC, false, false>(a, tiles, s);
  if (e != cudaSuccess) return e;
  const long long total = (long long)a.B * a.T * a.G * 2 * Cfg<T, LPC>::NP;
  const long long columns = (long long)a.D * (a.N + (a.dskip != nullptr || a.ddt_bias != nullptr ? 2 : 0));
  const unsigned column_blocks = (unsigned)((columns + 31) / 32);
  scan_sums_kernel<T><<<column_blocks + (unsigned)((total + 255) / 256), 256, 0, s>>>(
      a, tiles, Cfg<T, LPC>::NP, a.B * a.segs, columns, column_blocks);
  return cudaGetLastError();
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

__global__ void selftest_kernel(unsigned int* words) { selftest_wait(words, &g_scan_bwd_failures); }

}  // namespace

ScanSegments scan_bwd_segments(int B, int T, int D, int G, int N) {
  const int CT = kWarps * 2 * 32 * 4 / scan_pad(N);
  return scan_cut(T, kTile, (long long)B * G * ((D / G + CT - 1) / CT), kSlots);
}

cudaError_t launch_scan_bwd_selftest(unsigned int* words, cudaStream_t s) {
  selftest_kernel<<<1, 1, 0, s>>>(words);
  return cudaGetLastError();
}
cudaError_t scan_bwd_flag(unsigned int** at) { return cudaGetSymbolAddress((void**)at, g_scan_bwd_failures); }

ScanBwdSizes scan_bwd_sizes(int B, int T, int D, int G, int N) {
  const int NP = scan_pad(N), CT = kWarps * 2 * 32 * 4 / NP;
  ScanBwdSizes z;
  z.tiles = (D / G + CT - 1) / CT;
  z.part_bc = (size_t)z.tiles * B * T * G * 2 * NP;
  const int segs = scan_bwd_segments(B, T, D, G, N).count;
  z.part_a = (size_t)segs * B * D * N;
  z.part_d = (size_t)segs * B * 2 * D;
  return z;
}

cudaError_t launch_scan_bwd(const ScanArgs& a, cudaStream_t s) {
  return a.dtype == 0 ? by_states<bf16>(a, s) : by_states<float>(a, s);
}

}  // namespace mlstm

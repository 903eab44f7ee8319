// Group norm with statistics over a whole sequence, for groups that a cluster of CTAs holds in its shared
// memory (the formulas are in group_norm.cu; norm_sequence.cu takes the larger ones).
//
// Every value is read from memory once: each CTA of the cluster brings its slab of tokens in, its warps
// sum it up, the warps' sums go to every CTA of the cluster through distributed shared memory, and after
// the cluster's barrier each warp joins them all and writes the outputs of what it holds.  No counters,
// no workspace for the statistics and no waiting on flags: what a small call costs is one reading, two
// barriers of the cluster and one writing.  It is bound by that latency while the clusters all run at
// once, above that by how much of its loads an SM hides behind the other CTAs it holds.
//
// Measured on one B200, forward / backward with the parameters' sums, in us: B1 T100 NH8 d64 bf16
// 3.9 / 6.0 (norm_sequence.cu 14.6 / 14.5), B3 T333 NH5 d67 fp32 5.8 / 9.0 (18.5 / 22.6), B8 T1024 NH32
// d128 bf16 42 / 86 (55 / 89), 0.50 / 0.36 of a copy of the tensors moved once.
//
// Means and variances are joined as (count, mean, sum of squared distances), never as a difference of
// squares, in a fixed order and in 64 bits.
#include "internal.h"
#include "norm_common.cuh"

namespace mlstm {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32, kMost = 8;  // kMost: CTAs of a cluster
constexpr int kStages = 4;  // commit groups of the first reading
constexpr int kFwdCtas = 3, kBwdCtas = 2;  // of an SM, as the registers allow
constexpr int kSms = 148;
// Dynamic shared memory of each of `ctas` CTAs on an SM: of its 228 KB, each takes one for the system and
// one for `sums`.
constexpr int share_of(int ctas) { return (228 / ctas - 2) * 1024; }
constexpr int kEach = 64;  // more tokens of a thread than ever fit: bounds the arithmetic below

// A CTA takes `slab` tokens of one group, `each` of them to a thread: lanes along the channels, eight to
// a lane, and its other threads along tokens.
struct Slabs {
  int lanes, rows;
  int ctas;   // of a cluster
  int slab, each;
};

constexpr int bytes_of(int each, int elem, bool gated, bool backward) {
  // the tensors' vectors, and in the backward the channels' sums [rows][2][lanes][8]
  return kThreads * (each * (1 + backward + gated) * 8 * elem + (backward ? 64 : 0));
}

// False for groups that norm_sequence.cu does faster: those that even eight CTAs hold only alone on their
// SM, which leaves nothing to run while they load, unless all clusters run at once.  At B8 T4096 NH32
// d128 bf16 the forward took 223 us here and 153 there, at B8 T4096 NH32 d64 the backward 226 and 159; with
// two CTAs on an SM, at B8 T6000 NH16 d64, the forward took 62 here and 72 there, and with 64 clusters'
// CTAs in all (B2 T4096 NH4 d128) 13 and 25.
bool slabs_for(int B, int T, int NH, int d, int elem, bool gated, bool backward, Slabs* p) {
  const int v = (d + 7) / 8;
  if (v > kThreads) return false;
  p->lanes = 1;
  while (p->lanes < v) p->lanes *= 2;
  p->rows = kThreads / p->lanes;
  const long long groups = (long long)B * NH;
  auto fits = [&](int bytes) {
    return p->each <= kEach && bytes_of(p->each, elem, gated, backward) <= bytes;
  };
  // The smallest cluster with as many CTAs to an SM as can be, and two to each SM in all.
  for (p->ctas = 1;; p->ctas *= 2) {
    p->slab = (T + p->ctas - 1) / p->ctas;
    p->each = (p->slab + p->rows - 1) / p->rows;
    if (p->ctas == kMost || p->each == 1) break;
    if (fits(share_of(backward ? kBwdCtas : kFwdCtas)) && groups * p->ctas >= 2 * kSms) break;
  }
  return fits(share_of(groups * p->ctas <= kSms ? 1 : 2));
}

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
// Stores v at the same place in the shared memory of CTA `rank` of the cluster.
__device__ __forceinline__ void store_at_peer(float4* here, int rank, float4 v) {
  uint32_t to;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(to)
               : "r"((uint32_t)__cvta_generic_to_shared(here)), "r"(rank));
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(to), "f"(v.x), "f"(v.y), "f"(v.z),
               "f"(v.w)
               : "memory");
}
__device__ __forceinline__ double warp_sum64(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <typename T, bool GATED, bool WIDE, bool BWD>
__global__ void __launch_bounds__(kThreads, BWD ? kBwdCtas : kFwdCtas)
    norm_resident_kernel(NormArgs a, Slabs p, float* param) {
  constexpr int TENSORS = 1 + BWD + GATED;
  constexpr bool LATE = GATED && !BWD;  // the gate is not needed before the outputs
  extern __shared__ __align__(16) unsigned char dynamic[];
  auto slots = reinterpret_cast<Raw<T, 8>(*)[TENSORS][kThreads]>(dynamic);  // x, then dy, then the gate
  float* cols = reinterpret_cast<float*>(dynamic + sizeof(Raw<T, 8>) * p.each * TENSORS * kThreads);
  __shared__ float4 sums[kMost * kWarps];  // of every warp of the cluster
  const int tid = threadIdx.x, warp = tid / 32, wl = tid & 31;
  const int group = blockIdx.x / p.ctas, rank = blockIdx.x % p.ctas;
  const int b = group / a.NH, head = group % a.NH;
  const int row = tid / p.lanes, lane = tid % p.lanes, c0 = lane * 8;
  const int n = max(0, min(8, a.d - c0));
  const int t0 = rank * p.slab + row;
  // this thread's tokens: t0, t0 + rows, ..; threads without channels have none
  const int behind = min((rank + 1) * p.slab, a.T);
  const int count = n > 0 && t0 < behind ? (behind - t0 + p.rows - 1) / p.rows : 0;
  cluster_arrive();  // the others may write here once this CTA runs
  auto at = [&](const Rows& r) { return b * r.sb + t0 * r.st + head * r.sh + c0; };
  {
    const T *x = (const T*)a.x.p + at(a.x), *dy = BWD ? (const T*)a.y.p + at(a.y) : nullptr,
            *gate = GATED ? (const T*)a.gate.p + at(a.gate) : nullptr;
    const long long sx = p.rows * a.x.st, sy = p.rows * a.y.st, sg = p.rows * a.gate.st;
    int u = 0;
#pragma unroll
    for (int j = 1; j <= kStages; ++j) {
      for (; u < min(p.each * j / kStages, count); ++u) {
        fetch_raw<WIDE>(&slots[u][0][tid], x + u * sx, n);
        if (BWD) fetch_raw<WIDE>(&slots[u][BWD][tid], dy + u * sy, n);
        if (GATED && !LATE) fetch_raw<WIDE>(&slots[u][TENSORS - 1][tid], gate + u * sg, n);
      }
      copies_commit();
    }
    if (LATE) {
      for (u = 0; u < count; ++u) fetch_raw<WIDE>(&slots[u][TENSORS - 1][tid], gate + u * sg, n);
      copies_commit();
    }
  }
  float2 wt[4], bias[4];
  load_affine<WIDE>(a, head * a.d + c0, n, wt, bias);
  const double inv = 1.0 / ((double)a.T * a.d);
  // work(u) for the tokens of the j-th commit group
  auto stage = [&](int j, auto&& work) {
    const int end = min(p.each * (j + 1) / kStages, count);
    for (int u = p.each * j / kStages; u < end; ++u) work(u);
  };
  auto stages = [&](auto&& work) {
    copies_wait<3 + LATE>();
    stage(0, work);
    copies_wait<2 + LATE>();
    stage(1, work);
    copies_wait<1 + LATE>();
    stage(2, work);
    copies_wait<LATE>();
    stage(3, work);
  };
  if constexpr (!BWD) {
    // A warp's own mean first, then the distances from it: what it reads twice is in shared memory.
    float2 s = make_float2(0.f, 0.f);
    stages([&](int u) {
      float2 v[4];
      expand(slots[u][0][tid], v);
      s = add2(s, add2(add2(v[0], v[1]), add2(v[2], v[3])));
    });
    const float cnt = (float)__reduce_add_sync(0xffffffffu, count * n);
    const float mean = cnt > 0.f ? warp_sum(s.x + s.y) / cnt : 0.f;
    const float2 neg = make_float2(-mean, -mean);
    float2 off = make_float2(0.f, 0.f), e = off;
    for (int u = 0; u < count; ++u) {
      float2 v[4];
      expand(slots[u][0][tid], v);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float2 d = add2(v[k], neg);
        if (!WIDE && 2 * k >= n) d.x = 0.f;
        if (!WIDE && 2 * k + 1 >= n) d.y = 0.f;
        off = add2(off, d);
        e = fma2(d, d, e);
      }
    }
    // the rounding of the mean, and what it added to the distances
    const float o = warp_sum(off.x + off.y), left = cnt > 0.f ? o / cnt : 0.f;
    const float m2 = fmaxf(warp_sum(e.x + e.y) - left * o, 0.f);
    cluster_wait();
    if (wl < p.ctas) store_at_peer(sums + rank * kWarps + warp, wl, make_float4(cnt, mean, left, m2));
  } else {
    const float2 ms = reinterpret_cast<const float2*>(a.stats)[group];
    const float2 neg = make_float2(-ms.x, -ms.x), rs = make_float2(ms.y, ms.y);
    float2 dw[4], db[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) dw[k] = db[k] = make_float2(0.f, 0.f);
    stages([&](int u) {
      float2 v[4], g[4], f[4], slope[4];
      expand(slots[u][0][tid], v);
      expand(slots[u][BWD][tid], g);
      if (GATED) expand(slots[u][TENSORS - 1][tid], f);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[k] = mul2(add2(v[k], neg), rs);
        if (!GATED) f[k] = fma2(v[k], wt[k], bias[k]);
      }
      slope8(a.act, f, slope);
      // Absent channels have dy = 0 and so add nothing.
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 dn = mul2(g[k], GATED ? f[k] : slope[k]);
        dw[k] = fma2(dn, v[k], dw[k]);
        db[k] = add2(db[k], dn);
      }
    });
    // the sums of dn w and dn w xhat are those of dn and dn xhat, each channel's times its weight
    float2 s1 = mul2(wt[0], db[0]), s2 = mul2(wt[0], dw[0]);
#pragma unroll
    for (int k = 1; k < 4; ++k) {
      s1 = fma2(wt[k], db[k], s1);
      s2 = fma2(wt[k], dw[k], s2);
    }
    const float w1 = warp_sum(s1.x + s1.y), w2 = warp_sum(s2.x + s2.y);
    if (param != nullptr) {  // each channel's sums over the CTA's tokens
      float4* c = reinterpret_cast<float4*>(cols + row * 2 * p.lanes * 8 + c0);
      c[0] = make_float4(dw[0].x, dw[0].y, dw[1].x, dw[1].y);
      c[1] = make_float4(dw[2].x, dw[2].y, dw[3].x, dw[3].y);
      c += p.lanes * 2;
      c[0] = make_float4(db[0].x, db[0].y, db[1].x, db[1].y);
      c[1] = make_float4(db[2].x, db[2].y, db[3].x, db[3].y);
    }
    cluster_wait();
    if (wl < p.ctas) store_at_peer(sums + rank * kWarps + warp, wl, make_float4(w1, w2, 0.f, 0.f));
  }
  cluster_arrive();
  copies_wait<0>();
  cluster_wait();
  const float4 none = make_float4(0.f, 0.f, 0.f, 0.f), q0 = wl < p.ctas * kWarps ? sums[wl] : none,
               q1 = wl + 32 < p.ctas * kWarps ? sums[wl + 32] : none;
  if constexpr (!BWD) {
    const double m0 = (double)q0.y + q0.z, m1 = (double)q1.y + q1.z;
    const double mean = warp_sum64(q0.x * m0 + q1.x * m1) * inv;
    const double d0 = m0 - mean, d1 = m1 - mean;
    const double m2 = warp_sum64(q0.w + q0.x * d0 * d0 + q1.w + q1.x * d1 * d1);
    const float2 r = make_float2((float)mean, (float)(1.0 / sqrt(m2 * inv + (double)a.eps)));
    if (a.stats != nullptr && rank == 0 && tid == 0) reinterpret_cast<float2*>(a.stats)[group] = r;
    const float2 neg = make_float2(-r.x, -r.x), rs = make_float2(r.y, r.y);
    T* y = (T*)a.y.p + at(a.y);
    for (int u = 0; u < count; ++u) {
      float2 v[4], g[4];
      expand(slots[u][0][tid], v);
      if (GATED) expand(slots[u][TENSORS - 1][tid], g);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = fma2(mul2(add2(v[k], neg), rs), wt[k], bias[k]);
      if (GATED) {
        act8(a.act, g);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = mul2(v[k], g[k]);
      } else {
        act8(a.act, v);
      }
      store_pairs<WIDE, 8, true>(y, v, n);
      y += p.rows * a.y.st;
    }
  } else {
    const float m1 = (float)(warp_sum64((double)q0.x + q1.x) * inv);
    const float m2 = (float)(warp_sum64((double)q0.y + q1.y) * inv);
    const float2 ms = reinterpret_cast<const float2*>(a.stats)[group];
    const float2 neg = make_float2(-ms.x, -ms.x), rs = make_float2(ms.y, ms.y);
    const float2 n1 = make_float2(-m1, -m1), n2 = make_float2(-m2, -m2);
    T* dx = (T*)a.dx.p + at(a.dx);
    T* dgate = GATED ? (T*)a.dgate.p + at(a.dgate) : nullptr;
    for (int u = 0; u < count; ++u) {
      float2 v[4], g[4], f[4], slope[4], nn[4];
      expand(slots[u][0][tid], v);
      expand(slots[u][BWD][tid], g);
      if (GATED) expand(slots[u][TENSORS - 1][tid], f);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[k] = mul2(add2(v[k], neg), rs);
        nn[k] = fma2(v[k], wt[k], bias[k]);
        if (!GATED) f[k] = nn[k];
      }
      slope8(a.act, f, slope);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 h = mul2(mul2(g[k], GATED ? f[k] : slope[k]), wt[k]);
        if (GATED) nn[k] = mul2(mul2(g[k], nn[k]), slope[k]);
        v[k] = mul2(rs, fma2(v[k], n2, add2(h, n1)));
      }
      store_pairs<WIDE, 8, true>(dx, v, n);
      if (GATED) store_pairs<WIDE, 8, true>(dgate, nn, n);
      dx += p.rows * a.dx.st;
      if (GATED) dgate += p.rows * a.dgate.st;
    }
    if (param != nullptr) {  // the barrier above made every thread's sums visible
      const int line = p.lanes * 8, D = a.NH * a.d;
      float* out = param + ((long long)b * p.ctas + rank) * 2 * D + head * a.d;
      for (int e = tid; e < 2 * line; e += kThreads) {
        const int which = e / line, ch = e % line;
        if (ch < a.d) {
          float s = 0.f;
#pragma unroll 8
          for (int k = 0; k < p.rows; ++k) s += cols[(k * 2 + which) * line + ch];
          out[(long long)which * D + ch] = s;
        }
      }
    }
  }
}

template <typename T, bool GATED, bool WIDE, bool BWD>
cudaError_t run(const NormArgs& a, const Slabs& p, cudaStream_t s) {
  const bool params = BWD && (a.dw != nullptr || a.dbias != nullptr);
  float* param = params ? a.ws : nullptr;
  auto* kernel = norm_resident_kernel<T, GATED, WIDE, BWD>;
  const int bytes = bytes_of(p.each, (int)sizeof(T), GATED, BWD);
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute cluster;
  cluster.id = cudaLaunchAttributeClusterDimension;
  cluster.val.clusterDim.x = p.ctas;
  cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.B * a.NH) * p.ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = s;
  cfg.attrs = &cluster;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kernel, a, p, param);
  if (e != cudaSuccess || !params) return e;
  return launch_param_sums(param, a.B * p.ctas, a.NH * a.d, 1, a.dw, a.dbias, s);
}
template <typename T, bool BWD>
cudaError_t by_kind(const NormArgs& a, const Slabs& p, cudaStream_t s) {
  if (a.gate.p != nullptr) return a.wide ? run<T, true, true, BWD>(a, p, s) : run<T, true, false, BWD>(a, p, s);
  return a.wide ? run<T, false, true, BWD>(a, p, s) : run<T, false, false, BWD>(a, p, s);
}

}  // namespace

bool norm_resident_workspace(int B, int T, int NH, int d, int dtype, bool gated, bool backward, size_t* bytes) {
  Slabs p;
  if (!slabs_for(B, T, NH, d, dtype == 0 ? 2 : 4, gated, backward, &p)) return false;
  *bytes = backward ? (size_t)B * p.ctas * 2 * NH * d * 4 : 0;
  return true;
}

bool launch_norm_resident(const NormArgs& a, bool backward, cudaStream_t s, cudaError_t* status) {
  Slabs p;
  if (!slabs_for(a.B, a.T, a.NH, a.d, a.dtype == 0 ? 2 : 4, a.gate.p != nullptr, backward, &p)) return false;
  if (backward)
    *status = a.dtype == 0 ? by_kind<bf16, true>(a, p, s) : by_kind<float, true>(a, p, s);
  else
    *status = a.dtype == 0 ? by_kind<bf16, false>(a, p, s) : by_kind<float, false>(a, p, s);
  return true;
}

}  // namespace mlstm

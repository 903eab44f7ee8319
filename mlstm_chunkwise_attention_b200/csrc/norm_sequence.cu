// Group norm with statistics over a whole sequence, forward and backward (the formulas are in
// group_norm.cu).
//
// Bound by HBM: the statistics need every value before the first output, so x (in the backward x and
// dy) is read twice, and a plain second pass reads it from memory again.  Here one persistent kernel
// works through a queue: the sums of one chunk of groups, then the next chunk's sums, then the first
// chunk's outputs, and so on, so that the second reading of a chunk finds it in L2 (two chunks and what
// is written between them stay far below its 126 MB).  CTAs take items from a counter in this order.
// An output item waits for its group's sums, all of which were taken earlier by CTAs that run, so some
// CTA can always go on; the wait is bounded like those of the tensor-core kernels.
//
// Means and variances are joined as (count, mean, sum of squared distances), never as a difference of
// squares, and in a fixed order whoever comes last.
#include "internal.h"
#include "norm_common.cuh"
#include "tc_common.cuh"

namespace mlstm {

namespace {

constexpr int kThreads = 256;
constexpr int slots_of(bool backward) { return 148 * (backward ? 2 : 3); }  // CTAs of the persistent grid
__device__ unsigned int g_norm_error = 0;  // epoch of the last launch that gave up a wait

// The problem's items.  A CTA takes a slab of tokens and a block of up to 2048 channels of a (batch,
// group): lanes along the channels, eight to a lane, and its other threads along tokens.
struct Plan {
  int lanes, rows;       // threads along channels / tokens
  int slab, slabs;       // tokens of an item, items along a sequence
  int cblocks;           // channel blocks of a group
  int groups;            // B NH
  int chunk, chunks;     // groups of a chunk
  __host__ __device__ int parts() const { return slabs * cblocks; }
  __host__ __device__ long long items() const { return 2LL * chunks * chunk * parts(); }
};

// Workspace: counters (next item; finished sums and readiness of each group, zero at the launch), each
// group's pair of results, each item's sums, and in the backward rows of parameter sums.
struct Layout {
  size_t zeroed, pair, part, param, total;  // bytes; the counters lie at 0
};

Plan plan_for(int B, int T, int NH, int d, bool backward) {
  const int slots = slots_of(backward);
  Plan p;
  const int v = (d + 7) / 8;
  p.lanes = 1;
  while (p.lanes < v && p.lanes < kThreads) p.lanes *= 2;
  p.rows = kThreads / p.lanes;
  p.cblocks = (v + p.lanes - 1) / p.lanes;
  p.groups = B * NH;
  // Eight tokens to a thread (32 KB of a bf16 tensor to an item), fewer where that leaves too few
  // items to fill the GPU.
  int each = 8;
  while (each > 1 && (long long)p.groups * p.cblocks * ((T + p.rows * each - 1) / (p.rows * each)) < slots)
    each /= 2;
  p.slab = p.rows * each;
  p.slabs = (T + p.slab - 1) / p.slab;
  // A chunk has at least as many items as CTAs, so that its sums are done when its outputs are taken.
  p.chunk = (slots + p.parts() - 1) / p.parts();
  if (p.chunk > p.groups) p.chunk = p.groups;
  p.chunks = (p.groups + p.chunk - 1) / p.chunk;
  p.chunk = (p.groups + p.chunks - 1) / p.chunks;
  return p;
}

Layout layout_for(const Plan& p, int B, int D, bool backward) {
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  Layout l;
  l.zeroed = ((size_t)p.groups * 2 + 1) * 4;
  l.pair = up(l.zeroed);
  l.part = up(l.pair + (size_t)p.groups * 8);
  l.param = up(l.part + (size_t)p.groups * p.parts() * 3 * 4);
  l.total = l.param + (backward ? (size_t)B * p.slabs * 2 * D * 4 : 0);
  return l;
}

struct Work {
  unsigned int *next, *done, *ready;
  float2* pair;  // [groups]: mean and 1 / deviation, or the two means of the backward
  float* part;   // [groups, parts, 3]
  float* param;  // [B, slabs, 2, NH d], or null
};

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

// One item of the queue, worked out by one thread for the CTA: the divisions of every thread cost as
// many instructions as the norm.
struct Item {
  int output;  // the second reading; -1: behind the end of the queue
  int group, b, head, part, slab, c0, t0, t1;  // group < 0: nothing to do
  __device__ __forceinline__ void set(const NormArgs& a, const Plan& p, unsigned int i) {
    output = -1;
    if (i >= (unsigned int)p.items()) return;
    const unsigned int block = (unsigned int)(p.chunk * p.parts()), k = i / block, r = i % block;
    // blocks in turn: sums 0, sums 1, outputs 0, sums 2, outputs 1, ..
    const unsigned int end = 2u * p.chunks - 1;
    output = k > 0 && (k == end || k % 2 == 0);
    const unsigned int c = k == 0 ? 0 : !output ? (k + 1) / 2 : k == end ? p.chunks - 1 : k / 2 - 1;
    group = (int)(c * p.chunk + r / p.parts());
    if (group >= p.groups) {
      group = -1;
      return;
    }
    part = (int)(r % p.parts());
    b = group / a.NH;
    head = group % a.NH;
    slab = part / p.cblocks;
    c0 = (part % p.cblocks) * p.lanes * 8;
    t0 = slab * p.slab;
    t1 = min(t0 + p.slab, a.T);
  }
  template <typename T>
  __device__ __forceinline__ T* at(const Rows& r, int row, int lane) const {
    return (T*)r.p + b * r.sb + (t0 + row) * r.st + head * r.sh + c0 + lane * 8;
  }
};

// Tokens that a thread has on their way from memory: as many as 64 KB hold, up to the eight of an item.
template <typename T, int TENSORS>
constexpr int kRing = 65536 / (kThreads * TENSORS * 8 * (int)sizeof(T)) < 8
                          ? 65536 / (kThreads * TENSORS * 8 * (int)sizeof(T))
                          : 8;

template <typename T, bool GATED, bool WIDE, bool BWD>
__global__ void __launch_bounds__(kThreads, BWD ? 2 : 3) norm_sequence_kernel(NormArgs a, Plan p, Work w,
                                                                            unsigned int epoch) {
  constexpr int TENSORS = 1 + BWD + GATED, RING = kRing<T, TENSORS>;
  extern __shared__ __align__(16) unsigned char dynamic[];
  // x, then dy, then the gate on their way; and in the backward the channels' sums [rows][2][lanes][8]
  auto ring = reinterpret_cast<Raw<T, 8>(*)[TENSORS][kThreads]>(dynamic);
  float* cols = reinterpret_cast<float*>(dynamic + sizeof(Raw<T, 8>) * RING * TENSORS * kThreads);
  __shared__ float red[kThreads / 32][3];
  __shared__ float2 result;
  __shared__ Item items[3];  // the one worked on, the one after it, and room for the next
  __shared__ int waited;
  const tc::Abort abort{&g_norm_error, epoch};
  const int tid = threadIdx.x, warp = tid / 32, row = tid / p.lanes, lane = tid % p.lanes;
  // -- fetching: one commit group to a token, and RING of them ahead --------------------------
  const T* src[3];
  const long long step[3] = {p.rows * a.x.st, p.rows * a.y.st, p.rows * a.gate.st};
  int ahead = 0, end = 0, width = 0, slot = 0;
  bool with_gate = false;
  auto fetch = [&](int to) {
    if (ahead < end && width > 0) {
      fetch_raw<WIDE>(&ring[to][0][tid], src[0], width);
      if (BWD) fetch_raw<WIDE>(&ring[to][BWD][tid], src[1], width);
      if (with_gate) fetch_raw<WIDE>(&ring[to][TENSORS - 1][tid], src[2], width);
    }
    ahead += p.rows;
    src[0] += step[0];
    if (BWD) src[1] += step[1];
    if (GATED) src[2] += step[2];
    copies_commit();
  };
  auto begin = [&](const Item& i) {  // the first tokens of an item, into the slots from `slot` on
    if (i.output < 0) return;
    ahead = i.t0 + row;
    end = i.group >= 0 ? i.t1 : 0;
    width = max(0, min(8, a.d - i.c0 - lane * 8));
    with_gate = GATED && (BWD || i.output);
    src[0] = i.template at<const T>(a.x, row, lane);
    if (BWD) src[1] = i.template at<const T>(a.y, row, lane);
    if (GATED) src[2] = i.template at<const T>(a.gate, row, lane);
    for (int k = 0, to = slot; k < RING; ++k, to = to + 1 == RING ? 0 : to + 1) fetch(to);
  };
  auto advance = [&]() {
    fetch(slot);
    slot = slot + 1 == RING ? 0 : slot + 1;
  };
  // Each CTA holds the item it works on and the one after it, whose first tokens it fetches early.  That
  // one may wait behind the first; but the earliest unfinished item of the queue never does, so it can
  // go on.
  if (tid == 0) {
    items[0].set(a, p, atomicAdd(w.next, 1u));
    items[1].set(a, p, atomicAdd(w.next, 1u));
  }
  __syncthreads();
  begin(items[0]);
  for (int at = 0;; at = at == 2 ? 0 : at + 1) {
    const Item& q = items[at];
    const Item& behind = items[at == 2 ? 0 : at + 1];
    if (q.output < 0) return;
    unsigned int after = 0;
    if (tid == 0) after = atomicAdd(w.next, 1u);
    const bool real = q.group >= 0;
    if (real) {
      const int n = max(0, min(8, a.d - q.c0 - lane * 8)), first = q.t0 + row;
      if (q.output) {
        if (tid == 0) {
          bool ok = true;
          const uint64_t began = tc::global_timer_ns();
          for (unsigned int i = 1;; ++i) {
            unsigned int v;
            asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(w.ready + q.group) : "memory");
            if (v != 0) break;
            if ((i & 63) == 0 && (abort.raised() || tc::global_timer_ns() - began > tc::kWaitTimeoutNs)) {
              abort.raise();
              ok = false;
              break;
            }
            __nanosleep(100);
          }
          waited = ok;
          result = __ldcg(w.pair + q.group);
        }
        __syncthreads();
        if (!waited) {
          copies_wait<0>();
          return;
        }
      }
      float2 wt[4], bias[4];
      load_affine<WIDE>(a, q.head * a.d + q.c0 + lane * 8, n, wt, bias);
      if constexpr (!BWD) {
        if (!q.output) {
          // -- forward, first reading: a thread sums its distances from the mean of its first
          // vector.  Were that vector far from the rest, its own distances would make m2 as large:
          // m2 loses at most a factor of the thread's tokens in precision, whatever the values.
          float cnt = 0.f, mean = 0.f, m2 = 0.f;
          if (n > 0 && first < q.t1) {
            float2 neg = make_float2(0.f, 0.f), s = neg, e = neg;
            int tokens = 0;
            for (int t = first; t < q.t1; t += p.rows) {
              copies_wait<RING - 1>();
              float2 v[4];
              expand(ring[slot][0][tid], v);
              if (tokens == 0) {
                float2 m = add2(add2(v[0], v[1]), add2(v[2], v[3]));
                m.x = -(m.x + m.y) / n;
                neg = make_float2(m.x, m.x);
              }
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                float2 d = add2(v[i], neg);
                if (!WIDE && 2 * i >= n) d.x = 0.f;
                if (!WIDE && 2 * i + 1 >= n) d.y = 0.f;
                s = add2(s, d);
                e = fma2(d, d, e);
              }
              ++tokens;
              advance();
            }
            cnt = (float)tokens * n;
            const float off = (s.x + s.y) / cnt;
            mean = off - neg.x;
            m2 = fmaxf((e.x + e.y) - off * (s.x + s.y), 0.f);
          }
          begin(behind);
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) {
            const float nb = __shfl_down_sync(0xffffffffu, cnt, o), mb = __shfl_down_sync(0xffffffffu, mean, o),
                        sb = __shfl_down_sync(0xffffffffu, m2, o);
            join(cnt, mean, m2, nb, mb, sb);
          }
          if ((tid & 31) == 0) {
            red[warp][0] = cnt;
            red[warp][1] = mean;
            red[warp][2] = m2;
          }
        } else {
          // -- forward, second reading
          const float2 neg = make_float2(-result.x, -result.x), rs = make_float2(result.y, result.y);
          T* dst = q.template at<T>(a.y, row, lane);
          for (int t = first; t < q.t1 && n > 0; t += p.rows) {
            copies_wait<RING - 1>();
            float2 v[4], g[4];
            expand(ring[slot][0][tid], v);
            if (GATED) expand(ring[slot][TENSORS - 1][tid], g);
            advance();
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = fma2(mul2(add2(v[i], neg), rs), wt[i], bias[i]);
            if (GATED) {
              act8(a.act, g);
#pragma unroll
              for (int i = 0; i < 4; ++i) v[i] = mul2(v[i], g[i]);
            } else {
              act8(a.act, v);
            }
            store_pairs<WIDE, 8, true>(dst, v, n);
            dst += p.rows * a.y.st;
          }
          begin(behind);
        }
      } else {
        const float2 ms = reinterpret_cast<const float2*>(a.stats)[q.group];
        const float2 neg = make_float2(-ms.x, -ms.x), rs = make_float2(ms.y, ms.y);
        const float2 n1 = make_float2(-result.x, -result.x), n2 = make_float2(-result.y, -result.y);
        float2 s1 = make_float2(0.f, 0.f), s2 = s1, dw[4], db[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) dw[i] = db[i] = make_float2(0.f, 0.f);
        T* ddx = q.template at<T>(a.dx, row, lane);
        T* ddg = GATED ? q.template at<T>(a.dgate, row, lane) : nullptr;
        for (int t = first; t < q.t1 && n > 0; t += p.rows) {
          copies_wait<RING - 1>();
          float2 v[4], r[4], f[4], slope[4], nn[4];  // f: the activation's argument, then its value
          expand(ring[slot][0][tid], v);
          expand(ring[slot][BWD][tid], r);
          if (GATED) expand(ring[slot][TENSORS - 1][tid], f);
          advance();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[i] = mul2(add2(v[i], neg), rs);
            nn[i] = fma2(v[i], wt[i], bias[i]);
            if (!GATED) f[i] = nn[i];
          }
          slope8(a.act, f, slope);
          if (!q.output) {
            // -- backward, first reading.  Absent channels have dy = 0 and so add nothing.
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 dn = mul2(r[i], GATED ? f[i] : slope[i]), g = mul2(dn, wt[i]);
              s1 = add2(s1, g);
              s2 = fma2(g, v[i], s2);
              dw[i] = fma2(dn, v[i], dw[i]);
              db[i] = add2(db[i], dn);
            }
          } else {
            // -- backward, second reading
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 g = mul2(mul2(r[i], GATED ? f[i] : slope[i]), wt[i]);
              if (GATED) nn[i] = mul2(mul2(r[i], nn[i]), slope[i]);
              v[i] = mul2(rs, fma2(v[i], n2, add2(g, n1)));
            }
            store_pairs<WIDE, 8, true>(ddx, v, n);
            ddx += p.rows * a.dx.st;
            if (GATED) {
              store_pairs<WIDE, 8, true>(ddg, nn, n);
              ddg += p.rows * a.dgate.st;
            }
          }
        }
        begin(behind);
        if (!q.output) {
          const float w1 = warp_sum(s1.x + s1.y), w2 = warp_sum(s2.x + s2.y);
          if ((tid & 31) == 0) {
            red[warp][0] = w1;
            red[warp][1] = w2;
          }
          if (w.param != nullptr) {  // each channel's sums over the item's tokens
            const int line = p.lanes * 8;
            reinterpret_cast<float4*>(cols + (row * 2 + 0) * line + lane * 8)[0] =
                make_float4(dw[0].x, dw[0].y, dw[1].x, dw[1].y);
            reinterpret_cast<float4*>(cols + (row * 2 + 0) * line + lane * 8)[1] =
                make_float4(dw[2].x, dw[2].y, dw[3].x, dw[3].y);
            reinterpret_cast<float4*>(cols + (row * 2 + 1) * line + lane * 8)[0] =
                make_float4(db[0].x, db[0].y, db[1].x, db[1].y);
            reinterpret_cast<float4*>(cols + (row * 2 + 1) * line + lane * 8)[1] =
                make_float4(db[2].x, db[2].y, db[3].x, db[3].y);
            __syncthreads();
            const int cb = q.c0, D = a.NH * a.d;
            float* out = w.param + ((long long)q.b * p.slabs + q.slab) * 2 * D + q.head * a.d + cb;
            for (int e = tid; e < 2 * line; e += kThreads) {
              const int which = e / line, c = e % line;
              if (cb + c < a.d) {
                float s = 0.f;
                for (int r = 0; r < p.rows; ++r) s += cols[(r * 2 + which) * line + c];
                out[(long long)which * D + c] = s;
              }
            }
          }
        }
      }
      if (!q.output) {
        // -- the item's sums, and the group's by whoever finishes it
        __syncthreads();
        if (warp == 0) {
          float* part = w.part + ((long long)q.group * p.parts() + q.part) * 3;
          unsigned int before = 0;
          if (tid == 0) {
            float s[3] = {red[0][0], red[0][1], BWD ? 0.f : red[0][2]};
            for (int i = 1; i < kThreads / 32; ++i) {
              if (BWD) {
                s[0] += red[i][0];
                s[1] += red[i][1];
              } else {
                join(s[0], s[1], s[2], red[i][0], red[i][1], red[i][2]);
              }
            }
            for (int i = 0; i < 3; ++i) __stcg(part + i, s[i]);
            __threadfence();
            before = atomicAdd(w.done + q.group, 1u);
          }
          before = __shfl_sync(0xffffffffu, before, 0);
          if (before == (unsigned int)p.parts() - 1) {
            __threadfence();
            double s0 = 0, s1 = 0, s2 = 0;
            const float* all = w.part + (long long)q.group * p.parts() * 3;
            for (int i = tid; i < p.parts(); i += 32) {
              const double v0 = __ldcg(all + 3 * i), v1 = __ldcg(all + 3 * i + 1), v2 = __ldcg(all + 3 * i + 2);
              if (BWD) {
                s0 += v0;
                s1 += v1;
              } else {
                join(s0, s1, s2, v0, v1, v2);
              }
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
              const double v0 = __shfl_down_sync(0xffffffffu, s0, o), v1 = __shfl_down_sync(0xffffffffu, s1, o),
                           v2 = __shfl_down_sync(0xffffffffu, s2, o);
              if (BWD) {
                s0 += v0;
                s1 += v1;
              } else {
                join(s0, s1, s2, v0, v1, v2);
              }
            }
            if (tid == 0) {
              float2 r;
              if (BWD) {
                const double inv = 1.0 / ((double)a.T * a.d);
                r = make_float2((float)(s0 * inv), (float)(s1 * inv));
              } else {
                r = make_float2((float)s1, (float)(1.0 / sqrt(s2 / s0 + (double)a.eps)));
                if (a.stats != nullptr) reinterpret_cast<float2*>(a.stats)[q.group] = r;
              }
              __stcg(w.pair + q.group, r);
              __threadfence();
              asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(w.ready + q.group) : "memory");
            }
          }
        }
      }
    }
    if (!real) begin(behind);
    // the slot of the item before this one, which nobody reads any more
    if (tid == 0) items[at == 0 ? 2 : at - 1].set(a, p, after);
    __syncthreads();
  }
}

template <typename T, bool GATED, bool WIDE, bool BWD>
cudaError_t run(const NormArgs& a, cudaStream_t s) {
  const Plan p = plan_for(a.B, a.T, a.NH, a.d, BWD);
  const Layout l = layout_for(p, a.B, a.NH * a.d, BWD);
  char* ws = (char*)a.ws;
  Work w;
  w.next = (unsigned int*)ws;
  w.done = w.next + 1;
  w.ready = w.done + p.groups;
  w.pair = (float2*)(ws + l.pair);
  w.part = (float*)(ws + l.part);
  const bool params = BWD && (a.dw != nullptr || a.dbias != nullptr);
  w.param = params ? (float*)(ws + l.param) : nullptr;
  cudaError_t e = cudaMemsetAsync(ws, 0, l.zeroed, s);
  if (e != cudaSuccess) return e;
  constexpr int tensors = 1 + BWD + GATED;
  constexpr int bytes = kThreads * (kRing<T, tensors> * tensors * 8 * (int)sizeof(T) + (BWD ? 64 : 0));
  e = cudaFuncSetAttribute(norm_sequence_kernel<T, GATED, WIDE, BWD>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  const long long items = p.items(), slots = slots_of(BWD);
  norm_sequence_kernel<T, GATED, WIDE, BWD>
      <<<(unsigned)(items < slots ? items : slots), kThreads, bytes, s>>>(a, p, w, next_epoch());
  e = cudaGetLastError();
  if (e != cudaSuccess || !params) return e;
  return launch_param_sums(w.param, a.B * p.slabs, a.NH * a.d, 1, a.dw, a.dbias, s);
}
template <typename T, bool BWD>
cudaError_t by_kind(const NormArgs& a, cudaStream_t s) {
  if (a.gate.p != nullptr) return a.wide ? run<T, true, true, BWD>(a, s) : run<T, true, false, BWD>(a, s);
  return a.wide ? run<T, false, true, BWD>(a, s) : run<T, false, false, BWD>(a, s);
}

}  // namespace

size_t norm_sequence_workspace(int B, int T, int NH, int d, bool backward) {
  return layout_for(plan_for(B, T, NH, d, backward), B, NH * d, backward).total;
}

cudaError_t launch_norm_sequence(const NormArgs& a, bool backward, cudaStream_t s) {
  if (backward) return a.dtype == 0 ? by_kind<bf16, true>(a, s) : by_kind<float, true>(a, s);
  return a.dtype == 0 ? by_kind<bf16, false>(a, s) : by_kind<float, false>(a, s);
}

cudaError_t fetch_norm_error(unsigned int* flag) {
  return cudaMemcpyFromSymbol(flag, g_norm_error, sizeof(unsigned int));
}

}  // namespace mlstm

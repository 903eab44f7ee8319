// Group norm with statistics over a whole sequence, forward and backward (the formulas are in
// group_norm.cu), for groups too large for a cluster's shared memory (norm_resident.cu).
//
// Bound by HBM: the statistics need every value before the first output, so x (in the backward x and
// dy) is read twice, and a plain second pass reads it from memory again.  Here one persistent kernel
// works through a queue: the sums of one chunk of groups, then the next chunk's sums, then the first
// chunk's outputs, and so on, so that the second reading of a chunk finds some of it in L2.  Between a
// chunk's two readings lie the next chunk's, and the last chunk's second reading and output: at T8192 d256
// bf16 (chunks of 448 items of 64 KB) about 117 MB, and the 126 MB of L2 served half of the forward's
// second readings and two thirds of the backward's (198 MB read for a tensor of 134, 357 for 268).  A
// single group larger than L2 is read from memory twice.  CTAs take items from a counter in this order.
// An output item waits for its group's sums, all of which were taken earlier by CTAs that run, so some
// CTA can always go on; the wait is bounded like those of the tensor-core kernels.
//
// Means and variances are joined as (count, mean, sum of squared distances), never as a difference of
// squares, and in a fixed order whoever comes last.
//
// Measured on one B200 at B4 T8192 NH16 d256 bf16 with SiLU: forward 144 us, backward 299 us (0.57 and
// 0.42 of a plain copy of the tensors moved once); one group of 268 MB (T32768 d4096): 214 and 450 us.  A
// second pass over memory took 165 and 324 us at its best; a chunk of half or twice as many items as CTAs
// 206 / 349 and 175 / 327 us (waits; L2).  The issue of instructions between the barriers takes 0.5 to 0.6
// of the cycles; the rest waits for the second readings that miss L2 and at the barriers.
#include "norm_common.cuh"

namespace mlstm {

namespace {

constexpr int kThreads = 256;
constexpr int slots_of(bool backward) { return 148 * (backward ? 2 : 3); }  // CTAs of the persistent grid
__device__ unsigned int g_norm_failures = 0;  // launches that gave up a wait

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

// Workspace: words that are zero at the launch (its abort word; the next item; finished sums and readiness
// of each group), each group's pair of results, each item's sums, and in the backward rows of parameter sums.
struct Layout {
  size_t zeroed, pair, part, param, total;  // bytes; the zeroed words lie at 0
};

// Tokens of an item that a thread takes, all of them on their way from memory at once: as many as 64 KB
// of shared memory hold.
constexpr int tokens_of(int n) { return n >= 16 ? 16 : n >= 8 ? 8 : n >= 4 ? 4 : n >= 2 ? 2 : 1; }
constexpr int each_of(int elem, int tensors) { return tokens_of(65536 / (kThreads * tensors * 8 * elem)); }

Plan plan_for(int B, int T, int NH, int d, int elem, bool gated, bool backward) {
  const int slots = slots_of(backward);
  Plan p;
  const int v = (d + 7) / 8;
  p.lanes = 1;
  while (p.lanes < v && p.lanes < kThreads) p.lanes *= 2;
  p.rows = kThreads / p.lanes;
  p.cblocks = (v + p.lanes - 1) / p.lanes;
  p.groups = B * NH;
  // As many tokens to a thread as its slots hold, fewer where that leaves too few items to fill the GPU.
  int each = each_of(elem, 1 + backward + gated);
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
  l.zeroed = ((size_t)p.groups * 2 + 2) * 4;
  l.pair = up(l.zeroed);
  l.part = up(l.pair + (size_t)p.groups * 8);
  l.param = up(l.part + (size_t)p.groups * p.parts() * 3 * 4);
  l.total = l.param + (backward ? (size_t)B * p.slabs * 2 * D * 4 : 0);
  return l;
}

struct Work {
  unsigned int *abort, *next, *done, *ready;
  float2* pair;  // [groups]: mean and 1 / deviation, or the two means of the backward
  float* part;   // [groups, parts, 3]
  float* param;  // [B, slabs, 2, NH d], or null
};

// Joins (count, mean, m2) pairs: Chan, Golub and LeVeque's pairwise update.  A side without values is left
// out: its mean says nothing, and the square of the distance to it may overflow (from 2^64 in fp32).
template <typename F>
__device__ __forceinline__ void join(F& n, F& mean, F& m2, F nb, F meanb, F m2b) {
  if (nb == F(0)) return;
  if (n == F(0)) {
    n = nb;
    mean = meanb;
    m2 = m2b;
    return;
  }
  const F tot = n + nb;
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

__device__ __forceinline__ void named_barrier(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Eight warps work on an item.  Meanwhile a ninth joins the sums of the item before it, and a tenth, the
// manager, takes and works out the item after the next one and looks whether the next one's sums are
// ready: each of these waits on memory about as long as the work on an item takes.  One barrier ends an
// item.
template <typename T, bool GATED, bool WIDE, bool BWD>
__global__ void __launch_bounds__(kThreads + 64, BWD ? 2 : 3)
    norm_sequence_kernel(NormArgs a, Plan p, Work w) {
  constexpr int TENSORS = 1 + BWD + GATED, EACH = each_of((int)sizeof(T), TENSORS), ALL = kThreads + 64;
  extern __shared__ __align__(16) unsigned char dynamic[];
  // x, then dy, then the gate on their way; and in the backward the channels' sums [rows][2][lanes][8]
  auto slots = reinterpret_cast<Raw<T, 8>(*)[TENSORS][kThreads]>(dynamic);
  float* cols = reinterpret_cast<float*>(dynamic + sizeof(Raw<T, 8>) * EACH * TENSORS * kThreads);
  __shared__ float red[2][kThreads / 32][3];
  __shared__ float2 result[2];
  __shared__ int ready[2];  // whether result is the item's, as seen a barrier before
  __shared__ int waited;    // how the wait of an item that was not ready ended
  __shared__ Item items[4];
  const int tid = threadIdx.x, warp = tid / 32;

  if (warp == kThreads / 32) {  // ---- the warp that joins sums --------------------------------
    const int lane = tid & 31;
    // Joins an item's sums, and those of its group if it is the last to finish.
    auto finish = [&](const Item& q, const float (*r)[3]) {
      float s[3] = {0.f, 0.f, 0.f};
      if (lane < kThreads / 32)
#pragma unroll
        for (int k = 0; k < 3; ++k) s[k] = r[lane][k];
#pragma unroll
      for (int o = kThreads / 64; o > 0; o >>= 1) {
        const float v0 = __shfl_down_sync(0xffffffffu, s[0], o), v1 = __shfl_down_sync(0xffffffffu, s[1], o),
                    v2 = __shfl_down_sync(0xffffffffu, s[2], o);
        if (BWD) {
          s[0] += v0;
          s[1] += v1;
        } else {
          join(s[0], s[1], s[2], v0, v1, v2);
        }
      }
      float* all = w.part + (long long)q.group * p.parts() * 3;
      unsigned int before = 0;
      if (lane == 0) {
#pragma unroll
        for (int k = 0; k < 3; ++k) __stcg(all + q.part * 3 + k, s[k]);
        __threadfence();
        before = atomicAdd(w.done + q.group, 1u);
      }
      before = __shfl_sync(0xffffffffu, before, 0);
      if (before != (unsigned int)p.parts() - 1) return;
      __threadfence();
      double s0 = 0, s1 = 0, s2 = 0;
      for (int i = lane; i < p.parts(); i += 32) {
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
      if (lane == 0) {
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
    };
    named_barrier(0, ALL);
    for (int i = 0;; ++i) {
      if (i > 0) {
        const Item& last = items[(i - 1) & 3];
        if (last.output == 0 && last.group >= 0) finish(last, red[(i - 1) & 1]);
      }
      const Item& q = items[i & 3];
      if (q.output < 0) return;
      if (q.output && q.group >= 0 && ready[i & 1] == 0) {
        named_barrier(1, ALL);
        if (waited == 0) return;
      }
      named_barrier(0, ALL);
    }
  }
  if (warp > kThreads / 32) {  // ---- the manager ---------------------------------------------
    const int lane = tid & 31;
    if (lane == 0) {
      items[0].set(a, p, atomicAdd(w.next, 1u));
      items[1].set(a, p, atomicAdd(w.next, 1u));
      ready[0] = 0;
    }
    __syncwarp();
    named_barrier(0, ALL);
    // A CTA holds items behind the one it works on, which may wait; but the earliest unfinished item of
    // the queue is never among them, so it can go on.
    for (int i = 0;; ++i) {
      const Item& q = items[i & 3];
      if (q.output < 0) return;
      if (q.output && q.group >= 0 && ready[i & 1] == 0) {
        if (lane == 0) {
          const bool ok = wait_at_least(w.ready + q.group, 1, LaunchAbort{w.abort, &g_norm_failures}, 100);
          result[i & 1] = __ldcg(w.pair + q.group);
          waited = ok;
        }
        __syncwarp();
        named_barrier(1, ALL);
        if (waited == 0) return;
      }
      if (lane == 0) {
        items[(i + 2) & 3].set(a, p, atomicAdd(w.next, 1u));
        const Item& next = items[(i + 1) & 3];
        int ok = 0;
        if (next.output > 0 && next.group >= 0 && load_acquire(w.ready + next.group) != 0) {
          result[(i + 1) & 1] = __ldcg(w.pair + next.group);
          ok = 1;
        }
        ready[(i + 1) & 1] = ok;
      }
      __syncwarp();
      named_barrier(0, ALL);
    }
  }

  // ---- the eight warps ---------------------------------------------------------------------
  const int row = tid / p.lanes, lane = tid % p.lanes;
  // The tokens of an item on their way, a commit group each.  A slot is filled for the next item as soon
  // as this one's token has been taken from it, so the loads go on through the sums and the barrier.
  const T *x = nullptr, *dy = nullptr, *gate = nullptr;
  const long long sx = p.rows * a.x.st, sy = p.rows * a.y.st, sg = p.rows * a.gate.st;
  int ahead = 0, until = 0, width = 0;
  bool with_gate = false;
  auto aim = [&](const Item& q) {
    until = 0;
    if (q.output < 0 || q.group < 0) return;
    width = min(8, a.d - q.c0 - lane * 8);
    if (width <= 0) return;
    until = q.t1;
    ahead = q.t0 + row;
    with_gate = GATED && (BWD || q.output);
    x = q.template at<const T>(a.x, row, lane);
    if (BWD) dy = q.template at<const T>(a.y, row, lane);
    if (GATED) gate = q.template at<const T>(a.gate, row, lane);
  };
  auto fetch = [&](int u) {
    if (ahead < until) {
      fetch_raw<WIDE>(&slots[u][0][tid], x, width);
      if (BWD) fetch_raw<WIDE>(&slots[u][BWD][tid], dy, width);
      if (with_gate) fetch_raw<WIDE>(&slots[u][TENSORS - 1][tid], gate, width);
    }
    copies_commit();
    ahead += p.rows;
    x += sx;
    if (BWD) dy += sy;
    if (GATED) gate += sg;
  };
  auto begin = [&](const Item& q) {
    aim(q);
#pragma unroll
    for (int u = 0; u < EACH; ++u) fetch(u);
  };
  named_barrier(0, ALL);
  begin(items[0]);
  for (int i = 0;; ++i) {
    const Item& q = items[i & 3];
    const Item& behind = items[(i + 1) & 3];
    if (q.output < 0) return;
    if (q.group < 0) {
      begin(behind);
      named_barrier(0, ALL);
      continue;
    }
    if (q.output && ready[i & 1] == 0) {
      named_barrier(1, ALL);
      if (waited == 0) {
        copies_wait<0>();
        return;
      }
    }
    const int n = max(0, min(8, a.d - q.c0 - lane * 8));
    const int end = n > 0 ? q.t1 : 0;  // threads without channels have no tokens
    int t = q.t0 + row;
    aim(behind);
    if (!BWD && !q.output) {
      // -- forward, first reading: a warp sums its distances from the mean of one of its vectors.  Were
      // that vector far from the rest, its own distances would make m2 as large: m2 loses at most a
      // factor of the warp's vectors in precision, whatever the values.
      const unsigned int valid = __ballot_sync(0xffffffffu, t < end);
      float2 neg = make_float2(0.f, 0.f), s = neg, e = neg;
      int tokens = 0;
#pragma unroll
      for (int u = 0; u < EACH; ++u) {
        copies_wait<EACH - 1>();  // the oldest of EACH groups
        float2 v[4];
        if (t < end) expand(slots[u][0][tid], v);
        fetch(u);
        if (u == 0) {
          float m = 0.f;
          if (t < end) {
            const float2 q4 = add2(add2(v[0], v[1]), add2(v[2], v[3]));
            m = -(q4.x + q4.y) / n;
          }
          m = __shfl_sync(0xffffffffu, m, valid != 0 ? __ffs(valid) - 1 : 0);
          neg = make_float2(m, m);
        }
        if (t < end) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float2 d = add2(v[k], neg);
            if (!WIDE && 2 * k >= n) d.x = 0.f;
            if (!WIDE && 2 * k + 1 >= n) d.y = 0.f;
            s = add2(s, d);
            e = fma2(d, d, e);
          }
          ++tokens;
        }
        t += p.rows;
      }
      const float cnt = (float)__reduce_add_sync(0xffffffffu, tokens * n);
      const float sum = warp_sum(s.x + s.y), sq = warp_sum(e.x + e.y);
      if ((tid & 31) == 0) {
        const float off = cnt > 0.f ? sum / cnt : 0.f;
        red[i & 1][warp][0] = cnt;
        red[i & 1][warp][1] = off - neg.x;
        // squares beyond fp32's range stay infinite, as in the other kernels: their difference would be NaN,
        // and fmaxf would make that a variance of 0
        red[i & 1][warp][2] = sq < INFINITY ? fmaxf(sq - off * sum, 0.f) : sq;
      }
    } else if (!BWD) {
      // -- forward, second reading
      const float2 r = result[i & 1];
      const float2 neg = make_float2(-r.x, -r.x), rs = make_float2(r.y, r.y);
      float2 wt[4], bias[4];
      load_affine<WIDE>(a, q.head * a.d + q.c0 + lane * 8, n, wt, bias);
      T* y = q.template at<T>(a.y, row, lane);
#pragma unroll
      for (int u = 0; u < EACH; ++u) {
        copies_wait<EACH - 1>();
        float2 v[4], g[4];
        if (t < end) {
          expand(slots[u][0][tid], v);
          if (GATED) expand(slots[u][TENSORS - 1][tid], g);
        }
        fetch(u);
        if (t < end) {
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
        }
        t += p.rows;
        y += p.rows * a.y.st;
      }
    } else {
      const float2 ms = reinterpret_cast<const float2*>(a.stats)[q.group], r = result[i & 1];
      const float2 neg = make_float2(-ms.x, -ms.x), rs = make_float2(ms.y, ms.y);
      const float2 n1 = make_float2(-r.x, -r.x), n2 = make_float2(-r.y, -r.y);
      float2 wt[4], bias[4], dw[4], db[4];
      load_affine<WIDE>(a, q.head * a.d + q.c0 + lane * 8, n, wt, bias);
#pragma unroll
      for (int k = 0; k < 4; ++k) dw[k] = db[k] = make_float2(0.f, 0.f);
      T* dx = q.template at<T>(a.dx, row, lane);
      T* dgate = GATED ? q.template at<T>(a.dgate, row, lane) : nullptr;
#pragma unroll 2
      for (int u = 0; u < EACH; ++u) {
        copies_wait<EACH - 1>();
        float2 v[4], g[4], f[4], slope[4], nn[4];  // f: the activation's argument, then its value
        if (t < end) {
          expand(slots[u][0][tid], v);
          expand(slots[u][BWD][tid], g);
          if (GATED) expand(slots[u][TENSORS - 1][tid], f);
        }
        fetch(u);
        if (t < end) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            v[k] = mul2(add2(v[k], neg), rs);
            nn[k] = fma2(v[k], wt[k], bias[k]);
            if (!GATED) f[k] = nn[k];
          }
          slope8(a.act, f, slope);
          if (!q.output) {
            // -- backward, first reading.  Absent channels have dy = 0 and so add nothing.
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 dn = mul2(g[k], GATED ? f[k] : slope[k]);
              dw[k] = fma2(dn, v[k], dw[k]);
              db[k] = add2(db[k], dn);
            }
          } else {
            // -- backward, second reading
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 h = mul2(mul2(g[k], GATED ? f[k] : slope[k]), wt[k]);
              if (GATED) nn[k] = mul2(mul2(g[k], nn[k]), slope[k]);
              v[k] = mul2(rs, fma2(v[k], n2, add2(h, n1)));
            }
            store_pairs<WIDE, 8, true>(dx, v, n);
            if (GATED) store_pairs<WIDE, 8, true>(dgate, nn, n);
          }
        }
        t += p.rows;
        dx += p.rows * a.dx.st;
        if (GATED) dgate += p.rows * a.dgate.st;
      }
      if (!q.output) {
        // the sums of dn w and dn w xhat are those of dn and dn xhat, each channel's times its weight
        float2 s1 = mul2(wt[0], db[0]), s2 = mul2(wt[0], dw[0]);
#pragma unroll
        for (int k = 1; k < 4; ++k) {
          s1 = fma2(wt[k], db[k], s1);
          s2 = fma2(wt[k], dw[k], s2);
        }
        const float w1 = warp_sum(s1.x + s1.y), w2 = warp_sum(s2.x + s2.y);
        if ((tid & 31) == 0) {
          red[i & 1][warp][0] = w1;
          red[i & 1][warp][1] = w2;
        }
        if (w.param != nullptr) {  // each channel's sums over the item's tokens
          const int line = p.lanes * 8;
          float4* c = reinterpret_cast<float4*>(cols + row * 2 * line + lane * 8);
          c[0] = make_float4(dw[0].x, dw[0].y, dw[1].x, dw[1].y);
          c[1] = make_float4(dw[2].x, dw[2].y, dw[3].x, dw[3].y);
          c += line / 4;
          c[0] = make_float4(db[0].x, db[0].y, db[1].x, db[1].y);
          c[1] = make_float4(db[2].x, db[2].y, db[3].x, db[3].y);
          named_barrier(2, kThreads);
          const int D = a.NH * a.d;
          float* out = w.param + ((long long)q.b * p.slabs + q.slab) * 2 * D + q.head * a.d + q.c0;
          for (int e = tid; e < 2 * line; e += kThreads) {
            const int which = e / line, ch = e % line;
            if (q.c0 + ch < a.d) {
              float s = 0.f;
              for (int k = 0; k < p.rows; ++k) s += cols[(k * 2 + which) * line + ch];
              out[(long long)which * D + ch] = s;
            }
          }
        }
      }
    }
    named_barrier(0, ALL);
  }
}

template <typename T, bool GATED, bool WIDE, bool BWD>
cudaError_t run(const NormArgs& a, cudaStream_t s) {
  const Plan p = plan_for(a.B, a.T, a.NH, a.d, (int)sizeof(T), GATED, BWD);
  const Layout l = layout_for(p, a.B, a.NH * a.d, BWD);
  char* ws = (char*)a.ws;
  Work w;
  w.abort = (unsigned int*)ws;
  w.next = w.abort + 1;
  w.done = w.next + 1;
  w.ready = w.done + p.groups;
  w.pair = (float2*)(ws + l.pair);
  w.part = (float*)(ws + l.part);
  const bool params = BWD && (a.dw != nullptr || a.dbias != nullptr);
  w.param = params ? (float*)(ws + l.param) : nullptr;
  cudaError_t e = cudaMemsetAsync(ws, 0, l.zeroed, s);
  if (e != cudaSuccess) return e;
  constexpr int tensors = 1 + BWD + GATED;
  constexpr int bytes =
      kThreads * (each_of((int)sizeof(T), tensors) * tensors * 8 * (int)sizeof(T) + (BWD ? 64 : 0));
  e = cudaFuncSetAttribute(norm_sequence_kernel<T, GATED, WIDE, BWD>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  const long long items = p.items(), slots = slots_of(BWD);
  norm_sequence_kernel<T, GATED, WIDE, BWD>
      <<<(unsigned)(items < slots ? items : slots), kThreads + 64, bytes, s>>>(a, p, w);
  e = cudaGetLastError();
  if (e != cudaSuccess || !params) return e;
  return launch_param_sums(w.param, a.B * p.slabs, a.NH * a.d, 1, a.dw, a.dbias, s);
}
template <typename T, bool BWD>
cudaError_t by_kind(const NormArgs& a, cudaStream_t s) {
  if (a.gate.p != nullptr) return a.wide ? run<T, true, true, BWD>(a, s) : run<T, true, false, BWD>(a, s);
  return a.wide ? run<T, false, true, BWD>(a, s) : run<T, false, false, BWD>(a, s);
}

__global__ void selftest_kernel(unsigned int* words) { selftest_wait(words, &g_norm_failures); }

}  // namespace

long long norm_sequence_items(int B, int T, int NH, int d) {
  long long most = 0;
  for (int kind = 0; kind < 8; ++kind) {
    const Plan p = plan_for(B, T, NH, d, kind & 1 ? 2 : 4, (kind & 2) != 0, (kind & 4) != 0);
    if (p.items() > most) most = p.items();
  }
  return most;
}

size_t norm_sequence_workspace(int B, int T, int NH, int d, int dtype, bool backward) {
  size_t most = 0;  // with a gate or without
  for (int gated = 0; gated < 2; ++gated) {
    size_t bytes;
    if (!norm_resident_workspace(B, T, NH, d, dtype, gated != 0, backward, &bytes))
      bytes = layout_for(plan_for(B, T, NH, d, dtype == 0 ? 2 : 4, gated != 0, backward), B, NH * d, backward).total;
    if (bytes > most) most = bytes;
  }
  return most;
}

cudaError_t launch_norm_sequence(const NormArgs& a, bool backward, cudaStream_t s) {
  cudaError_t status;
  if (launch_norm_resident(a, backward, s, &status)) return status;
  if (backward) return a.dtype == 0 ? by_kind<bf16, true>(a, s) : by_kind<float, true>(a, s);
  return a.dtype == 0 ? by_kind<bf16, false>(a, s) : by_kind<float, false>(a, s);
}

cudaError_t launch_norm_selftest(unsigned int* words, cudaStream_t s) {
  selftest_kernel<<<1, 1, 0, s>>>(words);
  return cudaGetLastError();
}
cudaError_t norm_flag(unsigned int** at) { return cudaGetSymbolAddress((void**)at, g_norm_failures); }

}  // namespace mlstm

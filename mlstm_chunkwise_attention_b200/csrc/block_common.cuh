// Device helpers shared by the kernels around the recurrence: vectors of eight
// channels in the I/O dtype, activations, and a fixed-order sum of partial rows.
#pragma once

#include "block.h"
#include "common.cuh"
#include "tc_common.cuh"

namespace mlstm {

// Eight consecutive channels as fp32.  WIDE: 16-byte accesses (the address is
// then 16-byte aligned and all eight exist); else the first `n` elements one by
// one, the rest read as zero.
template <bool WIDE>
__device__ __forceinline__ void load8(const bf16* p, float* v, int n) {
  if (WIDE) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? to_f32(p[i]) : 0.f;
  }
}
template <bool WIDE>
__device__ __forceinline__ void load8(const float* p, float* v, int n) {
  if (WIDE) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : 0.f;
  }
}
template <bool WIDE>
__device__ __forceinline__ void store8(bf16* p, const float* v, int n) {
  if (WIDE) {
    uint4 u;
    uint32_t* w = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = u;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = from_f32<bf16>(v[i]);
  }
}
template <bool WIDE>
__device__ __forceinline__ void store8(float* p, const float* v, int n) {
  if (WIDE) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = v[i];
  }
}

// Four or eight consecutive channels as they lie in memory: loads into these stay in flight while
// earlier ones are worked on (converting at once would wait for each).
template <typename T, int C> struct Raw;
template <> struct Raw<bf16, 4> { uint2 u; };
template <> struct Raw<bf16, 8> { uint4 u; };
template <> struct Raw<float, 4> { float4 u; };
template <> struct Raw<float, 8> { float4 u, v; };

// WIDE as in load8; else the first n elements, the rest zero.
template <bool WIDE, int C>
__device__ __forceinline__ void load_raw(const bf16* p, Raw<bf16, C>& r, int n) {
  if (WIDE) {
    r.u = *reinterpret_cast<const decltype(r.u)*>(p);
  } else {
    uint32_t w[C / 2];
    const unsigned short* q = reinterpret_cast<const unsigned short*>(p);
#pragma unroll
    for (int i = 0; i < C / 2; ++i)
      w[i] = (2 * i < n ? (uint32_t)q[2 * i] : 0u) | (2 * i + 1 < n ? (uint32_t)q[2 * i + 1] << 16 : 0u);
    r.u = *reinterpret_cast<decltype(r.u)*>(w);
  }
}
template <bool WIDE>
__device__ __forceinline__ void load_raw(const float* p, Raw<float, 4>& r, int n) {
  if (WIDE)
    r.u = *reinterpret_cast<const float4*>(p);
  else
    r.u = make_float4(n > 0 ? p[0] : 0.f, n > 1 ? p[1] : 0.f, n > 2 ? p[2] : 0.f, n > 3 ? p[3] : 0.f);
}
template <bool WIDE>
__device__ __forceinline__ void load_raw(const float* p, Raw<float, 8>& r, int n) {
  Raw<float, 4> a, b;
  load_raw<WIDE>(p, a, n);
  load_raw<WIDE>(p + 4, b, n - 4);
  r.u = a.u;
  r.v = b.u;
}
template <typename T, int C>
__device__ __forceinline__ void zero_raw(Raw<T, C>& r) { r = Raw<T, C>{}; }
// As pairs of neighbouring channels.
template <int C>
__device__ __forceinline__ void expand(const Raw<bf16, C>& r, float2* v) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(&r);
#pragma unroll
  for (int i = 0; i < C / 2; ++i)
    v[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
template <int C>
__device__ __forceinline__ void expand(const Raw<float, C>& r, float2* v) {
  const float2* w = reinterpret_cast<const float2*>(&r);
#pragma unroll
  for (int i = 0; i < C / 2; ++i) v[i] = w[i];
}
// STREAM: what is stored will not be read soon, and makes room in L2 first.
template <bool WIDE, int C, bool STREAM = false>
__device__ __forceinline__ void store_pairs(bf16* p, const float2* v, int n) {
  if (WIDE) {
    uint32_t w[C / 2];
#pragma unroll
    for (int i = 0; i < C / 2; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[i].x, v[i].y);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    Raw<bf16, C> r;
    r.u = *reinterpret_cast<decltype(r.u)*>(w);
    if (STREAM)
      __stcs(reinterpret_cast<decltype(r.u)*>(p), r.u);
    else
      *reinterpret_cast<decltype(r.u)*>(p) = r.u;
  } else {
#pragma unroll
    for (int i = 0; i < C; ++i)
      if (i < n) p[i] = from_f32<bf16>(i & 1 ? v[i / 2].y : v[i / 2].x);
  }
}
template <bool WIDE, int C, bool STREAM = false>
__device__ __forceinline__ void store_pairs(float* p, const float2* v, int n) {
  if (WIDE) {
#pragma unroll
    for (int i = 0; i < C / 4; ++i) {
      const float4 r = make_float4(v[2 * i].x, v[2 * i].y, v[2 * i + 1].x, v[2 * i + 1].y);
      if (STREAM)
        __stcs(reinterpret_cast<float4*>(p) + i, r);
      else
        reinterpret_cast<float4*>(p)[i] = r;
    }
  } else {
#pragma unroll
    for (int i = 0; i < C; ++i)
      if (i < n) p[i] = i & 1 ? v[i / 2].y : v[i / 2].x;
  }
}

// A copy of 4, 8 or 16 bytes into shared memory that completes in the background.
template <int BYTES = 16>
__device__ __forceinline__ void copy_async(void* smem, const void* gmem) {
  const uint32_t to = (uint32_t)__cvta_generic_to_shared(smem);
  if (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(gmem) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(gmem), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copies_wait() {  // all but the newest LEFT groups are done
  asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}
// Brings a thread's channels into its own slot of shared memory, in the background unless they are
// single bf16 values (there is no such copy of two bytes).  The thread reads them after its own
// wait; no barrier is needed.
template <bool WIDE, typename T, int C>
__device__ __forceinline__ void fetch_raw(Raw<T, C>* to, const T* from, int n) {
  if (WIDE) {
    constexpr int size = (int)sizeof(Raw<T, C>), piece = size < 16 ? 8 : 16;
#pragma unroll
    for (int i = 0; i < size; i += piece) copy_async<piece>((char*)to + i, (const char*)from + i);
  } else if (sizeof(T) == 4) {
    float* slot = reinterpret_cast<float*>(to);
#pragma unroll
    for (int i = 0; i < C; ++i) {
      if (i < n)
        copy_async<4>(slot + i, from + i);
      else
        slot[i] = 0.f;
    }
  } else {
    Raw<T, C> r;
    load_raw<false>(from, r, n);
    *to = r;
  }
}

// Packed fp32 arithmetic: two lanes of fp32 in one instruction, each rounded as fmaf / + / * round.
__device__ __forceinline__ unsigned long long as_u64(float2 a) {
  return *reinterpret_cast<unsigned long long*>(&a);
}
__device__ __forceinline__ float2 as_f2(unsigned long long a) { return *reinterpret_cast<float2*>(&a); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  unsigned long long d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(as_u64(a)), "l"(as_u64(b)), "l"(as_u64(c)));
  return as_f2(d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  unsigned long long d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(as_u64(a)), "l"(as_u64(b)));
  return as_f2(d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  unsigned long long d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(as_u64(a)), "l"(as_u64(b)));
  return as_f2(d);
}

// The abort state of one launch whose CTAs wait for one another.  `word` lies in the launch's workspace
// and is zeroed with its counters, by a memset that a graph captures too, so a replayed launch starts
// clean whatever became of the ones before it.  `failures` is the kernel family's count of launches that
// gave up since mlstm_device_status last took it, so a second failure of the same graph is news as well.
struct LaunchAbort {
  unsigned int *word, *failures;
  __device__ __forceinline__ bool raised() const { return *reinterpret_cast<volatile unsigned int*>(word) != 0; }
  __device__ __forceinline__ void raise() const {
    if (atomicExch(word, 1u) == 0) atomicAdd(failures, 1u);
  }
};
__device__ __forceinline__ unsigned int load_acquire(const unsigned int* at) {
  unsigned int v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(at) : "memory");
  return v;
}
// One thread waits until *at >= least; false if it gave up, after the 2 s of the tensor-core kernels' waits
// or because another CTA of the launch did.
__device__ __forceinline__ bool wait_at_least(const unsigned int* at, unsigned int least,
                                              const LaunchAbort& abort, unsigned int nap_ns) {
  const uint64_t began = tc::global_timer_ns();
  for (unsigned int i = 1; load_acquire(at) < least; ++i) {
    if ((i & 63) == 0 && (abort.raised() || tc::global_timer_ns() - began > tc::kWaitTimeoutNs)) {
      abort.raise();
      return false;
    }
    __nanosleep(nap_ns);
  }
  return true;
}
// A launch whose wait runs out: word 0 is its abort word, word 1 what nothing raises.
__device__ __forceinline__ void selftest_wait(unsigned int* words, unsigned int* failures) {
  wait_at_least(words + 1, 1, LaunchAbort{words, failures}, 200);
}

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// 2^x, relative error about 2^-22, 0 far below zero; 1 / x, one ulp.  The .ftz forms: the others
// spend instructions on results below 2^-126.
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float2 exp2_pair(float2 v) {
  return make_float2(exp2_fast(v.x), exp2_fast(v.y));
}

// 1 / (1 + exp(-v)); 0 and 1 at the far ends, NaN for NaN.
__device__ __forceinline__ float2 sigmoid_pair(float2 v) {
  const float2 e = add2(exp2_pair(mul2(v, make_float2(-kLog2e, -kLog2e))), make_float2(1.f, 1.f));
  return make_float2(rcp_fast(e.x), rcp_fast(e.y));
}

// max(v, -100), NaN for NaN: silu is below 2^-126 from there on, and -inf would make it inf times 0.
__device__ __forceinline__ float2 above_minus_100(float2 v) {
  asm("max.NaN.f32 %0, %0, 0fC2C80000;" : "+f"(v.x));
  asm("max.NaN.f32 %0, %0, 0fC2C80000;" : "+f"(v.y));
  return v;
}

// The activation, and with its slope.
template <int ACT>
__device__ __forceinline__ float2 act_pair(float2 v) {
  if (ACT == kActNone) return v;
  if (ACT == kActSigmoid) return sigmoid_pair(v);
  v = above_minus_100(v);
  return mul2(v, sigmoid_pair(v));
}
template <int ACT>
__device__ __forceinline__ void slope_pair(float2 v, float2* value, float2* slope) {
  const float2 one = make_float2(1.f, 1.f), minus = make_float2(-1.f, -1.f);
  if (ACT == kActNone) {
    *value = v;
    *slope = one;
    return;
  }
  if (ACT == kActSilu) v = above_minus_100(v);
  const float2 s = sigmoid_pair(v), rest = fma2(s, minus, one);
  if (ACT == kActSigmoid) {
    *value = s;
    *slope = mul2(s, rest);
  } else {
    *value = mul2(v, s);
    *slope = fma2(*value, rest, s);
  }
}

}  // namespace mlstm

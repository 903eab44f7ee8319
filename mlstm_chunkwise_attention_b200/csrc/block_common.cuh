// Device helpers shared by the kernels around the recurrence: vectors of eight
// channels in the I/O dtype, activations, and a fixed-order sum of partial rows.
#pragma once

#include "block.h"
#include "common.cuh"

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

// 1 / (1 + exp(-v)); 0 and 1 at the far ends, NaN for NaN.
__device__ __forceinline__ float sigmoidf(float v) { return __fdividef(1.f, 1.f + __expf(-v)); }

// The activation and its slope.  silu(v) = v sigmoid(v): 0 at -inf, where the product would be NaN.
template <int ACT>
__device__ __forceinline__ float act_value(float v) {
  if (ACT == kActNone) return v;
  const float s = sigmoidf(v);
  if (ACT == kActSigmoid) return s;
  return s == 0.f ? 0.f : v * s;
}
template <int ACT>
__device__ __forceinline__ void act_slope(float v, float* value, float* slope) {
  if (ACT == kActNone) {
    *value = v;
    *slope = 1.f;
    return;
  }
  const float s = sigmoidf(v);
  if (ACT == kActSigmoid) {
    *value = s;
    *slope = s * (1.f - s);
    return;
  }
  *value = s == 0.f ? 0.f : v * s;
  *slope = s == 0.f ? 0.f : fmaf(*value, 1.f - s, s);
}

}  // namespace mlstm

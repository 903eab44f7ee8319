// What the group norm's kernels share.
#pragma once

#include "block_common.cuh"

namespace mlstm {

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

}  // namespace mlstm

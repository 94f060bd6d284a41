// decay_common.cuh -- the decay of the decayed linear attention, shared by its kernels.
#pragma once

#include <cuda_runtime.h>

namespace gdr {

// l^n with l = exp(g).  n = 0 is 1 for every g (g = -inf, a head that forgets at once, included).
__device__ __forceinline__ float decay_pow(float g, int64_t n) {
  return n == 0 ? 1.0f : expf(g * static_cast<float>(n));
}

// H <- l^n H + add as a H + (b H + add).  Where l^n is near 1 (slow heads), a = 1 and
// b = l^n - 1 by expm1: rounding l^n itself to 32 bits would be a relative error of up to
// 2^-25 in every step, all of one sign, which a memory of 1 / |g n| steps adds up (3e-3 at
// g n = -1e-5).  Elsewhere a = 0 and b = l^n.
struct DecayStep {
  float a, b;
  __device__ __forceinline__ float apply(float H, float add) const { return fmaf(a, H, fmaf(b, H, add)); }
  __device__ __forceinline__ float2 apply2(float2 H, float2 add) const {
    return __ffma2_rn(make_float2(a, a), H, __ffma2_rn(make_float2(b, b), H, add));
  }
};
__device__ __forceinline__ DecayStep decay_step(float g, int64_t n) {
  const float x = n == 0 ? 0.0f : g * static_cast<float>(n);
  DecayStep s;
  const bool near1 = x > -0.5f && x < 0.5f;
  s.a = near1 ? 1.0f : 0.0f;
  s.b = near1 ? expm1f(x) : expf(x);
  return s;
}

}  // namespace gdr

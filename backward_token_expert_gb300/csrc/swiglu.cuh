// The gated activation phi = silu(a) b, silu(a) = a / (1 + exp(-a)), and its
// derivative, in fp32.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "f32x2.cuh"

namespace lrm {

__device__ __forceinline__ float silu_grad(float a, float& silu) {
  const float s = 1.0f / (1.0f + expf(-a));
  silu = a * s;
  return s * (1.0f + a * (1.0f - s));
}

// The logistic functions of two values, one exponential and one reciprocal each, both approximate and without
// denormals: within (2 + |a|) 2^-22 of the value, relative, and 0 below a = -87 (less than 1e-37).
__device__ __forceinline__ F2 sigmoid2(F2 a) {
  const float2 t = mul2(a, F2(-1.4426950408889634f, -1.4426950408889634f)).get();
  F2 e;
  {
    float x, y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(x) : "f"(t.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(t.y));
    e = add2(F2(x, y), F2(1.0f, 1.0f));
  }
  const float2 d = e.get();
  float x, y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(x) : "f"(d.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(d.y));
  return F2(x, y);
}

__device__ __forceinline__ F2 silu2(F2 a) { return mul2(a, sigmoid2(a)); }

// silu'(a) and silu(a) of two values, from those: within (2 + |a|) 2^-22 of 1 + |a|.
__device__ __forceinline__ F2 silu_grad2(F2 a, F2& silu) {
  const F2 s = sigmoid2(a);
  silu = mul2(a, s);
  return fma2(silu, fma2(s, F2(-1.0f, -1.0f), F2(1.0f, 1.0f)), s);
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t pack_bf16x2(F2 v) {
  const float2 f = v.get();
  return pack_bf16x2(f.x, f.y);
}

}  // namespace lrm

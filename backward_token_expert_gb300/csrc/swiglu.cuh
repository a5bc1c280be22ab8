// The gated activation phi = silu(a) b, silu(a) = a / (1 + exp(-a)), and its
// derivative, in fp32.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace lrm {

// One exponential and one quotient, both approximate: within (2 + |a|) 2^-22 of the value, relative, and 0 below
// a = -87 (a value that would be smaller than 1e-36).
__device__ __forceinline__ float silu(float a) { return __fdividef(a, 1.0f + __expf(-a)); }

__device__ __forceinline__ float silu_grad(float a, float& silu) {
  const float s = 1.0f / (1.0f + expf(-a));
  silu = a * s;
  return s * (1.0f + a * (1.0f - s));
}

// The same from approximate functions, as silu() above: within (2 + |a|) 2^-22 of 1 + |a|.
__device__ __forceinline__ float silu_grad_fast(float a, float& silu) {
  const float s = __fdividef(1.0f, 1.0f + __expf(-a));
  silu = a * s;
  return fmaf(silu, 1.0f - s, s);
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&r);
}

}  // namespace lrm

// SwiGLU and its derivatives in fp32, shared by the glue and the kernels that
// work from kept activations (gfx950).
//
// sigmoid uses e = exp(-|g|) in (0, 1]: sigmoid(|g|) = 1 / (1 + e) and
// sigmoid(-|g|) = e / (1 + e), so neither 1 - sigmoid nor a large exponent
// is ever formed.  1 + e lies in (1, 2], so its reciprocal is the hardware
// one (V_RCP_F32, within 1 ulp; no denormal can occur) instead of a
// correctly rounded division sequence.
#pragma once

#include "mx_device.h"

namespace mx {

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// silu(g) and the two sigmoids sigmoid(g), sigmoid(-g).
__device__ __forceinline__ float silu_parts(float g, float& s, float& sm) {
  const float e = expf(-fabsf(g));
  const float r = __builtin_amdgcn_rcpf(1.0f + e);
  const float er = e * r;
  s = g >= 0.0f ? r : er;
  sm = g >= 0.0f ? er : r;
  return g * s;
}

__device__ __forceinline__ float swiglu1(float g, float u) {
  float s, sm;
  return silu_parts(g, s, sm) * u;
}

// dL/dg and dL/du of silu(g) u for dL/d(silu(g) u) = d.
__device__ __forceinline__ float swiglu_dgate(float g, float u, float d) {
  float s, sm;
  silu_parts(g, s, sm);
  return d * u * s * (1.0f + g * sm);
}

__device__ __forceinline__ float swiglu_dup(float g, float d) {
  float s, sm;
  return d * silu_parts(g, s, sm);
}

}  // namespace mx

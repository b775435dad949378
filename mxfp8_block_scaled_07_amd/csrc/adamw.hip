// AdamW step over many tensors (gfx950), with fp32 states or states in MXFP8.
//
//   g = grad * grad_scale;  m = b1 m + (1 - b1) g;  v = b2 v + (1 - b2) g^2
//   p = p (1 - lr wd) - (lr / (1 - b1^t)) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// Bound: HBM.  Everything is read and written once: 8 + 4 + 16 bytes per
// element of fp32 parameters, gradients and states, 8 + 2 + 4.125 (+ 2 for a
// bf16 copy) with bf16 gradients and 8-bit states.
//
// One launch takes up to kBatch tensors: their pointers travel in the kernel
// arguments, so the call needs no table in device memory and can be captured.
// A block takes one chunk of one tensor, a thread 4 consecutive elements (16
// bytes of fp32) per pass.
//
// 8-bit states are MX blocks of 32 consecutive elements (E4M3 codes, one E8M0
// scale).  m is kept as it is and v as its root: E4M3 spans 2^-9 .. 448 inside
// a block, which as v itself would be 17 binary orders of the gradient's
// square, as its root it is 17 of the gradient.  With b2 = 0.999 one step moves
// v by about 0.1%, far less than a code's step (6 to 12%), so rounding to
// nearest would never let it move; the states are therefore rounded up or
// down at random, up with probability the fraction, which keeps them right on
// average.  A positive root is never rounded to zero (m would then be divided
// by eps alone).  The scale is the smallest power of two with which the
// block's largest value is not above 448, so nothing saturates.  bf16
// parameters without an fp32 master are rounded in the same way: lr times a
// step is usually less than half their spacing.
// The random bits are a function of (seed, step, tensor, element) only.

#include "mx_device.h"

namespace mx {
namespace {

constexpr int kAdamThreads = 256;
constexpr int kPass = 4 * kAdamThreads;   // elements of a block per pass
constexpr int kBatch = 48;                // tensors per launch (the arguments stay below 4 KB)

struct Batch {
  mx_adamw_tensor_t t[kBatch];
  int32_t first[kBatch + 1];   // chunks before each tensor
  int32_t count, base;         // tensors here; the index of t[0] in the call
  int32_t passes;              // a chunk's passes
};
static_assert(sizeof(Batch) <= 3500, "kernel arguments");

struct Hyper {
  const float *lr, *grad_scale;
  const int32_t* step;
  double b1, b2;
  float eps, wd;
  uint32_t seed_lo, seed_hi;
};

constexpr uint32_t kGold = 0x9E3779B1u;

__device__ __forceinline__ uint32_t mix(uint32_t x) {
  x ^= x >> 16;
  x *= 0x6A09E667u;
  x ^= x >> 15;
  x *= 0xBB67AE85u;
  return x ^ (x >> 16);
}

// 1 - b^t, the power by repeated squaring in fp64 (1 - b^t cancels for small t).
__device__ __forceinline__ double one_minus_pow(double b, uint32_t t) {
  double r = 1.0;
  for (; t; t >>= 1) {
    if (t & 1) r *= b;
    b *= b;
  }
  return 1.0 - r;
}

__device__ __forceinline__ bool finite(float x) { return (__float_as_uint(x) & 0x7F800000u) != 0x7F800000u; }

// Largest of a block's 32 elements: 8 consecutive lanes hold it.
__device__ __forceinline__ float octet_max(float v) {
  v = fmaxf(v, __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(v), 0xB1, 0xF, 0xF, false)));
  v = fmaxf(v, __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(v), 0x4E, 0xF, 0xF, false)));
  // row_half_mirror: lane i of 8 takes lane 7 - i
  return fmaxf(v, __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(v), 0x141, 0xF, 0xF, false)));
}

// The block's scale byte: the smallest with amax / 2^(byte - 127) <= 448 = 1.75 * 2^8.
__device__ __forceinline__ uint32_t state_scale(float amax) {
  const uint32_t e = (__float_as_uint(amax) + 0x1FFFFFu) >> 23;   // one more above a mantissa of 1.75
  return e > 8u ? e - 8u : 0u;
}

// E4M3 code of y in [0, 448], rounded up with probability (u + 1/2^16's worth
// of) its fraction: u has 16 bits.
__device__ __forceinline__ uint32_t stochastic_e4m3(float y, uint32_t u) {
  const uint32_t b = __float_as_uint(y);
  const uint32_t normal = ((b + (u << 4)) >> 20) - 960u;
  const uint32_t small = (uint32_t)(y * 512.0f + (float)u * 0x1p-16f);
  return b >= 0x3C800000u ? normal : small;   // 2^-6, the smallest normal code
}

__device__ __forceinline__ uint32_t stochastic_bf16(float x, uint32_t u) {
  const uint32_t b = __float_as_uint(x);
  return finite(x) ? (b + u) >> 16 : (b >> 16) | ((b & 0xFFFFu) ? 0x40u : 0u);
}

template <bool kF32>
__device__ __forceinline__ void load4(const void* p, int64_t i, int n, float (&x)[4]) {
  if (n == 4) {
    if constexpr (kF32) {
      const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
      x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
      x[0] = __uint_as_float(v.x << 16); x[1] = __uint_as_float(v.x & 0xFFFF0000u);
      x[2] = __uint_as_float(v.y << 16); x[3] = __uint_as_float(v.y & 0xFFFF0000u);
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x[k] = 0.0f;
    if (k < n) {
      if constexpr (kF32) x[k] = static_cast<const float*>(p)[i + k];
      else x[k] = __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i + k] << 16);
    }
  }
}

__device__ __forceinline__ void store4_f32(void* p, int64_t i, int n, const float (&x)[4]) {
  float* d = static_cast<float*>(p) + i;
  if (n == 4) {
    *reinterpret_cast<float4*>(d) = make_float4(x[0], x[1], x[2], x[3]);
    return;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (k < n) d[k] = x[k];
}

__device__ __forceinline__ void store4_u16(void* p, int64_t i, int n, uint32_t lo, uint32_t hi) {
  uint16_t* d = static_cast<uint16_t*>(p) + i;
  if (n == 4) {
    *reinterpret_cast<uint2*>(d) = make_uint2(lo, hi);
    return;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (k < n) d[k] = (uint16_t)((k < 2 ? lo : hi) >> (16 * (k & 1)));
}

__device__ __forceinline__ uint32_t load4_u8(const void* p, int64_t i, int n) {
  const uint8_t* s = static_cast<const uint8_t*>(p) + i;
  if (n == 4) return *reinterpret_cast<const uint32_t*>(s);
  uint32_t v = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (k < n) v |= (uint32_t)s[k] << (8 * k);
  return v;
}

__device__ __forceinline__ void store4_u8(void* p, int64_t i, int n, uint32_t v) {
  uint8_t* d = static_cast<uint8_t*>(p) + i;
  if (n == 4) {
    *reinterpret_cast<uint32_t*>(d) = v;
    return;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (k < n) d[k] = (uint8_t)(v >> (8 * k));
}

// Four codes of a block to fp32.
__device__ __forceinline__ void decode4(uint32_t codes, uint32_t byte, float (&x)[4]) {
  const float s = e8m0_to_f32(byte);
  const v2f lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(codes, s, false);
  const v2f hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(codes, s, true);
  x[0] = lo[0]; x[1] = lo[1]; x[2] = hi[0]; x[3] = hi[1];
}

// Four values of a block to codes (the block's scale byte in `byte`).
template <bool kLeast>
__device__ __forceinline__ uint32_t encode4(const float (&x)[4], const uint32_t (&u)[4], uint32_t& byte) {
  float amax = 0.0f;
#pragma unroll
  for (int k = 0; k < 4; ++k) amax = fmaxf(amax, finite(x[k]) ? fabsf(x[k]) : 0.0f);
  byte = state_scale(octet_max(amax));
  const float inv = __uint_as_float((254u - byte) << 23);
  uint32_t codes = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t c = stochastic_e4m3(fabsf(x[k]) * inv, u[k]);
    if (kLeast && x[k] > 0.0f && c == 0) c = 1;
    if (!finite(x[k])) c = 0x7Fu;   // NaN
    codes |= (c | ((__float_as_uint(x[k]) >> 24) & 0x80u)) << (8 * k);
  }
  return codes;
}

template <bool kP32, bool kG32, bool kS8>
__global__ void __launch_bounds__(kAdamThreads) k_adamw(Batch b, Hyper hp) {
  // the block's tensor: the last with first[i] <= blockIdx.x
  int lo = 0, hi = b.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (b.first[mid] <= (int)blockIdx.x) lo = mid; else hi = mid;
  }
  const mx_adamw_tensor_t& t = b.t[lo];
  const int64_t begin = (int64_t)((int)blockIdx.x - b.first[lo]) * b.passes * kPass;

  const int32_t st = *hp.step;
  const uint32_t step = st < 1 ? 1u : (uint32_t)st;
  const float lr = *hp.lr;
  const float gs = hp.grad_scale ? *hp.grad_scale : 1.0f;
  const float b1 = (float)hp.b1, b2 = (float)hp.b2;
  const float c1 = (float)(1.0 - hp.b1), c2 = (float)(1.0 - hp.b2);
  const float size = lr / (float)one_minus_pow(hp.b1, step);
  const float root2 = (float)(1.0 / sqrt(one_minus_pow(hp.b2, step)));
  const float decay = 1.0f - lr * hp.wd;
  uint32_t key = mix(hp.seed_lo ^ kGold);
  key = mix(key ^ hp.seed_hi);
  key = mix(key ^ step);
  key = mix(key ^ (uint32_t)(b.base + lo));

  for (int pass = 0; pass < b.passes; ++pass) {
    const int64_t i = begin + (int64_t)pass * kPass + 4 * threadIdx.x;
    if (i - 4 * (int64_t)threadIdx.x >= t.n) break;
    // lanes past the end stay, so that whole blocks of 32 reduce together
    const int n = i >= t.n ? 0 : (t.n - i < 4 ? (int)(t.n - i) : 4);
    float p[4], g[4], m[4], v[4];
    load4<kP32>(t.param, i, n, p);
    load4<kG32>(t.grad, i, n, g);
    if constexpr (kS8) {
      const int64_t blk = i >> 5;
      const uint32_t mc = load4_u8(t.m, i, n), vc = load4_u8(t.v, i, n);
      decode4(mc, n ? t.m_scale[blk] : 0u, m);
      decode4(vc, n ? t.v_scale[blk] : 0u, v);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] *= v[k];
    } else {
      load4<true>(t.m, i, n, m);
      load4<true>(t.v, i, n, v);
    }
    float root[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float gk = g[k] * gs;
      m[k] = fmaf(b1, m[k], c1 * gk);
      v[k] = fmaf(b2, v[k], c2 * (gk * gk));
      root[k] = sqrtf(v[k]);
      p[k] = fmaf(-size, m[k] / fmaf(root[k], root2, hp.eps), p[k] * decay);
    }
    uint32_t h[4];
    if constexpr (kS8 || !kP32) {
#pragma unroll
      for (int k = 0; k < 4; ++k) h[k] = mix((key + (uint32_t)(i + k) * kGold) ^ (uint32_t)((i + k) >> 32));
    }
    if constexpr (kS8) {
      uint32_t um[4], uv[4], bm, bv;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        um[k] = h[k] >> 16;
        uv[k] = h[k] & 0xFFFFu;
        if (k >= n) m[k] = root[k] = 0.0f;   // not in the block
      }
      const uint32_t cm = encode4<false>(m, um, bm), cv = encode4<true>(root, uv, bv);
      store4_u8(t.m, i, n, cm);
      store4_u8(t.v, i, n, cv);
      if ((threadIdx.x & 7) == 0 && n) {
        t.m_scale[i >> 5] = (uint8_t)bm;
        t.v_scale[i >> 5] = (uint8_t)bv;
      }
    } else {
      store4_f32(t.m, i, n, m);
      store4_f32(t.v, i, n, v);
    }
    if constexpr (kP32) {
      store4_f32(t.param, i, n, p);
      if (t.copy) store4_u16(t.copy, i, n, bf16x2_rne(p[0], p[1]), bf16x2_rne(p[2], p[3]));
    } else {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = stochastic_bf16(p[k], mix(h[k] ^ kGold) >> 16);
      const uint32_t a = w[0] | (w[1] << 16), c = w[2] | (w[3] << 16);
      store4_u16(t.param, i, n, a, c);
      if (t.copy) store4_u16(t.copy, i, n, a, c);
    }
  }
}

template <bool kP32, bool kG32>
void launch_adamw(bool s8, unsigned blocks, hipStream_t st, const Batch& b, const Hyper& hp) {
  if (s8) hipLaunchKernelGGL((k_adamw<kP32, kG32, true>), dim3(blocks), dim3(kAdamThreads), 0, st, b, hp);
  else hipLaunchKernelGGL((k_adamw<kP32, kG32, false>), dim3(blocks), dim3(kAdamThreads), 0, st, b, hp);
}

}  // namespace
}  // namespace mx

using namespace mx;

extern "C" int mx_adamw(const mx_adamw_tensor_t* tensors, int32_t count, int32_t param_dtype, int32_t grad_dtype,
                        int32_t state_bits, const float* lr, const int32_t* step, const float* grad_scale,
                        double beta1, double beta2, double eps, double weight_decay, uint64_t seed,
                        mx_stream_t stream) {
  if (count < 0 || (count > 0 && !tensors) || !lr || !step) return MX_EINVAL;
  if ((param_dtype != MX_OUT_F32 && param_dtype != MX_OUT_BF16) || (grad_dtype != MX_OUT_F32 && grad_dtype != MX_OUT_BF16))
    return MX_EINVAL;
  if (state_bits != 8 && state_bits != 32) return MX_EINVAL;
  if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0)) return MX_EINVAL;
  if (!(eps >= 0.0 && eps <= 1e30) || !(weight_decay >= -1e30 && weight_decay <= 1e30)) return MX_EINVAL;
  if (((uintptr_t)lr | (uintptr_t)step | (uintptr_t)grad_scale) & 3) return MX_EINVAL;
  int64_t total = 0;
  for (int32_t i = 0; i < count; ++i) {
    const mx_adamw_tensor_t& t = tensors[i];
    if (t.n < 0) return MX_EINVAL;
    if (t.n == 0) continue;
    if (!t.param || !t.grad || !t.m || !t.v) return MX_EINVAL;
    if (state_bits == 8 && (!t.m_scale || !t.v_scale)) return MX_EINVAL;
    // 16-byte accesses
    if (((uintptr_t)t.param | (uintptr_t)t.grad | (uintptr_t)t.m | (uintptr_t)t.v | (uintptr_t)t.copy) & 15)
      return MX_EINVAL;
    if (t.n >= (1ll << 40) || total >= (1ll << 40)) return MX_EUNSUPPORTED;
    total += t.n;
  }
  if (total == 0) return MX_OK;
  // passes per block: one while that still gives every CU its eight blocks,
  // up to eight so that large steps do not pay a block's start per 1024 elements
  int64_t passes = total / (256ll * 8 * kPass);
  passes = passes < 1 ? 1 : (passes > 8 ? 8 : passes);
  while (total / (passes * kPass) >= (1ll << 30)) passes *= 2;
  Hyper hp;
  hp.lr = lr;
  hp.grad_scale = grad_scale;
  hp.step = step;
  hp.b1 = beta1;
  hp.b2 = beta2;
  hp.eps = (float)eps;
  hp.wd = (float)weight_decay;
  hp.seed_lo = (uint32_t)seed;
  hp.seed_hi = (uint32_t)(seed >> 32);
  const hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  for (int32_t base = 0; base < count; base += kBatch) {
    Batch b;
    b.count = count - base < kBatch ? count - base : kBatch;
    b.base = base;
    b.passes = (int32_t)passes;
    int64_t chunks = 0;
    for (int32_t i = 0; i < b.count; ++i) {
      b.t[i] = tensors[base + i];
      b.first[i] = (int32_t)chunks;
      chunks += (b.t[i].n + passes * kPass - 1) / (passes * kPass);
    }
    b.first[b.count] = (int32_t)chunks;
    if (chunks == 0) continue;
    const bool s8 = state_bits == 8, g32 = grad_dtype == MX_OUT_F32;
    if (param_dtype == MX_OUT_F32) {
      if (g32) launch_adamw<true, true>(s8, (unsigned)chunks, st, b, hp);
      else launch_adamw<true, false>(s8, (unsigned)chunks, st, b, hp);
    } else {
      if (g32) launch_adamw<false, true>(s8, (unsigned)chunks, st, b, hp);
      else launch_adamw<false, false>(s8, (unsigned)chunks, st, b, hp);
    }
    const int rc = launch_status();
    if (rc != MX_OK) return rc;
  }
  return MX_OK;
}

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
// A block takes 1024 elements of one tensor, a thread 4 consecutive ones (16
// bytes of fp32); more per block is slower (fp32 states 144, 145, 149 us for 1,
// 2, 4 times as many on 30M elements; 8-bit states 1.80, 1.91, 1.94 ms on 671M).
// Now 141 us, and 1.74 to 1.79 ms (6.0 to 6.2 TB/s).
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
constexpr int kChunk = 4 * kAdamThreads;  // elements of a block
constexpr int kBatch = 48;                // tensors per launch (the arguments stay below 4 KB)

struct Batch {
  mx_adamw_tensor_t t[kBatch];
  int32_t first[kBatch + 1];   // chunks before each tensor
  int32_t count, base;         // tensors here; the index of t[0] in the call
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

// Four elements from i on; n of them where not kFull.  Each byte is used once:
// non-temporal accesses leave the caches alone (97 tensors of 30M elements,
// fp32: 144 us, against 191 with default ones).
typedef float f4 __attribute__((ext_vector_type(4)));
typedef unsigned int u2 __attribute__((ext_vector_type(2)));

template <bool kF32>
struct Raw4 {
  f4 f;
};
template <>
struct Raw4<false> {
  u2 f;
};

template <bool kF32, bool kFull>
__device__ __forceinline__ Raw4<kF32> load4(const void* p, int64_t i, int n) {
  Raw4<kF32> r;
  if constexpr (kF32) {
    const float* s = static_cast<const float*>(p) + i;
    if (kFull) {
      r.f = __builtin_nontemporal_load(reinterpret_cast<const f4*>(s));
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) r.f[k] = k < n ? s[k] : 0.0f;
    }
  } else {
    const uint16_t* s = static_cast<const uint16_t*>(p) + i;
    if (kFull) {
      r.f = __builtin_nontemporal_load(reinterpret_cast<const u2*>(s));
    } else {
      r.f = u2{0, 0};
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (k < n) r.f[k >> 1] |= (uint32_t)s[k] << (16 * (k & 1));
    }
  }
  return r;
}

__device__ __forceinline__ void widen(const Raw4<true>& r, float (&x)[4]) {
  x[0] = r.f[0]; x[1] = r.f[1]; x[2] = r.f[2]; x[3] = r.f[3];
}
__device__ __forceinline__ void widen(const Raw4<false>& r, float (&x)[4]) {
  x[0] = __uint_as_float(r.f[0] << 16); x[1] = __uint_as_float(r.f[0] & 0xFFFF0000u);
  x[2] = __uint_as_float(r.f[1] << 16); x[3] = __uint_as_float(r.f[1] & 0xFFFF0000u);
}

template <bool kFull>
__device__ __forceinline__ void store4_f32(void* p, int64_t i, int n, const float (&x)[4]) {
  float* d = static_cast<float*>(p) + i;
  if (kFull) {
    __builtin_nontemporal_store(f4{x[0], x[1], x[2], x[3]}, reinterpret_cast<f4*>(d));
    return;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (k < n) d[k] = x[k];
}

template <bool kFull>
__device__ __forceinline__ void store4_u16(void* p, int64_t i, int n, uint32_t lo, uint32_t hi) {
  uint16_t* d = static_cast<uint16_t*>(p) + i;
  if (kFull) {
    __builtin_nontemporal_store(u2{lo, hi}, reinterpret_cast<u2*>(d));
    return;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (k < n) d[k] = (uint16_t)((k < 2 ? lo : hi) >> (16 * (k & 1)));
}

template <bool kFull>
__device__ __forceinline__ uint32_t load4_u8(const void* p, int64_t i, int n) {
  const uint8_t* s = static_cast<const uint8_t*>(p) + i;
  if (kFull) return __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(s));
  uint32_t v = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (k < n) v |= (uint32_t)s[k] << (8 * k);
  return v;
}

template <bool kFull>
__device__ __forceinline__ void store4_u8(void* p, int64_t i, int n, uint32_t v) {
  uint8_t* d = static_cast<uint8_t*>(p) + i;
  if (kFull) {
    __builtin_nontemporal_store(v, reinterpret_cast<uint32_t*>(d));
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

struct Step {
  float b1, b2, c1, c2, size, root2, decay, eps, gs;
  uint32_t key;
};

// What a thread reads of four elements.
template <bool kP32, bool kG32, bool kS8>
struct In {
  Raw4<kP32> p;
  Raw4<kG32> g;
  Raw4<true> m, v;         // fp32 states
  uint32_t mc, vc, ms, vs; // or codes and scales
};

template <bool kP32, bool kG32, bool kS8, bool kFull>
__device__ __forceinline__ void read(In<kP32, kG32, kS8>& in, const mx_adamw_tensor_t& t, int64_t i, int n) {
  in.p = load4<kP32, kFull>(t.param, i, n);
  in.g = load4<kG32, kFull>(t.grad, i, n);
  if constexpr (kS8) {
    in.mc = load4_u8<kFull>(t.m, i, n);
    in.vc = load4_u8<kFull>(t.v, i, n);
    in.ms = kFull || n ? t.m_scale[i >> 5] : 0u;
    in.vs = kFull || n ? t.v_scale[i >> 5] : 0u;
  } else {
    in.m = load4<true, kFull>(t.m, i, n);
    in.v = load4<true, kFull>(t.v, i, n);
  }
}

template <bool kP32, bool kG32, bool kS8, bool kFull>
__device__ __forceinline__ void update(const In<kP32, kG32, kS8>& in, const mx_adamw_tensor_t& t, int64_t i, int n,
                                       const Step& s) {
  float p[4], g[4], m[4], v[4], root[4];
  widen(in.p, p);
  widen(in.g, g);
  if constexpr (kS8) {
    decode4(in.mc, in.ms, m);
    decode4(in.vc, in.vs, v);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] *= v[k];
  } else {
    widen(in.m, m);
    widen(in.v, v);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float gk = g[k] * s.gs;
    m[k] = fmaf(s.b1, m[k], s.c1 * gk);
    v[k] = fmaf(s.b2, v[k], s.c2 * (gk * gk));
    // hardware root and reciprocal, each within a unit (exact ones cost the 8-bit
    // step 8% of its time)
    root[k] = __builtin_amdgcn_sqrtf(v[k]);
    p[k] = fmaf(-s.size, m[k] * __builtin_amdgcn_rcpf(fmaf(root[k], s.root2, s.eps)), p[k] * s.decay);
  }
  uint32_t h[4];
  if constexpr (kS8 || !kP32) {
#pragma unroll
    for (int k = 0; k < 4; ++k) h[k] = mix((s.key + (uint32_t)(i + k) * kGold) ^ (uint32_t)(i >> 32));
  }
  if constexpr (kS8) {
    uint32_t um[4], uv[4], bm, bv;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      um[k] = h[k] >> 16;
      uv[k] = h[k] & 0xFFFFu;
      if (!kFull && k >= n) m[k] = root[k] = 0.0f;   // not in the block
    }
    const uint32_t cm = encode4<false>(m, um, bm), cv = encode4<true>(root, uv, bv);
    store4_u8<kFull>(t.m, i, n, cm);
    store4_u8<kFull>(t.v, i, n, cv);
    if ((threadIdx.x & 7) == 0 && (kFull || n)) {
      t.m_scale[i >> 5] = (uint8_t)bm;
      t.v_scale[i >> 5] = (uint8_t)bv;
    }
  } else {
    store4_f32<kFull>(t.m, i, n, m);
    store4_f32<kFull>(t.v, i, n, v);
  }
  if constexpr (kP32) {
    store4_f32<kFull>(t.param, i, n, p);
    if (t.copy) store4_u16<kFull>(t.copy, i, n, bf16x2_rne(p[0], p[1]), bf16x2_rne(p[2], p[3]));
  } else {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = stochastic_bf16(p[k], mix(h[k] ^ kGold) >> 16);
    const uint32_t a = w[0] | (w[1] << 16), c = w[2] | (w[3] << 16);
    store4_u16<kFull>(t.param, i, n, a, c);
    if (t.copy) store4_u16<kFull>(t.copy, i, n, a, c);
  }
}

template <bool kP32, bool kG32, bool kS8>
__global__ void __launch_bounds__(kAdamThreads) k_adamw(Batch b, Hyper hp) {
  // the block's tensor: the last with first[i] <= blockIdx.x (one load, by lane)
  const int lane = threadIdx.x & 63;
  const bool at = lane < b.count && b.first[lane < kBatch ? lane : 0] <= (int)blockIdx.x;
  const int which = __builtin_amdgcn_readfirstlane(63 - __clzll((long long)__ballot(at)));
  const mx_adamw_tensor_t t = b.t[which];
  const int64_t begin = (int64_t)((int)blockIdx.x - b.first[which]) * kChunk;
  const int64_t i = begin + 4 * threadIdx.x;
  // a whole chunk, or the tensor's last one: there lanes past the end stay, so
  // that whole blocks of 32 reduce together
  const bool full = begin + kChunk <= t.n;
  const int n = full ? 4 : (i >= t.n ? 0 : (t.n - i < 4 ? (int)(t.n - i) : 4));
  In<kP32, kG32, kS8> in;
  if (full) read<kP32, kG32, kS8, true>(in, t, i, n);
  else read<kP32, kG32, kS8, false>(in, t, i, n);

  // the step's constants, by one wave (about a hundred fp64 operations)
  __shared__ Step shared;
  if (threadIdx.x < 64) {
    const int32_t st = *hp.step;
    const uint32_t step = st < 1 ? 1u : (uint32_t)st;
    const float lr = *hp.lr;
    Step c;
    c.gs = hp.grad_scale ? *hp.grad_scale : 1.0f;
    c.b1 = (float)hp.b1;
    c.b2 = (float)hp.b2;
    c.c1 = (float)(1.0 - hp.b1);
    c.c2 = (float)(1.0 - hp.b2);
    c.size = lr / (float)one_minus_pow(hp.b1, step);
    c.root2 = (float)(1.0 / sqrt(one_minus_pow(hp.b2, step)));
    c.decay = 1.0f - lr * hp.wd;
    c.eps = hp.eps;
    uint32_t key = mix(hp.seed_lo ^ kGold);
    key = mix(key ^ hp.seed_hi);
    key = mix(key ^ step);
    c.key = mix(key ^ (uint32_t)(b.base + which));
    if (threadIdx.x == 0) shared = c;
  }
  __syncthreads();
  const Step s = shared;

  if (full) update<kP32, kG32, kS8, true>(in, t, i, n, s);
  else update<kP32, kG32, kS8, false>(in, t, i, n, s);
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
  bool any = false;
  int64_t blocks = 0;   // of one launch
  for (int32_t i = 0; i < count; ++i) {
    if (i % kBatch == 0) blocks = 0;
    const mx_adamw_tensor_t& t = tensors[i];
    if (t.n < 0) return MX_EINVAL;
    if (t.n == 0) continue;
    if (!t.param || !t.grad || !t.m || !t.v) return MX_EINVAL;
    if (state_bits == 8 && (!t.m_scale || !t.v_scale)) return MX_EINVAL;
    // 16-byte accesses
    if (((uintptr_t)t.param | (uintptr_t)t.grad | (uintptr_t)t.m | (uintptr_t)t.v | (uintptr_t)t.copy) & 15)
      return MX_EINVAL;
    if (t.n >= (1ll << 40)) return MX_EUNSUPPORTED;
    blocks += (t.n + kChunk - 1) / kChunk;
    if (blocks * kAdamThreads >= (1ll << 32)) return MX_EUNSUPPORTED;   // threads of a launch
    any = true;
  }
  if (!any) return MX_OK;
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
    int64_t chunks = 0;
    for (int32_t i = 0; i < b.count; ++i) {
      b.t[i] = tensors[base + i];
      b.first[i] = (int32_t)chunks;
      chunks += (b.t[i].n + kChunk - 1) / kChunk;
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

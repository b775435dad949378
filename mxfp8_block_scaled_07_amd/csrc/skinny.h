// Products of weight rows with a few token rows (gfx950): the device code that
// the few-token layer and the single-token form of the bf16 product share.
//
//   acc[t][n] += sum_k x[t, k] w[n, k]
//
// With at most a few dozen tokens the weights are read once and used 2 T
// times per element, far below the matrix cores' ratio: the stream of weights
// from HBM bounds everything here, and the matrix instruction only keeps the
// arithmetic out of its way.  One wave takes 16 weight rows as the first
// operand and 16 token rows as the second of V_MFMA_F32_16X16X32_BF16, in
// steps of 128 k: lane (r = l & 15, h = l >> 4) loads the 32 consecutive
// elements k0 + 32 h .. + 31 of weight row r and of token row r, so a wave
// reads whole 128-byte lines of every fp8 row (256 bytes of a bf16 row), and
// the four instructions of a step use elements 8 i .. 8 i + 7 of each lane's
// 32.  (The order of k inside a dot product is free as long as both operands
// share it.)  The lane's 32 elements are exactly one MX block: its scale is
// one byte of the panel dword, and the codes become bf16 in registers
// (V_CVT_SCALEF32_PK_BF16_FP8; an E4M3 code times a power of two is exact in
// bf16), so MX weights are used unrounded and tokens stay in bf16.
//
// Result: lane l, register r holds weight row 4 (l >> 4) + r, token l & 15.
#pragma once

#include "mx_device.h"

namespace mx {

typedef __bf16 v8bf_s __attribute__((ext_vector_type(8)));
typedef float v4f_s __attribute__((ext_vector_type(4)));
typedef unsigned int v4u_s __attribute__((ext_vector_type(4)));

constexpr int kStepK = 128;                 // k elements of one step
constexpr uint32_t kNoRow = 0x80000000u;    // an offset past every buffer: reads as zero

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buf(const void* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}

__device__ __forceinline__ uint32_t step_uniform(uint32_t v) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)v); }

// One step's share of a lane: 32 weights of its row.
template <bool kMx>
struct WStep {
  v4u_s q[kMx ? 2 : 4];
  uint32_t s;   // kMx: the panel dword of the row
};

struct XStep {
  v4u_s q[4];   // 32 bf16 of the lane's token row
};

// Weight rows of one matrix as a wave reads them.
template <bool kMx>
struct WRows {
  __amdgpu_buffer_rsrc_t q, s;   // codes (or bf16) of the matrix; scales from the matrix's first row on
  uint32_t panel;                // bytes between scale panels
};

// row: the lane's weight row; k0 a multiple of 128.  Blocks past K read as
// zero (a whole step past K keeps the scalar offset inside the buffer).
template <bool kMx>
__device__ __forceinline__ void load_w(WStep<kMx>& w, const WRows<kMx>& m, uint32_t row, uint32_t K, uint32_t k0,
                                       bool row_ok) {
  const uint32_t h = (threadIdx.x & 63) >> 4;
  const bool ok = row_ok & (k0 + 32 * h < K);
  const uint32_t ks = k0 < K ? k0 : 0;
  if constexpr (kMx) {
    const uint32_t off = ok ? row * K + 32 * h : kNoRow;
    w.q[0] = __builtin_amdgcn_raw_buffer_load_b128(m.q, (int)off, (int)ks, 0);
    w.q[1] = __builtin_amdgcn_raw_buffer_load_b128(m.q, (int)off + 16, (int)ks, 0);
    w.s = __builtin_amdgcn_raw_buffer_load_b32(m.s, (int)(ok ? 4 * row : kNoRow), (int)((ks >> 7) * m.panel), 0);
  } else {
    const uint32_t off = ok ? 2 * (row * K + 32 * h) : kNoRow;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w.q[i] = __builtin_amdgcn_raw_buffer_load_b128(m.q, (int)off + 16 * i, (int)(2 * ks), 0);
  }
}

// off: byte offset of the lane's token row, or kNoRow for a lane without one.
__device__ __forceinline__ void load_x(XStep& x, __amdgpu_buffer_rsrc_t m, uint32_t off, uint32_t K, uint32_t k0) {
  const uint32_t h = (threadIdx.x & 63) >> 4;
  const bool ok = (k0 + 32 * h < K) & (off != kNoRow);
  const uint32_t o = ok ? off + 64 * h : kNoRow;
  const uint32_t ks = k0 < K ? k0 : 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) x.q[i] = __builtin_amdgcn_raw_buffer_load_b128(m, (int)o + 16 * i, (int)(2 * ks), 0);
}

// The lane's 8 weights of instruction i as bf16.
template <bool kMx>
__device__ __forceinline__ v8bf_s weights8(const WStep<kMx>& w, int i, float scale) {
  if constexpr (kMx) {
    const v4u_s& c = w.q[i >> 1];
    const uint32_t a = c[2 * (i & 1)], b = c[2 * (i & 1) + 1];
    const uint2 lo = cvt4_bf16(a, scale), hi = cvt4_bf16(b, scale);
    const v4u_s v = {lo.x, lo.y, hi.x, hi.y};
    return __builtin_bit_cast(v8bf_s, v);
  } else {
    return __builtin_bit_cast(v8bf_s, w.q[i]);
  }
}

template <bool kMx>
__device__ __forceinline__ float step_scale(const WStep<kMx>& w) {
  if constexpr (kMx) {
    const uint32_t h = (threadIdx.x & 63) >> 4;
    return e8m0_to_f32((w.s >> (8 * h)) & 0xFFu);
  }
  return 1.0f;
}

template <bool kMx>
__device__ __forceinline__ void mma_step(v4f_s& acc, const WStep<kMx>& w, const XStep& x) {
  const float scale = step_scale<kMx>(w);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(weights8<kMx>(w, i, scale), __builtin_bit_cast(v8bf_s, x.q[i]), acc,
                                                  0, 0, 0);
}

}  // namespace mx

// A stream of weight rows from HBM through LDS into matrix fragments (gfx950):
// what the few-token layer and the few-row form of the bf16 product share.
//
//   acc[t][n] += sum_k x[t, k] w[n, k]
//
// With a few tokens the weights are read once and used 2 T times per element,
// far below the matrix cores' ratio: the stream from HBM bounds everything.
// Non-temporal LDS-direct loads of whole 128-byte lines go into a ring of each
// wave's own, so that waiting needs no barrier and no registers.  A read-only
// stream of whole lines runs at 7.1 TB/s here non-temporally and at 6.3 TB/s
// otherwise, one of half lines (as matrix fragments loaded straight into
// registers) at 5.0 and 6.3.
//
// A wave's products: 16 weight rows as the first operand and 16 token rows as
// the second of V_MFMA_F32_16X16X32_BF16.  Of a 128-byte line of weight row r,
// lane (r = l & 15, h = l >> 4) takes the bytes 32 h .. 32 h + 31 and the same
// elements of token row r (the order of k inside a dot product is free as long
// as both operands share it).  For fp8 these are one MX block: its scale is one
// byte of the panel dword, and the codes become bf16 in registers (an E4M3 code
// times a power of two is exact in bf16), so weights are used unrounded and
// tokens stay in bf16.  Result: lane l, register r holds weight row
// 4 (l >> 4) + r, token l & 15.
#pragma once

#include "mx_device.h"

// The LDS-direct loads below set M0 in inline asm.
#pragma clang diagnostic ignored "-Winline-asm"

namespace mx {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef unsigned int v4u __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;

constexpr int kCus = 256;                // MI355X
constexpr uint32_t kOob = 0x80000000u;   // an offset that reads as zero

__device__ __forceinline__ v4u rsrc(const void* base, int64_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  const uint32_t n = bytes <= 0 ? 0u : (bytes > 0x7FFFFFFF ? 0x7FFFFFFFu : (uint32_t)bytes);
  return v4u{(uint32_t)a, (uint32_t)(a >> 32) & 0xFFFFu, n, 0x00020000u};
}

// The same for compiled loads.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buf(const void* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}

// LDS-direct loads of 16 (4) bytes per lane to LDS byte lds + 16 (4) lane.
// Inline asm, so that the compiler puts no wait of its own before LDS reads:
// every wait on these loads is an explicit vmcnt.
__device__ __forceinline__ void dma16(const v4u& r, uint32_t lds, uint32_t voff, uint32_t soff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :
               : "s"(lds), "v"(voff), "s"(r), "s"(soff)
               : "m0", "memory");
}
__device__ __forceinline__ void dma16_nt(const v4u& r, uint32_t lds, uint32_t voff, uint32_t soff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen nt lds"
               :
               : "s"(lds), "v"(voff), "s"(r), "s"(soff)
               : "m0", "memory");
}
__device__ __forceinline__ void dma4(const v4u& r, uint32_t lds, uint32_t voff, uint32_t soff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds"
               :
               : "s"(lds), "v"(voff), "s"(r), "s"(soff)
               : "m0", "memory");
}

__device__ __forceinline__ uint32_t uniform(uint32_t v) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)v); }

__device__ __forceinline__ uint32_t lds_addr(const void* p) { return (uint32_t)(uintptr_t)(const lds_void*)p; }

constexpr int waitcnt_vm(int n) { return (n & 0xF) | ((n >> 4) << 14) | (0x7 << 4) | (0xF << 8); }
constexpr int kWaitLgkm0 = 0xF | (0x3 << 14) | (0x7 << 4);

__device__ __forceinline__ void fence() { asm volatile("" ::: "memory"); }

// A workgroup barrier for LDS alone: the loads in flight go on.
__device__ __forceinline__ void lds_barrier() {
  fence();
  __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
  __builtin_amdgcn_s_barrier();
  fence();
}

// Elements of a 128-byte weight line.
template <bool kMx> constexpr int kLineK = kMx ? 128 : 64;
// 16-byte pieces of token elements that go with a lane's 32 weight bytes.
template <bool kMx> constexpr int kXp = kMx ? 4 : 2;

// A block of 16 weight rows x 128 bytes in LDS, its 16-byte chunks swizzled by
// row so that a fragment's reads fall on all banks.  Load q (0, 1) of it covers
// rows 8 q .. 8 q + 7: lane l holds row 8 q + l / 8.
__device__ __forceinline__ int chunk_swizzle(int r) { return (r >> 1) & 7; }

struct Fragment {
  uint4 lo, hi;   // the lane's 32 bytes
  uint32_t s;     // the panel dword of its row
};

// scales: the 16 rows' panel dwords (kMx)
template <bool kMx>
__device__ __forceinline__ Fragment read_fragment(const uint8_t* block, const uint8_t* scales) {
  const int lane = threadIdx.x & 63, r = lane & 15, h = lane >> 4, sw = chunk_swizzle(r);
  Fragment f;
  f.lo = *reinterpret_cast<const uint4*>(block + r * 128 + 16 * ((2 * h) ^ sw));
  f.hi = *reinterpret_cast<const uint4*>(block + r * 128 + 16 * ((2 * h + 1) ^ sw));
  f.s = kMx ? *reinterpret_cast<const uint32_t*>(scales + 4 * r) : 0u;
  return f;
}

// The lane's weights of instruction i as bf16.
template <bool kMx>
__device__ __forceinline__ v8bf weights8(const Fragment& f, int i, float scale) {
  if constexpr (kMx) {
    const uint4& c = i < 2 ? f.lo : f.hi;
    const uint2 a = cvt4_bf16((i & 1) ? c.z : c.x, scale), b = cvt4_bf16((i & 1) ? c.w : c.y, scale);
    return __builtin_bit_cast(v8bf, make_uint4(a.x, a.y, b.x, b.y));
  } else {
    return __builtin_bit_cast(v8bf, i == 0 ? f.lo : f.hi);
  }
}

template <bool kMx>
__device__ __forceinline__ float fragment_scale(const Fragment& f) {
  return kMx ? e8m0_to_f32((f.s >> (8 * ((threadIdx.x & 63) >> 4))) & 0xFFu) : 1.0f;
}

}  // namespace mx

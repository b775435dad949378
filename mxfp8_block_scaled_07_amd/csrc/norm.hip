// The root-mean-square norm in front of the expert layer, with the residual's
// addition and the MXFP8 rowwise quantize of its result fused in, and its
// backward (gfx950).
//
//   r = x + residual (rounded to the stream's type),  s = 1 / sqrt(mean(r^2) + eps)
//   y = RNE_bf16(r s w),  MX of y                     (w [cols])
//   dr = s (dy w - r s^2 mean(dy w r)) + dsum,  dw = sum_rows dy r s
//
// Both are HBM-bound streams: every element is read once, held in registers
// over the row's reduction, and written once.  A workgroup takes a row at a
// time, a thread 8 of its columns (N times 8 above 8192 columns), w of them in
// registers over all rows.  Sums are fp32 in a fixed order.

#include <type_traits>

#include "stream.h"
#include "tile_quant.h"

namespace mx {
namespace {

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

struct F8 {
  float v[8];
};

__device__ __forceinline__ F8 widen(const uint4& a) {
  return F8{{bf_lo(a.x), bf_hi(a.x), bf_lo(a.y), bf_hi(a.y), bf_lo(a.z), bf_hi(a.z), bf_lo(a.w), bf_hi(a.w)}};
}

__device__ __forceinline__ uint4 narrow(const F8& f) {
  return make_uint4(bf16x2_rne(f.v[0], f.v[1]), bf16x2_rne(f.v[2], f.v[3]), bf16x2_rne(f.v[4], f.v[5]),
                    bf16x2_rne(f.v[6], f.v[7]));
}

// A row of a tensor as a buffer: columns past its end load as zeros and are not
// stored, and a thread keeps one offset per chunk for all rows and tensors (as
// pointers and predicates these took more registers than the row itself).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_of(const void* p, int64_t r, int64_t row_bytes, bool ok) {
  return buf(static_cast<const uint8_t*>(p) + r * row_bytes, ok && p ? row_bytes : 0);
}

constexpr int kNt = 2;   // non-temporal: rows pass through once

__device__ __forceinline__ uint4 load16(__amdgpu_buffer_rsrc_t b, uint32_t at) {
  return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(b, (int)at, 0, kNt));
}

__device__ __forceinline__ void store16(__amdgpu_buffer_rsrc_t b, uint32_t at, const uint4& v) {
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4u, v), b, (int)at, 0, kNt);
}

// Keeps a row's bf16 packed over the reduction: widened before it, they would
// be held twice as large.
__device__ __forceinline__ void pin16(uint4& v) { asm volatile("" : "+v"(v.x), "+v"(v.y), "+v"(v.z), "+v"(v.w)); }

// 8 elements of the residual stream, bf16 or fp32, as they are stored; at: the
// offset of 8 bf16.
template <bool kF32> struct Raw;
template <> struct Raw<false> {
  uint4 a;
  __device__ void load(__amdgpu_buffer_rsrc_t b, uint32_t at) { a = load16(b, at); }
  __device__ void store(__amdgpu_buffer_rsrc_t b, uint32_t at) const { store16(b, at, a); }
  __device__ F8 value() const { return widen(a); }
  __device__ void set(const F8& f) { a = narrow(f); }
  __device__ void pin() { pin16(a); }
};
template <> struct Raw<true> {
  uint4 a, b;
  __device__ void load(__amdgpu_buffer_rsrc_t r, uint32_t at) {
    a = load16(r, 2 * at);
    b = load16(r, 2 * at + 16);
  }
  __device__ void store(__amdgpu_buffer_rsrc_t r, uint32_t at) const {
    store16(r, 2 * at, a);
    store16(r, 2 * at + 16, b);
  }
  __device__ F8 value() const {
    F8 f;
    __builtin_memcpy(f.v, &a, 16);
    __builtin_memcpy(f.v + 4, &b, 16);
    return f;
  }
  __device__ void set(const F8& f) {
    __builtin_memcpy(&a, f.v, 16);
    __builtin_memcpy(&b, f.v + 4, 16);
  }
  __device__ void pin() {}
};

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d, 64);
  return v;
}

// Sums over the workgroup, the same bits in each thread.  slot: one of two LDS
// slices in turn, so that one barrier per row is enough.
constexpr int kMaxWaves = 16;

template <int K>
__device__ __forceinline__ void row_sums(float (&v)[K], float (*slot)[K], int waves) {
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = wave_sum(v[k]);
  if (waves == 1) return;
  if ((threadIdx.x & 63) == 0) {
#pragma unroll
    for (int k = 0; k < K; ++k) slot[threadIdx.x >> 6][k] = v[k];
  }
  lds_barrier();   // the next row's loads stay in flight
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = 0.0f;
#pragma unroll
  for (int w = 0; w < kMaxWaves; ++w) {   // (waves that are not there left zeros)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += slot[w][k];
  }
}

template <int K>
__device__ __forceinline__ void clear_slots(float (*slots)[kMaxWaves][K]) {
  for (int i = threadIdx.x; i < 2 * kMaxWaves * K; i += blockDim.x) reinterpret_cast<float*>(slots)[i] = 0.0f;
  __syncthreads();
}

// The weights of a thread's chunks (1 without weights, 0 past the row's end).
template <int N>
__device__ __forceinline__ void load_weights(F8 (&w)[N], const float* weight, int64_t cols) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int64_t c = 8 * (int64_t)(threadIdx.x + blockDim.x * i);
#pragma unroll
    for (int k = 0; k < 8; ++k) w[i].v[k] = c < cols ? (weight ? weight[c + k] : 1.0f) : 0.0f;
  }
}

struct Norm {
  const uint16_t* x;       // bf16 [rows, cols] or null
  const void* residual;    // [rows, cols] of the stream's type or null
  const float* weight;
  int64_t rows, cols;
  float eps;
  void* sum;
  uint16_t* y;
  uint8_t* row_q;
  uint8_t* row_s;
};

// Workgroup b takes rows b, b + gridDim, ...: the card walks through the rows
// together, the next row on the way while one is finished (two rows ahead
// measure the same).  32768 x 7168 with every output: 370 us, 5.7 TB/s, 32768 x
// 4096 197 us, 6.2 TB/s (a copy reaches 6.6).  Rows above 16384 columns overflow the
// registers: by 6 of them, 61 with the fp32 stream, up to 32768 (5.5 and 4.3 TB/s
// there), by 218 and 316 above (2.9 and 1.9 TB/s at 65536).
template <int N, bool kF32>
__global__ void __launch_bounds__(1024) k_rmsnorm(const Norm p) {
  __shared__ float slots[2][kMaxWaves][1];
  const int T = blockDim.x, t = threadIdx.x, waves = T >> 6;
  if (waves > 1) clear_slots(slots);
  F8 w[N];
  load_weights<N>(w, p.weight, p.cols);
  const float inv_cols = 1.0f / (float)p.cols;

  uint4 rx[N];
  Raw<kF32> rr[N];
  auto load = [&](int64_t r) {
    const bool ok = r < p.rows;
    const __amdgpu_buffer_rsrc_t bx = row_of(p.x, r, 2 * p.cols, ok);
    const __amdgpu_buffer_rsrc_t br = row_of(p.residual, r, (kF32 ? 4 : 2) * p.cols, ok);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      rx[i] = load16(bx, 16u * (t + T * i));   // (without x or a residual: zeros)
      rr[i].load(br, 16u * (t + T * i));
    }
  };
  // workgroup b runs on XCD b % 8: each takes a run of the rows in work, so that the
  // lines of scales, 4 bytes of each of 32 rows, are written in one L2 (131072 x 512:
  // 96 us against 111; 32768 x 5120: 253 against 260)
  const uint32_t b = gridDim.x % 8 ? blockIdx.x : blockIdx.x % 8 * (gridDim.x / 8) + blockIdx.x / 8;
  load(b);
  int odd = 0;
  for (int64_t r = b; r < p.rows; r += gridDim.x, odd ^= 1) {
    const __amdgpu_buffer_rsrc_t bs = row_of(p.sum, r, (kF32 ? 4 : 2) * p.cols, true), by = row_of(p.y, r, 2 * p.cols, true);
    const __amdgpu_buffer_rsrc_t bq = row_of(p.row_q, r, p.cols, true);
    Raw<kF32> v[N];   // r as it is stored
    float ss[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < N; ++i) {
      F8 f = widen(rx[i]);
      if (p.residual) {
        const F8 a = rr[i].value();
#pragma unroll
        for (int k = 0; k < 8; ++k) f.v[k] = p.x ? f.v[k] + a.v[k] : a.v[k];   // (0 + -0 is no -0)
      }
      v[i].set(f);
      if (p.sum) v[i].store(bs, 16u * (t + T * i));
      f = v[i].value();
      float s[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) s[k] = f.v[k] * f.v[k];
      ss[0] += ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
    }
    load(r + gridDim.x);
    row_sums(ss, slots[odd], waves);
    const float s = rsqrtf(fmaf(ss[0], inv_cols, p.eps));
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int chunk = t + T * i;
      v[i].pin();
      F8 f = v[i].value();
#pragma unroll
      for (int k = 0; k < 8; ++k) f.v[k] = f.v[k] * s * w[i].v[k];
      // (past the row's end zeros, whatever s is: a quad of lanes is in or out)
      const uint4 o = 8 * chunk < p.cols ? narrow(f) : make_uint4(0, 0, 0, 0);
      if (p.y) store16(by, 16u * chunk, o);
      if (p.row_q) {
        // a quad of lanes holds a block, 16 lanes a panel of 4 blocks
        const uint32_t sb = scale_byte_from_amax(quad_max(amax8(o)));
        const float sc = e8m0_to_f32(sb);
        typedef unsigned int v2u __attribute__((ext_vector_type(2)));
        __builtin_amdgcn_raw_buffer_store_b64(v2u{cvt4_e4m3(o.x, o.y, sc), cvt4_e4m3(o.z, o.w, sc)}, bq, 8 * chunk, 0, kNt);
        const int ch = t & 15, panel = chunk >> 4;
        uint32_t d = sb << (8 * (ch >> 2));
        d |= dpp_row_shr(d, 4);
        d |= dpp_row_shr(d, 8);
        if (ch == 12 && 128 * (int64_t)panel < p.cols) reinterpret_cast<uint32_t*>(p.row_s)[(int64_t)panel * p.rows + r] = d;
      }
    }
  }
}

struct NormBwd {
  const uint16_t* dy;
  const void* sum;
  const void* dsum;
  const float* weight;
  int64_t rows, cols;
  float eps;
  void* dres;
  uint16_t* dx;
  float* part;             // [workgroups, cols] or null
};

// The same walk; a thread adds up its columns of dw over the workgroup's rows, and
// k_norm_join the workgroups' sums.  32768 x 7168 with dsum: 298 us, 6.3 TB/s.  Rows
// above 16384 columns, 8192 with the fp32 stream, overflow the registers: the latter
// by 20 up to 16384 (3.9 TB/s there), both by 144 to 194 up to 32768 (1.7 TB/s) and by
// 526 and 701 above (0.7 and 0.9 TB/s at 65536).
template <int N, bool kF32>
__global__ void __launch_bounds__(1024) k_rmsnorm_bwd(const NormBwd p) {
  __shared__ float slots[2][kMaxWaves][2];
  const int T = blockDim.x, t = threadIdx.x, waves = T >> 6;
  if (waves > 1) clear_slots(slots);
  F8 w[N], dw[N];
  load_weights<N>(w, p.weight, p.cols);
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) dw[i].v[k] = 0.0f;
  const float inv_cols = 1.0f / (float)p.cols;

  uint4 nd[N];
  Raw<kF32> nr[N], ns[N];
  auto load = [&](int64_t r) {
    const bool ok = r < p.rows;
    const int64_t bytes = (kF32 ? 4 : 2) * p.cols;
    const __amdgpu_buffer_rsrc_t br = row_of(p.sum, r, bytes, ok), bd = row_of(p.dy, r, 2 * p.cols, ok);
    const __amdgpu_buffer_rsrc_t bs = row_of(p.dsum, r, bytes, ok);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      nr[i].load(br, 16u * (t + T * i));
      nd[i] = load16(bd, 16u * (t + T * i));
      ns[i].load(bs, 16u * (t + T * i));   // (without one: zeros)
    }
  };
  load(blockIdx.x);
  int odd = 0;
  for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x, odd ^= 1) {
    uint4 rd[N];
    Raw<kF32> rr[N], rs[N];
    float s2[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < N; ++i) {
      rr[i] = nr[i];
      rd[i] = nd[i];
      rs[i] = ns[i];
      const F8 a = rr[i].value(), d = widen(rd[i]);
      float s[8], h[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        s[k] = a.v[k] * a.v[k];
        h[k] = d.v[k] * w[i].v[k] * a.v[k];
      }
      s2[0] += ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
      s2[1] += ((h[0] + h[1]) + (h[2] + h[3])) + ((h[4] + h[5]) + (h[6] + h[7]));
    }
    load(r + gridDim.x);
    row_sums(s2, slots[odd], waves);
    const float s = rsqrtf(fmaf(s2[0], inv_cols, p.eps));
    const float m = s * s * (s2[1] * inv_cols);
    const __amdgpu_buffer_rsrc_t bo = row_of(p.dres, r, (kF32 ? 4 : 2) * p.cols, true), bx = row_of(p.dx, r, 2 * p.cols, true);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      rr[i].pin();
      pin16(rd[i]);
      const F8 a = rr[i].value(), d = widen(rd[i]), e = rs[i].value();
      F8 o;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        o.v[k] = s * fmaf(-m, a.v[k], d.v[k] * w[i].v[k]) + e.v[k];
        dw[i].v[k] = fmaf(d.v[k], a.v[k] * s, dw[i].v[k]);
      }
      if (p.dres) {
        Raw<kF32> x;
        x.set(o);
        x.store(bo, 16u * (t + T * i));
      }
      if (p.dx) store16(bx, 16u * (t + T * i), narrow(o));
    }
  }
  if (!p.part) return;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int64_t c = 8 * (int64_t)(t + T * i);
    if (c < p.cols) {
      float4* o = reinterpret_cast<float4*>(p.part + (int64_t)blockIdx.x * p.cols + c);
      o[0] = make_float4(dw[i].v[0], dw[i].v[1], dw[i].v[2], dw[i].v[3]);
      o[1] = make_float4(dw[i].v[4], dw[i].v[5], dw[i].v[6], dw[i].v[7]);
    }
  }
}

// dweight from the workgroups' sums: 32 columns per workgroup, 32 threads to a
// column, each a run of partial sums in order, then the runs in order.
__global__ void __launch_bounds__(1024) k_norm_join(const float* __restrict__ part, int32_t blocks, int64_t cols,
                                                    float* __restrict__ dweight) {
  __shared__ float sum[32][33];
  const int c = threadIdx.x & 31, run = threadIdx.x >> 5;
  const int64_t j = 32 * (int64_t)blockIdx.x + c;   // cols % 32 == 0: always a column
  const int per = (blocks + 31) / 32;
  const int b1 = (run + 1) * per < blocks ? (run + 1) * per : blocks;
  float t = 0.0f;
#pragma unroll 8
  for (int b = run * per; b < b1; ++b) t += part[b * cols + j];
  sum[run][c] = t;
  __syncthreads();
  if (run == 0) {
    for (int r = 1; r < 32; ++r) t += sum[r][c];
    dweight[j] = t;
  }
}

// ---------------------------------------------------------------- host side
constexpr int64_t kMaxCols = 65536;

// Chunks per thread and threads of a row.  Two chunks to a thread above 4096
// columns (backward at 32768 x 7168: 299 us, with one 319), but for the fp32
// stream's backward, whose registers they overflow (911 us, with one 674).
struct Split {
  int n, threads;
};

Split split_row(int64_t cols, bool f32_bwd) {
  const int64_t chunks = cols / 8;
  int n = 1;
  while ((n == 1 && !f32_bwd ? 512 : 1024) * n < chunks) n *= 2;
  return Split{n, (int)((chunks + 64 * n - 1) / (64 * n) * 64)};
}

// Workgroups for rows that move `bytes` an element: few rows in work, near each
// other, 40 KB to a CU.  32768 x 7168, backward with dsum (8 bytes): 298 us with
// one per CU, 345 with two; 32768 x 4096, x to y (4 bytes): 89 us with two, 124
// with one; 131072 x 512 with all outputs (9 bytes): 97 us with 9, 139 with 4.  (A row
// takes a wave at least: of 128 columns 16 lanes of 64 are at work, 524288 x 128 takes
// 155 us, 3.9 TB/s; 262144 x 256 takes 105, 5.8 TB/s.)
int32_t blocks_for(int64_t rows, int64_t cols, int64_t bytes) {
  const int64_t row = bytes * cols / 8;
  const int64_t per_cu = (5000 + row / 2) / row;
  const int64_t most = kCus * (per_cu < 1 ? 1 : per_cu);
  return (int32_t)(rows < most ? rows : most);
}

template <int N, typename F>
int with_stream(bool f32, F f) {
  return f32 ? f(std::integral_constant<int, N>(), std::true_type()) : f(std::integral_constant<int, N>(), std::false_type());
}

template <typename F>
int dispatch(int n, bool f32, F f) {
  switch (n) {
    case 1: return with_stream<1>(f32, f);
    case 2: return with_stream<2>(f32, f);
    case 4: return with_stream<4>(f32, f);
    default: return with_stream<8>(f32, f);
  }
}

inline bool misaligned(const void* p, uintptr_t a) { return p && (reinterpret_cast<uintptr_t>(p) & (a - 1)); }

// Arguments both directions share.
int check(int32_t stream_dtype, const float* weight, int64_t rows, int64_t cols, double eps) {
  if (stream_dtype != MX_OUT_BF16 && stream_dtype != MX_OUT_F32) return MX_EINVAL;
  if (rows < 0 || cols <= 0 || cols % 32 || !(eps >= 1e-37) || eps > 1e30 || misaligned(weight, 4)) return MX_EINVAL;
  if (cols > kMaxCols || rows >= (1ll << 31)) return MX_EUNSUPPORTED;
  return MX_OK;
}

}  // namespace
}  // namespace mx

using namespace mx;

extern "C" int mx_rmsnorm(const uint16_t* x, const void* residual, int32_t stream_dtype, const float* weight,
                          int64_t rows, int64_t cols, double eps, void* sum, uint16_t* y, uint8_t* row_q,
                          uint8_t* row_s, mx_stream_t stream) {
  const int rc = check(stream_dtype, weight, rows, cols, eps);
  if (rc == MX_EINVAL) return rc;
  if ((!x && !residual) || (row_q == nullptr) != (row_s == nullptr) || (!sum && !y && !row_q)) return MX_EINVAL;
  if (misaligned(x, 16) || misaligned(residual, 16) || misaligned(sum, 16) || misaligned(y, 16) ||
      misaligned(row_q, 8) || misaligned(row_s, 4))
    return MX_EINVAL;
  if (rc != MX_OK || rows == 0) return rc;
  const Split s = split_row(cols, false);
  const Norm p{x, residual, weight, rows, cols, (float)eps, sum, y, row_q, row_s};
  const int64_t wide = stream_dtype == MX_OUT_F32 ? 4 : 2;
  const dim3 grid((unsigned)blocks_for(rows, cols, (x ? 2 : 0) + (residual ? wide : 0) + (sum ? wide : 0) + (y ? 2 : 0) + (row_q ? 1 : 0)));
  return dispatch(s.n, stream_dtype == MX_OUT_F32, [&](auto n, auto f32) {
    hipLaunchKernelGGL((k_rmsnorm<decltype(n)::value, decltype(f32)::value>), grid, dim3(s.threads), 0,
                       reinterpret_cast<hipStream_t>(stream), p);
    return launch_status();
  });
}

extern "C" size_t mx_rmsnorm_bwd_workspace_size(int64_t rows, int64_t cols) {
  if (rows <= 0 || check(MX_OUT_BF16, nullptr, rows, cols, 1.0) != MX_OK) return 0;
  return (size_t)(blocks_for(rows, cols, 6) * cols * 4);   // (the most workgroups: bf16 without dsum)
}

extern "C" int mx_rmsnorm_bwd(const uint16_t* dy, const void* sum, const void* dsum, int32_t stream_dtype,
                              const float* weight, int64_t rows, int64_t cols, double eps, void* dres, uint16_t* dx,
                              float* dweight, void* workspace, size_t workspace_bytes, mx_stream_t stream) {
  const int rc = check(stream_dtype, weight, rows, cols, eps);
  if (rc == MX_EINVAL) return rc;
  if (!dy || !sum || (!dres && !dx && !dweight)) return MX_EINVAL;
  if (misaligned(dy, 16) || misaligned(sum, 16) || misaligned(dsum, 16) || misaligned(dres, 16) || misaligned(dx, 16) ||
      misaligned(dweight, 4) || misaligned(workspace, 16))
    return MX_EINVAL;
  if (rc != MX_OK) return rc;
  const hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (dweight && rows > 0 && (!workspace || workspace_bytes < mx_rmsnorm_bwd_workspace_size(rows, cols))) return MX_EINVAL;
  int32_t blocks = 0;
  if (rows > 0) {
    const Split s = split_row(cols, stream_dtype == MX_OUT_F32);
    // (whatever outputs are asked for: dweight keeps its bits)
    const int64_t wide = stream_dtype == MX_OUT_F32 ? 4 : 2;
    blocks = blocks_for(rows, cols, 2 + wide * (dsum ? 3 : 2));
    const NormBwd p{dy, sum, dsum, weight, rows, cols, (float)eps, dres, dx, dweight ? static_cast<float*>(workspace) : nullptr};
    const int launched = dispatch(s.n, stream_dtype == MX_OUT_F32, [&](auto n, auto f32) {
      hipLaunchKernelGGL((k_rmsnorm_bwd<decltype(n)::value, decltype(f32)::value>), dim3((unsigned)blocks),
                         dim3(s.threads), 0, st, p);
      return launch_status();
    });
    if (launched != MX_OK) return launched;
  }
  if (!dweight) return MX_OK;
  hipLaunchKernelGGL(k_norm_join, dim3((unsigned)(cols / 32)), dim3(1024), 0, st,
                     static_cast<const float*>(workspace), blocks, cols, dweight);
  return launch_status();
}

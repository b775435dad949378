// The root-mean-square norm in front of the expert layer, with the residual's
// addition and the MXFP8 rowwise quantize of its result fused in, and its
// backward (gfx950).
//
//   r = x + residual (rounded to the stream's type),  s = 1 / sqrt(mean(r^2) + eps)
//   y = RNE_bf16(r s w),  MX of y                     (w [cols])
//   dr = s (dy w - r s^2 mean(dy w r)) + dsum,  dw = sum_rows dy r s
//
// Both are HBM-bound streams: every element is read once, held in registers
// over the row's reduction, and written once.  G threads share a row, a thread
// holds N chunks of 8 columns (chunk t + G i), w of its columns in registers
// over all rows of its workgroup.  Sums are fp32 in a fixed order.

#include <type_traits>

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

// 8 elements of the residual stream, bf16 or fp32, as they are loaded.
template <bool kF32> struct Raw;
template <> struct Raw<false> {
  uint4 a;
  __device__ void load(const void* p, int64_t at) { a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at); }
  __device__ F8 value() const { return widen(a); }
};
template <> struct Raw<true> {
  float4 a, b;
  __device__ void load(const void* p, int64_t at) {
    const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
    a = f[0];
    b = f[1];
  }
  __device__ F8 value() const { return F8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}}; }
};

template <bool kF32>
__device__ __forceinline__ void store_stream(void* p, int64_t at, const F8& f) {
  if constexpr (kF32) {
    float4* o = reinterpret_cast<float4*>(static_cast<float*>(p) + at);
    o[0] = make_float4(f.v[0], f.v[1], f.v[2], f.v[3]);
    o[1] = make_float4(f.v[4], f.v[5], f.v[6], f.v[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + at) = narrow(f);
  }
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d, 64);
  return v;
}

// Sums over the G threads of a row, the same bits in each of them.  slot: one
// of two LDS slices in turn, so that one barrier per row is enough.
template <int G, int K>
__device__ __forceinline__ void row_sums(float (&v)[K], float* slot) {
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = wave_sum(v[k]);
  if constexpr (G > 64) {
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    if (lane == 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) slot[wave * K + k] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float t = 0.0f;
#pragma unroll
      for (int w = 0; w < G / 64; ++w) t += slot[w * K + k];
      v[k] = t;
    }
  }
}

template <int G> constexpr int kThreads = G < 256 ? 256 : G;
template <int G> constexpr int kGroups = kThreads<G> / G;   // rows in work at once

// The columns' weights of a thread's chunks (1 without weights, 0 past the row's end).
template <int G, int N>
__device__ __forceinline__ void load_weights(F8 (&w)[N], const float* weight, int t, int64_t cols) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int64_t c = 8 * (int64_t)(t + G * i);
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
  int32_t band;            // rows per workgroup
  bool staged;             // scales go through LDS
};

template <int G, int N, bool kF32>
__global__ void __launch_bounds__(kThreads<G>) k_rmsnorm(const Norm p) {
  extern __shared__ uint32_t panels[];   // [ceil(cols / 128)][band] panel dwords
  __shared__ float slots[2][kThreads<G> / 64];
  const int g = threadIdx.x / G, t = threadIdx.x % G;
  const int64_t r0 = (int64_t)blockIdx.x * p.band;
  const int32_t band = p.rows - r0 < p.band ? (int32_t)(p.rows - r0) : p.band;
  F8 w[N];
  load_weights<G, N>(w, p.weight, t, p.cols);
  const float inv_cols = 1.0f / (float)p.cols;

  for (int32_t j = 0; j < band; j += kGroups<G>) {
    const bool ok = j + g < band;
    const int64_t r = r0 + j + g;
    uint4 rx[N];
    Raw<kF32> rr[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int64_t c = 8 * (int64_t)(t + G * i);
      if (ok && c < p.cols) {
        if (p.x) rx[i] = *reinterpret_cast<const uint4*>(p.x + r * p.cols + c);
        if (p.residual) rr[i].load(p.residual, r * p.cols + c);
      }
    }
    F8 v[N];
    float ss[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int64_t c = 8 * (int64_t)(t + G * i);
      if (ok && c < p.cols) {
        if (p.x) v[i] = widen(rx[i]);
        if (p.residual) {
          const F8 a = rr[i].value();
#pragma unroll
          for (int k = 0; k < 8; ++k) v[i].v[k] = p.x ? v[i].v[k] + a.v[k] : a.v[k];
          if constexpr (!kF32) v[i] = widen(narrow(v[i]));   // the norm is of the stored value
        }
        if (p.sum) store_stream<kF32>(p.sum, r * p.cols + c, v[i]);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[i].v[k] = 0.0f;
      }
      float q[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) q[k] = v[i].v[k] * v[i].v[k];
      ss[0] += ((q[0] + q[1]) + (q[2] + q[3])) + ((q[4] + q[5]) + (q[6] + q[7]));
    }
    row_sums<G>(ss, slots[(j / kGroups<G>) & 1]);
    const float s = rsqrtf(fmaf(ss[0], inv_cols, p.eps));
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int64_t c = 8 * (int64_t)(t + G * i);
      const bool in = ok && c < p.cols;
      F8 f;
#pragma unroll
      for (int k = 0; k < 8; ++k) f.v[k] = v[i].v[k] * s * w[i].v[k];
      // (past the row's end or the band's: zeros, whatever s is)
      const uint4 o = in ? narrow(f) : make_uint4(0, 0, 0, 0);
      if (p.y && in) *reinterpret_cast<uint4*>(p.y + r * p.cols + c) = o;
      if (p.row_q) {
        // a quad of lanes holds a block, 16 lanes a panel of 4 blocks
        const uint32_t sb = scale_byte_from_amax(quad_max(amax8(o)));
        const float sc = e8m0_to_f32(sb);
        if (in) *reinterpret_cast<uint2*>(p.row_q + r * p.cols + c) = make_uint2(cvt4_e4m3(o.x, o.y, sc), cvt4_e4m3(o.z, o.w, sc));
        const int ch = threadIdx.x & 15;
        uint32_t d = sb << (8 * (ch >> 2));
        d |= dpp_row_shr(d, 4);
        d |= dpp_row_shr(d, 8);
        const int32_t panel = (t + G * i) >> 4;
        if (ok && ch == 12 && 128 * (int64_t)panel < p.cols) {
          if (p.staged) panels[panel * p.band + j + g] = d;
          else reinterpret_cast<uint32_t*>(p.row_s)[(int64_t)panel * p.rows + r] = d;
        }
      }
    }
  }
  if (p.row_q && p.staged) {
    __syncthreads();
    const int32_t n = (int32_t)((p.cols + 127) / 128) * p.band;
    for (int32_t e = threadIdx.x; e < n; e += kThreads<G>) {
      const int32_t panel = e / p.band, j = e % p.band;
      if (j < band) reinterpret_cast<uint32_t*>(p.row_s)[(int64_t)panel * p.rows + r0 + j] = panels[e];
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
  int32_t band;            // rows per workgroup
};

template <int G, int N, bool kF32>
__global__ void __launch_bounds__(kThreads<G>) k_rmsnorm_bwd(const NormBwd p) {
  __shared__ float slots[2][2 * kThreads<G> / 64];
  __shared__ float cols_sum[kGroups<G> > 1 ? kGroups<G> - 1 : 1][kGroups<G> > 1 ? 8 * G * N : 1];
  const int g = threadIdx.x / G, t = threadIdx.x % G;
  const int64_t r0 = (int64_t)blockIdx.x * p.band;
  const int32_t band = p.rows - r0 < p.band ? (int32_t)(p.rows - r0) : p.band;
  F8 w[N], dw[N];
  load_weights<G, N>(w, p.weight, t, p.cols);
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) dw[i].v[k] = 0.0f;
  const float inv_cols = 1.0f / (float)p.cols;

  for (int32_t j = 0; j < band; j += kGroups<G>) {
    const bool ok = j + g < band;
    const int64_t r = r0 + j + g;
    uint4 rd[N];
    Raw<kF32> rr[N], rs[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int64_t c = 8 * (int64_t)(t + G * i);
      if (ok && c < p.cols) {
        rr[i].load(p.sum, r * p.cols + c);
        rd[i] = *reinterpret_cast<const uint4*>(p.dy + r * p.cols + c);
        if (p.dsum) rs[i].load(p.dsum, r * p.cols + c);
      }
    }
    float s2[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int64_t c = 8 * (int64_t)(t + G * i);
      if (ok && c < p.cols) {
        const F8 a = rr[i].value(), d = widen(rd[i]);
        float q[8], h[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          q[k] = a.v[k] * a.v[k];
          h[k] = d.v[k] * w[i].v[k] * a.v[k];
        }
        s2[0] += ((q[0] + q[1]) + (q[2] + q[3])) + ((q[4] + q[5]) + (q[6] + q[7]));
        s2[1] += ((h[0] + h[1]) + (h[2] + h[3])) + ((h[4] + h[5]) + (h[6] + h[7]));
      }
    }
    row_sums<G>(s2, slots[(j / kGroups<G>) & 1]);
    const float s = rsqrtf(fmaf(s2[0], inv_cols, p.eps));
    const float m = s * s * (s2[1] * inv_cols);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int64_t c = 8 * (int64_t)(t + G * i);
      if (ok && c < p.cols) {
        const F8 a = rr[i].value(), d = widen(rd[i]);
        F8 o;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          o.v[k] = s * fmaf(-m, a.v[k], d.v[k] * w[i].v[k]);
          dw[i].v[k] = fmaf(d.v[k], a.v[k] * s, dw[i].v[k]);
        }
        if (p.dsum) {
          const F8 e = rs[i].value();
#pragma unroll
          for (int k = 0; k < 8; ++k) o.v[k] += e.v[k];
        }
        if (p.dres) store_stream<kF32>(p.dres, r * p.cols + c, o);
        if (p.dx) *reinterpret_cast<uint4*>(p.dx + r * p.cols + c) = narrow(o);
      }
    }
  }
  if (!p.part) return;
  // the row groups' sums in order, then one row of partial sums per workgroup
  if constexpr (kGroups<G> > 1) {
    if (g > 0) {
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) cols_sum[g - 1][k * G * N + t + G * i] = dw[i].v[k];
    }
    __syncthreads();
    if (g > 0) return;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k)
#pragma unroll
        for (int o = 0; o < kGroups<G> - 1; ++o) dw[i].v[k] += cols_sum[o][k * G * N + t + G * i];
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int64_t c = 8 * (int64_t)(t + G * i);
    if (c < p.cols) store_stream<true>(p.part, (int64_t)blockIdx.x * p.cols + c, dw[i]);
  }
}

// dweight from the workgroups' sums: 16 columns per workgroup, 16 threads to a
// column, each a run of partial sums in order, then the runs in order.
__global__ void __launch_bounds__(256) k_norm_join(const float* __restrict__ part, int32_t blocks, int64_t cols,
                                                   float* __restrict__ dweight) {
  __shared__ float sum[16][17];
  const int c = threadIdx.x & 15, run = threadIdx.x >> 4;
  const int64_t j = 16 * (int64_t)blockIdx.x + c;   // cols % 32 == 0: always a column
  const int per = (blocks + 15) / 16;
  const int b1 = (run + 1) * per < blocks ? (run + 1) * per : blocks;
  float t = 0.0f;
#pragma unroll 8
  for (int b = run * per; b < b1; ++b) t += part[b * cols + j];
  sum[run][c] = t;
  __syncthreads();
  if (run == 0) {
    for (int r = 1; r < 16; ++r) t += sum[r][c];
    dweight[j] = t;
  }
}

// ---------------------------------------------------------------- host side
constexpr int64_t kMaxCols = 65536;
constexpr int kCus = 256;   // MI355X

// Threads per row (64, 256, 1024) and chunks per thread.
struct Split {
  int g, n;
};

Split split_row(int64_t rows, int64_t cols) {
  const int64_t chunks = (cols + 7) / 8;
  int g = chunks <= 4 * 64 ? 64 : chunks <= 4 * 256 ? 256 : 1024;
  // few rows: more threads to each
  while (g < 1024 && chunks > g && rows * g < 1024 * (int64_t)kCus) g *= 4;
  int n = 1;
  while (n * g < chunks) n *= 2;
  return Split{g, n};
}

int32_t bwd_band(int64_t rows, const Split& s) {
  const int groups = s.g < 256 ? 256 / s.g : 1;
  const int64_t want = (int64_t)kCus * (s.g == 1024 ? 1 : 3);
  int64_t band = (rows + want - 1) / want;
  band = (band + groups - 1) / groups * groups;
  return (int32_t)band;
}

template <int G, int N, typename F>
int with_stream(bool f32, F f) {
  return f32 ? f(std::integral_constant<int, G>(), std::integral_constant<int, N>(), std::true_type())
             : f(std::integral_constant<int, G>(), std::integral_constant<int, N>(), std::false_type());
}

template <typename F>
int dispatch(const Split& s, bool f32, F f) {
  switch (s.g * 16 + s.n) {
    case 64 * 16 + 1: return with_stream<64, 1>(f32, f);
    case 64 * 16 + 2: return with_stream<64, 2>(f32, f);
    case 64 * 16 + 4: return with_stream<64, 4>(f32, f);
    case 256 * 16 + 1: return with_stream<256, 1>(f32, f);
    case 256 * 16 + 2: return with_stream<256, 2>(f32, f);
    case 256 * 16 + 4: return with_stream<256, 4>(f32, f);
    case 1024 * 16 + 1: return with_stream<1024, 1>(f32, f);
    case 1024 * 16 + 2: return with_stream<1024, 2>(f32, f);
    case 1024 * 16 + 4: return with_stream<1024, 4>(f32, f);
    default: return with_stream<1024, 8>(f32, f);
  }
}

inline bool misaligned(const void* p, uintptr_t a) { return p && (reinterpret_cast<uintptr_t>(p) & (a - 1)); }

// Arguments both directions share.
int check(int32_t stream_dtype, const float* weight, int64_t rows, int64_t cols, double eps) {
  if (stream_dtype != MX_OUT_BF16 && stream_dtype != MX_OUT_F32) return MX_EINVAL;
  if (rows < 0 || cols <= 0 || cols % 32 || !(eps > 0.0) || eps > 1e30 || misaligned(weight, 4)) return MX_EINVAL;
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
  const Split s = split_row(rows, cols);
  Norm p{x, residual, weight, rows, cols, (float)eps, sum, y, row_q, row_s, 1, false};
  const int groups = s.g < 256 ? 256 / s.g : 1;
  // bands of up to 32 rows, so that a panel's scales leave as whole lines, while the card is filled
  int64_t band = (rows + 8 * kCus - 1) / (8 * kCus);
  band = band > 32 ? 32 : (band + groups - 1) / groups * groups;
  p.band = (int32_t)band;
  p.staged = row_q && band > groups;
  const size_t lds = p.staged ? (size_t)((cols + 127) / 128) * band * 4 : 0;
  const dim3 grid((unsigned)((rows + band - 1) / band));
  return dispatch(s, stream_dtype == MX_OUT_F32, [&](auto g, auto n, auto f32) {
    constexpr int G = decltype(g)::value, N = decltype(n)::value;
    hipLaunchKernelGGL((k_rmsnorm<G, N, decltype(f32)::value>), grid, dim3(kThreads<G>), lds,
                       reinterpret_cast<hipStream_t>(stream), p);
    return launch_status();
  });
}

extern "C" size_t mx_rmsnorm_bwd_workspace_size(int64_t rows, int64_t cols) {
  if (rows <= 0 || check(MX_OUT_BF16, nullptr, rows, cols, 1.0) != MX_OK) return 0;
  const int32_t band = bwd_band(rows, split_row(rows, cols));
  return (size_t)((rows + band - 1) / band * cols * 4);
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
    const Split s = split_row(rows, cols);
    NormBwd p{dy, sum, dsum, weight, rows, cols, (float)eps, dres, dx, dweight ? static_cast<float*>(workspace) : nullptr,
              bwd_band(rows, s)};
    blocks = (int32_t)((rows + p.band - 1) / p.band);
    const int launched = dispatch(s, stream_dtype == MX_OUT_F32, [&](auto g, auto n, auto f32) {
      constexpr int G = decltype(g)::value, N = decltype(n)::value;
      hipLaunchKernelGGL((k_rmsnorm_bwd<G, N, decltype(f32)::value>), dim3((unsigned)blocks), dim3(kThreads<G>), 0, st, p);
      return launch_status();
    });
    if (launched != MX_OK) return launched;
  }
  if (!dweight) return MX_OK;
  hipLaunchKernelGGL(k_norm_join, dim3((unsigned)(cols / 16)), dim3(256), 0, st,
                     static_cast<const float*>(workspace), blocks, cols, dweight);
  return launch_status();
}

// The dense bf16 product with an epilogue, and its backward (gfx950):
//
//   z = x w^T + bias,  out = act(z) + residual            (x [M, K], w [N, K])
//   dz = dout act'(z), dx = dz w (+ dx_add), dw = dz^T x, dbias = sum_m dz
//
// All three products run in the tiles of product.h.
//
// Up to 16 rows the forward streams w once through the code of stream.h.

#include "few_rows.h"
#include "product.h"

namespace mx {
namespace {

// ---------------------------------------------------------------- activations
// e^x for x <= 0 by the hardware's 2^x: its relative error grows with |x| (the
// rounding of x log2 e), its absolute error |x| e^x 2^-24 stays below a unit of
// the sums it goes into.
__device__ __forceinline__ float exp_neg(float x) { return __builtin_amdgcn_exp2f(x * 1.4426950408889634f); }

// sigmoid(x) and sigmoid(-x) from e^-|x| in (0, 1]: neither is a difference.
// 1 + e lies in (1, 2], where the hardware reciprocal is within a unit.
__device__ __forceinline__ float sigmoid2(float x, float& minus) {
  const float e = exp_neg(-fabsf(x));
  const float r = __builtin_amdgcn_rcpf(1.0f + e), q = e * r;
  minus = x >= 0.0f ? q : r;
  return x >= 0.0f ? r : q;
}

__device__ __forceinline__ float sigmoid(float x) {
  float m;
  return sigmoid2(x, m);
}

// Phi(z) of gelu, g = e^(-z^2 / 2): 1 + erf(z / sqrt 2) would cancel for negative
// z (one rounding of that sum is 10% of the value at z = -5), so the tail below
// -|z| is formed by itself, as g t P(t) with t = 1 / (1 + 0.34 |z|).  P: the
// polynomial with the least largest relative error over |z| <= 14 (half a unit;
// with the fp32 arithmetic six), beyond which g is 0.  8192 x 8192 x 64 takes 71
// us, 105 with erfcf in its place (1 + erff: 79).
__device__ __forceinline__ float normal_cdf(float z, float g) {
  const float t = __builtin_amdgcn_rcpf(fmaf(0.34f, fabsf(z), 1.0f));
  float y = -0.026120487600564957f;
  y = fmaf(y, t, 0.13949955999851227f);
  y = fmaf(y, t, -0.27313289046287537f);
  y = fmaf(y, t, 0.2021828293800354f);
  y = fmaf(y, t, -0.044718559831380844f);
  y = fmaf(y, t, 0.11535920947790146f);
  y = fmaf(y, t, 0.11519765108823776f);
  y = fmaf(y, t, 0.13611219823360443f);
  y = fmaf(y, t, 0.13562050461769104f);
  const float q = g * (t * y);
  return z < 0.0f ? q : 1.0f - q;
}

constexpr float kGeluC = 0.7978845608028654f;   // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

__device__ __forceinline__ float act_value(float z, int act) {
  switch (act) {
    case MX_ACT_RELU: return z > 0.0f ? z : (z == z ? 0.0f : z);
    case MX_ACT_GELU: return z * normal_cdf(z, exp_neg(-0.5f * z * z));
    // 0.5 (1 + tanh(y)) = sigmoid(2 y)
    case MX_ACT_GELU_TANH: return z * sigmoid(2.0f * kGeluC * (z + kGeluA * z * z * z));
    case MX_ACT_SILU: return z * sigmoid(z);
    default: return z;
  }
}

__device__ __forceinline__ float act_slope(float z, int act) {
  switch (act) {
    case MX_ACT_RELU: return z > 0.0f ? 1.0f : (z == z ? 0.0f : z);
    case MX_ACT_GELU: {
      const float g = exp_neg(-0.5f * z * z);
      return normal_cdf(z, g) + z * (0.39894228040143268f * g);
    }
    case MX_ACT_GELU_TANH: {
      if (fabsf(z) > 20.0f) return z > 0.0f ? 1.0f : 0.0f;   // to fp32 (and z^3 could overflow)
      float m;
      const float s = sigmoid2(2.0f * kGeluC * (z + kGeluA * z * z * z), m);
      return s + z * s * m * 2.0f * kGeluC * (1.0f + 3.0f * kGeluA * z * z);
    }
    case MX_ACT_SILU: {
      float m;
      const float s = sigmoid2(z, m);
      return s * (1.0f + z * m);
    }
    default: return 1.0f;
  }
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ float bf1(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

// ---------------------------------------------------------------- epilogue
struct Epi {
  const float* bias;         // [J] or null
  const uint16_t* residual;  // [I, J] or null
  uint16_t* z;               // [I, J] or null
  void* out;                 // [I, J]
  int32_t act;
  bool f32;
  bool wide;                 // J % 8 == 0: 16-byte accesses
};

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]), bf16x2_rne(v[4], v[5]), bf16x2_rne(v[6], v[7]));
}

template <bool kNt>
__device__ __forceinline__ void store16(void* to, const uint4& v) {
  const v4u w = {v.x, v.y, v.z, v.w};
  if constexpr (kNt) __builtin_nontemporal_store(w, static_cast<v4u*>(to));
  else *static_cast<v4u*>(to) = w;
}

// z of 8 consecutive columns of one row (bias added) to the results; res: the
// residual's 8 values where accesses are wide.  kNt: non-temporal wide stores.
template <bool kNt>
__device__ __forceinline__ void finish8(const Epi& e, int act, float (&v)[8], const uint4& res, int64_t i, int64_t j,
                                        int64_t J) {
  const int64_t at = i * J + j;
  if (e.wide) {
    if (e.z) store16<kNt>(e.z + at, pack8(v));
    if (act != MX_ACT_NONE) {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = act_value(v[k], act);
    }
    if (e.residual) {
      const uint32_t w[4] = {res.x, res.y, res.z, res.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[2 * k] += bf_lo(w[k]);
        v[2 * k + 1] += bf_hi(w[k]);
      }
    }
    if (e.f32) {
      float* o = static_cast<float*>(e.out) + at;
      const v4f lo = {v[0], v[1], v[2], v[3]}, hi = {v[4], v[5], v[6], v[7]};
      store16<kNt>(o, __builtin_bit_cast(uint4, lo));
      store16<kNt>(o + 4, __builtin_bit_cast(uint4, hi));
    } else {
      store16<kNt>(static_cast<uint16_t*>(e.out) + at, pack8(v));
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    if (j + k < J) {
      float x = v[k];
      if (e.z) e.z[at + k] = (uint16_t)bf16x2_rne(x, x);
      x = act_value(x, act);
      if (e.residual) x += bf1(e.residual[at + k]);
      if (e.f32) static_cast<float*>(e.out)[at + k] = x;
      else static_cast<uint16_t*>(e.out)[at + k] = (uint16_t)bf16x2_rne(x, x);
    }
  }
}

// 32 rows of kStageCols<TN> columns: the lane's bias, the residual, the results.
template <int TN>
struct Rows32 {
  static constexpr int W = kStageCols<TN>, kPitch = W * 4 + 16;
  static constexpr int kLpr = W / 8, kRpp = 64 / kLpr, kIt = 32 / kRpp;   // lanes per row, rows per pass, passes
  float bias[8];
  int64_t j;   // the lane's first column

  __device__ __forceinline__ void init(const Epi& e, int64_t j0, int64_t J) {
    j = j0 + 8 * ((threadIdx.x & 63) % kLpr);
#pragma unroll
    for (int k = 0; k < 8; ++k) bias[k] = e.bias && j + k < J ? e.bias[j + k] : 0.0f;
  }
  __device__ __forceinline__ void fetch(const Epi& e, uint4 (&res)[kIt], int64_t i0, int64_t I, int64_t J) const {
#pragma unroll
    for (int it = 0; it < kIt; ++it) {
      const int64_t i = i0 + kRpp * it + (threadIdx.x & 63) / kLpr;
      res[it] = make_uint4(0, 0, 0, 0);
      if (e.residual && e.wide && i < I && j < J) res[it] = *reinterpret_cast<const uint4*>(e.residual + i * J + j);
    }
  }
  template <int kAct, bool kNt>
  __device__ __forceinline__ void finish(const Epi& e, const v16f* acc, uint8_t* slice, const uint4 (&res)[kIt],
                                         int64_t i0, int64_t I, int64_t J) const {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int n = 0; n < W / 32; ++n)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        *reinterpret_cast<float4*>(slice + (lane & 31) * kPitch + (32 * n + 8 * g + 4 * (lane >> 5)) * 4) =
            make_float4(acc[n][4 * g], acc[n][4 * g + 1], acc[n][4 * g + 2], acc[n][4 * g + 3]);
    // exchanged between the wave's lanes, whose LDS accesses run in order
    asm volatile("" ::: "memory");
#pragma unroll
    for (int it = 0; it < kIt; ++it) {
      const int row = kRpp * it + lane / kLpr;
      const float4 x = *reinterpret_cast<const float4*>(slice + row * kPitch + 32 * (lane % kLpr));
      const float4 y = *reinterpret_cast<const float4*>(slice + row * kPitch + 32 * (lane % kLpr) + 16);
      const int64_t i = i0 + row;
      if (i < I && j < J) {
        float v[8] = {x.x + bias[0], x.y + bias[1], x.z + bias[2], x.w + bias[3],
                      y.x + bias[4], y.y + bias[5], y.z + bias[6], y.w + bias[7]};
        finish8<kNt>(e, kAct, v, res[it], i, j, J);
      }
    }
    asm volatile("" ::: "memory");
  }
};

// The accumulators hold 4 consecutive columns of one row per lane (32 rows of W
// fp32 columns are staged at a time), rows of 8 columns per lane go out.  The
// residual of the next 32 rows is fetched while these are finished: read where
// it is added, its latency costs more than the products of a 256 x 256 tile's
// last quarter.
template <int TM, int TN, int kAct, typename Sums>
__device__ __forceinline__ void epilogue(const Epi& e, v16f (&acc)[TM / 32][TN / 32], uint8_t* slice, int64_t i0,
                                         int64_t j0, int64_t I, int64_t J, Sums sums) {
  constexpr int FM = TM / 32, FN = TN / 32, W = kStageCols<TN>;
#pragma unroll
  for (int n0 = 0; n0 < FN; n0 += W / 32) {
    Rows32<TN> rows;
    uint4 res[2][Rows32<TN>::kIt];
    rows.init(e, j0 + 32 * n0, J);
    rows.fetch(e, res[0], i0, I, J);
    if (n0 == 0) sums();
#pragma unroll
    for (int m = 0; m < FM; ++m) {
      if (m + 1 < FM) rows.fetch(e, res[(m + 1) & 1], i0 + 32 * (m + 1), I, J);
      rows.template finish<kAct, false>(e, &acc[m][n0], slice, res[m & 1], i0 + 32 * m, I, J);
    }
  }
}
template <int kAct>
struct Dense {
  typedef Epi Args;
  static constexpr int kSide = 32;   // (the other shape's sums run in another order)
  template <int TM, int TN, typename Sums>
  __device__ static __forceinline__ void run(const Epi& e, v16f (&acc)[TM / 32][TN / 32], uint8_t* slice, int64_t i0,
                                             int64_t j0, int64_t I, int64_t J, Sums sums) {
    epilogue<TM, TN, kAct>(e, acc, slice, i0, j0, I, J, sums);
  }
};

// Contractions of at most 64 (A stored by rows): the output is all the cost.
// A workgroup keeps a B tile of 256 columns, each wave 64 of them as fragments
// in registers, and goes over blocks of 32 rows, every `splits`-th, so that the
// card writes whole rows together; the next block's rows of A and its residual
// are on the way while one is finished.
constexpr int kShortCols = 256;
constexpr int kShortPerCu = 3;

template <bool kBRows, int kAct>
__global__ void __launch_bounds__(256, kShortPerCu) k_short(Product<Epi> p) {
  constexpr int kTile = kShortCols * 64 * 2;
  constexpr int kLds = kTile > 4 * kStageBytes<64> ? kTile : 4 * kStageBytes<64>;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kLds];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t j0 = (int64_t)(blockIdx.x % p.tiles_j) * kShortCols, jw = j0 + 64 * wave;
  TileLoads<kBRows, kShortCols, 4, 64> lb;
  FragAt<kBRows, kShortCols, 64> fb;
  lb.init(p.b, j0, p.J, p.C);
  fb.init();
  const auto tb = lb.prepare(0, p.C);
#pragma unroll
  for (int i = 0; i < lb.kLoads; ++i) lb.template load<false>(tb, i, (uint32_t)(uintptr_t)(const lds_void*)lds);
  __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
  bare_barrier();
  v8bf b[4][2];
#pragma unroll
  for (int kk = 0; kk < 4; ++kk)
#pragma unroll
    for (int n = 0; n < 2; ++n) b[kk][n] = fb.read(lds, 64 * wave + 32 * n, kk);
  __syncthreads();   // read: the waves' slices take the tile's place
  if (jw >= p.J) return;
  uint8_t* slice = lds + wave * kStageBytes<64>;
  Rows32<64> rows;
  rows.init(p.epi, jw, p.J);

  const int64_t blocks = (p.I + 31) / 32;
  v8bf a[4];
  uint4 res[Rows32<64>::kIt];
  auto fetch = [&](int64_t blk) {
    const int64_t left = p.I - 32 * blk;   // rows (none past the end: nothing is read)
    const int64_t n = left < 0 ? 0 : (left < 32 ? left : 32);
    const __amdgpu_buffer_rsrc_t r = buf(p.a.p + (n ? 32 * blk : 0) * p.a.ld, n * p.a.ld * 2);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      const int c = 16 * kk + 8 * (lane >> 5);
      const uint32_t off = (uint32_t)(lane & 31) * (uint32_t)p.a.ld * 2u + 2u * (uint32_t)c;
      a[kk] = __builtin_bit_cast(v8bf, __builtin_amdgcn_raw_buffer_load_b128(r, (int)(c < p.C ? off : kOob), 0, 0));
    }
    rows.fetch(p.epi, res, 32 * blk, p.I, p.J);
  };
  int64_t blk = blockIdx.x / p.tiles_j;
  fetch(blk);
  for (; blk < blocks; blk += p.splits) {
    v16f acc[2];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[n][r] = 0.f;
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
      for (int n = 0; n < 2; ++n) acc[n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b[kk][n], a[kk], acc[n], 0, 0, 0);
    uint4 now[Rows32<64>::kIt];
#pragma unroll
    for (int it = 0; it < Rows32<64>::kIt; ++it) now[it] = res[it];
    fetch(blk + p.splits);
    rows.template finish<kAct, true>(p.epi, acc, slice, now, 32 * blk, p.I, p.J);
  }
}
// ---------------------------------------------------------------- few rows
// What k_skinny's sums become: the epilogue.  What it adds is fetched ahead, as a
// compiled load that is waited for between the items would wait for the stream's
// loads too.
struct FewDense {
  Epi epi;
  struct Ahead {
    float bias[8];
    uint4 res;
  };
  struct State {};
  __device__ __forceinline__ Ahead fetch(bool in, int m, int64_t j, int64_t N) const {
    Ahead t{};
    if (in) {
      if (epi.bias) {
        if (epi.wide) {
          __builtin_memcpy(t.bias, epi.bias + j, 32);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (j + k < N) t.bias[k] = epi.bias[j + k];
        }
      }
      if (epi.residual && epi.wide) t.res = *reinterpret_cast<const uint4*>(epi.residual + m * N + j);
    }
    return t;
  }
  __device__ __forceinline__ void finish(State&, const Ahead& t, float (&v)[8], int m, int64_t j, int64_t N) const {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] += t.bias[k];
    finish8<false>(epi, epi.act, v, t.res, m, j, N);
  }
  __device__ __forceinline__ void end(State&, float*, int, int, int64_t) const {}
};

// ---------------------------------------------------------------- dz and dbias
// dz = dout act'(z) in bf16 with rows of pitch elements (zeros past N): the type
// of the matrix instruction's operand, in which a bf16 dout comes anyway; an fp32
// one is rounded here too, as keeping its lower half would double both products
// (dx and dw are then off by 0.0023 of their size, of which their own rounding
// is 0.0017).  And fp32 column sums of the unrounded dz over the block's rows:
// `part` [gridDim.y, N].  256 threads: ct groups of 8 columns x 256 / ct rows.
template <typename T>
__device__ __forceinline__ T load_once(const void* p) { return __builtin_nontemporal_load(static_cast<const T*>(p)); }

template <bool kF32>
__global__ void __launch_bounds__(256) k_dz(const void* __restrict__ dout, const uint16_t* __restrict__ z, int64_t M,
                                            int64_t N, int64_t pitch, int32_t act, int32_t ct, int64_t rows_per,
                                            uint16_t* __restrict__ dz, float* __restrict__ part) {
  __shared__ float sum[256][8];
  const int cg = threadIdx.x % ct, rl = threadIdx.x / ct, rt = 256 / ct;
  const int64_t j = 8 * ((int64_t)blockIdx.x * ct + cg);
  const int64_t r0 = (int64_t)blockIdx.y * rows_per;
  const int64_t r1 = r0 + rows_per < M ? r0 + rows_per : M;
  const bool wide = N % 8 == 0;
  float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (j < N) {
    const int n = N - j < 8 ? (int)(N - j) : 8;
#pragma unroll 2
    for (int64_t r = r0 + rl; r < r1; r += rt) {
      float v[8];
      const int64_t at = r * N + j;
      if (wide) {
        if constexpr (kF32) {
          const v4f a = load_once<v4f>(static_cast<const float*>(dout) + at);
          const v4f b = load_once<v4f>(static_cast<const float*>(dout) + at + 4);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            v[k] = a[k];
            v[4 + k] = b[k];
          }
        } else {
          const v4u w = load_once<v4u>(static_cast<const uint16_t*>(dout) + at);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            v[2 * k] = bf_lo(w[k]);
            v[2 * k + 1] = bf_hi(w[k]);
          }
        }
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          v[k] = 0.0f;
          if (k < n) v[k] = kF32 ? static_cast<const float*>(dout)[at + k] : bf1(static_cast<const uint16_t*>(dout)[at + k]);
        }
      }
      if (act != MX_ACT_NONE) {
        if (wide) {
          const v4u w = load_once<v4u>(z + at);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            v[2 * k] *= act_slope(bf_lo(w[k]), act);
            v[2 * k + 1] *= act_slope(bf_hi(w[k]), act);
          }
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (k < n) v[k] *= act_slope(bf1(z[at + k]), act);
        }
      }
      if (dz)
        *reinterpret_cast<uint4*>(dz + r * pitch + j) = make_uint4(bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]),
                                                                   bf16x2_rne(v[4], v[5]), bf16x2_rne(v[6], v[7]));
#pragma unroll
      for (int k = 0; k < 8; ++k) s[k] += v[k];
    }
  }
  if (!part) return;
#pragma unroll
  for (int k = 0; k < 8; ++k) sum[threadIdx.x][k] = s[k];
  __syncthreads();
  // one thread per column sums the row lanes in order
  for (int c = threadIdx.x; c < 8 * ct; c += 256) {
    const int64_t col = 8 * (int64_t)blockIdx.x * ct + c;
    if (col >= N) continue;
    float t = 0.0f;
    for (int l = 0; l < rt; ++l) t += sum[l * ct + (c >> 3)][c & 7];
    part[(int64_t)blockIdx.y * N + col] = t;
  }
}

// dbias from the blocks' sums: 16 columns per workgroup, 16 threads to a
// column, each a run of blocks in order, then the runs in order (one thread
// per column takes 16 to 31 us for 256 blocks, their latencies in a row).
__global__ void __launch_bounds__(256) k_dbias(const float* __restrict__ part, int32_t blocks, int64_t N,
                                               float* __restrict__ dbias) {
  __shared__ float sum[16][17];
  const int c = threadIdx.x & 15, run = threadIdx.x >> 4;
  const int64_t j = 16 * (int64_t)blockIdx.x + c;
  const int per = (blocks + 15) / 16;
  const int b1 = (run + 1) * per < blocks ? (run + 1) * per : blocks;
  float t = 0.0f;
  if (j < N) {
#pragma unroll 8
    for (int b = run * per; b < b1; ++b) t += part[b * N + j];
  }
  sum[run][c] = t;
  __syncthreads();
  if (run == 0 && j < N) {
    for (int r = 1; r < 16; ++r) t += sum[r][c];
    dbias[j] = t;
  }
}

// ---------------------------------------------------------------- host side
bool grid_fits(int64_t I, int64_t J, int64_t C, bool a_rows) {
  return (a_rows && C <= 64) || tiles_fit(I, J, C);   // (k_short has a few workgroups per CU)
}

template <bool kBRows, int kAct>
int launch_short(Product<Epi>& p, hipStream_t st) {
  const int64_t tj = (p.J + kShortCols - 1) / kShortCols, blocks = (p.I + 31) / 32;
  int64_t s = kShortPerCu * kCus / tj;
  s = s > blocks ? blocks : s;
  p.tiles_j = (int32_t)tj;
  p.splits = (int32_t)(s < 1 ? 1 : s);
  hipLaunchKernelGGL((k_short<kBRows, kAct>), dim3((unsigned)(tj * p.splits)), dim3(256), 0, st, p);
  return launch_status();
}
template <bool kARows, bool kBRows, int kAct>
int launch_product(const Operand& a, const Operand& b, int64_t I, int64_t J, int64_t C, const Epi& epi, float* part,
                   hipStream_t st) {
  if constexpr (kARows) {
    if (C <= 64) {
      Product<Epi> p{a, b, I, J, C};
      p.epi = epi;
      return launch_short<kBRows, kAct>(p, st);
    }
  }
  return launch_tiles<kARows, kBRows, Dense<kAct>>(a, b, I, J, C, epi, part, st);
}

// Sections of the backward's workspace.
struct BwdSpace {
  int64_t pitch, dz, sums, part;   // dz row pitch; byte sizes
  int32_t ct, blocks;              // column groups per block, row blocks of k_dz
  int64_t rows_per;
};

BwdSpace bwd_space(int64_t M, int64_t N, int64_t K) {
  BwdSpace s;
  s.pitch = up(N, 8);
  s.dz = up(2 * M * s.pitch, 256);
  s.ct = 1;
  while (s.ct < 64 && 8 * s.ct < N) s.ct *= 2;
  // row blocks: about eight workgroups per CU, at least four rows per thread row
  const int64_t gx = (N + 8 * s.ct - 1) / (8 * s.ct);
  int64_t want = 8 * kCus / gx;
  const int64_t most = (M + 4 * (256 / s.ct) - 1) / (4 * (256 / s.ct));
  want = want < 1 ? 1 : (want > most ? most : want);
  if (want > 256) want = 256;
  s.rows_per = want ? up((M + want - 1) / want, 256 / s.ct) : 1;
  s.blocks = (int32_t)((M + s.rows_per - 1) / s.rows_per);
  s.sums = up(4 * (int64_t)s.blocks * N, 256);
  const int64_t a = plan_product(M, K, N).part_bytes, b = plan_product(N, K, M).part_bytes;
  s.part = a > b ? a : b;
  return s;
}

}  // namespace
}  // namespace mx

using namespace mx;

extern "C" size_t mx_bf16_linear_workspace_size(int64_t rows, int64_t n, int64_t k) {
  if (rows <= 0 || n <= 0 || k <= 0 || few_rows(rows, k) || too_large(rows, n, k)) return 0;
  return (size_t)plan_product(rows, n, k).part_bytes;
}

extern "C" int mx_bf16_linear(const uint16_t* x, const uint16_t* w, const float* bias, const uint16_t* residual,
                              int64_t rows, int64_t n, int64_t k, int32_t act, uint16_t* z, void* out,
                              int32_t out_dtype, void* workspace, size_t workspace_bytes, mx_stream_t stream) {
  if (rows < 0 || n <= 0 || k <= 0 || k % 32) return MX_EINVAL;
  if (!x || !w || !out || act < MX_ACT_NONE || act > MX_ACT_SILU) return MX_EINVAL;
  if (out_dtype != MX_OUT_BF16 && out_dtype != MX_OUT_F32) return MX_EINVAL;
  if (misaligned(x) || misaligned(w) || misaligned(residual) || misaligned(z) || misaligned(out)) return MX_EINVAL;
  if (((uintptr_t)bias & 3) || misaligned(workspace)) return MX_EINVAL;
  if (too_large(rows, n, k)) return MX_EUNSUPPORTED;
  if (rows == 0) return MX_OK;
  if (!few_rows(rows, k) && !grid_fits(rows, n, k, true)) return MX_EUNSUPPORTED;
  const hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  Epi epi;
  epi.bias = bias;
  epi.residual = residual;
  epi.z = z;
  epi.out = out;
  epi.act = act;
  epi.f32 = out_dtype == MX_OUT_F32;
  epi.wide = n % 8 == 0;
  if (few_rows(rows, k)) {
    hipLaunchKernelGGL(k_skinny<FewDense>, dim3(skinny_grid(n)), dim3(64 * kSkWaves), 0, st, x, w, rows, n, k,
                       FewDense{epi});
    return launch_status();
  }
  const int64_t need = plan_product(rows, n, k).part_bytes;
  if (need && (!workspace || (int64_t)workspace_bytes < need)) return MX_EINVAL;
  const Operand a{x, k}, b{w, k};
  float* part = static_cast<float*>(workspace);
  switch (act) {   // (the epilogue of a large tile is compiled per activation)
    case MX_ACT_RELU: return launch_product<true, true, MX_ACT_RELU>(a, b, rows, n, k, epi, part, st);
    case MX_ACT_GELU: return launch_product<true, true, MX_ACT_GELU>(a, b, rows, n, k, epi, part, st);
    case MX_ACT_GELU_TANH: return launch_product<true, true, MX_ACT_GELU_TANH>(a, b, rows, n, k, epi, part, st);
    case MX_ACT_SILU: return launch_product<true, true, MX_ACT_SILU>(a, b, rows, n, k, epi, part, st);
    default: return launch_product<true, true, MX_ACT_NONE>(a, b, rows, n, k, epi, part, st);
  }
}

extern "C" size_t mx_bf16_linear_bwd_workspace_size(int64_t rows, int64_t n, int64_t k, int32_t act) {
  if (rows <= 0 || n <= 0 || k <= 0 || too_large(rows, n, k) || act < MX_ACT_NONE || act > MX_ACT_SILU) return 0;
  const BwdSpace s = bwd_space(rows, n, k);
  return (size_t)(s.dz + s.sums + s.part);
}

extern "C" int mx_bf16_linear_bwd(const void* dout, int32_t dout_dtype, const uint16_t* z, const uint16_t* x,
                                  const uint16_t* w, const uint16_t* dx_add, int64_t rows, int64_t n, int64_t k,
                                  int32_t act, uint16_t* dx, uint16_t* dw, float* dbias, void* workspace,
                                  size_t workspace_bytes, mx_stream_t stream) {
  if (rows < 0 || n <= 0 || k <= 0 || k % 32 || act < MX_ACT_NONE || act > MX_ACT_SILU) return MX_EINVAL;
  if (dout_dtype != MX_OUT_BF16 && dout_dtype != MX_OUT_F32) return MX_EINVAL;
  if (!dout || (act != MX_ACT_NONE && !z) || (!dx && !dw && !dbias)) return MX_EINVAL;
  if ((dx && !w) || (dw && !x) || (dx_add && !dx)) return MX_EINVAL;
  if (misaligned(dout) || misaligned(z) || misaligned(x) || misaligned(w) || misaligned(dx_add) || misaligned(dx) ||
      misaligned(dw) || ((uintptr_t)dbias & 3) || misaligned(workspace))
    return MX_EINVAL;
  if (too_large(rows, n, k)) return MX_EUNSUPPORTED;
  if ((dx && !grid_fits(rows, k, n, true)) || (dw && !grid_fits(n, k, rows, false))) return MX_EUNSUPPORTED;
  const hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  const BwdSpace s = bwd_space(rows, n, k);
  if (rows > 0 && (!workspace || (int64_t)workspace_bytes < s.dz + s.sums + s.part)) return MX_EINVAL;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  float* sums = reinterpret_cast<float*>(ws + s.dz);
  float* part = reinterpret_cast<float*>(ws + s.dz + s.sums);
  // dout itself serves as dz where it is bf16, linear and has 16-byte rows
  const bool same = act == MX_ACT_NONE && dout_dtype == MX_OUT_BF16 && n % 8 == 0;
  const uint16_t* dzp = same ? static_cast<const uint16_t*>(dout) : reinterpret_cast<uint16_t*>(ws);
  const int64_t pitch = same ? n : s.pitch;
  if (rows > 0 && (!same || dbias)) {
    const dim3 grid((unsigned)((n + 8 * s.ct - 1) / (8 * s.ct)), (unsigned)s.blocks);
    uint16_t* dz = same ? nullptr : reinterpret_cast<uint16_t*>(ws);
    float* sp = dbias ? sums : nullptr;
    if (dout_dtype == MX_OUT_F32)
      hipLaunchKernelGGL(k_dz<true>, grid, dim3(256), 0, st, dout, z, rows, n, pitch, act, s.ct, s.rows_per, dz, sp);
    else
      hipLaunchKernelGGL(k_dz<false>, grid, dim3(256), 0, st, dout, z, rows, n, pitch, act, s.ct, s.rows_per, dz, sp);
  }
  if (dbias)
    hipLaunchKernelGGL(k_dbias, dim3((unsigned)((n + 15) / 16)), dim3(256), 0, st, sums, rows > 0 ? s.blocks : 0, n,
                       dbias);
  Epi epi;
  epi.bias = nullptr;
  epi.residual = nullptr;
  epi.z = nullptr;
  epi.act = MX_ACT_NONE;
  epi.f32 = false;
  epi.wide = true;   // K % 32 == 0
  if (dx && rows > 0) {
    epi.out = dx;
    epi.residual = dx_add;
    const int rc = launch_product<true, false, MX_ACT_NONE>(Operand{dzp, pitch}, Operand{w, k}, rows, k, n, epi, part, st);
    if (rc != MX_OK) return rc;
  }
  if (dw) {
    epi.out = dw;
    epi.residual = nullptr;
    const int rc = launch_product<false, false, MX_ACT_NONE>(Operand{dzp, pitch}, Operand{x, k}, n, k, rows, epi, part, st);
    if (rc != MX_OK) return rc;
  }
  return launch_status();
}

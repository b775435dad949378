// The dense bf16 product with an epilogue, and its backward (gfx950):
//
//   z = x w^T + bias,  out = act(z) + residual            (x [M, K], w [N, K])
//   dz = dout act'(z), dx = dz w (+ dx_add), dw = dz^T x, dbias = sum_m dz
//
// All three products are C[i, j] = sum_c A(i, c) B(j, c) and run in one
// kernel: an operand is stored either with c contiguous ("rows": x and w in
// the forward, dz in dx) or with i or j contiguous ("columns": w in dx, dz and
// x in dw).  Tiles of 64 c come into LDS by LDS-direct loads in their stored
// layout.  Rows are read as fragments with 16-byte LDS reads, columns with
// the transposing reads (ds_read_b64_tr_b16), so no operand is ever
// transposed in memory.
//
// Up to 16 rows the forward streams w once through the code of stream.h.
// Sums are fp32 in a fixed order; where the tiles are too few for the card
// the contraction is split over workgroups, whose fp32 partial sums are
// added in order by a second launch with the same epilogue.

#include "stream.h"

namespace mx {
namespace {

typedef float v16f __attribute__((ext_vector_type(16)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s lds_v4s;

constexpr int kXcds = 8;

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

// ---------------------------------------------------------------- tiled product
struct Operand {
  const uint16_t* p;
  int64_t ld;        // elements between stored rows
};

struct Product {
  Operand a, b;
  int64_t I, J, C;       // rows and columns of the result, contraction length
  int32_t tiles_i, tiles_j;
  int32_t full;          // tiles computed whole; the others are split over the contraction
  int32_t splits;
  int32_t split_c;       // contraction elements per split (a multiple of 64)
  float* part;           // fp32 sums of the split tiles [splits, tiles - full, BM x BN in register order]
  Epi epi;
};

// The q-th tile: bands of 8 row tiles, so that tiles that run together share
// operands in an XCD's L2.
__device__ __forceinline__ void tile_at(const Product& p, int32_t q, int bm, int bn, int64_t& i0, int64_t& j0) {
  constexpr int kBand = 8;
  const int32_t band = q / (kBand * p.tiles_j), in = q % (kBand * p.tiles_j);
  const int32_t rows = p.tiles_i - band * kBand < kBand ? p.tiles_i - band * kBand : kBand;
  i0 = (int64_t)(band * kBand + in % rows) * bm;
  j0 = (int64_t)(in / rows) * bn;
}

// A barrier that waits for nothing by itself (a fence's wait would include
// loads still in flight); nothing may be moved across it.
__device__ __forceinline__ void bare_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// Swizzles of 16-byte chunks.  Rows: 128-byte LDS rows, chunk ^ (r >> 1) & 7,
// so the 16-byte reads of 32 consecutive rows spread over all banks.  Columns:
// an LDS row is one c with R columns; a transposing read takes 64 bytes of 4
// consecutive c at once, which the swizzle moves to different 64-byte banks.
template <int kC>
__device__ __forceinline__ int row_swizzle(int r) { return kC == 64 ? (r >> 1) & 7 : (r >> 2) & 3; }
template <int R>
__device__ __forceinline__ int col_swizzle(int c) { return R >= 128 ? (c & 3) << 2 : ((c >> 1) & 1) << 2; }

// The LDS-direct loads of one operand tile: kLoads per wave and 64-c tile.
template <bool kRows, int R, int kNw, int kC>
struct TileLoads {
  static constexpr int kLoads = R * kC * 2 / 1024 / kNw;
  static_assert(R * kC * 2 % (1024 * kNw) == 0, "whole loads per wave");
  uint32_t voff[kLoads];
  int32_t kc;   // rows: the lane's first c in a tile
  const uint8_t* base;
  int64_t bytes, step;

  // first: the tile's first row (i or j), n: rows of the operand, C: contraction length
  __device__ void init(const Operand& o, int64_t first, int64_t n, int64_t C) {
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if constexpr (kRows) {
      const int64_t rows = n - first < R ? n - first : R;
      base = reinterpret_cast<const uint8_t*>(o.p + first * o.ld);
      bytes = rows * o.ld * 2;
      step = 0;
      kc = 0;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        constexpr int kPer = kC / 8;         // chunks per LDS row
        const int r = 64 / kPer * (w + kNw * i) + lane / kPer;
        const int ch = (lane % kPer) ^ row_swizzle<kC>(r);
        kc = 8 * ch;   // the same for every i (kNw is even)
        voff[i] = (uint32_t)r * (uint32_t)o.ld * 2u + 16u * (uint32_t)ch;
      }
    } else {
      base = reinterpret_cast<const uint8_t*>(o.p + first);
      bytes = C * o.ld * 2 - first * 2;
      step = kC * o.ld * 2;
      kc = 0;
      constexpr int kPer = R / 8;          // chunks per LDS row
      constexpr int kRowsPer = 64 / kPer;  // LDS rows of one load
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int c = kRowsPer * (w + kNw * i) + lane / kPer;
        const int ch = (lane % kPer) ^ col_swizzle<R>(c);
        // columns past the operand's are other rows' data, or past the end: masked
        voff[i] = first + 8 * ch < n ? (uint32_t)c * (uint32_t)o.ld * 2u + 16u * (uint32_t)ch : kOob;
      }
    }
  }

  // The loads of a tile: prepare() once per tile, then load(i).
  struct Tile {
    v4u r;
    uint32_t soff;
    bool ok;
  };
  __device__ Tile prepare(int64_t tile, int64_t C) const {
    Tile t;
    if constexpr (kRows) {
      t.r = rsrc(base, bytes);
      t.soff = (uint32_t)(tile * kC * 2);
      t.ok = tile * kC + kc < C;
    } else {
      t.r = rsrc(base + tile * step, bytes - tile * step);
      t.soff = 0;
      t.ok = true;
    }
    return t;
  }
  template <bool kOnce>
  __device__ void load(const Tile& t, int i, uint32_t lds) const {
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t to = lds + 1024u * (uint32_t)(w + kNw * i), from = kRows && !t.ok ? kOob : voff[i];
    if constexpr (kOnce) dma16_nt(t.r, to, from, t.soff);
    else dma16(t.r, to, from, t.soff);
  }
};

// Lane offsets of a 32 (i) x 16 (c) fragment; kk = 0..3 in a 64-c tile.
template <bool kRows, int R, int kC>
struct FragAt {
  int row, sw, lo, hi;
  __device__ void init() {
    const int lane = threadIdx.x & 63;
    if constexpr (kRows) {
      row = (lane & 31) * (2 * kC);
      sw = row_swizzle<kC>(lane & 31);
      lo = lane >> 5;
    } else {
      const int l = lane & 15, half = (lane >> 4) & 1, h = lane >> 5;
      const int c = 8 * h + (l >> 2);
      row = c * (2 * R);
      sw = col_swizzle<R>(c);
      lo = 2 * half + ((l & 3) >> 1);   // 16-byte chunk inside the fragment's 32 columns
      hi = 8 * (l & 1);
    }
  }
  // i0: the fragment's first row inside the tile, a multiple of 32
  __device__ v8bf read(const uint8_t* tile, int i0, int kk) const {
    if constexpr (kRows) {
      return *reinterpret_cast<const v8bf*>(tile + i0 * (2 * kC) + row + 16 * ((2 * kk + lo) ^ sw));
    } else {
      const uint8_t* p = tile + kk * 16 * 2 * R + row + 16 * ((i0 / 8 + lo) ^ sw) + hi;
      // c .. c + 3 and c + 4 .. c + 7: the swizzle depends on c & 3 only
      const v4s a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(p));
      const v4s b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(p + 4 * 2 * R));
      return __builtin_bit_cast(v8bf, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  }
};

// Epilogue of a wave's TM x TN sums through its LDS slice: the accumulators
// hold 4 consecutive columns of one row per lane (32 rows of W fp32 columns
// are staged at a time), rows of 8 columns per lane go out.  The residual of the next 32 rows is fetched while these are
// finished: read where it is added, its latency costs more than the products
// of a 256 x 256 tile's last quarter.  sums(): brings the accumulators, after
// the first fetches.
template <int TN>
constexpr int kStageCols = TN < 64 ? TN : 64;
template <int TN>
constexpr int kStageBytes = 32 * (kStageCols<TN> * 4 + 16);

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

// The operand whose every element one workgroup alone reads (the other has one
// row of tiles): its loads are non-temporal.
enum { kOnceNone, kOnceA, kOnceB };

// BM x BN result tile, kWm x kWn waves, kSlots LDS tiles of kC contraction
// elements in flight.
template <int BM, int BN, int kWm, int kWn, int kC, int kSlots, bool kARows, bool kBRows, int kAct, int kOnce>
__global__ void __launch_bounds__(64 * kWm * kWn) k_product(Product p) {
  constexpr int kNw = kWm * kWn;
  constexpr int TM = BM / kWm, TN = BN / kWn, FM = TM / 32, FN = TN / 32;
  constexpr int kABytes = BM * kC * 2, kSlot = (BM + BN) * kC * 2;
  constexpr int kLds = kSlots * kSlot > kNw * kStageBytes<TN> ? kSlots * kSlot : kNw * kStageBytes<TN>;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kLds];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / kWn, wn = wave % kWn;

  // Workgroup b runs on XCD b % 8: each XCD takes a contiguous range of the
  // whole tiles, then one of the split tiles' parts.
  const int32_t tiles = p.tiles_i * p.tiles_j, tail = tiles - p.full;
  const int32_t full8 = (p.full + kXcds - 1) / kXcds * kXcds;
  const bool whole = (int32_t)blockIdx.x < full8;
  const int32_t bid = whole ? blockIdx.x : blockIdx.x - full8;
  const int32_t total = whole ? p.full : tail * p.splits;
  const int32_t per = (total + kXcds - 1) / kXcds;
  const int32_t L = (bid % kXcds) * per + bid / kXcds;
  if (bid / kXcds >= per || L >= total) return;
  const int32_t split = whole ? 0 : L / tail;
  int64_t i0, j0;
  tile_at(p, whole ? L : p.full + L % tail, BM, BN, i0, j0);
  const int64_t all = (p.C + kC - 1) / kC;
  const int64_t t0 = whole ? 0 : (int64_t)split * (p.split_c / kC);
  const int64_t t1 = whole || t0 + p.split_c / kC > all ? all : t0 + p.split_c / kC;

  TileLoads<kARows, BM, kNw, kC> la;
  TileLoads<kBRows, BN, kNw, kC> lb;
  la.init(p.a, i0, p.I, p.C);
  lb.init(p.b, j0, p.J, p.C);
  constexpr int kLoads = TileLoads<kARows, BM, kNw, kC>::kLoads + TileLoads<kBRows, BN, kNw, kC>::kLoads;
  const uint32_t base = (uint32_t)(uintptr_t)(const lds_void*)lds;
  FragAt<kARows, BM, kC> fa;
  FragAt<kBRows, BN, kC> fb;
  fa.init();
  fb.init();

  v16f acc[FM][FN];
#pragma unroll
  for (int m = 0; m < FM; ++m)
#pragma unroll
    for (int n = 0; n < FN; ++n)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[m][n][r] = 0.f;

  // Tiles t0 .. t0 + kSlots - 1 into the slots; tile t0 has to be there.
  constexpr int kLa = decltype(la)::kLoads;
  typename decltype(la)::Tile ta;
  typename decltype(lb)::Tile tb;
  uint32_t dst = 0;
  auto load = [&](int i) {   // load i of the tile in hand
    if (i < kLa) la.template load<kOnce == kOnceA>(ta, i, dst);
    else lb.template load<kOnce == kOnceB>(tb, i - kLa, dst + kABytes);
  };
  auto hand = [&](int64_t t, int s) {
    ta = la.prepare(t, p.C);
    tb = lb.prepare(t, p.C);
    dst = base + (uint32_t)s * kSlot;
  };
#pragma unroll
  for (int s = 0; s < kSlots; ++s)
    if (t0 + s < t1) {
      hand(t0 + s, s);
#pragma unroll
      for (int i = 0; i < kLoads; ++i) load(i);
    }
  if (t0 + kSlots <= t1) __builtin_amdgcn_s_waitcnt(waitcnt_vm(kLoads * (kSlots - 1)));
  else __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
  bare_barrier();

  // A tile's products go in kC / 16 parts of 16 c.  The fragments of a part
  // are read during the part before it, and the loads into the slot that the
  // last tile left are spread over a tile's parts, all placed between the
  // products: a burst of either stalls the products behind it.
  constexpr int kParts = kC / 16, kMfma = FM * FN, kFrags = FM + FN;
  // with two slots a tile has one tile's time to arrive: its loads all go into the first part
  constexpr int kPerPart = kSlots == 2 ? kLoads : (kLoads + kParts - 1) / kParts;
  v8bf a[2][FM], b[2][FN];
  // part of fragments q; `tile` and kk: where part 1 - q is read; loads from `first` on
  auto part = [&](int q, const uint8_t* tile, int kk, bool fill, int first) {
#pragma unroll
    for (int i = 0; i < kMfma; ++i) {
      const int m = i / FN, n = i % FN;
      acc[m][n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b[q][n], a[q][m], acc[m][n], 0, 0, 0);
#pragma unroll
      for (int f = i * kFrags / kMfma; f < (i + 1) * kFrags / kMfma; ++f) {
        if (f < FN) b[1 - q][f] = fb.read(tile + kABytes, wn * TN + 32 * f, kk);
        else a[1 - q][f - FN] = fa.read(tile, wm * TM + 32 * (f - FN), kk);
      }
      if (fill) {
#pragma unroll
        for (int l = i * kPerPart / kMfma; l < (i + 1) * kPerPart / kMfma; ++l)
          if (first + l < kLoads) load(first + l);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
#pragma unroll
  for (int n = 0; n < FN; ++n) b[0][n] = fb.read(lds + kABytes, wn * TN + 32 * n, 0);
#pragma unroll
  for (int m = 0; m < FM; ++m) a[0][m] = fa.read(lds, wm * TM + 32 * m, 0);
  int slot = 0;
  bool fill = false;   // whether the tile in hand is loaded
  for (int64_t t = t0; t < t1; ++t) {
    const uint8_t* tile = lds + slot * kSlot;
    const int next = slot + 1 == kSlots ? 0 : slot + 1;
#pragma unroll
    for (int kk = 1; kk < kParts; ++kk) part((kk & 1) ^ 1, tile, kk, fill, kk * kPerPart);
    // this wave has read its share of the slot, and its loads of tile t + 1
    // are done (the kSlots - 2 tiles after it may be in flight; near the end
    // fewer are, so everything is waited for) ...
    __builtin_amdgcn_s_waitcnt(0xF | (0x3 << 14) | (0x7 << 4));   // lgkmcnt(0)
    if (kSlots > 2 && t + kSlots <= t1) __builtin_amdgcn_s_waitcnt(waitcnt_vm(kLoads * (kSlots > 2 ? kSlots - 2 : 0)));
    else __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
    // ... and after the barrier every wave's: the slot takes tile t + kSlots
    bare_barrier();
    fill = t + kSlots < t1;
    hand(t + kSlots, slot);
    // (after the last tile this reads an old slot, which is not used)
    part(1, lds + next * kSlot, 0, fill, 0);
    slot = next;
  }
  __syncthreads();

  if (!whole) {
    float4* o = reinterpret_cast<float4*>(p.part) + (int64_t)L * (BM * BN / 4) + wave * (TM * TN / 4) + lane;
#pragma unroll
    for (int m = 0; m < FM; ++m)
#pragma unroll
      for (int n = 0; n < FN; ++n)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          o[((m * FN + n) * 4 + g) * 64] =
              make_float4(acc[m][n][4 * g], acc[m][n][4 * g + 1], acc[m][n][4 * g + 2], acc[m][n][4 * g + 3]);
    return;
  }
  epilogue<TM, TN, kAct>(p.epi, acc, lds + wave * kStageBytes<TN>, i0 + wm * TM, j0 + wn * TN, p.I, p.J, [] {});
}

// Contractions of at most 64 (A stored by rows): the output is all the cost.
// A workgroup keeps a B tile of 256 columns, each wave 64 of them as fragments
// in registers, and goes over blocks of 32 rows, every `splits`-th, so that the
// card writes whole rows together; the next block's rows of A and its residual
// are on the way while one is finished.
constexpr int kShortCols = 256;
constexpr int kShortPerCu = 3;

template <bool kBRows, int kAct>
__global__ void __launch_bounds__(256, kShortPerCu) k_short(Product p) {
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

// The split tiles: one wave per 32 rows of a wave's share of a tile adds the
// partial sums in the splits' order, then the epilogue.
template <int BM, int BN, int kWm, int kWn, int kAct>
__global__ void __launch_bounds__(64) k_join(Product p) {
  constexpr int TM = BM / kWm, TN = BN / kWn, FM = TM / 32, FN = TN / 32;
  __shared__ __attribute__((aligned(16))) uint8_t slice[kStageBytes<TN>];
  const int32_t tail = p.tiles_i * p.tiles_j - p.full;
  const int32_t t = blockIdx.x / (kWm * kWn * FM), in = blockIdx.x % (kWm * kWn * FM);
  const int32_t wave = in / FM, m = in % FM;
  int64_t i0, j0;
  tile_at(p, p.full + t, BM, BN, i0, j0);
  v16f acc[1][FN];
#pragma unroll
  for (int n = 0; n < FN; ++n)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[0][n][r] = 0.f;
  const float4* o = reinterpret_cast<const float4*>(p.part) + (int64_t)t * (BM * BN / 4) + wave * (TM * TN / 4) +
                    m * (FN * 256) + threadIdx.x;
  auto sums = [&] {
#pragma unroll 2
    for (int s = 0; s < p.splits; ++s, o += (int64_t)tail * (BM * BN / 4)) {
#pragma unroll
      for (int n = 0; n < FN; ++n)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const float4 v = o[(n * 4 + g) * 64];
          acc[0][n][4 * g] += v.x;
          acc[0][n][4 * g + 1] += v.y;
          acc[0][n][4 * g + 2] += v.z;
          acc[0][n][4 * g + 3] += v.w;
        }
    }
  };
  epilogue<32, TN, kAct>(p.epi, acc, slice, i0 + wave / kWn * TM + 32 * m, j0 + wave % kWn * TN, p.I, p.J, sums);
}

// ---------------------------------------------------------------- few rows
// At most 16 rows of x: items of 16 rows of w, each workgroup a run of them.
// Its eight waves take the chunks of 256 bytes of the items' rows in turn, from
// rings that go on from one item to the next, and add up through LDS.  x stays
// in registers, kSkSteps chunks of a wave.  8192 x 5120 (84 MB): 16.7 us for one
// row (5.0 TB/s), 19.7 for 16; 128 x 64 tiles take 23.5 for 1 to 64 rows, of
// which the split tiles' join is 4: above 16 rows x no longer fits the registers
// beside the stream.  (With k above 8192 x would have to be read again for each
// item: 1408 x 16384 took 22 us for one row and 30 for 16, the tiles take 22.5.)
constexpr int kSkWaves = 8;
constexpr int kSkDepth = 3;                  // chunks of a wave in flight
constexpr int kSkItems = 4;                  // items whose sums wait for each other
constexpr int kSkSlot = 2 * 2048;            // two lines of 16 rows
constexpr int kSkSteps = 8;
constexpr int kSkRows = 16;
constexpr int64_t kSkK = 128 * kSkWaves * kSkSteps;
bool few_rows(int64_t rows, int64_t k) { return rows <= kSkRows && k <= kSkK; }

__global__ void __launch_bounds__(64 * kSkWaves, 2) k_skinny(const uint16_t* __restrict__ x,
                                                             const uint16_t* __restrict__ w, int64_t M, int64_t N,
                                                             int64_t K, Epi epi) {
  __shared__ __attribute__((aligned(16))) float red[kSkItems][kSkWaves][4][64];
  __shared__ __attribute__((aligned(1024))) uint8_t ring[kSkWaves][kSkDepth][kSkSlot];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, h = lane >> 4;
  const int items = (int)((N + 15) / 16);
  const int begin = (int)((int64_t)items * blockIdx.x / gridDim.x), end = (int)((int64_t)items * (blockIdx.x + 1) / gridDim.x);
  const int64_t row_bytes = 2 * K;
  const int chunks = (int)((row_bytes + 255) / 256);
  const int per = (chunks + kSkWaves - 1) / kSkWaves;   // a wave takes chunks wave, wave + 8, ...

  // the loads' cursor
  int li = begin, ls = 0, seq = 0;
  v4u lq;
  auto open = [&](int item) {
    const int64_t n0 = 16 * (int64_t)item;
    lq = rsrc(w + n0 * K, (N - n0 < 16 ? N - n0 : 16) * row_bytes);
  };
  open(begin);
  uint32_t lane_off[2];
  int32_t lane_c[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int row = 8 * q + (lane >> 3);
    lane_c[q] = 16 * ((lane & 7) ^ chunk_swizzle(row));
    lane_off[q] = (uint32_t)row * (uint32_t)row_bytes + (uint32_t)lane_c[q];
  }
  auto load = [&]() {
    const uint32_t dst = lds_addr(ring[wave][0]) + (uint32_t)(seq % kSkDepth) * kSkSlot;
    const int c = wave + kSkWaves * ls;
    const bool in = li < end && c < chunks;
    const int32_t left = in ? (int32_t)(row_bytes - 256 * (int64_t)c) : 0;   // bytes of the rows from here on
    const uint32_t soff = in ? 256u * (uint32_t)c : 0u;
#pragma unroll
    for (int q = 0; q < 4; ++q)   // (rows past N are past the buffer's end)
      dma16_nt(lq, dst + 1024u * q, lane_c[q & 1] + 128 * (q >> 1) < left ? lane_off[q & 1] + 128u * (q >> 1) : kOob, soff);
    ++seq;
    if (++ls == per) {
      ls = 0;
      if (++li < end) open(li);
    }
  };

  v8bf xv[kSkSteps][2][2];
  const __amdgpu_buffer_rsrc_t xr = buf(x, M * row_bytes);
  auto tokens = [&] {
#pragma unroll
    for (int s = 0; s < kSkSteps; ++s) {
      if (s >= per) break;
#pragma unroll
      for (int i = 0; i < 4; ++i) {   // line i >> 1 of the chunk, half of the lane's 32 bytes
        const int64_t at = 256 * (int64_t)(wave + kSkWaves * s) + 128 * (i >> 1) + 32 * h + 16 * (i & 1);
        const uint32_t off = r < M && at < row_bytes ? (uint32_t)r * (uint32_t)row_bytes + (uint32_t)at : kOob;
        xv[s][i >> 1][i & 1] = __builtin_bit_cast(v8bf, __builtin_amdgcn_raw_buffer_load_b128(xr, (int)off, 0, 0));
      }
    }
  };

  // The items are finished kSkItems at a time: after each, the waves would wait
  // for each other with the stream running dry.  A thread takes 8 of the 16
  // columns of one row; what it adds is fetched ahead, as a compiled load that
  // is waited for in between would wait for the stream's loads too.
  struct Tail {
    float bias[8];
    uint4 res;
  };
  const int ti = tid >> 5, m = (tid & 31) >> 1, c0 = 8 * (tid & 1);
  auto tail = [&](int item0) {
    Tail t{};
    const int64_t j = 16 * (int64_t)(item0 + ti) + c0;
    if (ti < kSkItems && m < M && item0 + ti < end && j < N) {
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
  };

  // x lies between the first chunks, and is waited for here: else the compiler
  // waits at each use, and for the stream's loads too
#pragma unroll 1
  for (int d = 0; d < kSkDepth - 1; ++d) load();
  Tail t = tail(begin);
  tokens();
  load();
  __builtin_amdgcn_s_waitcnt(waitcnt_vm(4));
  int used = 0;
  for (int item = begin; item < end; ++item) {
    v4f acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < kSkSteps; ++s) {
      if (s < per) {
        // the oldest chunk's loads are done, the others may be in flight
        fence();
        __builtin_amdgcn_s_waitcnt(waitcnt_vm(4 * (kSkDepth - 1)));
        fence();
        const uint8_t* slot = ring[wave][used % kSkDepth];
        const Fragment f0 = read_fragment<false>(slot, nullptr), f1 = read_fragment<false>(slot + 2048, nullptr);
        fence();
        __builtin_amdgcn_s_waitcnt(kWaitLgkm0);   // read: the slot is free
        fence();
        load();
        ++used;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(weights8<false>(f0, j, 1.0f), xv[s][0][j], acc, 0, 0, 0);
          acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(weights8<false>(f1, j, 1.0f), xv[s][1][j], acc, 0, 0, 0);
        }
      }
    }
    const int at = (item - begin) % kSkItems;
#pragma unroll
    for (int i = 0; i < 4; ++i) red[at][wave][i][lane] = acc[i];
    if (at < kSkItems - 1 && item + 1 < end) continue;
    lds_barrier();
    const int64_t j = 16 * (int64_t)(item - at + ti) + c0;
    if (ti <= at && m < M && j < N) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int c = c0 + k;
        v[k] = 0.0f;
#pragma unroll
        for (int g = 0; g < kSkWaves; ++g) v[k] += red[ti][g][c & 3][16 * (c >> 2) + m];
        v[k] += t.bias[k];
      }
      finish8<false>(epi, epi.act, v, t.res, m, j, N);
    }
    if (item + 1 < end) {
      t = tail(item + 1);
      lds_barrier();
    }
  }
  // loads past the last item may still be writing LDS
  __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
}

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
constexpr int64_t up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

// Tile shapes.
enum Shape { k256x256, k128x128, k128x64, k64x128, k64x64, kShapes };
constexpr struct {
  int bm, bn, per_cu;   // workgroups per CU (LDS)
  double us;            // microseconds per 64 c of a round with all slots busy and operands in L2
  double stream;        // bytes per microsecond at which it streams operands that are read once
} kShape[kShapes] = {
    {256, 256, 1, 1.75, 4.9e6},   // 8192 x 5120 x 8192: 570 us, against 710 with 128 x 128 and 1240 with 64 x 64
    {128, 128, 2, 1.13, 4.9e6},
    {128, 64, 1, 0.70, 6.3e6},    // 32768 x 64 x 7168: 75 us, against 107 with 128 x 128
    {64, 128, 1, 0.70, 5.0e6},    // 64 x 7168 x 8191: 31 us, against 36 with 64 x 64
    {64, 64, 2, 0.50, 4.0e6}};    // 1000 x 1408 x 2048: 18 us, against 22 to 23 with the others

// Tile and split of a product.  Tiles run in rounds of `slots` workgroups; the
// tiles of the last, partly filled round are split over the contraction so
// that it is filled.
struct Plan {
  int shape;
  int32_t full, splits, split_c;
  int64_t part_bytes;
};

Plan plan_product(int64_t I, int64_t J, int64_t C) {
  const int64_t all = (C + 63) / 64;
  Plan best{};
  double least = 1e30;
  for (int id = 0; id < kShapes; ++id) {
    const auto& sh = kShape[id];
    const int64_t ti = (I + sh.bm - 1) / sh.bm, tj = (J + sh.bn - 1) / sh.bn, t = ti * tj;
    const int64_t slots = sh.per_cu * kCus, rounds = t / slots, rem = t - rounds * slots;
    int64_t s = rem ? slots / rem : 1;
    if (s > all / 8) s = all / 8;     // at least 512 c per split
    if (s < 1) s = 1;
    const int64_t per = all ? (all + s - 1) / s : 1;
    s = all ? (all + per - 1) / per : 1;
    double us = sh.us * ((double)rounds * all + (rem ? (double)per : 0.0)) + 3.0 * (rounds + (rem != 0));
    if (us < 2.0 * C * (I + J) / sh.stream) us = 2.0 * C * (I + J) / sh.stream;
    const double part = 4.0 * s * rem * sh.bm * sh.bn;
    if (s > 1) us += 4.0 + 2.0 * part / 4e6;   // the join's launch, its bytes at 4 TB/s
    if (us < least) {
      least = us;
      best.shape = id;
      best.full = (int32_t)(s > 1 ? rounds * slots : t);
      best.splits = (int32_t)s;
      best.split_c = (int32_t)(64 * per);
      best.part_bytes = s > 1 ? (int64_t)part : 0;
    }
  }
  return best;
}

// Whether a product's launch stays below 2^32 threads (the split tiles' parts are at most 2 kCus workgroups).
bool grid_fits(int64_t I, int64_t J, int64_t C, bool a_rows) {
  if (a_rows && C <= 64) return true;   // k_short
  const int shape = plan_product(I, J, C).shape;
  const int64_t tiles = (I + kShape[shape].bm - 1) / kShape[shape].bm * ((J + kShape[shape].bn - 1) / kShape[shape].bn);
  return (tiles + 4 * kCus) * (shape == k256x256 ? 512 : 256) < (1ll << 32);
}

template <int BM, int BN, int kWm, int kWn, int kC, int kSlots, bool kARows, bool kBRows, int kAct, int kOnce = kOnceNone>
void launch_shape(const Product& p, hipStream_t st) {
  auto up8 = [](int32_t v) { return (v + kXcds - 1) / kXcds * kXcds; };
  const int32_t tail = p.tiles_i * p.tiles_j - p.full;
  const dim3 grid((unsigned)(up8(p.full) + up8(tail * p.splits)));
  hipLaunchKernelGGL((k_product<BM, BN, kWm, kWn, kC, kSlots, kARows, kBRows, kAct, kOnce>), grid, dim3(64 * kWm * kWn), 0, st, p);
  if (tail)
    hipLaunchKernelGGL((k_join<BM, BN, kWm, kWn, kAct>), dim3((unsigned)(BM / 32 * kWn * tail)), dim3(64), 0, st, p);
}

// A narrow tile's launch.
template <int BM, int BN, int kSlots, bool kARows, bool kBRows, int kAct>
void launch_narrow(const Product& p, hipStream_t st) {
  if (p.tiles_j == 1) launch_shape<BM, BN, 2, 2, 64, kSlots, kARows, kBRows, kAct, kOnceA>(p, st);
  else if (p.tiles_i == 1) launch_shape<BM, BN, 2, 2, 64, kSlots, kARows, kBRows, kAct, kOnceB>(p, st);
  else launch_shape<BM, BN, 2, 2, 64, kSlots, kARows, kBRows, kAct>(p, st);
}

template <bool kBRows, int kAct>
int launch_short(Product& p, hipStream_t st) {
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
  Product p;
  p.a = a;
  p.b = b;
  p.I = I;
  p.J = J;
  p.C = C;
  p.epi = epi;
  if constexpr (kARows) {
    if (C <= 64) return launch_short<kBRows, kAct>(p, st);
  }
  const Plan pl = plan_product(I, J, C);
  const auto& sh = kShape[pl.shape];
  const int64_t ti = (I + sh.bm - 1) / sh.bm, tj = (J + sh.bn - 1) / sh.bn;
  p.tiles_i = (int32_t)ti;
  p.tiles_j = (int32_t)tj;
  p.full = pl.full;
  p.splits = pl.splits;
  p.split_c = pl.split_c;
  p.part = part;
  switch (pl.shape) {
    case k256x256: launch_shape<256, 256, 2, 4, 64, 2, kARows, kBRows, kAct>(p, st); break;
    case k128x128: launch_shape<128, 128, 2, 2, 64, 2, kARows, kBRows, kAct>(p, st); break;
    case k128x64: launch_narrow<128, 64, 5, kARows, kBRows, kAct>(p, st); break;
    case k64x128: launch_narrow<64, 128, 5, kARows, kBRows, kAct>(p, st); break;
    default: launch_narrow<64, 64, 4, kARows, kBRows, kAct>(p, st); break;
  }
  return launch_status();
}

bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) != 0; }

// Sizes the 32-bit offsets of the tiles allow (256 rows of an operand below 2^31 bytes).
bool too_large(int64_t rows, int64_t n, int64_t k) {
  return k >= (1 << 21) || n >= (1 << 21) || rows >= (1ll << 31);
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
    const int64_t items = (n + 15) / 16;
    const dim3 grid((unsigned)(items < kCus ? items : kCus));
    hipLaunchKernelGGL(k_skinny, grid, dim3(64 * kSkWaves), 0, st, x, w, rows, n, k, epi);
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

// The tiled bf16 product behind the dense product, its backward and the cross
// entropy (gfx950): C[i, j] = sum_c A(i, c) B(j, c), each operand stored either
// with c contiguous ("rows") or with i or j contiguous ("columns").  Tiles of 64
// c come into LDS by LDS-direct loads in their stored layout.  Rows are read as
// fragments with 16-byte LDS reads, columns with the transposing reads
// (ds_read_b64_tr_b16), so no operand is ever transposed in memory.
//
// Sums are fp32 in a fixed order; where the tiles are too few for the card the
// contraction is split over workgroups, whose fp32 partial sums are added in
// order by a second launch with the same epilogue.
//
// What becomes of the sums is an epilogue's matter, a class E with
//   struct Args;                     passed by value to the kernels
//   kSide                            32 or 16: the 256 x 256 tiles' matrix instruction
//   template <int TM, int TN, typename Sums>
//   static void run(const Args&, v16f (&acc)[TM / 32][TN / 32], uint8_t* slice, int64_t i0, int64_t j0, int64_t I,
//                   int64_t J, Sums sums);
// run() gets a wave's TM x TN sums at (i0, j0) of the I x J result and an LDS
// slice of kStageBytes<TN> of its own, and calls sums() once before it reads
// them.  Lane l, register r of acc[m][n] holds row i0 + 32 m + (l & 31), column
// j0 + 32 n + 8 (r >> 2) + 4 (l >> 5) + (r & 3).
#pragma once

#include "stream.h"

namespace mx {
namespace {

typedef float v16f __attribute__((ext_vector_type(16)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s lds_v4s;

constexpr int kXcds = 8;

struct Operand {
  const uint16_t* p;
  int64_t ld;        // elements between stored rows
};

template <class Args>
struct Product {
  Operand a, b;
  int64_t I, J, C;       // rows and columns of the result, contraction length
  int32_t tiles_i, tiles_j;
  int32_t full;          // tiles computed whole; the others are split over the contraction
  int32_t splits;
  int32_t split_c;       // contraction elements per split (a multiple of 64)
  float* part;           // fp32 sums of the split tiles [splits, tiles - full, BM x BN in register order]
  Args epi;              // of the epilogue
};

// The q-th tile: bands of 8 row tiles, so that tiles that run together share
// operands in an XCD's L2.
template <class Args>
__device__ __forceinline__ void tile_at(const Product<Args>& p, int32_t q, int bm, int bn, int64_t& i0, int64_t& j0) {
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
// (Fragments of 16 columns take 32 bytes of c and of c + 8, which it parts too.)
template <int R, int kSide>
__device__ __forceinline__ int col_swizzle(int c) {
  return (R >= 128 ? (c & 3) << 2 : ((c >> 1) & 1) << 2) | (kSide == 16 ? ((c >> 3) & 1) << 1 : 0);
}

// The LDS-direct loads of one operand tile: kLoads per wave and 64-c tile.
template <bool kRows, int R, int kNw, int kC, int kSide = 32>
struct TileLoads {
  static constexpr int kLoads = R * kC * 2 / 1024 / kNw;
  static_assert(R * kC * 2 % (1024 * kNw) == 0, "whole loads per wave");
  uint32_t voff[kLoads];
  int32_t kc;   // rows: the lane's first c in a tile
  int32_t w;    // the wave
  const uint8_t* base;
  int64_t bytes, step;

  // first: the tile's first row (i or j), n: rows of the operand, C: contraction length
  __device__ void init(const Operand& o, int64_t first, int64_t n, int64_t C) {
    const int lane = threadIdx.x & 63;
    w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
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
        const int ch = (lane % kPer) ^ col_swizzle<R, kSide>(c);
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
    const uint32_t to = lds + 1024u * (uint32_t)(w + kNw * i), from = kRows && !t.ok ? kOob : voff[i];
    if constexpr (kOnce) dma16_nt(t.r, to, from, t.soff);
    else dma16(t.r, to, from, t.soff);
  }
};

// Lane offsets of a fragment of kSide (i) x 512 / kSide (c), its number in the
// tile's contraction kk: 32 x 16 or 16 x 32.
template <bool kRows, int R, int kC, int kSide = 32>
struct FragAt {
  static constexpr int kK = 512 / kSide;
  int row, sw, lo, hi;
  __device__ void init() {
    const int lane = threadIdx.x & 63;
    if constexpr (kRows) {
      row = (lane & (kSide - 1)) * (2 * kC);
      sw = row_swizzle<kC>(lane & (kSide - 1));
      lo = lane / kSide;
    } else {
      const int l = lane & 15, half = kSide == 32 ? (lane >> 4) & 1 : 0, h = lane / kSide;
      const int c = 8 * h + (l >> 2);
      row = c * (2 * R);
      sw = col_swizzle<R, kSide>(c);
      lo = 2 * half + ((l & 3) >> 1);   // 16-byte chunk inside the fragment's columns
      hi = 8 * (l & 1);
    }
  }
  // i0: the fragment's first row inside the tile, a multiple of kSide
  __device__ v8bf read(const uint8_t* tile, int i0, int kk) const {
    if constexpr (kRows) {
      return *reinterpret_cast<const v8bf*>(tile + i0 * (2 * kC) + row + 16 * ((kK / 8 * kk + lo) ^ sw));
    } else {
      const uint8_t* p = tile + kk * kK * 2 * R + row + 16 * ((i0 / 8 + lo) ^ sw) + hi;
      // c .. c + 3 and c + 4 .. c + 7: the swizzle does not depend on c & 4
      const v4s a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(p));
      const v4s b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(p + 4 * 2 * R));
      return __builtin_bit_cast(v8bf, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  }
};
// A wave's LDS slice of the epilogue: 32 rows of fp32 sums, at most 64 columns at a time.
template <int TN>
constexpr int kStageCols = TN < 64 ? TN : 64;
template <int TN>
constexpr int kStageBytes = 32 * (kStageCols<TN> * 4 + 16);

// The operand whose every element one workgroup alone reads (the other has one
// row of tiles): its loads are non-temporal.
enum { kOnceNone, kOnceA, kOnceB };

// BM x BN result tile, kWm x kWn waves, LDS for kSlots tiles of kC contraction
// elements; kSlots 0: for two and a half tiles, five halves (A or B) in a ring, so
// that A is on the way for two tiles' time, B for one, and only B's loads are
// waited for at short notice (two whole slots: one tile's time for both).
//
// What bounds the large products is the power of the matrix units: 4096 x 65536 x
// 5120 takes 2.05 ms with normal values and 1.52 ms with zeros, all else alike.
// From registers 16 x 16 x 32 reaches 2.1 PFLOP/s where 32 x 32 x 16 reaches 1.85
// (zeros: 2.4 both); in this loop they take 1.99 ms and 2.09 ms.  4 waves of 128 x
// 128 read a third less from LDS and take 2.17 ms (one wave of a SIMD has nothing
// beside it at a wait).  As it stands the loop takes 1.95 ms, 1.59 with zeros.
template <int BM, int BN, int kWm, int kWn, int kC, int kSlots, bool kARows, bool kBRows, class E, int kOnce>
__global__ void __launch_bounds__(64 * kWm * kWn) k_product(Product<typename E::Args> p) {
  constexpr int kNw = kWm * kWn;
  constexpr int TM = BM / kWm, TN = BN / kWn, FM = TM / 32, FN = TN / 32;
  constexpr int kABytes = BM * kC * 2, kSlot = (BM + BN) * kC * 2;
  constexpr bool kHalves = kSlots == 0;
  static_assert(!kHalves || BM == BN, "halves of one size");
  constexpr int kRing = kHalves ? 5 * kABytes : kSlots * kSlot;
  constexpr int kLds = kRing > kNw * kStageBytes<TN> ? kRing : kNw * kStageBytes<TN>;
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

  constexpr int kSide = kHalves ? E::kSide : 32;
  TileLoads<kARows, BM, kNw, kC, kSide> la;
  TileLoads<kBRows, BN, kNw, kC, kSide> lb;
  la.init(p.a, i0, p.I, p.C);
  lb.init(p.b, j0, p.J, p.C);
  constexpr int kLoads = decltype(la)::kLoads + decltype(lb)::kLoads;
  const uint32_t base = (uint32_t)(uintptr_t)(const lds_void*)lds;
  FragAt<kARows, BM, kC, kSide> fa;
  FragAt<kBRows, BN, kC, kSide> fb;
  fa.init();
  fb.init();

  v16f acc[FM][FN];
#pragma unroll
  for (int m = 0; m < FM; ++m)
#pragma unroll
    for (int n = 0; n < FN; ++n)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[m][n][r] = 0.f;

  // A tile's products go in kC / 16 parts of 16 c.  The fragments of a part
  // are read during the part before it, and the loads into what the last tile
  // left are spread over a tile's parts, all placed between the products: a
  // burst of either stalls the products behind it.  The loads behind the last
  // tile are issued too, of nothing: no branch stands between the products.
  constexpr int kLa = decltype(la)::kLoads, kLb = decltype(lb)::kLoads;
  constexpr int kParts = kC / 16, kMfma = FM * FN, kFrags = FM + FN;
  typename decltype(la)::Tile ta;
  typename decltype(lb)::Tile tb;
  v8bf a[2][FM], b[2][FN];
  const int32_t tn = (int32_t)(t1 - t0);
  // part of fragments q; ap, bp and kk: where part 1 - q is read; loads: `count` of load(first ..)
  auto part = [&](int q, const uint8_t* ap, const uint8_t* bp, int kk, int first, int count, auto load) {
#pragma unroll
    for (int i = 0; i < kMfma; ++i) {
      const int m = i / FN, n = i % FN;
      acc[m][n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b[q][n], a[q][m], acc[m][n], 0, 0, 0);
#pragma unroll
      for (int f = i * kFrags / kMfma; f < (i + 1) * kFrags / kMfma; ++f) {
        if (f < FN) b[1 - q][f] = fb.read(bp, wn * TN + 32 * f, kk);
        else a[1 - q][f - FN] = fa.read(ap, wm * TM + 32 * (f - FN), kk);
      }
#pragma unroll
      for (int l = i * count / kMfma; l < (i + 1) * count / kMfma; ++l) load(first + l);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // the first tile's first fragments
  auto start = [&] {
#pragma unroll
    for (int n = 0; n < FN; ++n) b[0][n] = fb.read(lds + kABytes, wn * TN + 32 * n, 0);
#pragma unroll
    for (int m = 0; m < FM; ++m) a[0][m] = fa.read(lds, wm * TM + 32 * m, 0);
  };

  if constexpr (kHalves) {
    // The ring takes A(t0), B(t0), A(t0 + 1), B(t0 + 1), ...: tile t's A in place
    // 2 (t - t0) mod 5, its B behind it.
    uint32_t da = 0, db = 0;
    auto load_a = [&](int i) {
      if (i < kLa) la.template load<kOnce == kOnceA>(ta, i, da);
    };
    auto load_b = [&](int i) { lb.template load<kOnce == kOnceB>(tb, i, db); };
    auto hand_a = [&](int32_t t, int at) {
      ta = la.prepare(t0 + t, p.C);
      if (t >= tn) ta.r[2] = 0;
      da = base + (uint32_t)(at * kABytes);
    };
    auto hand_b = [&](int32_t t, int at) {
      tb = lb.prepare(t0 + t, p.C);
      if (t >= tn) tb.r[2] = 0;
      db = base + (uint32_t)(at * kABytes);
    };
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      hand_a(s, 2 * s);
#pragma unroll
      for (int i = 0; i < kLa; ++i) load_a(i);
      hand_b(s, 2 * s + 1);
#pragma unroll
      for (int i = 0; i < kLb; ++i) load_b(i);
    }
    hand_a(2, 4);   // (loaded in the first tile's time)
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(kLa + kLb));   // the first tile is there
    bare_barrier();
    int at = 0;          // A's place
    auto place = [](int v) { return v >= 5 ? v - 5 : v; };
    if constexpr (kSide == 16) {
      // Two parts of 32 c.  A fragment of A is used by one row of products and read
      // anew behind it; those of B have two sets.  Nothing is moved past two rows, or
      // one where a fragment of A takes two reads: 4096 x 65536 x 5120 with both
      // gradients 6.33 ms, one row for all 6.39, left to the compiler 6.62, branches
      // around the loads instead 6.50.  kAhead: the rows of the second part in front
      // of the waits; 1 takes 6.46, 3 and 4 6.38.
      constexpr int GM = TM / 16, GN = TN / 16, kAhead = 2, kLeft = GM - kAhead;
      static_assert(kParts == 4, "two parts of 32 c");
      v4f s[GM][GN];
      v8bf x[GM], y[2][GN];
#pragma unroll
      for (int n = 0; n < GN; ++n) y[0][n] = fb.read(lds + kABytes, wn * TN + 16 * n, 0);
#pragma unroll
      for (int m = 0; m < GM; ++m) {
        x[m] = fa.read(lds, wm * TM + 16 * m, 0);
#pragma unroll
        for (int n = 0; n < GN; ++n) s[m][n] = v4f{0.f, 0.f, 0.f, 0.f};
      }
      auto row = [&](int q, int m) {
#pragma unroll
        for (int i = 0; i < GN; ++i) {
          const int n = m & 1 ? GN - 1 - i : i;
          s[m][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(y[q][n], x[m], s[m][n], 0, 0, 0);
        }
      };
      for (int32_t t = 0; t < tn; ++t) {
        const uint8_t *ap = lds + at * kABytes, *bp = lds + place(at + 1) * kABytes;
#pragma unroll
        for (int m = 0; m < GM; ++m) {
          row(0, m);
#pragma unroll
          for (int n = m * GN / GM; n < (m + 1) * GN / GM; ++n) y[1][n] = fb.read(bp, wn * TN + 16 * n, 1);
          x[m] = fa.read(ap, wm * TM + 16 * m, 1);
#pragma unroll
          for (int l = m * kLa / GM; l < (m + 1) * kLa / GM; ++l) load_a(l);
          if (m & 1 || !kARows) __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int m = 0; m < kAhead; ++m) row(1, m);
        // This wave has read its share of tile t, and its loads of tile t + 1 are done
        // (A of tile t + 2 is in flight); after the barrier every wave's: B of tile t +
        // 2 goes where A of tile t was, A of tile t + 3 where its B was.
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(0xF | (0x3 << 14) | (0x7 << 4));   // lgkmcnt(0)
        __builtin_amdgcn_s_waitcnt(waitcnt_vm(kLa));
        bare_barrier();
        hand_b(t + 2, at);
        hand_a(t + 3, place(at + 1));
        at = place(at + 2);
        ap = lds + at * kABytes;
        bp = lds + place(at + 1) * kABytes;
#pragma unroll
        for (int m = kAhead; m < GM; ++m) {
          row(1, m);
          const int k = m - kAhead;
#pragma unroll
          for (int n = k * GN / kLeft; n < (k + 1) * GN / kLeft; ++n) y[0][n] = fb.read(bp, wn * TN + 16 * n, 0);
#pragma unroll
          for (int i = k * GM / kLeft; i < (k + 1) * GM / kLeft; ++i) x[i] = fa.read(ap, wm * TM + 16 * i, 0);
#pragma unroll
          for (int l = k * kLb / kLeft; l < (k + 1) * kLb / kLeft; ++l) load_b(l);
          if (m & 1 || !kARows) __builtin_amdgcn_sched_barrier(0);
        }
      }
      // to the layout of the 32 x 32 instruction: there the lane's bits 4 and 5 are
      // i's bit 4 and j's bit 2, here j's bits 2 and 3
#pragma unroll
      for (int m = 0; m < FM; ++m)
#pragma unroll
        for (int n = 0; n < FN; ++n)
#pragma unroll
          for (int g = 0; g < 2; ++g)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const auto u = __builtin_amdgcn_permlane16_swap(__float_as_uint(s[2 * m][2 * n + g][r]),
                                                              __float_as_uint(s[2 * m + 1][2 * n + g][r]), false, false);
              const auto v = __builtin_amdgcn_permlane32_swap(u[0], u[1], false, false);
              acc[m][n][8 * g + r] = __uint_as_float(v[0]);
              acc[m][n][8 * g + 4 + r] = __uint_as_float(v[1]);
            }
    } else {
      start();
      constexpr int kPer = (kLa + kParts - 2) / (kParts - 1);
      for (int32_t t = 0; t < tn; ++t) {
        const uint8_t *ap = lds + at * kABytes, *bp = lds + place(at + 1) * kABytes;
#pragma unroll
        for (int kk = 1; kk < kParts; ++kk) part((kk & 1) ^ 1, ap, bp, kk, (kk - 1) * kPer, kPer, load_a);
        // this wave has read its share of tile t, and its loads of tile t + 1 are
        // done (A of tile t + 2 may be in flight) ...
        __builtin_amdgcn_s_waitcnt(0xF | (0x3 << 14) | (0x7 << 4));   // lgkmcnt(0)
        __builtin_amdgcn_s_waitcnt(waitcnt_vm(kLa));
        // ... and after the barrier every wave's: B of tile t + 2 goes where A of
        // tile t was, A of tile t + 3 where its B was
        bare_barrier();
        hand_b(t + 2, at);
        hand_a(t + 3, place(at + 1));
        at = place(at + 2);
        // (after the last tile this reads old halves, which are not used)
        part(1, lds + at * kABytes, lds + place(at + 1) * kABytes, 0, 0, kLb, load_b);
      }
    }
  } else {
    // Tiles t0 .. t0 + kSlots - 1 into the slots; tile t0 has to be there.
    uint32_t dst = 0;
    auto load = [&](int i) {   // load i of the tile in hand
      if (i >= kLoads) return;
      if (i < kLa) la.template load<kOnce == kOnceA>(ta, i, dst);
      else lb.template load<kOnce == kOnceB>(tb, i - kLa, dst + kABytes);
    };
    auto hand = [&](int32_t t, int s) {
      ta = la.prepare(t0 + t, p.C);
      tb = lb.prepare(t0 + t, p.C);
      if (t >= tn) ta.r[2] = tb.r[2] = 0;
      dst = base + (uint32_t)s * kSlot;
    };
    // with two slots a tile has one tile's time to arrive: its loads all go into the first part
    constexpr int kPerPart = kSlots == 2 ? kLoads : (kLoads + kParts - 1) / kParts;
#pragma unroll
    for (int s = 0; s < kSlots; ++s) {
      hand(s, s);
#pragma unroll
      for (int i = 0; i < (s + 1 < kSlots ? kLoads : kPerPart); ++i) load(i);   // (the last tile's others: in the first's time)
    }
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(kLoads * (kSlots > 2 ? kSlots - 2 : 0) + kPerPart));
    bare_barrier();
    start();
    int slot = 0;
    for (int32_t t = 0; t < tn; ++t) {
      const uint8_t* tile = lds + slot * kSlot;
      const int next = slot + 1 == kSlots ? 0 : slot + 1;
#pragma unroll
      for (int kk = 1; kk < kParts; ++kk) part((kk & 1) ^ 1, tile, tile + kABytes, kk, kk * kPerPart, kPerPart, load);
      // this wave has read its share of the slot, and its loads of tile t + 1
      // are done (the kSlots - 2 tiles after it may be in flight) ...
      __builtin_amdgcn_s_waitcnt(0xF | (0x3 << 14) | (0x7 << 4));   // lgkmcnt(0)
      __builtin_amdgcn_s_waitcnt(waitcnt_vm(kLoads * (kSlots > 2 ? kSlots - 2 : 0)));
      // ... and after the barrier every wave's: the slot takes tile t + kSlots
      bare_barrier();
      hand(t + kSlots, slot);
      // (after the last tile this reads an old slot, which is not used)
      part(1, lds + next * kSlot, lds + next * kSlot + kABytes, 0, 0, kPerPart, load);
      slot = next;
    }
  }
  __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));   // (the loads of nothing too are done with the LDS)
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
  E::template run<TM, TN>(p.epi, acc, lds + wave * kStageBytes<TN>, i0 + wm * TM, j0 + wn * TN, p.I, p.J, [] {});
}
// The split tiles: one wave per 32 rows of a wave's share of a tile adds the
// partial sums in the splits' order, then the epilogue.
template <int BM, int BN, int kWm, int kWn, class E>
__global__ void __launch_bounds__(64) k_join(Product<typename E::Args> p) {
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
  E::template run<32, TN>(p.epi, acc, slice, i0 + wave / kWn * TM + 32 * m, j0 + wave % kWn * TN, p.I, p.J, sums);
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
    {256, 256, 1, 1.75, 4.9e6},   // 8192 x 5120 x 8192: 530 us, against 710 with 128 x 128 and 1240 with 64 x 64
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
bool tiles_fit(int64_t I, int64_t J, int64_t C) {
  const int shape = plan_product(I, J, C).shape;
  const int64_t tiles = (I + kShape[shape].bm - 1) / kShape[shape].bm * ((J + kShape[shape].bn - 1) / kShape[shape].bn);
  return (tiles + 4 * kCus) * (shape == k256x256 ? 512 : 256) < (1ll << 32);
}

template <int BM, int BN, int kWm, int kWn, int kC, int kSlots, bool kARows, bool kBRows, class E, int kOnce = kOnceNone>
void launch_shape(const Product<typename E::Args>& p, hipStream_t st) {
  auto up8 = [](int32_t v) { return (v + kXcds - 1) / kXcds * kXcds; };
  const int32_t tail = p.tiles_i * p.tiles_j - p.full;
  const dim3 grid((unsigned)(up8(p.full) + up8(tail * p.splits)));
  hipLaunchKernelGGL((k_product<BM, BN, kWm, kWn, kC, kSlots, kARows, kBRows, E, kOnce>), grid, dim3(64 * kWm * kWn), 0, st, p);
  if (tail)
    hipLaunchKernelGGL((k_join<BM, BN, kWm, kWn, E>), dim3((unsigned)(BM / 32 * kWn * tail)), dim3(64), 0, st, p);
}

// A narrow tile's launch.
template <int BM, int BN, int kSlots, bool kARows, bool kBRows, class E>
void launch_narrow(const Product<typename E::Args>& p, hipStream_t st) {
  if (p.tiles_j == 1) launch_shape<BM, BN, 2, 2, 64, kSlots, kARows, kBRows, E, kOnceA>(p, st);
  else if (p.tiles_i == 1) launch_shape<BM, BN, 2, 2, 64, kSlots, kARows, kBRows, E, kOnceB>(p, st);
  else launch_shape<BM, BN, 2, 2, 64, kSlots, kARows, kBRows, E>(p, st);
}
// The product of A [I, C] and B [J, C] with the epilogue E; part: plan_product(I, J, C).part_bytes.
template <bool kARows, bool kBRows, class E>
int launch_tiles(const Operand& a, const Operand& b, int64_t I, int64_t J, int64_t C, const typename E::Args& epi, float* part,
                   hipStream_t st) {
  Product<typename E::Args> p;
  p.a = a;
  p.b = b;
  p.I = I;
  p.J = J;
  p.C = C;
  p.epi = epi;
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
    case k256x256: launch_shape<256, 256, 2, 4, 64, 0, kARows, kBRows, E>(p, st); break;
    case k128x128: launch_shape<128, 128, 2, 2, 64, 2, kARows, kBRows, E>(p, st); break;
    case k128x64: launch_narrow<128, 64, 5, kARows, kBRows, E>(p, st); break;
    case k64x128: launch_narrow<64, 128, 5, kARows, kBRows, E>(p, st); break;
    default: launch_narrow<64, 64, 4, kARows, kBRows, E>(p, st); break;
  }
  return launch_status();
}

bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) != 0; }

// Sizes the 32-bit offsets of the tiles allow (256 rows of an operand below 2^31 bytes).
bool too_large(int64_t rows, int64_t n, int64_t k) {
  return k >= (1 << 21) || n >= (1 << 21) || rows >= (1ll << 31);
}

}  // namespace
}  // namespace mx

// Activations of the SwiGLU expert FFN kept in MXFP8 between the forward and
// the backward (gfx950).
//
// The forward keeps H = [g | u] as rowwise MX codes and the tokens as the codes
// the permute took; the backward rebuilds from them what else it needs:
//   A' = silu(g') u'        columnwise MX (the down weight gradient's operand)
//   dH = [dA u' s (1 + g' (1 - s)) | dA silu(g')], s = sigmoid(g')   row and column MX
//   dots[r] = sum_f dA[r, f] A'[r, f]
//   X^T                     columnwise MX in permuted order, from the tokens' codes
// with g', u' the decoded values.  dA = w_j W2^T dout, so dots[r] = w_j <dout,
// W2 A'> of the pair (t, j) in row r: the router's gradient needs neither the
// down product's rows nor another pass over H columns,
//   dlogit[t, e_j] = dots_j - w_j sum_i dots_i.
// A pair's activations between the passes are 33/32 2F bytes instead of 4F of H
// in bf16, 33/32 F of A^T and 2H of the down product.
//
// All are HBM-bound streams in the tiles and orders of the tile quantizer.

#include "stream.h"
#include "swiglu.h"
#include "tile_quant.h"

namespace mx {
namespace {

// 8 codes with their block's scale byte (not 255) to bf16, as the dequantize does it.
__device__ __forceinline__ uint4 decode8(const uint2& c, uint32_t sb) {
  const float sc = e8m0_to_f32(sb);
  const uint2 a = cvt4_bf16(c.x, sc), b = cvt4_bf16(c.y, sc);
  return make_uint4(a.x, a.y, b.x, b.y);
}

// A block of scale 255 is NaN: sets the block's 8 values to it.
__device__ __forceinline__ void nan_scale(uint4& v, uint32_t sb) {
  if (sb == 255u) v = make_uint4(0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u);
}

// tq_store_rows for columns base + c0 .. of a matrix where base is a multiple of
// 32 but panels may be shared with another tile: scales go out as bytes, the
// last block's lane zeroes the panel's pad bytes.
__device__ __forceinline__ void store_rows_bytes(const uint4 (&v)[8], uint8_t* row_q, uint8_t* row_s, int64_t R,
                                                 int64_t cols, int64_t r, int64_t rows, int64_t col, bool col_ok) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const bool ok = r + i < rows && col_ok;
    const uint32_t sb = scale_byte_from_amax(quad_max(amax8(v[i])));
    const float sc = e8m0_to_f32(sb);
    if (ok)
      *reinterpret_cast<uint2*>(row_q + (r + i) * cols + col) =
          make_uint2(cvt4_e4m3(v[i].x, v[i].y, sc), cvt4_e4m3(v[i].z, v[i].w, sc));
    if (ok && !(threadIdx.x & 3)) put_scale(row_s, R, r + i, col >> 5, cols >> 5, sb);
  }
}

// Half (gate or up) of a matrix [rows, 2F], at the tile's columns c0 .. of it.
// kWhole: F % 128 == 0, no panel holds columns of both halves.
template <bool kWhole>
__device__ __forceinline__ void store_half(const uint4 (&v)[8], uint8_t* q, uint8_t* s, int64_t rows, int64_t F, int64_t r,
                                           int64_t half, int64_t c0, bool col_ok) {
  if constexpr (kWhole)
    tq_store_rows<true, false>(v, q, s, nullptr, rows, 2 * F, r, r, rows, half + c0, col_ok);
  else
    store_rows_bytes(v, q, s, rows, 2 * F, r, rows, half + c0 + 8 * (threadIdx.x & 15), col_ok);
}

// The forward: a thread takes 8 columns of a row, so that a wave's accesses are
// 1 KB of it (the tile quantizer's are four pieces of 256 bytes: 194 us at 67,584
// x 2048, where this took 173 in turn with it, 5.7 TB/s; 2 rows a thread the same, 4
// rows 193; over processes and buffers this form's calls vary from 173 to 210).
// Workgroups go to the XCDs in runs of 32, so that the lines of scales, 4 bytes of
// each of 32 rows, are written in one L2 (8192 x 2048: 23.2 us against 25.9).
template <bool kWhole>
__global__ void __launch_bounds__(256) k_swiglu_keep(const uint16_t* __restrict__ h, int64_t rows, int64_t F,
                                                     uint32_t chunks, uint8_t* __restrict__ row_q,
                                                     uint8_t* __restrict__ row_s, uint8_t* __restrict__ keep_q,
                                                     uint8_t* __restrict__ keep_s) {
  typedef unsigned int v4 __attribute__((ext_vector_type(4)));
  typedef unsigned int v2 __attribute__((ext_vector_type(2)));
  uint32_t b = blockIdx.x;
  if ((b | 255) < gridDim.x) b = (b & ~255u) | (b & 7) << 5 | (b >> 3 & 31);
  const uint32_t id = b * 256u + threadIdx.x;
  const int64_t r = id / chunks, col = 8 * (int64_t)(id % chunks);   // a quad of lanes shares r
  const bool ok = r < rows;
  uint4 g = make_uint4(0, 0, 0, 0), u = g;
  if (ok) {
    const uint16_t* p = h + r * 2 * F + col;
    g = __builtin_bit_cast(uint4, __builtin_nontemporal_load(reinterpret_cast<const v4*>(p)));
    u = __builtin_bit_cast(uint4, __builtin_nontemporal_load(reinterpret_cast<const v4*>(p + F)));
  }
  // the codes of 8 values into q [rows, cols], the block's scale byte into s
  auto put = [&](const uint4& v, uint8_t* q, uint8_t* s, int64_t cols, int64_t c) {
    const uint32_t sb = scale_byte_from_amax(quad_max(amax8(v)));
    const float sc = e8m0_to_f32(sb);
    if (ok)
      __builtin_nontemporal_store(v2{cvt4_e4m3(v.x, v.y, sc), cvt4_e4m3(v.z, v.w, sc)},
                                  reinterpret_cast<v2*>(q + r * cols + c));
    if constexpr (kWhole) {   // 16 lanes hold a panel of 4 blocks
      const int ch = threadIdx.x & 15;
      uint32_t d = sb << (8 * (ch >> 2));
      d |= dpp_row_shr(d, 4);
      d |= dpp_row_shr(d, 8);
      if (ok && ch == 12) reinterpret_cast<uint32_t*>(s)[(c >> 7) * rows + r] = d;
    } else {
      if (ok && !(threadIdx.x & 3)) put_scale(s, rows, r, c >> 5, cols >> 5, sb);
    }
  };
  uint32_t o[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t x = tq_comp(g, k), y = tq_comp(u, k);
    o[k] = bf16x2_rne(swiglu1(bf_lo(x), bf_lo(y)), swiglu1(bf_hi(x), bf_hi(y)));
  }
  put(make_uint4(o[0], o[1], o[2], o[3]), row_q, row_s, F, col);
  put(g, keep_q, keep_s, 2 * F, col);
  put(u, keep_q, keep_s, 2 * F, F + col);
}

struct KeptBwd {
  const uint8_t* q;      // codes [rows, 2F]
  const uint8_t* s;      // their scales
  const uint16_t* da;    // bf16 [rows, F]
  int64_t rows, F;
  int32_t n_tc;
  uint8_t *row_q, *row_s, *col_q, *col_s;   // dH
  uint8_t *a_q, *a_s;                       // A' columnwise
  float* dots;           // [n_tc, rows] partial sums, or the sums where n_tc is 1; or null
};

// Sum over the 16 lanes of a DPP row.
__device__ __forceinline__ float row16_sum(float v) {
#define MX_DPP_ADD(ctrl) v += __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), ctrl, 0xF, 0xF, true))
  MX_DPP_ADD(0xB1);    // lane ^ 1
  MX_DPP_ADD(0x4E);    // lane ^ 2
  MX_DPP_ADD(0x141);   // the other quad of 8 lanes
  MX_DPP_ADD(0x140);   // the other 8 lanes
#undef MX_DPP_ADD
  return v;
}

// The backward in the quantizer's tiles of 128 rows x 128 columns: dH's two halves
// and A' are made from one reading of the codes and of dA, held in registers as
// bf16, and go out by rows and, through LDS, by columns.  67,584 x 2048: 273 us by
// itself, 4.7 TB/s; the arithmetic bounds it (65 instructions an element, exponential
// and five quantizes among them: 230 us of the vector units' issue).  67,520 rows take
// 284, as every second column's run of codes starts inside a line, and 312 between
// the other kernels of a backward, with the time of what they left to write.  Left to
// itself the compiler took 512 registers and spilled; bound to three tiles a CU,
// whole halves fit, and halves that share panels spill 13 registers.
// A row's tiles on one XCD and non-temporal columns leave whole lines as they are
// and mend shared ones: 67,584 x 2080 takes 295 us, 343 without (67,520: 314).
template <bool kWhole>
__global__ void __launch_bounds__(kTqThreads, 3) k_swiglu_bwd_kept(const KeptBwd p) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[kTq * kTq * 2];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, ch = lane & 15;
  // workgroup b runs on XCD b % 8: each takes a run of the tiles, by rows
  const uint32_t xcd = blockIdx.x % 8, each = gridDim.x / 8, more = gridDim.x % 8;
  const uint32_t b = xcd * each + (xcd < more ? xcd : more) + blockIdx.x / 8;
  const int32_t tc = (int32_t)(b % (uint32_t)p.n_tc);
  const int64_t r0 = (int64_t)(b / (uint32_t)p.n_tc) * kTq, r = r0 + 32 * w + 8 * (lane >> 4);
  const int64_t F = p.F, c0 = (int64_t)tc * kTq, col = c0 + 8 * ch;
  const bool col_ok = col < F;
  uint2 gq[8], uq[8];
  uint32_t gs[8], us[8];
  uint4 d[8];
  // Loads through buffers: past the rows' end they give zeros, and a lane keeps
  // one offset for all of its rows (as pointers they do not fit the registers).
  const int64_t left = p.rows - r0 < kTq ? p.rows - r0 : kTq;
  const __amdgpu_buffer_rsrc_t bq = buf(p.q + r0 * 2 * F, left * 2 * F), bd = buf(p.da + r0 * F, left * 2 * F);
  const uint32_t lr = (uint32_t)(r - r0), stride = (uint32_t)(2 * F);   // (both have rows of 2 F bytes)
  const uint32_t og = col_ok ? lr * stride + (uint32_t)col : kOob, od = col_ok ? lr * stride + 2u * (uint32_t)col : kOob;
  const uint32_t ou = col_ok ? og + (uint32_t)F : kOob;
  const uint8_t* sg = p.s + scale_index(p.rows, r, col >> 5);   // the rows' bytes are 4 apart
  const uint8_t* su = p.s + scale_index(p.rows, r, (F + col) >> 5);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    gq[i] = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(bq, (int)(og + i * stride), 0, 0));
    uq[i] = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(bq, (int)(ou + i * stride), 0, 0));
    d[i] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(bd, (int)(od + i * stride), 0, 0));
    gs[i] = us[i] = 0;
    if (r + i < p.rows && col_ok) {
      gs[i] = sg[4 * i];
      us[i] = su[4 * i];
    }
  }
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) most = max(most, max(gs[i], us[i]));
  const bool nans = __any(most == 255u);   // (looked at once for the wave: hardly ever)
  uint4 vg[8], vu[8], va[8];
  float mine = 0.0f;   // lane ch < 8: the dot of row r + ch
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint4 g4 = decode8(gq[i], gs[i]), u4 = decode8(uq[i], us[i]);
    if (nans) {
      nan_scale(g4, gs[i]);
      nan_scale(u4, us[i]);
    }
    float dot = 0.0f;
    uint32_t wg[4], wu[4], wa[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t x = tq_comp(g4, k), y = tq_comp(u4, k), z = tq_comp(d[i], k);
      const float gl = bf_lo(x), gh = bf_hi(x), ul = bf_lo(y), uh = bf_hi(y), dl = bf_lo(z), dh = bf_hi(z);
      const float al = swiglu1(gl, ul), ah = swiglu1(gh, uh);
      wg[k] = bf16x2_rne(swiglu_dgate(gl, ul, dl), swiglu_dgate(gh, uh, dh));
      wu[k] = bf16x2_rne(swiglu_dup(gl, dl), swiglu_dup(gh, dh));
      wa[k] = bf16x2_rne(al, ah);
      // rounded here: put off to their uses, the unrounded values of all rows would have to be kept
      asm volatile("" : "+v"(wg[k]), "+v"(wu[k]), "+v"(wa[k]));
      dot = fmaf(dl, al, dot);
      dot = fmaf(dh, ah, dot);
    }
    vg[i] = make_uint4(wg[0], wg[1], wg[2], wg[3]);
    vu[i] = make_uint4(wu[0], wu[1], wu[2], wu[3]);
    va[i] = make_uint4(wa[0], wa[1], wa[2], wa[3]);
    if (p.dots) {
      dot = row16_sum(dot);
      mine = ch == i ? dot : mine;
    }
    __builtin_amdgcn_sched_barrier(0);   // a row at a time: interleaved, the rows' terms do not fit the registers
  }
  if (p.dots && ch < 8 && r + ch < p.rows) p.dots[(int64_t)tc * p.rows + r + ch] = mine;
  if (p.row_q) {
    store_half<kWhole>(vg, p.row_q, p.row_s, p.rows, F, r, 0, c0, col_ok);
    store_half<kWhole>(vu, p.row_q, p.row_s, p.rows, F, r, F, c0, col_ok);
  }
  if (p.col_q) {
    tq_store_cols<true>(vg, lds, p.col_q, p.col_s, 2 * F, c0, F - c0, p.rows, r0);
    __syncthreads();
    tq_store_cols<true>(vu, lds, p.col_q, p.col_s, 2 * F, F + c0, F - c0, p.rows, r0);
  }
  if (p.a_q) {
    if (p.col_q) __syncthreads();
    tq_store_cols<true>(va, lds, p.a_q, p.a_s, F, c0, F - c0, p.rows, r0);
  }
}

// The tiles' partial sums of a row, in order (latency: 5 us at 16 x 67,584).
__global__ void __launch_bounds__(256) k_dots_join(const float* __restrict__ part, int64_t rows, int32_t n_tc,
                                                   float* __restrict__ dots) {
  const int64_t r = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (r >= rows) return;
  float t = 0.0f;
#pragma unroll 8
  for (int32_t c = 0; c < n_tc; ++c) t += part[(int64_t)c * rows + r];
  dots[r] = t;
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d, 64);
  return v;
}

// One wave per token: lane j holds the dot of its pair j (latency: 5 us at 8192
// tokens, top-8 of 64).
__global__ void __launch_bounds__(256) k_router_bwd_dots(const float* __restrict__ dots, int64_t rows,
                                                         const int32_t* __restrict__ dst_row,
                                                         const int32_t* __restrict__ ids,
                                                         const float* __restrict__ weights, int64_t tokens, int32_t E,
                                                         int32_t topk, float* __restrict__ dlogits) {
  const int64_t t = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (t >= tokens) return;
  const int lane = threadIdx.x & 63;
  float p = 0.0f, w = 0.0f;
  int32_t esel = -1;
  if (lane < topk) {
    const int32_t r = dst_row[t * topk + lane];
    if (r >= 0 && r < rows) p = dots[r];
    w = weights[t * topk + lane];
    esel = ids[t * topk + lane];
  }
  const float gsel = p - w * wave_sum(p);
  for (int e0 = 0; e0 < E; e0 += 64) {   // every lane stays in the loop: the others read its pair
    const int e = e0 + lane;
    float val = 0.0f;
    for (int32_t j = 0; j < topk; ++j) {
      const int32_t ej = __shfl(esel, j, 64);
      const float gj = __shfl(gsel, j, 64);
      if (ej == e) val += gj;   // (a repeated expert sums its terms)
    }
    if (e < E) dlogits[t * E + e] = val;
  }
}

// Source of the tile quantizer: rowwise MX rows, decoded; gathered or in order.
// The rows' scale dwords of the workgroup's column tiles come with the row table:
// loaded a byte at a time beside the codes they cost more than these.  8192 x 7168
// gathered to 67,584 rows: 129 us by itself, 184 between the other kernels of a
// backward, whose writes are still on their way (67,520 rows, whose columns start
// inside lines: 131 and 206); 560 MB in pieces of 128 bytes, which alone reach 5.3
// TB/s.  In order, 67,584 x 2048: 55 us, 5.1 TB/s; 67,520: 62.
template <bool kGather, int kTiles>
struct SrcMx {
  const uint8_t* q;
  const uint8_t* s;
  const int32_t* gather;
  int64_t rows_in, cols;
  struct Table {
    int32_t src[kTq];
    uint32_t sc[kTiles][kTq];
  };
  static constexpr bool kTable = true;
  static constexpr bool kGathered = kGather;
  static constexpr int kSub = kTiles;
  static constexpr bool kFetchAll = false;
  static constexpr bool kAhead = kTiles > 1;
  __device__ void fill_table(Table& tb, int64_t, int64_t r0, int64_t rows_out, int32_t tc0) const {
    const int t = threadIdx.x & (kTq - 1), half = threadIdx.x / kTq;
    const int64_t r = r0 + t;
    int64_t g = r < rows_out ? (kGather ? gather[r] : r) : -1;
    if (g >= rows_in) g = -1;
    if (half == 0) tb.src[t] = (int32_t)g;
    const uint32_t* sc = reinterpret_cast<const uint32_t*>(s) + (int64_t)tc0 * rows_in + g;
#pragma unroll
    for (int k = 0; k < (kTiles + 1) / 2; ++k) {
      const int i = 2 * k + half;
      if (i < kTiles) tb.sc[i][t] = g >= 0 && 128 * (int64_t)(tc0 + i) < cols ? sc[i * rows_in] : 0u;
    }
  }
  struct Row {
    bool ok;
    int32_t r;
    uint32_t sc;   // the lane's scale bytes of the tiles
  };
  __device__ Row row(const Table& tb, int64_t, int64_t, int lr, bool in_range) const {
    Row w;
    w.r = tb.src[lr];
    w.ok = in_range && w.r >= 0;
    w.sc = 0;
#pragma unroll
    for (int i = 0; i < kTiles; ++i) w.sc |= (tb.sc[i][lr] >> (8 * ((threadIdx.x & 15) >> 2)) & 0xFFu) << (8 * i);
    return w;
  }
  typedef uint2 Raw;
  __device__ Raw fetch(const Row& w, int64_t col, bool) const { return *reinterpret_cast<const uint2*>(q + w.r * cols + col); }
  __device__ uint4 finish(const Raw& x, const Row& w, int64_t col) const {
    const uint32_t sb = w.sc >> (kTiles > 1 ? 8 * ((uint32_t)(col >> 7) % kTiles) : 0) & 0xFFu;
    uint4 v = decode8(x, sb);
    nan_scale(v, sb);
    return v;
  }
};

template <bool kGather>
int launch_requantize(const uint8_t* q, const uint8_t* s, int64_t rows, int64_t cols, const int32_t* gather,
                      const TqShape& sh, unsigned tiles, const TqOut& o, hipStream_t st) {
  // four column tiles to a workgroup share the row table, where that leaves enough workgroups
  if (tiles >= 4 * 4 * 256) {
    const unsigned grid = (unsigned)((int64_t)sh.n_tr * ((sh.n_tc + 3) / 4));
    hipLaunchKernelGGL((k_tile_quant<SrcMx<kGather, 4>, false, true, false>), dim3(grid), dim3(kTqThreads), 0, st,
                       SrcMx<kGather, 4>{q, s, gather, rows, cols}, sh, o);
  } else {
    hipLaunchKernelGGL((k_tile_quant<SrcMx<kGather, 1>, false, true, false>), dim3(tiles), dim3(kTqThreads), 0, st,
                       SrcMx<kGather, 1>{q, s, gather, rows, cols}, sh, o);
  }
  return launch_status();
}

// 128 rows of H in bytes stay below the 2^31 of a buffer's offsets.
constexpr int64_t kMaxF = 1 << 22;

inline bool misaligned(const void* p, uintptr_t a) { return p && (reinterpret_cast<uintptr_t>(p) & (a - 1)); }

// A pair of codes and scales: both or none, codes aligned to `a`.
inline bool bad_pair(const uint8_t* q, const uint8_t* s, uintptr_t a) {
  return (q == nullptr) != (s == nullptr) || misaligned(q, a) || misaligned(s, 4);
}

}  // namespace
}  // namespace mx

using namespace mx;

extern "C" int mx_swiglu_keep(const uint16_t* h, int64_t rows, int64_t F, uint8_t* row_q, uint8_t* row_s,
                              uint8_t* keep_q, uint8_t* keep_s, mx_stream_t stream) {
  if (!h || !row_q || !keep_q || rows < 0 || F <= 0 || F % 32) return MX_EINVAL;
  if (misaligned(h, 16) || bad_pair(row_q, row_s, 8) || bad_pair(keep_q, keep_s, 8)) return MX_EINVAL;
  if (rows == 0) return MX_OK;
  const int64_t chunks = F / 8;
  if (F > kMaxF || rows >= (1ll << 32) / chunks) return MX_EUNSUPPORTED;   // threads of a launch
  const int64_t grid = (rows * chunks + 255) / 256;
  hipLaunchKernelGGL(F % 128 ? k_swiglu_keep<false> : k_swiglu_keep<true>, dim3((unsigned)grid), dim3(256), 0,
                     reinterpret_cast<hipStream_t>(stream), h, rows, F, (uint32_t)chunks, row_q, row_s, keep_q, keep_s);
  return launch_status();
}

extern "C" size_t mx_swiglu_bwd_kept_workspace_size(int64_t rows, int64_t F) {
  TqShape sh;
  unsigned grid;
  if (rows <= 0 || F <= 0 || F % 32 || F > kMaxF || !tq_shape(1, rows, F, sh, grid) || sh.n_tc == 1) return 0;
  return (size_t)(4 * rows * sh.n_tc);
}

extern "C" int mx_swiglu_bwd_kept(const uint8_t* keep_q, const uint8_t* keep_s, const uint16_t* da, int64_t rows,
                                  int64_t F, uint8_t* row_q, uint8_t* row_s, uint8_t* col_q, uint8_t* col_s,
                                  uint8_t* a_col_q, uint8_t* a_col_s, float* dots, void* workspace,
                                  size_t workspace_bytes, mx_stream_t stream) {
  if (!keep_q || !keep_s || !da || rows < 0 || F <= 0 || F % 32) return MX_EINVAL;
  if (bad_pair(keep_q, keep_s, 8) || misaligned(da, 16) || bad_pair(row_q, row_s, 8) || bad_pair(col_q, col_s, 16) ||
      bad_pair(a_col_q, a_col_s, 16) || misaligned(dots, 4) || misaligned(workspace, 16))
    return MX_EINVAL;
  if ((!row_q && !col_q && !a_col_q && !dots) || ((col_q || a_col_q) && rows % 32)) return MX_EINVAL;
  if (F > kMaxF) return MX_EUNSUPPORTED;
  if (rows == 0) return MX_OK;
  TqShape sh;
  unsigned grid;
  if (!tq_shape(1, rows, F, sh, grid)) return MX_EINVAL;
  const size_t need = dots ? mx_swiglu_bwd_kept_workspace_size(rows, F) : 0;
  if (need && (!workspace || workspace_bytes < need)) return MX_EINVAL;
  const hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  const KeptBwd p{keep_q, keep_s, da, rows, F, sh.n_tc, row_q, row_s, col_q, col_s, a_col_q, a_col_s,
                  need ? static_cast<float*>(workspace) : dots};
  hipLaunchKernelGGL((F % 128 ? k_swiglu_bwd_kept<false> : k_swiglu_bwd_kept<true>), dim3(grid), dim3(kTqThreads), 0, st, p);
  if (need)
    hipLaunchKernelGGL(k_dots_join, dim3((unsigned)((rows + 255) / 256)), dim3(256), 0, st,
                       static_cast<const float*>(workspace), rows, sh.n_tc, dots);
  return launch_status();
}

extern "C" int mx_router_bwd_dots(const float* dots, int64_t rows, const int32_t* dst_row, const int32_t* expert_ids,
                                  const float* weights, int64_t tokens, int32_t num_experts, int32_t topk,
                                  float* dlogits, mx_stream_t stream) {
  if (!dots || !dst_row || !expert_ids || !weights || !dlogits || rows < 0 || tokens < 0) return MX_EINVAL;
  if (num_experts < 1 || topk < 1 || topk > 64) return MX_EINVAL;
  if (tokens == 0) return MX_OK;
  const int64_t blocks = (tokens + 3) / 4;
  if (blocks > 0x7FFFFFFF) return MX_EINVAL;
  hipLaunchKernelGGL(k_router_bwd_dots, dim3((unsigned)blocks), dim3(256), 0, reinterpret_cast<hipStream_t>(stream),
                     dots, rows, dst_row, expert_ids, weights, tokens, num_experts, topk, dlogits);
  return launch_status();
}

extern "C" int mx_requantize(const uint8_t* q, const uint8_t* s, int64_t rows, int64_t cols, const int32_t* gather,
                             int64_t rows_out, uint8_t* col_q, uint8_t* col_s, mx_stream_t stream) {
  if (!q || !s || !col_q || rows < 0 || cols <= 0 || cols % 32 || rows_out < 0 || rows_out % 32) return MX_EINVAL;
  if (bad_pair(q, s, 8) || bad_pair(col_q, col_s, 16) || misaligned(gather, 4)) return MX_EINVAL;
  if (rows >= (1ll << 31)) return MX_EUNSUPPORTED;
  if (rows_out == 0) return MX_OK;
  TqShape sh;
  unsigned grid;
  if (!tq_shape(1, rows_out, cols, sh, grid)) return MX_EINVAL;
  const TqOut o = {nullptr, nullptr, col_q, col_s, nullptr};
  const hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  return gather ? launch_requantize<true>(q, s, rows, cols, gather, sh, grid, o, st)
                : launch_requantize<false>(q, s, rows, cols, gather, sh, grid, o, st);
}

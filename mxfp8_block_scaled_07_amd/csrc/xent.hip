// Softmax cross entropy over a large vocabulary, from the hidden rows and the
// output weights, with its gradient (gfx950):
//
//   z = x w^T,  lse_i = log sum_v exp z_iv,  loss_i = lse_i - z_{i, t_i}
//   dz = g_i (softmax(z_i) - onehot(t_i)),  dx = dz w,  dw = dz^T x
//
// The product's epilogue reduces a wave's columns of a row to their largest value
// m and the sum of exp(z - m) (a strip of 32 or 64 columns); a second launch joins
// a row's strips.  Without a gradient no logit is kept.  For the gradient the
// epilogue also leaves log2 exp(z - m) of a chunk of rows in 16 bits, so that a
// second product of the logits (a quarter of all the work) is saved; dz = g
// (exp(z - lse) - onehot) is rounded to bf16, the matrix instruction's operand,
// once.  The logarithm goes in even steps of 2^-10 from 0 to -64: half a step is
// 2^-11.5 of an exponential however small, an eleventh of the most that dz is rounded
// by afterwards, and one below 2^-64 of its strip's largest is zero.  (As fp16 the
// exponentials of the same 16 bits lose theirs from 2^-14 on and are zero below
// 2^-25: the gradients of words 10 to 17 nats under a neighbour.)  Chunks bound
// the workspace; with several, dw is added up in fp32.
//
// The products run in the tiles of product.h and bound the call: 4096 rows, 65536
// words, k 5120 with both gradients takes 6.3 ms (1.3 PFLOP/s), 2.0 the loss, 2.0 dx,
// 2.1 dw, 0.2 k_xent_dz; a library's three plain products of these shapes take
// 7.24.  Everything is added in a fixed order: repeated calls give the same bits.

#include "few_rows.h"
#include "product.h"

namespace mx {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }   // x <= 0

// Differences x <= 0 of logits as they are kept: -x log2 e in steps of kStep, to
// nearest; kNone and what is past it stand for exponentials of zero.  NaN may
// become anything (its row's lse is NaN).
constexpr float kStep = 64.0f / 65535.0f;
constexpr uint32_t kNone = 65535;
__device__ __forceinline__ uint32_t keep2(float a, float b) {
  constexpr float f = -kLog2e / 64.0f;
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pknorm_u16(a * f, b * f));   // of 65535, clamped
}

__device__ __forceinline__ float other_half(float v) { return __shfl_xor(v, 32, 64); }

struct XentArgs {
  const int32_t* targets;   // [I]
  float2* part;             // [strips, I]: a strip's largest logit and sum of exponentials
  float* zt;                // [I]: the target's logit
  uint16_t* e;              // [I, pitch]: z - m as keep2 gives it, kNone to the next multiple of 8 columns
  int64_t pitch;
};

template <bool kGrad>
struct XentEpi {
  typedef XentArgs Args;
  static constexpr int kSide = 16;
  template <int TM, int TN, typename Sums>
  __device__ static __forceinline__ void run(const XentArgs& p, v16f (&acc)[TM / 32][TN / 32], uint8_t* slice, int64_t i0,
                                             int64_t j0, int64_t I, int64_t J, Sums sums) {
    constexpr int FM = TM / 32, FN = TN / 32, kPitch = 2 * TN + 16;
    static_assert(32 * kPitch <= kStageBytes<TN>, "the slice holds 32 rows of 16 bits");
    const int lane = threadIdx.x & 63, h = lane >> 5;
    sums();
#pragma unroll
    for (int m = 0; m < FM; ++m) {
      const int64_t i = i0 + 32 * m + (lane & 31);
      float z[FN * 16];
#pragma unroll
      for (int r = 0; r < FN * 16; ++r) z[r] = acc[m][r / 16][r % 16];
      // the lane's column of register r: j0 + at(r) + 4 h
      auto at = [](int r) { return 32 * (r / 16) + 8 * (r % 16 / 4) + r % 4; };
      if (j0 + TN > J) {
#pragma unroll
        for (int r = 0; r < FN * 16; ++r)
          if (j0 + at(r) + 4 * h >= J) z[r] = -INFINITY;
      }
      float top = z[0];
#pragma unroll
      for (int r = 1; r < FN * 16; ++r) top = fmaxf(top, z[r]);
      top = fmaxf(top, other_half(top));
      const int64_t t = i < I ? p.targets[i] : -1;
      const int32_t rel = t >= j0 && t < J && t - j0 < TN ? (int32_t)(t - j0) : -1;   // the target's column, if it is here
      if (__any(rel >= 0)) {
#pragma unroll
        for (int r = 0; r < FN * 16; ++r)
          if (rel == at(r) + 4 * h) p.zt[i] = z[r];
      }
      const float ref = top == -INFINITY ? 0.0f : top;   // (a strip of nothing: exponentials of zero)
#pragma unroll
      for (int r = 0; r < FN * 16; ++r) z[r] -= ref;
      if constexpr (kGrad) {
#pragma unroll
        for (int g = 0; g < FN * 4; ++g)
          *reinterpret_cast<uint2*>(slice + (lane & 31) * kPitch + 2 * (at(4 * g) + 4 * h)) =
              make_uint2(keep2(z[4 * g], z[4 * g + 1]), keep2(z[4 * g + 2], z[4 * g + 3]));
        asm volatile("" ::: "memory");   // exchanged between the wave's lanes, whose LDS accesses run in order
        constexpr int kLpr = TN / 8, kRpp = 64 / kLpr;
#pragma unroll
        for (int it = 0; it < 32 / kRpp; ++it) {
          const int row = kRpp * it + lane / kLpr, c = 8 * (lane % kLpr);
          const uint4 v = *reinterpret_cast<const uint4*>(slice + row * kPitch + 2 * c);
          const int64_t ri = i0 + 32 * m + row;
          if (ri < I && j0 + c < J) *reinterpret_cast<uint4*>(p.e + ri * p.pitch + j0 + c) = v;
        }
        asm volatile("" ::: "memory");
      }
#pragma unroll
      for (int r = 0; r < FN * 16; ++r) z[r] = exp_of(z[r]);
#pragma unroll
      for (int w = FN * 8; w > 0; w /= 2)
#pragma unroll
        for (int r = 0; r < w; ++r) z[r] += z[r + w];
      const float s = z[0] + other_half(z[0]);
      if (h == 0 && i < I) p.part[j0 / TN * I + i] = make_float2(top, s);
      __builtin_amdgcn_sched_barrier(0);   // 32 rows at a time: interleaved, they do not fit the registers
    }
  }
};

// (m, s) and another strip's (m, s) to those of both.  A sum of zero stands for
// no words at all, whatever its m; a NaN is something.
__device__ __forceinline__ void join_strip(float& m, float& s, float m2, float s2) {
  const float n = fmaxf(s == 0.0f ? -INFINITY : m, s2 == 0.0f ? -INFINITY : m2);
  s = (s == 0.0f ? 0.0f : s * exp_of(m - n)) + (s2 == 0.0f ? 0.0f : s2 * exp_of(m2 - n));
  m = n;
}

// What k_skinny's sums become: a workgroup's strip of each row, in part [gridDim, M].
struct FewXent {
  const int32_t* targets;
  float2* part;
  float* zt;
  struct Ahead {
    int32_t t;
  };
  struct State {
    float m = -INFINITY, s = 0.0f;
  };
  __device__ __forceinline__ Ahead fetch(bool in, int m, int64_t, int64_t) const { return Ahead{in ? targets[m] : -1}; }
  __device__ __forceinline__ void finish(State& st, const Ahead& a, float (&v)[8], int m, int64_t j, int64_t N) const {
    float top = -INFINITY, s = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (j + k >= N) v[k] = -INFINITY;
      else if (j + k == a.t) zt[m] = v[k];
      top = fmaxf(top, v[k]);
    }
    const float ref = top == -INFINITY ? 0.0f : top;
#pragma unroll
    for (int k = 0; k < 8; ++k) s += exp_of(v[k] - ref);
    join_strip(st.m, st.s, top, s);
  }
  __device__ __forceinline__ void end(State& st, float* lds, int m, int item, int64_t M) const {
    float2* strips = reinterpret_cast<float2*>(lds);   // [2 kSkItems][kSkRows]
    lds_barrier();   // (the sums have been read)
    if (item < kSkItems && m < M) strips[(2 * item + (threadIdx.x & 1)) * kSkRows + m] = make_float2(st.m, st.s);
    lds_barrier();
    if ((int)threadIdx.x >= M) return;
    float top = -INFINITY, s = 0.0f;
    for (int k = 0; k < 2 * kSkItems; ++k) {
      const float2 v = strips[k * kSkRows + threadIdx.x];
      join_strip(top, s, v.x, v.y);
    }
    part[(int64_t)blockIdx.x * M + threadIdx.x] = make_float2(top, s);
  }
};

// Joins the rows' strips, and beside that copies x with zeros in the rows without
// a target: what they hold, infinities and NaN among it, must not reach dw (their
// dz is zero, which does not hide them).
struct JoinArgs {
  const float2* part;       // [strips, rows]
  int64_t rows;
  int32_t strips;
  const int32_t* targets;
  int64_t vocab;
  const float* zt;
  float* lse;               // for the gradient, or null
  float* lse_out;           // or null
  float* loss;              // or null
  uint32_t blocks;          // workgroups that join; those behind them copy
  const uint16_t* x;
  uint16_t* live;           // [rows, k]
  int64_t k;
};

// 16 rows per workgroup, 64 threads to a row: each takes every 64th strip, eight
// at a time, then the threads' strips are joined in a fixed order (a latency: 4.8
// us for 1000 rows of 512 strips, 20 with 4096 rows of 1024 and the copy of 42 MB).
__global__ void __launch_bounds__(1024) k_xent_join(const JoinArgs p) {
  if (blockIdx.x >= p.blocks) {
    const int64_t at = 8 * ((int64_t)(blockIdx.x - p.blocks) * 1024 + threadIdx.x);
    if (at >= p.rows * p.k) return;
    const int32_t t = p.targets[at / p.k];
    uint4 v = make_uint4(0, 0, 0, 0);
    if (t >= 0 && t < p.vocab) v = *reinterpret_cast<const uint4*>(p.x + at);
    *reinterpret_cast<uint4*>(p.live + at) = v;
    return;
  }
  __shared__ float2 sum[16][16];
  const int rl = threadIdx.x & 15, sl = threadIdx.x >> 4;
  const int64_t i = 16 * (int64_t)blockIdx.x + rl;
  float m = -INFINITY, s = 0.0f;
  if (i < p.rows) {
    for (int32_t k0 = sl; k0 < p.strips; k0 += 8 * 64) {
      float2 v[8];
      float top = -INFINITY, add = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = k0 + 64 * k < p.strips ? p.part[(int64_t)(k0 + 64 * k) * p.rows + i] : make_float2(0.0f, 0.0f);
#pragma unroll
      for (int k = 0; k < 8; ++k) top = fmaxf(top, v[k].y == 0.0f ? -INFINITY : v[k].x);
#pragma unroll
      for (int k = 0; k < 8; ++k) add += v[k].y == 0.0f ? 0.0f : v[k].y * exp_of(v[k].x - top);
      join_strip(m, s, top, add);
    }
  }
#pragma unroll
  for (int d = 16; d < 64; d *= 2) join_strip(m, s, __shfl_xor(m, d, 64), __shfl_xor(s, d, 64));
  if ((threadIdx.x & 63) < 16) sum[threadIdx.x >> 6][rl] = make_float2(m, s);
  __syncthreads();
  if (sl > 0 || i >= p.rows) return;
  for (int k = 1; k < 16; ++k) join_strip(m, s, sum[k][rl].x, sum[k][rl].y);
  const float l = m + logf(s);
  const int32_t t = p.targets[i];
  if (p.lse) p.lse[i] = l;
  if (p.lse_out) p.lse_out[i] = l;
  if (p.loss) p.loss[i] = t >= 0 && t < p.vocab ? l - p.zt[i] : 0.0f;
}

// dz in place of the kept logarithms: a thread takes 8 columns of a row in each of
// kDzStrips strips.  Rows without a target are zeros whatever they held.  HBM-bound:
// 4096 x 65536 takes 187 us, 5.7 TB/s.
constexpr int kDzStrips = 8;

template <int TN>
__global__ void __launch_bounds__(256) k_xent_dz(const float2* __restrict__ part, const float* __restrict__ lse,
                                                 const int32_t* __restrict__ targets,
                                                 const float* __restrict__ row_weight, int64_t rows, int64_t vocab,
                                                 int64_t pitch, uint32_t blocks_j, uint16_t* __restrict__ e) {
  constexpr int kLpr = TN / 8, kRows = 256 / kLpr;
  const int64_t i = (int64_t)(blockIdx.x / blocks_j) * kRows + threadIdx.x / kLpr;
  if (i >= rows) return;
  const int32_t t = targets[i];
  const bool live = t >= 0 && t < vocab;
  const float g = row_weight ? row_weight[i] : 1.0f, l = lse[i];
  const int32_t s0 = (int32_t)(blockIdx.x % blocks_j) * kDzStrips;
  uint4 v[kDzStrips];
  float m[kDzStrips];
#pragma unroll
  for (int s = 0; s < kDzStrips; ++s) {
    const int64_t c = (int64_t)(s0 + s) * TN + 8 * (threadIdx.x % kLpr);
    if (c < vocab) {
      v[s] = *reinterpret_cast<const uint4*>(e + i * pitch + c);
      m[s] = part[(int64_t)(s0 + s) * rows + i].x;
    }
  }
#pragma unroll
  for (int s = 0; s < kDzStrips; ++s) {
    const int64_t c = (int64_t)(s0 + s) * TN + 8 * (threadIdx.x % kLpr);
    if (c >= vocab) break;
    const float f = (m[s] - l) * kLog2e, none = f - INFINITY;   // (NaN in a row whose lse is NaN)
    auto exp_at = [&](uint32_t n) { return __builtin_amdgcn_exp2f(n == kNone ? none : fmaf((float)n, -kStep, f)); };
    const uint32_t w[4] = {v[s].x, v[s].y, v[s].z, v[s].w};
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float lo = g * exp_at(w[k] & 0xFFFFu), hi = g * exp_at(w[k] >> 16);
      if (c + 2 * k == t) lo -= g;
      if (c + 2 * k + 1 == t) hi -= g;
      o[k] = live ? bf16x2_rne(lo, hi) : 0u;
    }
    *reinterpret_cast<uint4*>(e + i * pitch + c) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// The gradients' epilogue: out = add + sums, in bf16 or fp32.  J % 8 == 0.
struct SumArgs {
  const float* add;   // fp32 [I, J] or null
  void* out;          // [I, J] (fp32: may be add)
  bool f32;
};

struct SumEpi {
  typedef SumArgs Args;
  static constexpr int kSide = 16;
  template <int TM, int TN, typename Sums>
  __device__ static __forceinline__ void run(const SumArgs& p, v16f (&acc)[TM / 32][TN / 32], uint8_t* slice, int64_t i0,
                                             int64_t j0, int64_t I, int64_t J, Sums sums) {
    constexpr int W = kStageCols<TN>, kPitch = W * 4 + 16, kLpr = W / 8, kRpp = 64 / kLpr;
    const int lane = threadIdx.x & 63;
    sums();
#pragma unroll
    for (int n0 = 0; n0 < TN / 32; n0 += W / 32) {
      const int64_t j = j0 + 32 * n0 + 8 * (lane % kLpr);
#pragma unroll
      for (int m = 0; m < TM / 32; ++m) {
#pragma unroll
        for (int n = 0; n < W / 32; ++n)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const v16f& a = acc[m][n0 + n];
            *reinterpret_cast<float4*>(slice + (lane & 31) * kPitch + (32 * n + 8 * g + 4 * (lane >> 5)) * 4) =
                make_float4(a[4 * g], a[4 * g + 1], a[4 * g + 2], a[4 * g + 3]);
          }
        asm volatile("" ::: "memory");   // exchanged between the wave's lanes, whose LDS accesses run in order
#pragma unroll
        for (int it = 0; it < 32 / kRpp; ++it) {
          const int row = kRpp * it + lane / kLpr;
          float4 x = *reinterpret_cast<const float4*>(slice + row * kPitch + 32 * (lane % kLpr));
          float4 y = *reinterpret_cast<const float4*>(slice + row * kPitch + 32 * (lane % kLpr) + 16);
          const int64_t i = i0 + 32 * m + row;
          if (i >= I || j >= J) continue;
          const int64_t o = i * J + j;
          if (p.add) {
            const float4 a = *reinterpret_cast<const float4*>(p.add + o), b = *reinterpret_cast<const float4*>(p.add + o + 4);
            x = make_float4(x.x + a.x, x.y + a.y, x.z + a.z, x.w + a.w);
            y = make_float4(y.x + b.x, y.y + b.y, y.z + b.z, y.w + b.w);
          }
          if (p.f32) {
            *reinterpret_cast<float4*>(static_cast<float*>(p.out) + o) = x;
            *reinterpret_cast<float4*>(static_cast<float*>(p.out) + o + 4) = y;
          } else {
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + o) =
                make_uint4(bf16x2_rne(x.x, x.y), bf16x2_rne(x.z, x.w), bf16x2_rne(y.x, y.y), bf16x2_rne(y.z, y.w));
          }
        }
        asm volatile("" ::: "memory");
      }
    }
  }
};

// ---------------------------------------------------------------- host side
// Columns of a wave in a tile shape.
int strip_cols(int shape) { return kShape[shape].bn >= 128 ? 64 : 32; }

int32_t strips_of(int64_t rows, int64_t vocab, int64_t k) {
  const int shape = plan_product(rows, vocab, k).shape;
  const int bn = kShape[shape].bn;
  return (int32_t)((vocab + bn - 1) / bn * (bn / strip_cols(shape)));
}

// Elements between the rows of z - m.  Long rows take whole lines, an odd
// number of 256 bytes, so that a column of rows falls on all of the memory's channels
// (4096 rows of 65536, k 5120, both gradients: 2.3% less time than a pitch of 65536);
// of short ones that would be a large part.
int64_t pitch_of(int64_t vocab) { return vocab < 4096 ? up(vocab, 8) : 128 * ((vocab + 127) / 128 | 1); }

// Rows that are in work together: their z - m and their copies of x
// (without a gradient: the strips' sums) take 2 GiB at most.
int64_t chunk_rows(int64_t rows, int64_t vocab, int64_t k, bool grad) {
  const int64_t row_bytes = grad ? 2 * (vocab > k ? pitch_of(vocab) : k) : (vocab + 255) / 256 * 8 * 8;
  int64_t most = (2ll << 30) / row_bytes / 256 * 256;
  if (most < 256) most = 256;
  if (rows <= most) return rows;
  const int64_t chunks = (rows + most - 1) / most;
  return up((rows + chunks - 1) / chunks, 256);
}

// Sections of the workspace.
struct XentSpace {
  int64_t chunk, pitch;
  int64_t e, part, row, x, acc, prod;   // bytes; row: of one float per row
};

// At most 16 rows without a gradient: w is streamed once through k_skinny.
bool streamed(int64_t rows, int64_t k, bool grad) { return !grad && few_rows(rows, k); }

XentSpace xent_space(int64_t rows, int64_t vocab, int64_t k, bool grad) {
  XentSpace s{};
  if (streamed(rows, k, grad)) {
    s.chunk = rows;
    s.part = up(8 * (int64_t)skinny_grid(vocab) * rows, 256);
    s.row = up(4 * rows, 256);
    return s;
  }
  s.chunk = chunk_rows(rows, vocab, k, grad);
  s.pitch = pitch_of(vocab);
  const int64_t last = rows % s.chunk ? rows % s.chunk : s.chunk;
  for (const int64_t r : {s.chunk, last}) {
    const int64_t part = up(8 * (int64_t)strips_of(r, vocab, k) * r, 256);
    if (part > s.part) s.part = part;
    int64_t prod = plan_product(r, vocab, k).part_bytes;
    if (grad) {
      const int64_t a = plan_product(r, k, vocab).part_bytes, b = plan_product(vocab, k, r).part_bytes;
      prod = prod > a ? prod : a;
      prod = prod > b ? prod : b;
    }
    if (prod > s.prod) s.prod = prod;
  }
  s.row = up(4 * s.chunk, 256);
  if (grad) {
    s.e = up(2 * s.chunk * s.pitch, 256);
    s.x = up(2 * s.chunk * k, 256);
    s.acc = s.chunk < rows ? 4 * vocab * k : 0;
  }
  return s;
}

int64_t total(const XentSpace& s) { return s.e + s.part + 2 * s.row + s.x + s.acc + s.prod; }

}  // namespace
}  // namespace mx

using namespace mx;

extern "C" size_t mx_bf16_xent_workspace_size(int64_t rows, int64_t vocab, int64_t k, int32_t backward) {
  if (rows <= 0 || vocab <= 0 || k <= 0 || k % 32 || too_large(rows, vocab, k)) return 0;
  return (size_t)total(xent_space(rows, vocab, k, backward != 0));
}

extern "C" int mx_bf16_xent(const uint16_t* x, const uint16_t* w, const int32_t* targets, const float* row_weight,
                            int64_t rows, int64_t vocab, int64_t k, float* loss, float* lse, uint16_t* dx, uint16_t* dw,
                            void* workspace, size_t workspace_bytes, mx_stream_t stream) {
  if (rows < 0 || vocab <= 0 || k <= 0 || k % 32 || !x || !w || !targets) return MX_EINVAL;
  if (!loss && !lse && !dx && !dw) return MX_EINVAL;
  if (misaligned(x) || misaligned(w) || misaligned(dx) || misaligned(dw) || misaligned(workspace)) return MX_EINVAL;
  if (((uintptr_t)targets | (uintptr_t)row_weight | (uintptr_t)loss | (uintptr_t)lse) & 3) return MX_EINVAL;
  if (too_large(rows, vocab, k)) return MX_EUNSUPPORTED;
  const bool grad = dx || dw;
  const hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (rows == 0) {
    if (!dw) return MX_OK;
    if (!tiles_fit(vocab, k, 0)) return MX_EUNSUPPORTED;
    return launch_tiles<false, false, SumEpi>(Operand{x, up(vocab, 8)}, Operand{x, k}, vocab, k, 0,
                                              SumArgs{nullptr, dw, false}, nullptr, st);   // a sum of nothing
  }
  const XentSpace s = xent_space(rows, vocab, k, grad);
  if (!workspace || (int64_t)workspace_bytes < total(s)) return MX_EINVAL;
  for (int64_t r0 = 0; r0 < rows; r0 += s.chunk) {
    const int64_t r = rows - r0 < s.chunk ? rows - r0 : s.chunk;
    if (streamed(rows, k, grad)) break;
    if (!tiles_fit(r, vocab, k) || (dx && !tiles_fit(r, k, vocab)) || (dw && !tiles_fit(vocab, k, r))) return MX_EUNSUPPORTED;
  }
  uint8_t* at = static_cast<uint8_t*>(workspace);
  auto take = [&](int64_t bytes) {
    uint8_t* p = at;
    at += bytes;
    return p;
  };
  uint16_t* e = reinterpret_cast<uint16_t*>(take(s.e));
  float2* part = reinterpret_cast<float2*>(take(s.part));
  float* zt = reinterpret_cast<float*>(take(s.row));
  float* own_lse = reinterpret_cast<float*>(take(s.row));
  uint16_t* xl = reinterpret_cast<uint16_t*>(take(s.x));
  float* acc = reinterpret_cast<float*>(take(s.acc));
  float* prod = reinterpret_cast<float*>(take(s.prod));

  for (int64_t r0 = 0; r0 < rows; r0 += s.chunk) {
    const int64_t r = rows - r0 < s.chunk ? rows - r0 : s.chunk;
    const uint16_t* xr = x + r0 * k;
    const int32_t* tr = targets + r0;
    const XentArgs a{tr, part, zt, e, s.pitch};
    const Operand ox{xr, k}, ow{w, k};
    JoinArgs j{part, r, 0, tr, vocab, zt, grad ? own_lse : nullptr, lse ? lse + r0 : nullptr, loss ? loss + r0 : nullptr,
               (uint32_t)((r + 15) / 16), xr, xl, k};
    int rc = MX_OK;
    if (streamed(rows, k, grad)) {
      j.strips = (int32_t)skinny_grid(vocab);
      hipLaunchKernelGGL(k_skinny<FewXent>, dim3(j.strips), dim3(64 * kSkWaves), 0, st, xr, w, r, vocab, k, FewXent{tr, part, zt});
    } else {
      j.strips = strips_of(r, vocab, k);
      rc = grad ? launch_tiles<true, true, XentEpi<true>>(ox, ow, r, vocab, k, a, prod, st)
                : launch_tiles<true, true, XentEpi<false>>(ox, ow, r, vocab, k, a, prod, st);
    }
    if (rc != MX_OK) return rc;
    const uint32_t copies = dw ? (uint32_t)((r * k / 8 + 1023) / 1024) : 0u;
    hipLaunchKernelGGL(k_xent_join, dim3(j.blocks + copies), dim3(1024), 0, st, j);
    if (!grad) continue;
    const int tn = strip_cols(plan_product(r, vocab, k).shape), per = 256 / (tn / 8);
    const uint32_t bj = (uint32_t)((vocab + kDzStrips * tn - 1) / (kDzStrips * tn));
    const dim3 grid((unsigned)(bj * ((r + per - 1) / per)));
    const float* rw = row_weight ? row_weight + r0 : nullptr;
    if (tn == 64) hipLaunchKernelGGL(k_xent_dz<64>, grid, dim3(256), 0, st, part, own_lse, tr, rw, r, vocab, s.pitch, bj, e);
    else hipLaunchKernelGGL(k_xent_dz<32>, grid, dim3(256), 0, st, part, own_lse, tr, rw, r, vocab, s.pitch, bj, e);
    const Operand dz{e, s.pitch};
    if (dx) {
      rc = launch_tiles<true, false, SumEpi>(dz, ow, r, k, vocab, SumArgs{nullptr, dx + r0 * k, false}, prod, st);
      if (rc != MX_OK) return rc;
    }
    if (dw) {
      const bool last = r0 + r == rows;
      const SumArgs sum{r0 ? acc : nullptr, last ? static_cast<void*>(dw) : acc, !last};
      rc = launch_tiles<false, false, SumEpi>(dz, Operand{xl, k}, vocab, k, r, sum, prod, st);
      if (rc != MX_OK) return rc;
    }
  }
  return launch_status();
}

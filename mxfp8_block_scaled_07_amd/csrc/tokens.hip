// The whole SwiGLU MoE layer for a few tokens (gfx950), from the router's
// logits to the combined rows, in two kernels:
//
//   [G; U] = W1_e x_t,  A = w_tj silu(G) U,  out_t = residual_t + sum_j W2_e A
//   with e = ids_tj the k largest logits of token t (equal logits to the lower
//   id, -inf never), w_tj their softmax.
//
// Bound: each active expert's weights have to come from HBM once (3 F H
// elements), and every other byte is small beside them.  The layer's path for
// many tokens pads each expert to 32 rows and makes eighteen launches; here
//   k_tokens_up    every workgroup routes all tokens by itself (a few hundred
//                  instructions per token, cheaper than a launch of its own),
//                  then takes items of 16 gate and 16 up rows of one active
//                  expert, its eight waves splitting H, and writes A;
//   k_tokens_down  a workgroup owns 16 rows of the output and reads them from
//                  every active expert's W2, its waves splitting experts and F.
// A is kept in bf16 (one rounding of w silu(G) U); everything else between
// the two roundings of bf16 inputs and outputs is fp32.  The weight goes into
// A so that the sum over a token's experts is one fp32 sum over its products.
// All sums have a fixed order: the result does not depend on scheduling.

#include "skinny.h"

namespace mx {
namespace {

constexpr int kMaxTokens = 64;     // one bit of a 64-bit mask each
constexpr int kTokExperts = 1024;  // as mx_route_topk
constexpr int kTokTopk = 64;
constexpr int kWaves = 8;
constexpr int kTokThreads = 64 * kWaves;

// Workspace: the routing table, then A [rows, F] in bf16.
//   int32 U; act[U] (expert), first[U + 1] (rows before it); uint8 token[rows]
struct Table {
  int32_t U, rows;
  int32_t pad[2];
  int32_t act[kTokExperts];
  int32_t first[kTokExperts + 1];
  int32_t pad2[3];
  uint8_t token[kMaxTokens * kTokTopk];
};
constexpr int64_t kTableBytes = (sizeof(Table) + 255) & ~(int64_t)255;

struct Routing {
  unsigned long long mask[kTokExperts];   // bit t: token t goes to the expert
  int32_t act[kTokExperts];
  int32_t first[kTokExperts + 1];
  int32_t U;
  float zmax[kMaxTokens], zsum[kMaxTokens];
  uint8_t token[kMaxTokens * kTokTopk];
  float weight[kMaxTokens * kTokTopk];
};

__device__ __forceinline__ float wave_max_f(float v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v = fmaxf(v, __shfl_xor(v, d, 64));
  return v;
}

__device__ __forceinline__ float wave_add_f(float v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d, 64);
  return v;
}

// Order-preserving integer key of a float (-0 as +0).
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}

__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

// One wave chooses token t's experts: the k-th largest key is built bit by
// bit from the top (the count of keys at or above a candidate is a ballot and
// a popcount; the search ends when a count is exactly k), ties at it go to
// the lowest ids.  Then the softmax statistics of the chosen.  kGroups: groups
// of 64 experts, one key of each per lane.
template <int kGroups>
__device__ __forceinline__ void route_token(Routing& rt, const float* __restrict__ row, int t, int E, int k) {
  const int lane = threadIdx.x & 63;
  uint32_t key[kGroups];
  uint32_t valid = 0, chosen = 0;
#pragma unroll
  for (int i = 0; i < kGroups; ++i) {
    const int e = lane + 64 * i;
    key[i] = order_key(e < E ? row[e] : 0.0f);
    valid |= (e < E ? 1u : 0u) << i;
  }
  uint32_t thr = 0;
  bool exact = false;
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t cand = thr | (1u << bit);
    int n = 0;
#pragma unroll
    for (int i = 0; i < kGroups; ++i) n += __popcll(__ballot((valid >> i & 1u) && key[i] >= cand));
    if (n >= k) thr = cand;
    if (n == k) {
      exact = true;
      break;
    }
  }
  int gt = 0;
#pragma unroll
  for (int i = 0; i < kGroups; ++i) {
    const bool in = (valid >> i & 1u) && (exact ? key[i] >= thr : key[i] > thr);
    if (in) chosen |= 1u << i;
    gt += __popcll(__ballot(in));
  }
  int left = k - gt;   // keys equal to the threshold still to take, lowest ids first
#pragma unroll
  for (int i = 0; i < kGroups; ++i) {
    const unsigned long long b = __ballot((valid >> i & 1u) && key[i] == thr);
    if ((b >> lane & 1u) && (int)__popcll(b & ((1ull << lane) - 1)) < left) chosen |= 1u << i;
    left -= __popcll(b);
  }
  float zm = -INFINITY;
#pragma unroll
  for (int i = 0; i < kGroups; ++i) {
    const float v = key_value(key[i]);
    if (v == -INFINITY) chosen &= ~(1u << i);   // masked: weight 0
    if (chosen >> i & 1u) zm = fmaxf(zm, v);
  }
  zm = wave_max_f(zm);
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < kGroups; ++i) {
    if (chosen >> i & 1u) {
      sum += expf(key_value(key[i]) - zm);
      atomicOr(&rt.mask[lane + 64 * i], 1ull << t);
    }
  }
  sum = wave_add_f(sum);
  if (lane == 0) {
    rt.zmax[t] = zm;
    rt.zsum[t] = sum;
  }
}

// The whole routing, by one workgroup.
__device__ void route_all(Routing& rt, const float* __restrict__ logits, int T, int E, int k) {
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  for (int e = tid; e < E; e += kTokThreads) rt.mask[e] = 0;
  __syncthreads();
  for (int t = wave; t < T; t += kWaves) {
    const float* row = logits + (int64_t)t * E;
    if (E <= 64) route_token<1>(rt, row, t, E, k);
    else if (E <= 256) route_token<4>(rt, row, t, E, k);
    else route_token<kTokExperts / 64>(rt, row, t, E, k);
  }
  __syncthreads();
  if (wave == 0) {
    int U = 0, rows = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
      const int e = e0 + lane;
      const int n = e < E ? __popcll(rt.mask[e]) : 0;
      const unsigned long long b = __ballot(n > 0);
      int s = n;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(s, d, 64);
        if (lane >= d) s += o;
      }
      if (n > 0) {
        const int u = U + __popcll(b & ((1ull << lane) - 1));
        rt.act[u] = e;
        rt.first[u] = rows + s - n;
      }
      U += __popcll(b);
      rows += __shfl(s, 63, 64);
    }
    if (lane == 0) {
      rt.first[U] = rows;
      rt.U = U;
    }
  }
  __syncthreads();
  // a thread per (active expert, token)
  for (int i = tid; i < 64 * rt.U; i += kTokThreads) {
    const int u = i >> 6, t = i & 63;
    const int e = rt.act[u];
    const unsigned long long m = rt.mask[e];
    if (m >> t & 1u) {
      const int r = rt.first[u] + __popcll(m & ((1ull << t) - 1));
      rt.token[r] = (uint8_t)t;
      rt.weight[r] = expf(logits[(int64_t)t * E + e] - rt.zmax[t]) / rt.zsum[t];
    }
  }
  __syncthreads();
}

struct TokensProblem {
  const uint16_t* x;
  const float* logits;
  int32_t T, k, E, H, F;
  const uint8_t *w1, *w1_s, *w2, *w2_s;
  const uint16_t* residual;
  uint16_t* out;
  Table* table;
  uint16_t* a;
};

template <bool kMx>
__device__ __forceinline__ WRows<kMx> expert_rows(const uint8_t* w, const uint8_t* s, int64_t e, int64_t E,
                                                  int64_t rows, int64_t cols) {
  WRows<kMx> m;
  m.q = buf(w + e * rows * cols * (kMx ? 1 : 2), rows * cols * (kMx ? 1 : 2));
  // scales of the expert's rows start 4 e rows into every panel
  m.s = kMx ? buf(s + 4 * e * rows, ((cols + 127) / 128 * E - e) * rows * 4) : m.q;
  m.panel = (uint32_t)(4 * E * rows);
  return m;
}

// One step of the up kernel in flight: gate and up weights, and the tokens of
// the item's first 16 rows.
template <bool kMx>
struct UpStep {
  WStep<kMx> g, u;
  XStep x;
};

// An item (active expert u, 16 columns f0 of F) as a wave walks it.
template <bool kMx>
struct UpItem {
  WRows<kMx> w;
  int32_t item, i, f0, lo, hi;   // i: the wave's step in the item
  uint32_t off;                  // the lane's token row of the first tile
};

template <bool kMx>
__device__ __forceinline__ void open_item(UpItem<kMx>& c, const TokensProblem& p, const Routing& rt, int item, int fb) {
  const int u = item / fb;
  const int e = __builtin_amdgcn_readfirstlane(rt.act[u]);
  c.item = item;
  c.i = 0;
  c.f0 = 16 * (item - u * fb);
  c.lo = __builtin_amdgcn_readfirstlane(rt.first[u]);
  c.hi = __builtin_amdgcn_readfirstlane(rt.first[u + 1]);
  c.w = expert_rows<kMx>(p.w1, p.w1_s, e, p.E, 2 * (int64_t)p.F, p.H);
  const int row = c.lo + (threadIdx.x & 15);
  c.off = row < c.hi ? 2u * (uint32_t)rt.token[row] * (uint32_t)p.H : kNoRow;
}

// kTiles: most tiles of 16 tokens an expert can have.  The loads run kDepth - 1
// steps ahead of the products, across items, so that the stream of weights does
// not pause for the reduction at an item's end.
template <bool kMx, int kTiles, int kDepth, int kOcc>
__global__ void __launch_bounds__(kTokThreads, kOcc) k_tokens_up(TokensProblem p) {
  __shared__ Routing rt;
  __shared__ float red[kWaves][2][4][64];
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int r = lane & 15;
  route_all(rt, p.logits, p.T, p.E, p.k);
  const int U = __builtin_amdgcn_readfirstlane(rt.U);
  if (blockIdx.x == 0) {
    if (tid == 0) {
      p.table->U = U;
      p.table->rows = rt.first[U];
    }
    for (int u = tid; u < U; u += kTokThreads) p.table->act[u] = rt.act[u];
    for (int u = tid; u <= U; u += kTokThreads) p.table->first[u] = rt.first[u];
    for (int i = tid; i < rt.first[U]; i += kTokThreads) p.table->token[i] = rt.token[i];
  }
  const int fb = p.F / 16, items = U * fb;
  if ((int)blockIdx.x >= items) return;
  const uint32_t H = (uint32_t)p.H;
  // a wave takes steps wave, wave + 8, ...; every wave as many (those past H read zeros)
  const int per = ((p.H + kStepK - 1) / kStepK + kWaves - 1) / kWaves;
  const __amdgpu_buffer_rsrc_t xr = buf(p.x, (int64_t)p.T * p.H * 2);
  UpItem<kMx> ld, cur;
  open_item(ld, p, rt, blockIdx.x, fb);
  cur = ld;
  bool more = true;
  UpStep<kMx> st[kDepth];
  auto load = [&](UpStep<kMx>& s) {
    if (!more) return;
    const uint32_t k0 = (uint32_t)(wave + kWaves * ld.i) * kStepK;
    load_w<kMx>(s.g, ld.w, (uint32_t)(ld.f0 + r), H, k0, true);
    load_w<kMx>(s.u, ld.w, (uint32_t)(p.F + ld.f0 + r), H, k0, true);
    load_x(s.x, xr, ld.off, H, k0);
    if (++ld.i == per) {
      more = ld.item + (int)gridDim.x < items;
      if (more) open_item(ld, p, rt, ld.item + gridDim.x, fb);
    }
  };
  v4f_s g[kTiles], up[kTiles];
#pragma unroll
  for (int t = 0; t < kTiles; ++t) g[t] = up[t] = v4f_s{0.f, 0.f, 0.f, 0.f};
  // one step's products; false after the workgroup's last item
  auto step = [&](UpStep<kMx>& s) -> bool {
    mma_step<kMx>(g[0], s.g, s.x);
    mma_step<kMx>(up[0], s.u, s.x);
#pragma unroll
    for (int t = 1; t < kTiles; ++t) {
      if (cur.lo + 16 * t < cur.hi) {   // an expert with more than 16 tokens
        const int row = cur.lo + 16 * t + r;
        XStep x;
        load_x(x, xr, row < cur.hi ? 2u * (uint32_t)rt.token[row] * H : kNoRow, H,
               (uint32_t)(wave + kWaves * cur.i) * kStepK);
        mma_step<kMx>(g[t], s.g, x);
        mma_step<kMx>(up[t], s.u, x);
      }
    }
    load(s);
    if (++cur.i < per) return true;
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      if (cur.lo + 16 * t < cur.hi) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          red[wave][0][i][lane] = g[t][i];
          red[wave][1][i][lane] = up[t][i];
        }
        g[t] = up[t] = v4f_s{0.f, 0.f, 0.f, 0.f};
        __syncthreads();
        // thread (token c, row f of 16): the waves' partial sums in order
        const int c = tid >> 4, f = tid & 15;
        const int row = cur.lo + 16 * t + c;
        if (tid < 256 && row < cur.hi) {
          float sg = 0.0f, su = 0.0f;
#pragma unroll
          for (int w = 0; w < kWaves; ++w) {
            sg += red[w][0][f & 3][16 * (f >> 2) + c];
            su += red[w][1][f & 3][16 * (f >> 2) + c];
          }
          const float a = rt.weight[row] * (sg / (1.0f + expf(-sg)) * su);
          p.a[(int64_t)row * p.F + cur.f0 + f] = (uint16_t)bf16x2_rne(a, a);
        }
        __syncthreads();
      }
    }
    if (cur.item + (int)gridDim.x >= items) return false;
    open_item(cur, p, rt, cur.item + gridDim.x, fb);
    return true;
  };
#pragma unroll
  for (int d = 0; d < kDepth; ++d) load(st[d]);
  bool on = true;
  while (on) {
#pragma unroll
    for (int d = 0; d < kDepth; ++d) on = on && step(st[d]);
  }
}

// One step of the down kernel in flight.
template <bool kMx>
struct DownStep {
  WStep<kMx> w;
  XStep x;
};

template <bool kMx>
struct DownUnit {
  WRows<kMx> w;
  int32_t c, s, s1, lo, hi;   // the unit; its step and end
  uint32_t off;
};

// Steps of a unit, the share of one expert's F that a wave takes at a time.
constexpr int kUnitSteps = 4;

// kNw waves: eight where the output's 16-row blocks give every CU two
// workgroups, sixteen where they are fewer.
template <bool kMx, int kNw, int kDepth, int kOcc>
__global__ void __launch_bounds__(64 * kNw, kOcc) k_tokens_down(TokensProblem p) {
  __shared__ int32_t act[kTokExperts], first[kTokExperts + 1];
  __shared__ uint8_t token[kMaxTokens * kTokTopk];
  __shared__ float sum[kNw][kMaxTokens][16];
  constexpr int kThreads = 64 * kNw;
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int r = lane & 15, h = lane >> 4;
  const int U = __builtin_amdgcn_readfirstlane(p.table->U);
  const int rows = __builtin_amdgcn_readfirstlane(p.table->rows);
  for (int u = tid; u < U; u += kThreads) act[u] = p.table->act[u];
  for (int u = tid; u <= U; u += kThreads) first[u] = p.table->first[u];
  for (int i = tid; i < rows; i += kThreads) token[i] = p.table->token[i];
  for (int i = lane; i < 16 * p.T; i += 64) (&sum[wave][0][0])[i] = 0.0f;
  __syncthreads();
  const uint32_t n0 = 16 * blockIdx.x, F = (uint32_t)p.F;
  const int steps = (p.F + kStepK - 1) / kStepK;
  const int per = (steps + kUnitSteps - 1) / kUnitSteps;
  const int units = U * per;
  const __amdgpu_buffer_rsrc_t ar = buf(p.a, (int64_t)rows * p.F * 2);
  auto open = [&](DownUnit<kMx>& q, int c) {
    const int u = c / per;
    q.c = c;
    q.s = (c - u * per) * kUnitSteps;
    q.s1 = q.s + kUnitSteps < steps ? q.s + kUnitSteps : steps;
    const int e = __builtin_amdgcn_readfirstlane(act[u]);
    q.lo = __builtin_amdgcn_readfirstlane(first[u]);
    q.hi = __builtin_amdgcn_readfirstlane(first[u + 1]);
    q.w = expert_rows<kMx>(p.w2, p.w2_s, e, p.E, p.H, p.F);
    q.off = q.lo + r < q.hi ? 2u * (uint32_t)(q.lo + r) * F : kNoRow;
  };
  if (wave < units) {
    DownUnit<kMx> ld, cur;
    open(ld, wave);
    cur = ld;
    bool more = true;
    DownStep<kMx> st[kDepth];
    auto load = [&](DownStep<kMx>& s) {
      if (!more) return;
      load_w<kMx>(s.w, ld.w, n0 + r, F, (uint32_t)(ld.s * kStepK), true);
      load_x(s.x, ar, ld.off, F, (uint32_t)(ld.s * kStepK));
      if (++ld.s == ld.s1) {
        more = ld.c + kNw < units;
        if (more) open(ld, ld.c + kNw);
      }
    };
    // the lane's sums of one tile's token
    auto flush = [&](const v4f_s& y, int row) {
      if (row < cur.hi) {
        float* d = sum[wave][token[row]] + 4 * h;
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] += y[i];
      }
    };
    v4f_s y = {0.f, 0.f, 0.f, 0.f};
    // one step's products; false after the wave's last unit
    auto step = [&](DownStep<kMx>& s) -> bool {
      mma_step<kMx>(y, s.w, s.x);
      for (int row0 = cur.lo + 16; row0 < cur.hi; row0 += 16) {   // an expert with more than 16 tokens
        XStep x;
        load_x(x, ar, row0 + r < cur.hi ? 2u * (uint32_t)(row0 + r) * F : kNoRow, F, (uint32_t)(cur.s * kStepK));
        v4f_s z = {0.f, 0.f, 0.f, 0.f};
        mma_step<kMx>(z, s.w, x);
        flush(z, row0 + r);
      }
      load(s);
      if (++cur.s < cur.s1) return true;
      flush(y, cur.lo + r);
      y = v4f_s{0.f, 0.f, 0.f, 0.f};
      if (cur.c + kNw >= units) return false;
      open(cur, cur.c + kNw);
      return true;
    };
#pragma unroll
    for (int d = 0; d < kDepth; ++d) load(st[d]);
    bool on = true;
    while (on) {
#pragma unroll
      for (int d = 0; d < kDepth; ++d) on = on && step(st[d]);
    }
  }
  __syncthreads();
  for (int i = tid; i < 16 * p.T; i += kThreads) {
    const int t = i >> 4, n = i & 15;
    float v = p.residual ? __uint_as_float((uint32_t)p.residual[(int64_t)t * p.H + n0 + n] << 16) : 0.0f;
#pragma unroll
    for (int w = 0; w < kNw; ++w) v += sum[w][t][n];
    p.out[(int64_t)t * p.H + n0 + n] = (uint16_t)bf16x2_rne(v, v);
  }
}

constexpr int kCus = 256;   // MI355X

template <bool kMx>
int launch_tokens(const TokensProblem& p, hipStream_t st) {
  const int64_t most = (int64_t)(p.E < p.T * p.k ? p.E : p.T * p.k) * (p.F / 16);
  // one up workgroup per CU with four (three) steps in flight per wave: 77 us for
  // one token of the 64-expert layer, against 84 with two workgroups and two steps
  const dim3 up((unsigned)(most < kCus ? most : kCus)), down(p.H / 16);
  if (p.T <= 16) hipLaunchKernelGGL((k_tokens_up<kMx, 1, 4, 2>), up, dim3(kTokThreads), 0, st, p);
  else hipLaunchKernelGGL((k_tokens_up<kMx, kMaxTokens / 16, 3, 2>), up, dim3(kTokThreads), 0, st, p);
  if (down.x > kCus) hipLaunchKernelGGL((k_tokens_down<kMx, 8, 3, 4>), down, dim3(512), 0, st, p);
  else hipLaunchKernelGGL((k_tokens_down<kMx, 16, 3, 4>), down, dim3(1024), 0, st, p);
  return launch_status();
}

int64_t tokens_bytes(int64_t tokens, int64_t topk, int64_t F) {
  return kTableBytes + ((tokens * topk * F * 2 + 255) & ~(int64_t)255);
}

int tokens_call(bool mxw, const uint16_t* x, const float* logits, int64_t tokens, int32_t topk, int32_t E, int64_t H,
                int64_t F, const void* w1, const uint8_t* w1_s, const void* w2, const uint8_t* w2_s,
                const uint16_t* residual, uint16_t* out, void* ws, size_t ws_bytes, mx_stream_t stream) {
  if (tokens < 0 || topk < 1 || E < 1 || topk > E || H <= 0 || F <= 0 || H % 32 || F % 32) return MX_EINVAL;
  if (!x || !logits || !w1 || !w2 || !out || !ws || (mxw && (!w1_s || !w2_s))) return MX_EINVAL;
  if (((uintptr_t)x | (uintptr_t)w1 | (uintptr_t)w2 | (uintptr_t)ws) & 15) return MX_EINVAL;
  if (((uintptr_t)logits | (uintptr_t)w1_s | (uintptr_t)w2_s) & 3) return MX_EINVAL;
  if (((uintptr_t)out | (uintptr_t)residual) & 1) return MX_EINVAL;
  if (tokens > kMaxTokens || E > kTokExperts || topk > kTokTopk) return MX_EUNSUPPORTED;
  // one expert's matrix and the scales are addressed with 31-bit byte offsets
  const int64_t eb = mxw ? 1 : 2;
  if (H >= (1ll << 24) || F >= (1ll << 24) || 2 * F * H * eb >= (1ll << 31)) return MX_EUNSUPPORTED;
  if (mxw && ((H + 127) / 128 * E * 2 * F * 4 >= (1ll << 31) || (F + 127) / 128 * E * H * 4 >= (1ll << 31)))
    return MX_EUNSUPPORTED;
  if (tokens * topk * F * 2 >= (1ll << 31) || tokens * H * 2 >= (1ll << 31)) return MX_EUNSUPPORTED;
  if (tokens == 0) return MX_OK;
  if ((int64_t)ws_bytes < tokens_bytes(tokens, topk, F)) return MX_EINVAL;
  TokensProblem p;
  p.x = x;
  p.logits = logits;
  p.T = (int32_t)tokens;
  p.k = topk;
  p.E = E;
  p.H = (int32_t)H;
  p.F = (int32_t)F;
  p.w1 = static_cast<const uint8_t*>(w1);
  p.w2 = static_cast<const uint8_t*>(w2);
  p.w1_s = w1_s;
  p.w2_s = w2_s;
  p.residual = residual;
  p.out = out;
  p.table = static_cast<Table*>(ws);
  p.a = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(ws) + kTableBytes);
  const hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  return mxw ? launch_tokens<true>(p, st) : launch_tokens<false>(p, st);
}

}  // namespace
}  // namespace mx

using namespace mx;

extern "C" size_t mx_moe_tokens_workspace_size(int64_t tokens, int32_t topk, int32_t num_experts, int64_t F) {
  if (tokens < 0 || topk < 1 || num_experts < 1 || F <= 0) return 0;
  if (tokens > kMaxTokens || topk > kTokTopk || F >= (1ll << 24)) return 0;
  return (size_t)tokens_bytes(tokens, topk, F);
}

extern "C" int mx_moe_tokens(const uint16_t* x, const float* logits, int64_t tokens, int32_t topk,
                             int32_t num_experts, int64_t H, int64_t F, const uint8_t* w1_q, const uint8_t* w1_s,
                             const uint8_t* w2_q, const uint8_t* w2_s, const uint16_t* residual, uint16_t* out,
                             void* workspace, size_t workspace_bytes, mx_stream_t stream) {
  return tokens_call(true, x, logits, tokens, topk, num_experts, H, F, w1_q, w1_s, w2_q, w2_s, residual, out,
                     workspace, workspace_bytes, stream);
}

extern "C" int mx_bf16_moe_tokens(const uint16_t* x, const float* logits, int64_t tokens, int32_t topk,
                                  int32_t num_experts, int64_t H, int64_t F, const uint16_t* w1, const uint16_t* w2,
                                  const uint16_t* residual, uint16_t* out, void* workspace, size_t workspace_bytes,
                                  mx_stream_t stream) {
  return tokens_call(false, x, logits, tokens, topk, num_experts, H, F, w1, nullptr, w2, nullptr, residual, out,
                     workspace, workspace_bytes, stream);
}

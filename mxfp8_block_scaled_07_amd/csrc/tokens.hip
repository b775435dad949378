// The whole SwiGLU MoE layer for a few tokens (gfx950), from the router's
// logits to the combined rows:
//
//   [G; U] = W1_e x_t,  A = w_tj silu(G) U,  out_t = residual_t + sum_j W2_e A
//   with e = ids_tj the k largest logits of token t (equal logits to the lower
//   id, -inf never), w_tj their softmax.
//
// Bound: each active expert's weights have to come from HBM once (3 F H
// elements), and every other byte is small beside them.  An expert with more
// rows than the up kernel's register tiles hold (16 above H = 4096, 32 above
// 2048, else 64) is several entries, and its weights are walked once for each:
// H = 7168, F = 2048, 2 experts, top-1, MXFP8 takes 33 us for 16 tokens (8 rows
// an expert) and 53 for 64.  The layer's path for many tokens pads each expert
// to 32 rows and makes eighteen launches; here
//   k_tokens_up    every workgroup routes all tokens by itself (a few hundred
//                  instructions per token, cheaper than a launch of its own),
//                  then takes a run of items: 16 gate and 16 up rows of one
//                  active expert, its eight waves splitting H; writes A
//   k_tokens_down  groups of 128 output rows, 16 per wave, over the active
//                  experts' F; the groups' work is cut evenly over the card
//   k_tokens_join  adds the pieces of a group in order (where it was cut)
//
// The weights stream through LDS as in stream.h.  What then costs is every
// other vector load beside the stream: reading the tokens again for each step
// took 10% of the up kernel and 28% of the down kernel (33 tokens).  So the up
// kernel keeps its waves' share of the tokens in registers while it stays with
// an expert, and the down kernel's waves share theirs through LDS.
//
// 64 experts of 2048 x 7168, top-8, MXFP8: one token 68 us (up 42, down 23, join
// 4.5; 5.3 TB/s of weights), 33 tokens 440 us (6.5 TB/s); 61 tokens, 8 experts of
// 1408 x 2048 in bf16 48 us.
//
// A is kept in bf16 (one rounding of w silu(G) U), the type of the matrix
// instruction's operand: a second bf16 term of it would double the down kernel's
// products and its loads beside the stream, for an error that goes from 0.0017
// to 0.0019-0.0023 of the result, whose own rounding is most of that.  Everything
// else between the bf16 inputs and outputs is fp32.  The weight goes into A so
// that the sum over a token's experts is one fp32 sum.  All sums have a fixed
// order: the result does not depend on scheduling.

#include "stream.h"

namespace mx {
namespace {

constexpr int kMaxTokens = 64;     // one bit of a 64-bit mask each
constexpr int kTokExperts = 1024;  // as mx_route_topk
constexpr int kTokTopk = 64;
constexpr int kMaxRows = kMaxTokens * kTokTopk;
constexpr int kEntries = kTokExperts + kMaxRows / 16;
constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;

// Entries: an active expert's rows (token, expert pairs) in groups of at most
// the up kernel's token tiles.  The workspace holds the table for the down
// kernel, the pieces of the output, then A [rows, F] in bf16.
struct Table {
  int32_t entries, rows;
  int32_t tiles;                    // 16-row tiles of all entries
  int32_t pad;
  int32_t expert[kEntries];
  int32_t first[kEntries + 1];      // rows before the entry
  int32_t tile[kEntries + 1];       // tiles before the entry
  uint8_t token[kMaxRows];
};
constexpr int64_t kTableBytes = (sizeof(Table) + 255) & ~(int64_t)255;

struct Routing {
  unsigned long long mask[kTokExperts];   // bit t: token t goes to the expert
  int32_t expert[kEntries];
  int32_t first[kEntries + 1];
  int32_t entries;
  float zmax[kMaxTokens], zsum[kMaxTokens];
  uint8_t token[kMaxRows];
  float weight[kMaxRows];
};

// Reductions over the wave by DPP: rows of 16 lanes, then their last lanes
// into the rows after them; lane 63 holds the result.
template <int kCtrl, int kRows>
__device__ __forceinline__ float dpp(float old, float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp((int)__float_as_uint(old), (int)__float_as_uint(v), kCtrl,
                                                               kRows, 0xF, false));
}
__device__ __forceinline__ float last_lane(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}
__device__ __forceinline__ float wave_max_f(float v) {
  v = fmaxf(v, dpp<0x111, 0xF>(v, v));        // row_shr 1, 2, 4, 8 (a lane without a source keeps its own)
  v = fmaxf(v, dpp<0x112, 0xF>(v, v));
  v = fmaxf(v, dpp<0x114, 0xF>(v, v));
  v = fmaxf(v, dpp<0x118, 0xF>(v, v));
  v = fmaxf(v, dpp<0x142, 0xA>(v, v));        // row_bcast 15 into rows 1 and 3
  v = fmaxf(v, dpp<0x143, 0xC>(v, v));        // row_bcast 31 into rows 2 and 3
  return last_lane(v);
}
__device__ __forceinline__ float wave_add_f(float v) {
  v += dpp<0x111, 0xF>(0.0f, v);
  v += dpp<0x112, 0xF>(0.0f, v);
  v += dpp<0x114, 0xF>(0.0f, v);
  v += dpp<0x118, 0xF>(0.0f, v);
  v += dpp<0x142, 0xA>(0.0f, v);
  v += dpp<0x143, 0xC>(0.0f, v);
  return last_lane(v);
}

// Order-preserving integer key of a float (-0 as +0).  A NaN of either sign has
// the largest, so that it is always chosen and its token's row becomes NaN: by
// its bits a negative one would sort below -inf and be dropped.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  return v != v ? 0xFFFFFFFFu : b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}

__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

// One wave chooses a token's experts: the k-th largest key is built bit by bit
// from the top (the count of keys at or above a candidate is a ballot and a
// popcount; the search ends when a count is exactly k), ties at it go to the
// lowest ids.  Then the softmax statistics of the chosen.  kGroups: groups of
// 64 experts, one key of each per lane; key 0, which no logit has, where there
// is no expert.
template <int kGroups>
__device__ __forceinline__ void route_token(Routing& rt, const uint32_t (&key)[kGroups], int t, int k) {
  const int lane = threadIdx.x & 63;
  uint32_t thr = 0;
  bool exact = false;
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t cand = thr | (1u << bit);
    int n = 0;
#pragma unroll
    for (int i = 0; i < kGroups; ++i) n += (int)__popcll(__ballot(key[i] >= cand));
    if (n >= k) thr = cand;
    if (n == k) {
      exact = true;
      break;
    }
  }
  uint32_t chosen = 0;
  int gt = 0;
#pragma unroll
  for (int i = 0; i < kGroups; ++i) {
    const bool in = key[i] >= thr + (exact ? 0u : 1u) && thr + (exact ? 0u : 1u) != 0u;
    chosen |= (in ? 1u : 0u) << i;
    gt += (int)__popcll(__ballot(in));
  }
  int left = k - gt;   // keys equal to the threshold still to take, lowest ids first
#pragma unroll
  for (int i = 0; i < kGroups; ++i) {
    const unsigned long long b = __ballot(!exact & (key[i] == thr) & (key[i] != 0u));
    const bool in = (b >> lane & 1u) && (int)__popcll(b & ((1ull << lane) - 1)) < left;
    chosen |= (in ? 1u : 0u) << i;
    left -= (int)__popcll(b);
  }
  float zm = -INFINITY;
#pragma unroll
  for (int i = 0; i < kGroups; ++i) {
    const float v = key_value(key[i]);
    if (v == -INFINITY) chosen &= ~(1u << i);   // masked: weight 0
    zm = (chosen >> i & 1u) ? fmaxf(zm, v) : zm;
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

template <int kGroups>
__device__ __forceinline__ void route_wave(Routing& rt, const float* __restrict__ logits, int T, int E, int k) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  uint32_t next[kGroups];
  auto fetch = [&](int t) {
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      const int e = lane + 64 * i;
      next[i] = e < E ? __float_as_uint(logits[(int64_t)t * E + e]) : 0u;
    }
  };
  if (wave < T) fetch(wave);
  for (int t = wave; t < T; t += kWaves) {
    uint32_t key[kGroups];
#pragma unroll
    for (int i = 0; i < kGroups; ++i) key[i] = lane + 64 * i < E ? order_key(__uint_as_float(next[i])) : 0u;
    if (t + kWaves < T) fetch(t + kWaves);   // in flight while this token is routed
    route_token<kGroups>(rt, key, t, k);
  }
}

// The routing, by one workgroup: entries of at most `group` rows ...
__device__ __forceinline__ void route_entries(Routing& rt, const float* __restrict__ logits, int T, int E, int k, int group) {
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  for (int e = tid; e < E; e += kThreads) rt.mask[e] = 0;
  __syncthreads();
  if (E > 256) route_wave<kTokExperts / 64>(rt, logits, T, E, k);
  else if (E > 64) route_wave<4>(rt, logits, T, E, k);
  else route_wave<1>(rt, logits, T, E, k);
  __syncthreads();
  if (wave == 0) {
    int V = 0, rows = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
      const int e = e0 + lane;
      const int n = e < E ? (int)__popcll(rt.mask[e]) : 0;
      const int g = (n + group - 1) / group;
      int s = n, v = g;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(s, d, 64), q = __shfl_up(v, d, 64);
        if (lane >= d) {
          s += o;
          v += q;
        }
      }
      for (int i = 0; i < g; ++i) {
        rt.expert[V + v - g + i] = e;
        rt.first[V + v - g + i] = rows + s - n + i * group;
      }
      V += __shfl(v, 63, 64);
      rows += __shfl(s, 63, 64);
    }
    if (lane == 0) {
      rt.first[V] = rows;
      rt.entries = V;
    }
  }
  __syncthreads();
}

// ... and then their rows' tokens and weights: a thread per (entry, token);
// the entries of one expert share its mask.  (The caller's barrier follows.)
__device__ __forceinline__ void route_rows(Routing& rt, const float* __restrict__ logits, int E) {
  const int tid = threadIdx.x;
  for (int i = tid; i < 64 * rt.entries; i += kThreads) {
    const int u = i >> 6, t = i & 63;
    const int e = rt.expert[u];
    const unsigned long long m = rt.mask[e];
    if ((m >> t & 1u) && (u == 0 || rt.expert[u - 1] != e)) {
      const int r = rt.first[u] + (int)__popcll(m & ((1ull << t) - 1));
      rt.token[r] = (uint8_t)t;
      rt.weight[r] = expf(logits[(int64_t)t * E + e] - rt.zmax[t]) / rt.zsum[t];
    }
  }
}

struct TokensProblem {
  const uint16_t* x;
  const float* logits;
  int32_t T, k, E, H, F;
  const uint8_t *w1, *w1_s, *w2, *w2_s;
  const uint16_t* residual;
  uint16_t* out;
  Table* table;
  float* part;      // pieces of the output, or null: one workgroup per group of rows writes it
  uint16_t* a;
};

// ---------------------------------------------------------------- the stream
// Scales of an expert's rows start 4 e rows into every panel.
__device__ __forceinline__ v4u scale_rsrc(const uint8_t* s, int64_t e, int64_t E, int64_t rows, int64_t cols) {
  return rsrc(s + 4 * e * rows, ((cols + 127) / 128 * E - e) * rows * 4);
}

// ---------------------------------------------------------------- up
constexpr int kUpDepth = 3;                        // steps of a wave in flight
constexpr int kUpSlot = 2 * 2048 + 256;            // gate and up blocks, their scale dwords

// The table for the down kernel, by one workgroup.
__device__ void write_table(const Routing& rt, Table* table) {
  const int tid = threadIdx.x, lane = tid & 63;
  const int V = rt.entries, rows = rt.first[V];
  for (int u = tid; u < V; u += kThreads) table->expert[u] = rt.expert[u];
  for (int u = tid; u <= V; u += kThreads) table->first[u] = rt.first[u];
  for (int i = tid; i < rows; i += kThreads) table->token[i] = rt.token[i];
  if (tid < 64) {   // tiles before each entry
    int before = 0;
    for (int u0 = 0; u0 < V; u0 += 64) {
      const int u = u0 + lane;
      const int n = u < V ? (rt.first[u + 1] - rt.first[u] + 15) / 16 : 0;
      int s = n;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(s, d, 64);
        if (lane >= d) s += o;
      }
      if (u < V) table->tile[u] = before + s - n;
      before += __shfl(s, 63, 64);
    }
    if (lane == 0) {
      table->tile[V] = before;
      table->tiles = before;
      table->entries = V;
      table->rows = rows;
    }
  }
}

// kSteps: steps of a wave whose tokens stay in registers, for kTiles tiles of
// 16 tokens (128 registers in all).  kSteps * 8 lines cover H, or the tokens
// are read again for each item.
template <bool kMx, int kSteps, int kTiles>
__global__ void __launch_bounds__(kThreads, 2) k_tokens_up(TokensProblem p) {
  __shared__ Routing rt;
  __shared__ __attribute__((aligned(16))) float red[kWaves][2][4][64];
  __shared__ __attribute__((aligned(1024))) uint8_t ring[kWaves][kUpDepth][kUpSlot];
  constexpr int kOps = kMx ? 5 : 4, eb = kMx ? 1 : 2, kK = kLineK<kMx>, kP = kXp<kMx>;
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int r = lane & 15, h = lane >> 4;
  route_entries(rt, p.logits, p.T, p.E, p.k, 16 * kTiles);
  // ahead of the stream: its reads of the logits are compiled loads, and waiting
  // for them would wait for the stream's too.  Behind the first loads 61 tokens
  // on 8 experts of 1408 x 2048 take 51 us, here 49; one token 67.5 either way.
  route_rows(rt, p.logits, p.E);
  lds_barrier();
  const int V = __builtin_amdgcn_readfirstlane(rt.entries);
  // the last workgroup writes the table; it has items too where every CU has
  const int takers = gridDim.x == kCus ? kCus : gridDim.x - 1;
  const bool scribe = blockIdx.x == gridDim.x - 1;
  if (scribe && takers < (int)gridDim.x) {
    write_table(rt, p.table);
    return;
  }
  const int fb = p.F / 16, items = V * fb;
  const int begin = (int)((int64_t)items * blockIdx.x / takers);
  const int end = (int)((int64_t)items * (blockIdx.x + 1) / takers);
  if (begin >= end) {
    if (scribe) write_table(rt, p.table);
    return;
  }
  const int lines = (p.H * eb + 127) / 128;
  const int per = (lines + kWaves - 1) / kWaves;   // a wave takes lines wave, wave + 8, ...
  const int64_t rows = 2 * (int64_t)p.F, row_bytes = (int64_t)p.H * eb;

  // the loads' cursor; a lane's offsets are the same for every item and line
  int li = begin, ls = 0, seq = 0;
  uint32_t lrow = 0, lrow_s = 0;   // the item's first row, in weight and scale bytes
  v4u lq, lsc;
  auto open = [&](int item) {
    const int u = item / fb;
    const int64_t e = __builtin_amdgcn_readfirstlane(rt.expert[u]);
    const int f = 16 * (item - u * fb);
    lrow = (uint32_t)f * (uint32_t)row_bytes;
    lrow_s = 4u * (uint32_t)f;
    lq = rsrc(p.w1 + e * rows * row_bytes, rows * row_bytes);
    if constexpr (kMx) lsc = scale_rsrc(p.w1_s, e, p.E, rows, p.H);
  };
  open(begin);
  const uint32_t half = (uint32_t)p.F * (uint32_t)row_bytes, panel = 4u * (uint32_t)p.E * (uint32_t)rows;
  uint32_t lane_off[2];
  int32_t lane_c[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int row = 8 * q + (lane >> 3);
    lane_c[q] = 16 * ((lane & 7) ^ chunk_swizzle(row));
    lane_off[q] = (uint32_t)row * (uint32_t)row_bytes + (uint32_t)lane_c[q];
  }
  const uint32_t lane_s = lane < 32 ? 4u * (uint32_t)((lane >> 4) * p.F + r) : kOob;
  auto load = [&]() {
    const uint32_t dst = lds_addr(ring[wave][0]) + (uint32_t)(seq % kUpDepth) * kUpSlot;
    const int line = wave + kWaves * ls;
    const bool in = li < end && line < lines;
    const uint32_t soff = in ? 128u * (uint32_t)line + lrow : 0u;
    const int32_t left = in ? (int32_t)(row_bytes - 128 * (int64_t)line) : 0;   // bytes of the row from here on
#pragma unroll
    for (int q = 0; q < 4; ++q)
      dma16_nt(lq, dst + 1024u * q, lane_c[q & 1] < left ? lane_off[q & 1] : kOob, soff + (in ? (q >> 1) * half : 0u));
    if constexpr (kMx) dma4(lsc, dst + 4096u, in ? lane_s : kOob, in ? (uint32_t)line * panel + lrow_s : 0u);
    ++seq;
    if (++ls == per) {
      ls = 0;
      if (++li < end) open(li);
    }
  };

  // the tokens of `line` .. of the entry's tiles
  v8bf x[kTiles][kSteps][kP];
  auto tokens = [&](int lo, int hi, int s0) {
    const __amdgpu_buffer_rsrc_t xr =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(p.x), (short)0, (int)(2 * p.T * p.H), 0x00020000);
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      const int row = lo + 16 * t + r;
      const uint32_t base = row < hi ? 2u * (uint32_t)rt.token[row] * (uint32_t)p.H : kOob;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const int k = (wave + kWaves * (s0 + s)) * kK + kK / 4 * h;
        const uint32_t off = (row < hi && k < p.H) ? base + 2u * (uint32_t)k : kOob;
#pragma unroll
        for (int j = 0; j < kP; ++j)
          x[t][s][j] = __builtin_bit_cast(v8bf, __builtin_amdgcn_raw_buffer_load_b128(xr, (int)off + 16 * j, 0, 0));
      }
    }
  };

  int entry = begin / fb, used = 0;
  tokens(__builtin_amdgcn_readfirstlane(rt.first[entry]), __builtin_amdgcn_readfirstlane(rt.first[entry + 1]), 0);
#pragma unroll 1
  for (int d = 0; d < kUpDepth; ++d) load();
  if (scribe) write_table(rt, p.table);
  // the tokens are waited for here, ahead of the stream (by itself the compiler
  // would wait at each use, and for the stream's loads too)
  __builtin_amdgcn_s_waitcnt(waitcnt_vm(kOps * kUpDepth));
  for (int item = begin; item < end; ++item) {
    const int u = item / fb, f0 = 16 * (item - u * fb);
    const int lo = __builtin_amdgcn_readfirstlane(rt.first[u]), hi = __builtin_amdgcn_readfirstlane(rt.first[u + 1]);
    v4f g[kTiles], up[kTiles];
#pragma unroll
    for (int t = 0; t < kTiles; ++t) g[t] = up[t] = v4f{0.f, 0.f, 0.f, 0.f};
    for (int s0 = 0; s0 < per; s0 += kSteps) {
      if (u != entry || (per > kSteps && (s0 || item > begin))) {
        tokens(lo, hi, s0);
        __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
        entry = u;
      }
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        if (s0 + s < per) {
          // the oldest step's loads are done, the others may be in flight
          fence();
          __builtin_amdgcn_s_waitcnt(waitcnt_vm(kOps * (kUpDepth - 1)));
          fence();
          const uint8_t* slot = ring[wave][used % kUpDepth];
          const Fragment fg = read_fragment<kMx>(slot, slot + 4096), fu = read_fragment<kMx>(slot + 2048, slot + 4096 + 64);
          fence();
          __builtin_amdgcn_s_waitcnt(kWaitLgkm0);   // read: the slot is free
          fence();
          load();
          ++used;
          const float sg = fragment_scale<kMx>(fg), su = fragment_scale<kMx>(fu);
#pragma unroll
          for (int j = 0; j < kP; ++j) {
            const v8bf wg = weights8<kMx>(fg, j, sg), wu = weights8<kMx>(fu, j, su);
#pragma unroll
            for (int t = 0; t < kTiles; ++t) {
              if (t == 0 || lo + 16 * t < hi) {
                g[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wg, x[t][s][j], g[t], 0, 0, 0);
                up[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wu, x[t][s][j], up[t], 0, 0, 0);
              }
            }
          }
        }
      }
    }
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      if (lo + 16 * t < hi) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          red[wave][0][i][lane] = g[t][i];
          red[wave][1][i][lane] = up[t][i];
        }
        lds_barrier();
        // thread (token c, row f of 16): the waves' partial sums in order
        const int c = tid >> 4, f = tid & 15;
        const int row = lo + 16 * t + c;
        if (tid < 256 && row < hi) {
          float sg = 0.0f, su = 0.0f;
#pragma unroll
          for (int w = 0; w < kWaves; ++w) {
            sg += red[w][0][f & 3][16 * (f >> 2) + c];
            su += red[w][1][f & 3][16 * (f >> 2) + c];
          }
          const float a = rt.weight[row] * (sg / (1.0f + expf(-sg)) * su);
          p.a[(int64_t)row * p.F + f0 + f] = (uint16_t)bf16x2_rne(a, a);
        }
        lds_barrier();
      }
    }
  }
  // loads past the last item may still be writing LDS
  __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
}

// ---------------------------------------------------------------- down
constexpr int kGroupRows = 16 * kWaves;            // output rows of a workgroup
constexpr int kDownDepth = 2;                      // chunks of a wave in flight
constexpr int kDownSlot = 2 * 2048 + 256;          // two lines of 16 rows, their scale dwords
constexpr int kXSlots = 3;

// Units of work: (group of rows, entry, chunk of two lines, tile), the tile
// innermost so that an entry's later tiles find the chunk in the cache.  A
// group has `each` units.  Where the work is cut over the card, workgroup b of
// kCus takes the units [total b / kCus, total (b + 1) / kCus) of all groups',
// or unit b where there are fewer units: the shares of a group's workgroups
// follow each other and none of them is empty.
__device__ __forceinline__ int64_t share(int64_t total, int32_t b) {
  if (total < kCus) return b < total ? b : total;
  return total * b / kCus;
}

// The workgroup whose share holds unit g each + y (0 <= y < each, each > 0).
__device__ __forceinline__ int32_t owner(int32_t groups, int64_t each, int32_t g, int64_t y) {
  const int64_t total = groups * each, x = g * each + y;
  if (total < kCus) return (int32_t)x;
  int32_t b = (int32_t)((y ? kCus * (g + 1) - 1 : kCus * g) / groups);   // near it: g each / total = g / groups
  while (share(total, b + 1) <= x) ++b;
  while (share(total, b) > x) --b;
  return b;
}

template <bool kMx>
__global__ void __launch_bounds__(kThreads, 2) k_tokens_down(TokensProblem p) {
  constexpr int kOps = kMx ? 6 : 5, eb = kMx ? 1 : 2, kK = kLineK<kMx>, kP = kXp<kMx>;
  constexpr int kXRow = 2 * kK * 2;                // bytes of a token row of a chunk
  __shared__ int32_t expert[kEntries], first[kEntries + 1], tile[kEntries + 1];
  __shared__ __attribute__((aligned(4))) uint8_t token[kMaxRows];
  __shared__ __attribute__((aligned(16))) float sum[kWaves][kMaxTokens][16];
  __shared__ __attribute__((aligned(1024))) uint8_t ring[kWaves][kDownDepth][kDownSlot];
  __shared__ __attribute__((aligned(1024))) uint8_t xs[kXSlots][16 * kXRow];
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int r = lane & 15, h = lane >> 4;
  // the table up to the most entries and rows there can be: no load waits for
  // another (what lies past the entries is not used)
  const int pairs = p.T * p.k, most = (p.E < pairs ? p.E : pairs) + pairs / 16;
  const int V = __builtin_amdgcn_readfirstlane(p.table->entries);
  const int rows = __builtin_amdgcn_readfirstlane(p.table->rows);
  const int tiles = __builtin_amdgcn_readfirstlane(p.table->tiles);
  for (int u = tid; u <= most; u += kThreads) {
    if (u < kEntries) expert[u] = p.table->expert[u];
    first[u] = p.table->first[u];
    tile[u] = p.table->tile[u];
  }
  for (int i = 4 * tid; i < pairs; i += 4 * kThreads)
    *reinterpret_cast<uint32_t*>(token + i) = *reinterpret_cast<const uint32_t*>(p.table->token + i);
  for (int i = lane; i < 16 * p.T; i += 64) (&sum[wave][0][0])[i] = 0.0f;
  __syncthreads();
  const int32_t groups = (p.H + kGroupRows - 1) / kGroupRows;
  const int64_t row_bytes = (int64_t)p.F * eb;
  const int chunks = (int)((row_bytes + 255) / 256);
  const int64_t each = (int64_t)tiles * chunks;    // units of a group
  const int64_t total = groups * each;
  const int64_t u0 = p.part ? share(total, blockIdx.x) : blockIdx.x * each;
  const int64_t u1 = p.part ? share(total, blockIdx.x + 1) : u0 + each;

  // a group's sums to their place: lane's 4 rows of 16 for each token
  auto put = [&](int64_t g) {
    const int64_t n0 = g * kGroupRows + 16 * wave;
    if (n0 < p.H) {
      float* part = nullptr;
      if (p.part) part = p.part + ((int32_t)blockIdx.x - owner(groups, each, (int32_t)g, 0)) * p.T * (int64_t)p.H;
      for (int i = lane; i < 16 * p.T; i += 64) {
        const int t = i >> 4;
        const int64_t at = (int64_t)t * p.H + n0 + (i & 15);
        float v = (&sum[wave][0][0])[i];
        (&sum[wave][0][0])[i] = 0.0f;
        if (part) {
          part[at] = v;
        } else {
          if (p.residual) v += __uint_as_float((uint32_t)p.residual[at] << 16);
          p.out[at] = (uint16_t)bf16x2_rne(v, v);
        }
      }
    }
  };
  if (u0 >= u1) {
    // (without pieces a workgroup owns its group even if no expert is active)
    if (!p.part) put(blockIdx.x);
    return;
  }

  struct Unit {
    int64_t g;
    int32_t u, c, t, nt;   // entry, chunk, tile of nt
  };
  auto at = [&](int64_t x) {
    Unit q;
    q.g = x / each;
    const int64_t y = x - q.g * each;
    int a = 0, b = V;      // tile[a] * chunks <= y < tile[b] * chunks
    while (b - a > 1) {
      const int m = (a + b) >> 1;
      if ((int64_t)__builtin_amdgcn_readfirstlane(tile[m]) * chunks <= y) a = m; else b = m;
    }
    const int before = __builtin_amdgcn_readfirstlane(tile[a]);
    q.u = a;
    q.nt = __builtin_amdgcn_readfirstlane(tile[a + 1]) - before;
    const int in = (int)(y - (int64_t)before * chunks);
    q.c = in / q.nt;
    q.t = in - q.c * q.nt;
    return q;
  };
  auto next = [&](Unit& q) {
    if (++q.t < q.nt) return;
    q.t = 0;
    if (++q.c < chunks) return;
    q.c = 0;
    if (++q.u == V) {
      q.u = 0;
      ++q.g;
    }
    q.nt = __builtin_amdgcn_readfirstlane(tile[q.u + 1]) - __builtin_amdgcn_readfirstlane(tile[q.u]);
  };

  Unit ld = at(u0), cur = ld;
  const int count = (int)(u1 - u0);
  int issued = 0;
  const v4u ar = rsrc(p.a, (int64_t)rows * p.F * 2);
  v4u wq, sr;
  uint32_t n_off = 0, n_off_s = 0;   // the wave's first row, in weight and scale bytes
  bool rows_in = false;
  int lo = 0, hi = 0, open_u = -1;
  int64_t open_g = -1;
  auto open = [&]() {
    if (ld.u != open_u) {
      const int64_t e = __builtin_amdgcn_readfirstlane(expert[ld.u]);
      lo = __builtin_amdgcn_readfirstlane(first[ld.u]);
      hi = __builtin_amdgcn_readfirstlane(first[ld.u + 1]);
      wq = rsrc(p.w2 + e * p.H * row_bytes, p.H * row_bytes);
      if constexpr (kMx) sr = scale_rsrc(p.w2_s, e, p.E, p.H, p.F);
      open_u = ld.u;
    }
    if (ld.g != open_g) {
      const int64_t n0 = ld.g * kGroupRows + 16 * wave;
      rows_in = n0 < p.H;
      n_off = rows_in ? (uint32_t)n0 * (uint32_t)row_bytes : 0u;
      n_off_s = rows_in ? 4u * (uint32_t)n0 : 0u;
      open_g = ld.g;
    }
  };
  uint32_t lane_off[2];
  int32_t lane_c[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int row = 8 * q + (lane >> 3);
    lane_c[q] = 16 * ((lane & 7) ^ chunk_swizzle(row));
    lane_off[q] = (uint32_t)row * (uint32_t)row_bytes + (uint32_t)lane_c[q];
  }
  const uint32_t panel = 4u * (uint32_t)p.E * (uint32_t)p.H;
  const uint32_t lane_s = (uint32_t)((lane >> 4) & 1) * panel + 4u * (uint32_t)r;
  constexpr int kChunks = kXRow / 16;              // 16-byte chunks of a token row
  const int xl = 2 * wave + lane / kChunks;        // the lane's token row of a tile, its chunk
  const int xc = 8 * ((lane % kChunks) ^ (xl & 15));
  auto load = [&]() {
    const bool on = issued < count;
    const bool in = on && rows_in;
    const uint32_t dst = lds_addr(ring[wave][0]) + (uint32_t)(issued % kDownDepth) * kDownSlot;
    const int32_t left = in ? (int32_t)(row_bytes - 256 * (int64_t)ld.c) : 0;   // bytes of the rows from here on
    const uint32_t soff = uniform(in ? n_off + 256u * (uint32_t)ld.c : 0u);
#pragma unroll
    for (int q = 0; q < 4; ++q)   // (a second line past the rows' end has no lane in range)
      dma16_nt(wq, dst + 1024u * q, lane_c[q & 1] + 128 * (q >> 1) < left ? lane_off[q & 1] + 128u * (q >> 1) : kOob, soff);
    if constexpr (kMx) {   // lanes 0..15: the first line's scale dwords, 16..31 the second's
      const bool ok = lane < 32 && 128 * ((lane >> 4) & 1) < left;
      dma4(sr, dst + 4096u, ok ? lane_s : kOob, uniform(in ? 2u * (uint32_t)ld.c * panel + n_off_s : 0u));
    }
    // this wave's two token rows of the chunk
    const uint32_t xd = lds_addr(xs[0]) + (uint32_t)(issued % kXSlots) * (16 * kXRow) + (uint32_t)wave * (2 * kXRow);
    if (lane < 2 * kChunks) {
      const int row = lo + 16 * ld.t + xl, k = ld.c * 2 * kK + xc;
      dma16(ar, xd, on && row < hi && k < p.F ? 2u * ((uint32_t)row * (uint32_t)p.F + (uint32_t)k) : kOob, 0);
    }
    if (++issued < count) {
      next(ld);
      open();
    }
  };

  open();
#pragma unroll
  for (int d = 0; d < kDownDepth; ++d) load();
  for (int seq = 0; seq < count; ++seq) {
    // this unit's loads are done, the next one's may be in flight; after the
    // barrier every wave's token rows are there, and every wave has read the
    // token slot that the loads below overwrite (two units ago)
    fence();
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(kOps * (kDownDepth - 1)));
    lds_barrier();
    const uint8_t* slot = ring[wave][seq % kDownDepth];
    const uint8_t* xt = xs[seq % kXSlots] + r * kXRow;
    Fragment f[2];
    v8bf xv[2][kP];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      f[i] = read_fragment<kMx>(slot + 2048 * i, slot + 4096 + 64 * i);
#pragma unroll
      for (int j = 0; j < kP; ++j)
        xv[i][j] = *reinterpret_cast<const v8bf*>(xt + 16 * ((4 * kP * i + kP * h + j) ^ r));
    }
    fence();
    __builtin_amdgcn_s_waitcnt(kWaitLgkm0);        // read: the ring's slot is free
    fence();
    load();
    v4f y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float s = fragment_scale<kMx>(f[i]);
#pragma unroll
      for (int j = 0; j < kP; ++j)
        y = __builtin_amdgcn_mfma_f32_16x16x32_bf16(weights8<kMx>(f[i], j, s), xv[i][j], y, 0, 0, 0);
    }
    const int row = __builtin_amdgcn_readfirstlane(first[cur.u]) + 16 * cur.t + r;
    if (row < __builtin_amdgcn_readfirstlane(first[cur.u + 1])) {   // the lane owns 4 sums of its token
      float4* d = reinterpret_cast<float4*>(sum[wave][token[row]] + 4 * h);
      float4 v = *d;
      v.x += y[0];
      v.y += y[1];
      v.z += y[2];
      v.w += y[3];
      *d = v;
    }
    const int64_t g = cur.g;
    next(cur);
    if (cur.g != g || seq + 1 == count) put(g);
  }
  // loads past the last unit may still be writing LDS
  __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
}

// The pieces of a group in the workgroups' order, the residual, the rounding.
__global__ void __launch_bounds__(256) k_tokens_join(TokensProblem p, int32_t chunks) {
  const int32_t i = 2 * (blockIdx.x * 256 + threadIdx.x);   // two columns of a token (T H < 2^30)
  const int32_t all = p.T * p.H;
  if (i >= all) return;
  const int32_t groups = (p.H + kGroupRows - 1) / kGroupRows;
  const int64_t each = (int64_t)p.table->tiles * chunks;
  float a = 0.0f, b = 0.0f;
  if (p.residual) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(p.residual + i);
    a = __uint_as_float(w << 16);
    b = __uint_as_float(w & 0xFFFF0000u);
  }
  if (each > 0) {
    const int32_t g = i % p.H / kGroupRows;
    const int32_t n = owner(groups, each, g, each - 1) - owner(groups, each, g, 0) + 1;
#pragma unroll 4
    for (int32_t s = 0; s < n; ++s) {
      const float2 v = *reinterpret_cast<const float2*>(p.part + (int64_t)s * all + i);
      a += v.x;
      b += v.y;
    }
  }
  *reinterpret_cast<uint32_t*>(p.out + i) = bf16x2_rne(a, b);
}

// Pieces of one group at most, times its columns over the card: where the
// groups are at most kCus, (kCus / groups + 2) * 128 groups.
constexpr int64_t kPartCols = 128 * 3 * (int64_t)kCus;

// Whether the groups' work is cut over the card: not where they fill it, nor
// where a group has at most six units (a unit takes its workgroup 0.8 us, the
// join and the reading of more pieces 5 us).
bool cut(const TokensProblem& p, bool mxw) {
  const int64_t groups = (p.H + kGroupRows - 1) / kGroupRows;
  const int64_t pairs = (int64_t)p.T * p.k;
  const int64_t units = (p.E < pairs ? p.E : pairs) * (((int64_t)p.F * (mxw ? 1 : 2) + 255) / 256);
  return groups < kCus && units > 6;
}

template <bool kMx>
int launch_tokens(TokensProblem p, hipStream_t st) {
  const int64_t pairs = (int64_t)p.T * p.k;
  const int64_t most = ((p.E < pairs ? p.E : pairs) + pairs / 16) * (p.F / 16);
  const dim3 up((unsigned)(most + 1 < kCus ? most + 1 : kCus));   // items at most, and the table's writer
  // steps of 8 waves x 128 bytes; registers hold 8 (fp8) or 16 (bf16) of one tile
  constexpr int kLong = kMx ? 8 : 16;
  if (p.H > 4096) hipLaunchKernelGGL((k_tokens_up<kMx, kLong, 1>), up, dim3(kThreads), 0, st, p);
  else if (p.H > 2048) hipLaunchKernelGGL((k_tokens_up<kMx, kLong / 2, 2>), up, dim3(kThreads), 0, st, p);
  else hipLaunchKernelGGL((k_tokens_up<kMx, kLong / 4, 4>), up, dim3(kThreads), 0, st, p);
  const int64_t groups = (p.H + kGroupRows - 1) / kGroupRows;
  if (cut(p, kMx)) {
    hipLaunchKernelGGL(k_tokens_down<kMx>, dim3(kCus), dim3(kThreads), 0, st, p);
    const int64_t n = (int64_t)p.T * p.H / 2;
    hipLaunchKernelGGL(k_tokens_join, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st, p,
                       (int32_t)(((int64_t)p.F * (kMx ? 1 : 2) + 255) / 256));
  } else {
    p.part = nullptr;
    hipLaunchKernelGGL(k_tokens_down<kMx>, dim3((unsigned)groups), dim3(kThreads), 0, st, p);
  }
  return launch_status();
}

int64_t tokens_bytes(int64_t tokens, int64_t topk, int64_t F) {
  return kTableBytes + 4 * tokens * kPartCols + ((tokens * topk * F * 2 + 255) & ~(int64_t)255);
}

int tokens_call(bool mxw, const uint16_t* x, const float* logits, int64_t tokens, int32_t topk, int32_t E, int64_t H,
                int64_t F, const void* w1, const uint8_t* w1_s, const void* w2, const uint8_t* w2_s,
                const uint16_t* residual, uint16_t* out, void* ws, size_t ws_bytes, mx_stream_t stream) {
  if (tokens < 0 || topk < 1 || E < 1 || topk > E || H <= 0 || F <= 0 || H % 32 || F % 32) return MX_EINVAL;
  if (!x || !logits || !w1 || !w2 || !out || !ws || (mxw && (!w1_s || !w2_s))) return MX_EINVAL;
  if (((uintptr_t)x | (uintptr_t)w1 | (uintptr_t)w2 | (uintptr_t)ws) & 15) return MX_EINVAL;
  if (((uintptr_t)logits | (uintptr_t)w1_s | (uintptr_t)w2_s) & 3) return MX_EINVAL;
  if (((uintptr_t)out | (uintptr_t)residual) & 3) return MX_EINVAL;
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
  p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kTableBytes);
  p.a = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(ws) + kTableBytes + 4 * tokens * kPartCols);
  const hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  return mxw ? launch_tokens<true>(p, st) : launch_tokens<false>(p, st);
}

}  // namespace
}  // namespace mx

using namespace mx;

extern "C" size_t mx_moe_tokens_workspace_size(int64_t tokens, int32_t topk, int32_t num_experts, int64_t F) {
  if (tokens < 0 || topk < 1 || topk > num_experts || F <= 0 || F % 32) return 0;
  if (tokens > kMaxTokens || num_experts > kTokExperts || topk > kTokTopk || F >= (1ll << 24)) return 0;
  if (tokens * topk * F * 2 >= (1ll << 31)) return 0;
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

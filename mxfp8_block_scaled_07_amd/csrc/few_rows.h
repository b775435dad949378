// The few-row form of the bf16 product (gfx950): x w^T for at most 16 rows of x,
// the weights streamed once through the rings of stream.h.
#pragma once

#include "stream.h"

namespace mx {
namespace {

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

// fin, a class F: what becomes of the sums, eight consecutive columns j .. of row
// m in one thread (thread 32 item + 2 m + half).
//   struct Ahead, State;
//   Ahead fetch(bool in, m, j, N) const      loads ahead of the sums
//   void finish(State&, const Ahead&, float (&v)[8], m, j, N) const
//   void end(State&, float* lds, m, item, M) const     by every thread; lds: kSkItems kSkWaves 256 floats
template <class F>
__global__ void __launch_bounds__(64 * kSkWaves, 2) k_skinny(const uint16_t* __restrict__ x,
                                                             const uint16_t* __restrict__ w, int64_t M, int64_t N,
                                                             int64_t K, F fin) {
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
  // columns of one row.
  const int ti = tid >> 5, m = (tid & 31) >> 1, c0 = 8 * (tid & 1);
  auto tail = [&](int item0) {
    const int64_t j = 16 * (int64_t)(item0 + ti) + c0;
    return fin.fetch(ti < kSkItems && m < M && item0 + ti < end && j < N, m, j, N);
  };

  // x lies between the first chunks, and is waited for here: else the compiler
  // waits at each use, and for the stream's loads too
#pragma unroll 1
  for (int d = 0; d < kSkDepth - 1; ++d) load();
  typename F::Ahead t = tail(begin);
  typename F::State state;
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
      }
      fin.finish(state, t, v, m, j, N);
    }
    if (item + 1 < end) {
      t = tail(item + 1);
      lds_barrier();
    }
  }
  // loads past the last item may still be writing LDS
  __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
  fin.end(state, reinterpret_cast<float*>(red), m, ti, M);
}

// Workgroups of k_skinny for n rows of w.
inline unsigned skinny_grid(int64_t n) {
  const int64_t items = (n + 15) / 16;
  return (unsigned)(items < kCus ? items : kCus);
}

}  // namespace
}  // namespace mx

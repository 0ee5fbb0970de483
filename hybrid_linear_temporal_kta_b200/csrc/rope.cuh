// rope.cuh -- rotary positions of query / key heads: part of each head (dims [begin, begin + rot))
// is cut into one section per position axis, and pair i of a section turns by t = pos * freq_i:
//     (a, b) -> m (a cos t - b sin t, a sin t + b cos t),
// b the dim next to a (interleaved) or half a section behind it (half). The gradient is the same
// map with -t (sgn = -1).
//
// Memory-bound: every element is read and written once, 2 x 2 bytes in bf16. A block takes tt tokens,
// forms their cosines and sines once in shared memory (angles as 64-bit turns reduced to [-1/2, 1/2],
// so a position of 2^31 still has an angle good to 2^-21), and each thread keeps those of its (token,
// item) in registers while it walks the heads of both tensors. q and k of 32,760 tokens x 16 heads x
// 128 dims (537 MB moved) take 93 us interleaved, 107 us half; a copy of as many bytes 85 us.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "mixer_common.cuh"

namespace kta {

constexpr int ROPE_THREADS = 256;
constexpr int ROPE_MAX_AXES = 4;
constexpr int ROPE_MAX_PAIRS = 64;   // d <= 128
constexpr int ROPE_MAX_ITEMS = 128;
// Heads loaded before the first is stored: one keeps the half layout (two pieces a head) in 64 registers
// and four blocks on an SM (two: 113 against 107 us on the shape below).
constexpr int ROPE_UNROLL_HALF = 1, ROPE_UNROLL_PAIR = 4;

struct RopeParams {
  const void* x[2];
  void* o[2];
  long long ld[2];        // elements from one token to the next
  int H[2];
  int copy[2];            // write the dims that do not turn (0 when o is x)
  long long rows;         // B * N
  int N, d, begin, rot, n_axes, n_items;
  int tt, lanes, head_step;      // tokens per block, threads that share a (token, item)'s heads, heads per block
  int pair_end[ROPE_MAX_AXES];   // pairs of axes 0..a
  const long long* pos;   // [B or 1][N][n_axes], or null (first axis = token of the sequence)
  long long pos_seq;      // elements from one sequence's positions to the next (0: shared)
  long long pos0;         // added to the first axis
  const double* freqs;    // radians per position, one per pair
  float mscale, sgn;
};

// One item = V dims of a head and, in the half layout, their partners half a section behind.
struct RopeItem {
  short lo, hi;    // element offsets in the head; hi < 0: no partner chunk
  short pair;      // first pair (interleaved: may begin before or run past the turned part)
  short turns;     // 0: copied
};

template <typename T, int V, bool HALF>
__global__ __launch_bounds__(ROPE_THREADS, 4) void rope_kernel(const RopeParams p) {
  constexpr int UNROLL = HALF ? ROPE_UNROLL_HALF : ROPE_UNROLL_PAIR;
  extern __shared__ float2 rope_cs[];              // [tt][pairs]
  __shared__ RopeItem items[ROPE_MAX_ITEMS];
  __shared__ long long s_pos[ROPE_THREADS][ROPE_MAX_AXES];
  const int tid = threadIdx.x, pairs = p.rot / 2;
  const unsigned r0 = blockIdx.x * static_cast<unsigned>(p.tt);
  const int nt = min(static_cast<unsigned>(p.tt), static_cast<unsigned>(p.rows) - r0);
  for (int tl = tid; tl < nt; tl += ROPE_THREADS) {
    const unsigned r = r0 + tl, b = r / static_cast<unsigned>(p.N), n = r - b * static_cast<unsigned>(p.N);
    const long long* src = p.pos + b * p.pos_seq + static_cast<long long>(n) * p.n_axes;
    for (int a = 0; a < p.n_axes; ++a) s_pos[tl][a] = (p.pos ? src[a] : n) + (a == 0 ? p.pos0 : 0);
  }
  if (tid < p.n_items) {
    RopeItem it;
    if (HALF) {
      const int nrot = pairs / V;
      if (tid < nrot) {
        const int pr = tid * V;
        int a = 0;
        while (a < p.n_axes - 1 && pr >= p.pair_end[a]) ++a;
        const int first = a ? p.pair_end[a - 1] : 0, half = p.pair_end[a] - first;
        it.lo = static_cast<short>(p.begin + 2 * first + (pr - first));
        it.hi = static_cast<short>(it.lo + half);
        it.pair = static_cast<short>(pr);
        it.turns = 1;
      } else {
        const int c = (tid - nrot) * V;
        it.lo = static_cast<short>(c < p.begin ? c : c + p.rot);
        it.hi = -1;
        it.pair = 0;
        it.turns = 0;
      }
    } else {
      it.lo = static_cast<short>(tid * V);
      it.hi = -1;
      it.pair = static_cast<short>((it.lo - p.begin) / 2);   // begin is even: exact
      it.turns = static_cast<short>(it.lo + V > p.begin && it.lo < p.begin + p.rot);
    }
    items[tid] = it;
  }
  __syncthreads();
  // a thread's pair is the same for all its tokens
  const int pr = tid % ROPE_MAX_PAIRS;
  if (pr < pairs) {
    int a = 0;
    while (a < p.n_axes - 1 && pr >= p.pair_end[a]) ++a;
    const double f = p.freqs[pr] * 0.15915494309189533577;   // turns of the circle per position
    for (int tl = tid / ROPE_MAX_PAIRS; tl < nt; tl += ROPE_THREADS / ROPE_MAX_PAIRS) {
      const double t = static_cast<double>(s_pos[tl][a]) * f;
      const float frac = static_cast<float>(t - rint(t));    // whole turns come off in 64 bits
      float s, c;
      sincospif(2.f * frac, &s, &c);
      rope_cs[tl * pairs + pr] = make_float2(c * p.mscale, s * p.mscale * p.sgn);
    }
  }
  __syncthreads();

  const int h0 = blockIdx.y * p.head_step, h1 = min(h0 + p.head_step, p.H[0] + p.H[1]);
  for (int slot = tid; slot < nt * p.lanes * p.n_items; slot += ROPE_THREADS) {
    const int row = slot / p.n_items, tl = row / p.lanes, hl = row - tl * p.lanes;
    const RopeItem it = items[slot - row * p.n_items];
    const long long r = r0 + tl;
    constexpr int NP = HALF ? V : V / 2;
    float2 cs[NP > 0 ? NP : 1];
    unsigned turned = 0;                    // interleaved: which pairs of the chunk turn
    if (it.turns) {
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        const int q = it.pair + j;
        const bool in = q >= 0 && q < pairs;
        cs[j] = in ? rope_cs[tl * pairs + q] : make_float2(1.f, 0.f);
        turned |= unsigned(in) << j;
      }
    }
#pragma unroll 1
    for (int w = 0; w < 2; ++w) {           // the heads of x, then of x2
      const int e0 = (w ? max(h0 - p.H[0], 0) : h0) + hl, e1 = w ? h1 - p.H[0] : min(h1, p.H[0]);
      if (!it.turns && !p.copy[w]) continue;
      const int hd = p.lanes * p.d;         // from one of the thread's heads to the next
      const T* src = static_cast<const T*>(p.x[w]) + r * p.ld[w] + static_cast<long long>(e0) * p.d + it.lo;
      T* dst = static_cast<T*>(p.o[w]) + r * p.ld[w] + static_cast<long long>(e0) * p.d + it.lo;
      const int step = it.hi - it.lo;
      for (int h = e0; h < e1; h += UNROLL * p.lanes) {
        VecPack<T, V> lo[UNROLL], hi[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u)
          if (h + u * p.lanes < e1) {
            lo[u].load(src + u * hd);
            if (HALF && it.turns) hi[u].load(src + u * hd + step);
          }
#pragma unroll
        for (int u = 0; u < UNROLL; ++u)
          if (h + u * p.lanes < e1) {
            if (it.turns) {
              if (HALF) {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                  const float x = to_f32(lo[u].e[j]), y = to_f32(hi[u].e[j]);
                  lo[u].e[j] = from_f32<T>(x * cs[j % NP].x - y * cs[j % NP].y);
                  hi[u].e[j] = from_f32<T>(x * cs[j % NP].y + y * cs[j % NP].x);
                }
                hi[u].store(dst + u * hd + step);
              } else {
#pragma unroll
                for (int j = 0; j < V / 2; ++j)
                  if (turned >> j & 1) {    // a pair outside the part keeps its bits
                    const float x = to_f32(lo[u].e[2 * j]), y = to_f32(lo[u].e[2 * j + 1]);
                    lo[u].e[2 * j] = from_f32<T>(x * cs[j].x - y * cs[j].y);
                    lo[u].e[2 * j + 1] = from_f32<T>(x * cs[j].y + y * cs[j].x);
                  }
              }
            }
            lo[u].store(dst + u * hd);
          }
        src += UNROLL * hd;
        dst += UNROLL * hd;
      }
    }
  }
}

}  // namespace kta

// rope.cuh -- rotary positions of query / key heads: part of each head (dims [begin, begin + rot))
// is cut into one section per position axis, and pair i of a section turns by t = pos * freq_i:
//     (a, b) -> m (a cos t - b sin t, a sin t + b cos t),
// b the dim next to a (interleaved) or half a section behind it (half). The gradient is the same
// map with -t (sgn = -1).
//
// Memory-bound: every element is read and written once, 2 x 2 bytes in bf16. A block takes TT
// tokens, forms their cosines and sines once in shared memory (angles as 64-bit turns reduced to
// [-1/2, 1/2], so a position of 2^31 still has an angle good to 2^-21), and each thread keeps those
// of its (token, item) in registers while it walks the heads of both tensors.
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
constexpr int ROPE_UNROLL = 4;       // heads loaded before the first is stored

struct RopeParams {
  const void* x[2];
  void* o[2];
  long long ld[2];        // elements from one token to the next
  int H[2];
  int copy[2];            // write the dims that do not turn (0 when o is x)
  long long rows;         // B * N
  int N, d, begin, rot, n_axes, n_items, tt, head_step;
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
__global__ __launch_bounds__(ROPE_THREADS) void rope_kernel(const RopeParams p) {
  extern __shared__ float2 rope_cs[];              // [tt][pairs]
  __shared__ RopeItem items[ROPE_MAX_ITEMS];
  const int tid = threadIdx.x, pairs = p.rot / 2;
  const long long r0 = static_cast<long long>(blockIdx.x) * p.tt;
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
  for (int i = tid; i < p.tt * pairs; i += ROPE_THREADS) {
    const int tl = i / pairs, pr = i - tl * pairs;
    const long long r = r0 + tl;
    if (r < p.rows) {
      int a = 0;
      while (a < p.n_axes - 1 && pr >= p.pair_end[a]) ++a;
      const long long b = r / p.N, n = r - b * p.N;
      long long pos = p.pos ? p.pos[b * p.pos_seq + n * p.n_axes + a] : n;
      if (a == 0) pos += p.pos0;
      // turns of the circle, the whole ones taken off in 64 bits
      const double t = static_cast<double>(pos) * (p.freqs[pr] * 0.15915494309189533577);
      const float f = static_cast<float>(t - rint(t));
      float s, c;
      sincospif(2.f * f, &s, &c);
      rope_cs[i] = make_float2(c * p.mscale, s * p.mscale * p.sgn);
    }
  }
  __syncthreads();

  const int Hall = p.H[0] + p.H[1];
  const int h0 = blockIdx.y * p.head_step, h1 = min(h0 + p.head_step, Hall);
  for (int slot = tid; slot < p.tt * p.n_items; slot += ROPE_THREADS) {
    const int tl = slot / p.n_items;
    const RopeItem it = items[slot - tl * p.n_items];
    const long long r = r0 + tl;
    if (r >= p.rows) break;
    constexpr int NP = HALF ? V : V / 2;
    float2 cs[NP > 0 ? NP : 1];
    unsigned turned = 0;                    // interleaved: which pairs of the chunk turn
    if (it.turns) {
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        const int pr = it.pair + j;
        const bool in = pr >= 0 && pr < pairs;
        cs[j] = in ? rope_cs[tl * pairs + pr] : make_float2(1.f, 0.f);
        turned |= unsigned(in) << j;
      }
    }
    for (int hb = h0; hb < h1; hb += ROPE_UNROLL) {
      VecPack<T, V> lo[ROPE_UNROLL], hi[ROPE_UNROLL];
#pragma unroll
      for (int u = 0; u < ROPE_UNROLL; ++u) {
        const int h = hb + u;
        if (h < h1) {
          const int w = h >= p.H[0];
          const T* src = static_cast<const T*>(p.x[w]) + r * p.ld[w] +
                         static_cast<long long>(w ? h - p.H[0] : h) * p.d;
          if (it.turns || p.copy[w]) {
            lo[u].raw = *reinterpret_cast<const decltype(lo[u].raw)*>(src + it.lo);
            if (HALF && it.turns) hi[u].raw = *reinterpret_cast<const decltype(hi[u].raw)*>(src + it.hi);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < ROPE_UNROLL; ++u) {
        const int h = hb + u;
        if (h < h1) {
          const int w = h >= p.H[0];
          T* dst = static_cast<T*>(p.o[w]) + r * p.ld[w] +
                   static_cast<long long>(w ? h - p.H[0] : h) * p.d;
          if (it.turns) {
            if (HALF) {
#pragma unroll
              for (int j = 0; j < V; ++j) {
                const float a = to_f32(lo[u].e[j]), b = to_f32(hi[u].e[j]);
                lo[u].e[j] = from_f32<T>(a * cs[j % NP].x - b * cs[j % NP].y);
                hi[u].e[j] = from_f32<T>(a * cs[j % NP].y + b * cs[j % NP].x);
              }
              *reinterpret_cast<decltype(hi[u].raw)*>(dst + it.hi) = hi[u].raw;
            } else {
#pragma unroll
              for (int j = 0; j < V / 2; ++j) {
                if (turned >> j & 1) {   // a pair outside the part keeps its bits
                  const float a = to_f32(lo[u].e[2 * j]), b = to_f32(lo[u].e[2 * j + 1]);
                  lo[u].e[2 * j] = from_f32<T>(a * cs[j].x - b * cs[j].y);
                  lo[u].e[2 * j + 1] = from_f32<T>(a * cs[j].y + b * cs[j].x);
                }
              }
            }
            *reinterpret_cast<decltype(lo[u].raw)*>(dst + it.lo) = lo[u].raw;
          } else if (p.copy[w]) {
            *reinterpret_cast<decltype(lo[u].raw)*>(dst + it.lo) = lo[u].raw;
          }
        }
      }
    }
  }
}

}  // namespace kta

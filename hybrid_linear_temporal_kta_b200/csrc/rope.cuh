// rope.cuh -- rotary positions of query / key heads: part of each head (dims [begin, begin + rot))
// is cut into one section per position axis, and pair i of a section turns by t = pos * freq_i:
//     (a, b) -> m (a cos t - b sin t, a sin t + b cos t),
// b the dim next to a (interleaved) or half a section behind it (half). The gradient is the same
// map with -t (sgn = -1).
//
// Memory-bound: every element is read and written once, 2 x 2 bytes in bf16. A block takes tt tokens and
// forms their cosines and sines once in shared memory (angles as 64-bit turns reduced to [-1/2, 1/2],
// so a position of 2^31 still has an angle good to 2^-21). A thread owns one 16-byte piece of the head: it
// keeps the piece's cosines and sines in registers and walks the heads of both tensors. Interleaved
// partners lie in the piece; in the half layout a warp puts its rows into shared memory as well and
// every thread fetches its partners there, so any section size moves 16-byte pieces.
// q and k of 32,760 tokens x 16 heads x 128 dims (537 MB moved): interleaved 87 us, half 94 us (102 with
// sections of any even size); a copy of as many bytes takes 85 us.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "mixer_common.cuh"

namespace kta {

constexpr int ROPE_THREADS = 256;
constexpr int ROPE_MAX_AXES = 4;
constexpr int ROPE_MAX_PAIRS = 64;   // d <= 128
constexpr int ROPE_UNROLL = 4;       // heads loaded before the first is stored (64 registers, four blocks on an SM)

struct RopeParams {
  const void* x[2];
  void* o[2];
  long long ld[2];        // elements from one token to the next
  int H[2];
  int copy[2];            // write the dims that do not turn (0 when o is x)
  long long rows;         // B * N
  int N, d, begin, rot, n_axes, n_items;   // n_items: 16-byte pieces of a head
  int tt, lanes, head_step;      // tokens per block, threads that share a (token, item)'s heads, heads per block
  int pair_end[ROPE_MAX_AXES];   // pairs of axes 0..a
  const long long* pos;   // [B or 1][N][n_axes], or null (first axis = token of the sequence)
  long long pos_seq;      // elements from one sequence's positions to the next (0: shared)
  long long pos0;         // added to the first axis
  const double* freqs;    // radians per position, one per pair
  float mscale, sgn;
};

template <typename T, int V> union RopePartners {   // V elements fetched W at a time
  T e[V];
  uint4 q;
  uint2 d[V * sizeof(T) / 8];
  uint32_t w[V * sizeof(T) / 4];
  uint16_t h[V * sizeof(T) / 2];
  __device__ __forceinline__ RopePartners() {}
};

// HALF: W = elements of partners that lie together and aligned (the largest power of two, up to a piece,
// that divides begin and every half section). Interleaved: W = 0.
template <typename T, int W>
__global__ __launch_bounds__(ROPE_THREADS, 4) void rope_kernel(const RopeParams p) {
  constexpr bool HALF = W > 0;
  constexpr int V = 16 / int(sizeof(T)), NP = HALF ? V : V / 2, PW = HALF ? W : 1;
  extern __shared__ float2 rope_cs[];              // [tt][pairs]
  __shared__ long long s_pos[ROPE_THREADS][ROPE_MAX_AXES];
  __shared__ uint4 rows[HALF ? ROPE_UNROLL : 1][HALF ? ROPE_THREADS : 1];
  const int tid = threadIdx.x, pairs = p.rot / 2;
  const unsigned r0 = blockIdx.x * static_cast<unsigned>(p.tt);
  const int nt = min(static_cast<unsigned>(p.tt), static_cast<unsigned>(p.rows) - r0);
  for (int tl = tid; tl < nt; tl += ROPE_THREADS) {
    const unsigned r = r0 + tl, b = r / static_cast<unsigned>(p.N), n = r - b * static_cast<unsigned>(p.N);
    const long long* src = p.pos + b * p.pos_seq + static_cast<long long>(n) * p.n_axes;
    for (int a = 0; a < p.n_axes; ++a) s_pos[tl][a] = (p.pos ? src[a] : n) + (a == 0 ? p.pos0 : 0);
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

  // thread = (token, head lane, piece); n_items divides 32, so a warp holds whole heads
  const int row = tid / p.n_items, tl = row / p.lanes, hl = row - tl * p.lanes, e0 = (tid - row * p.n_items) * V;
  const bool on = tl < nt;
  const long long r = r0 + (on ? tl : 0);
  float2 cs[NP];                            // HALF: (cos, +-sin) of each element; else of each pair
  short part[HALF ? V / PW : 1];            // where partners begin, in elements from the head's first
  unsigned turned = 0;                      // elements (interleaved: pairs) that turn
#pragma unroll
  for (int g = 0; g < NP / PW; ++g) {       // HALF: PW elements of one half of one section, or of no section
    const int at = (HALF ? e0 + g * PW : e0 + 2 * g) - p.begin;   // in the turned part
    const bool in = on && at >= 0 && at < p.rot;
    int pair = at / 2, move = 0;            // (interleaved pairs are numbered through)
    bool hi = true;
    if (HALF && in) {
      int a = 0;
      while (a < p.n_axes - 1 && at >= 2 * p.pair_end[a]) ++a;
      const int first = a ? p.pair_end[a - 1] : 0, half = p.pair_end[a] - first, o = at - 2 * first;
      hi = o >= half;
      pair = first + (hi ? o - half : o);
      move = hi ? -half : half;
    }
    if (HALF) part[g] = static_cast<short>(e0 + g * PW + move);
    if (in) turned |= ((1u << PW) - 1) << (g * PW);
#pragma unroll
    for (int j = 0; j < PW; ++j) {
      float2 v = in ? rope_cs[tl * pairs + pair + j] : make_float2(1.f, 0.f);
      if (!hi) v.y = -v.y;
      cs[g * PW + j] = v;
    }
  }
  const int h0 = blockIdx.y * p.head_step, h1 = min(h0 + p.head_step, p.H[0] + p.H[1]);
#pragma unroll 1
  for (int w = 0; w < 2; ++w) {             // the heads of x, then of x2
    const int b0 = w ? max(h0 - p.H[0], 0) : h0, b1 = w ? h1 - p.H[0] : min(h1, p.H[0]);
    if (b0 >= b1) continue;
    // heads of this thread (none if its piece neither turns nor is copied: it is no one's partner then)
    // and of the warp's first head lane
    const int most = (b1 - b0 + p.lanes - 1) / p.lanes;
    const int mine = on && (turned || p.copy[w]) ? (b1 - b0 - hl + p.lanes - 1) / p.lanes : 0;
    if (!HALF && !mine) continue;
    const int hd = p.lanes * p.d;           // from one of the thread's heads to the next
    const T* src = static_cast<const T*>(p.x[w]) + r * p.ld[w] + static_cast<long long>(b0 + hl) * p.d + e0;
    T* dst = static_cast<T*>(p.o[w]) + r * p.ld[w] + static_cast<long long>(b0 + hl) * p.d + e0;
    for (int i = 0; i < (HALF ? most : mine); i += ROPE_UNROLL) {
      VecPack<T, V> x[ROPE_UNROLL];
#pragma unroll
      for (int u = 0; u < ROPE_UNROLL; ++u)
        if (i + u < mine) x[u].load(src + u * hd);
      if (HALF) {
        __syncwarp();                       // the partners of the heads before have been read
#pragma unroll
        for (int u = 0; u < ROPE_UNROLL; ++u) rows[u][tid] = x[u].raw;
        __syncwarp();
      }
#pragma unroll
      for (int u = 0; u < ROPE_UNROLL; ++u) {
        if (i + u < mine) {
          if (HALF) {
            const T* head = reinterpret_cast<const T*>(&rows[u][tid - e0 / V]);
            RopePartners<T, V> q;
            constexpr int WB = PW * int(sizeof(T));
#pragma unroll
            for (int j = 0; j < V / PW; ++j) {
              if constexpr (WB == 16)
                q.q = *reinterpret_cast<const uint4*>(head + part[j]);
              else if constexpr (WB == 8)
                q.d[j] = *reinterpret_cast<const uint2*>(head + part[j]);
              else if constexpr (WB == 4)
                q.w[j] = *reinterpret_cast<const uint32_t*>(head + part[j]);
              else
                q.h[j] = *reinterpret_cast<const uint16_t*>(head + part[j]);
            }
#pragma unroll
            for (int j = 0; j < V; ++j)
              if (turned >> j & 1)
                x[u].e[j] = from_f32<T>(fmaf(to_f32(q.e[j]), cs[j % NP].y, to_f32(x[u].e[j]) * cs[j % NP].x));
          } else {
#pragma unroll
            for (int j = 0; j < V / 2; ++j)
              if (turned >> j & 1) {        // a pair outside the part keeps its bits
                const float a = to_f32(x[u].e[2 * j]), b = to_f32(x[u].e[2 * j + 1]);
                x[u].e[2 * j] = from_f32<T>(a * cs[j].x - b * cs[j].y);
                x[u].e[2 * j + 1] = from_f32<T>(a * cs[j].y + b * cs[j].x);
              }
          }
          x[u].store(dst + u * hd);
        }
      }
      src += ROPE_UNROLL * hd;
      dst += ROPE_UNROLL * hd;
    }
  }
}

}  // namespace kta

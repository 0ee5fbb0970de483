// short_conv.cuh -- short causal convolution along the tokens, one filter of K taps per channel:
//     pre_t = bias + sum_j w_j x_{t-K+1+j},   y_t = act(pre_t),   act = silu or identity,
// rows before the sequence's first come from a carried state S0 (K - 1 rows) or are zero; the end
// state is the last K - 1 rows of [S0; x]. Backward, with dp_t = dy_t act'(pre_t):
//     dx_t = sum_j w_j dp_{t+K-1-j},   dw_j = sum_t dp_t x_{t-K+1+j},   dbias = sum_t dp_t.
//
// A thread owns 4 channels and walks a run of tokens with the last K - 1 rows in registers, so every row
// is read once per run plus the K - 1 rows before it, which its neighbour has brought into L2. Weights and
// sums are fp32. Forward: memory-bound, 2 x 65,536 x 2,048 bf16 (1.07 GB moved) in 192 us, a copy of as
// many bytes 171 us; 8 channels to a thread need twice the registers: 260 us. Backward: 2 x 8,191 x 2,048 bf16
// (201 MB) in 64 us, where the bytes alone take 31 and the issue of its 36 instructions per element 33: the two
// follow each other instead of overlapping.
#pragma once
#include "mixer_common.cuh"

namespace kta {

constexpr int SC_THREADS = 128;
constexpr int SC_V = 4;             // channels per thread
constexpr int SC_UNROLL = 4;        // rows loaded before the first is used (forward)
constexpr int SC_RUN = 64;          // tokens of a run, at most (backward: of one that is not stretched)
constexpr int SC_MIN_RUN = 8;       // and at least: more than K - 1
constexpr int SC_RING = 4;          // rows in flight per thread (backward)
constexpr int SC_BWD_UNROLL = 8;    // rows between two register renamings of the windows (backward)
constexpr int SC_BWD_X = 32;        // pieces of the channels per block (backward)
constexpr int SC_BWD_Y = 4;         // runs per block (backward)
constexpr int SC_BWD_BLOCKS = 4;    // blocks on an SM (backward)

struct ConvParams {
  const void *x, *S0, *dout, *dS_out;
  void *o, *S_out, *dx, *dS0;
  const float *w, *bias;   // [D][K], [D]
  const int* lens;
  float* part;             // backward: [blocks][K + 1][D] partial sums of dw_0..dw_{K-1}, dbias
  int B, L, D, silu, run, runs;   // tokens per run, runs per sequence
  int nch;                 // pieces of the channels
};

template <typename T, int V, int K>
__device__ __forceinline__ void conv_load_w(const ConvParams& p, int c, float (&w)[K][V]) {
  // [D][K] rows: the thread's V * K weights are contiguous
  float f[V * K];
#pragma unroll
  for (int i = 0; i < V * K / 4; ++i)
    *reinterpret_cast<float4*>(f + 4 * i) =
        reinterpret_cast<const float4*>(p.w + static_cast<long long>(c) * K)[i];
#pragma unroll
  for (int j = 0; j < K; ++j)
#pragma unroll
    for (int v = 0; v < V; ++v) w[j][v] = f[v * K + j];
}

// Row t of [S0; x] (t >= -(K-1)) of one sequence, as fp32; zero where there is none.
template <typename T, int V, int K>
__device__ __forceinline__ void conv_row(const ConvParams& p, int b, int t, int c, float (&f)[V]) {
  VecPack<T, V> v;
  if (t >= 0)
    v.load(static_cast<const T*>(p.x) + (static_cast<long long>(b) * p.L + t) * p.D + c);
  else if (p.S0)
    v.load(static_cast<const T*>(p.S0) + (static_cast<long long>(b) * (K - 1) + t + K - 1) * p.D + c);
  else
    v.zero();
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] = to_f32(v.e[i]);
}

template <typename T, int K, bool SILU>
__global__ __launch_bounds__(SC_THREADS) void short_conv_fwd_kernel(const ConvParams p) {
  constexpr int V = SC_V;
  const long long gid = static_cast<long long>(blockIdx.x) * SC_THREADS + threadIdx.x;
  const long long rid = gid / p.nch;
  const int c = static_cast<int>(gid - rid * p.nch) * V;
  if (rid >= static_cast<long long>(p.B) * p.runs) return;
  const int b = static_cast<int>(rid / p.runs), run = static_cast<int>(rid - static_cast<long long>(b) * p.runs);
  const int len = seq_len(p.lens, b, p.L);
  const int t0 = run * p.run, t1 = min(t0 + p.run, len);
  const long long base = static_cast<long long>(b) * p.L * p.D + c;

  float win[K - 1][V];
  if (t0 < t1) {
#pragma unroll
    for (int j = 0; j < K - 1; ++j) conv_row<T, V, K>(p, b, t0 - (K - 1) + j, c, win[j]);
  }
  if (run == 0 && p.S_out) {
    // rows len .. len + K - 2 of [S0; x]; all are read before any is written (S_out may be S0)
    VecPack<T, V> e[K - 1];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      const int t = len + j - (K - 1);
      if (t >= 0)
        e[j].load(static_cast<const T*>(p.x) + base + static_cast<long long>(t) * p.D);
      else if (p.S0)
        e[j].load(static_cast<const T*>(p.S0) + (static_cast<long long>(b) * (K - 1) + t + K - 1) * p.D + c);
      else
        e[j].zero();
    }
#pragma unroll
    for (int j = 0; j < K - 1; ++j)
      e[j].store(static_cast<T*>(p.S_out) + (static_cast<long long>(b) * (K - 1) + j) * p.D + c);
  }
  if (t0 >= t1) return;

  float w[K][V], bias[V];
  conv_load_w<T, V, K>(p, c, w);
#pragma unroll
  for (int i = 0; i < V; ++i) bias[i] = p.bias ? p.bias[c + i] : 0.f;
  const T* x = static_cast<const T*>(p.x) + base + static_cast<long long>(t0) * p.D;
  T* o = static_cast<T*>(p.o) + base + static_cast<long long>(t0) * p.D;
  auto row = [&](const VecPack<T, V>& r, T* dst) {
    VecPack<T, V> y;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float xv = to_f32(r.e[i]);
      float a = bias[i];
#pragma unroll
      for (int j = 0; j < K - 1; ++j) a = fmaf(w[j][i], win[j][i], a);
      a = fmaf(w[K - 1][i], xv, a);
#pragma unroll
      for (int j = 0; j + 1 < K - 1; ++j) win[j][i] = win[j + 1][i];
      win[K - 2][i] = xv;
      y.e[i] = from_f32<T>(SILU ? a * sigmoid_f32(a) : a);
    }
    y.store(dst);
  };
  // whole groups of rows without a test, so that the window moves by renaming registers
  int t = t0;
  for (; t + SC_UNROLL <= t1; t += SC_UNROLL) {
    VecPack<T, V> r[SC_UNROLL];
#pragma unroll
    for (int u = 0; u < SC_UNROLL; ++u) r[u].load(x + static_cast<long long>(u) * p.D);
#pragma unroll
    for (int u = 0; u < SC_UNROLL; ++u) row(r[u], o + static_cast<long long>(u) * p.D);
    x += static_cast<long long>(SC_UNROLL) * p.D;
    o += static_cast<long long>(SC_UNROLL) * p.D;
  }
  for (; t < t1; ++t, x += p.D, o += p.D) {
    VecPack<T, V> r;
    r.load(x);
    row(r, o);
  }
}

// Two fp32 values per element pair of a bf16 or fp32 piece.
__device__ __forceinline__ uint64_t conv_pair(const VecPack<__nv_bfloat16, 4>& v, int i) {
  const uint32_t x = i ? v.raw.y : v.raw.x;
  return f32x2_pack(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}
__device__ __forceinline__ uint64_t conv_pair(const VecPack<float, 4>& v, int i) {
  return f32x2_pack(v.e[2 * i], v.e[2 * i + 1]);
}

// Backward. One block = SC_BWD_X pieces of 4 channels x SC_BWD_Y runs of one sequence. Rows come through
// a ring of the thread's own pieces in shared memory, SC_RING ahead, so nothing waits for a load but the
// first; arithmetic runs on packed pairs of channels.
template <typename T, int K, bool SILU>
__global__ __launch_bounds__(SC_BWD_X* SC_BWD_Y, SC_BWD_BLOCKS) void short_conv_bwd_kernel(const ConvParams p) {
  constexpr int V = SC_V, P = V / 2;
  __shared__ typename VecPack<T, V>::Raw ring[SC_RING][2][SC_BWD_X * SC_BWD_Y];
  __shared__ __align__(16) float red[SC_BWD_Y][K + 1][SC_BWD_X * V + 4];
  chain_start();
  const int xb = (p.nch + SC_BWD_X - 1) / SC_BWD_X, yb = (p.runs + SC_BWD_Y - 1) / SC_BWD_Y;
  const long long blk = blockIdx.x / xb;     // (sequence, block of runs)
  const int cx = static_cast<int>(blockIdx.x - blk * xb) * SC_BWD_X + (threadIdx.x % SC_BWD_X);
  const int ry = threadIdx.x / SC_BWD_X;
  const int b = static_cast<int>(blk / yb), run = static_cast<int>(blk - static_cast<long long>(b) * yb) * SC_BWD_Y + ry;
  const int c = cx * V;
  const int len = seq_len(p.lens, b, p.L);
  const int t0 = run * p.run, t1 = min(t0 + p.run, len);
  uint64_t dw[K + 1][P];
#pragma unroll
  for (int j = 0; j <= K; ++j)
#pragma unroll
    for (int i = 0; i < P; ++i) dw[j][i] = 0;

  const bool own = cx < p.nch && run < p.runs && (t0 < t1 || (run == 0 && p.dS0));
  if (own) {
    uint64_t w[K][P], bias[P], win[K][P], dp[K][P];   // rows s-K+1..s; dp_{s-K+1}..dp_s
    {
      float f[K][V];
      conv_load_w<T, V, K>(p, c, f);
#pragma unroll
      for (int j = 0; j < K; ++j)
#pragma unroll
        for (int i = 0; i < P; ++i) {
          w[j][i] = f32x2_pack(f[j][2 * i], f[j][2 * i + 1]);
          dp[j][i] = 0;
        }
#pragma unroll
      for (int j = 1; j < K; ++j) {
        conv_row<T, V, K>(p, b, t0 - K + j, c, f[0]);
#pragma unroll
        for (int i = 0; i < P; ++i) win[j][i] = f32x2_pack(f[0][2 * i], f[0][2 * i + 1]);
      }
#pragma unroll
      for (int i = 0; i < P; ++i)
        bias[i] = p.bias ? f32x2_pack(p.bias[c + 2 * i], p.bias[c + 2 * i + 1]) : 0;
    }
    const long long base = static_cast<long long>(b) * p.L * p.D + c;
    // Rows past the sequence's end come as zeros.
    const int s_end = t1 + K - 1;
    auto fetch = [&](int s, int slot) {
      if (s < s_end) {
        const bool on = s < len;
        const long long at = on ? base + static_cast<long long>(s) * p.D : 0;
        piece_async<V * int(sizeof(T))>(&ring[slot][0][threadIdx.x], static_cast<const T*>(p.x) + at, on);
        piece_async<V * int(sizeof(T))>(&ring[slot][1][threadIdx.x], static_cast<const T*>(p.dout) + at, on);
      }
      piece_commit();
    };
#pragma unroll
    for (int u = 0; u < SC_RING; ++u) fetch(t0 + u, u);
    int slot = 0;
    // One row s: its dp, its share of dw and dbias (rows of the run alone), and dx of row s - K + 1, which
    // it completes.
    auto row = [&](int s, bool mine) {
      piece_wait<SC_RING - 1>();
      VecPack<T, V> xr, gr, out;
      xr.raw = ring[slot][0][threadIdx.x];
      gr.raw = ring[slot][1][threadIdx.x];
      fetch(s + SC_RING, slot);
      slot = (slot + 1) % SC_RING;
      const int t = s - (K - 1);
      const bool end = p.dS_out && t - len + (K - 1) >= 0;   // row t is one of the end state's
      VecPack<T, V> ev;
      if (end)
        ev.load(static_cast<const T*>(p.dS_out) + (static_cast<long long>(b) * (K - 1) + t - len + K - 1) * p.D + c);
#pragma unroll
      for (int i = 0; i < P; ++i) {
#pragma unroll
        for (int j = 0; j + 1 < K; ++j) {
          win[j][i] = win[j + 1][i];
          dp[j][i] = dp[j + 1][i];
        }
        win[K - 1][i] = conv_pair(xr, i);
        uint64_t g = conv_pair(gr, i);
        if (SILU) {
          uint64_t a = bias[i];
#pragma unroll
          for (int j = 0; j < K; ++j) a = ffma2(w[j][i], win[j][i], a);
          const float2 e = f32x2_unpack(fmul2(a, f32x2_pack(-1.4426950408889634f, -1.4426950408889634f)));
          const float2 q = f32x2_unpack(fadd2(f32x2_pack(ex2_approx(e.x), ex2_approx(e.y)), f32x2_pack(1.f, 1.f)));
          const uint64_t sg = f32x2_pack(rcp_approx(q.x), rcp_approx(q.y));
          const uint64_t cg = ffma2(sg, f32x2_pack(-1.f, -1.f), f32x2_pack(1.f, 1.f));
          g = fmul2(g, fmul2(sg, ffma2(a, cg, f32x2_pack(1.f, 1.f))));
          if (!mine && s >= len) g = 0;       // no row: 0 times the slope of what is not finite is no 0
        }
        dp[K - 1][i] = g;
        if (mine) {
#pragma unroll
          for (int j = 0; j < K; ++j) dw[j][i] = ffma2(g, win[j][i], dw[j][i]);
          dw[K][i] = fadd2(dw[K][i], g);
        }
        uint64_t d = fmul2(w[0][i], dp[K - 1][i]);
#pragma unroll
        for (int j = 1; j < K; ++j) d = ffma2(w[j][i], dp[K - 1 - j][i], d);
        if (end) d = fadd2(d, conv_pair(ev, i));
        const float2 o = f32x2_unpack(d);
        out.e[2 * i] = from_f32<T>(o.x);
        out.e[2 * i + 1] = from_f32<T>(o.y);
      }
      if (t >= t0)
        out.store(static_cast<T*>(p.dx) + base + static_cast<long long>(t) * p.D);
      else if (run == 0 && p.dS0)
        out.store(static_cast<T*>(p.dS0) + (static_cast<long long>(b) * (K - 1) + t + K - 1) * p.D + c);
    };
    int s = t0;
    for (; s + SC_BWD_UNROLL <= t1; s += SC_BWD_UNROLL) {
#pragma unroll
      for (int u = 0; u < SC_BWD_UNROLL; ++u) row(s + u, true);
    }
#pragma unroll 1
    for (; s < t1; ++s) row(s, true);
#pragma unroll 1
    for (; s < s_end; ++s) row(s, false);     // the next run's first rows complete dx of this one's last
    piece_wait<0>();
  }
  // sums over the block's runs, in run order
#pragma unroll
  for (int j = 0; j <= K; ++j)
#pragma unroll
    for (int i = 0; i < P; ++i)
      *reinterpret_cast<float2*>(&red[ry][j][(threadIdx.x % SC_BWD_X) * V + 2 * i]) = f32x2_unpack(dw[j][i]);
  __syncthreads();
  const int c0 = static_cast<int>(blockIdx.x - blk * xb) * SC_BWD_X * V;
  for (int i = threadIdx.x; i < (K + 1) * SC_BWD_X * V; i += SC_BWD_X * SC_BWD_Y) {
    const int j = i / (SC_BWD_X * V), cc = i - j * (SC_BWD_X * V);
    if (c0 + cc < p.D) {
      float a = 0.f;
#pragma unroll
      for (int y = 0; y < SC_BWD_Y; ++y) a += red[y][j][cc];
      p.part[(blk * (K + 1) + j) * p.D + c0 + cc] = a;
    }
  }
}

// dw [D][K] and dbias [D] from the partial sums, in block order: 32 columns x 8 lanes of blocks.
template <int K>
__global__ __launch_bounds__(256) void short_conv_dw_kernel(const float* part, long long blocks, int D,
                                                            float* dw, float* dbias) {
  __shared__ float red[8][33];
  const int n = (K + 1) * D, x = threadIdx.x % 32, y = threadIdx.x / 32;
  chain_wait();
  const int i = blockIdx.x * 32 + x;
  float a = 0.f;
  if (i < n)
    for (long long r = y; r < blocks; r += 8) a += part[r * n + i];
  red[y][x] = a;
  __syncthreads();
  if (y == 0 && i < n) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) s += red[k][x];
    const int j = i / D, d = i - j * D;
    if (j < K)
      dw[static_cast<long long>(d) * K + j] = s;
    else if (dbias)
      dbias[d] = s;
  }
}

}  // namespace kta

// short_conv.cuh -- short causal convolution along the tokens, one filter of K taps per channel:
//     pre_t = bias + sum_j w_j x_{t-K+1+j},   y_t = act(pre_t),   act = silu or identity,
// rows before the sequence's first come from a carried state S0 (K - 1 rows) or are zero; the end
// state is the last K - 1 rows of [S0; x]. Backward, with dp_t = dy_t act'(pre_t):
//     dx_t = sum_j w_j dp_{t+K-1-j},   dw_j = sum_t dp_t x_{t-K+1+j},   dbias = sum_t dp_t.
//
// Memory-bound (2 elements moved per output, 3 in the backward pass). A thread owns one 16-byte
// (backward: 8-byte) piece of the channels and walks a run of tokens with the last K - 1 rows in
// registers, so every row is read once per run plus the K - 1 rows before it, which its neighbour
// has brought into L2. Weights and sums are fp32.
#pragma once
#include "mixer_common.cuh"

namespace kta {

constexpr int SC_THREADS = 128;
constexpr int SC_UNROLL = 8;        // rows in flight per thread (forward); runs are multiples of it
constexpr int SC_BWD_X = 32;        // channel pieces per block (backward)
constexpr int SC_BWD_Y = 4;         // runs per block (backward)

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

template <typename T, int K>
__global__ __launch_bounds__(SC_THREADS) void short_conv_fwd_kernel(const ConvParams p) {
  constexpr int V = 16 / int(sizeof(T));
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
  const T* x = static_cast<const T*>(p.x) + base;
  T* o = static_cast<T*>(p.o) + base;
  for (int t = t0; t < t1; t += SC_UNROLL) {
    VecPack<T, V> r[SC_UNROLL];
#pragma unroll
    for (int u = 0; u < SC_UNROLL; ++u)
      if (t + u < t1) r[u].load(x + static_cast<long long>(t + u) * p.D);
#pragma unroll
    for (int u = 0; u < SC_UNROLL; ++u) {
      if (t + u < t1) {
        VecPack<T, V> y;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float xv = to_f32(r[u].e[i]);
          float a = bias[i];
#pragma unroll
          for (int j = 0; j < K - 1; ++j) a = fmaf(w[j][i], win[j][i], a);
          a = fmaf(w[K - 1][i], xv, a);
#pragma unroll
          for (int j = 0; j + 1 < K - 1; ++j) win[j][i] = win[j + 1][i];
          win[K - 2][i] = xv;
          y.e[i] = from_f32<T>(p.silu ? a * sigmoid_f32(a) : a);
        }
        y.store(o + static_cast<long long>(t + u) * p.D);
      }
    }
  }
}

// One block = SC_BWD_X pieces of the channels x SC_BWD_Y runs of one sequence.
template <typename T, int K>
__global__ __launch_bounds__(SC_BWD_X* SC_BWD_Y) void short_conv_bwd_kernel(const ConvParams p) {
  constexpr int V = 4;
  __shared__ float red[SC_BWD_Y][K + 1][SC_BWD_X * V + 4];
  const int xb = (p.nch + SC_BWD_X - 1) / SC_BWD_X, yb = (p.runs + SC_BWD_Y - 1) / SC_BWD_Y;
  const long long blk = blockIdx.x / xb;     // (sequence, block of runs)
  const int cx = static_cast<int>(blockIdx.x - blk * xb) * SC_BWD_X + (threadIdx.x % SC_BWD_X);
  const int ry = threadIdx.x / SC_BWD_X;
  const int b = static_cast<int>(blk / yb), run = static_cast<int>(blk - static_cast<long long>(b) * yb) * SC_BWD_Y + ry;
  const int c = cx * V;
  const int len = seq_len(p.lens, b, p.L);
  const int t0 = run * p.run, t1 = min(t0 + p.run, len);
  float dw[K + 1][V];
#pragma unroll
  for (int j = 0; j <= K; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) dw[j][i] = 0.f;

  const bool own = cx < p.nch && run < p.runs && (t0 < t1 || (run == 0 && p.dS0));
  if (own) {
    float w[K][V], bias[V], win[K][V], dp[K][V];   // rows s-K+1..s; dp_{s-K+1}..dp_s
    conv_load_w<T, V, K>(p, c, w);
#pragma unroll
    for (int i = 0; i < V; ++i) bias[i] = p.bias ? p.bias[c + i] : 0.f;
#pragma unroll
    for (int j = 0; j < K; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) dp[j][i] = 0.f;
#pragma unroll
    for (int j = 1; j < K; ++j) conv_row<T, V, K>(p, b, t0 - K + j, c, win[j]);
    const long long base = static_cast<long long>(b) * p.L * p.D + c;
    // s runs past the run's end to complete dx of its last K - 1 rows
    for (int s = t0; s < t1 + K - 1; ++s) {
#pragma unroll
      for (int j = 0; j + 1 < K; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          win[j][i] = win[j + 1][i];
          dp[j][i] = dp[j + 1][i];
        }
      if (s < len) {
        VecPack<T, V> xv, gv;
        xv.load(static_cast<const T*>(p.x) + base + static_cast<long long>(s) * p.D);
        gv.load(static_cast<const T*>(p.dout) + base + static_cast<long long>(s) * p.D);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          win[K - 1][i] = to_f32(xv.e[i]);
          float g = to_f32(gv.e[i]);
          if (p.silu) {
            float a = bias[i];
#pragma unroll
            for (int j = 0; j < K; ++j) a = fmaf(w[j][i], win[j][i], a);
            const float sg = sigmoid_f32(a);
            g *= sg * fmaf(a, 1.f - sg, 1.f);
          }
          dp[K - 1][i] = g;
        }
        if (s < t1) {
#pragma unroll
          for (int i = 0; i < V; ++i) {
#pragma unroll
            for (int j = 0; j < K; ++j) dw[j][i] = fmaf(dp[K - 1][i], win[j][i], dw[j][i]);
            dw[K][i] += dp[K - 1][i];
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) dp[K - 1][i] = 0.f;
      }
      // dx of row t = s - K + 1 takes dp_t .. dp_s
      const int t = s - (K - 1);
      if (t >= t0 || (run == 0 && p.dS0)) {
        float d[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
          d[i] = 0.f;
#pragma unroll
          for (int j = 0; j < K; ++j) d[i] = fmaf(w[j][i], dp[K - 1 - j][i], d[i]);
        }
        const int e = t - len + (K - 1);        // row of the end state, if it is one
        if (p.dS_out && e >= 0) {
          VecPack<T, V> ev;
          ev.load(static_cast<const T*>(p.dS_out) + (static_cast<long long>(b) * (K - 1) + e) * p.D + c);
#pragma unroll
          for (int i = 0; i < V; ++i) d[i] += to_f32(ev.e[i]);
        }
        VecPack<T, V> out;
#pragma unroll
        for (int i = 0; i < V; ++i) out.e[i] = from_f32<T>(d[i]);
        if (t >= 0)
          out.store(static_cast<T*>(p.dx) + base + static_cast<long long>(t) * p.D);
        else
          out.store(static_cast<T*>(p.dS0) + (static_cast<long long>(b) * (K - 1) + t + K - 1) * p.D + c);
      }
    }
  }
  // sums over the block's runs, in run order
#pragma unroll
  for (int j = 0; j <= K; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) red[ry][j][(threadIdx.x % SC_BWD_X) * V + i] = dw[j][i];
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

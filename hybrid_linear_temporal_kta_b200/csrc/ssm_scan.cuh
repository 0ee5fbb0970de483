// ssm_scan.cuh -- selective state-space scan. Per sequence, channel c and state n, with
// d_t = softplus(dt_t + dt_bias):
//     h_t = exp(d_t A) h_{t-1} + d_t u_t B_t,    y_t = (C_t . h_t + Dskip u_t) silu(z_t),
// B and C shared by the channels of a group. States, gates and sums are fp32.
//
// Bound by the exponential unit: one exponential per (token, channel, state), a warp's 32 in 8 cycles
// of its scheduler, against 8 bytes per (token, channel) in bf16.
#pragma once
#include "mixer_common.cuh"

namespace kta {

constexpr int SSM_THREADS = 128;
constexpr int SSM_CH = 32;      // channels per warp (forward) or block (backward)
constexpr int SSM_TT = 8;       // tokens per tile (forward)
constexpr int SSM_MAX_N = 32;

struct SsmParams {
  const void *u, *dt, *Bm, *Cm, *z;
  const float *A, *Dskip, *dt_bias, *S0;
  const int* lens;
  void* y;
  float* S_out;
  int B, L, D, N, G, Dg;         // Dg = D / G channels per group
  int cbg;                       // channel blocks per group
  int nseg, seg;                 // segments of the sequence and their tokens (a multiple of SSM_TT)
  int bc_bytes;                  // rows of B and C may be read in pieces of 16, 8 or 4 bytes; 0: elements
  float *seg_h, *seg_d;          // end states of segments from zero, sums of d
};

struct SsmBlock {
  int b, s, g, c0, cw;           // sequence, segment, group, first channel, channels
};

__device__ __forceinline__ SsmBlock ssm_block(const SsmParams& p, long long blk, int nseg) {
  SsmBlock k;
  const int ncb = p.G * p.cbg;
  const long long rest = blk / ncb;
  const int cb = static_cast<int>(blk - rest * ncb);
  k.b = static_cast<int>(rest / nseg);
  k.s = static_cast<int>(rest - static_cast<long long>(k.b) * nseg);
  k.g = cb / p.cbg;
  const int o = (cb - k.g * p.cbg) * SSM_CH;
  k.c0 = k.g * p.Dg + o;
  k.cw = min(SSM_CH, p.Dg - o);
  return k;
}

// States q NS .. of one channel's row of N (16-byte aligned where N = 4 NS); zero past N.
template <int NS>
__device__ __forceinline__ void ssm_load_states(const float* row, int q, int N, float (&f)[NS]) {
  if (NS % 4 == 0 && N == 4 * NS) {
#pragma unroll
    for (int i = 0; i < NS / 4; ++i)
      *reinterpret_cast<float4*>(f + 4 * i) = reinterpret_cast<const float4*>(row + q * NS)[i];
  } else {
#pragma unroll
    for (int i = 0; i < NS; ++i) f[i] = q * NS + i < N ? row[q * NS + i] : 0.f;
  }
}

template <int NS>
__device__ __forceinline__ void ssm_store_states(float* row, int q, int N, const float (&f)[NS]) {
  if (NS % 4 == 0 && N == 4 * NS) {
#pragma unroll
    for (int i = 0; i < NS / 4; ++i)
      reinterpret_cast<float4*>(row + q * NS)[i] =
          make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < NS; ++i)
      if (q * NS + i < N) row[q * NS + i] = f[i];
  }
}

template <int NS>
__device__ __forceinline__ void lds_states(const float* s, float (&f)[NS]) {
  if constexpr (NS % 4 == 0) {
#pragma unroll
    for (int i = 0; i < NS / 4; ++i)
      *reinterpret_cast<float4*>(f + 4 * i) = reinterpret_cast<const float4*>(s)[i];
  } else if constexpr (NS == 2) {
    *reinterpret_cast<float2*>(f) = *reinterpret_cast<const float2*>(s);
  } else {
    f[0] = s[0];
  }
}

// Copies rows t0 .. t0 + TT - 1 of B (or C), group g, to fp32 rows of 4 NS; rows from `end` on are 0.
template <typename T, int NS, int TT>
__device__ __forceinline__ void ssm_stage_bc(const SsmParams& p, const void* src, int b, int g, int t0,
                                             int end, float* dst) {
  constexpr int V = 16 / int(sizeof(T));
  const T* rows = static_cast<const T*>(src);
  const long long ld = static_cast<long long>(p.G) * p.N;
  const long long r0 = (static_cast<long long>(b) * p.L + t0) * ld + g * p.N;
  if (p.bc_bytes == 16) {
    const int nv = p.N / V;
    for (int i = threadIdx.x; i < TT * nv; i += SSM_THREADS) {
      const int t = i / nv, v = i - t * nv;
      VecPack<T, V> x;
      x.zero();
      if (t0 + t < end) x.load(rows + r0 + t * ld + v * V);
#pragma unroll
      for (int k = 0; k < V; ++k) dst[t * 4 * NS + v * V + k] = to_f32(x.e[k]);
    }
  } else {
    for (int i = threadIdx.x; i < TT * p.N; i += SSM_THREADS) {
      const int t = i / p.N, n = i - t * p.N;
      dst[t * 4 * NS + n] = t0 + t < end ? to_f32(rows[r0 + t * ld + n]) : 0.f;
    }
  }
}

// Forward. A warp takes 32 channels of a group over one segment, a lane all states of one channel: rows
// of B and C are then the same for the whole warp (broadcast reads), and lanes exchange nothing. Raw
// tiles of 8 tokens arrive by asynchronous copies, two (fp32: one) ahead; a lane turns its channel's dt
// and u into (d, d u) for the tile, walks the tokens with its states in registers as packed pairs, gates
// the 8 outputs, and the tile leaves as 16-byte rows. Warps of a block share nothing; blocks have four so
// that each scheduler of the SM gets one. 128 registers keep 4 warps on a scheduler, which hide each
// other's exponentials: 206 cycles a token and warp against the unit's 152.
//
// (Four lanes per channel with the sum over states exchanged between them needed twice the
// instructions and shared-memory reads per token: 1.3 times the time. Computing one exponential in four
// or eight on the FMA pipe by a polynomial gained nothing: the issue slots are as short.)
template <typename T, int NP, bool OUT>
struct SsmFwdSmem {
  static constexpr int STAGES = sizeof(T) == 2 ? 3 : 2;
  struct Raw {                             // every part is the target of 16-byte copies
    alignas(16) T u[SSM_TT][SSM_CH];
    alignas(16) T d[SSM_TT][SSM_CH];
    alignas(16) T z[OUT ? SSM_TT : 1][SSM_CH];
    alignas(16) T b[SSM_TT][NP];
    alignas(16) T c[OUT ? SSM_TT : 1][NP];
  };
  Raw raw[STAGES];
  alignas(16) float bc[SSM_TT][OUT ? 2 : 1][NP];   // rows of B (and C) of the current tile, fp32
  alignas(16) float2 dd[SSM_TT][SSM_CH];           // d, d u; then (x) the token's C . h
};

static_assert(sizeof(SsmFwdSmem<__nv_bfloat16, 4, false>) % 16 == 0 &&
                  sizeof(SsmFwdSmem<__nv_bfloat16, 4, false>::Raw) % 16 == 0,
              "warps' and stages' parts stay 16-byte aligned");

// One piece size of a tile's rows of B and C.
template <typename T, int NP, bool OUT, int BYTES, typename Raw>
__device__ __forceinline__ void ssm_fetch_bc(const SsmParams& p, Raw& r, long long row0, int g, int t0, int t_end,
                                             int lane) {
  constexpr int V = BYTES / int(sizeof(T)) > 0 ? BYTES / int(sizeof(T)) : 1, NV = (NP + V - 1) / V;
#pragma unroll
  for (int m = 0; m < (SSM_TT * NV + 31) / 32; ++m) {
    const int it = lane + m * 32, t = it / NV, n = it % NV * V;
    if (it < SSM_TT * NV && n < p.N) {
      const bool on = t0 + t < t_end;
      const long long at = on ? ((row0 + t0 + t) * p.G + g) * p.N + n : 0;
      piece_async<BYTES>(&r.b[t][n], static_cast<const T*>(p.Bm) + at, on);
      if (OUT) piece_async<BYTES>(&r.c[t][n], static_cast<const T*>(p.Cm) + at, on);
    }
  }
}

// OUT: outputs (and, past the last segment, the end state) from the state that enters the segment.
// Otherwise: the segment's end state from zero (seg_h [B][nseg][NP][D]) and its sum of d.
template <typename T, int NP, bool OUT>
__global__ __launch_bounds__(SSM_THREADS, NP > 16 ? 3 : 4) void ssm_fwd_kernel(const SsmParams p) {
  using Smem = SsmFwdSmem<T, NP, OUT>;
  constexpr int V = 16 / int(sizeof(T)), CPR = SSM_CH / V, STAGES = Smem::STAGES;
  extern __shared__ __align__(16) unsigned char ssm_smem[];
  Smem& sm = reinterpret_cast<Smem*>(ssm_smem)[threadIdx.x / 32];
  const int lane = threadIdx.x % 32;
  const int nseg = OUT ? p.nseg : p.nseg - 1;
  const long long wid = blockIdx.x * static_cast<long long>(SSM_THREADS / 32) + threadIdx.x / 32;
  if (wid >= static_cast<long long>(p.B) * nseg * p.G * p.cbg) return;
  const SsmBlock k = ssm_block(p, wid, nseg);
  const bool live = lane < k.cw;
  const int c = k.c0 + (live ? lane : 0);
  const int len = seq_len(p.lens, k.b, p.L);
  const int t_begin = k.s * p.seg, t_end = min(t_begin + p.seg, len);
  const long long row0 = static_cast<long long>(k.b) * p.L;

  auto fetch = [&](int t0, int stage) {
    typename Smem::Raw& r = sm.raw[stage];
#pragma unroll
    for (int m = 0; m < SSM_TT * CPR / 32; ++m) {
      const int it = lane + m * 32, t = it / CPR, cc = it % CPR * V;
      const bool on = t0 + t < t_end && cc < k.cw;
      const long long at = on ? (row0 + t0 + t) * p.D + k.c0 + cc : 0;
      piece_async<16>(&r.u[t][cc], static_cast<const T*>(p.u) + at, on);
      piece_async<16>(&r.d[t][cc], static_cast<const T*>(p.dt) + at, on);
      if (OUT && p.z) piece_async<16>(&r.z[t][cc], static_cast<const T*>(p.z) + at, on);
    }
    if (p.bc_bytes == 16)
      ssm_fetch_bc<T, NP, OUT, 16>(p, r, row0, k.g, t0, t_end, lane);
    else if (p.bc_bytes == 8)
      ssm_fetch_bc<T, NP, OUT, 8>(p, r, row0, k.g, t0, t_end, lane);
    else if (p.bc_bytes == 4)
      ssm_fetch_bc<T, NP, OUT, 4>(p, r, row0, k.g, t0, t_end, lane);
    piece_commit();
  };
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) fetch(t_begin + s * SSM_TT, s);

  float2 A2[NP / 2], h[NP / 2];                          // pairs of states; zero past N
  const float* Arow = p.A + static_cast<long long>(c) * p.N;
#pragma unroll
  for (int i = 0; i < NP / 2; ++i) {
    A2[i].x = 2 * i < p.N ? Arow[2 * i] * 1.4426950408889634f : 0.f;
    A2[i].y = 2 * i + 1 < p.N ? Arow[2 * i + 1] * 1.4426950408889634f : 0.f;
    h[i] = make_float2(0.f, 0.f);
  }
  if (OUT && p.nseg > 1) {                               // entering states, left by ssm_fwd_carry
    const float* s = p.seg_h + (static_cast<long long>(k.b) * p.nseg + k.s) * NP * p.D + c;
#pragma unroll
    for (int i = 0; i < NP / 2; ++i) {
      h[i].x = s[static_cast<long long>(2 * i) * p.D];
      h[i].y = s[static_cast<long long>(2 * i + 1) * p.D];
    }
  } else if (OUT && p.S0) {
    const float* s = p.S0 + (static_cast<long long>(k.b) * p.D + c) * p.N;
#pragma unroll
    for (int i = 0; i < NP / 2; ++i) {
      h[i].x = 2 * i < p.N ? s[2 * i] : 0.f;
      h[i].y = 2 * i + 1 < p.N ? s[2 * i + 1] : 0.f;
    }
  }
  for (int i = lane; i < SSM_TT * (OUT ? 2 : 1) * NP; i += 32) (&sm.bc[0][0][0])[i] = 0.f;

  const float bias = p.dt_bias ? p.dt_bias[c] : 0.f, skip = OUT && p.Dskip ? p.Dskip[c] : 0.f;
  float sum_d = 0.f;
  int stage = 0;
  for (int t0 = t_begin; t0 < t_end; t0 += SSM_TT) {
    piece_wait<STAGES - 2>();
    __syncwarp();                                        // every lane's pieces are there; dd, bc are free
    typename Smem::Raw& r = sm.raw[stage];
#pragma unroll
    for (int j = 0; j < SSM_TT; ++j) {                   // past the end d = 0: the state stays
      float d = softplus_f32(to_f32(r.d[j][lane]) + bias);
      d = t0 + j < t_end ? d : 0.f;
      if (!OUT) sum_d += d;
      sm.dd[j][lane] = make_float2(d, d * to_f32(r.u[j][lane]));
    }
    if (p.bc_bytes) {
      constexpr int NQ = NP / 4;
#pragma unroll
      for (int m = 0; m < (SSM_TT * NQ + 31) / 32; ++m) {
        const int it = lane + m * 32, t = it / NQ, n = it % NQ * 4;
        if (it < SSM_TT * NQ && n < p.N) {
#pragma unroll
          for (int w = 0; w < (OUT ? 2 : 1); ++w) {
            VecPack<T, 4> x;
            x.load(w ? &r.c[OUT ? t : 0][n] : &r.b[t][n]);
            float4 f = make_float4(to_f32(x.e[0]), to_f32(x.e[1]), to_f32(x.e[2]), to_f32(x.e[3]));
            if (n + 4 > p.N) {                           // the row ends inside the quad
              f.y = n + 1 < p.N ? f.y : 0.f;
              f.z = n + 2 < p.N ? f.z : 0.f;
              f.w = 0.f;
            }
            *reinterpret_cast<float4*>(&sm.bc[t][w][n]) = f;
          }
        }
      }
    } else {                                             // an odd row of 2-byte elements
      for (int it = lane; it < SSM_TT * p.N; it += 32) {
        const int t = it / p.N, n = it - t * p.N;
        const bool on = t0 + t < t_end;
        const long long at = on ? ((row0 + t0 + t) * p.G + k.g) * p.N + n : 0;
        sm.bc[t][0][n] = on ? to_f32(static_cast<const T*>(p.Bm)[at]) : 0.f;
        if (OUT) sm.bc[t][OUT ? 1 : 0][n] = on ? to_f32(static_cast<const T*>(p.Cm)[at]) : 0.f;
      }
    }
    __syncwarp();
    fetch(t0 + (STAGES - 1) * SSM_TT, stage == 0 ? STAGES - 1 : stage - 1);   // into the tile before's place
#pragma unroll
    for (int j = 0; j < SSM_TT; ++j) {
      const float2 dd = sm.dd[j][lane];
      const uint64_t d2 = f32x2_pack(dd.x, dd.x), du2 = f32x2_pack(dd.y, dd.y);
      uint64_t acc[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < NP / 2; i += 2) {
        const ulonglong2 b4 = *reinterpret_cast<const ulonglong2*>(&sm.bc[j][0][2 * i]);
        ulonglong2 c4;
        if (OUT) c4 = *reinterpret_cast<const ulonglong2*>(&sm.bc[j][OUT ? 1 : 0][2 * i]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float2 x = f32x2_unpack(fmul2(d2, f32x2_pack(A2[i + e])));
          const uint64_t a = f32x2_pack(ex2_approx(x.x), ex2_approx(x.y));
          const uint64_t hn = ffma2(a, f32x2_pack(h[i + e]), fmul2(du2, e ? b4.y : b4.x));
          h[i + e] = f32x2_unpack(hn);
          if (OUT) acc[e] = ffma2(hn, e ? c4.y : c4.x, acc[e]);
        }
      }
      if (OUT) {
        const float2 y = f32x2_unpack(fadd2(acc[0], acc[1]));
        sm.dd[j][lane].x = y.x + y.y;
      }
    }
    if (OUT) {
#pragma unroll
      for (int j = 0; j < SSM_TT; ++j) {                 // the outputs take the place of u
        float y = fmaf(skip, to_f32(r.u[j][lane]), sm.dd[j][lane].x);
        if (p.z) {
          const float z = to_f32(r.z[j][lane]);
          y *= z * sigmoid_f32(z);
        }
        r.u[j][lane] = from_f32<T>(y);
      }
      __syncwarp();
#pragma unroll
      for (int m = 0; m < SSM_TT * CPR / 32; ++m) {
        const int it = lane + m * 32, t = it / CPR, cc = it % CPR * V;
        if (t0 + t < t_end && cc < k.cw)
          *reinterpret_cast<uint4*>(static_cast<T*>(p.y) + (row0 + t0 + t) * p.D + k.c0 + cc) =
              *reinterpret_cast<const uint4*>(&r.u[t][cc]);
      }
    }
    stage = stage == STAGES - 1 ? 0 : stage + 1;
  }
  if (!live) return;
  if (OUT) {
    if (p.S_out && k.s == p.nseg - 1) {
      float* s = p.S_out + (static_cast<long long>(k.b) * p.D + c) * p.N;
#pragma unroll
      for (int i = 0; i < NP / 2; ++i) {
        if (2 * i < p.N) s[2 * i] = h[i].x;
        if (2 * i + 1 < p.N) s[2 * i + 1] = h[i].y;
      }
    }
  } else {
    const long long r = static_cast<long long>(k.b) * p.nseg + k.s;
    float* s = p.seg_h + r * NP * p.D + c;
#pragma unroll
    for (int i = 0; i < NP / 2; ++i) {
      s[static_cast<long long>(2 * i) * p.D] = h[i].x;
      s[static_cast<long long>(2 * i + 1) * p.D] = h[i].y;
    }
    p.seg_d[r * p.D + c] = sum_d;
  }
}

// One thread per (sequence, state, channel): in place, end states of segments from zero become the
// states that enter them. Loads of SSM_CARRY_UNROLL segments are in flight at once.
constexpr int SSM_CARRY_UNROLL = 8;

__global__ __launch_bounds__(256) void ssm_fwd_carry_kernel(const SsmParams p, int NP) {
  const long long per = static_cast<long long>(p.D) * NP;
  const long long gid = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (gid >= per * p.B) return;
  const int b = static_cast<int>(gid / per);
  const int n = static_cast<int>(gid % per / p.D), c = static_cast<int>(gid % p.D);
  const long long e = static_cast<long long>(c) * p.N + n;
  const bool on = n < p.N;
  const float A2 = on ? p.A[e] * 1.4426950408889634f : 0.f;
  float h = on && p.S0 ? p.S0[static_cast<long long>(b) * p.D * p.N + e] : 0.f;
  float* hs = p.seg_h + (static_cast<long long>(b) * p.nseg * NP + n) * p.D + c;
  const float* ds = p.seg_d + static_cast<long long>(b) * p.nseg * p.D + c;
  for (int s0 = 0; s0 < p.nseg; s0 += SSM_CARRY_UNROLL) {
    float v[SSM_CARRY_UNROLL], d[SSM_CARRY_UNROLL];
#pragma unroll
    for (int i = 0; i < SSM_CARRY_UNROLL; ++i)
      if (s0 + i < p.nseg - 1) {
        v[i] = hs[(s0 + i) * per];
        d[i] = ds[static_cast<long long>(s0 + i) * p.D];
      }
#pragma unroll
    for (int i = 0; i < SSM_CARRY_UNROLL; ++i)
      if (s0 + i < p.nseg) {
        hs[(s0 + i) * per] = h;
        if (s0 + i < p.nseg - 1) h = fmaf(ex2_approx(d[i] * A2), h, v[i]);
      }
  }
}

// One token: memory-bound, the state read and written once (8 bytes per state against 8 per channel
// of u, dt, z and y). A lane owns a state quarter of one channel and walks SSM_STEP_B sequences with
// its row of A in registers.
constexpr int SSM_STEP_B = 4;

template <typename T, int NS>
__global__ __launch_bounds__(SSM_THREADS) void ssm_step_kernel(const SsmParams p) {
  const int q = threadIdx.x % 4;
  const long long item = (static_cast<long long>(blockIdx.x) * SSM_THREADS + threadIdx.x) / 4;
  const int b0 = static_cast<int>(item / p.D) * SSM_STEP_B;   // D % 8 == 0: the same for a warp
  const int c = static_cast<int>(item % p.D), g = c / p.Dg;
  if (b0 >= p.B) return;
  const int nb = min(SSM_STEP_B, p.B - b0);
  const bool vec = NS % 4 == 0 && p.N == 4 * NS && p.bc_bytes == 16;
  float h[SSM_STEP_B][NS], bv[SSM_STEP_B][NS], cv[SSM_STEP_B][NS], u[SSM_STEP_B], d[SSM_STEP_B], z[SSM_STEP_B];
#pragma unroll
  for (int j = 0; j < SSM_STEP_B; ++j) {
    if (j < nb) {
      const long long r = static_cast<long long>(b0 + j) * p.D + c;
      const long long bc = (static_cast<long long>(b0 + j) * p.G + g) * p.N;
      ssm_load_states<NS>(p.S0 + r * p.N, q, p.N, h[j]);
      u[j] = to_f32(static_cast<const T*>(p.u)[r]);
      d[j] = to_f32(static_cast<const T*>(p.dt)[r]);
      if (p.z) z[j] = to_f32(static_cast<const T*>(p.z)[r]);
      if (vec) {
        constexpr int V = NS * int(sizeof(T)) > 16 ? 16 / int(sizeof(T)) : NS;
#pragma unroll
        for (int v = 0; v < NS / V; ++v) {
          VecPack<T, V> x, y;
          x.load(static_cast<const T*>(p.Bm) + bc + q * NS + v * V);
          y.load(static_cast<const T*>(p.Cm) + bc + q * NS + v * V);
#pragma unroll
          for (int i = 0; i < V; ++i) {
            bv[j][v * V + i] = to_f32(x.e[i]);
            cv[j][v * V + i] = to_f32(y.e[i]);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          const int n = q * NS + i;
          bv[j][i] = n < p.N ? to_f32(static_cast<const T*>(p.Bm)[bc + n]) : 0.f;
          cv[j][i] = n < p.N ? to_f32(static_cast<const T*>(p.Cm)[bc + n]) : 0.f;
        }
      }
    }
  }
  float A2[NS];
  ssm_load_states<NS>(p.A + static_cast<long long>(c) * p.N, q, p.N, A2);
#pragma unroll
  for (int i = 0; i < NS; ++i) A2[i] *= 1.4426950408889634f;
  const float bias = p.dt_bias ? p.dt_bias[c] : 0.f, skip = p.Dskip ? p.Dskip[c] : 0.f;
#pragma unroll
  for (int j = 0; j < SSM_STEP_B; ++j) {
    if (j < nb) {                                        // the same for a warp
      const long long r = static_cast<long long>(b0 + j) * p.D + c;
      const float dl = softplus_f32(d[j] + bias), du = dl * u[j];
      float y = 0.f;
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        h[j][i] = fmaf(ex2_approx(dl * A2[i]), h[j][i], du * bv[j][i]);
        y = fmaf(h[j][i], cv[j][i], y);
      }
      ssm_store_states<NS>(p.S_out + r * p.N, q, p.N, h[j]);
      y += __shfl_xor_sync(0xffffffffu, y, 1);
      y += __shfl_xor_sync(0xffffffffu, y, 2);
      if (q == 0) {
        y = fmaf(skip, u[j], y);
        if (p.z) y *= z[j] * sigmoid_f32(z[j]);
        static_cast<T*>(p.y)[r] = from_f32<T>(y);
      }
    }
  }
}

// ---------------------------------------------------------------------------------- backward
//
// With dy_t = dout_t silu(z_t) and G_t = dL/dh_t = dy_t C_t + exp(d_{t+1} A) G_{t+1}:
//     dC_t = sum_c dy_t h_t,        dB_t = sum_c G_t d_t u_t,      dx_t = sum_n G_t B_t,
//     w_t = G_t exp(d_t A) h_{t-1}, dd_t = dx_t u_t + sum_n w_t A, dA = sum_t w_t d_t,
//     du_t = dx_t d_t + Dskip dy_t, ddt_t = dd_t sigmoid(dt_t + dt_bias),
//     dz_t = dout_t y_t silu'(z_t), dDskip = sum_t dy_t u_t,       ddt_bias = sum_t ddt_t.
// Three launches over segments of SEG tokens, all segments at once:
//  1. ssm_bwd_local: each segment's end state from zero, its share of the adjoint that leaves it at
//     its start (P_t the running product of decays: sum_t P_t dy_t C_t), and its sum of d;
//  2. ssm_bwd_carry: folds both along the sequence: the state that enters each segment and the
//     adjoint that enters it from behind (and dS0);
//  3. ssm_bwd_main: a forward walk keeps the state before every GT tokens in shared memory; then,
//     last group first, the group's states are formed again in registers and the adjoint walks back.
// Sums over channels (dB, dC) are joined over a warp by halving exchanges, then over the block, the
// channel blocks and finally by ssm_bwd_bc in a fixed order; dA, dDskip and ddt_bias likewise.

template <int NS> struct SsmBwdCfg {
  static constexpr int GT = NS <= 4 ? 8 : 4;       // tokens whose states fit in registers
  static constexpr int GROUPS = 8;
  static constexpr int SEG = GT * GROUPS;
};

struct SsmBwdParams {
  SsmParams f;                   // inputs; nseg / seg of the backward; seg_h: entering states
  const void *dout;
  const float* dS_out;
  void *du, *ddt, *dz, *dB, *dC;
  float *dA, *dD, *ddt_bias, *dS0;
  float* seg_g;                  // [B][nseg][D][N]: adjoint entering each segment from behind
  float* part_bc;                // [G * cbg][B * L][2 N]
  float* part_c;                 // [B][nseg][2][D]: dDskip, ddt_bias
};

// (d, d u) and dy of a segment in shared memory; zero past its end.
template <typename T, int SEG>
__device__ __forceinline__ void ssm_bwd_stage(const SsmBwdParams& p, const SsmBlock& k, int t0, int t_end,
                                              float2 (*s_d)[SSM_CH], float (*s_dy)[SSM_CH]) {
  constexpr int V = 16 / int(sizeof(T)), CPR = SSM_CH / V;
  for (int it = threadIdx.x; it < SEG * CPR; it += SSM_THREADS) {
    const int t = it / CPR, cc = it % CPR * V;
    const bool on = t0 + t < t_end && cc < k.cw;
    VecPack<T, V> u, d, z, o;
    if (on) {
      const long long at = (static_cast<long long>(k.b) * p.f.L + t0 + t) * p.f.D + k.c0 + cc;
      u.load(static_cast<const T*>(p.f.u) + at);
      d.load(static_cast<const T*>(p.f.dt) + at);
      o.load(static_cast<const T*>(p.dout) + at);
      if (p.f.z) z.load(static_cast<const T*>(p.f.z) + at);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float2 v = make_float2(0.f, 0.f);
      float dy = 0.f;
      if (on) {
        v.x = softplus_f32(to_f32(d.e[i]) + (p.f.dt_bias ? p.f.dt_bias[k.c0 + cc + i] : 0.f));
        v.y = v.x * to_f32(u.e[i]);
        dy = to_f32(o.e[i]);
        if (p.f.z) {
          const float zf = to_f32(z.e[i]);
          dy *= zf * sigmoid_f32(zf);
        }
      }
      s_d[t][cc + i] = v;
      s_dy[t][cc + i] = dy;
    }
  }
}

template <typename T, int NS>
__global__ __launch_bounds__(SSM_THREADS) void ssm_bwd_local_kernel(const SsmBwdParams p) {
  using Cfg = SsmBwdCfg<NS>;
  __shared__ __align__(16) float2 s_d[Cfg::SEG][SSM_CH];
  __shared__ __align__(16) float s_dy[Cfg::SEG][SSM_CH];
  __shared__ __align__(16) float s_b[Cfg::SEG * 4 * NS], s_c[Cfg::SEG * 4 * NS];
  const int tid = threadIdx.x, lane = tid % 32, q = lane % 4;
  const SsmBlock k = ssm_block(p.f, blockIdx.x, p.f.nseg);
  const int ch = tid / 32 * 8 + lane / 4;
  const bool live = ch < k.cw;
  const long long c = k.c0 + (live ? ch : 0);
  const int len = seq_len(p.f.lens, k.b, p.f.L);
  const int t0 = k.s * Cfg::SEG, t_end = min(t0 + Cfg::SEG, len);
  float A2[NS], h[NS], g[NS], P[NS], sum_d = 0.f;
  ssm_load_states<NS>(p.f.A + c * p.f.N, q, p.f.N, A2);
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    A2[i] *= 1.4426950408889634f;
    h[i] = g[i] = 0.f;
    P[i] = 1.f;
  }
  if (t0 < t_end) {
    for (int i = tid; i < Cfg::SEG * 4 * NS; i += SSM_THREADS) s_b[i] = s_c[i] = 0.f;
    __syncthreads();
    ssm_stage_bc<T, NS, Cfg::SEG>(p.f, p.f.Bm, k.b, k.g, t0, t_end, s_b);
    ssm_stage_bc<T, NS, Cfg::SEG>(p.f, p.f.Cm, k.b, k.g, t0, t_end, s_c);
    ssm_bwd_stage<T, Cfg::SEG>(p, k, t0, t_end, s_d, s_dy);
    __syncthreads();
#pragma unroll 4
    for (int t = 0; t < Cfg::SEG; ++t) {
      const float2 d = s_d[t][ch];
      const float dy = s_dy[t][ch];
      float bv[NS], cv[NS];
      lds_states<NS>(s_b + t * 4 * NS + q * NS, bv);
      lds_states<NS>(s_c + t * 4 * NS + q * NS, cv);
      sum_d += d.x;
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const float a = ex2_approx(d.x * A2[i]);
        h[i] = fmaf(a, h[i], d.y * bv[i]);
        P[i] *= a;
        g[i] = fmaf(P[i], dy * cv[i], g[i]);
      }
    }
  }
  if (!live) return;
  const long long r = (static_cast<long long>(k.b) * p.f.nseg + k.s) * p.f.D + c;
  ssm_store_states<NS>(p.f.seg_h + r * p.f.N, q, p.f.N, h);
  ssm_store_states<NS>(p.seg_g + r * p.f.N, q, p.f.N, g);
  if (q == 0) p.f.seg_d[r] = sum_d;
}

// One thread per (sequence, channel, state): in place, local end states become entering states and
// local adjoints become the adjoints entering from behind.
__global__ __launch_bounds__(256) void ssm_bwd_carry_kernel(const SsmBwdParams p) {
  const long long per = static_cast<long long>(p.f.D) * p.f.N;
  const long long gid = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (gid >= per * p.f.B) return;
  const int b = static_cast<int>(gid / per);
  const long long e = gid - b * per, c = e / p.f.N;
  const float A2 = p.f.A[e] * 1.4426950408889634f;
  const int S = p.f.nseg;
  float* hs = p.f.seg_h + static_cast<long long>(b) * S * per + e;
  float* gs = p.seg_g + static_cast<long long>(b) * S * per + e;
  const float* ds = p.f.seg_d + static_cast<long long>(b) * S * p.f.D + c;
  float h = p.f.S0 ? p.f.S0[b * per + e] : 0.f;
  for (int s0 = 0; s0 < S; s0 += SSM_CARRY_UNROLL) {
    float v[SSM_CARRY_UNROLL], d[SSM_CARRY_UNROLL];
#pragma unroll
    for (int i = 0; i < SSM_CARRY_UNROLL; ++i)
      if (s0 + i < S) {
        v[i] = hs[(s0 + i) * per];
        d[i] = ds[static_cast<long long>(s0 + i) * p.f.D];
      }
#pragma unroll
    for (int i = 0; i < SSM_CARRY_UNROLL; ++i)
      if (s0 + i < S) {
        hs[(s0 + i) * per] = h;
        h = fmaf(ex2_approx(d[i] * A2), h, v[i]);
      }
  }
  float g = p.dS_out ? p.dS_out[b * per + e] : 0.f;
  for (int s0 = S - 1; s0 >= 0; s0 -= SSM_CARRY_UNROLL) {
    float v[SSM_CARRY_UNROLL], d[SSM_CARRY_UNROLL];
#pragma unroll
    for (int i = 0; i < SSM_CARRY_UNROLL; ++i)
      if (s0 - i >= 0) {
        v[i] = gs[(s0 - i) * per];
        d[i] = ds[static_cast<long long>(s0 - i) * p.f.D];
      }
#pragma unroll
    for (int i = 0; i < SSM_CARRY_UNROLL; ++i)
      if (s0 - i >= 0) {
        gs[(s0 - i) * per] = g;
        g = fmaf(ex2_approx(d[i] * A2), g, v[i]);
      }
  }
  if (p.dS0) p.dS0[b * per + e] = g;
}

template <typename T, int NS>
struct SsmBwdSmem {
  using Cfg = SsmBwdCfg<NS>;
  alignas(16) float2 d[Cfg::SEG][SSM_CH];       // d, d u; then dx, sum_n w A of the tokens walked
  alignas(16) float dy[Cfg::SEG][SSM_CH];       // dy; then C . h
  alignas(16) float b[Cfg::SEG * 4 * NS];
  alignas(16) float c[Cfg::SEG * 4 * NS];
  float ck[Cfg::GROUPS][NS][SSM_THREADS];       // state before each group
  float red[SSM_THREADS / 32][Cfg::GT][8 * NS]; // a group's dB, dC, one sum per warp
  float cs[2][SSM_THREADS / (SSM_CH / (16 / int(sizeof(T))))][SSM_CH];  // dDskip, ddt_bias
};

template <typename T, int NS>
__global__ __launch_bounds__(SSM_THREADS) void ssm_bwd_main_kernel(const SsmBwdParams p) {
  using Cfg = SsmBwdCfg<NS>;
  constexpr int V = 16 / int(sizeof(T)), CPR = SSM_CH / V, GT = Cfg::GT;
  extern __shared__ __align__(16) unsigned char ssm_smem[];
  auto& sm = *reinterpret_cast<SsmBwdSmem<T, NS>*>(ssm_smem);
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, q = lane % 4;
  const SsmBlock k = ssm_block(p.f, blockIdx.x, p.f.nseg);
  const int ch = warp * 8 + lane / 4;
  const bool live = ch < k.cw;
  const long long c = k.c0 + (live ? ch : 0);
  const int len = seq_len(p.f.lens, k.b, p.f.L);
  const int t0 = k.s * Cfg::SEG, t_end = min(t0 + Cfg::SEG, len);
  const long long r = (static_cast<long long>(k.b) * p.f.nseg + k.s) * p.f.D + c;
  const int N = p.f.N;

  float dA[NS];
#pragma unroll
  for (int i = 0; i < NS; ++i) dA[i] = 0.f;
  if (t0 < t_end) {
    float A[NS], h[NS], g[NS];
    ssm_load_states<NS>(p.f.A + c * N, q, N, A);
    ssm_load_states<NS>(p.f.seg_h + r * N, q, N, h);
    ssm_load_states<NS>(p.seg_g + r * N, q, N, g);
    for (int i = tid; i < Cfg::SEG * 4 * NS; i += SSM_THREADS) sm.b[i] = sm.c[i] = 0.f;
    __syncthreads();
    ssm_stage_bc<T, NS, Cfg::SEG>(p.f, p.f.Bm, k.b, k.g, t0, t_end, sm.b);
    ssm_stage_bc<T, NS, Cfg::SEG>(p.f, p.f.Cm, k.b, k.g, t0, t_end, sm.c);
    ssm_bwd_stage<T, Cfg::SEG>(p, k, t0, t_end, sm.d, sm.dy);
    __syncthreads();
    // forward: the state before each group
#pragma unroll 1
    for (int gr = 0; gr < Cfg::GROUPS; ++gr) {
#pragma unroll
      for (int i = 0; i < NS; ++i) sm.ck[gr][i][tid] = h[i];
      if (gr + 1 < Cfg::GROUPS) {
#pragma unroll
        for (int j = 0; j < GT; ++j) {
          const float2 d = sm.d[gr * GT + j][ch];
          float bv[NS];
          lds_states<NS>(sm.b + (gr * GT + j) * 4 * NS + q * NS, bv);
#pragma unroll
          for (int i = 0; i < NS; ++i)
            h[i] = fmaf(ex2_approx(d.x * (A[i] * 1.4426950408889634f)), h[i], d.y * bv[i]);
        }
      }
    }
    // backward, last group first
#pragma unroll 1
    for (int gr = Cfg::GROUPS - 1; gr >= 0; --gr) {
      float a[GT][NS], ah[GT][NS], yv[GT], xv[GT], sv[GT];
#pragma unroll
      for (int i = 0; i < NS; ++i) h[i] = sm.ck[gr][i][tid];
#pragma unroll
      for (int j = 0; j < GT; ++j) {
        const int t = gr * GT + j;
        const float2 d = sm.d[t][ch];
        float bv[NS], cv[NS];
        lds_states<NS>(sm.b + t * 4 * NS + q * NS, bv);
        lds_states<NS>(sm.c + t * 4 * NS + q * NS, cv);
        yv[j] = 0.f;
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          a[j][i] = ex2_approx(d.x * (A[i] * 1.4426950408889634f));
          ah[j][i] = a[j][i] * h[i];
          h[i] = fmaf(d.y, bv[i], ah[j][i]);
          yv[j] = fmaf(h[i], cv[i], yv[j]);
        }
      }
#pragma unroll
      for (int j = GT - 1; j >= 0; --j) {
        const int t = gr * GT + j;
        const float2 d = sm.d[t][ch];
        const float dy = sm.dy[t][ch];
        float bv[NS], cv[NS], bc[2 * NS];
        lds_states<NS>(sm.b + t * 4 * NS + q * NS, bv);
        lds_states<NS>(sm.c + t * 4 * NS + q * NS, cv);
        xv[j] = sv[j] = 0.f;
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          g[i] = fmaf(dy, cv[i], g[i]);
          bc[i] = live ? g[i] * d.y : 0.f;
          bc[NS + i] = live ? dy * fmaf(d.y, bv[i], ah[j][i]) : 0.f;
          xv[j] = fmaf(g[i], bv[i], xv[j]);
          const float w = g[i] * ah[j][i];
          sv[j] = fmaf(w, A[i], sv[j]);
          dA[i] = fmaf(w, d.x, dA[i]);
          g[i] *= a[j][i];
        }
        // over the warp's 8 channels: lane bits 4, 3, 2 pick which sums are kept
        constexpr int C0 = 2 * NS;
        int at = 0;
        if constexpr (C0 >= 2) {
          halve_sum(bc, C0, 16, lane & 16);
          at += lane & 16 ? C0 / 2 : 0;
        }
        if constexpr (C0 >= 4) {
          halve_sum(bc, C0 / 2, 8, lane & 8);
          at += lane & 8 ? C0 / 4 : 0;
        } else {
          bc[0] += __shfl_xor_sync(0xffffffffu, bc[0], 8);
        }
        if constexpr (C0 >= 8) {
          halve_sum(bc, C0 / 4, 4, lane & 4);
          at += lane & 4 ? C0 / 8 : 0;
        } else {
          bc[0] += __shfl_xor_sync(0xffffffffu, bc[0], 4);
        }
        constexpr int KEEP = C0 >= 8 ? C0 / 8 : 1;
#pragma unroll
        for (int i = 0; i < KEEP; ++i) sm.red[warp][j][q * C0 + at + i] = bc[i];
      }
      // y, dx, sum w A: over the 4 state quarters; lane q keeps GT / 4 tokens from q GT / 4
      halve_sum(yv, GT, 2, q & 2);
      halve_sum(yv, GT / 2, 1, q & 1);
      halve_sum(xv, GT, 2, q & 2);
      halve_sum(xv, GT / 2, 1, q & 1);
      halve_sum(sv, GT, 2, q & 2);
      halve_sum(sv, GT / 2, 1, q & 1);
      __syncwarp();                              // the warp is done with the group's d and dy
#pragma unroll
      for (int i = 0; i < GT / 4; ++i) {
        const int t = gr * GT + q * (GT / 4) + i;
        sm.d[t][ch] = make_float2(xv[i], sv[i]);
        sm.dy[t][ch] = yv[i];
      }
      __syncthreads();
      for (int i = tid; i < GT * 8 * NS; i += SSM_THREADS) {
        const int j = i / (8 * NS), e = i - j * (8 * NS);
        const int qq = e / (2 * NS), f = e - qq * (2 * NS);   // quarter; dB_0.., dC_0..
        const int n = qq * NS + (f < NS ? f : f - NS), t = t0 + gr * GT + j;
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < SSM_THREADS / 32; ++w) s += sm.red[w][j][e];
        if (n < N && t < t_end) {
          const long long cb = k.g * p.f.cbg + (k.c0 - k.g * p.f.Dg) / SSM_CH;
          const long long row = (cb * p.f.B + k.b) * p.f.L + t;
          p.part_bc[row * 2 * N + (f < NS ? n : N + n)] = s;
        }
      }
      __syncthreads();                           // the sums are read before the next group's
    }
    // whole rows: du, ddt, dz, and the sums over tokens of dDskip, ddt_bias
    float sD[V], sT[V];
#pragma unroll
    for (int i = 0; i < V; ++i) sD[i] = sT[i] = 0.f;
    for (int it = tid; it < Cfg::SEG * CPR; it += SSM_THREADS) {
      const int t = it / CPR, cc = it % CPR * V;
      if (t0 + t < t_end && cc < k.cw) {
        const long long at = (static_cast<long long>(k.b) * p.f.L + t0 + t) * p.f.D + k.c0 + cc;
        VecPack<T, V> u, d, z, o, ou, od, oz;
        u.load(static_cast<const T*>(p.f.u) + at);
        d.load(static_cast<const T*>(p.f.dt) + at);
        o.load(static_cast<const T*>(p.dout) + at);
        if (p.f.z) z.load(static_cast<const T*>(p.f.z) + at);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float bias = p.f.dt_bias ? p.f.dt_bias[k.c0 + cc + i] : 0.f;
          const float skip = p.f.Dskip ? p.f.Dskip[k.c0 + cc + i] : 0.f;
          const float raw = to_f32(d.e[i]) + bias, dl = softplus_f32(raw), uf = to_f32(u.e[i]);
          const float2 xs = sm.d[t][cc + i];
          float dy = to_f32(o.e[i]);
          if (p.f.z) {
            const float zf = to_f32(z.e[i]), sg = sigmoid_f32(zf);
            const float y = fmaf(skip, uf, sm.dy[t][cc + i]);
            oz.e[i] = from_f32<T>(dy * y * (sg * fmaf(zf, 1.f - sg, 1.f)));
            dy *= zf * sg;
          }
          const float dt = fmaf(xs.x, uf, xs.y) * sigmoid_f32(raw);
          ou.e[i] = from_f32<T>(fmaf(xs.x, dl, skip * dy));
          od.e[i] = from_f32<T>(dt);
          sD[i] = fmaf(dy, uf, sD[i]);
          sT[i] += dt;
        }
        ou.store(static_cast<T*>(p.du) + at);
        od.store(static_cast<T*>(p.ddt) + at);
        if (p.f.z) oz.store(static_cast<T*>(p.dz) + at);
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      sm.cs[0][tid / CPR][tid % CPR * V + i] = sD[i];
      sm.cs[1][tid / CPR][tid % CPR * V + i] = sT[i];
    }
    __syncthreads();
    if (tid < 2 * SSM_CH) {
      const int w = tid / SSM_CH, cc = tid % SSM_CH;
      float s = 0.f;
      for (int i = 0; i < SSM_THREADS / CPR; ++i) s += sm.cs[w][i][cc];
      if (cc < k.cw)
        p.part_c[((static_cast<long long>(k.b) * p.f.nseg + k.s) * 2 + w) * p.f.D + k.c0 + cc] = s;
    }
  } else if (tid < 2 * SSM_CH && tid % SSM_CH < k.cw) {
    p.part_c[((static_cast<long long>(k.b) * p.f.nseg + k.s) * 2 + tid / SSM_CH) * p.f.D + k.c0 +
             tid % SSM_CH] = 0.f;
  }
  // this segment's dA takes the place of its entering state, which only this block reads
  if (live) ssm_store_states<NS>(p.f.seg_h + r * N, q, N, dA);
}

// dB, dC [B][L][G][N] from the channel blocks' sums; rows past a sequence's end are left.
template <typename T>
__global__ __launch_bounds__(256) void ssm_bwd_bc_kernel(const SsmBwdParams p) {
  const int N = p.f.N, G = p.f.G;
  const long long rows = static_cast<long long>(p.f.B) * p.f.L;
  const long long gid = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  const long long row = gid / (2 * N * G);
  if (row >= rows) return;
  const int e = static_cast<int>(gid - row * (2 * N * G)), g = e / (2 * N), f = e - g * (2 * N);
  const int b = static_cast<int>(row / p.f.L);
  if (p.f.lens && row - static_cast<long long>(b) * p.f.L >= seq_len(p.f.lens, b, p.f.L)) return;
  float s = 0.f;
  const float* src = p.part_bc + (static_cast<long long>(g) * p.f.cbg * rows + row) * 2 * N + f;
#pragma unroll 8
  for (int i = 0; i < p.f.cbg; ++i) s += src[i * rows * 2 * N];
  T* dst = static_cast<T*>(f < N ? p.dB : p.dC);
  dst[(row * G + g) * N + (f < N ? f : f - N)] = from_f32<T>(s);
}

// dA [D][N], dDskip [D], ddt_bias [D]: sums over sequences and segments in a fixed order, 32 columns
// x 8 lanes of segments per block.
__global__ __launch_bounds__(256) void ssm_bwd_param_kernel(const SsmBwdParams p) {
  __shared__ float red[8][33];
  const int x = threadIdx.x % 32, y = threadIdx.x / 32;
  const long long nA = static_cast<long long>(p.f.D) * p.f.N, nC = 2LL * p.f.D;
  const long long blocksA = (nA + 31) / 32;
  const bool isA = blockIdx.x < blocksA;
  const long long i = (isA ? blockIdx.x : blockIdx.x - blocksA) * 32LL + x;
  const long long n = isA ? nA : nC;
  const float* src = isA ? p.f.seg_h : p.part_c;
  float a = 0.f;
  if (i < n) {
    const long long R = static_cast<long long>(p.f.B) * p.f.nseg;
#pragma unroll 4
    for (long long r = y; r < R; r += 8) a += src[r * n + i];
  }
  red[y][x] = a;
  __syncthreads();
  if (y == 0 && i < n) {
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) s += red[j][x];
    if (isA)
      p.dA[i] = s;
    else if (i < p.f.D) {
      if (p.dD) p.dD[i] = s;
    } else if (p.ddt_bias) {
      p.ddt_bias[i - p.f.D] = s;
    }
  }
}

}  // namespace kta

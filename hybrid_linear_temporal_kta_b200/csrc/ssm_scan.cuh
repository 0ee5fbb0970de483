// ssm_scan.cuh -- selective state-space scan. Per sequence, channel c and state n, with
// d_t = softplus(dt_t + dt_bias):
//     h_t = exp(d_t A) h_{t-1} + d_t u_t B_t,    y_t = (C_t . h_t + Dskip u_t) silu(z_t),
// B and C shared by the channels of a group. States, gates and sums are fp32.
//
// Bound by the exponential unit: one exponential per (token, channel, state), a warp's 32 in 8 cycles
// of its scheduler, against 8 bytes per (token, channel) in bf16.
#pragma once
#include <float.h>

#include <type_traits>

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

// Warp `wid` of a grid over (sequence, segment, group, channel block of CH).
__device__ __forceinline__ SsmBlock ssm_block(const SsmParams& p, long long wid, int nseg, int cbg, int CH) {
  SsmBlock k;
  const int ncb = p.G * cbg;
  const long long rest = wid / ncb;
  const int cb = static_cast<int>(wid - rest * ncb);
  k.b = static_cast<int>(rest / nseg);
  k.s = static_cast<int>(rest - static_cast<long long>(k.b) * nseg);
  k.g = cb / cbg;
  const int o = (cb - k.g * cbg) * CH;
  k.c0 = k.g * p.Dg + o;
  k.cw = min(CH, p.Dg - o);
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

// A = -inf as the lowest finite value (a NaN stays one): every step d > 0 forgets, and where d = 0, as in the
// rows that pad a tile, the state stays.
__device__ __forceinline__ float ssm_finite(float x) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(-FLT_MAX));
  return y;
}
__device__ __forceinline__ float ssm_log2(float A) { return ssm_finite(A * 1.4426950408889634f); }

// Starts the copies of TT rows of B (and of C, if C) to their raw tile.
template <typename T, int NP, int TT, bool C, int BYTES>
__device__ __forceinline__ void ssm_rows_fetch_as(const SsmParams& p, T (*rb)[NP], T (*rc)[NP], long long row0, int g,
                                                  int t0, int t_end, int lane) {
  constexpr int V = BYTES / int(sizeof(T)) > 0 ? BYTES / int(sizeof(T)) : 1, NV = (NP + V - 1) / V;
#pragma unroll
  for (int m = 0; m < (TT * NV + 31) / 32; ++m) {
    const int it = lane + m * 32, t = it / NV, n = it % NV * V;
    if (it < TT * NV && n < p.N) {
      const bool on = t0 + t < t_end;
      const long long at = on ? ((row0 + t0 + t) * p.G + g) * p.N + n : 0;
      piece_async<BYTES>(&rb[t][n], static_cast<const T*>(p.Bm) + at, on);
      if (C) piece_async<BYTES>(&rc[t][n], static_cast<const T*>(p.Cm) + at, on);
    }
  }
}
template <typename T, int NP, int TT, bool C>
__device__ __forceinline__ void ssm_rows_fetch(const SsmParams& p, T (*rb)[NP], T (*rc)[NP], long long row0, int g,
                                               int t0, int t_end, int lane) {
  if (p.bc_bytes == 16)
    ssm_rows_fetch_as<T, NP, TT, C, 16>(p, rb, rc, row0, g, t0, t_end, lane);
  else if (p.bc_bytes == 8)
    ssm_rows_fetch_as<T, NP, TT, C, 8>(p, rb, rc, row0, g, t0, t_end, lane);
  else if (p.bc_bytes == 4)
    ssm_rows_fetch_as<T, NP, TT, C, 4>(p, rb, rc, row0, g, t0, t_end, lane);
}

// The raw rows (or, for odd rows of 2-byte elements, rows from memory) as fp32; columns from N on are
// left as they are (zeros, set once).
template <typename T, int NP, int TT, bool C>
__device__ __forceinline__ void ssm_rows_f32(const SsmParams& p, const T (*rb)[NP], const T (*rc)[NP],
                                             float (*bc)[C ? 2 : 1][NP], long long row0, int g, int t0, int t_end,
                                             int lane) {
  if (p.bc_bytes) {
    constexpr int NQ = NP / 4;
#pragma unroll
    for (int m = 0; m < (TT * NQ + 31) / 32; ++m) {
      const int it = lane + m * 32, t = it / NQ, n = it % NQ * 4;
      if (it < TT * NQ && n < p.N) {
#pragma unroll
        for (int w = 0; w < (C ? 2 : 1); ++w) {
          VecPack<T, 4> x;
          x.load(w ? &rc[t][n] : &rb[t][n]);
          float4 f = make_float4(to_f32(x.e[0]), to_f32(x.e[1]), to_f32(x.e[2]), to_f32(x.e[3]));
          if (n + 4 > p.N) {                             // the row ends inside the quad
            f.y = n + 1 < p.N ? f.y : 0.f;
            f.z = n + 2 < p.N ? f.z : 0.f;
            f.w = 0.f;
          }
          *reinterpret_cast<float4*>(&bc[t][w][n]) = f;
        }
      }
    }
  } else {
    for (int it = lane; it < TT * p.N; it += 32) {
      const int t = it / p.N, n = it - t * p.N;
      const bool on = t0 + t < t_end;
      const long long at = on ? ((row0 + t0 + t) * p.G + g) * p.N + n : 0;
      bc[t][0][n] = on ? to_f32(static_cast<const T*>(p.Bm)[at]) : 0.f;
      if (C) bc[t][C ? 1 : 0][n] = on ? to_f32(static_cast<const T*>(p.Cm)[at]) : 0.f;
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
  const SsmBlock k = ssm_block(p, wid, nseg, p.cbg, SSM_CH);
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
    ssm_rows_fetch<T, NP, SSM_TT, OUT>(p, r.b, r.c, row0, k.g, t0, t_end, lane);
    piece_commit();
  };
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) fetch(t_begin + s * SSM_TT, s);

  float2 A2[NP / 2], h[NP / 2];                          // pairs of states; zero past N
  const float* Arow = p.A + static_cast<long long>(c) * p.N;
#pragma unroll
  for (int i = 0; i < NP / 2; ++i) {
    A2[i].x = 2 * i < p.N ? ssm_log2(Arow[2 * i]) : 0.f;
    A2[i].y = 2 * i + 1 < p.N ? ssm_log2(Arow[2 * i + 1]) : 0.f;
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
    ssm_rows_f32<T, NP, SSM_TT, OUT>(p, r.b, r.c, sm.bc, row0, k.g, t0, t_end, lane);
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
  piece_wait<0>();
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

// 2^x h + v; a state still at zero stays there. GROW: where a segment's growth alone overflows (A > 0), 2^126 of
// it goes to h first (exactly), so that 2^x h is formed whenever h and it are normal numbers.
template <bool GROW>
__device__ __forceinline__ float ssm_carry(float x, float h, float v) {
  const bool up = GROW && x >= 128.f;
  const float e = ex2_approx(up ? x - 126.f : x);
  return h == 0.f ? v : fmaf(e, up ? h * 0x1p126f : h, v);
}

// Up to SSM_CARRY_UNROLL segments in a row, `vstep` elements apart: their end states from zero (v, loaded from vs)
// become the states that enter them; d: their sums of d.
__device__ __forceinline__ void ssm_carry_batch(float* vs, long long vstep, const float (&v)[SSM_CARRY_UNROLL],
                                                const float (&d)[SSM_CARRY_UNROLL], float A2, int left, float& h) {
  bool grow = false;                                     // uncommon, and one test for all
#pragma unroll
  for (int i = 0; i < SSM_CARRY_UNROLL; ++i) grow |= d[i] * A2 >= 128.f;
  auto walk = [&](auto up) {
#pragma unroll
    for (int i = 0; i < SSM_CARRY_UNROLL; ++i)
      if (i < left) {
        vs[i * vstep] = h;
        h = ssm_carry<decltype(up)::value>(d[i] * A2, h, v[i]);
      }
  };
  if (grow)
    walk(std::true_type());
  else
    walk(std::false_type());
}

__global__ __launch_bounds__(256) void ssm_fwd_carry_kernel(const SsmParams p, int NP) {
  const long long per = static_cast<long long>(p.D) * NP;
  const long long gid = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (gid >= per * p.B) return;
  const int b = static_cast<int>(gid / per);
  const int n = static_cast<int>(gid % per / p.D), c = static_cast<int>(gid % p.D);
  const long long e = static_cast<long long>(c) * p.N + n;
  const bool on = n < p.N;
  const float A2 = on ? ssm_log2(p.A[e]) : 0.f;
  float h = on && p.S0 ? p.S0[static_cast<long long>(b) * p.D * p.N + e] : 0.f;
  float* hs = p.seg_h + (static_cast<long long>(b) * p.nseg * NP + n) * p.D + c;
  const float* ds = p.seg_d + static_cast<long long>(b) * p.nseg * p.D + c;
  for (int s0 = 0; s0 < p.nseg; s0 += SSM_CARRY_UNROLL) {
    float v[SSM_CARRY_UNROLL], d[SSM_CARRY_UNROLL];
#pragma unroll
    for (int i = 0; i < SSM_CARRY_UNROLL; ++i)
      if (s0 + i < p.nseg - 1) {                         // (what follows the last segment is not wanted)
        v[i] = hs[(s0 + i) * per];
        d[i] = ds[static_cast<long long>(s0 + i) * p.D];
      } else {
        v[i] = d[i] = 0.f;
      }
    ssm_carry_batch(hs + s0 * per, per, v, d, A2, p.nseg - s0, h);
  }
}

// One token: memory-bound, the state read and written once (8 bytes per state against 8 per channel
// of u, dt, z and y in bf16). A lane owns a state quarter of one channel (16 bytes for N = 16) of
// SSM_STEP_B sequences, whose loads are in flight together and share its row of A: 64 x 4,096 x 16
// states in 11.2 us with two; one takes 1.1 times as long, four 1.4 times (fewer warps).
constexpr int SSM_STEP_B = 2;

template <typename T, int NS>
__global__ __launch_bounds__(SSM_THREADS) void ssm_step_kernel(const SsmParams p) {
  const int q = threadIdx.x % 4;
  const int c = (blockIdx.x * SSM_THREADS + threadIdx.x) / 4;   // D % 8 == 0: a warp's 8 channels all live or none
  const int b0 = blockIdx.y * SSM_STEP_B;
  if (c >= p.D) return;
  const int nb = min(SSM_STEP_B, p.B - b0), g = c / p.Dg;
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
  for (int i = 0; i < NS; ++i) A2[i] = ssm_log2(A2[i]);
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
// Launches over segments of SEG tokens, all segments at once:
//  1. ssm_bwd_local: each segment's end state from zero, its share of the adjoint that leaves it at
//     its start (P_t the running product of decays: sum_t P_t dy_t C_t), and its sum of d;
//  2. ssm_bwd_carry: folds both along the sequence: the state that enters each segment and the
//     adjoint that enters it from behind (and dS0);
//  3. ssm_bwd_main: a forward walk keeps the state before every GT tokens in shared memory; then,
//     last group first, the group's states are formed again in registers and the adjoint walks back:
//     three exponentials per (token, channel, state) in all, and no state but the segments' in memory;
//  4. ssm_bwd_sums: sums over channel blocks, and over segments, in a fixed order.

template <int NP> struct SsmBwdCfg {
  static constexpr int NH = NP == 32 ? 8 : NP >= 8 ? 4 : 2;   // states of one lane, for each of two channels
  static constexpr int SPL = NP / NH;                // lanes that share a channel's states (2 or 4)
  static constexpr int CH = 64 / SPL;                // channels of a warp
  static constexpr int BCH = CH * SSM_THREADS / 32;  // channels of a block
  static constexpr int GT = 4;                       // tokens whose decays and states fit in registers
  static constexpr int GROUPS = 8;
  static constexpr int SEG = GT * GROUPS;
  // sums over the warp's channel pairs: NH values are halved log2(NH) times; where a lane bit is left,
  // it tells dB from dC
  static constexpr bool SPLIT = 32 / SPL > NH;
};
constexpr int SSM_BWD_SEG = 32;

struct SsmBwdParams {
  SsmParams f;                   // inputs; nseg / seg of the backward; seg_h [B][nseg][NP][D]
  const void *dout;
  const float* dS_out;
  void *du, *ddt, *dz, *dB, *dC;
  float *dA, *dD, *ddt_bias, *dS0;
  int cbg;                       // channel blocks per group of the main pass (f.cbg: of the local one)
  float* seg_g;                  // [B][nseg][NP][D]: adjoint entering each segment from behind
  float* part_bc;                // [G * cbg][B * L][2 N]
  float* part_c;                 // [B][nseg][2][D]: dDskip, ddt_bias
};

// Shared memory of one warp of the local pass: as in the forward, with dout and C beside.
template <typename T, int NP>
struct SsmLocalSmem {
  struct Raw {
    alignas(16) T u[SSM_TT][SSM_CH];
    alignas(16) T d[SSM_TT][SSM_CH];
    alignas(16) T z[SSM_TT][SSM_CH];
    alignas(16) T o[SSM_TT][SSM_CH];
    alignas(16) T b[SSM_TT][NP];
    alignas(16) T c[SSM_TT][NP];
  };
  Raw raw[2];
  alignas(16) float bc[SSM_TT][2][NP];
  alignas(16) float2 dd[SSM_TT][SSM_CH];   // d, d u
  alignas(16) float dy[SSM_TT][SSM_CH];
};

// One warp = 32 channels of a group over one segment, a lane all states of one channel.
template <typename T, int NP>
__global__ __launch_bounds__(SSM_THREADS, NP > 16 ? 2 : 4) void ssm_bwd_local_kernel(const SsmBwdParams p) {
  using Smem = SsmLocalSmem<T, NP>;
  constexpr int V = 16 / int(sizeof(T)), CPR = SSM_CH / V;
  extern __shared__ __align__(16) unsigned char ssm_smem[];
  Smem& sm = reinterpret_cast<Smem*>(ssm_smem)[threadIdx.x / 32];
  chain_start();
  const int lane = threadIdx.x % 32;
  const long long wid = blockIdx.x * static_cast<long long>(SSM_THREADS / 32) + threadIdx.x / 32;
  if (wid >= static_cast<long long>(p.f.B) * p.f.nseg * p.f.G * p.f.cbg) return;
  const SsmBlock k = ssm_block(p.f, wid, p.f.nseg, p.f.cbg, SSM_CH);
  const bool live = lane < k.cw;
  const int c = k.c0 + (live ? lane : 0);
  const int len = seq_len(p.f.lens, k.b, p.f.L);
  const int t_begin = k.s * p.f.seg, t_end = min(t_begin + p.f.seg, len);
  const long long row0 = static_cast<long long>(k.b) * p.f.L;

  auto fetch = [&](int t0, int stage) {
    typename Smem::Raw& r = sm.raw[stage];
#pragma unroll
    for (int m = 0; m < SSM_TT * CPR / 32; ++m) {
      const int it = lane + m * 32, t = it / CPR, cc = it % CPR * V;
      const bool on = t0 + t < t_end && cc < k.cw;
      const long long at = on ? (row0 + t0 + t) * p.f.D + k.c0 + cc : 0;
      piece_async<16>(&r.u[t][cc], static_cast<const T*>(p.f.u) + at, on);
      piece_async<16>(&r.d[t][cc], static_cast<const T*>(p.f.dt) + at, on);
      piece_async<16>(&r.o[t][cc], static_cast<const T*>(p.dout) + at, on);
      if (p.f.z) piece_async<16>(&r.z[t][cc], static_cast<const T*>(p.f.z) + at, on);
    }
    ssm_rows_fetch<T, NP, SSM_TT, true>(p.f, r.b, r.c, row0, k.g, t0, t_end, lane);
    piece_commit();
  };
  fetch(t_begin, 0);

  float2 A2[NP / 2], h[NP / 2], g[NP / 2], P[NP / 2];
  const float* Arow = p.f.A + static_cast<long long>(c) * p.f.N;
#pragma unroll
  for (int i = 0; i < NP / 2; ++i) {
    A2[i].x = 2 * i < p.f.N ? ssm_log2(Arow[2 * i]) : 0.f;
    A2[i].y = 2 * i + 1 < p.f.N ? ssm_log2(Arow[2 * i + 1]) : 0.f;
    h[i] = g[i] = make_float2(0.f, 0.f);
    P[i] = make_float2(1.f, 1.f);
  }
  for (int i = lane; i < SSM_TT * 2 * NP; i += 32) (&sm.bc[0][0][0])[i] = 0.f;
  const float bias = p.f.dt_bias ? p.f.dt_bias[c] : 0.f;
  float sum_d = 0.f;
  int stage = 0;
  for (int t0 = t_begin; t0 < t_end; t0 += SSM_TT, stage ^= 1) {
    piece_wait<0>();
    __syncwarp();                                        // the pieces are there; dd, dy, bc are free
    fetch(t0 + SSM_TT, stage ^ 1);
    typename Smem::Raw& r = sm.raw[stage];
#pragma unroll
    for (int j = 0; j < SSM_TT; ++j) {
      float d = softplus_f32(to_f32(r.d[j][lane]) + bias);
      d = t0 + j < t_end ? d : 0.f;
      sum_d += d;
      float dy = to_f32(r.o[j][lane]);
      if (p.f.z) {
        const float z = to_f32(r.z[j][lane]);
        dy *= z * sigmoid_f32(z);
      }
      sm.dd[j][lane] = make_float2(d, d * to_f32(r.u[j][lane]));
      sm.dy[j][lane] = dy;                               // (past the end 0: dout is)
    }
    ssm_rows_f32<T, NP, SSM_TT, true>(p.f, r.b, r.c, sm.bc, row0, k.g, t0, t_end, lane);
    __syncwarp();
#pragma unroll 4
    for (int j = 0; j < SSM_TT; ++j) {
      const float2 dd = sm.dd[j][lane];
      const float dy = sm.dy[j][lane];
      const uint64_t d2 = f32x2_pack(dd.x, dd.x), du2 = f32x2_pack(dd.y, dd.y), dy2 = f32x2_pack(dy, dy);
#pragma unroll
      for (int i = 0; i < NP / 2; i += 2) {
        const ulonglong2 b4 = *reinterpret_cast<const ulonglong2*>(&sm.bc[j][0][2 * i]);
        const ulonglong2 c4 = *reinterpret_cast<const ulonglong2*>(&sm.bc[j][1][2 * i]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float2 x = f32x2_unpack(fmul2(d2, f32x2_pack(A2[i + e])));
          const uint64_t a = f32x2_pack(ex2_approx(x.x), ex2_approx(x.y));
          h[i + e] = f32x2_unpack(ffma2(a, f32x2_pack(h[i + e]), fmul2(du2, e ? b4.y : b4.x)));
          const uint64_t q = fmul2(a, f32x2_pack(P[i + e]));
          P[i + e] = f32x2_unpack(q);
          g[i + e] = f32x2_unpack(ffma2(q, fmul2(dy2, e ? c4.y : c4.x), f32x2_pack(g[i + e])));
        }
      }
    }
  }
  piece_wait<0>();
  if (!live) return;
  const long long r = static_cast<long long>(k.b) * p.f.nseg + k.s;
  float* sh = p.f.seg_h + r * NP * p.f.D + c;
  float* sg = p.seg_g + r * NP * p.f.D + c;
#pragma unroll
  for (int i = 0; i < NP / 2; ++i) {
    const long long a = static_cast<long long>(2 * i) * p.f.D, b = a + p.f.D;
    sh[a] = h[i].x;
    sh[b] = h[i].y;
    sg[a] = g[i].x;
    sg[b] = g[i].y;
  }
  p.f.seg_d[r * p.f.D + c] = sum_d;
}

// One thread per (sequence, state, channel), in place: local end states become entering states
// (blockIdx.y 0), local adjoints the adjoints entering from behind (1).
__global__ __launch_bounds__(256) void ssm_bwd_carry_kernel(const SsmBwdParams p, int NP) {
  chain_start();
  chain_wait();
  const long long per = static_cast<long long>(p.f.D) * NP;
  const long long gid = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (gid >= per * p.f.B) return;
  const int b = static_cast<int>(gid / per);
  const int n = static_cast<int>(gid % per / p.f.D), c = static_cast<int>(gid % p.f.D);
  const bool on = n < p.f.N, back = blockIdx.y;
  const long long e = static_cast<long long>(c) * p.f.N + n, eb = static_cast<long long>(b) * p.f.D * p.f.N + e;
  const float A2 = on ? ssm_log2(p.f.A[e]) : 0.f;
  const int S = p.f.nseg;
  const long long first = back ? S - 1 : 0, step = back ? -1 : 1;
  float* vs = (back ? p.seg_g : p.f.seg_h) + (static_cast<long long>(b) * S + first) * per + gid % per;
  const float* ds = p.f.seg_d + (static_cast<long long>(b) * S + first) * p.f.D + c;
  const float* in = back ? p.dS_out : p.f.S0;
  float h = on && in ? in[eb] : 0.f;
  for (int s0 = 0; s0 < S; s0 += SSM_CARRY_UNROLL) {
    float v[SSM_CARRY_UNROLL], d[SSM_CARRY_UNROLL];
#pragma unroll
    for (int i = 0; i < SSM_CARRY_UNROLL; ++i)
      if (s0 + i < S) {
        v[i] = vs[step * (s0 + i) * per];
        d[i] = ds[step * (s0 + i) * p.f.D];
      } else {
        v[i] = d[i] = 0.f;
      }
    ssm_carry_batch(vs + step * s0 * per, step * per, v, d, A2, S - s0, h);
  }
  if (back && on && p.dS0) p.dS0[eb] = h;
}

// Shared memory of a block of the main pass: four warps' own parts, and the rows of B and C.
template <typename T, int NP>
struct SsmMainSmem {
  using Cfg = SsmBwdCfg<NP>;
  struct Raw {
    alignas(16) T d[Cfg::SEG][Cfg::CH];
    alignas(16) T z[Cfg::SEG][Cfg::CH];
    alignas(16) T o[Cfg::SEG][Cfg::CH];
  };
  struct Keep {
    alignas(16) float4 h[Cfg::GROUPS - 1][Cfg::NH / 2][32];   // state before groups 1 .., by lane
  };
  struct Warp {
    union {                                          // the raw rows are gone before a state is kept
      Raw raw;
      Keep ck;
    };
    alignas(16) T u[Cfg::SEG][Cfg::CH];
    alignas(16) float d[Cfg::SEG][Cfg::CH];
    alignas(16) float dy[Cfg::SEG][Cfg::CH];
  };
  Warp w[SSM_THREADS / 32];
  union {
    struct {
      alignas(16) T b[Cfg::SEG][NP];
      alignas(16) T c[Cfg::SEG][NP];
    } raw;
    alignas(16) float red[2][SSM_THREADS / 32][Cfg::GT][2 * NP];   // warps' sums of dB and dC of two groups
  };
  alignas(16) float bc[Cfg::SEG][2][NP];
};

__device__ __forceinline__ float2 ssm_pair(const float* p) { return *reinterpret_cast<const float2*>(p); }
__device__ __forceinline__ float2 ssm_pair(const __nv_bfloat16* p) {
  const uint32_t x = *reinterpret_cast<const uint32_t*>(p);
  return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}

// H2 packed pairs of neighbouring states.
template <int H2>
__device__ __forceinline__ void ssm_lds_pairs(const float* s, uint64_t (&v)[H2]) {
  if constexpr (H2 % 2 == 0) {
#pragma unroll
    for (int i = 0; i < H2 / 2; ++i) {
      const ulonglong2 x = reinterpret_cast<const ulonglong2*>(s)[i];
      v[2 * i] = x.x;
      v[2 * i + 1] = x.y;
    }
  } else {
    v[0] = *reinterpret_cast<const unsigned long long*>(s);
  }
}

// CNT values summed over the lanes of mask bits [lowest, 16]: halved from mask 16 down while more than
// one is left, then added. The kept value's index comes back in `at`.
template <int CNT>
__device__ __forceinline__ float ssm_sum_lanes(float (&v)[CNT], int lane, int lowest, int& at) {
  int n = CNT;
  at = 0;
#pragma unroll
  for (int mask = 16; mask >= 1; mask /= 2) {
    if (mask >= lowest) {
      if (n > 1) {
        halve_sum(v, n, mask, lane & mask);
        n /= 2;
        at += lane & mask ? n : 0;
      } else {
        v[0] += __shfl_xor_sync(0xffffffffu, v[0], mask);
      }
    }
  }
  return v[0];
}

// One block = one segment x BCH channels of a group. A lane holds NH states of two neighbouring channels,
// SPL lanes a channel pair: two channels to a lane halve the exchanges that sum dB and dC over channels,
// and 2 x NH states x 4 tokens of decays and decayed states stay in registers.
template <typename T, int NP>
__global__ __launch_bounds__(SSM_THREADS, NP > 16 ? 2 : 3) void ssm_bwd_main_kernel(const SsmBwdParams p) {
  using Cfg = SsmBwdCfg<NP>;
  using Smem = SsmMainSmem<T, NP>;
  constexpr int NH = Cfg::NH, H2 = NH / 2, SPL = Cfg::SPL, CH = Cfg::CH, GT = Cfg::GT, SEG = Cfg::SEG,
                V = 16 / int(sizeof(T)), CPR = CH / V, FT = GT / (SPL / 2);
  static_assert(SEG == SSM_BWD_SEG, "the plan cuts segments of this length");
  static_assert(SPL == 2 || SPL == 4, "two or four lanes share a channel pair");
  extern __shared__ __align__(16) unsigned char ssm_smem[];
  Smem& sb = *reinterpret_cast<Smem*>(ssm_smem);
  chain_start();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, q = lane % SPL, cp = lane / SPL, N = p.f.N;
  typename Smem::Warp& sm = sb.w[warp];
  const SsmBlock k = ssm_block(p.f, blockIdx.x, p.f.nseg, p.cbg, Cfg::BCH);
  const int wc = warp * CH, lc = 2 * cp;               // the warp's first channel in the block, the lane's in the warp
  const bool live = wc + lc < k.cw;                    // (a group's last block may leave whole warps idle)
  const int fc = lc + q % 2;                           // the channel whose rows this lane finishes
  const int c = k.c0 + (live ? wc + lc : 0), cf = k.c0 + (live ? wc + fc : 0);
  const int len = seq_len(p.f.lens, k.b, p.f.L);
  const int t0 = k.s * SEG, t_end = min(t0 + SEG, len);
  const long long row0 = static_cast<long long>(k.b) * p.f.L;
  const long long seg = static_cast<long long>(k.b) * p.f.nseg + k.s;
  float* seg_h = p.f.seg_h + (seg * NP + q * NH) * p.f.D + c;
  float2 dA[2][H2];                                    // [channel][pair of states]
  float sD = 0.f, sT = 0.f;
#pragma unroll
  for (int e = 0; e < 2; ++e)
#pragma unroll
    for (int i = 0; i < H2; ++i) dA[e][i] = make_float2(0.f, 0.f);

  if (t0 < t_end) {
    // raw rows of the segment
#pragma unroll
    for (int m = 0; m < SEG * CPR / 32; ++m) {
      const int it = lane + m * 32, t = it / CPR, cc = it % CPR * V;
      const bool on = t0 + t < t_end && wc + cc < k.cw;
      const long long at = on ? (row0 + t0 + t) * p.f.D + k.c0 + wc + cc : 0;
      piece_async<16>(&sm.u[t][cc], static_cast<const T*>(p.f.u) + at, on);
      piece_async<16>(&sm.raw.d[t][cc], static_cast<const T*>(p.f.dt) + at, on);
      piece_async<16>(&sm.raw.o[t][cc], static_cast<const T*>(p.dout) + at, on);
      if (p.f.z) piece_async<16>(&sm.raw.z[t][cc], static_cast<const T*>(p.f.z) + at, on);
    }
    if (warp == 0) ssm_rows_fetch<T, NP, SEG, true>(p.f, sb.raw.b, sb.raw.c, row0, k.g, t0, t_end, lane);
    piece_commit();
    for (int i = threadIdx.x; i < SEG * 2 * NP; i += SSM_THREADS) (&sb.bc[0][0][0])[i] = 0.f;

    // a lane without a channel works on zeros
    float2 A[2][H2], g[2][H2], h[2][H2];
    const float* sg = p.seg_g + (seg * NP + q * NH) * p.f.D + c;
    auto load_pairs = [&](const float* src, float2 (&v)[2][H2]) {
#pragma unroll
      for (int i = 0; i < H2; ++i) {
        const float2 z2 = make_float2(0.f, 0.f);
        const float2 a = live ? ssm_pair(src + static_cast<long long>(2 * i) * p.f.D) : z2;
        const float2 b = live ? ssm_pair(src + static_cast<long long>(2 * i + 1) * p.f.D) : z2;
        v[0][i] = make_float2(a.x, b.x);
        v[1][i] = make_float2(a.y, b.y);
      }
    };
#pragma unroll
    for (int i = 0; i < H2; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int n = q * NH + 2 * i;
        const float* Arow = p.f.A + static_cast<long long>(c + e) * N;
        A[e][i].x = live && n < N ? Arow[n] : 0.f;
        A[e][i].y = live && n + 1 < N ? Arow[n + 1] : 0.f;
      }
    const float fbias = p.f.dt_bias ? p.f.dt_bias[cf] : 0.f, skip = p.f.Dskip ? p.f.Dskip[cf] : 0.f;
    chain_wait();
    load_pairs(seg_h, h);
    load_pairs(sg, g);
    piece_wait<0>();
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 2; ++e)                        // (here the loads of A are in without a wait of their own)
#pragma unroll
      for (int i = 0; i < H2; ++i) A[e][i] = make_float2(ssm_finite(A[e][i].x), ssm_finite(A[e][i].y));
    {
      const int cc = lane % CH;                        // a lane's items have one channel
      const bool con = wc + cc < k.cw;
      const float bias = p.f.dt_bias && con ? p.f.dt_bias[k.c0 + wc + cc] : 0.f;
#pragma unroll 4
      for (int m = 0; m < SEG * CH / 32; ++m) {
        const int t = (lane + m * 32) / CH;
        const bool on = t0 + t < t_end && con;
        const float d = softplus_f32(to_f32(sm.raw.d[t][cc]) + bias);
        float dy = to_f32(sm.raw.o[t][cc]);
        if (p.f.z) {
          const float z = to_f32(sm.raw.z[t][cc]);
          dy *= z * sigmoid_f32(z);
        }
        sm.d[t][cc] = on ? d : 0.f;                    // past the end: the state and the adjoint stay
        sm.dy[t][cc] = on ? dy : 0.f;
      }
    }
    if (warp == 0) ssm_rows_f32<T, NP, SEG, true>(p.f, sb.raw.b, sb.raw.c, sb.bc, row0, k.g, t0, t_end, lane);
    __syncthreads();                                   // the raw rows are used up

    const int last = (t_end - t0 - 1) / GT;            // groups behind this one leave all as it is
    // forward: the state before each group
#pragma unroll 1
    for (int gr = 0; gr < last; ++gr) {
#pragma unroll
      for (int j = 0; j < GT; ++j) {
        const int t = gr * GT + j;
        const float2 d = ssm_pair(&sm.d[t][lc]), u = ssm_pair(&sm.u[t][lc]);
        uint64_t b2[H2];
        ssm_lds_pairs<H2>(&sb.bc[t][0][q * NH], b2);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float de = e ? d.y : d.x, due = de * (e ? u.y : u.x), dl = de * 1.4426950408889634f;
          const uint64_t d2 = f32x2_pack(dl, dl), du2 = f32x2_pack(due, due);
#pragma unroll
          for (int i = 0; i < H2; ++i) {
            const float2 x = f32x2_unpack(fmul2(d2, f32x2_pack(A[e][i])));
            const uint64_t a = f32x2_pack(ex2_approx(x.x), ex2_approx(x.y));
            h[e][i] = f32x2_unpack(ffma2(a, f32x2_pack(h[e][i]), fmul2(du2, b2[i])));
          }
        }
      }
#pragma unroll
      for (int i = 0; i < H2; ++i) sm.ck.h[gr][i][lane] = make_float4(h[0][i].x, h[0][i].y, h[1][i].x, h[1][i].y);
    }
    // where dB and dC of this lane's share go, and where the block's sums go
    int at = 0;
    int buf = 0;
    const long long cb = static_cast<long long>(k.g) * p.cbg + (k.c0 - k.g * p.f.Dg) / Cfg::BCH;
    float* part = p.part_bc + ((cb * p.f.B + k.b) * p.f.L + t0) * 2 * N;
    // backward, last group first
#pragma unroll 1
    for (int gr = last; gr >= 0; --gr, buf ^= 1) {
      // what finishing the group's rows reads again
      const int ft = gr * GT + (SPL > 2 ? q / 2 * FT : 0);   // the first row this lane finishes
      const long long fo = (row0 + t0 + ft) * p.f.D + cf;
      T rd[FT], ro[FT], rz[FT];
#pragma unroll
      for (int j = 0; j < FT; ++j)
        if (live && t0 + ft + j < t_end) {
          rd[j] = static_cast<const T*>(p.f.dt)[fo + j * static_cast<long long>(p.f.D)];
          ro[j] = static_cast<const T*>(p.dout)[fo + j * static_cast<long long>(p.f.D)];
          if (p.f.z) rz[j] = static_cast<const T*>(p.f.z)[fo + j * static_cast<long long>(p.f.D)];
        }
      if (gr > 0) {
#pragma unroll
        for (int i = 0; i < H2; ++i) {
          const float4 v = sm.ck.h[gr - 1][i][lane];
          h[0][i] = make_float2(v.x, v.y);
          h[1][i] = make_float2(v.z, v.w);
        }
      } else {
        load_pairs(seg_h, h);
      }
      uint64_t a[GT][2][H2], ah[GT][2][H2];
      float yv[GT][2], xv[GT][2], sv[GT][2], vc[GT];
#pragma unroll
      for (int j = 0; j < GT; ++j) {
        const int t = gr * GT + j;
        const float2 d = ssm_pair(&sm.d[t][lc]), u = ssm_pair(&sm.u[t][lc]), dy = ssm_pair(&sm.dy[t][lc]);
        uint64_t b2[H2], c2[H2], qc[H2];
        ssm_lds_pairs<H2>(&sb.bc[t][0][q * NH], b2);
        ssm_lds_pairs<H2>(&sb.bc[t][1][q * NH], c2);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float de = e ? d.y : d.x, due = de * (e ? u.y : u.x), dl = de * 1.4426950408889634f;
          const float dye = e ? dy.y : dy.x;
          const uint64_t d2 = f32x2_pack(dl, dl), du2 = f32x2_pack(due, due), dy2 = f32x2_pack(dye, dye);
          uint64_t y2 = 0;
#pragma unroll
          for (int i = 0; i < H2; ++i) {
            const float2 x = f32x2_unpack(fmul2(d2, f32x2_pack(A[e][i])));
            a[j][e][i] = f32x2_pack(ex2_approx(x.x), ex2_approx(x.y));
            ah[j][e][i] = fmul2(a[j][e][i], f32x2_pack(h[e][i]));
            const uint64_t hn = ffma2(du2, b2[i], ah[j][e][i]);
            h[e][i] = f32x2_unpack(hn);
            y2 = i ? ffma2(hn, c2[i], y2) : fmul2(hn, c2[i]);
            qc[i] = e ? ffma2(dy2, hn, qc[i]) : fmul2(dy2, hn);
          }
          const float2 y = f32x2_unpack(y2);
          yv[j][e] = y.x + y.y;
        }
        float cs[NH];
#pragma unroll
        for (int i = 0; i < H2; ++i) f32x2_unpack(qc[i], cs[2 * i], cs[2 * i + 1]);
        vc[j] = ssm_sum_lanes<NH>(cs, lane, Cfg::SPLIT ? 2 * SPL : SPL, at);
      }
#pragma unroll
      for (int j = GT - 1; j >= 0; --j) {
        const int t = gr * GT + j;
        const float2 d = ssm_pair(&sm.d[t][lc]), u = ssm_pair(&sm.u[t][lc]), dy = ssm_pair(&sm.dy[t][lc]);
        uint64_t b2[H2], c2[H2], qb[H2];
        ssm_lds_pairs<H2>(&sb.bc[t][0][q * NH], b2);
        ssm_lds_pairs<H2>(&sb.bc[t][1][q * NH], c2);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float de = e ? d.y : d.x, due = de * (e ? u.y : u.x), dye = e ? dy.y : dy.x;
          const uint64_t d2 = f32x2_pack(de, de), du2 = f32x2_pack(due, due), dy2 = f32x2_pack(dye, dye);
          uint64_t x2 = 0, s2 = 0;
#pragma unroll
          for (int i = 0; i < H2; ++i) {
            const uint64_t gn = ffma2(dy2, c2[i], f32x2_pack(g[e][i]));
            qb[i] = e ? ffma2(du2, gn, qb[i]) : fmul2(du2, gn);
            x2 = i ? ffma2(gn, b2[i], x2) : fmul2(gn, b2[i]);
            const uint64_t w = fmul2(gn, ah[j][e][i]);
            s2 = i ? ffma2(w, f32x2_pack(A[e][i]), s2) : fmul2(w, f32x2_pack(A[e][i]));
            dA[e][i] = f32x2_unpack(ffma2(w, d2, f32x2_pack(dA[e][i])));
            g[e][i] = f32x2_unpack(fmul2(gn, a[j][e][i]));
          }
          const float2 x = f32x2_unpack(x2), s = f32x2_unpack(s2);
          xv[j][e] = x.x + x.y;
          sv[j][e] = s.x + s.y;
        }
        float bs[NH];
#pragma unroll
        for (int i = 0; i < H2; ++i) f32x2_unpack(qb[i], bs[2 * i], bs[2 * i + 1]);
        const float vb = ssm_sum_lanes<NH>(bs, lane, Cfg::SPLIT ? 2 * SPL : SPL, at);
        // this warp's sums of dB and dC over its channels
        float* red = &sb.red[buf][warp][j][q * NH + at];
        if constexpr (Cfg::SPLIT) {                    // the last lane bit: one of the two is left to add
          const bool up = lane & SPL;
          red[up ? NP : 0] = (up ? vc[j] : vb) + __shfl_xor_sync(0xffffffffu, up ? vb : vc[j], SPL);
        } else {
          red[0] = vb;
          red[NP] = vc[j];
        }
      }
      // y, dx, sum w A over the lanes of a channel: bit 0 picks the channel, bit 1 (if any) the tokens
#pragma unroll
      for (int j = 0; j < GT; ++j) {
        halve_sum(yv[j], 2, 1, q & 1);
        halve_sum(xv[j], 2, 1, q & 1);
        halve_sum(sv[j], 2, 1, q & 1);
      }
#pragma unroll
      for (int j = 0; j < FT; ++j) {
        float fy = yv[j][0], fx = xv[j][0], fs = sv[j][0];
        if constexpr (SPL == 4) {
          const bool up = q & 2;
          fy = (up ? yv[j + FT][0] : fy) + __shfl_xor_sync(0xffffffffu, up ? fy : yv[j + FT][0], 2);
          fx = (up ? xv[j + FT][0] : fx) + __shfl_xor_sync(0xffffffffu, up ? fx : xv[j + FT][0], 2);
          fs = (up ? sv[j + FT][0] : fs) + __shfl_xor_sync(0xffffffffu, up ? fs : sv[j + FT][0], 2);
        }
        const int tl = ft + j;
        if (live && t0 + tl < t_end) {
          const float u = to_f32(sm.u[tl][fc]), d = sm.d[tl][fc], dy = sm.dy[tl][fc];
          const float ddt = fmaf(fx, u, fs) * sigmoid_f32(to_f32(rd[j]) + fbias);
          const long long o = fo + j * static_cast<long long>(p.f.D);
          static_cast<T*>(p.du)[o] = from_f32<T>(fmaf(fx, d, skip * dy));
          static_cast<T*>(p.ddt)[o] = from_f32<T>(ddt);
          sD = fmaf(dy, u, sD);
          sT += ddt;
          if (p.f.z) {
            const float z = to_f32(rz[j]), s = sigmoid_f32(z);
            static_cast<T*>(p.dz)[o] = from_f32<T>(to_f32(ro[j]) * fmaf(skip, u, fy) * (s * fmaf(z, 1.f - s, 1.f)));
          }
        }
      }
      // the block's sums of dB and dC; the next group's go to the other buffer, and the one after comes
      // behind this barrier's successor
      __syncthreads();
      for (int i = threadIdx.x; i < GT * 2 * NP; i += SSM_THREADS) {
        const int j = i / (2 * NP), f = i % (2 * NP), n = f % NP, t = gr * GT + j;
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < SSM_THREADS / 32; ++w) s += sb.red[buf][w][j][f];
        if (n < N && t0 + t < t_end) part[t * 2 * N + (f < NP ? n : N + n)] = s;
      }
    }
  }
  if (t0 >= t_end) chain_wait();                       // (it has no states to load, but one to write over)
  if constexpr (SPL > 2) {                             // lanes that finished other tokens of the channel
    sD += __shfl_xor_sync(0xffffffffu, sD, 2);
    sT += __shfl_xor_sync(0xffffffffu, sT, 2);
  }
  if (!live) return;
  if (q < 2) {
    float* pc = p.part_c + seg * 2 * p.f.D + cf;
    pc[0] = sD;
    pc[p.f.D] = sT;
  }
  // this segment's dA takes the place of its entering state, which only this warp reads
#pragma unroll
  for (int i = 0; i < H2; ++i) {
    *reinterpret_cast<float2*>(seg_h + static_cast<long long>(2 * i) * p.f.D) = make_float2(dA[0][i].x, dA[1][i].x);
    *reinterpret_cast<float2*>(seg_h + static_cast<long long>(2 * i + 1) * p.f.D) = make_float2(dA[0][i].y, dA[1][i].y);
  }
}

// The call's last launch. Its first `bc_blocks` blocks: dB, dC [B][L][G][N] from the channel blocks' sums;
// rows past a sequence's end are left. The others: dA [D][N], dDskip [D], ddt_bias [D], sums over
// sequences and segments, 32 columns x 8 lanes of segments per block. All in a fixed order.
template <typename T>
__global__ __launch_bounds__(256) void ssm_bwd_sums_kernel(const SsmBwdParams p, int NP, unsigned bc_blocks) {
  __shared__ float red[8][33];
  const int N = p.f.N, G = p.f.G;
  chain_wait();
  if (blockIdx.x < bc_blocks) {
    const long long rows = static_cast<long long>(p.f.B) * p.f.L;
    const long long gid = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
    const long long row = gid / (2 * N * G);
    if (row >= rows) return;
    const int e = static_cast<int>(gid - row * (2 * N * G)), g = e / (2 * N), f = e - g * (2 * N);
    const int b = static_cast<int>(row / p.f.L);
    if (p.f.lens && row - static_cast<long long>(b) * p.f.L >= seq_len(p.f.lens, b, p.f.L)) return;
    float s = 0.f;
    const float* src = p.part_bc + (static_cast<long long>(g) * p.cbg * rows + row) * 2 * N + f;
#pragma unroll 8
    for (int i = 0; i < p.cbg; ++i) s += src[i * rows * 2 * N];
    T* dst = static_cast<T*>(f < N ? p.dB : p.dC);
    dst[(row * G + g) * N + (f < N ? f : f - N)] = from_f32<T>(s);
    return;
  }
  const int x = threadIdx.x % 32, y = threadIdx.x / 32;
  const long long nA = static_cast<long long>(p.f.D) * N, nC = 2LL * p.f.D;   // columns [N][D], [2][D]
  const long long blocksA = (nA + 31) / 32, blk = blockIdx.x - bc_blocks;
  const bool isA = blk < blocksA;
  const long long i = (isA ? blk : blk - blocksA) * 32 + x;
  const long long n = isA ? nA : nC, step = isA ? static_cast<long long>(p.f.D) * NP : nC;
  const float* src = isA ? p.f.seg_h : p.part_c;
  float a = 0.f;
  if (i < n) {
    const long long R = static_cast<long long>(p.f.B) * p.f.nseg;
#pragma unroll 8
    for (long long r = y; r < R; r += 8) a += src[r * step + i];
  }
  red[y][x] = a;
  __syncthreads();
  if (y == 0 && i < n) {
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) s += red[j][x];
    if (isA)
      p.dA[i % p.f.D * N + i / p.f.D] = s;
    else if (i < p.f.D) {
      if (p.dD) p.dD[i] = s;
    } else if (p.ddt_bias) {
      p.ddt_bias[i - p.f.D] = s;
    }
  }
}

}  // namespace kta

// mixer_common.cuh -- element access and scalar functions shared by the rotary, short-convolution
// and state-space kernels.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kta_ptx.cuh"

namespace kta {

template <typename T> __device__ __forceinline__ float to_f32(T x);
template <> __device__ __forceinline__ float to_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 x) {
  return __bfloat162float(x);
}
template <typename T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

// V elements of T moved as one access of 2, 4, 8 or 16 bytes.
template <int BYTES> struct RawVec;
template <> struct RawVec<16> { using type = uint4; };
template <> struct RawVec<8> { using type = uint2; };
template <> struct RawVec<4> { using type = uint32_t; };
template <> struct RawVec<2> { using type = uint16_t; };

template <typename T, int V> union VecPack {
  using Raw = typename RawVec<V * int(sizeof(T))>::type;
  Raw raw;
  T e[V];
  __device__ __forceinline__ VecPack() {}
  __device__ __forceinline__ void load(const T* p) { raw = *reinterpret_cast<const Raw*>(p); }
  __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<Raw*>(p) = raw; }
  __device__ __forceinline__ void zero() { raw = Raw(); }
};

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 1 / (1 + e^-x): 0 and 1 are reached where e^-x over- or underflows.
__device__ __forceinline__ float sigmoid_f32(float x) {
  return rcp_approx(1.f + ex2_approx(x * -1.4426950408889634f));
}

// log(1 + e^x) = max(x, 0) + log(1 + e^-|x|). log(1 + e) / e on 0 <= e <= 1 is a polynomial of degree 8 (a
// least-squares fit on Chebyshev nodes, reweighted towards equal relative errors: 3e-8), so that small e loses
// nothing to the 1. The relative error is that of e^-|x|, whose argument is rounded to fp32: below
// (1.25 |x| + 8) 2^-24, 1e-6 at step sizes of 1e-3 (x = -7); results below 2^-126 (x < -87.3) are 0.
__device__ __forceinline__ float softplus_f32(float x) {
  const float e = ex2_approx(fabsf(x) * -1.4426950408889634f);
  float r = 0.0052326880395412445f;
  r = fmaf(r, e, -0.029505213722586632f);
  r = fmaf(r, e, 0.07822591066360474f);
  r = fmaf(r, e, -0.13663242757320404f);
  r = fmaf(r, e, 0.19106005132198334f);
  r = fmaf(r, e, -0.2484298199415207f);
  r = fmaf(r, e, 0.3331909775733948f);
  r = fmaf(r, e, -0.4999949336051941f);
  r = fmaf(r, e, 0.9999999403953552f);
  return fmaf(r, e, fmaxf(x, 0.f));
}

__device__ __forceinline__ uint64_t fmul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ uint64_t f32x2_pack(float2 v) { return f32x2_pack(v.x, v.y); }
__device__ __forceinline__ float2 f32x2_unpack(uint64_t v) {
  float2 r;
  f32x2_unpack(v, r.x, r.y);
  return r;
}

// Kernels of one call in a row: a kernel lets the next be set up while it still runs, and the next one
// waits, before it touches what the earlier ones write, until they have ended. Both do nothing in a
// launch without the attribute.
__device__ __forceinline__ void chain_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void chain_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <int BYTES>
__device__ __forceinline__ void piece_async(void* dst, const void* src, bool on) {
  const uint32_t n = on ? BYTES : 0;       // 0: filled with zeros
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(smem_u32(dst)), "l"(src), "n"(BYTES), "r"(n)
                 : "memory");
}
__device__ __forceinline__ void piece_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void piece_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

// One halving step of a sum over lanes: n values per lane, each summed with lane ^ mask; the lane
// whose `mask` bit is clear keeps the lower n / 2 sums, the other the upper ones.
template <int CNT>
__device__ __forceinline__ void halve_sum(float (&v)[CNT], int n, int mask, bool upper) {
#pragma unroll
  for (int i = 0; i < CNT / 2; ++i) {
    if (i < n / 2) {
      const float send = upper ? v[i] : v[i + n / 2];
      const float keep = upper ? v[i + n / 2] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, mask);
    }
  }
}

// Rows of sequence b: its length if lengths are given (kept within the tensor), else all L.
__device__ __forceinline__ int seq_len(const int* lens, int b, int L) {
  return lens ? min(max(lens[b], 0), L) : L;
}

}  // namespace kta

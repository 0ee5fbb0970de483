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

// log(1 + e^x) = max(x, 0) + log(1 + e^-|x|), relative error a few 2^-23 everywhere: with e = e^-|x|
// and s = e / (2 + e) <= 1/3, log(1 + e) = 2 artanh(s) = 2 s (1 + s^2/3 + s^4/5 + ...), cut where
// the rest is below 2^-26 of the sum ((1/9)^8 / 17).
__device__ __forceinline__ float softplus_f32(float x) {
  const float e = ex2_approx(fabsf(x) * -1.4426950408889634f);
  const float s = e * rcp_approx(2.f + e), q = s * s;
  float r = 1.f / 15.f;
  r = fmaf(r, q, 1.f / 13.f);
  r = fmaf(r, q, 1.f / 11.f);
  r = fmaf(r, q, 1.f / 9.f);
  r = fmaf(r, q, 1.f / 7.f);
  r = fmaf(r, q, 1.f / 5.f);
  r = fmaf(r, q, 1.f / 3.f);
  r = fmaf(r, q, 1.f);
  return fmaxf(x, 0.f) + 2.f * s * r;
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

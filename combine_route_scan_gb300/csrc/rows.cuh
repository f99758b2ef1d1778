// Rows of fp16 / bf16 as fp32 numbers and back, for combine and the gradients of
// combine and dispatch.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace crs {

// Element traits: 16-byte vectors of T, fp32 accumulators.
template <int DT>
struct Vec;
template <>
struct Vec<MOE_F16> {
  __device__ static void unpack(float (&f)[8], int4 v) {
    const __half2* h = reinterpret_cast<const __half2*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = __half22float2(h[i]);
      f[2 * i] = a.x;
      f[2 * i + 1] = a.y;
    }
  }
  __device__ static void fma(float* acc, float w, int4 v) {
    const __half2* h = reinterpret_cast<const __half2*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(h[i]);
      acc[2 * i] = __fmaf_rn(w, f.x, acc[2 * i]);
      acc[2 * i + 1] = __fmaf_rn(w, f.y, acc[2 * i + 1]);
    }
  }
  __device__ static int4 pack(const float* acc) {
    int4 o;
    __half2* h = reinterpret_cast<__half2*>(&o);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(acc[2 * i], acc[2 * i + 1]);
    return o;
  }
};
template <>
struct Vec<MOE_BF16> {
  __device__ static void unpack(float (&f)[8], int4 v) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = __bfloat1622float2(h[i]);
      f[2 * i] = a.x;
      f[2 * i + 1] = a.y;
    }
  }
  __device__ static void fma(float* acc, float w, int4 v) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __bfloat1622float2(h[i]);
      acc[2 * i] = __fmaf_rn(w, f.x, acc[2 * i]);
      acc[2 * i + 1] = __fmaf_rn(w, f.y, acc[2 * i + 1]);
    }
  }
  __device__ static int4 pack(const float* acc) {
    int4 o;
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&o);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(acc[2 * i], acc[2 * i + 1]);
    return o;
  }
};

template <int DT>
__device__ __forceinline__ float elem_to_float(uint16_t b) {
  return DT == MOE_F16 ? __half2float(__ushort_as_half(b)) : __bfloat162float(__ushort_as_bfloat16(b));
}
template <int DT>
__device__ __forceinline__ uint16_t float_to_elem(float f) {
  return DT == MOE_F16 ? __half_as_ushort(__float2half_rn(f)) : __bfloat16_as_ushort(__float2bfloat16_rn(f));
}

// 16 bytes that the kernel may write to as well.
__device__ __forceinline__ int4 ld_v4(const void* p) {
  int4 v;
  asm volatile("ld.global.v4.s32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}

// The flat row of each lane's routed pick (class cls >= 0; lanes beyond the token's picks have another) without a
// pick -> row map: the rows of a segment (expert, source rank) are at most bs, so that a warp looks through 32 of a pick's
// at a time. -1 where no row names the pick, or counts are out of range. All lanes of a warp take part.
__device__ __forceinline__ long long find_rows(const CombineParams& p, size_t tau, int cls) {
  const Shape& sh = p.sh;
  const int lane = threadIdx.x & 31, s = (int)(tau / sh.bs), t = (int)(tau % sh.bs), LW = sh.L * sh.W;
  int lo = 0, hi = 0;
  if (cls >= 0) {
    const int32_t* ep = p.ep_recv_count + (size_t)(cls / sh.L) * LW;
    const int seg = cls % sh.L * sh.W + s;
    hi = ep[seg];
    lo = seg ? ep[seg - 1] : 0;
    if (lo < 0 || hi < lo || hi > sh.A || ep[LW - 1] > sh.A) lo = hi = 0;
  }
  const long long first = (long long)(cls >= 0 ? cls / sh.L : 0) * sh.A;
  long long found = -1;
  // the first 32 rows of all picks are asked for before any is looked at
  constexpr int kAhead = 8;
  for (int k0 = 0; k0 < sh.K; k0 += kAhead) {
    int at[kAhead], ak[kAhead], as[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const long long base = __shfl_sync(0xffffffffu, first + lo, (k0 + j) & 31);
      const int n = k0 + j < sh.K ? __shfl_sync(0xffffffffu, hi - lo, (k0 + j) & 31) : 0;
      as[j] = -1;
      if (lane < n) {
        const int32_t* a = p.assist + (base + lane) * 3;
        as[j] = a[0], at[j] = a[1], ak[j] = a[2];
      }
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int k = k0 + j;
      if (k >= sh.K) break;
      const long long base = __shfl_sync(0xffffffffu, first + lo, k);
      const int n = __shfl_sync(0xffffffffu, hi - lo, k);
      uint32_t match = __ballot_sync(0xffffffffu, as[j] == s && at[j] == t && ak[j] == k);
      int r = 0;
      for (; !match && r + 32 < n; r += 32) {
        bool here = false;
        if (r + 32 + lane < n) {
          const int32_t* a = p.assist + (base + r + 32 + lane) * 3;
          here = a[0] == s && a[1] == t && a[2] == k;
        }
        match = __ballot_sync(0xffffffffu, here);
      }
      if (lane == k && match) found = base + r + __ffs(match) - 1;
    }
  }
  return found;
}

}  // namespace crs

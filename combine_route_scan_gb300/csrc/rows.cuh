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

// The flat row of pick (s, t, k), routed to expert e, without a pick -> row map: a warp looks through the rows of the
// segment (e, s), at most bs of them, 32 at a time; of more than 32, which dispatch leaves in ascending t, first where t
// should be and then, should the rows be in another order, through all. -1 where none names the pick, or counts are out
// of range.
__device__ __forceinline__ long long find_row(const CombineParams& p, int s, int t, int k, int e) {
  const Shape& sh = p.sh;
  const int lane = threadIdx.x & 31, d = e / sh.L, seg = e % sh.L * sh.W + s, LW = sh.L * sh.W;
  const int32_t* ep = p.ep_recv_count + (size_t)d * LW;
  const int hi = ep[seg], lo = seg ? ep[seg - 1] : 0;
  if (lo < 0 || hi > sh.A || ep[LW - 1] > sh.A) return -1;
  const int32_t* assist = p.assist + (long long)d * sh.A * 3;
  const auto look = [&](int from, int to) {
    for (int r = from; r < to; r += 32) {
      bool here = false;
      if (r + lane < to) {
        const int32_t* a = assist + (long long)(r + lane) * 3;
        here = a[0] == s && a[1] == t && a[2] == k;
      }
      const uint32_t match = __ballot_sync(0xffffffffu, here);
      if (match) return (long long)d * sh.A + r + __ffs(match) - 1;
    }
    return -1ll;
  };
  if (hi - lo > 32) {
    const int step = (hi - lo + 31) / 32, probe = lo + lane * step;
    const uint32_t below = __ballot_sync(0xffffffffu, probe < hi && assist[(long long)probe * 3 + 1] <= t);
    const int at = lo + max(0, __popc(below) - 1) * step;
    const long long r = look(at, min(hi, at + step));
    if (r >= 0) return r;
  }
  return look(lo, hi);
}

// The rows of a token's picks into s_row[K], by all warps of the block; ends with a barrier.
__device__ __forceinline__ void find_rows(const CombineParams& p, size_t tau, long long* s_row) {
  const Shape& sh = p.sh;
  for (int k = threadIdx.x >> 5; k < sh.K; k += blockDim.x >> 5) {
    const int c = classify_pick(p.ids, p.mask, sh, tau, k);
    const long long r = c >= 0 ? find_row(p, (int)(tau / sh.bs), (int)(tau % sh.bs), k, c) : -1;
    if ((threadIdx.x & 31) == 0) s_row[k] = r;
  }
  __syncthreads();
}

}  // namespace crs

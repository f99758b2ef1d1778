// Routing scores to expert ids and weights (moe_route) and the gradient of the
// weights (moe_route_backward); include/moe_experts.h has the formulas.
//
// One warp a token, a lane holding E / 32 neighbouring experts (rounded up to a power
// of two) in registers, in one load. A large batch is bound by instructions and by their
// latency: 65521 tokens x 256 experts in 8 groups take 480 warp instructions a token,
// some 160 of them (20 a key) for the keys and the rest for the choice, on 68% of the issue
// slots with 37% of the warps resident. The keys of all experts are needed, the
// weights of the picks alone: keys come from the fast exponential and reciprocal
// (within 2^-21 of the formula and 2^-16 of the score; equal logits and biases give
// equal keys), and the lanes that end up with a pick compute its weight with expf and
// IEEE division. Picking the K largest keys one by one costs a warp-wide argmax and a
// rescan each (73 us where this took 57, 65521 tokens x 256 experts); instead
//   * the K-th largest of the 32 lanes' maxima bounds the K-th largest key from below,
//     since at least K keys are not below it: each lane counts the maxima ahead of
//     its own;
//   * the keys that reach it, mostly little more than K of them, are listed in shared
//     memory by ballots, one a lane comes back, and each counts the keys ahead of it
//     (larger, or equal with a lower index): its rank is its place in the output.
// More than 32 such keys (ties, large K) are picked one by one. Groups of experts that
// do not fall on lanes, and more than 512 experts (their keys would not fit the
// registers), take route_any_kernel, which keeps the row in shared memory. Experts that are not
// 32 times a power of two leave lanes idle and are loaded an element at a time. 65521 tokens,
// fp32: 256 experts 34 us, 384 84 us, 160 49 us; in 8 groups 256 experts 40 us, 160 114 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "../../include/moe_experts.h"
#include "common.cuh"
#include "experts_host.h"

namespace crs {

constexpr int kRouterWarps = 4;
// From here on two tokens a warp. One / two at 4096, 8192 and 65521 tokens: 256 experts in 8
// groups 5.8 / 6.5, 9.6 / 8.1 and 52 / 39 us, 128 experts 4.6 / 4.2, 6.6 / 5.3 and 37 / 26 us, 256
// experts without groups 4.6 / 6.5, 7.9 / 8.2 and 46 / 38 us.
constexpr int kPairTokens = 8192;
// The gradient's row is most of its work. One / two at 4096, 8192 and 65536 tokens: 128 experts 2.4 /
// 2.2, 3.5 / 2.7 and 18.7 / 12.7 us, 256 experts (every gradient) 3.2 / 3.9, 4.9 / 5.4 and 32 / 28 us, the
// two lines of which meet at some 16000.
constexpr int kGradPairTokens = 4096, kGradPairTokensWide = 16384;
constexpr int kBoundSteps = 12;    // halvings of the interval that a bound on the picks' keys is sought in
constexpr uint32_t kAll = 0xffffffffu;

struct RouterParams {
  const void* logits;
  const float* bias;
  const int32_t* ids_in;
  const float* grad;
  int32_t* ids;
  float* weights;
  void* grad_logits;
  long long stride, grad_stride;
  int T, E, K, G, KG, top2, sigmoid, renorm;
  int T_step;        // tokens a warp takes at once
  int vec;           // whole lanes at once: E = 32 * EPL and the rows that are held by lanes aligned for it
  float scaling;
};

// Keys as unsigned integers that order like the floats: -inf (masked and NaN
// keys) stays above 0, which stands for an expert that cannot be picked.
constexpr uint32_t kMaskedKey = 0x007fffffu;
__device__ __forceinline__ uint32_t ordered_number(float f) {
  const uint32_t b = __float_as_uint(__fadd_rn(f, 0.f));  // -0 and +0 are equal keys
  return b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ uint32_t ordered_key(float f) { return f == f ? ordered_number(f) : kMaskedKey; }
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

template <int DT>
__device__ __forceinline__ float load_logit(const void* row, int e) {
  if (DT == MOE_F32) return __ldg(static_cast<const float*>(row) + e);
  const uint16_t b = __ldg(static_cast<const uint16_t*>(row) + e);
  return DT == MOE_F16 ? __half2float(__ushort_as_half(b)) : __bfloat162float(__ushort_as_bfloat16(b));
}
template <int DT>
__device__ __forceinline__ const void* logit_row(const void* base, long long t, long long stride) {
  return static_cast<const uint8_t*>(base) + t * stride * (DT == MOE_F32 ? 4 : 2);
}
template <int DT>
__device__ __forceinline__ void store_logit(void* row, int e, float v) {
  if (DT == MOE_F32) static_cast<float*>(row)[e] = v;
  else if (DT == MOE_F16) static_cast<__half*>(row)[e] = __float2half_rn(v);
  else static_cast<__nv_bfloat16*>(row)[e] = __float2bfloat16_rn(v);
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(kAll, v, o));
  return v;
}

// 1 / (1 + exp(-x)); the reciprocal rounded to nearest is the division's result.
__device__ __forceinline__ float sigmoid_of(float x) { return __frcp_rn(__fadd_rn(1.f, expf(-x))); }

// Scores for the keys: the special functions' exponential and reciprocal, subnormal numbers as
// zeros (an exponential of those changes nothing next to 1, a score of those is far within
// the keys' 2^-21). Their plain forms' care for subnormals cost a tenth of the time (44 -> 40 us).
__device__ __forceinline__ float fast_sigmoid(float x) {
  float e, s;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.44269504088896f));  // 2^(-x / ln 2)
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.f + e));
  return s;
}
// A bias of NaN counts as -inf: then no sum with a score is NaN, or -0.
__device__ __forceinline__ float load_bias(const float* bias, int e) {
  const float b = __ldg(bias + e);
  return b == b ? b : -INFINITY;
}
__device__ __forceinline__ uint32_t score_key(float x, float score, float bias) {
  const uint32_t b = __float_as_uint(__fadd_rn(score, bias));
  return x == -INFINITY ? kMaskedKey : b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
}

// The index of the largest key among a lane's best (key, index) pairs, the
// lowest index among equal keys.
__device__ __forceinline__ int warp_argmax(uint32_t key, int index, uint32_t* best) {
  const uint32_t m = __reduce_max_sync(kAll, key);
  *best = m;
  return __reduce_min_sync(kAll, key == m ? (unsigned)index : 0x7fffffffu);
}

template <int DT>
__global__ void __launch_bounds__(kRouterWarps * 32) route_any_kernel(RouterParams p) {
  extern __shared__ uint32_t rsm[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t* key = rsm + warp * (2 * p.E + p.G);
  float* score = reinterpret_cast<float*>(key + p.E);
  uint32_t* value = key + 2 * p.E;
  pdl_wait();
  pdl_launch_dependents();
  for (long long t = (long long)blockIdx.x * kRouterWarps + warp; t < p.T; t += (long long)gridDim.x * kRouterWarps) {
    const void* row = logit_row<DT>(p.logits, t, p.stride);
    const bool by_score = p.bias || p.top2;
    float top = -INFINITY;
    for (int e = lane; e < p.E; e += 32) {
      const float x = load_logit<DT>(row, e);
      score[e] = x == x ? x : -INFINITY;
      top = fmaxf(top, score[e]);
    }
    top = warp_max(top);
    float sum = 0.f;
    if (!p.sigmoid) {
      for (int e = lane; e < p.E; e += 32) {
        const float x = score[e];
        key[e] = ordered_key(x);
        const float v = x == -INFINITY ? 0.f : x == top ? 1.f : expf(__fsub_rn(x, top));
        score[e] = v;
        sum = __fadd_rn(sum, v);
      }
      sum = warp_sum(sum);
    }
    for (int e = lane; e < p.E; e += 32) {
      float s;
      bool masked;
      if (p.sigmoid) {
        const float x = score[e];
        masked = x == -INFINITY;
        s = masked ? 0.f : sigmoid_of(x);
        key[e] = ordered_key(x);
      } else {
        masked = key[e] == kMaskedKey;
        s = sum > 0.f ? __fdiv_rn(score[e], sum) : 0.f;
      }
      score[e] = s;
      if (by_score) key[e] = masked ? kMaskedKey : ordered_key(p.bias ? __fadd_rn(s, __ldg(p.bias + e)) : s);
    }
    __syncwarp();
    if (p.G > 1) {
      const int gs = p.E / p.G;
      for (int g = lane; g < p.G; g += 32) {
        uint32_t a = 0, b = 0;
        for (int i = 0; i < gs; ++i) {
          const uint32_t k = key[g * gs + i];
          if (k > a) { b = a; a = k; }
          else if (k > b) b = k;
        }
        if (p.top2 && b > kMaskedKey) a = ordered_key(__fadd_rn(key_value(a), key_value(b)));
        value[g] = a;
      }
      __syncwarp();
      for (int i = 0; i < p.KG; ++i) {
        uint32_t best = 0;
        int at = 0x7fffffff;
        for (int g = lane; g < p.G; g += 32)
          if (value[g] > best) { best = value[g]; at = g; }
        uint32_t m;
        const int g = warp_argmax(best, at, &m);
        if (lane == 0) value[g] = 0;  // open
        __syncwarp();
      }
      for (int e = lane; e < p.E; e += 32)
        if (value[e / gs] != 0) key[e] = 0;
      __syncwarp();
    }
    int my_id = 0;
    float my_score = 0.f;
    for (int k = 0; k < p.K; ++k) {
      uint32_t best = 0;
      int at = 0x7fffffff;
      for (int e = lane; e < p.E; e += 32)
        if (key[e] > best) { best = key[e]; at = e; }
      uint32_t m;
      const int e = warp_argmax(best, at, &m);
      if (lane == k) { my_id = e; my_score = score[e]; }
      __syncwarp();
      if (lane == 0) key[e] = 0;
      __syncwarp();
    }
    float w = my_score;
    if (p.renorm) {
      const float total = warp_sum(lane < p.K ? my_score : 0.f);
      w = total > 0.f ? __fdiv_rn(my_score, total) : 0.f;
    }
    if (lane < p.K) {
      p.ids[t * p.K + lane] = my_id;
      p.weights[t * p.K + lane] = __fmul_rn(w, p.scaling);
    }
    __syncwarp();
  }
}

// A lane's EPL neighbouring logits; past the row's end they read as masked.
template <int DT, int EPL>
__device__ __forceinline__ void load_lane(const void* row, int E, bool vec, int lane, float (&x)[EPL]) {
  const int e0 = lane * EPL;
  constexpr int kBytes = EPL * (DT == MOE_F32 ? 4 : 2);
  if (vec) {
    alignas(16) uint32_t w[(kBytes + 3) / 4];
    const uint8_t* q = static_cast<const uint8_t*>(row) + (size_t)e0 * (DT == MOE_F32 ? 4 : 2);
    if (kBytes >= 16) {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i) *reinterpret_cast<int4*>(&w[i * 4]) = ld_nc_v4(q + i * 16);
    } else if (kBytes == 8) {
      *reinterpret_cast<uint2*>(&w[0]) = __ldg(reinterpret_cast<const uint2*>(q));
    } else if (kBytes == 4) {
      w[0] = __ldg(reinterpret_cast<const uint32_t*>(q));
    } else {
      w[0] = __ldg(reinterpret_cast<const uint16_t*>(q));
    }
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      if (DT == MOE_F32) x[j] = __uint_as_float(w[j]);
      else if (DT == MOE_BF16) x[j] = __uint_as_float(j & 1 ? w[j / 2] & 0xffff0000u : w[j / 2] << 16);
      else x[j] = __half2float(__ushort_as_half((uint16_t)(w[j / 2] >> (16 * (j & 1)))));
    }
  } else {
#pragma unroll
    for (int j = 0; j < EPL; ++j) x[j] = e0 + j < E ? load_logit<DT>(row, e0 + j) : -INFINITY;
  }
}

// A warp's keys and logits by expert, and the candidates among them: index, then key
// and inverted index (the order of these pairs is the order of the picks).
template <int EPL>
struct RouteScratch {
  uint32_t key[32 * EPL];
  float x[32 * EPL];
  unsigned long long order[32];
  int list[32];
  uint32_t best[32];
};

template <int DT, int EPL>
__global__ void __launch_bounds__(kRouterWarps * 32) route_kernel(RouterParams p) {
  __shared__ alignas(16) RouteScratch<EPL> scratch[kRouterWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e0 = lane * EPL;
  const int mine = min(EPL, max(0, p.E - e0));  // experts of this lane
  RouteScratch<EPL>& sc = scratch[warp];
  const bool by_score = p.bias || p.top2;
  pdl_wait();
  pdl_launch_dependents();
  float bias[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) bias[j] = p.bias && j < mine ? load_bias(p.bias, e0 + j) : 0.f;
  for (long long t = (long long)blockIdx.x * kRouterWarps + warp; t < p.T; t += (long long)gridDim.x * kRouterWarps) {
    float x[EPL];
    uint32_t key[EPL];
    load_lane<DT, EPL>(logit_row<DT>(p.logits, t, p.stride), p.E, p.vec, lane, x);
#pragma unroll
    for (int j = 0; j < EPL; ++j) x[j] = fmaxf(x[j], -INFINITY);  // NaN becomes -inf
    float top = -INFINITY, sum = 1.f;
    if (!by_score) {
#pragma unroll
      for (int j = 0; j < EPL; ++j) key[j] = ordered_number(x[j]);
    }
    if (p.sigmoid) {
      if (by_score) {
#pragma unroll
        for (int j = 0; j < EPL; ++j) key[j] = score_key(x[j], fast_sigmoid(x[j]), bias[j]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < EPL; ++j) top = fmaxf(top, x[j]);
      top = key_value(__reduce_max_sync(kAll, ordered_number(top)));
      sum = 0.f;
      float v[EPL];
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        // exp(-inf) is 0; a row without experts and +inf leave no number in the difference
        const float d = __fsub_rn(x[j], top);
        v[j] = d == d ? expf(d) : top > 0.f ? 1.f : 0.f;
        sum = __fadd_rn(sum, v[j]);
      }
      sum = warp_sum(sum);
      if (by_score) {
        const float share = sum > 0.f ? __fdiv_rn(1.f, sum) : 0.f;
#pragma unroll
        for (int j = 0; j < EPL; ++j) key[j] = score_key(x[j], __fmul_rn(v[j], share), bias[j]);
      }
    }
    if (!p.vec) {
#pragma unroll
      for (int j = 0; j < EPL; ++j)
        if (j >= mine) key[j] = 0;  // past the last expert: not to be picked
    }
    uint32_t best = 0;
#pragma unroll
    for (int j = 0; j < EPL; ++j) best = max(best, key[j]);
    if (p.G > 1) {
      // 32 / G lanes a group
      uint32_t second = 0;
      if (p.top2) {
        uint32_t a = 0;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
          second = max(second, min(a, key[j]));
          a = max(a, key[j]);
        }
      }
      uint32_t value = best;
      for (int o = 16 / p.G; o; o >>= 1) {
        const uint32_t v = __shfl_xor_sync(kAll, value, o), w = __shfl_xor_sync(kAll, second, o);
        second = max(max(second, w), min(value, v));
        value = max(value, v);
      }
      if (p.top2 && second > kMaskedKey) value = ordered_key(__fadd_rn(key_value(value), key_value(second)));
      const uint32_t group = (uint32_t)lane & ~(uint32_t)(32 / p.G - 1);  // its first lane
      bool open = false;
      for (int i = 0; i < p.KG; ++i) {
        const uint32_t m = __reduce_max_sync(kAll, value);
        if (group == (uint32_t)(__ffs(__ballot_sync(kAll, value == m)) - 1)) {
          open = true;
          value = 0;
        }
      }
      if (!open) {
        best = 0;
#pragma unroll
        for (int j = 0; j < EPL; ++j) key[j] = 0;
      }
    }
    uint32_t bound = 1;  // fewer lanes than picks: every key that may be picked
    if (__popc(__ballot_sync(kAll, best != 0)) >= p.K) {
      // the least of the K largest lanes' maxima, each lane counting those ahead of its own
      sc.best[lane] = best;
      __syncwarp();
      int ahead = 0;
#pragma unroll
      for (int i = 0; i < 32; i += 4) {
        const uint4 o = *reinterpret_cast<const uint4*>(&sc.best[i]);
        ahead += (o.x > best) + (o.y > best) + (o.z > best) + (o.w > best);
      }
      bound = __reduce_min_sync(kAll, best && ahead < p.K ? best : 0xffffffffu);
    }
    uint32_t in = 0;
#pragma unroll
    for (int j = 0; j < EPL; ++j) in |= (key[j] >= bound ? 1u : 0u) << j;
    // keys and logits to shared memory, candidates' indexes listed a round a lane's next one
#pragma unroll
    for (int j = 0; j < EPL; j += 4) {
      if (EPL >= 4) {
        *reinterpret_cast<uint4*>(&sc.key[e0 + j]) = make_uint4(key[j], key[(j + 1) % EPL], key[(j + 2) % EPL], key[(j + 3) % EPL]);
        *reinterpret_cast<float4*>(&sc.x[e0 + j]) = make_float4(x[j], x[(j + 1) % EPL], x[(j + 2) % EPL], x[(j + 3) % EPL]);
      } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i) sc.key[e0 + i] = key[i], sc.x[e0 + i] = x[i];
      }
    }
    int count = 0;
    for (uint32_t who; (who = __ballot_sync(kAll, in != 0)) != 0 && count <= 32;) {
      const int at = count + __popc(who & lanemask_lt());
      if (in && at < 32) sc.list[at] = e0 + __ffs(in) - 1;
      in &= in - 1;
      count += __popc(who);
    }
    __syncwarp();
    int rank = 32, id = 0;
    if (count <= 32) {
      unsigned long long own = 0;
      if (lane < count) {
        id = sc.list[lane];
        own = ((unsigned long long)sc.key[id] << 32) | (uint32_t)~id;
      }
      sc.order[lane] = own;
      __syncwarp();
      rank = 0;
      for (int i = 0; i < count; i += 2) {
        const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(&sc.order[i]);
        rank += (o.x > own) + (o.y > own);
      }
      if (lane >= count) rank = 32;
    } else {
      for (int k = 0; k < p.K; ++k) {
        uint32_t b = 0, m;
        int at = 0x7fffffff;
#pragma unroll
        for (int j = 0; j < EPL; ++j)
          if (key[j] > b) b = key[j], at = e0 + j;
        const int e = warp_argmax(b, at, &m);
        if (lane == k) rank = k, id = e;
#pragma unroll
        for (int j = 0; j < EPL; ++j)
          if (e0 + j == e) key[j] = 0;
      }
    }
    const bool picked = rank < p.K;
    const float at = sc.x[id];
    __syncwarp();
    float score;
    if (p.sigmoid) {
      score = sigmoid_of(at);  // of -inf: 0
    } else {
      const float d = __fsub_rn(at, top);
      score = sum > 0.f ? __fdiv_rn(d == d ? expf(d) : top > 0.f ? 1.f : 0.f, sum) : 0.f;
    }
    float w = score;
    if (p.renorm) {
      const float total = warp_sum(picked ? score : 0.f);
      w = total > 0.f ? __fdiv_rn(score, total) : 0.f;
    }
    if (picked) {
      p.ids[t * p.K + rank] = id;
      p.weights[t * p.K + rank] = __fmul_rn(w, p.scaling);
    }
  }
}

// Two tokens a warp, 16 lanes each (E = 16 EPL, K <= 16): what a token costs beside
// its experts' keys, rather more than half, is then spent once for two. The steps are
// route_kernel's; where that asks the whole warp, the halves use shuffles within
// themselves, and ranks by counting in place of repeated maxima. 65521 tokens: 256
// experts in 8 groups 52 -> 39 us, 128 without groups 37 -> 26 us (seven CTAs an SM by
// their registers; six take 41 us, eight 40, nine 43). Below some 8192 tokens there are warps
// enough for one token each, and those are done sooner.
// A lane's experts lie kRow words from the next lane's (no bank conflicts).
template <int EPL>
struct PairScratch {
  static constexpr int kRow = EPL >= 8 ? EPL + 4 : EPL;
  static __device__ __forceinline__ int place(int e) { return e / EPL * kRow + e % EPL; }
  uint32_t key[2][16 * kRow];
  float x[2][16 * kRow];
  unsigned long long order[2][16];
  int list[2][16];
};

__device__ __forceinline__ float half_max(float v) {
#pragma unroll
  for (int o = 8; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}
__device__ __forceinline__ float half_sum(float v) {
#pragma unroll
  for (int o = 8; o; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(kAll, v, o));
  return v;
}

template <int DT, int EPL>
__global__ void __launch_bounds__(kRouterWarps * 32, 7) route_pair_kernel(RouterParams p) {
  __shared__ alignas(16) PairScratch<EPL> scratch[kRouterWarps];
  using Scratch = PairScratch<EPL>;
  __shared__ alignas(16) float bias[16 * Scratch::kRow];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, half = lane >> 4, hl = lane & 15, e0 = hl * EPL, s0 = hl * PairScratch<EPL>::kRow;
  const uint32_t half_lanes = 0xffffu << (16 * half), below = lanemask_lt() & half_lanes;
  PairScratch<EPL>& sc = scratch[warp];
  const bool by_score = p.bias || p.top2;
  pdl_wait();
  pdl_launch_dependents();
  for (int e = threadIdx.x; e < 16 * EPL; e += kRouterWarps * 32) bias[Scratch::place(e)] = p.bias ? load_bias(p.bias, e) : 0.f;
  __syncthreads();
  const bool plenty = 16 * p.KG / p.G >= 2 * p.K;  // open lanes for each pick
  const long long pairs = ((long long)p.T + 1) / 2;
  for (long long w = (long long)blockIdx.x * kRouterWarps + warp; w < pairs; w += (long long)gridDim.x * kRouterWarps) {
    const bool there = 2 * w + half < p.T;  // an odd last token is done twice and stored once
    const long long t = there ? 2 * w + half : p.T - 1;
    float x[EPL];
    uint32_t key[EPL];
    if (DT == MOE_F32 && EPL == 16) {
      // 64 bytes a lane: loaded 16 bytes a lane in turn and handed over in shared memory
      const float* row = static_cast<const float*>(logit_row<DT>(p.logits, t, p.stride));
      float4 v[EPL / 4];
#pragma unroll
      for (int i = 0; i < EPL / 4; ++i) {
        const int4 w4 = ld_nc_v4(row + i * 64 + hl * 4);
        v[i] = make_float4(fmaxf(__int_as_float(w4.x), -INFINITY), fmaxf(__int_as_float(w4.y), -INFINITY),
                           fmaxf(__int_as_float(w4.z), -INFINITY), fmaxf(__int_as_float(w4.w), -INFINITY));
      }
#pragma unroll
      for (int i = 0; i < EPL / 4; ++i) *reinterpret_cast<float4*>(&sc.x[half][Scratch::place(i * 64 + hl * 4)]) = v[i];
      __syncwarp();
#pragma unroll
      for (int j = 0; j < EPL; j += 4) {
        const float4 a = *reinterpret_cast<const float4*>(&sc.x[half][s0 + j]);
        x[j] = a.x, x[j + 1] = a.y, x[j + 2] = a.z, x[j + 3] = a.w;
      }
    } else {
      load_lane<DT, EPL>(logit_row<DT>(p.logits, t, p.stride), p.E, true, hl, x);
#pragma unroll
      for (int j = 0; j < EPL; ++j) x[j] = fmaxf(x[j], -INFINITY);  // NaN becomes -inf
#pragma unroll
      for (int j = 0; j < EPL; j += 4) *reinterpret_cast<float4*>(&sc.x[half][s0 + j]) = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
    }
    float top = -INFINITY, sum = 1.f;
    if (!by_score) {
#pragma unroll
      for (int j = 0; j < EPL; ++j) key[j] = ordered_number(x[j]);
    }
    if (p.sigmoid) {
      if (by_score) {
#pragma unroll
        for (int j = 0; j < EPL; j += 4) {
          const float4 b = *reinterpret_cast<const float4*>(&bias[s0 + j]);
          const float bj[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) key[j + i] = score_key(x[j + i], fast_sigmoid(x[j + i]), bj[i]);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < EPL; ++j) top = fmaxf(top, x[j]);
      top = half_max(top);
      sum = 0.f;
      float v[EPL];
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        const float d = __fsub_rn(x[j], top);
        v[j] = d == d ? expf(d) : top > 0.f ? 1.f : 0.f;
        sum = __fadd_rn(sum, v[j]);
      }
      sum = half_sum(sum);
      if (by_score) {
        const float share = sum > 0.f ? __fdiv_rn(1.f, sum) : 0.f;
#pragma unroll
        for (int j = 0; j < EPL; ++j) key[j] = score_key(x[j], __fmul_rn(v[j], share), bias[s0 + j]);
      }
    }
    uint32_t best = 0, next = 0;  // the lane's two largest
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      next = max(next, min(best, key[j]));
      best = max(best, key[j]);
    }
    if (p.G > 1) {
      // 16 / G lanes a group
      uint32_t second = next, value = best;
      const int lanes = 16 / p.G;
      for (int o = lanes / 2; o; o >>= 1) {
        const uint32_t v = __shfl_xor_sync(kAll, value, o), w2 = __shfl_xor_sync(kAll, second, o);
        second = max(max(second, w2), min(value, v));
        value = max(value, v);
      }
      if (p.top2 && second > kMaskedKey) value = ordered_key(__fadd_rn(key_value(value), key_value(second)));
      int ahead = 0;  // groups that come first
      for (int o = lanes; o < 16; o += lanes) {
        const uint32_t v = __shfl_xor_sync(kAll, value, o);
        ahead += v > value || (v == value && (hl ^ o) < hl);
      }
      if (ahead >= p.KG) {
        best = next = 0;
#pragma unroll
        for (int j = 0; j < EPL; ++j) key[j] = 0;
      }
    }
#pragma unroll
    for (int j = 0; j < EPL; j += 4) *reinterpret_cast<uint4*>(&sc.key[half][s0 + j]) = make_uint4(key[j], key[j + 1], key[j + 2], key[j + 3]);
    uint32_t bound;
    if (plenty) {
      // the least of the K largest lanes' maxima, each lane counting those ahead of its own
      int ahead = 0;
#pragma unroll
      for (int o = 1; o < 16; ++o) ahead += __shfl_xor_sync(kAll, best, o) > best;
      bound = best && ahead < p.K ? best : 0xffffffffu;
#pragma unroll
      for (int o = 8; o; o >>= 1) bound = min(bound, __shfl_xor_sync(kAll, bound, o));
    } else {
      // that K of the lanes' two largest reach it, found by halving (the few lanes of the open groups have too
      // few maxima); 1, and so every open key, where there are fewer
      uint32_t high = best, low = next ? next : best ? best : 0xffffffffu;
#pragma unroll
      for (int o = 8; o; o >>= 1) {
        high = max(high, __shfl_xor_sync(kAll, high, o));
        low = min(low, __shfl_xor_sync(kAll, low, o));
      }
      const auto reach = [&](uint32_t v) {
        return __popc(__ballot_sync(kAll, best >= v) & half_lanes) + __popc(__ballot_sync(kAll, next >= v) & half_lanes);
      };
      bool going = reach(1) >= p.K;
      if (!going) low = 1;
      for (int i = 0; i < kBoundSteps; ++i) {
        going = going && low < high;
        if (!__any_sync(kAll, going)) break;
        const uint32_t mid = low + (high - low) / 2 + 1;
        const int n = reach(mid);
        if (going) {
          if (n >= p.K) low = mid;
          else high = mid - 1;
          going = n < p.K || n > p.K + 1;
        }
      }
      bound = low;
    }
    uint32_t in = 0;
#pragma unroll
    for (int j = 0; j < EPL; ++j) in |= (key[j] >= bound ? 1u : 0u) << j;
    int count = 0;
    for (uint32_t who; (who = __ballot_sync(kAll, in != 0)) != 0;) {
      const int at = count + __popc(who & below);
      if (in && at < 16) sc.list[half][at] = e0 + __ffs(in) - 1;
      in &= in - 1;
      count += __popc(who & half_lanes);
    }
    __syncwarp();
    int rank = 16, id = 0;
    const int most = max(count, __shfl_xor_sync(kAll, count, 16));
    if (most <= 16) {
      unsigned long long own = 0;
      if (hl < count) {
        id = sc.list[half][hl];
        own = ((unsigned long long)sc.key[half][Scratch::place(id)] << 32) | (uint32_t)~id;
      }
      sc.order[half][hl] = own;
      __syncwarp();
      rank = 0;
      for (int i = 0; i < most; i += 2) {
        const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(&sc.order[half][i]);
        rank += (o.x > own) + (o.y > own);
      }
      if (hl >= count) rank = 16;
    } else {
      for (int k = 0; k < p.K; ++k) {
        unsigned long long b = 0;  // the largest pair of key and inverted index
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
          const unsigned long long c = ((unsigned long long)key[j] << 32) | (uint32_t) ~(e0 + j);
          if (key[j] && c > b) b = c;
        }
#pragma unroll
        for (int o = 8; o; o >>= 1) {
          const unsigned long long c = __shfl_xor_sync(kAll, b, o);
          if (c > b) b = c;
        }
        const int e = (int)~(uint32_t)b;
        if (hl == k) rank = k, id = e;
#pragma unroll
        for (int j = 0; j < EPL; ++j)
          if (e0 + j == e) key[j] = 0;
      }
    }
    const bool picked = rank < p.K;
    const float at = sc.x[half][Scratch::place(id)];
    __syncwarp();
    float score;
    if (p.sigmoid) {
      score = sigmoid_of(at);  // of -inf: 0
    } else {
      const float d = __fsub_rn(at, top);
      score = sum > 0.f ? __fdiv_rn(d == d ? expf(d) : top > 0.f ? 1.f : 0.f, sum) : 0.f;
    }
    float w8 = score;
    if (p.renorm) {
      const float total = half_sum(picked ? score : 0.f);
      w8 = total > 0.f ? __fdiv_rn(score, total) : 0.f;
    }
    if (picked && there) {
      p.ids[t * p.K + rank] = id;
      p.weights[t * p.K + rank] = __fmul_rn(w8, p.scaling);
    }
  }
}

// A lane's EPL neighbouring gradients, stored at once.
template <int DT, int EPL>
__device__ __forceinline__ void store_lane(void* row, int lane, const float (&x)[EPL]) {
  constexpr int kBytes = EPL * (DT == MOE_F32 ? 4 : 2);
  alignas(16) uint32_t w[(kBytes + 3) / 4] = {};
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    if (DT == MOE_F32) w[j] = __float_as_uint(x[j]);
    else if (DT == MOE_BF16) w[j / 2] |= (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(x[j])) << (16 * (j & 1));
    else w[j / 2] |= (uint32_t)__half_as_ushort(__float2half_rn(x[j])) << (16 * (j & 1));
  }
  uint8_t* q = static_cast<uint8_t*>(row) + (size_t)lane * kBytes;
  if (kBytes >= 16) {
#pragma unroll
    for (int i = 0; i < kBytes / 16; ++i) st_v4(q + i * 16, *reinterpret_cast<int4*>(&w[i * 4]));
  } else if (kBytes == 8) {
    *reinterpret_cast<uint2*>(q) = make_uint2(w[0], w[kBytes == 8 ? 1 : 0]);
  } else if (kBytes == 4) {
    *reinterpret_cast<uint32_t*>(q) = w[0];
  } else {
    *reinterpret_cast<uint16_t*>(q) = (uint16_t)w[0];
  }
}

// A row over LANES lanes, where it does not matter which of its elements a lane has: 16
// bytes a lane in turn (neighbouring lanes' 32 bytes apart would fetch and write each
// sector twice), or a lane's neighbouring ones where they are fewer, or an element a lane in
// turn where rows are not aligned (34056 rows of 425 gradients, bf16 78 -> 44 us, fp32 67 -> 28).
// `vec` says which, so a row that is loaded and stored has the same for both.
template <int DT, int EPL, int LANES>
__device__ __forceinline__ void load_row(const void* row, int E, bool vec, int lane, float (&x)[EPL]) {
  constexpr int kVec = DT == MOE_F32 ? 4 : 8;
  if constexpr (EPL % kVec == 0) {
    if (vec) {
#pragma unroll
      for (int i = 0; i < EPL / kVec; ++i) {
        float part[kVec];
        load_lane<DT, kVec>(static_cast<const uint8_t*>(row) + i * LANES * 16, E, true, lane, part);
#pragma unroll
        for (int j = 0; j < kVec; ++j) x[i * kVec + j] = part[j];
      }
      return;
    }
  }
  if (vec) {
    load_lane<DT, EPL>(row, E, true, lane, x);
    return;
  }
#pragma unroll
  for (int j = 0; j < EPL; ++j) x[j] = j * LANES + lane < E ? load_logit<DT>(row, j * LANES + lane) : -INFINITY;
}
template <int DT, int EPL, int LANES>
__device__ __forceinline__ void store_row(void* row, int E, bool vec, int lane, const float (&x)[EPL]) {
  constexpr int kVec = DT == MOE_F32 ? 4 : 8;
  if constexpr (EPL % kVec == 0) {
    if (vec) {
#pragma unroll
      for (int i = 0; i < EPL / kVec; ++i) {
        float part[kVec];
#pragma unroll
        for (int j = 0; j < kVec; ++j) part[j] = x[i * kVec + j];
        store_lane<DT, kVec>(static_cast<uint8_t*>(row) + i * LANES * 16, lane, part);
      }
      return;
    }
  }
  if (vec) {
    store_lane<DT, EPL>(row, lane, x);
    return;
  }
#pragma unroll
  for (int j = 0; j < EPL; ++j)
    if (j * LANES + lane < E) store_logit<DT>(row, j * LANES + lane, x[j]);
}

template <int LANES>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
  for (int o = LANES / 2; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(kAll, v, o));
  return v;
}

// exp(x - top); an expert that is masked out has none, and +inf ones share the sum.
__device__ __forceinline__ float exp_below(float x, float top) {
  const float d = __fsub_rn(x, top);
  return d == d ? expf(d) : top > 0.f ? 1.f : 0.f;
}

// The gradient: LANES lanes (a warp, or half of one for large batches, where what a
// token costs beside its row counts) write a token's whole row (zeros, or the softmax's
// share in every expert), then the lanes that hold its picks write theirs over it.
// Each logit is read once at most, each gradient written once. 65536 x 256 fp32 softmax
// logits, every gradient: 29 us, 4.7 TB/s (a warp a token 31 us; with one side's rows not
// aligned 31 us, the aligned batch 26 us beside it). Neither HBM (71% of a copy's rate) nor the
// issue slots (66%) are full: a third of the warps are resident, and a token's chain of
// loads, exponentials and reductions is what they wait for.
template <int DT, int EPL, int LANES>
__global__ void __launch_bounds__(kRouterWarps * 32, LANES == 16 ? 6 : 1) route_grad_kernel(RouterParams p) {
  const int lane = threadIdx.x & (LANES - 1);
  pdl_wait();
  pdl_launch_dependents();
  const bool dense = !p.sigmoid && !p.renorm;
  const long long step = (long long)gridDim.x * (kRouterWarps * 32 / LANES);
  // a token's row, picks and their gradients are loaded while the one before is worked
  // on, its chosen logits at the end of that
  long long t = (long long)blockIdx.x * (kRouterWarps * 32 / LANES) + threadIdx.x / LANES;
  float ahead[EPL];
  int id_ahead = -1;
  float g_ahead = 0.f, raw_ahead = -INFINITY;
  const auto load = [&](long long k) {
    if (k >= p.T) return;
    if (dense) load_row<DT, EPL, LANES>(logit_row<DT>(p.logits, k, p.stride), p.E, p.vec, lane, ahead);
    if (lane < p.K) {
      id_ahead = __ldg(p.ids_in + k * p.K + lane);
      g_ahead = __ldg(p.grad + k * p.K + lane);
    }
  };
  const auto load_chosen = [&](long long k) {
    if (k < p.T && (unsigned)id_ahead < (unsigned)p.E) raw_ahead = load_logit<DT>(logit_row<DT>(p.logits, k, p.stride), id_ahead);
  };
  load(t);
  load_chosen(t);
  // the warp stays together: its last token may be missing
  for (long long first = t - (threadIdx.x & 31) / LANES; first < p.T; first += step, t += step) {
    const bool there = t < p.T;
    uint8_t* out = static_cast<uint8_t*>(p.grad_logits) + t * p.grad_stride * (DT == MOE_F32 ? 4 : 2);
    float v[EPL];
    if (dense) {
#pragma unroll
      for (int j = 0; j < EPL; ++j) v[j] = fmaxf(ahead[j], -INFINITY);  // NaN becomes -inf
    }
    const int id = there && lane < p.K && (unsigned)id_ahead < (unsigned)p.E ? id_ahead : -1;
    const float x = id >= 0 ? fmaxf(raw_ahead, -INFINITY) : -INFINITY;
    // a masked pick's weight is 0 whatever the logits: nothing of its gradient, infinite or NaN, reaches the others
    const float g = x > -INFINITY ? __fmul_rn(g_ahead, p.scaling) : 0.f;
    load(t + step);
    float d;
    if (p.sigmoid) {
      const float s = sigmoid_of(x), other = sigmoid_of(-x);  // 1 - s without the cancellation near s = 1
      if (p.renorm) {
        const float total = lanes_sum<LANES>(s);
        const float r = total > 0.f ? __fdiv_rn(s, total) : 0.f;
        d = r * (g - lanes_sum<LANES>(g * r)) * other;
      } else {
        d = g * s * other;
      }
    } else {
      // the chosen logits alone when renormalised, else the whole row
      float top = x, sum = 0.f;
      if (dense) {
#pragma unroll
        for (int j = 0; j < EPL; ++j) top = fmaxf(top, v[j]);
      }
      top = lanes_max<LANES>(top);
      const float mine = exp_below(x, top);
      if (dense) {
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
          v[j] = exp_below(v[j], top);
          sum += v[j];
        }
      } else {
        sum = mine;
      }
      sum = lanes_sum<LANES>(sum);
      const float r = sum > 0.f ? __fdiv_rn(mine, sum) : 0.f;
      const float mean = lanes_sum<LANES>(g * r);
      d = r * (g - mean);
      if (dense) {
        const float share = sum > 0.f ? -__fdiv_rn(mean, sum) : 0.f;
#pragma unroll
        for (int j = 0; j < EPL; ++j) v[j] *= share;
      }
    }
    if (!dense) {
#pragma unroll
      for (int j = 0; j < EPL; ++j) v[j] = 0.f;
    }
    if (there) store_row<DT, EPL, LANES>(out, p.E, p.vec, lane, v);
    __syncwarp();
    if (id >= 0) store_logit<DT>(out, id, d);
    load_chosen(t + step);
  }
}

namespace {

moe_status_t check_router(const moe_router_config_t* c) {
  if (!c) return MOE_ERR_INVALID_ARG;
  if (c->tokens < 0 || c->expert_num < 1 || c->expert_num > 1024 || c->topk < 1 || c->topk > 32)
    return MOE_ERR_INVALID_ARG;
  if (c->group_num < 1 || c->group_num > c->expert_num || c->expert_num % c->group_num) return MOE_ERR_INVALID_ARG;
  if (c->topk_group < 1 || c->topk_group > c->group_num) return MOE_ERR_INVALID_ARG;
  if (c->topk > c->topk_group * (c->expert_num / c->group_num)) return MOE_ERR_INVALID_ARG;
  if (c->group_score < MOE_GROUP_MAX || c->group_score > MOE_GROUP_TOP2_SUM) return MOE_ERR_INVALID_ARG;
  if (c->score_func < MOE_SCORE_SOFTMAX || c->score_func > MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARG;
  if (c->renormalize < 0 || c->renormalize > 1) return MOE_ERR_INVALID_ARG;
  if (c->logits_dtype != MOE_F32 && c->logits_dtype != MOE_F16 && c->logits_dtype != MOE_BF16)
    return MOE_ERR_INVALID_ARG;
  if (!isfinite(c->scaling) || c->logits_stride < c->expert_num) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

bool aligned_to(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

RouterParams params_of(const moe_router_config_t* c) {
  RouterParams p{};
  p.T = c->tokens;
  p.T_step = 1;
  p.E = c->expert_num;
  p.K = c->topk;
  p.G = c->group_num;
  p.KG = c->topk_group;
  p.top2 = c->group_num > 1 && c->group_score == MOE_GROUP_TOP2_SUM;
  p.sigmoid = c->score_func == MOE_SCORE_SIGMOID;
  p.renorm = c->renormalize;
  p.scaling = c->scaling;
  p.stride = c->logits_stride;
  return p;
}

typedef void (*RouterKernel)(RouterParams);

// Experts a lane: the least power of two that 32 lanes cover E with.
int lane_experts(int E) {
  int n = 1;
  while (32 * n < E) n *= 2;
  return n;
}

template <int DT>
RouterKernel route_of(int epl) {
  switch (epl) {
    case 1: return route_kernel<DT, 1>;
    case 2: return route_kernel<DT, 2>;
    case 4: return route_kernel<DT, 4>;
    case 8: return route_kernel<DT, 8>;
    default: return route_kernel<DT, 16>;
  }
}
template <int DT>
RouterKernel route_pair_of(int epl) {
  return epl == 4 ? route_pair_kernel<DT, 4> : epl == 8 ? route_pair_kernel<DT, 8> : route_pair_kernel<DT, 16>;
}
template <int DT>
RouterKernel route_grad_of(int epl) {
  switch (epl) {
    case 1: return route_grad_kernel<DT, 1, 32>;
    case 2: return route_grad_kernel<DT, 2, 32>;
    case 4: return route_grad_kernel<DT, 4, 32>;
    case 8: return route_grad_kernel<DT, 8, 32>;
    case 16: return route_grad_kernel<DT, 16, 32>;
    default: return route_grad_kernel<DT, 32, 32>;
  }
}
template <int DT>
RouterKernel route_grad_pair_of(int epl) {
  return epl == 4 ? route_grad_kernel<DT, 4, 16> : epl == 8 ? route_grad_kernel<DT, 8, 16> : route_grad_kernel<DT, 16, 16>;
}

// Whether a lane's EPL elements load or store at once.
bool whole_lanes(const void* base, int64_t stride, int E, int epl, int es, int lanes = 32) {
  const size_t bytes = (size_t)epl * es, align = bytes < 16 ? bytes : 16;
  return E == lanes * epl && aligned_to(base, align) && (size_t)stride * es % align == 0;
}

moe_status_t launch(RouterKernel kernel, const RouterParams& p, size_t smem, void* stream) {
  const int nsm = num_sms_of_current_device();
  int per_sm = 0;
  if (nsm <= 0 || resident_blocks((const void*)kernel, kRouterWarps * 32, smem, &per_sm) != cudaSuccess || per_sm < 1)
    return MOE_ERR_CUDA;
  const int tokens = kRouterWarps * p.T_step;
  const long long need = ((long long)p.T + tokens - 1) / tokens, most = (long long)nsm * per_sm;
  PdlLaunch L(dim3((unsigned)(need < most ? need : most)), dim3(kRouterWarps * 32), smem,
              static_cast<cudaStream_t>(stream));
  if (cudaLaunchKernelEx(&L.cfg, kernel, p) != cudaSuccess) return MOE_ERR_CUDA;
  note_launches(1);
  return MOE_OK;
}

}  // namespace
}  // namespace crs

extern "C" moe_status_t moe_route(const moe_router_config_t* rc, const void* logits, const float* bias,
                                  int32_t* expert_ids, float* expert_scales, void* stream) {
  using namespace crs;
  const moe_status_t st = check_router(rc);
  if (st != MOE_OK) return st;
  const size_t es = rc->logits_dtype == MOE_F32 ? 4 : 2;
  if (rc->tokens > 0 && (!logits || !expert_ids || !expert_scales)) return MOE_ERR_INVALID_ARG;
  if (!aligned_to(logits, es) || !aligned_to(bias, 4) || !aligned_to(expert_ids, 4) || !aligned_to(expert_scales, 4))
    return MOE_ERR_INVALID_ARG;
  if (rc->tokens == 0) return MOE_OK;
  RouterParams p = params_of(rc);
  p.logits = logits;
  p.bias = bias;
  p.ids = expert_ids;
  p.weights = expert_scales;
  const int epl = lane_experts(p.E);
  p.vec = whole_lanes(logits, p.stride, p.E, epl, (int)es);
  const int pair_epl = 2 * epl;
  if (p.T >= kPairTokens && p.K <= 16 && pair_epl >= 4 && pair_epl <= 16 && 16 % p.G == 0 &&
      whole_lanes(logits, p.stride, p.E, pair_epl, (int)es, 16)) {
    p.T_step = 2;
    return launch(rc->logits_dtype == MOE_F32   ? route_pair_of<MOE_F32>(pair_epl)
                  : rc->logits_dtype == MOE_F16 ? route_pair_of<MOE_F16>(pair_epl)
                                                : route_pair_of<MOE_BF16>(pair_epl),
                  p, 0, stream);
  }
  // over 512 experts, or groups that do not fall on lanes
  if (epl > 16 || (p.G > 1 && (p.E != 32 * epl || 32 % p.G))) {
    const size_t smem = (size_t)kRouterWarps * (2 * p.E + p.G) * 4;
    return launch(rc->logits_dtype == MOE_F32   ? route_any_kernel<MOE_F32>
                  : rc->logits_dtype == MOE_F16 ? route_any_kernel<MOE_F16>
                                                : route_any_kernel<MOE_BF16>,
                  p, smem, stream);
  }
  return launch(rc->logits_dtype == MOE_F32   ? route_of<MOE_F32>(epl)
                : rc->logits_dtype == MOE_F16 ? route_of<MOE_F16>(epl)
                                              : route_of<MOE_BF16>(epl),
                p, 0, stream);
}

extern "C" moe_status_t moe_route_backward(const moe_router_config_t* rc, const void* logits,
                                           const int32_t* expert_ids, const float* grad_scales, void* grad_logits,
                                           int64_t grad_stride, void* stream) {
  using namespace crs;
  const moe_status_t st = check_router(rc);
  if (st != MOE_OK) return st;
  const size_t es = rc->logits_dtype == MOE_F32 ? 4 : 2;
  if (grad_stride < rc->expert_num) return MOE_ERR_INVALID_ARG;
  if (rc->tokens > 0 && (!logits || !expert_ids || !grad_scales || !grad_logits)) return MOE_ERR_INVALID_ARG;
  if (!aligned_to(logits, es) || !aligned_to(grad_logits, es) || !aligned_to(expert_ids, 4) ||
      !aligned_to(grad_scales, 4))
    return MOE_ERR_INVALID_ARG;
  if (rc->tokens == 0) return MOE_OK;
  RouterParams p = params_of(rc);
  p.logits = logits;
  p.ids_in = expert_ids;
  p.grad = grad_scales;
  p.grad_logits = grad_logits;
  p.grad_stride = grad_stride;
  // the softmax's gradient loads the row that it stores: both in whole lanes, or neither
  const bool dense = !p.sigmoid && !p.renorm;
  const auto whole = [&](int epl, int lanes) {
    return whole_lanes(grad_logits, grad_stride, p.E, epl, (int)es, lanes) &&
           (!dense || whole_lanes(logits, p.stride, p.E, epl, (int)es, lanes));
  };
  const int epl = lane_experts(p.E), pair_epl = 2 * epl;
  if (p.T >= (pair_epl > 8 ? kGradPairTokensWide : kGradPairTokens) && p.K <= 16 && pair_epl >= 4 && pair_epl <= 16 &&
      whole(pair_epl, 16)) {
    p.T_step = 2;
    p.vec = 1;
    return launch(rc->logits_dtype == MOE_F32   ? route_grad_pair_of<MOE_F32>(pair_epl)
                  : rc->logits_dtype == MOE_F16 ? route_grad_pair_of<MOE_F16>(pair_epl)
                                                : route_grad_pair_of<MOE_BF16>(pair_epl),
                  p, 0, stream);
  }
  p.vec = whole(epl, 32);
  return launch(rc->logits_dtype == MOE_F32   ? route_grad_of<MOE_F32>(epl)
                : rc->logits_dtype == MOE_F16 ? route_grad_of<MOE_F16>(epl)
                                              : route_grad_of<MOE_BF16>(epl),
                p, 0, stream);
}

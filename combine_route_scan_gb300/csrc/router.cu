// Routing scores to expert ids and weights (moe_route) and the gradient of the
// weights (moe_route_backward); include/moe_experts.h has the formulas.
//
// One warp a token, its keys and scores in shared memory: softmax statistics,
// group values and each of the topk argmax steps are warp reductions.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "../../include/moe_experts.h"
#include "common.cuh"

namespace crs {

constexpr int kRouterWarps = 4;
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
  float scaling;
};

// Keys as unsigned integers that order like the floats: -inf (masked and NaN
// keys) stays above 0, which stands for an expert that cannot be picked.
constexpr uint32_t kMaskedKey = 0x007fffffu;
__device__ __forceinline__ uint32_t ordered_key(float f) {
  if (f != f) return kMaskedKey;
  const uint32_t b = __float_as_uint(__fadd_rn(f, 0.f));  // -0 and +0 are equal keys
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
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

__device__ __forceinline__ float sigmoid_of(float x) { return __fdiv_rn(1.f, __fadd_rn(1.f, expf(-x))); }

// The index of the largest key among a lane's best (key, index) pairs, the
// lowest index among equal keys.
__device__ __forceinline__ int warp_argmax(uint32_t key, int index, uint32_t* best) {
  const uint32_t m = __reduce_max_sync(kAll, key);
  *best = m;
  return __reduce_min_sync(kAll, key == m ? (unsigned)index : 0x7fffffffu);
}

template <int DT>
__global__ void __launch_bounds__(kRouterWarps * 32) route_scores_kernel(RouterParams p) {
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

template <int DT>
__global__ void __launch_bounds__(kRouterWarps * 32) route_grad_kernel(RouterParams p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();
  for (long long t = (long long)blockIdx.x * kRouterWarps + warp; t < p.T; t += (long long)gridDim.x * kRouterWarps) {
    const void* row = logit_row<DT>(p.logits, t, p.stride);
    uint8_t* out = static_cast<uint8_t*>(p.grad_logits) + t * p.grad_stride * (DT == MOE_F32 ? 4 : 2);
    int id = lane < p.K ? p.ids_in[t * p.K + lane] : -1;
    if (id >= p.E) id = -1;
    const float g = id >= 0 ? __fmul_rn(p.grad[t * p.K + lane], p.scaling) : 0.f;
    const float raw = id >= 0 ? load_logit<DT>(row, id) : -INFINITY;
    const float x = raw == raw ? raw : -INFINITY;
    float top = -INFINITY, sum = 0.f, d = 0.f;
    if (p.sigmoid) {
      const float s = x == -INFINITY ? 0.f : sigmoid_of(x);
      const float other = x == -INFINITY ? 1.f : sigmoid_of(-x);  // 1 - s without the cancellation near s = 1
      if (p.renorm) {
        const float total = warp_sum(s);
        const float r = total > 0.f ? __fdiv_rn(s, total) : 0.f;
        const float mean = warp_sum(g * r);
        d = r * (g - mean) * other;
      } else {
        d = g * s * other;
      }
    } else {
      // the chosen logits alone when renormalised, else the whole row
      if (p.renorm) {
        top = warp_max(x);
      } else {
        for (int e = lane; e < p.E; e += 32) {
          const float v = load_logit<DT>(row, e);
          top = fmaxf(top, v);
        }
        top = warp_max(top);
        for (int e = lane; e < p.E; e += 32) {
          const float v = load_logit<DT>(row, e);
          sum += v == -INFINITY || v != v ? 0.f : v == top ? 1.f : expf(v - top);
        }
        sum = warp_sum(sum);
      }
      const float v = x == -INFINITY ? 0.f : x == top ? 1.f : expf(x - top);
      if (p.renorm) sum = warp_sum(v);
      const float r = sum > 0.f ? __fdiv_rn(v, sum) : 0.f;
      const float mean = warp_sum(g * r);
      d = r * (g - mean);
      if (!p.renorm) {
        for (int e = lane; e < p.E; e += 32) {
          const float l = load_logit<DT>(row, e);
          const float ve = l == -INFINITY || l != l ? 0.f : l == top ? 1.f : expf(l - top);
          store_logit<DT>(out, e, sum > 0.f ? -mean * __fdiv_rn(ve, sum) : 0.f);
        }
      }
    }
    if (p.sigmoid || p.renorm)
      for (int e = lane; e < p.E; e += 32) store_logit<DT>(out, e, 0.f);
    __syncwarp();
    if (id >= 0) store_logit<DT>(out, id, d);
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

moe_status_t launch(RouterKernel kernel, const RouterParams& p, size_t smem, void* stream) {
  const int nsm = num_sms_of_current_device();
  int per_sm = 0;
  if (nsm <= 0 || resident_blocks((const void*)kernel, kRouterWarps * 32, smem, &per_sm) != cudaSuccess || per_sm < 1)
    return MOE_ERR_CUDA;
  const long long need = ((long long)p.T + kRouterWarps - 1) / kRouterWarps, most = (long long)nsm * per_sm;
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
  const size_t smem = (size_t)kRouterWarps * (2 * p.E + p.G) * 4;
  return launch(rc->logits_dtype == MOE_F32   ? route_scores_kernel<MOE_F32>
                : rc->logits_dtype == MOE_F16 ? route_scores_kernel<MOE_F16>
                                              : route_scores_kernel<MOE_BF16>,
                p, smem, stream);
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
  return launch(rc->logits_dtype == MOE_F32   ? route_grad_kernel<MOE_F32>
                : rc->logits_dtype == MOE_F16 ? route_grad_kernel<MOE_F16>
                                              : route_grad_kernel<MOE_BF16>,
                p, 0, stream);
}

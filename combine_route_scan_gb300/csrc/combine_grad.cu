// The gradient of combine (moe_combine_backward; include/moe_experts.h). With g the
// gradient of x_out[token] and y_k, w_k a routed pick's expert-output row and weight:
//   grad_expert_out[row of k] = w_k * g,   grad_scales[token, k] = <g, y_k>,
// and a copy pick adds w_k to the factor of grad_x[token] = (sum of w_k) * g, with
// <g, x> as its weight's gradient.
//
// A block has one token, so that g is read once for all of its picks (from expert to
// expert, row after row, it would come K times from L2), and goes through the row's
// 16-byte vectors with the loads of up to 8 picks in flight; the products' sums stay
// in registers and are joined over the lanes and then the warps in a fixed order.
// The rows come from the pick -> row map of the dispatch, checked against assist_info as combine's reduce does, or, where
// the workspace has no such map, by looking through assist_info (rows.cuh). Bound by HBM: the tokens and the rows,
// read, and the rows, written: 4096 tokens of hidden 7168 with 27000 rows 150 us, 5.9 TB/s.
#include "rows.cuh"

namespace crs {

constexpr int kGradBatch = 8;     // picks whose loads are in flight together
constexpr int kGradThreads = 256; // at most

// VEC: rows of 16-byte vectors; else an element at a time. SEARCH: without a row map (rows.cuh).
template <int DT, bool VEC, bool SEARCH>
__global__ void __launch_bounds__(kGradThreads, 4) combine_grad_kernel(CombineGradParams p, int active) {
  __shared__ const uint8_t* s_src[32];
  __shared__ uint8_t* s_dst[32];
  __shared__ float s_w[32];
  __shared__ int s_pick[32];
  __shared__ float s_dot[kGradThreads / 32][kGradBatch];
  __shared__ int s_n;
  __shared__ float s_copy;
  __shared__ bool s_copies;
  __shared__ long long s_row[SEARCH ? 32 : 1];
  const Shape sh = p.sh;
  // the threads that go through the row: with a map or without, sums have one order
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = active >> 5;
  const size_t begin = (int)threadIdx.x < active ? threadIdx.x : (size_t)1 << 32;
  const size_t tau = blockIdx.x;
  pdl_wait();
  pdl_launch_dependents();

  if (SEARCH) find_rows(p, tau, s_row);
  // the token's contributing picks, in ascending k; every block of the token has all
  // of them and takes its own batches
  long long r = -1;
  int d = -1;
  bool check = false;
  if (warp == 0) {
    const uint8_t* src = nullptr;
    uint8_t* dst = nullptr;
    float w = 0.f;
    bool has = false, copies = false;
    const int cls = lane < sh.K ? classify_pick(p.ids, p.mask, sh, tau, lane) : kPickInactive;
    if (lane < sh.K) {
      const size_t pk = tau * sh.K + lane;
      r = SEARCH ? s_row[lane] : (long long)p.inv[pk];
      w = static_cast<const float*>(p.scales)[pk];
      if (cls >= 0) {
        d = cls / sh.L;
        const long long row = r - (long long)d * sh.A;
        if (row >= 0 && row < sh.A && MOE_IN_BOUNDS(p.status, r, (long long)sh.W * sh.A)) {
          src = static_cast<const uint8_t*>(p.expert_out) + r * (long long)sh.row_in;
          if (p.grad_rows) dst = static_cast<uint8_t*>(p.grad_rows) + r * (long long)sh.row_in;
          has = true;
          check = !SEARCH;
        } else {
          set_error(p.status, MOE_ERR_BAD_ASSIST);
        }
      } else if (cls == kPickCopy) {
        src = static_cast<const uint8_t*>(p.x) + tau * (size_t)sh.row_in;
        has = copies = true;
      } else if (cls == kPickBad) {
        set_error(p.status, MOE_ERR_BAD_EXPERT_ID);
      }
      if (!has && p.grad_scales && blockIdx.y == 0) p.grad_scales[pk] = 0.f;
    }
    const uint32_t m = __ballot_sync(0xffffffffu, has);
    if (has) {
      const int j = __popc(m & lanemask_lt());
      s_src[j] = src;
      s_dst[j] = dst;
      s_w[j] = w;
      s_pick[j] = lane;
    }
    // the copies' weights, k ascending
    uint32_t left = __ballot_sync(0xffffffffu, copies);
    if (lane == 0) {
      s_n = __popc(m);
      s_copies = left != 0;
    }
    float total = 0.f;
    for (; left; left &= left - 1) total += __shfl_sync(0xffffffffu, w, __ffs(left) - 1);
    if (lane == 0) s_copy = total;
  }
  __syncthreads();
  const int n = s_n;

  // a row is what assist_info says: asked now, compared last
  int a0 = 0, a1 = 0, a2 = 0, cnt = 0;
  check = check && blockIdx.y == 0;
  if (check) {
    const int32_t* a = p.assist + r * 3;
    a0 = a[0];
    a1 = a[1];
    a2 = a[2];
    cnt = p.ep_recv_count[(size_t)d * sh.L * sh.W + sh.L * sh.W - 1];
  }

  const size_t row0 = tau * (size_t)sh.row_in;
  const uint8_t* g_row = static_cast<const uint8_t*>(p.grad_out) + row0;
  const bool dots = p.grad_scales != nullptr;
  constexpr int kStep = VEC ? 16 : 2;  // bytes a thread takes at a time
  for (int j0 = blockIdx.y * kGradBatch; j0 < n; j0 += gridDim.y * kGradBatch) {
    const int here = min(kGradBatch, n - j0);
    float acc[kGradBatch];
#pragma unroll
    for (int j = 0; j < kGradBatch; ++j) acc[j] = 0.f;
    for (size_t off = begin * kStep; off < (size_t)sh.row_in; off += (size_t)active * kStep) {
      if constexpr (VEC) {
        int4 y[kGradBatch];
        const int4 gv = ld_nc_v4(g_row + off);
#pragma unroll
        for (int j = 0; j < kGradBatch; ++j)
          if (dots && j < here) y[j] = ld_nc_v4(s_src[j0 + j] + off);
        float g[8];
        Vec<DT>::unpack(g, gv);
#pragma unroll
        for (int j = 0; j < kGradBatch; ++j) {
          if (j >= here) break;
          uint8_t* dst = s_dst[j0 + j];
          if (dst) {
            const float w = s_w[j0 + j];
            float o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = __fmul_rn(w, g[i]);
            __stcs(reinterpret_cast<int4*>(dst + off), Vec<DT>::pack(o));
          }
          if (dots) {
            float f[8];
            Vec<DT>::unpack(f, y[j]);
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[j] = __fmaf_rn(g[i], f[i], acc[j]);
          }
        }
      } else {
        const float g = elem_to_float<DT>(*reinterpret_cast<const uint16_t*>(g_row + off));
#pragma unroll
        for (int j = 0; j < kGradBatch; ++j) {
          if (j >= here) break;
          uint8_t* dst = s_dst[j0 + j];
          if (dst) *reinterpret_cast<uint16_t*>(dst + off) = float_to_elem<DT>(__fmul_rn(s_w[j0 + j], g));
          if (dots) acc[j] = __fmaf_rn(g, elem_to_float<DT>(*reinterpret_cast<const uint16_t*>(s_src[j0 + j] + off)), acc[j]);
        }
      }
    }
    if (dots) {
#pragma unroll
      for (int j = 0; j < kGradBatch; ++j) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], o);
      }
      __syncthreads();  // the batch before has read s_dot
#pragma unroll
      for (int j = 0; j < kGradBatch; ++j)
        if (lane == j) s_dot[warp][j] = acc[j];
      __syncthreads();
      if ((int)threadIdx.x < here) {
        float sum = 0.f;
        for (int v = 0; v < warps; ++v) sum += s_dot[v][threadIdx.x];
        p.grad_scales[tau * sh.K + s_pick[j0 + threadIdx.x]] = sum;
      }
    }
  }

  if (p.grad_x && blockIdx.y == 0) {
    const float w = s_copy;
    const bool some = s_copies;  // without one grad_out is not read: zeros, whatever it holds
    uint8_t* out = static_cast<uint8_t*>(p.grad_x) + row0;
    for (size_t off = begin * kStep; off < (size_t)sh.row_in; off += (size_t)active * kStep) {
      if constexpr (VEC) {
        float g[8];
        if (some) {
          Vec<DT>::unpack(g, ld_nc_v4(g_row + off));
#pragma unroll
          for (int i = 0; i < 8; ++i) g[i] = __fmul_rn(w, g[i]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) g[i] = 0.f;
        }
        st_v4(out + off, Vec<DT>::pack(g));
      } else {
        const float g = some ? __fmul_rn(w, elem_to_float<DT>(*reinterpret_cast<const uint16_t*>(g_row + off))) : 0.f;
        *reinterpret_cast<uint16_t*>(out + off) = float_to_elem<DT>(g);
      }
    }
  }

  if (check) {
    const int s = (int)(tau / sh.bs), t = (int)(tau % sh.bs);
    if (a0 != s || a1 != t || a2 != lane || r - (long long)d * sh.A >= cnt) set_error(p.status, MOE_ERR_BAD_ASSIST);
  }
}

// Dispatch's gradient where a batch is too small for a row map to pay: a block has one token, as above.
template <int DT, bool VEC>
__global__ void __launch_bounds__(kGradThreads) dispatch_grad_token_kernel(DispatchGradParams p) {
  __shared__ const uint8_t* s_src[32];
  __shared__ long long s_row[32];
  __shared__ int s_n;
  const Shape sh = p.sh;
  const int lane = threadIdx.x & 31;
  const size_t tau = blockIdx.x;
  pdl_wait();
  pdl_launch_dependents();
  find_rows(p, tau, s_row);
  if (threadIdx.x < 32) {
    const uint8_t* src = nullptr;
    if (lane < sh.K) {
      const int cls = classify_pick(p.ids, p.mask, sh, tau, lane);
      const long long r = s_row[lane];
      if (cls >= 0 && r >= 0 && MOE_IN_BOUNDS(p.status, r, (long long)sh.W * sh.A)) {
        src = static_cast<const uint8_t*>(p.expert_out) + r * (long long)sh.row_in;
      } else if (cls >= 0 || cls == kPickBad) {
        set_error(p.status, cls >= 0 ? MOE_ERR_BAD_ASSIST : MOE_ERR_BAD_EXPERT_ID);
      }
      if (p.pick_weights) p.pick_weights[tau * sh.K + lane] = src ? p.row_weights[r] : 0.f;
    }
    const uint32_t m = __ballot_sync(0xffffffffu, src != nullptr);
    if (src) s_src[__popc(m & lanemask_lt())] = src;
    if (lane == 0) s_n = __popc(m);
  }
  __syncthreads();
  const int n = s_n;
  const size_t row0 = tau * (size_t)sh.row_in;
  const uint8_t* residual = p.residual ? static_cast<const uint8_t*>(p.residual) + row0 : nullptr;
  uint8_t* out = static_cast<uint8_t*>(p.x_out) + row0;
  constexpr int kStep = VEC ? 16 : 2;
  for (size_t off = (size_t)threadIdx.x * kStep; off < (size_t)sh.row_in; off += (size_t)blockDim.x * kStep) {
    if constexpr (VEC) {
      float acc[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = 0.f;
      // an ordinary load: the residual may be what this thread then writes
      if (residual) Vec<DT>::fma(acc, 1.f, ld_v4(residual + off));
      for (int j0 = 0; j0 < n; j0 += kGradBatch) {
        int4 y[kGradBatch];
#pragma unroll
        for (int j = 0; j < kGradBatch; ++j)
          if (j0 + j < n) y[j] = ld_nc_v4(s_src[j0 + j] + off);
#pragma unroll
        for (int j = 0; j < kGradBatch; ++j)
          if (j0 + j < n) Vec<DT>::fma(acc, 1.f, y[j]);
      }
      st_v4(out + off, Vec<DT>::pack(acc));
    } else {
      float acc = residual ? elem_to_float<DT>(*reinterpret_cast<const uint16_t*>(residual + off)) : 0.f;
      for (int j = 0; j < n; ++j) acc += elem_to_float<DT>(*reinterpret_cast<const uint16_t*>(s_src[j] + off));
      *reinterpret_cast<uint16_t*>(out + off) = float_to_elem<DT>(acc);
    }
  }
}

// As few threads as go through a row in as many steps as 256 would; where rows are looked for, a warp for each pick.
static int grad_threads(const Shape& sh, bool search) {
  const int items = sh.row_in % 16 == 0 ? sh.row_in / 16 : sh.h;
  const int steps = (items + kGradThreads - 1) / kGradThreads;
  const int threads = ((items + steps - 1) / steps + 31) / 32 * 32, picks = 32 * (sh.K < 8 ? sh.K : 8);
  return search && threads < picks ? picks : threads;
}

template <bool SEARCH>
static cudaError_t launch_grad(const CombineGradParams& p, cudaStream_t st, int num_sms) {
  const Shape& sh = p.sh;
  const long long n_tok = (long long)sh.W * sh.bs;
  if (n_tok == 0) return cudaSuccess;
  const int batches = (sh.K + kGradBatch - 1) / kGradBatch, active = grad_threads(sh, false);
  PdlLaunch L(dim3((unsigned)n_tok, (unsigned)(n_tok < num_sms * 4LL ? batches : 1)), dim3(grad_threads(sh, SEARCH)), 0, st);
  if (sh.row_in % 16 == 0)
    return sh.x_dtype == MOE_F16 ? cudaLaunchKernelEx(&L.cfg, combine_grad_kernel<MOE_F16, true, SEARCH>, p, active)
                                 : cudaLaunchKernelEx(&L.cfg, combine_grad_kernel<MOE_BF16, true, SEARCH>, p, active);
  return sh.x_dtype == MOE_F16 ? cudaLaunchKernelEx(&L.cfg, combine_grad_kernel<MOE_F16, false, SEARCH>, p, active)
                               : cudaLaunchKernelEx(&L.cfg, combine_grad_kernel<MOE_BF16, false, SEARCH>, p, active);
}

cudaError_t launch_combine_grad(const CombineGradParams& p, bool search, cudaStream_t st, int num_sms) {
  return search ? launch_grad<true>(p, st, num_sms) : launch_grad<false>(p, st, num_sms);
}

cudaError_t launch_dispatch_grad(const DispatchGradParams& p, bool search, cudaStream_t st, int num_sms) {
  if (!search) return launch_dispatch_grad_reduce(p, st, num_sms);
  const Shape& sh = p.sh;
  PdlLaunch L(dim3((unsigned)(sh.W * sh.bs)), dim3(grad_threads(sh, true)), 0, st);
  if (sh.row_in % 16 == 0)
    return sh.x_dtype == MOE_F16 ? cudaLaunchKernelEx(&L.cfg, dispatch_grad_token_kernel<MOE_F16, true>, p)
                                 : cudaLaunchKernelEx(&L.cfg, dispatch_grad_token_kernel<MOE_BF16, true>, p);
  return sh.x_dtype == MOE_F16 ? cudaLaunchKernelEx(&L.cfg, dispatch_grad_token_kernel<MOE_F16, false>, p)
                               : cudaLaunchKernelEx(&L.cfg, dispatch_grad_token_kernel<MOE_BF16, false>, p);
}

}  // namespace crs

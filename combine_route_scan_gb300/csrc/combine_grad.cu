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
// The rows come from the pick -> row map of the dispatch, checked against assist_info
// as combine's reduce does, or, where the workspace has no such map, by looking
// through assist_info. Bound by HBM: the tokens and the rows, read, and the
// rows, written: 4096 tokens of hidden 7168 with 27000 rows 143 us, 6.3 TB/s. A small
// batch is one block's chain of steps: 16 tokens of hidden 256 4.1 us.
//
// Rows that do not align to 16 bytes are taken in pieces of 8, 4 or 2 bytes, eight
// elements a thread at a time: 2048 tokens of hidden 2048 29 us, 2044 38, 2046 43, 2047
// 64 (an element at a time 117).
#include "gradients.h"
#include "rows.cuh"

namespace crs {

constexpr int kGradBatch = 8;     // picks whose loads are in flight together
constexpr int kGradThreads = 256; // at most

// 8 elements of a row in pieces of BYTES (16, 8, 4 or 2), `apart` bytes from one another from `off` on; those beyond the
// row's end are zeros, and not stored. load_own: of what the kernel may write too.
template <int BYTES>
struct RowUnit {
  static constexpr int kPieces = 16 / BYTES;
  template <class F>
  static __device__ __forceinline__ int4 gather(uint32_t off, uint32_t apart, uint32_t end, F read) {
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < kPieces; ++q) {
      const uint32_t at = off + q * apart;
      if constexpr (BYTES == 8) {
        const uint2 v = at < end ? read(at, uint2{}) : uint2{0, 0};
        w[2 * q] = v.x, w[2 * q + 1] = v.y;
      } else if constexpr (BYTES == 4) {
        w[q] = at < end ? read(at, uint32_t{}) : 0u;
      } else {
        const uint32_t v = at < end ? (uint32_t)read(at, uint16_t{}) : 0u;
        if (q & 1) w[q / 2] |= v << 16;
        else w[q / 2] = v;
      }
    }
    return make_int4((int)w[0], (int)w[1], (int)w[2], (int)w[3]);
  }
  static __device__ __forceinline__ int4 load(const uint8_t* row, uint32_t off, uint32_t apart, uint32_t end) {
    if constexpr (BYTES == 16) return ld_nc_v4(row + off);
    else return gather(off, apart, end, [&](uint32_t at, auto t) { return __ldg(reinterpret_cast<const decltype(t)*>(row + at)); });
  }
  static __device__ __forceinline__ int4 load_own(const uint8_t* row, uint32_t off, uint32_t apart, uint32_t end) {
    if constexpr (BYTES == 16) return ld_v4(row + off);
    else return gather(off, apart, end, [&](uint32_t at, auto t) { return *reinterpret_cast<const decltype(t)*>(row + at); });
  }
  static __device__ __forceinline__ void store(uint8_t* row, uint32_t off, uint32_t apart, uint32_t end, int4 v) {
    if constexpr (BYTES == 16) {
      __stcs(reinterpret_cast<int4*>(row + off), v);
    } else {
      const uint32_t w[4] = {(uint32_t)v.x, (uint32_t)v.y, (uint32_t)v.z, (uint32_t)v.w};
#pragma unroll
      for (int q = 0; q < kPieces; ++q) {
        const uint32_t at = off + q * apart;
        if (at >= end) break;
        if constexpr (BYTES == 8) *reinterpret_cast<uint2*>(row + at) = make_uint2(w[2 * q], w[2 * q + 1]);
        else if constexpr (BYTES == 4) *reinterpret_cast<uint32_t*>(row + at) = w[q];
        else *reinterpret_cast<uint16_t*>(row + at) = (uint16_t)(w[q / 2] >> (16 * (q & 1)));
      }
    }
  }
};

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

// BYTES: what a load takes of a row, 16, 8, 4 or 2 as rows align (RowUnit). SEARCH: without a row map.
template <int DT, int BYTES, bool SEARCH>
__global__ void __launch_bounds__(kGradThreads, BYTES == 16 ? 4 : 3) combine_grad_kernel(CombineGradParams p, int active) {
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
  const uint32_t begin = (int)threadIdx.x < active ? threadIdx.x * BYTES : 0x7fffffffu;  // rows are 2^30 bytes at most
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
  using Unit = RowUnit<BYTES>;
  const uint32_t apart = active * BYTES;  // a unit's pieces
  for (int j0 = blockIdx.y * kGradBatch; j0 < n; j0 += gridDim.y * kGradBatch) {
    const int here = min(kGradBatch, n - j0);
    float acc[kGradBatch];
#pragma unroll
    for (int j = 0; j < kGradBatch; ++j) acc[j] = 0.f;
    for (uint32_t off = begin; off < (uint32_t)sh.row_in; off += apart * Unit::kPieces) {
      int4 y[kGradBatch];
      const int4 gv = Unit::load(g_row, off, apart, sh.row_in);
#pragma unroll
      for (int j = 0; j < kGradBatch; ++j)
        if (dots && j < here) y[j] = Unit::load(s_src[j0 + j], off, apart, sh.row_in);
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
          Unit::store(dst, off, apart, sh.row_in, Vec<DT>::pack(o));
        }
        if (dots) {
          float f[8];
          Vec<DT>::unpack(f, y[j]);
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[j] = __fmaf_rn(g[i], f[i], acc[j]);
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
    for (uint32_t off = begin; off < (uint32_t)sh.row_in; off += apart * Unit::kPieces) {
      float g[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = 0.f;
      if (some) {
        Vec<DT>::unpack(g, Unit::load(g_row, off, apart, sh.row_in));
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = __fmul_rn(w, g[i]);
      }
      Unit::store(out, off, apart, sh.row_in, Vec<DT>::pack(g));
    }
  }

  if (check) {
    const int s = (int)(tau / sh.bs), t = (int)(tau % sh.bs);
    if (a0 != s || a1 != t || a2 != lane || r - (long long)d * sh.A >= cnt) set_error(p.status, MOE_ERR_BAD_ASSIST);
  }
}

// Dispatch's gradient where a batch is too small for a row map to pay: a block has one token, as above.
template <int DT, int BYTES>
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
  using Unit = RowUnit<BYTES>;
  const uint32_t apart = blockDim.x * BYTES;
  for (uint32_t off = threadIdx.x * BYTES; off < (uint32_t)sh.row_in; off += apart * Unit::kPieces) {
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
    if (residual) Vec<DT>::fma(acc, 1.f, Unit::load_own(residual, off, apart, sh.row_in));
    for (int j0 = 0; j0 < n; j0 += kGradBatch) {
      int4 y[kGradBatch];
#pragma unroll
      for (int j = 0; j < kGradBatch; ++j)
        if (j0 + j < n) y[j] = Unit::load(s_src[j0 + j], off, apart, sh.row_in);
#pragma unroll
      for (int j = 0; j < kGradBatch; ++j)
        if (j0 + j < n) Vec<DT>::fma(acc, 1.f, y[j]);
    }
    Unit::store(out, off, apart, sh.row_in, Vec<DT>::pack(acc));
  }
}

// The widest pieces that rows, which lie one after the other, align for.
static int row_piece(const Shape& sh) { return sh.row_in % 16 == 0 ? 16 : sh.row_in % 8 == 0 ? 8 : sh.row_in % 4 == 0 ? 4 : 2; }

// As few threads as go through a row in as many steps as 256 would; where rows are looked for, a warp for each pick.
static int grad_threads(const Shape& sh, bool search) {
  const int items = (sh.row_in + 15) / 16;
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
  const auto launch = [&](auto f16, auto bf16) {
    return sh.x_dtype == MOE_F16 ? cudaLaunchKernelEx(&L.cfg, f16, p, active) : cudaLaunchKernelEx(&L.cfg, bf16, p, active);
  };
  switch (row_piece(sh)) {
    case 16: return launch(combine_grad_kernel<MOE_F16, 16, SEARCH>, combine_grad_kernel<MOE_BF16, 16, SEARCH>);
    case 8: return launch(combine_grad_kernel<MOE_F16, 8, SEARCH>, combine_grad_kernel<MOE_BF16, 8, SEARCH>);
    case 4: return launch(combine_grad_kernel<MOE_F16, 4, SEARCH>, combine_grad_kernel<MOE_BF16, 4, SEARCH>);
    default: return launch(combine_grad_kernel<MOE_F16, 2, SEARCH>, combine_grad_kernel<MOE_BF16, 2, SEARCH>);
  }
}

cudaError_t launch_combine_grad(const CombineGradParams& p, bool search, cudaStream_t st, int num_sms) {
  return search ? launch_grad<true>(p, st, num_sms) : launch_grad<false>(p, st, num_sms);
}

cudaError_t launch_dispatch_grad(const DispatchGradParams& p, bool search, cudaStream_t st, int num_sms) {
  const Shape& sh = p.sh;
  if (!search && sh.row_in % 16 == 0) return launch_dispatch_grad_reduce(p, st, num_sms);
  PdlLaunch L(dim3((unsigned)(sh.W * sh.bs)), dim3(grad_threads(sh, true)), 0, st);
  const auto launch = [&](auto f16, auto bf16) {
    return sh.x_dtype == MOE_F16 ? cudaLaunchKernelEx(&L.cfg, f16, p) : cudaLaunchKernelEx(&L.cfg, bf16, p);
  };
  switch (row_piece(sh)) {
    case 16: return launch(dispatch_grad_token_kernel<MOE_F16, 16>, dispatch_grad_token_kernel<MOE_BF16, 16>);
    case 8: return launch(dispatch_grad_token_kernel<MOE_F16, 8>, dispatch_grad_token_kernel<MOE_BF16, 8>);
    case 4: return launch(dispatch_grad_token_kernel<MOE_F16, 4>, dispatch_grad_token_kernel<MOE_BF16, 4>);
    default: return launch(dispatch_grad_token_kernel<MOE_F16, 2>, dispatch_grad_token_kernel<MOE_BF16, 2>);
  }
}

}  // namespace crs

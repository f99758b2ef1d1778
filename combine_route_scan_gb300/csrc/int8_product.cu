// The experts' product on dispatched int8 rows (moe_expert_product_int8;
// include/moe_experts.h): z[r][j] = xs[r] * ws[e(r)][j] * sum_i x[r][i] * w[e(r)][j][i] over
// the rows that ep_recv_count gives to each expert, then the epilogue.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/moe_experts.h"
#include "common.cuh"
#include "experts_host.h"

namespace crs {

struct Int8ProductParams {
  const int8_t* x;    // [W*A][K]
  const float* xs;    // [W*A], or null
  const int32_t* ep;  // [W][L*W]
  const int8_t* w;    // [E][N][K]
  const float* ws;    // [E][N]
  void* y;            // [W*A][C]
  int W, L, E, N, K, C;
  long long A;
  int* status;
};

// SwiGLU of a gate and what it gates. exp and the reciprocal are the fast ones, within a
// few ulps (exp: plus |gate| / 2^23 of its value), far below the rounding to 16 bits that
// follows; the divisor stays within [1, 2], where the fast reciprocal holds.
__device__ __forceinline__ float int8_swiglu(float gate, float up) {
  const float t = __expf(-fabsf(gate));
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + t));
  return (gate < 0.f ? gate * t : gate) * r * up;
}

// The experts' rows: running tiles of `tile` rows pre[E + 1], first flat row [E], row
// count [E] behind one another; false (for every thread) where counts overlap to more tiles
// than dispatch's can make. All threads of the block take part.
template <int THREADS>
__device__ __forceinline__ bool int8_expert_rows(const Int8ProductParams& p, int tile, int* pre, long long* scratch) {
  int* first = pre + p.E + 1;
  int* count = first + p.E;
  long long carry = 0;
  for (int e0 = 0; e0 < p.E; e0 += THREADS) {
    const int e = e0 + (int)threadIdx.x;
    int lo = 0, n = 0;
    if (e < p.E) {
      const int le = e % p.L;
      const int32_t* ep = p.ep + (size_t)(e / p.L) * p.L * p.W;
      const int hi = ep[le * p.W + p.W - 1];
      lo = le ? ep[le * p.W - 1] : 0;
      n = hi - lo;
      if (lo < 0 || hi < lo || hi > p.A) {
        if (blockIdx.x == 0) set_error(p.status, MOE_ERR_BAD_ASSIST);
        n = 0;
        lo = 0;
      }
      first[e] = (int)(e / p.L * p.A) + lo;  // flat rows fit 32 bits
      count[e] = n;
    }
    const long long tiles = (n + tile - 1) / tile;
    const long long before = carry + block_exclusive_scan(tiles, scratch);
    if (e < p.E) {
      pre[e] = (int)min(before, 1ll << 30);
      if (e == p.E - 1) pre[p.E] = (int)min(before + tiles, 1ll << 30);
    }
    __syncthreads();
    const int last = min(p.E, e0 + THREADS) - 1;
    carry = pre[last] + (count[last] + tile - 1) / tile;
  }
  return pre[p.E] <= (long long)p.W * p.A / tile + p.E;
}

// ------------------------------------------------------------- any k and alignment

// Rows whose length the tensor kernel's copies cannot take (k not a multiple of 16): 32 rows
// x 64 features a unit, four products an instruction (dp4a), 32-bit sums. Bound by those
// instructions; a shape of this kind is no one's production size.
constexpr int kPlainThreads = 256, kPlainRows = 32, kPlainCols = 64, kPlainK = 128;

template <int YT, bool SWIGLU>
__global__ void __launch_bounds__(kPlainThreads) int8_product_plain_kernel(Int8ProductParams p) {
  __shared__ int s_x[kPlainRows][kPlainK / 4 + 1], s_w[kPlainCols][kPlainK / 4 + 1];
  __shared__ long long scratch[32];
  extern __shared__ int pre[];
  pdl_wait();
  pdl_launch_dependents();
  if (!int8_expert_rows<kPlainThreads>(p, kPlainRows, pre, scratch)) return;
  const int* first = pre + p.E + 1;
  const int* count = first + p.E;
  const int n_tiles = (p.N + kPlainCols - 1) / kPlainCols;
  const long long units = (long long)pre[p.E] * n_tiles;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const int mt = (int)(u / n_tiles), n0 = (int)(u % n_tiles) * kPlainCols;
    int e = 0;  // the last expert whose tiles begin at or before mt
    for (int half = 512; half; half >>= 1)
      if (e + half < p.E && pre[e + half] <= mt) e += half;
    const int before = (mt - pre[e]) * kPlainRows, rows = min(kPlainRows, count[e] - before);
    const long long row0 = first[e] + before;
    int acc[2][4] = {};
    for (int k0 = 0; k0 < p.K; k0 += kPlainK) {
      __syncthreads();
      for (int i = threadIdx.x; i < (kPlainRows + kPlainCols) * kPlainK; i += kPlainThreads) {
        const int r = i / kPlainK, c = i % kPlainK;
        int8_t v = 0;
        if (r < kPlainRows) {
          if (r < rows && k0 + c < p.K) v = p.x[(size_t)(row0 + r) * p.K + k0 + c];
          reinterpret_cast<int8_t*>(s_x[r])[c] = v;
        } else {
          const int j = r - kPlainRows;
          if (n0 + j < p.N && k0 + c < p.K) v = p.w[((size_t)e * p.N + n0 + j) * p.K + k0 + c];
          reinterpret_cast<int8_t*>(s_w[j])[c] = v;
        }
      }
      __syncthreads();
#pragma unroll 4
      for (int k = 0; k < kPlainK / 4; ++k)
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
          for (int b = 0; b < 4; ++b) acc[a][b] = __dp4a(s_x[ty * 2 + a][k], s_w[tx * 4 + b][k], acc[a][b]);
    }
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      const int r = ty * 2 + a;
      if (r >= rows) continue;
      const float xs = p.xs ? p.xs[row0 + r] : 1.f;
      float z[4];
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int j = n0 + tx * 4 + b;
        z[b] = j < p.N ? (float)acc[a][b] * xs * p.ws[(size_t)e * p.N + j] : 0.f;
      }
#pragma unroll
      for (int b = 0; b < (SWIGLU ? 2 : 4); ++b) {
        const int c = (SWIGLU ? n0 / 2 + tx * 2 : n0 + tx * 4) + b;
        if (c >= p.C) continue;
        const float v = SWIGLU ? int8_swiglu(z[(2 * b) & 3], z[(2 * b + 1) & 3]) : z[b];
        static_cast<uint16_t*>(p.y)[(size_t)(row0 + r) * p.C + c] =
            YT == MOE_F16 ? __half_as_ushort(__float2half_rn(v)) : __bfloat16_as_ushort(__float2bfloat16_rn(v));
      }
    }
  }
}

// ------------------------------------------------------------- host side

typedef void (*Int8PlainKernel)(Int8ProductParams);

}  // namespace crs

extern "C" moe_status_t moe_expert_product_int8(const moe_config_t* cfg, const int8_t* x, const float* x_scales,
                                                const int32_t* ep_recv_count, const int8_t* w, const float* w_scales,
                                                int32_t n, int32_t k, int32_t epilogue, int32_t y_dtype, void* y,
                                                void* ws, size_t ws_bytes, void* stream) {
  using namespace crs;
  size_t need = 0;
  int64_t A = 0;
  const moe_status_t st = moe_get_workspace_size(cfg, &need, &A);
  if (st != MOE_OK) return st;
  if (n < 1 || k < 1 || k > 131071 || epilogue < MOE_EPI_NONE || epilogue > MOE_EPI_SWIGLU) return MOE_ERR_INVALID_ARG;
  const int E = cfg->moe_expert_num, W = cfg->ep_world_size;
  if (epilogue == MOE_EPI_SWIGLU && n % 2) return MOE_ERR_INVALID_ARG;
  if (y_dtype != MOE_F16 && y_dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if ((long long)E * n >= 2147483647LL) return MOE_ERR_INVALID_ARG;
  if (!ep_recv_count || (A > 0 && (!x || !w || !w_scales || !y))) return MOE_ERR_INVALID_ARG;
  auto aligned = [](const void* p, size_t a) { return ((uintptr_t)p % a) == 0; };
  if (!aligned(x, 16) || !aligned(x_scales, 4) || !aligned(ep_recv_count, 4) || !aligned(w, 16) || !aligned(w_scales, 4) ||
      !aligned(y, 16))
    return MOE_ERR_INVALID_ARG;
  if (!ws || ws_bytes < need || !aligned(ws, 256)) return MOE_ERR_WORKSPACE;
  if (A == 0) return MOE_OK;
  const int nsm = num_sms_of_current_device();
  if (nsm <= 0) return MOE_ERR_CUDA;
  Int8ProductParams p{};
  p.x = x;
  p.xs = x_scales;
  p.ep = ep_recv_count;
  p.w = w;
  p.ws = w_scales;
  p.y = y;
  p.W = W;
  p.L = E / W;
  p.E = E;
  p.N = n;
  p.K = k;
  p.C = epilogue == MOE_EPI_SWIGLU ? n / 2 : n;
  p.A = A;
  p.status = &static_cast<WsHeader*>(ws)->status;
  const bool sw = epilogue == MOE_EPI_SWIGLU;
  const Int8PlainKernel plain =
      y_dtype == MOE_F16 ? (sw ? int8_product_plain_kernel<MOE_F16, true> : int8_product_plain_kernel<MOE_F16, false>)
                         : (sw ? int8_product_plain_kernel<MOE_BF16, true> : int8_product_plain_kernel<MOE_BF16, false>);
  const size_t smem = (3 * (size_t)E + 1) * 4;
  int per_sm = 0;
  if (resident_blocks((const void*)plain, kPlainThreads, smem, &per_sm) != cudaSuccess || per_sm < 1) return MOE_ERR_CUDA;
  PdlLaunch L(dim3((unsigned)(nsm * per_sm)), dim3(kPlainThreads), smem, static_cast<cudaStream_t>(stream));
  if (cudaLaunchKernelEx(&L.cfg, plain, p) != cudaSuccess) return MOE_ERR_CUDA;
  note_launches(1);
  return MOE_OK;
}

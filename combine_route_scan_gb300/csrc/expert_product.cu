// The experts' product on dispatched MX FP4 rows (moe_expert_product;
// include/moe_experts.h).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/moe_experts.h"
#include "quant_common.cuh"

namespace crs {

struct ProductParams {
  const uint8_t* x;        // [W*A][K/2]
  const uint8_t* xs;       // [W*A][K/32]
  const int32_t* ep;       // [W][L*W]
  const uint8_t* w;        // [E][N][K/2]
  const uint8_t* wsf;      // tiles of 128 x 4 scales
  void* y;                 // [W*A][C]
  uint8_t* ys;             // [W*A][ceil(C/32)], MX FP4 output
  int W, L, E, N, K, C;    // C output columns
  long long A;
  int swiglu, y_dtype;
  int* status;
  uint64_t timeout_ns;
};

constexpr int kRowTile = 16, kColTile = 64;

// One CTA a (expert, 64 weight rows) unit, 16 rows at a time: 256 threads, 4
// sums each, operands decoded to fp32 in shared memory 32 elements at a time.
__global__ void __launch_bounds__(256) expert_product_kernel(ProductParams p) {
  __shared__ float sx[kRowTile][33], sw[kColTile][33], sz[kRowTile][kColTile + 1];
  __shared__ float lut[16];
  pdl_wait();
  pdl_launch_dependents();
  if (threadIdx.x < 16) {
    const int c = threadIdx.x, ex = (c >> 1) & 3, m = c & 1;
    const float v = ex == 0 ? 0.5f * m : (1.f + 0.5f * m) * (1 << (ex - 1));
    lut[c] = c & 8 ? -v : v;
  }
  __syncthreads();
  const int tiles = (p.N + kColTile - 1) / kColTile, blocks = p.K / 32, bt = (blocks + 3) / 4;
  for (int u = blockIdx.x; u < p.E * tiles; u += gridDim.x) {
    const int e = u / tiles, n0 = u % tiles * kColTile, d = e / p.L, le = e % p.L;
    const int32_t* ep = p.ep + (size_t)d * p.L * p.W;
    const int lo = le ? ep[le * p.W - 1] : 0, hi = ep[le * p.W + p.W - 1];
    if (lo < 0 || hi < lo || hi > p.A) {
      if (threadIdx.x == 0) set_error(p.status, MOE_ERR_BAD_ASSIST);
      continue;
    }
    for (int r0 = lo; r0 < hi; r0 += kRowTile) {
      const long long row0 = d * p.A + r0;
      const int nr = min(kRowTile, hi - r0);
      float acc[4] = {};
      const int tr = threadIdx.x >> 4, tc = threadIdx.x & 15;
      for (int b = 0; b < blocks; ++b) {
        __syncthreads();
        for (int i = threadIdx.x; i < (kRowTile + kColTile) * 16; i += 256) {
          const int r = i >> 4, j = i & 15;
          uint32_t byte = 0;
          float s = 0.f;
          if (r < kRowTile) {
            if (r < nr) {
              byte = p.x[(size_t)(row0 + r) * (p.K / 2) + b * 16 + j];
              s = exp2_exact((int)p.xs[(size_t)(row0 + r) * blocks + b] - 127);
            }
            sx[r][2 * j] = lut[byte & 15] * s;
            sx[r][2 * j + 1] = lut[byte >> 4] * s;
          } else {
            const int n = n0 + r - kRowTile;
            if (n < p.N) {
              byte = p.w[((size_t)e * p.N + n) * (p.K / 2) + b * 16 + j];
              const size_t tile = ((size_t)e * ((p.N + 127) / 128) + n / 128) * bt + b / 4;
              s = exp2_exact((int)p.wsf[tile * 512 + n % 32 * 16 + n % 128 / 32 * 4 + b % 4] - 127);
            }
            sw[r - kRowTile][2 * j] = lut[byte & 15] * s;
            sw[r - kRowTile][2 * j + 1] = lut[byte >> 4] * s;
          }
        }
        __syncthreads();
#pragma unroll 8
        for (int j = 0; j < 32; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[q] = fmaf(sx[tr][j], sw[tc + 16 * q][j], acc[q]);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) sz[tr][tc + 16 * q] = acc[q];
      __syncthreads();
      const int width = p.swiglu ? kColTile / 2 : kColTile, c0 = p.swiglu ? n0 / 2 : n0;
      if (p.swiglu) {
        float h[2];
        for (int q = 0; q < 2; ++q) {
          const float g = sz[tr][2 * (tc + 16 * q)], v = sz[tr][2 * (tc + 16 * q) + 1];
          h[q] = g / (1.f + expf(-g)) * v;
        }
        __syncthreads();
        for (int q = 0; q < 2; ++q) sz[tr][tc + 16 * q] = h[q];
        __syncthreads();
      }
      if (p.y_dtype == MOE_MXFP4) {
        if (threadIdx.x < kRowTile * (width / 32)) {
          const int r = threadIdx.x / (width / 32), q = threadIdx.x % (width / 32), c = c0 + 32 * q;
          const int n = min(32, p.C - c);
          if (r < nr && n > 0) {
            float m = 0.f;
            for (int j = 0; j < n; ++j) m = fmaxf(m, fabsf(sz[r][32 * q + j]));
            const int se = mx_exponent(m, 2);
            const float inv = exp2_exact(-se);
            uint8_t* out = static_cast<uint8_t*>(p.y) + (size_t)(row0 + r) * (p.C / 2) + c / 2;
            for (int j = 0; j < n; j += 2)
              out[j / 2] = (uint8_t)cvt_fp4x2(sz[r][32 * q + j] * inv, sz[r][32 * q + j + 1] * inv);
            p.ys[(size_t)(row0 + r) * ((p.C + 31) / 32) + c / 32] = (uint8_t)(se + 127);
          }
        }
      } else {
        for (int c = tc; c < width; c += 16)
          if (tr < nr && c0 + c < p.C) {
            const size_t at = (size_t)(row0 + tr) * p.C + c0 + c;
            if (p.y_dtype == MOE_F16) static_cast<__half*>(p.y)[at] = __float2half_rn(sz[tr][c]);
            else static_cast<__nv_bfloat16*>(p.y)[at] = __float2bfloat16_rn(sz[tr][c]);
          }
      }
    }
  }
}

}  // namespace crs

extern "C" moe_status_t moe_expert_product(const moe_config_t* cfg, const void* x, const uint8_t* x_scales,
                                           const int32_t* ep_recv_count, const void* w, const uint8_t* w_scales,
                                           int32_t n, int32_t k, int32_t epilogue, int32_t y_dtype, void* y,
                                           uint8_t* y_scales, void* ws, size_t ws_bytes, void* stream) {
  using namespace crs;
  size_t need = 0;
  int64_t A = 0;
  const moe_status_t st = moe_get_workspace_size(cfg, &need, &A);
  if (st != MOE_OK) return st;
  if (n < 1 || k < 1 || epilogue < MOE_EPI_NONE || epilogue > MOE_EPI_SWIGLU) return MOE_ERR_INVALID_ARG;
  if (k % 32) return MOE_ERR_UNSUPPORTED;
  const int E = cfg->moe_expert_num, W = cfg->ep_world_size;
  if (epilogue == MOE_EPI_SWIGLU && n % 2) return MOE_ERR_INVALID_ARG;
  const int C = epilogue == MOE_EPI_SWIGLU ? n / 2 : n;
  if (y_dtype != MOE_F16 && y_dtype != MOE_BF16 && y_dtype != MOE_MXFP4) return MOE_ERR_INVALID_ARG;
  if (y_dtype == MOE_MXFP4 ? C % 2 != 0 || !y_scales : y_scales != nullptr) return MOE_ERR_INVALID_ARG;
  if ((long long)E * n >= 2147483647LL) return MOE_ERR_INVALID_ARG;
  if (!ep_recv_count) return MOE_ERR_INVALID_ARG;
  if (A > 0 && (!x || !x_scales || !w || !w_scales || !y)) return MOE_ERR_INVALID_ARG;
  auto aligned = [](const void* p, size_t a) { return ((uintptr_t)p % a) == 0; };
  if (!aligned(x, 16) || !aligned(x_scales, 4) || !aligned(ep_recv_count, 4) || !aligned(w, 16) ||
      !aligned(w_scales, 16) || !aligned(y, 16))
    return MOE_ERR_INVALID_ARG;
  if (!ws || ws_bytes < need || !aligned(ws, 256)) return MOE_ERR_WORKSPACE;
  if (A == 0) return MOE_OK;
  const int nsm = num_sms_of_current_device();
  if (nsm <= 0) return MOE_ERR_CUDA;
  ProductParams p{};
  p.x = static_cast<const uint8_t*>(x);
  p.xs = x_scales;
  p.ep = ep_recv_count;
  p.w = static_cast<const uint8_t*>(w);
  p.wsf = w_scales;
  p.y = y;
  p.ys = y_scales;
  p.W = W;
  p.L = E / W;
  p.E = E;
  p.N = n;
  p.K = k;
  p.C = C;
  p.A = A;
  p.swiglu = epilogue == MOE_EPI_SWIGLU;
  p.y_dtype = y_dtype;
  p.status = &static_cast<WsHeader*>(ws)->status;
  p.timeout_ns = (uint64_t)cfg->wait_timeout_us * 1000ull;
  const long long units = (long long)E * ((n + kColTile - 1) / kColTile);
  PdlLaunch L(dim3((unsigned)(units < nsm * 8ll ? units : nsm * 8ll)), dim3(256), 0,
              static_cast<cudaStream_t>(stream));
  if (cudaLaunchKernelEx(&L.cfg, expert_product_kernel, p) != cudaSuccess) return MOE_ERR_CUDA;
  note_launches(1);
  return MOE_OK;
}

// Microscaled 4-bit quantisation of whole matrices (moe_mx_quantize;
// include/moe_experts.h): blocks of 32 elements share a power of two, codes are
// E2M1, with the arithmetic of dispatch's quant_mode 4 (quant_common.cuh).
#include "../../include/moe_experts.h"
#include "quant_common.cuh"

namespace crs {

struct MxQuantParams {
  const void* x;
  uint8_t* codes;
  uint8_t* scales;
  long long rows, row_stride, expert_stride;  // rows of one matrix
  int experts, cols, blocks;                  // blocks = ceil(cols / 32)
  int tiled;
};

template <int DT>
__device__ __forceinline__ float mx_load(const void* x, size_t i) {
  if (DT == MOE_F32) return static_cast<const float*>(x)[i];
  return load_elem(x, i, DT);
}

__device__ __forceinline__ size_t mx_scale_at(const MxQuantParams& p, long long e, long long r, int b) {
  if (!p.tiled) return ((size_t)e * p.rows + r) * p.blocks + b;
  const size_t nt = (p.rows + 127) / 128, bt = (p.blocks + 3) / 4;
  return (((size_t)e * nt + r / 128) * bt + b / 4) * 512 + (r % 32) * 16 + (r % 128) / 32 * 4 + b % 4;
}

// One thread a block; with tiled scales the threads beyond the edges of the
// last tiles write their zero bytes.
template <int DT>
__global__ void __launch_bounds__(256) mx_quantize_kernel(MxQuantParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const long long rows = p.tiled ? (p.rows + 127) / 128 * 128 : p.rows;
  const long long blocks = p.tiled ? (p.blocks + 3) / 4 * 4 : p.blocks;
  const long long total = p.experts * rows * blocks;
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
    const int b = (int)(i % blocks);
    const long long r = i / blocks % rows, e = i / blocks / rows;
    const size_t at = mx_scale_at(p, e, r, b);
    if (r >= p.rows || b >= p.blocks) {
      p.scales[at] = 0;
      continue;
    }
    const size_t from = (size_t)(e * p.expert_stride + r * p.row_stride) + (size_t)b * 32;
    const int n = min(32, p.cols - b * 32);
    float m = 0.f;
    for (int j = 0; j < n; ++j) m = fmaxf(m, fabsf(mx_load<DT>(p.x, from + j)));
    const int se = mx_exponent(m, 2);
    const float inv = exp2_exact(-se);
    uint8_t* out = p.codes + ((size_t)e * p.rows + r) * (p.cols / 2) + (size_t)b * 16;
    for (int j = 0; j < n; j += 2)
      out[j / 2] = (uint8_t)cvt_fp4x2(__fmul_rn(mx_load<DT>(p.x, from + j), inv),
                                      __fmul_rn(mx_load<DT>(p.x, from + j + 1), inv));
    p.scales[at] = (uint8_t)(se + 127);
  }
}

}  // namespace crs

extern "C" uint64_t moe_mx_scale_bytes(int32_t experts, int64_t rows, int32_t cols, int32_t sf_layout) {
  if (experts < 0 || rows < 0 || cols < 2 || cols % 2 || cols > (1 << 30)) return 0;
  if (rows >= 2147483648LL || experts * rows >= 2147483648LL) return 0;
  const uint64_t blocks = ((uint64_t)cols + 31) / 32;
  if (sf_layout == MOE_SF_ROWS) return (uint64_t)experts * rows * blocks;
  if (sf_layout == MOE_SF_TILED) return (uint64_t)experts * (((uint64_t)rows + 127) / 128) * ((blocks + 3) / 4) * 512;
  return 0;
}

extern "C" moe_status_t moe_mx_quantize(const void* x, int32_t x_dtype, int32_t experts, int64_t rows, int32_t cols,
                                        int64_t row_stride, int64_t expert_stride, int32_t sf_layout, uint8_t* codes,
                                        uint8_t* scales, void* stream) {
  using namespace crs;
  if (x_dtype != MOE_F32 && x_dtype != MOE_F16 && x_dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (experts < 0 || rows < 0 || cols < 2 || cols % 2 || cols > (1 << 30)) return MOE_ERR_INVALID_ARG;
  if (rows >= 2147483648LL || experts * rows >= 2147483648LL) return MOE_ERR_INVALID_ARG;
  if (row_stride < cols || expert_stride < 0) return MOE_ERR_INVALID_ARG;
  if (sf_layout != MOE_SF_ROWS && sf_layout != MOE_SF_TILED) return MOE_ERR_INVALID_ARG;
  if (experts == 0 || rows == 0) return MOE_OK;
  if (!x || !codes || !scales || (uintptr_t)x % (x_dtype == MOE_F32 ? 4 : 2)) return MOE_ERR_INVALID_ARG;
  const int nsm = num_sms_of_current_device();
  if (nsm <= 0) return MOE_ERR_CUDA;
  MxQuantParams p{x, codes, scales, rows, row_stride, expert_stride, experts, cols, (cols + 31) / 32,
                  sf_layout == MOE_SF_TILED};
  void (*kernel)(MxQuantParams) = x_dtype == MOE_F32   ? mx_quantize_kernel<MOE_F32>
                                  : x_dtype == MOE_F16 ? mx_quantize_kernel<MOE_F16>
                                                       : mx_quantize_kernel<MOE_BF16>;
  const long long total = (long long)moe_mx_scale_bytes(experts, rows, cols, sf_layout);
  const long long need = (total + 255) / 256, most = nsm * 8ll;
  PdlLaunch L(dim3((unsigned)(need < most ? need : most)), dim3(256), 0, static_cast<cudaStream_t>(stream));
  if (cudaLaunchKernelEx(&L.cfg, kernel, p) != cudaSuccess) return MOE_ERR_CUDA;
  note_launches(1);
  return MOE_OK;
}

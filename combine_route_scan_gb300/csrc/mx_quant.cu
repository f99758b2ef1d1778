// Microscaled 4-bit quantisation of whole matrices (moe_mx_quantize;
// include/moe_experts.h): blocks of 32 elements share a power of two, codes are
// E2M1, with the arithmetic of dispatch's quant_mode 4 (quant_common.cuh).
//
// One pass over the data, bound by HBM: mx_quantize_vec_kernel gives each block of
// 32 to two neighbouring lanes, 16 elements each, so that a warp reads and writes
// 16 blocks in a row; the block's maximum takes one shuffle, and four blocks' scale
// bytes leave as one word. The next 16 elements are loaded before the present ones
// are worked on. (Eight elements a lane spent as many instructions on addresses as
// on them: 223 us for 128 x 1024 x 2048 bf16.) Rows that 16-byte loads do not fit go
// through mx_quantize_kernel, a thread a block.
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

// 16 elements as loaded, and as fp32 pairs.
template <int DT>
struct MxVec {
  static constexpr int kLoads = DT == MOE_F32 ? 4 : 2;
  int4 v[kLoads];
  __device__ void load(const uint8_t* x) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) v[i] = __ldg(reinterpret_cast<const int4*>(x) + i);
  }
  __device__ void pairs(f32x2 (&o)[8]) const {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      if (DT == MOE_F32) {
        o[2 * i] = f2_pack(__int_as_float(v[i].x), __int_as_float(v[i].y));
        o[2 * i + 1] = f2_pack(__int_as_float(v[i].z), __int_as_float(v[i].w));
      } else {
        f32x2 q[4];
        unpack8x2<DT == MOE_F32 ? MOE_BF16 : DT>(v[i], q);
#pragma unroll
        for (int j = 0; j < 4; ++j) o[(4 * i + j) & 7] = q[j];
      }
    }
  }
};

// cols a multiple of 32, rows of x 16-byte aligned, codes 8-byte and scales 4-byte
// aligned. Codes and MOE_SF_ROWS scales run on from block to block over all rows and
// matrices; x (STRIDED) and the tiles need the block's matrix, row and place.
template <int DT, bool TILED, bool STRIDED>
__global__ void __launch_bounds__(256) mx_quantize_vec_kernel(MxQuantParams p) {
  pdl_wait();
  pdl_launch_dependents();
  constexpr int kEs = DT == MOE_F32 ? 4 : 2;
  const int lane = threadIdx.x & 31, half = lane & 1;
  const int rows = (int)p.rows, blocks = p.blocks;
  const long long total = (long long)p.experts * rows * blocks;
  const long long step = gridDim.x * 128ll;
  long long i = blockIdx.x * 128ll + (threadIdx.x >> 1);
  int b = 0, r = 0, e = 0, db = 0, dr = 0, de = 0;
  if (TILED || STRIDED) {
    b = (int)(i % blocks), r = (int)(i / blocks % rows), e = (int)(i / blocks / rows);
    db = (int)(step % blocks), dr = (int)(step / blocks % rows), de = (int)(step / blocks / rows);
  }
  const auto advance = [&] {
    b += db;
    r += dr;
    e += de;
    if (b >= blocks) {
      b -= blocks;
      ++r;
    }
    if (r >= rows) {
      r -= rows;
      ++e;
    }
  };
  const uint8_t* x = static_cast<const uint8_t*>(p.x) + half * (16 * kEs);
  const auto from = [&](long long k) {
    return x + (STRIDED ? (size_t)(e * p.expert_stride + r * p.row_stride + b * 32) : (size_t)k * 32) * kEs;
  };
  const bool words = (blocks & 3) == 0;  // four blocks from a multiple of 4 on are in one row, and four neighbouring pairs
  const int nt = (rows + 127) >> 7, bt = (blocks + 3) >> 2;
  MxVec<DT> next{};
  if (i < total) next.load(from(i));
  for (long long first = i - (lane >> 1); first < total; first += step, i += step) {
    f32x2 v[8];
    next.pairs(v);
    const bool valid = i < total;
    uint8_t* sf = p.scales + i;
    if (TILED) sf = p.scales + ((size_t)(e * nt + (r >> 7)) * bt + (b >> 2)) * 512 + ((r & 31) * 16 + ((r & 127) >> 5) * 4 + (b & 3));
    if (TILED || STRIDED) advance();
    if (i + step < total) next.load(from(i + step));
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float lo, hi;
      f2_split(v[j], lo, hi);
      m = fmax_abs3(m, lo, hi);
    }
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    const int se = mx_exponent(m, 2);
    const float inv = exp2_exact(-se);
    const f32x2 inv2 = f2_pack(inv, inv);
    uint32_t q[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float lo, hi;
      f2_split(f2_mul(v[j], inv2), lo, hi);
      q[j >> 2] |= cvt_fp4x2(lo, hi) << (8 * (j & 3));
    }
    uint32_t word = (uint32_t)(se + 127) << (8 * ((lane >> 1) & 3));
    if (words) {
      word |= __shfl_xor_sync(0xffffffffu, word, 2);
      word |= __shfl_xor_sync(0xffffffffu, word, 4);
    }
    if (!valid) continue;
    *reinterpret_cast<uint2*>(p.codes + (size_t)i * 16 + half * 8) = make_uint2(q[0], q[1]);
    if (words) {
      if ((lane & 7) == 0) *reinterpret_cast<uint32_t*>(sf) = word;
    } else if (half == 0) {
      *sf = (uint8_t)(se + 127);
    }
  }
  if (TILED) {
    // the zero bytes beyond the edges of the last tiles
    const int rows4 = nt * 128, blocks4 = bt * 4;
    const long long below = (long long)(rows4 - rows) * blocks4, beside = (long long)rows * (blocks4 - blocks);
    const long long pad = (below + beside) * p.experts;
    for (long long k = blockIdx.x * 256ll + threadIdx.x; k < pad; k += gridDim.x * 256ll) {
      const long long ke = k / (below + beside), o = k % (below + beside);
      if (o < below) p.scales[mx_scale_at(p, ke, rows + o / blocks4, (int)(o % blocks4))] = 0;
      else p.scales[mx_scale_at(p, ke, (o - below) / (blocks4 - blocks), blocks + (int)((o - below) % (blocks4 - blocks)))] = 0;
    }
  }
}

template <int DT>
void (*mx_kernel(bool vec, bool tiled, bool strided))(MxQuantParams) {
  if (!vec) return mx_quantize_kernel<DT>;
  if (tiled) return strided ? mx_quantize_vec_kernel<DT, true, true> : mx_quantize_vec_kernel<DT, true, false>;
  return strided ? mx_quantize_vec_kernel<DT, false, true> : mx_quantize_vec_kernel<DT, false, false>;
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
  const int es = x_dtype == MOE_F32 ? 4 : 2;
  const bool vec = cols % 32 == 0 && (uintptr_t)x % 16 == 0 && row_stride * es % 16 == 0 &&
                   (experts == 1 || expert_stride * es % 16 == 0) && (uintptr_t)codes % 8 == 0 && (uintptr_t)scales % 4 == 0;
  const bool strided = (rows > 1 && row_stride != cols) || (experts > 1 && expert_stride != rows * cols);
  const auto kernel = x_dtype == MOE_F32   ? mx_kernel<MOE_F32>(vec, p.tiled, strided)
                      : x_dtype == MOE_F16 ? mx_kernel<MOE_F16>(vec, p.tiled, strided)
                                           : mx_kernel<MOE_BF16>(vec, p.tiled, strided);
  int per_sm = 0;
  if (resident_blocks((const void*)kernel, 256, 0, &per_sm) != cudaSuccess || per_sm < 1) return MOE_ERR_CUDA;
  const long long items = vec ? (long long)experts * rows * p.blocks * 2
                              : (long long)moe_mx_scale_bytes(experts, rows, cols, sf_layout);
  const long long need = (items + 255) / 256, most = (long long)nsm * per_sm;
  PdlLaunch L(dim3((unsigned)(need < most ? need : most)), dim3(256), 0, static_cast<cudaStream_t>(stream));
  if (cudaLaunchKernelEx(&L.cfg, kernel, p) != cudaSuccess) return MOE_ERR_CUDA;
  note_launches(1);
  return MOE_OK;
}

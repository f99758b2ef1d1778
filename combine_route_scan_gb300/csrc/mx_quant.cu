// Microscaled 4-bit quantisation of whole matrices (moe_mx_quantize;
// include/moe_experts.h): blocks of 32 elements share a power of two, codes are
// E2M1, with the arithmetic of dispatch's quant_mode 4 (quant_common.cuh).
//
// One pass over the data, bound by HBM: mx_quantize_vec_kernel gives each block of
// 32 to two neighbouring lanes, 16 elements each, so that a warp reads and writes
// 16 blocks in a row; the block's maximum takes one shuffle, and four blocks' scale
// bytes leave as one word. The next 16 elements are loaded before the present ones
// are worked on. (Eight elements a lane spent as many instructions on addresses as
// on them: 223 us for 128 x 1024 x 2048 bf16.) Rows that 16-byte loads do not fit, or
// that end inside a block, go through mx_quantize_pairs_kernel: a warp takes 16 blocks
// of a row, two at a time, a pair of elements a lane. (64 x 1024 rows of 2048 bf16
// 52 us, 6.5 TB/s; of 2046 104 us; as pairs all would take the latter.)
#include "../../include/moe_experts.h"
#include "experts_host.h"
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

// The zero bytes beyond the edges of the last tiles (MOE_SF_TILED).
__device__ __forceinline__ void mx_pad_tiles(const MxQuantParams& p) {
  const long long rows4 = (p.rows + 127) / 128 * 128, blocks4 = (p.blocks + 3) / 4 * 4;
  const long long below = (rows4 - p.rows) * blocks4, beside = p.rows * (blocks4 - p.blocks);
  const long long pad = (below + beside) * p.experts;
  for (long long k = blockIdx.x * 256ll + threadIdx.x; k < pad; k += gridDim.x * 256ll) {
    const long long e = k / (below + beside), o = k % (below + beside);
    if (o < below) p.scales[mx_scale_at(p, e, p.rows + o / blocks4, (int)(o % blocks4))] = 0;
    else p.scales[mx_scale_at(p, e, (o - below) / (blocks4 - p.blocks), p.blocks + (int)((o - below) % (blocks4 - p.blocks)))] = 0;
  }
}

// Two neighbouring elements; PAIRED: aligned for one load.
template <int DT, bool PAIRED>
__device__ __forceinline__ float2 mx_load_pair(const void* x, size_t i) {
  if (!PAIRED) return make_float2(mx_load<DT>(x, i), mx_load<DT>(x, i + 1));
  if (DT == MOE_F32) return __ldg(reinterpret_cast<const float2*>(static_cast<const float*>(x) + i));
  const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(x) + i));
  if (DT == MOE_BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

template <int DT, bool PAIRED>
__global__ void __launch_bounds__(256) mx_quantize_pairs_kernel(MxQuantParams p) {
  pdl_wait();
  pdl_launch_dependents();
  constexpr int kSteps = 8;  // of two blocks
  const int lane = threadIdx.x & 31;
  const int parts = (p.blocks + 2 * kSteps - 1) / (2 * kSteps);
  const long long total = p.experts * p.rows * parts;
  for (long long i = (blockIdx.x * 256ll + threadIdx.x) >> 5; i < total; i += gridDim.x * 8ll) {
    const long long row = i / parts, e = row / p.rows, r = row - e * p.rows;
    const int b0 = (int)(i - row * parts) * 2 * kSteps;
    const size_t from = (size_t)(e * p.expert_stride + r * p.row_stride);
    float2 v[kSteps];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int c = (b0 + 2 * s) * 32 + lane * 2;
      v[s] = c < p.cols ? mx_load_pair<DT, PAIRED>(p.x, from + c) : make_float2(0.f, 0.f);
    }
    uint8_t* out = p.codes + (size_t)row * (p.cols / 2) + b0 * 16 + lane;
    // the maxima of the half warp's 8 blocks, halving the blocks that a lane looks after each time: a lane ends
    // up with one, of step 4 bit 0 + 2 bit 1 + bit 2 of its number
    float m[kSteps];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) m[s] = fmaxf(fabsf(v[s].x), fabsf(v[s].y));
#pragma unroll
    for (int o = 1, n = kSteps / 2; n; o *= 2, n /= 2) {
      const bool upper = lane & o;
#pragma unroll
      for (int k = 0; k < n; ++k)
        m[k] = fmaxf(upper ? m[k + n] : m[k], __shfl_xor_sync(0xffffffffu, upper ? m[k] : m[k + n], o));
    }
    const int se = mx_exponent(fmaxf(m[0], __shfl_xor_sync(0xffffffffu, m[0], 8)), 2);
    const float inv = exp2_exact(-se);
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const float f = __shfl_sync(0xffffffffu, inv, (lane & 16) | (s >> 2) | (s & 2) | (s & 1) << 2);
      if ((b0 + 2 * s) * 32 + lane * 2 < p.cols) out[s * 32] = (uint8_t)cvt_fp4x2(__fmul_rn(v[s].x, f), __fmul_rn(v[s].y, f));
    }
    const int b = b0 + 2 * (4 * (lane & 1) + (lane & 2) + (lane >> 2 & 1)) + (lane >> 4);
    if (!(lane & 8) && b < p.blocks) p.scales[mx_scale_at(p, e, r, b)] = (uint8_t)(se + 127);
  }
  if (p.tiled) mx_pad_tiles(p);
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
  const unsigned rows = (unsigned)p.rows;  // with a step added, and rounded up, beyond 31 bits
  const int blocks = p.blocks;
  const long long total = (long long)p.experts * rows * blocks;
  const long long step = gridDim.x * 128ll;
  long long i = blockIdx.x * 128ll + (threadIdx.x >> 1);
  int b = 0, e = 0, db = 0, de = 0;
  unsigned r = 0, dr = 0;
  if (TILED || STRIDED) {
    b = (int)(i % blocks), r = (unsigned)(i / blocks % rows), e = (int)(i / blocks / rows);
    db = (int)(step % blocks), dr = (unsigned)(step / blocks % rows), de = (int)(step / blocks / rows);
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
  const int nt = (int)((rows + 127) >> 7), bt = (blocks + 3) >> 2;
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
  if (TILED) mx_pad_tiles(p);
}

template <int DT>
void (*mx_kernel(bool vec, bool paired, bool tiled, bool strided))(MxQuantParams) {
  if (!vec) return paired ? mx_quantize_pairs_kernel<DT, true> : mx_quantize_pairs_kernel<DT, false>;
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
  const bool paired = (uintptr_t)x % (2 * es) == 0 && (rows == 1 || row_stride % 2 == 0) && (experts == 1 || expert_stride % 2 == 0);
  const bool strided = (rows > 1 && row_stride != cols) || (experts > 1 && expert_stride != rows * cols);
  const auto kernel = x_dtype == MOE_F32   ? mx_kernel<MOE_F32>(vec, paired, p.tiled, strided)
                      : x_dtype == MOE_F16 ? mx_kernel<MOE_F16>(vec, paired, p.tiled, strided)
                                           : mx_kernel<MOE_BF16>(vec, paired, p.tiled, strided);
  int per_sm = 0;
  if (resident_blocks((const void*)kernel, 256, 0, &per_sm) != cudaSuccess || per_sm < 1) return MOE_ERR_CUDA;
  const long long items = vec ? (long long)experts * rows * p.blocks * 2 : (long long)experts * rows * ((p.blocks + 15) / 16) * 32;
  const long long need = (items + 255) / 256, most = (long long)nsm * per_sm;
  PdlLaunch L(dim3((unsigned)(need < most ? need : most)), dim3(256), 0, static_cast<cudaStream_t>(stream));
  if (cudaLaunchKernelEx(&L.cfg, kernel, p) != cudaSuccess) return MOE_ERR_CUDA;
  note_launches(1);
  return MOE_OK;
}

// Rows quantised to 8-bit integers with a scale each (moe_int8_quantize;
// include/moe_experts.h), with the arithmetic of dispatch's quant_mode 2
// (quant_common.cuh): scale = amax / 127, code = round(x / scale).
//
// One pass over the data, bound by HBM: a row stays in registers between its maximum
// and its codes, in a warp's where it has up to 2048 elements, in a block's up to
// 32768; as the codes of its elements are made, the next row's take their registers.
// Rows go in pieces of 8 elements (16-byte loads), 2 or 1, as they align. Longer rows are
// read twice, the second time from cache; of narrow pieces, shorter ones too.
//
// Measured, bf16: 131072 rows of 2048 130 us, 6.2 TB/s; of 2046, in pieces of 2 elements, 129; of 2047, one by one,
// 319 (waiting for its loads of 2 bytes a lane); 4096 rows of 512 3.1 us; 16384 rows of 16384 125 us, 6.4 TB/s, of 18432
// 162, 5.6 TB/s, of 65536 (read twice) 781, 4.1 TB/s.
#include "../../include/moe_experts.h"
#include "experts_host.h"
#include "quant_common.cuh"

#include <type_traits>

namespace crs {

constexpr int kInt8Threads = 256;
constexpr int kInt8CountedMats = 1024;  // matrices with row counts: one for each rank

struct Int8QuantParams {
  const void* x;
  const int32_t* counts;  // [mats][counts_len], or null
  int8_t* codes;
  float* scales;
  long long rows, row_stride, mat_stride;
  int mats, cols, counts_len;
};

// The rows to work on, numbered through: matrix and row of number i, found in ascending order.
struct Int8Rows {
  const Int8QuantParams& p;
  const int* pre;  // running row counts [mats + 1], with counts
  long long total;
  int m = 0;
  __device__ Int8Rows(const Int8QuantParams& p_, int* s_pre) : p(p_), pre(s_pre) {
    total = (long long)p.mats * p.rows;
    if (!p.counts) return;
    if (threadIdx.x < 32) {
      int carry = 0;
      for (int m0 = 0; m0 < p.mats; m0 += 32) {
        const int mine = m0 + (int)threadIdx.x;
        int n = mine < p.mats ? p.counts[(size_t)mine * p.counts_len + p.counts_len - 1] : 0;
        n = n < 0 ? 0 : n > p.rows ? (int)p.rows : n;
        int sum = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int below = __shfl_up_sync(0xffffffffu, sum, o);
          if ((int)threadIdx.x >= o) sum += below;
        }
        if (mine < p.mats) s_pre[mine] = carry + sum - n;
        carry += __shfl_sync(0xffffffffu, sum, 31);
      }
      if (threadIdx.x == 0) s_pre[p.mats] = carry;
    }
    __syncthreads();
    total = s_pre[p.mats];
  }
  // where row i begins in x (elements) and its place among all rows of codes and scales
  __device__ size_t find(long long i, size_t& place) {
    long long r;
    if (p.counts) {
      while (i >= pre[m + 1]) ++m;
      r = i - pre[m];
    } else {
      m = (int)(i / p.rows);
      r = i - (long long)m * p.rows;
    }
    place = (size_t)m * p.rows + r;
    return (size_t)(m * p.mat_stride + r * p.row_stride);
  }
};

// 8 elements of a row as loaded, and as fp32 pairs: PIECE neighbours (8, 2 or 1, as the rows align) at a time, unit j's
// pieces THREADS * PIECE elements apart; zeros beyond the row's end.
template <int DT, int PIECE, int THREADS>
struct Int8Unit {
  static constexpr int kLoads = DT == MOE_F32 ? 2 : 1, kPieces = 8 / PIECE;
  int4 v[kLoads];
  static __device__ int element(int t, int j, int piece) { return ((j * kPieces + piece) * THREADS + t) * PIECE; }
  // `row` begins at the row's first element
  __device__ void load(const uint8_t* row, int t, int j, int cols) {
    if constexpr (PIECE == 8) {
      const int c = element(t, j, 0);
#pragma unroll
      for (int i = 0; i < kLoads; ++i)
        v[i] = c < cols ? ld_nc_v4(row + (size_t)c * (DT == MOE_F32 ? 4 : 2) + i * 16) : make_int4(0, 0, 0, 0);
    } else {
      uint32_t w[4 * kLoads];
#pragma unroll
      for (int q = 0; q < kPieces; ++q) {
        const int c = element(t, j, q);
        if constexpr (DT == MOE_F32 && PIECE == 2) {
          const float2 f = c < cols ? __ldg(reinterpret_cast<const float2*>(reinterpret_cast<const float*>(row) + c)) : float2{0.f, 0.f};
          w[2 * q] = __float_as_uint(f.x), w[2 * q + 1] = __float_as_uint(f.y);
        } else if constexpr (DT == MOE_F32) {
          w[q] = c < cols ? __float_as_uint(__ldg(reinterpret_cast<const float*>(row) + c)) : 0u;
        } else if constexpr (PIECE == 2) {
          w[q] = c < cols ? __ldg(reinterpret_cast<const uint32_t*>(reinterpret_cast<const uint16_t*>(row) + c)) : 0u;
        } else {
          const uint32_t h = c < cols ? (uint32_t)__ldg(reinterpret_cast<const uint16_t*>(row) + c) : 0u;
          if (q & 1) w[q / 2] |= h << 16;
          else w[q / 2] = h;
        }
      }
#pragma unroll
      for (int i = 0; i < kLoads; ++i) v[i] = make_int4((int)w[4 * i], (int)w[4 * i + 1], (int)w[4 * i + 2], (int)w[4 * i + 3]);
    }
  }
  static __device__ void store(int8_t* out, int t, int j, int cols, uint2 codes) {
#pragma unroll
    for (int q = 0; q < kPieces; ++q) {
      const int c = element(t, j, q);
      if (c >= cols) break;
      if constexpr (PIECE == 8) *reinterpret_cast<uint2*>(out + c) = codes;
      else if constexpr (PIECE == 2)
        *reinterpret_cast<uint16_t*>(out + c) = (uint16_t)((q < 2 ? codes.x : codes.y) >> (16 * (q & 1)));
      else out[c] = (int8_t)((q < 4 ? codes.x : codes.y) >> (8 * (q & 3)));
    }
  }
  // The largest magnitude: of 16-bit elements pair by pair, in their own type.
  __device__ float amax(float m) const {
    if constexpr (DT == MOE_F32) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        m = fmax_abs3(m, __int_as_float(v[i].x), __int_as_float(v[i].y));
        m = fmax_abs3(m, __int_as_float(v[i].z), __int_as_float(v[i].w));
      }
      return m;
    } else {
      using T = typename std::conditional<DT == MOE_F16, __half2, __nv_bfloat162>::type;
      const T* h = reinterpret_cast<const T*>(v);
      const T a = __hmax2(__hmax2(__habs2(h[0]), __habs2(h[1])), __hmax2(__habs2(h[2]), __habs2(h[3])));
      return fmax_abs3(m, __low2float(a), __high2float(a));
    }
  }
  // Keeps what was computed from the elements so far from being held in registers in their place.
  __device__ void forget() {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) asm volatile("" : "+r"(v[i].x), "+r"(v[i].y), "+r"(v[i].z), "+r"(v[i].w));
  }
  __device__ void pairs(f32x2 (&o)[4]) const {
    if constexpr (DT == MOE_F32) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        o[2 * i] = f2_pack(__int_as_float(v[i].x), __int_as_float(v[i].y));
        o[2 * i + 1] = f2_pack(__int_as_float(v[i].z), __int_as_float(v[i].w));
      }
    } else {
      unpack8x2<DT>(v[0], o);
    }
  }
};

// The largest magnitude among the THREADS threads of a warp or of the block.
template <int THREADS>
__device__ __forceinline__ float int8_amax(float m, float (&s_max)[THREADS / 32]) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (THREADS == 32) return m;
  __syncthreads();  // the row before is done with s_max
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
  __syncthreads();
  m = s_max[threadIdx.x & (THREADS / 32 - 1)];
#pragma unroll
  for (int o = THREADS / 64; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

template <int DT>
__device__ __forceinline__ float int8_load(const void* x, size_t i) {
  if constexpr (DT == MOE_F32) return static_cast<const float*>(x)[i];
  else return load_elem(x, i, DT);
}

// The codes of 8 elements, round(v / scale), from r = 1 / scale rounded to nearest: y = v * r is up to 1.5 ulps off the
// quotient, and y + r * (v - y * scale), by fused multiply-adds, off it by a rounding and less than 2^-20 of an ulp before
// that (after Markstein 1990, whose y is within one ulp); adding 1.5 * 2^23 leaves the integer in the low byte. That no
// code differs from the division's was compared next to every half step for each of the 2^23 mantissas that a row's
// largest magnitude may have (tests/test_int8_half_steps_gpu.py); powers of two change nothing, for scales whose residuals
// do not underflow (int8_rcp_ok); a quotient of smaller elements is 0 in any case. (dispatch's token_codes8
// takes the division where a product is near a half, which of bf16 rows is every other eight: half the largest
// magnitude, 63.5, is a frequent number.)
__device__ __forceinline__ bool int8_rcp_ok(float scale) { return scale >= 7.8886091e-31f && scale <= 3.40282347e38f; }  // 2^-100
__device__ __forceinline__ uint2 int8_codes(const f32x2 (&v)[4], f32x2 scale2, f32x2 rcp2) {
  const f32x2 shift2 = f2_pack(kRoundShift, kRoundShift);
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f32x2 y = f2_mul(v[i], rcp2);
    const f32x2 t = f2_add(f2_fma(f2_fma(y, scale2, v[i]), rcp2, y), shift2);
    float tl, th;
    f2_split(t, tl, th);
    c[2 * i] = __float_as_uint(tl);
    c[2 * i + 1] = __float_as_uint(th);
  }
  return pack8_low(c);
}

// Rows that a warp's or (THREADS > 32) the block's threads hold as NV units each; x, its strides, cols and codes
// aligned for pieces of PIECE elements (with 8: 16 bytes of x).
template <int DT, int PIECE, int NV, int THREADS>
__global__ void __launch_bounds__(THREADS > 32 ? THREADS : kInt8Threads,
                                  ((DT == MOE_F32 ? 2 * NV : NV) > 8 ? 2 : 4) / (THREADS > kInt8Threads ? 2 : 1))
    int8_quantize_kernel(Int8QuantParams p) {
  constexpr bool BLOCK = THREADS > 32;
  __shared__ int s_pre[kInt8CountedMats + 1];
  __shared__ float s_max[THREADS / 32];
  pdl_wait();
  pdl_launch_dependents();
  const int t = BLOCK ? threadIdx.x : threadIdx.x & 31;
  const uint8_t* x = static_cast<const uint8_t*>(p.x);
  constexpr size_t kEs = DT == MOE_F32 ? 4 : 2;
  Int8Rows rows(p, s_pre);
  const long long first = BLOCK ? blockIdx.x : blockIdx.x * (kInt8Threads / 32ll) + (threadIdx.x >> 5);
  const long long step = BLOCK ? gridDim.x : gridDim.x * (kInt8Threads / 32ll);
  if (first >= rows.total) return;
  size_t place;
  size_t from = rows.find(first, place);
  Int8Unit<DT, PIECE, THREADS> u[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) u[j].load(x + from * kEs, t, j, p.cols);
  for (long long i = first; i < rows.total; i += step) {
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      m = u[j].amax(m);
      u[j].forget();
    }
    m = int8_amax<THREADS>(m, s_max);
    const float scale = __fdiv_rn(m, 127.0f);
    const float rcp = __frcp_rn(scale);
    const f32x2 rcp2 = f2_pack(rcp, rcp), scale2 = f2_pack(-scale, -scale);
    int8_t* out = p.codes + place * p.cols;
    if (t == 0) p.scales[place] = scale;
    if (!int8_rcp_ok(scale)) {  // zeros, infinities, the smallest numbers: by the division, an element at a time
#pragma unroll 1
      for (int c = t; c < p.cols; c += THREADS) out[c] = (int8_t)(m == 0.f ? 0 : token_q(int8_load<DT>(p.x, from + c), scale));
    }
    const bool fast = int8_rcp_ok(scale), more = i + step < rows.total;
    if (more) from = rows.find(i + step, place);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (u[j].element(t, j, 0) >= p.cols) break;
      f32x2 v[4];
      u[j].pairs(v);
      if (more) u[j].load(x + from * kEs, t, j, p.cols);  // of the next row, under way while this one's codes are made
      if (fast) u[j].store(out, t, j, p.cols, int8_codes(v, scale2, rcp2));
    }
  }
}

// Rows that a block's registers do not hold: read twice, the second time from cache.
template <int DT, int PIECE>
__global__ void __launch_bounds__(kInt8Threads, 4) int8_quantize_long_kernel(Int8QuantParams p) {
  __shared__ int s_pre[kInt8CountedMats + 1];
  __shared__ float s_max[kInt8Threads / 32];
  pdl_wait();
  pdl_launch_dependents();
  using Unit = Int8Unit<DT, PIECE, kInt8Threads>;
  const int t = threadIdx.x;
  Int8Rows rows(p, s_pre);
  for (long long i = blockIdx.x; i < rows.total; i += gridDim.x) {
    size_t place;
    const size_t from = rows.find(i, place);
    const uint8_t* x = static_cast<const uint8_t*>(p.x) + from * (DT == MOE_F32 ? 4 : 2);
    float m = 0.f;
#pragma unroll 8
    for (int j = 0; Unit::element(t, j, 0) < p.cols; ++j) {
      Unit u;
      u.load(x, t, j, p.cols);
      m = u.amax(m);
    }
    m = int8_amax<kInt8Threads>(m, s_max);
    const float scale = __fdiv_rn(m, 127.0f);
    int8_t* out = p.codes + place * p.cols;
    if (int8_rcp_ok(scale)) {
      const float rcp = __frcp_rn(scale);
      const f32x2 rcp2 = f2_pack(rcp, rcp), scale2 = f2_pack(-scale, -scale);
#pragma unroll 8
      for (int j = 0; Unit::element(t, j, 0) < p.cols; ++j) {
        Unit u;
        u.load(x, t, j, p.cols);
        f32x2 v[4];
        u.pairs(v);
        u.store(out, t, j, p.cols, int8_codes(v, scale2, rcp2));
      }
    } else {
#pragma unroll 1
      for (int c = t; c < p.cols; c += kInt8Threads) out[c] = (int8_t)(m == 0.f ? 0 : token_q(int8_load<DT>(p.x, from + c), scale));
    }
    if (t == 0) p.scales[place] = scale;
  }
}

struct Int8QuantKernel {
  void (*kernel)(Int8QuantParams);
  int threads;  // to a row
};

// The narrowest group of threads that holds a row.
template <int DT, int PIECE>
Int8QuantKernel int8_quant_kernel(int cols) {
  if (cols <= 256) return {int8_quantize_kernel<DT, PIECE, 1, 32>, 32};
  if (cols <= 512) return {int8_quantize_kernel<DT, PIECE, 2, 32>, 32};
  if (cols <= 1024) return {int8_quantize_kernel<DT, PIECE, 4, 32>, 32};
  if (cols <= 2048) return {int8_quantize_kernel<DT, PIECE, 8, 32>, 32};
  // A block holds longer rows as far as their pieces are wide. One by one the kernel that reads rows twice is faster (bf16,
  // 16384 rows of 16383 223 us, held 310; 32768 of 4095 159 and 183; but 65536 of 2047 202, held by a warp 165), by twos
  // it is as fast above 16384 (16384 of 18430 183, held 188), in 16-byte pieces slower (18432 216, held 162).
  if constexpr (PIECE > 1) {
    if (cols <= 8192) return {int8_quantize_kernel<DT, PIECE, 4, 256>, 256};
    if (cols <= 16384) return {int8_quantize_kernel<DT, PIECE, 8, 256>, 256};
  }
  if constexpr (PIECE == 8) {
    if (cols <= 32768) return {int8_quantize_kernel<DT, PIECE, 8, 512>, 512};
  }
  return {int8_quantize_long_kernel<DT, PIECE>, kInt8Threads};
}
template <int DT>
Int8QuantKernel int8_quant_kernel(int cols, int piece) {
  return piece == 8 ? int8_quant_kernel<DT, 8>(cols) : piece == 2 ? int8_quant_kernel<DT, 2>(cols) : int8_quant_kernel<DT, 1>(cols);
}

}  // namespace crs

extern "C" moe_status_t moe_int8_quantize(const void* x, int32_t x_dtype, int32_t mats, int64_t rows, int32_t cols,
                                          int64_t row_stride, int64_t mat_stride, const int32_t* counts,
                                          int32_t counts_len, int8_t* codes, float* scales, void* stream) {
  using namespace crs;
  if (x_dtype != MOE_F32 && x_dtype != MOE_F16 && x_dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (mats < 0 || rows < 0 || cols < 1 || cols > (1 << 30)) return MOE_ERR_INVALID_ARG;
  if (rows >= 2147483648LL || mats * rows >= 2147483648LL) return MOE_ERR_INVALID_ARG;
  if (row_stride < cols || mat_stride < 0) return MOE_ERR_INVALID_ARG;
  if (counts && (counts_len < 1 || mats > kInt8CountedMats || (uintptr_t)counts % 4)) return MOE_ERR_INVALID_ARG;
  if (mats == 0 || rows == 0) return MOE_OK;
  const int es = x_dtype == MOE_F32 ? 4 : 2;
  if (!x || !codes || !scales || (uintptr_t)x % es || (uintptr_t)scales % 4) return MOE_ERR_INVALID_ARG;
  const int nsm = num_sms_of_current_device();
  if (nsm <= 0) return MOE_ERR_CUDA;
  const Int8QuantParams p{x, counts, codes, scales, rows, row_stride, mat_stride, mats, cols, counts_len};
  const auto fits = [&](int piece, unsigned bytes) {  // of x that a piece's load takes
    return cols % piece == 0 && (uintptr_t)x % bytes == 0 && (mats * rows == 1 || row_stride * es % bytes == 0) &&
           (mats == 1 || mat_stride * es % bytes == 0) && (uintptr_t)codes % piece == 0;
  };
  const int piece = fits(8, 16) ? 8 : fits(2, 2 * es) ? 2 : 1;
  const Int8QuantKernel k = x_dtype == MOE_F32   ? int8_quant_kernel<MOE_F32>(cols, piece)
                            : x_dtype == MOE_F16 ? int8_quant_kernel<MOE_F16>(cols, piece)
                                                 : int8_quant_kernel<MOE_BF16>(cols, piece);
  int per_sm = 0;
  const int threads = k.threads > 32 ? k.threads : kInt8Threads;
  if (resident_blocks((const void*)k.kernel, threads, 0, &per_sm) != cudaSuccess || per_sm < 1) return MOE_ERR_CUDA;
  const long long need = k.threads > 32 ? mats * rows : (mats * rows + kInt8Threads / 32 - 1) / (kInt8Threads / 32);
  const long long most = (long long)nsm * per_sm;
  PdlLaunch L(dim3((unsigned)(need < most ? need : most)), dim3(threads), 0, static_cast<cudaStream_t>(stream));
  if (cudaLaunchKernelEx(&L.cfg, k.kernel, p) != cudaSuccess) return MOE_ERR_CUDA;
  note_launches(1);
  return MOE_OK;
}

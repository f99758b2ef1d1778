// The experts' product on dispatched MX FP4 rows (moe_expert_product;
// include/moe_experts.h): z[r][j] = sum_i x[r][i] * w[e(r)][j][i] over the rows
// that ep_recv_count gives to each expert, then the epilogue.
//
// On the tensor cores' block-scaled path (tcgen05.mma kind::mxf4: E2M1 codes, one
// E8M0 scale for 32 elements of K, fp32 accumulators in TMEM):
//   * a unit is 128 rows of one expert (the MMA's A operand) against up to 256
//     of its weight rows (B). The rows are A although an expert may have only a
//     few: streaming weights from HBM takes 23 bytes a clock and SM, the MMA eats
//     64 of them a clock, so the unused rows cost nothing that is short, and
//     each epilogue thread has one row with neighbouring features in registers;
//   * codes come by TMA in 128-byte-swizzled boxes, 256 elements of K a stage;
//     only as many 32-row boxes of A as the unit has rows;
//   * the weights' scales, laid out in the tensor cores' order (MOE_SF_TILED), come
//     by one bulk copy for 128 rows and 256 elements; the rows' scales lie a row
//     after the other as dispatch wrote them: a warp brings them into the same
//     order with 4-byte cp.async. tcgen05.cp then takes both to TMEM, in the
//     MMA's own issue order;
//   * warps: 0 TMA, 1 MMA, 2 row scales, 4..11 epilogue (two for each quarter of
//     the accumulator's lanes). An epilogue thread takes its whole share of the
//     accumulator into registers (128 of them) and hands it back at once, so one
//     accumulator is enough: the next unit's MMAs run while this one is stored;
//   * one persistent CTA an SM; units are dealt out round-robin over all experts
//     (their running tile counts are scanned in shared memory), n-tiles of one
//     row tile adjacent, so that rows and weights are read from L2 but once from HBM.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <mutex>

#include "../../include/moe_experts.h"
#include "quant_common.cuh"
#include "tcgen05.cuh"

namespace crs {

struct ProductParams {
  const uint8_t* xs;       // [W*A][K/32]
  const int32_t* ep;       // [W][L*W]
  const uint8_t* wsf;      // [E][nt128][kt128][512]
  void* y;                 // [W*A][C]
  uint8_t* ys;             // [W*A][ceil(C/32)], MX FP4 output
  int W, L, E, N, K, C;    // C output columns
  long long A;
  int* status;
  uint64_t timeout_ns;
};

constexpr int kProductThreads = 384;
constexpr int kProductStages = 4;
constexpr int kEpilogueWarp = 4;             // first of the eight
constexpr int kRowsTile = 128;               // MMA M
constexpr int kMaxBoxes = 4;                 // of 64 weight rows: MMA N <= 256
constexpr int kKStage = 256;                 // elements of K a stage: 128 bytes a row
constexpr uint32_t kABytes = kRowsTile * 128;
constexpr uint32_t kBBox = 64 * 128;
constexpr uint32_t kBBytes = kMaxBoxes * kBBox;
constexpr uint32_t kSfaBytes = 2 * 512;      // 128 rows x 8 scales
constexpr uint32_t kSfbBytes = 2 * 1024;     // 2 x 128 rows x 8 scales
constexpr uint32_t kProductStage = kABytes + kBBytes + kSfaBytes + kSfbBytes;
static_assert(kProductStage % 1024 == 0, "stages stay 1024-byte aligned");
constexpr uint32_t kSfCols = 24;             // TMEM columns of a stage's scales: 2 x 4 of the rows, 2 x 8 of the weights
constexpr uint32_t kAccCols = 256;

// Shared memory behind the stages: running row tiles [E+1], first row [E], row count [E].
__host__ __device__ inline size_t product_smem(int E) {
  return 1024 + (size_t)kProductStages * kProductStage + ((size_t)3 * E + 1) * 4;
}

struct ProductUnit {
  int e, n0, rows;
  long long row0;
};

__device__ __forceinline__ ProductUnit product_unit(const ProductParams& p, const int* pre, int u, int n_tiles, int width) {
  const int mt = u / n_tiles;
  int lo = 0, hi = p.E;  // the expert whose tiles [pre[e], pre[e+1]) hold mt
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= mt) lo = mid;
    else hi = mid;
  }
  const int* first = pre + p.E + 1;
  const int* count = first + p.E;
  const int at = (mt - pre[lo]) * kRowsTile;
  ProductUnit x;
  x.e = lo;
  x.n0 = (u - mt * n_tiles) * width;
  x.rows = min(kRowsTile, count[lo] - at);
  x.row0 = (long long)(lo / p.L) * p.A + first[lo] + at;
  return x;
}

struct ProductAbort {
  volatile int* flag;
  int* status;
  uint64_t limit;
};

__device__ __forceinline__ bool product_wait(uint64_t* bar, uint32_t parity, const ProductAbort& a) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t it = 0;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 63u) == 63u) {
      if (*a.flag) return false;
      if (globaltimer_ns() - t0 > a.limit) {
        set_error(a.status, MOE_ERR_TIMEOUT);
        *a.flag = 1;
        return false;
      }
    }
  }
}

// Scales of rows [row0, row0 + rows) for one stage, in the tensor cores' order:
// the 4 bytes of row r and k-group j at j * 512 + (r % 32) * 16 + (r / 32) * 4.
// Whole 4-byte groups (K % 128 == 0) go by cp.async; other row lengths leave
// unaligned rows, whose bytes are gathered by plain loads.
__device__ __forceinline__ void load_row_scales(const ProductParams& p, const ProductUnit& un, int kb, uint8_t* dst) {
  const int lane = threadIdx.x & 31, blocks = p.K / 32, left = blocks - kb * 8;
  const uint8_t* src = p.xs + (size_t)un.row0 * blocks + kb * 8;
  if ((blocks & 3) == 0) {
    const int groups = left >= 8 ? 2 : 1;
    for (int r = lane; r < un.rows; r += 32)
      for (int j = 0; j < groups; ++j)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst + j * 512 + lane * 16 + (r >> 5) * 4)),
                     "l"(src + (size_t)r * blocks + j * 4)
                     : "memory");
  } else {
    for (int r = lane; r < un.rows; r += 32)
      for (int j = 0; j < 2; ++j) {
        uint32_t v = 0;
        for (int b = 0; b < 4; ++b)
          if (j * 4 + b < left) v |= (uint32_t)__ldg(src + (size_t)r * blocks + j * 4 + b) << (8 * b);
        *reinterpret_cast<uint32_t*>(dst + j * 512 + lane * 16 + (r >> 5) * 4) = v;
      }
  }
}

template <int YT>
__device__ __forceinline__ uint32_t pack_y(float lo, float hi) {
  if (YT == MOE_F16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// CNT neighbouring results of one row from column c on.
template <int YT, int CNT>
__device__ __forceinline__ void store_results(const ProductParams& p, long long row, int c, const float (&v)[CNT]) {
  if (YT == MOE_MXFP4) {
#pragma unroll
    for (int b = 0; b < CNT / 32; ++b) {
      const int cb = c + 32 * b, n = min(32, p.C - cb);
      if (n <= 0) return;
      float m = 0.f;
#pragma unroll
      for (int j = 0; j < 32; ++j) m = fmaxf(m, fabsf(v[32 * b + j]));  // columns beyond C are zeros
      const int se = mx_exponent(m, 2);
      const float inv = exp2_exact(-se);
      uint32_t q[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        q[i] = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          q[i] |= cvt_fp4x2(__fmul_rn(v[32 * b + 8 * i + 2 * j], inv), __fmul_rn(v[32 * b + 8 * i + 2 * j + 1], inv)) << (8 * j);
      }
      uint8_t* out = static_cast<uint8_t*>(p.y) + (size_t)row * (p.C / 2) + cb / 2;
      if (n == 32 && (p.C & 31) == 0) {
        st_v4(out, make_int4(q[0], q[1], q[2], q[3]));
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (2 * i < n) out[i] = (uint8_t)(q[i / 4] >> (8 * (i % 4)));
      }
      p.ys[(size_t)row * ((p.C + 31) / 32) + cb / 32] = (uint8_t)(se + 127);
    }
  } else {
    uint16_t* out = static_cast<uint16_t*>(p.y) + (size_t)row * p.C + c;
    if ((p.C & 7) == 0) {
#pragma unroll
      for (int i = 0; i < CNT; i += 8)
        if (c + i < p.C)
          st_v4(out + i, make_int4(pack_y<YT>(v[i], v[i + 1]), pack_y<YT>(v[i + 2], v[i + 3]), pack_y<YT>(v[i + 4], v[i + 5]),
                                   pack_y<YT>(v[i + 6], v[i + 7])));
    } else {
#pragma unroll
      for (int i = 0; i < CNT; i += 2) {
        const uint32_t w = pack_y<YT>(v[i], v[i + 1]);
        if (c + i < p.C) out[i] = (uint16_t)w;
        if (c + i + 1 < p.C) out[i + 1] = (uint16_t)(w >> 16);
      }
    }
  }
}

template <int YT, bool SWIGLU>
__global__ void __launch_bounds__(kProductThreads, 1)
    expert_product_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                          ProductParams p) {
  extern __shared__ __align__(1024) uint8_t psm_raw[];
  __shared__ __align__(8) uint64_t full[kProductStages], empty[kProductStages], acc_full, acc_empty, drained;
  __shared__ uint32_t tmem_slot;
  __shared__ long long scan_scratch[32];
  __shared__ volatile int s_abort;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* sm = psm_raw + ((1024u - (smem_u32(psm_raw) & 1023u)) & 1023u);
  int* pre = reinterpret_cast<int*>(sm + (size_t)kProductStages * kProductStage);

  if (threadIdx.x == 0) {
    for (int i = 0; i < kProductStages; ++i) {
      mbar_init(&full[i], 2);  // the TMA thread's expect_tx and the row-scale warp
      mbar_init(&empty[i], 1);
    }
    mbar_init(&acc_full, 1);
    mbar_init(&acc_empty, kProductThreads / 32 - kEpilogueWarp);
    mbar_init(&drained, 1);
    mbar_fence_init();
    s_abort = 0;
  }
  if (warp == 1) {
    tmem_alloc(&tmem_slot, 512);
    tmem_relinquish();
  }
  pdl_wait();
  pdl_launch_dependents();

  // running row tiles of the experts
  {
    int* first = pre + p.E + 1;
    int* count = first + p.E;
    long long carry = 0;
    for (int e0 = 0; e0 < p.E; e0 += kProductThreads) {
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
        }
        first[e] = lo;
        count[e] = n;
      }
      const long long tiles = (n + kRowsTile - 1) / kRowsTile;
      const long long before = carry + block_exclusive_scan(tiles, scan_scratch);
      if (e < p.E) {
        pre[e] = (int)before;
        if (e == p.E - 1) pre[p.E] = (int)(before + tiles);
      }
      __syncthreads();
      // the last expert of this pass carries on
      const int last = min(p.E, e0 + kProductThreads) - 1;
      carry = pre[last] + (count[last] + kRowsTile - 1) / kRowsTile;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const uint32_t tmem_sf = tmem + kAccCols;

  const int m_tiles = pre[p.E], KB = (p.K + kKStage - 1) / kKStage;
  // weight rows a unit: the width whose rounds of units cost least, a unit's
  // cost being its weight rows and half a box for its rows and its ends
  int boxes = 1;
  {
    long long best = 1ll << 62;
    for (int b = kMaxBoxes; b >= 1; --b) {
      const long long units = (long long)m_tiles * ((p.N + 64 * b - 1) / (64 * b));
      const long long cost = (units + gridDim.x - 1) / gridDim.x * (2 * b + 1);
      if (cost < best) {
        best = cost;
        boxes = b;
      }
    }
  }
  const int width = boxes * 64, n_tiles = (p.N + width - 1) / width;
  const int units = m_tiles * n_tiles;
  const ProductAbort ab{&s_abort, p.status, p.timeout_ns};

  if (warp == 0) {
    if (lane == 0) {
      const int nt128 = (p.N + 127) / 128, kt128 = (p.K + 127) / 128;
      uint32_t it = 0;
      for (int u = blockIdx.x; u < units && !s_abort; u += gridDim.x) {
        const ProductUnit un = product_unit(p, pre, u, n_tiles, width);
        const int a_boxes = (un.rows + 31) >> 5;
        const int c0 = un.n0 >> 7, chunks = min(nt128, (un.n0 + width + 127) >> 7) - c0;
        const uint8_t* sf = p.wsf + ((size_t)un.e * nt128 + c0) * kt128 * 512;
        for (int kb = 0; kb < KB; ++kb, ++it) {
          const uint32_t stage = it % kProductStages, round = it / kProductStages;
          if (round > 0 && !product_wait(&empty[stage], (round - 1) & 1u, ab)) break;
          uint8_t* st = sm + stage * kProductStage;
          const uint32_t sf_bytes = 512u * (uint32_t)min(2, kt128 - 2 * kb);
          mbar_arrive_expect_tx(&full[stage], (uint32_t)a_boxes * 4096u + (uint32_t)boxes * kBBox + (uint32_t)chunks * sf_bytes);
          for (int b = 0; b < boxes; ++b)
            tma_load_3d(st + kABytes + b * kBBox, &map_w, kb * 128, un.n0 + b * 64, un.e, &full[stage]);
          for (int b = 0; b < a_boxes; ++b)
            tma_load_2d(st + b * 4096, &map_x, kb * 128, (int)(un.row0 + b * 32), &full[stage]);
          for (int c = 0; c < chunks; ++c)
            bulk_g2s(st + kABytes + kBBytes + kSfaBytes + c * 1024, sf + ((size_t)c * kt128 + 2 * kb) * 512, sf_bytes,
                     &full[stage]);
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = idesc_mxf4(width);
      uint32_t it = 0, done = 0;
      for (int u = blockIdx.x; u < units && !s_abort; u += gridDim.x, ++done) {
        const ProductUnit un = product_unit(p, pre, u, n_tiles, width);
        const int c0 = un.n0 >> 7, chunks = ((un.n0 + width + 127) >> 7) - c0;
        const uint32_t shift = (un.n0 & 127) >> 5;  // columns before the unit's first weight row: 0 or 2
        if (done > 0 && !product_wait(&acc_empty, (done - 1) & 1u, ab)) break;
        tc_fence_after();
        for (int kb = 0; kb < KB; ++kb, ++it) {
          const uint32_t stage = it % kProductStages, round = it / kProductStages;
          if (!product_wait(&full[stage], round & 1u, ab)) break;
          tc_fence_after();
          const uint8_t* st = sm + stage * kProductStage;
          const uint8_t* sfa = st + kABytes + kBBytes;
          const uint32_t ta = tmem_sf + stage * kSfCols, tb = ta + 8;
          const int steps = min(4, (p.K - kb * kKStage + 63) / 64);
          for (int j = 0; j < (steps + 1) / 2; ++j) {
            tc_cp_scales(ta + 4 * j, sf_desc(sfa + j * 512));
            for (int c = 0; c < chunks; ++c) tc_cp_scales(tb + 8 * j + 4 * c, sf_desc(sfa + kSfaBytes + c * 1024 + j * 512));
          }
          const uint64_t adesc = sw128_desc(st), bdesc = sw128_desc(st + kABytes);
          for (int kk = 0; kk < steps; ++kk) {
            const uint32_t id = (kk & 1) * 2;  // which two of a column's four scales
            tc_mma_mxf4(tmem, adesc + 2 * kk, bdesc + 2 * kk, idesc | (id << 4) | (id << 29), ta + 4 * (kk >> 1),
                        tb + 8 * (kk >> 1) + shift, (kb | kk) != 0);
          }
          tc_commit(&empty[stage]);
        }
        tc_commit(&acc_full);
      }
      tc_commit(&drained);
    }
  } else if (warp == 2) {
    // row scales: cp.async of stage it, arrival for the stage two before
    uint32_t it = 0;
    const auto arrive = [&](uint32_t stage) {
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[stage]);
    };
    bool ok = true;
    for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
      const ProductUnit un = product_unit(p, pre, u, n_tiles, width);
      for (int kb = 0; kb < KB; ++kb, ++it) {
        const uint32_t stage = it % kProductStages, round = it / kProductStages;
        if (round > 0) {
          ok = product_wait(&empty[stage], (round - 1) & 1u, ab);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
        }
        load_row_scales(p, un, kb, sm + stage * kProductStage + kABytes + kBBytes);
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (it >= 2) {
          asm volatile("cp.async.wait_group 2;" ::: "memory");
          arrive((it - 2) % kProductStages);
        }
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (ok)
      for (uint32_t i = it >= 2 ? it - 2 : 0; i < it; ++i) arrive(i % kProductStages);
  } else if (warp >= kEpilogueWarp) {
    const int q = warp & 3, half = (warp - kEpilogueWarp) >> 2;
    uint32_t done = 0;
    for (int u = blockIdx.x; u < units && !s_abort; u += gridDim.x, ++done) {
      const ProductUnit un = product_unit(p, pre, u, n_tiles, width);
      if (!product_wait(&acc_full, done & 1u, ab)) break;
      tc_fence_after();
      const int r = 32 * q + lane;
      const bool mine = 32 * q < un.rows && half < boxes;
      uint32_t v[2][64];
      if (mine) {
        const uint32_t t = tmem + ((uint32_t)(32 * q) << 16) + half * 64;
        tc_ld64(t, v[0]);
        if (half + 2 < boxes) tc_ld64(t + 128, v[1]);
        tc_wait_ld();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty);
      if (mine && r < un.rows) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int n = un.n0 + (half + 2 * i) * 64;
          if (half + 2 * i >= boxes || n >= p.N) break;
          if (SWIGLU) {
            float h[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const float g = __uint_as_float(v[i][2 * j]), up = __uint_as_float(v[i][2 * j + 1]);
              // __fdividef is within 2 ulps, far below the rounding to 16 or 4 bits that follows
              h[j] = __fdividef(g, 1.0f + expf(-g)) * up;
            }
            store_results<YT>(p, un.row0 + r, n / 2, h);
          } else {
            float h[64];
#pragma unroll
            for (int j = 0; j < 64; ++j) h[j] = __uint_as_float(v[i][j]);
            store_results<YT>(p, un.row0 + r, n, h);
          }
        }
      }
    }
  }

  __syncthreads();
  if (threadIdx.x == 0) {
    // the MMAs, and after an abort the copies in flight, end before their memory is given back
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(&drained, 0) && globaltimer_ns() - t0 < 1000000ull) {}
    if (s_abort)
      while (globaltimer_ns() - t0 < 1000000ull) {}
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------- host side

static PFN_cuTensorMapEncodeTiled_v12000 product_encode_fn() {
  static std::once_flag once;
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// Packed codes [depth][rows][bytes], boxes of 128 bytes x box_rows rows; beyond
// the ends of a matrix they read as zeros.
static bool product_map(CUtensorMap* m, const void* base, unsigned long long bytes, unsigned long long rows,
                        unsigned long long depth, unsigned box_rows) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = product_encode_fn();
  if (!enc) return false;
  cuuint64_t dims[3] = {bytes, rows, depth};
  cuuint64_t strides[2] = {bytes, bytes * rows};
  cuuint32_t box[3] = {128, box_rows, 1};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, depth ? 3 : 2, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

typedef void (*ProductKernel)(CUtensorMap, CUtensorMap, ProductParams);
template <int YT>
ProductKernel product_kernel(bool swiglu) {
  return swiglu ? expert_product_kernel<YT, true> : expert_product_kernel<YT, false>;
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
  // units of 128 rows x 64 weight rows are counted in 32 bits
  if ((long long)E * n >= 2147483647LL || ((long long)W * A / kRowsTile + E) * ((n + 63) / 64) >= 2147483647LL)
    return MOE_ERR_INVALID_ARG;
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

  CUtensorMap mx, mw;
  if (!product_map(&mx, x, (unsigned long long)k / 2, (unsigned long long)W * A, 0, 32) ||
      !product_map(&mw, w, (unsigned long long)k / 2, (unsigned long long)n, (unsigned long long)E, 64))
    return MOE_ERR_CUDA;
  ProductParams p{};
  p.xs = x_scales;
  p.ep = ep_recv_count;
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
  p.status = &static_cast<WsHeader*>(ws)->status;
  p.timeout_ns = (uint64_t)cfg->wait_timeout_us * 1000ull;
  const bool sw = epilogue == MOE_EPI_SWIGLU;
  const ProductKernel kernel = y_dtype == MOE_F16    ? product_kernel<MOE_F16>(sw)
                               : y_dtype == MOE_BF16 ? product_kernel<MOE_BF16>(sw)
                                                     : product_kernel<MOE_MXFP4>(sw);
  const size_t smem = product_smem(E);
  int per_sm = 0;
  if (resident_blocks((const void*)kernel, kProductThreads, smem, &per_sm) != cudaSuccess || per_sm < 1)
    return MOE_ERR_CUDA;
  // a unit is at least 64 weight rows of an expert's tile: no more CTAs than that
  const long long most = ((long long)W * A / kRowsTile + E) * ((n + 63) / 64);
  PdlLaunch L(dim3((unsigned)(most < nsm ? most : nsm)), dim3(kProductThreads), smem, static_cast<cudaStream_t>(stream));
  if (cudaLaunchKernelEx(&L.cfg, kernel, mx, mw, p) != cudaSuccess) return MOE_ERR_CUDA;
  note_launches(1);
  return MOE_OK;
}

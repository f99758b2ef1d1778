// The experts' product on dispatched MX FP4 rows (moe_expert_product;
// include/moe_experts.h): z[r][j] = sum_i x[r][i] * w[e(r)][j][i] over the rows
// that ep_recv_count gives to each expert, then the epilogue.
//
// On the tensor cores' block-scaled path (tcgen05.mma kind::mxf4: E2M1 codes, one
// E8M0 scale for 32 elements of K, fp32 accumulators in TMEM):
//   * a unit is 128 rows of one expert (the MMA's A operand) against up to 192
//     of its weight rows (B). The rows are A although an expert may have only a
//     few: streaming weights from HBM takes 23 bytes a clock and SM, the MMA eats
//     64 of them a clock, so the unused rows cost nothing that is short, and
//     each epilogue thread has one row with neighbouring features in registers;
//   * codes come by TMA in 128-byte-swizzled boxes, 256 elements of K a stage, as
//     many boxes of 32 rows of A as the unit has rows for; where every expert has
//     few rows the stages are that much smaller and more;
//   * the weights' scales, laid out in the tensor cores' order (MOE_SF_TILED), come
//     in boxes of 2 x 1 KB for 256 rows (untiled bulk copies of 1 KB kept the copy
//     engine busy for longer than the codes did); the rows' scales lie a row
//     after the other as dispatch wrote them: a lane loads 8 bytes of its rows
//     (r, r + 32, ..) and stores them in that order; the same warp's
//     tcgen05.cp takes both to TMEM, and its commit arrives on the barrier of the
//     stage's codes, so that the MMA warp is left with one wait, four MMAs and one
//     commit a stage (what it has to issue bounds a stage);
//   * warps: 0 TMA, 1 MMA, 2..5 scales, 6..13 epilogue (four for each of the two
//     accumulators). Two accumulators of 192 columns and the scales fill
//     TMEM, so that the next unit's MMAs run while this one is read (256 columns
//     would leave room for one: the hand-over then stood still for each unit);
//   * one persistent CTA an SM; units are dealt out round-robin over all experts
//     (their running tile counts are scanned in shared memory), n-tiles of one
//     row tile adjacent, so that rows and weights are read from L2 but once from HBM.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <mutex>

#include "../../include/moe_experts.h"
#include "experts_host.h"
#include "quant_common.cuh"
#include "tcgen05.cuh"

namespace crs {

struct ProductParams {
  const uint8_t* xs;       // [W*A][K/32]
  const int32_t* ep;       // [W][L*W]
  void* y;                 // [W*A][C]
  uint8_t* ys;             // [W*A][ceil(C/32)], MX FP4 output
  int W, L, E, N, K, C;    // C output columns
  int xs_align;            // bytes that a copy of row scales may take: 8, 4 or 1
  long long A;
  long long most_tiles;    // of 128 rows, with counts that dispatch can write
  int* status;
  uint64_t timeout_ns;
};

// Boxes of 32 rows of x, of 64 rows of w and of the scales of 2 x 128 rows of w. (A stage's
// rows in one box each, with a map for every size, took the same time.)
struct ProductMaps {
  CUtensorMap x, w, wsf;
};

constexpr int kProductThreads = 448;
constexpr int kMaxStages = 8;
constexpr int kEpilogueWarp = 6;             // first of the eight
constexpr int kRowsTile = 128;               // MMA M
constexpr int kRowsBox = 32;
constexpr int kMaxBoxes = 3;                 // of 64 weight rows: MMA N <= 192
constexpr int kKStage = 256;                 // elements of K a stage: 128 bytes a row
constexpr uint32_t kSfbBytes = 2 * 1024;     // 2 x 128 rows x 8 scales
// Four warps bring the scales to the tensor cores, each those of every fourth place
// of the stage ring (a place's barriers have one and the same waiter, which cannot
// be a round ahead). They have rings of their own, so that a stage's scales are in
// TMEM when its codes arrive: with them in the stages, a stage's way from its release
// through copy, tcgen05.cp and their barriers back to the MMA took 2600 clocks, a
// third of which were the scales'. One stage ahead of the present one is under way: the
// weights' scales in a slot, the rows' in registers.
constexpr int kScaleWarps = 4, kScaleSlots = 2;
constexpr uint32_t kScaleStage = 128 * 8;
// An epilogue warp turns 32 rows x 64 bytes around in shared memory before it
// stores them (rows 80 bytes apart: no bank is hit twice): stored a row a lane, every
// store touched 32 lines, and the epilogue was what the scale warps waited for.
constexpr uint32_t kTurnRow = 80, kTurnWarp = 32 * kTurnRow;
constexpr size_t kProductSmem = 227 * 1024 - 1024;  // dynamic; the barriers and 1 KB of alignment aside

// Shared memory behind the stages: row scales in order, scales under way (copies want
// them on 128 bytes), the epilogue warps' turning places, running row tiles [E+1],
// first flat row [E], row count [E].
__host__ __device__ constexpr uint32_t product_fixed_smem(int E) {
  return (uint32_t)kScaleWarps * (kScaleStage + kScaleSlots * kSfbBytes) + 8 * kTurnWarp + ((3u * E + 1) * 4 + 127) / 128 * 128;
}

static_assert(kProductSmem % 128 == 0 && kScaleStage % 128 == 0 && kTurnWarp % 128 == 0, "copies' places");
static_assert((kProductSmem - 1024 - product_fixed_smem(1024)) / ((kRowsTile + kMaxBoxes * 64) * 128) >= kScaleWarps,
              "every scale warp has a place in the smallest ring");

// How a launch cuts its work: weight rows a unit, rows of A kept for a stage, and
// as many stages as shared memory holds.
struct ProductShape {
  int width, n_tiles, stages;
  uint32_t a_bytes, stage_bytes, sf_cols;
};

__device__ __forceinline__ ProductShape product_shape(int N, int E, int m_tiles, int most_rows) {
  int boxes = 1;
  uint32_t best = 0xffffffffu;
  // The width whose rounds of units cost least: where experts have a row tile or two,
  // a unit streams its weights from HBM (its cost is their bytes); where they have
  // many, its rows and weights come from L2 and a wider unit saves rows. Measured
  // with 64 / 128 / 192 weight rows: 8 rows of 8 experts 5.9 / 6.2 / 6.9 us, 32 rows an
  // expert 30.9 / 27.6 / 28.7 us, 128 rows (k 7168) 239 / 182 / 188 us, 1024 rows 224 /
  // 137 / 124 us (short runs; at the power limit the last takes 137 us). Between one tile an expert and eight
  // nothing was measured, nor batches whose rows are with a few of the experts.
  const bool streams = m_tiles < 3 * E;
  for (int b = kMaxBoxes; b >= 1; --b) {
    const uint32_t units = (uint32_t)m_tiles * (uint32_t)((N + 64 * b - 1) / (64 * b));
    const uint32_t cost = (units + gridDim.x - 1) / gridDim.x * (uint32_t)(streams ? 4 * b + 1 : b + 2);
    if (cost < best) {
      best = cost;
      boxes = b;
    }
  }
  ProductShape s;
  s.width = boxes * 64;
  s.n_tiles = (N + s.width - 1) / s.width;
  s.a_bytes = (uint32_t)min(kRowsTile, (most_rows + kRowsBox - 1) / kRowsBox * kRowsBox) * 128;
  s.stage_bytes = s.a_bytes + s.width * 128;
  s.stages = min(kMaxStages, (int)(((uint32_t)kProductSmem - 1024 - product_fixed_smem(E)) / s.stage_bytes));
  // TMEM: two accumulators, then 2 x 4 columns of the rows' scales and 2 x 4 for
  // every 128 weight rows of a stage
  s.sf_cols = 8 + (boxes == 3 ? 16 : 8);
  s.stages = min(s.stages, (512 - 2 * s.width) / (int)s.sf_cols);
  return s;
}

struct ProductUnit {
  int e, n0, rows;
  long long row0;
};

// A CTA's units in turn: row tile mt and n-tile ni of unit u, u + gridDim.x, ..
struct ProductCursor {
  int u, mt, ni, m_step, n_step, n_tiles;
  __device__ ProductCursor(int n_tiles_) : u(blockIdx.x), n_tiles(n_tiles_) {
    mt = u / n_tiles;
    ni = u - mt * n_tiles;
    m_step = (int)gridDim.x / n_tiles;
    n_step = (int)gridDim.x - m_step * n_tiles;
  }
  __device__ void next() {
    u += gridDim.x;
    mt += m_step;
    ni += n_step;
    if (ni >= n_tiles) {
      ni -= n_tiles;
      ++mt;
    }
  }
};

// Its expert and rows, found by a whole warp: the expert whose tiles [pre[e],
// pre[e+1]) hold mt, first among every (E/32)th expert, then among those between.
__device__ __forceinline__ ProductUnit product_unit(const ProductParams& p, const int* pre, const ProductCursor& at, int width) {
  const int lane = threadIdx.x & 31, step = (p.E + 31) >> 5;
  const int far = lane * step;
  const int block = (31 - __clz(__ballot_sync(0xffffffffu, far < p.E && pre[far] <= at.mt))) * step;
  const int near = block + lane;
  const int e = block + 31 - __clz(__ballot_sync(0xffffffffu, lane < step && near < p.E && pre[near] <= at.mt));
  const int* first = pre + p.E + 1;
  const int* count = first + p.E;
  const int before = (at.mt - pre[e]) * kRowsTile;
  ProductUnit x;
  x.e = e;
  x.n0 = at.ni * width;
  x.rows = min(kRowsTile, count[e] - before);
  x.row0 = first[e] + before;
  return x;
}

struct ProductAbort {
  volatile int* flag;
  int* status;
  uint64_t limit;
};

// A wait of the pipeline, bounded by `limit` once it has lasted a while: reading
// the global timer at every wait that has to wait at all cost more than the wait.
__device__ __forceinline__ bool product_wait(uint32_t bar, uint32_t parity, const ProductAbort& a) {
#pragma unroll 1
  for (int it = 0; it < 64; ++it)
    if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
#pragma unroll 1
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

// The same for a whole warp: one lane asks, so that waiting warps leave the
// shared-memory pipe to those at work.
__device__ __forceinline__ bool product_wait_warp(uint32_t bar, uint32_t parity, const ProductAbort& a) {
  bool ok = true;
  if ((threadIdx.x & 31) == 0) ok = product_wait(bar, parity, a);
  return __all_sync(0xffffffffu, ok);
}

// The same where all lanes ask, for the warps that others wait for: nothing of it diverges
// when the phase is there at once.
__device__ __forceinline__ bool product_wait_all(uint32_t bar, uint32_t parity, const ProductAbort& a) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, product_wait(bar, parity, a));
}

// The 8 scale bytes of rows lane, lane + 32, .. of a unit for stage kb, by the widest loads
// that the row length (K / 32 bytes) and x_scales' address align; zeros beyond the
// row's end and the unit's rows.
__device__ __forceinline__ void load_row_scales(const ProductParams& p, const ProductUnit& un, int kb, uint2 (&v)[4]) {
  const int lane = threadIdx.x & 31, blocks = p.K / 32, left = min(8, blocks - kb * 8);
  const uint8_t* src = p.xs + (size_t)(un.row0 + lane) * blocks + kb * 8;
  const size_t step = (size_t)32 * blocks;
#pragma unroll
  for (int c = 0; c < 4; ++c) v[c] = make_uint2(0, 0);
  if (p.xs_align == 8) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (lane + 32 * c < un.rows) v[c] = __ldg(reinterpret_cast<const uint2*>(src + c * step));
  } else if (p.xs_align == 4) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (lane + 32 * c < un.rows) {
        v[c].x = __ldg(reinterpret_cast<const uint32_t*>(src + c * step));
        if (left > 4) v[c].y = __ldg(reinterpret_cast<const uint32_t*>(src + c * step) + 1);
      }
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (lane + 32 * c < un.rows)
        for (int b = 0; b < left; ++b) {
          const uint32_t w = (uint32_t)__ldg(src + c * step + b) << (8 * (b & 3));
          if (b < 4) v[c].x |= w;
          else v[c].y |= w;
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

// 32 neighbouring results (columns c ..) of each lane's row, row0 + lane, of which the
// first `rows` lanes' exist; the whole warp takes part. Rows that 16-byte stores fit
// leave as such, others an element (or a byte of codes) a lane, row by row.
template <int YT>
__device__ __forceinline__ void store_results(const ProductParams& p, uint32_t turn, long long row0, int rows, int c,
                                              const float (&v)[32]) {
  const int lane = threadIdx.x & 31;
  if (c >= p.C) return;
  const uint32_t own = turn + lane * kTurnRow;
  if constexpr (YT == MOE_MXFP4) {
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < 32; ++j) m = fmaxf(m, fabsf(v[j]));  // columns beyond C are zeros
    const int se = mx_exponent(m, 2);
    const float inv = exp2_exact(-se);
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      q[i] = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        q[i] |= cvt_fp4x2(__fmul_rn(v[8 * i + 2 * j], inv), __fmul_rn(v[8 * i + 2 * j + 1], inv)) << (8 * j);
    }
    uint8_t* out = static_cast<uint8_t*>(p.y) + (size_t)row0 * (p.C / 2) + c / 2;
    if (lane < rows) p.ys[(size_t)(row0 + lane) * ((p.C + 31) / 32) + c / 32] = (uint8_t)(se + 127);
    if ((p.C & 31) == 0) {
      if (lane < rows) st_v4(out + (size_t)lane * (p.C / 2), make_int4(q[0], q[1], q[2], q[3]));
    } else {
      asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(own), "r"(q[0]), "r"(q[1]), "r"(q[2]), "r"(q[3]) : "memory");
      __syncwarp();
      const int b = lane & 15, last = c / 2 + b < p.C / 2 ? rows : 0;
#pragma unroll 4
      for (int r = lane >> 4; r < last; r += 2) {
        uint32_t w;
        asm volatile("ld.shared.u8 %0, [%1];" : "=r"(w) : "r"(turn + r * kTurnRow + b));
        out[(size_t)r * (p.C / 2) + b] = (uint8_t)w;
      }
      __syncwarp();
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(own + i * 16), "r"(pack_y<YT>(v[8 * i], v[8 * i + 1])),
                   "r"(pack_y<YT>(v[8 * i + 2], v[8 * i + 3])), "r"(pack_y<YT>(v[8 * i + 4], v[8 * i + 5])),
                   "r"(pack_y<YT>(v[8 * i + 6], v[8 * i + 7]))
                   : "memory");
    __syncwarp();
    uint16_t* out = static_cast<uint16_t*>(p.y) + (size_t)row0 * p.C + c;
    if ((p.C & 7) == 0) {
      // 8 rows x 64 bytes a store
      const int part = (lane & 3) * 8, r0 = lane >> 2;
      int4 w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[i].x), "=r"(w[i].y), "=r"(w[i].z), "=r"(w[i].w)
                     : "r"(turn + (8 * i + r0) * kTurnRow + (lane & 3) * 16));
      const int last = c + part < p.C ? rows : 0;
      out += (size_t)r0 * p.C + part;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (8 * i + r0 < last) st_v4(out + (size_t)(8 * i) * p.C, w[i]);
    } else {
      const int last = c + lane < p.C ? rows : 0;
#pragma unroll 4
      for (int r = 0; r < last; ++r) {
        uint16_t w;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(w) : "r"(turn + r * kTurnRow + lane * 2));
        out[(size_t)r * p.C + lane] = w;
      }
    }
    __syncwarp();
  }
}

template <int YT, bool SWIGLU>
__global__ void __launch_bounds__(kProductThreads, 1)
    expert_product_kernel(const __grid_constant__ ProductMaps maps, ProductParams p) {
  extern __shared__ __align__(1024) uint8_t psm_raw[];
  __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], drained;
  __shared__ __align__(8) uint64_t landed[kScaleWarps][kScaleSlots], taken[kScaleWarps];
  __shared__ uint32_t tmem_slot;
  __shared__ long long scan_scratch[32];
  __shared__ volatile int s_abort;

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  uint8_t* sm = psm_raw + ((1024u - (smem_u32(psm_raw) & 1023u)) & 1023u);
  uint8_t* ring = sm + kProductSmem - 1024 - product_fixed_smem(p.E);
  uint8_t* slots = ring + kScaleWarps * kScaleStage;
  uint8_t* turn = slots + kScaleWarps * kScaleSlots * kSfbBytes;
  int* pre = reinterpret_cast<int*>(turn + 8 * kTurnWarp);

  if (threadIdx.x == 0) {
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(&full[i], 2);  // the codes' copies, and the scales' tcgen05.cp
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 4);
    }
    for (int i = 0; i < kScaleWarps * kScaleSlots; ++i) mbar_init(&landed[0][i], 1);
    for (int i = 0; i < kScaleWarps; ++i) mbar_init(&taken[i], 1);
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
  int most_rows = 0;
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
        most_rows = max(most_rows, n);
        first[e] = (int)(e / p.L * p.A) + lo;  // flat rows fit 32 bits
        count[e] = n;
      }
      const long long tiles = (n + kRowsTile - 1) / kRowsTile;
      const long long before = carry + block_exclusive_scan(tiles, scan_scratch);
      if (e < p.E) {
        pre[e] = (int)min(before, 1ll << 30);
        if (e == p.E - 1) pre[p.E] = (int)min(before + tiles, 1ll << 30);
      }
      __syncthreads();
      // the last expert of this pass carries on
      const int last = min(p.E, e0 + kProductThreads) - 1;
      carry = pre[last] + (count[last] + kRowsTile - 1) / kRowsTile;
    }
  }
  most_rows = __reduce_max_sync(0xffffffffu, most_rows);
  if (lane == 0) scan_scratch[warp] = most_rows;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  most_rows = (int)(lane < kProductThreads / 32 ? scan_scratch[lane] : 0);
  most_rows = __reduce_max_sync(0xffffffffu, most_rows);
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_slot, 0);
  // overlapping experts (counts that fall and rise again, reported above) can have more
  // row tiles than the units' numbers hold: then none is worked on
  const int m_tiles = pre[p.E] <= p.most_tiles ? __shfl_sync(0xffffffffu, pre[p.E], 0) : 0, KB = (p.K + kKStage - 1) / kKStage;
  const ProductShape shape = product_shape(p.N, p.E, m_tiles, most_rows);
  const int width = __shfl_sync(0xffffffffu, shape.width, 0), n_tiles = __shfl_sync(0xffffffffu, shape.n_tiles, 0);
  const uint32_t stages = __shfl_sync(0xffffffffu, shape.stages, 0), a_bytes = __shfl_sync(0xffffffffu, shape.a_bytes, 0);
  const uint32_t stage_bytes = __shfl_sync(0xffffffffu, shape.stage_bytes, 0), sf_cols = __shfl_sync(0xffffffffu, shape.sf_cols, 0);
  const uint32_t tmem_sf = tmem + 2 * width, b_step = width > 128 ? 8 : 4;
  const int units = m_tiles * n_tiles;
  const bool whole = p.K % kKStage == 0;
  const uint32_t full0 = smem_u32(full), empty0 = smem_u32(empty);
  const ProductAbort ab{&s_abort, p.status, p.timeout_ns};

  // Every role walks the same units and stages. The copying, scaling and multiplying
  // warps run theirs with all lanes on values that the compiler can see are uniform,
  // one elected lane's instructions predicated: what the MMA warp has to issue bounds a
  // stage. Under a divergent branch every descriptor took the slow way into uniform
  // registers, and coming together again cost 120 clocks.
  if (warp == 0) {
    const uint32_t sm0 = smem_u32(sm);
    const int w_boxes = width >> 6;
    const bool leader = elect_one();
    uint32_t stage = 0, phase = 1;
    bool ok = true;
    for (ProductCursor at(n_tiles); at.u < units && ok; at.next()) {
      const ProductUnit un = product_unit(p, pre, at, width);
      const int rows = __shfl_sync(0xffffffffu, un.rows, 0), e = __shfl_sync(0xffffffffu, un.e, 0),
                row = __shfl_sync(0xffffffffu, (int)un.row0, 0), n0 = at.ni * width;
      const int a_boxes = (rows + kRowsBox - 1) / kRowsBox;
      const uint32_t bytes = (uint32_t)(width + a_boxes * kRowsBox) * 128u;
      for (int kb = 0; kb < KB; ++kb) {
        ok = product_wait_all(empty0 + stage * 8, phase, ab);
        if (!ok) break;
        const uint32_t st = sm0 + stage * stage_bytes, bar = full0 + stage * 8;
        mbar_expect_tx_if(leader, bar, bytes);
#pragma unroll
        for (int b = 0; b < kMaxBoxes; ++b)
          tma_load_3d_if(leader && b < w_boxes, st + a_bytes + b * (64 * 128), &maps.w, kb * 128, n0 + b * 64, e, bar);
#pragma unroll
        for (int b = 0; b < kRowsTile / kRowsBox; ++b)
          tma_load_2d_if(leader && b < a_boxes, st + b * (kRowsBox * 128), &maps.x, kb * 128, row + b * kRowsBox, bar);
        if (++stage == stages) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
  } else if (warp == 1) {
    const uint64_t adesc0 = sw128_desc(sm), bdesc0 = sw128_desc(sm + a_bytes);
    const bool leader = elect_one();
    uint32_t stage = 0, phase = 0, done = 0;
    bool ok = true;
    for (ProductCursor at(n_tiles); at.u < units && ok; at.next(), ++done) {
      const int n0 = at.ni * width, cols = min(width, (p.N - n0 + 63) & ~63);
      const uint32_t shift = (n0 & 127) >> 5;  // columns before the unit's first weight row: 0 or 2
      const uint32_t idesc = idesc_mxf4(cols), buf = done & 1, acc = tmem + buf * width;
      ok = product_wait_all(smem_u32(&acc_empty[buf]), ((done >> 1) & 1) ^ 1, ab);
      for (int kb = 0; kb < KB && ok; ++kb) {
        ok = product_wait_all(full0 + stage * 8, phase, ab);
        if (!ok) break;
        tc_fence_after();
        const uint32_t step = stage * (stage_bytes >> 4), here = stage;
        const uint32_t ta = tmem_sf + stage * sf_cols, tb = ta + 8 + shift;
        if (++stage == stages) {
          stage = 0;
          phase ^= 1;
        }
        const int steps = whole || kb + 1 < KB ? 4 : (p.K - kb * kKStage + 63) / 64;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          constexpr uint32_t kPair = (2u << 4) | (2u << 29);  // the upper two of a column's four scales
          tc_mma_mxf4_if(leader && kk < steps, acc, adesc0 + step + 2 * kk, bdesc0 + step + 2 * kk, idesc | (kk & 1 ? kPair : 0),
                         ta + 4 * (kk >> 1), tb + b_step * (kk >> 1), kk > 0 || kb > 0);
        }
        tc_commit_if(leader, empty0 + here * 8);
        tc_commit_if(leader && kb + 1 == KB, smem_u32(&acc_full[buf]));
      }
    }
    if (leader) tc_commit(&drained);
  } else if (warp < 2 + kScaleWarps) {
    // scales of the stages in this warp's places of the ring
    const uint32_t mine = warp - 2;
    const uint8_t* my_slots = slots + mine * kScaleSlots * kSfbBytes;
    const uint8_t* my_ring = ring + mine * kScaleStage;
    const uint32_t slot0 = smem_u32(my_slots), dst = smem_u32(my_ring) + lane * 16;
    const uint64_t asf = sf_desc(my_ring), bsf0 = sf_desc(my_slots);
    const int nt128 = (p.N + 127) / 128;
    const bool leader = elect_one();
    // from one of its places to the next one's stage; true where that is in the ring's next round
    const auto hop = [&](ProductCursor& at, int& kb, uint32_t& place, bool& moved) {
      const bool around = place + kScaleWarps >= stages;
      kb += around ? (int)(stages - place + mine) : kScaleWarps;
      place = around ? mine : place + kScaleWarps;
      while (kb >= KB) {
        kb -= KB;
        at.next();
        moved = true;
      }
      return around;
    };
    const auto first = [&](ProductCursor& at, int& kb) {
      for (kb = (int)mine; kb >= KB; kb -= KB) at.next();
    };
    ProductCursor load(n_tiles), at(n_tiles);
    int load_kb, kb;
    uint32_t load_slot = 0, load_stage = mine;
    bool fresh = true;
    ProductUnit ahead{};
    uint2 v[4];  // the lane's own rows: word i of row c is 128-element group i
    first(load, load_kb);
    first(at, kb);
    const auto load_next = [&] {
      if (load.u < units) {
        if (fresh) ahead = product_unit(p, pre, load, width);
        fresh = false;
        const uint32_t bar = smem_u32(&landed[mine][load_slot]);
        load_row_scales(p, ahead, load_kb, v);
        mbar_expect_tx_if(leader, bar, kSfbBytes);
        tma_load_2d_if(leader, slot0 + load_slot * kSfbBytes, &maps.wsf, load_kb * 256, ahead.e * nt128 + (ahead.n0 >> 7), bar);
        load_slot ^= 1;
        hop(load, load_kb, load_stage, fresh);
      }
    };
    load_next();
    uint32_t stage = mine, phase = 1, slot = 0, landed_phase = 0, taken_phase = 1;
    for (bool moved; at.u < units; phase ^= hop(at, kb, stage, moved)) {
      // tcgen05.cp has taken the stage before: its slot and the ordered scales are free
      if (!product_wait_all(smem_u32(&taken[mine]), taken_phase, ab)) break;
      taken_phase ^= 1;
      // the 4 bytes of row r and group i at i * 512 + (r % 32) * 16 + (r / 32) * 4
      asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(v[0].x), "r"(v[1].x), "r"(v[2].x), "r"(v[3].x)
                   : "memory");
      asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst + 512), "r"(v[0].y), "r"(v[1].y), "r"(v[2].y), "r"(v[3].y)
                   : "memory");
      fence_proxy_async_smem();
      __syncwarp();
      load_next();
      // the weights' scales are there, and the MMAs of the round before are done with the TMEM columns
      if (!product_wait_all(smem_u32(&landed[mine][slot]), landed_phase, ab)) break;
      if (!product_wait_all(empty0 + stage * 8, phase, ab)) break;
      tc_fence_after();
      const int n0 = at.ni * width;
      const bool two = (n0 & 127) + min(width, (p.N - n0 + 63) & ~63) > 128;
      const bool more = p.K - kb * kKStage > 128;  // than one 128-element group
      const uint32_t ta = tmem_sf + stage * sf_cols;
      const uint64_t bsf = bsf0 + slot * (kSfbBytes >> 4);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const bool go = leader && (j == 0 || more);
        tc_cp_scales_if(go, ta + 4 * j, asf + j * 32);
        tc_cp_scales_if(go, ta + 8 + b_step * j, bsf + j * 32);
        tc_cp_scales_if(go && two, ta + 8 + b_step * j + 4, bsf + 64 + j * 32);
      }
      tc_commit_if(leader, full0 + stage * 8);
      tc_commit_if(leader, smem_u32(&taken[mine]));
      slot ^= 1;
      landed_phase ^= slot == 0;
    }
    // the last stage's arrival: the MMAs' end, which the kernel waits for, does not say that it has come
    product_wait_all(smem_u32(&taken[mine]), taken_phase, ab);
  } else if (warp >= kEpilogueWarp) {
    // quarter q: rows 32 q ..; four warps take the even units, four the odd ones (an
    // accumulator each): what a unit costs a warp besides its columns, some 650
    // clocks, then falls to it every other unit
    const int q = warp & 3;
    const uint32_t buf = (warp - kEpilogueWarp) >> 2;
    const uint32_t acc = tmem + ((uint32_t)(32 * q) << 16) + buf * width;
    const uint32_t my_turn = smem_u32(turn) + (warp - kEpilogueWarp) * kTurnWarp;
    uint32_t done = 0;
    // ended by an abort at the wait alone, which answers for the whole warp: lanes that read the flag by themselves
    // could part before the next ballot
    for (ProductCursor at(n_tiles); at.u < units; at.next(), ++done) {
      if ((done & 1) != buf) continue;
      const ProductUnit un = product_unit(p, pre, at, width);
      if (!product_wait_warp(smem_u32(&acc_full[buf]), (done >> 1) & 1, ab)) break;
      tc_fence_after();
      const int rows = min(32, un.rows - 32 * q), parts = rows > 0 ? (min(width, p.N - un.n0) + 63) / 64 : 0;
#pragma unroll 1
      for (int g = 0; g < parts; ++g) {  // 64 columns
        const int n = un.n0 + g * 64;
        uint32_t v[64];
        tc_ld64(acc + g * 64, v);
        tc_wait_ld();
        if (g + 1 == parts) {
          // the last part is in registers: the accumulator goes back before it is stored
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&acc_empty[buf]);
        }
        float h[32];
        if (SWIGLU) {
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const float a = __uint_as_float(v[2 * j]), b = __uint_as_float(v[2 * j + 1]);
            // both within a few ulps (exp: plus |a| / 2^23 of its value), far below the rounding to 16 or 4
            // bits that follows; the divisor stays within [1, 2], where the fast reciprocal holds (as a / (1 + exp(-a)),
            // gates below -87 came out as 0, whatever they were to be multiplied by)
            const float t = __expf(-fabsf(a));
            float r;
            asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + t));
            h[j] = (a < 0.f ? a * t : a) * r * b;
          }
          store_results<YT>(p, my_turn, un.row0 + 32 * q, rows, n / 2, h);
        } else {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int j = 0; j < 32; ++j) h[j] = __uint_as_float(v[32 * i + j]);
            store_results<YT>(p, my_turn, un.row0 + 32 * q, rows, n + 32 * i, h);
          }
        }
      }
      if (parts == 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[buf]);
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

// Rows of scale tiles (512 bytes for every 128 elements of K), boxes of 1 KB x 2 rows.
static bool scale_map(CUtensorMap* m, const void* base, unsigned long long bytes, unsigned long long rows) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = product_encode_fn();
  if (!enc) return false;
  cuuint64_t dims[2] = {bytes / 4, rows};
  cuuint64_t strides[1] = {bytes};
  cuuint32_t box[2] = {256, 2};
  cuuint32_t es[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

typedef void (*ProductKernel)(ProductMaps, ProductParams);
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
  if (n < 1 || k < 1 || k > (1 << 30) || epilogue < MOE_EPI_NONE || epilogue > MOE_EPI_SWIGLU) return MOE_ERR_INVALID_ARG;
  if (k % 32) return MOE_ERR_UNSUPPORTED;
  const int E = cfg->moe_expert_num, W = cfg->ep_world_size;
  if (epilogue == MOE_EPI_SWIGLU && n % 2) return MOE_ERR_INVALID_ARG;
  const int C = epilogue == MOE_EPI_SWIGLU ? n / 2 : n;
  if (y_dtype != MOE_F16 && y_dtype != MOE_BF16 && y_dtype != MOE_MXFP4) return MOE_ERR_INVALID_ARG;
  if (y_dtype == MOE_MXFP4 ? C % 2 != 0 || !y_scales : y_scales != nullptr) return MOE_ERR_INVALID_ARG;
  // units of 128 rows x 64 weight rows are counted in 32 bits, and a CTA looks some of its units ahead
  const long long most_tiles = (long long)W * A / kRowsTile + E, most_units = most_tiles * ((n + 63LL) / 64);
  if ((long long)E * n >= 2147483647LL || most_units >= 2147483647LL - 65536) return MOE_ERR_INVALID_ARG;
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

  ProductMaps maps;
  const unsigned long long row_bytes = (unsigned long long)k / 2, rows = (unsigned long long)W * A;
  if (!product_map(&maps.x, x, row_bytes, rows, 0, kRowsBox) ||
      !scale_map(&maps.wsf, w_scales, (unsigned long long)(k + 127) / 128 * 512, (unsigned long long)E * ((n + 127) / 128)) ||
      !product_map(&maps.w, w, row_bytes, (unsigned long long)n, (unsigned long long)E, 64))
    return MOE_ERR_CUDA;
  ProductParams p{};
  p.xs = x_scales;
  p.ep = ep_recv_count;
  p.y = y;
  p.ys = y_scales;
  p.W = W;
  p.L = E / W;
  p.E = E;
  p.N = n;
  p.K = k;
  p.C = C;
  p.xs_align = k % 256 == 0 && aligned(x_scales, 8) ? 8 : k % 128 == 0 ? 4 : 1;
  p.A = A;
  p.most_tiles = most_tiles;
  p.status = &static_cast<WsHeader*>(ws)->status;
  p.timeout_ns = (uint64_t)cfg->wait_timeout_us * 1000ull;
  const bool sw = epilogue == MOE_EPI_SWIGLU;
  const ProductKernel kernel = y_dtype == MOE_F16    ? product_kernel<MOE_F16>(sw)
                               : y_dtype == MOE_BF16 ? product_kernel<MOE_BF16>(sw)
                                                     : product_kernel<MOE_MXFP4>(sw);
  const size_t smem = kProductSmem;
  int per_sm = 0;
  if (resident_blocks((const void*)kernel, kProductThreads, smem, &per_sm) != cudaSuccess || per_sm < 1)
    return MOE_ERR_CUDA;
  // a unit is at least 64 weight rows of an expert's tile: no more CTAs than that
  PdlLaunch L(dim3((unsigned)(most_units < nsm ? most_units : nsm)), dim3(kProductThreads), smem, static_cast<cudaStream_t>(stream));
  if (cudaLaunchKernelEx(&L.cfg, kernel, maps, p) != cudaSuccess) return MOE_ERR_CUDA;
  note_launches(1);
  return MOE_OK;
}

// The experts' product on dispatched int8 rows (moe_expert_product_int8;
// include/moe_experts.h): z[r][j] = xs[r] * ws[e(r)][j] * sum_i x[r][i] * w[e(r)][j][i] over
// the rows that ep_recv_count gives to each expert, then the epilogue.
//
// sm_103a's integer tensor rate is a small part of its fp16 rate, and fp16 holds every
// int8 exactly, products below 2^14 and sums to 2^24 in fp32 too: the codes are
// widened to fp16 on the way from shared memory to the tensor cores.
//   * two CTAs share a unit (cta_group::2): 256 weight rows of an expert, 128 each (the MMA's A
//     operand), against up to 192 of its rows (B, half of them widened in each). Weights are A
//     because A may come from TMEM: a weight goes TMA -> shared memory -> registers -> TMEM, 2
//     bytes of shared-memory traffic for each; a row's element, written back as fp16 and
//     read by the MMA, takes 6. Shared memory's 128 bytes a clock bound a unit of many rows: in one CTA
//     128 x 192 took 235 bytes for each clock of the MMA, in a pair 139;
//   * four bytes become two fp16 pairs, bytes 0 and 2 and bytes 1 and 3 (widen4). The order of K
//     that this gives is the same for both operands;
//   * copies bring 128 elements of K a stage; four sets of four warps widen them in turn, a stage
//     each, into a slot of TMEM and shared memory that each has. Two accumulators of more than
//     128 columns leave TMEM for half as much: then a slot is half a stage, and so is a set's turn;
//   * warps: 0 TMA, 1 MMA (of the pair's first CTA), 2..17 widen, 18..21 epilogue. Two accumulators, so
//     that the next unit's MMAs run while this one is read.
//
// Measured: 4096 rows of 128 experts, 2048 -> 1024 with SwiGLU, 50 us, 5.6 TB/s; 512 -> 2048, 35 us;
// 32768 rows of 256 experts, 7168 -> 1024, 458 us, 4.7 TB/s and 1.05 PFLOP/s; 131072 rows of 128 experts, 2048
// -> 1024, 390 us, 1.4 PFLOP/s; 8 rows 10.2 us. Few rows are bound by HBM, and by some 5 us before
// the first product and behind the last (a unit's copies, widening, MMAs and epilogue end to end). Many
// are bound by the widening and the way of a slot through it: without widening prefill takes 273 us of 387,
// without x 318, without weights 313, without the epilogue 356.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <mutex>

#include "../../include/moe_experts.h"
#include "experts_host.h"
#include "quant_common.cuh"
#include "tcgen05_pair.cuh"

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
  uint64_t timeout_ns;
  uint8_t raw_stages[6];  // of the copies' ring, for row tiles of 32, 64, ..
};

// SwiGLU of a gate and what it gates. exp and the reciprocal are the fast ones, within a few ulps (exp: plus
// |gate| / 2^23 of its value), far below the rounding to 16 bits that follows; a gate below -87, whose exponential is
// beyond the reciprocal's range, gives 0.
__device__ __forceinline__ float int8_swiglu(float gate, float up) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + __expf(-gate)));
  return gate * r * up;
}

// A barrier of the block's first THREADS threads.
template <int THREADS>
__device__ __forceinline__ void int8_barrier() {
  asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory");
}

// The experts' rows: first flat row [E] and row count [E] behind the tiles pre[E + 1]. Thread t has experts per * t, ..;
// its largest count is returned; no barrier.
template <int THREADS>
__device__ __forceinline__ int int8_expert_rows(const Int8ProductParams& p, int* pre) {
  int* first = pre + p.E + 1;
  int* count = first + p.E;
  const int per = (p.E + THREADS - 1) / THREADS;
  int e = per * (int)threadIdx.x, d = e / p.L, le = e - d * p.L;
  int most = 0;
  for (int i = 0; i < per && e < p.E; ++i, ++e) {
    const int32_t* ep = p.ep + (size_t)d * p.L * p.W;
    const int hi = ep[le * p.W + p.W - 1], lo = le ? ep[le * p.W - 1] : 0;
    const bool good = lo >= 0 && hi >= lo && hi <= p.A;
    if (!good && blockIdx.x == 0) set_error(p.status, MOE_ERR_BAD_ASSIST);
    first[e] = (int)(d * p.A) + (good ? lo : 0);  // flat rows fit 32 bits
    count[e] = good ? hi - lo : 0;
    most = max(most, count[e]);
    if (++le == p.L) {
      le = 0;
      ++d;
    }
  }
  return most;
}

// Running tiles of `tile` rows, pre[E + 1], of counts that the same threads have written; false
// (for every thread) where counts overlap to more tiles than dispatch's can make. The block's first THREADS threads take
// part; ends with their barrier. s_warp: a word for each warp, and one that is 0.
template <int THREADS>
__device__ __forceinline__ bool int8_row_tiles(const Int8ProductParams& p, int tile, int* pre, uint32_t* s_warp) {
  constexpr int kWarps = THREADS / 32;
  const int* count = pre + 2 * p.E + 1;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, per = (p.E + THREADS - 1) / THREADS;
  const int e0 = per * (int)threadIdx.x, e1 = min(p.E, e0 + per);
  const auto running = [lane](uint32_t sum) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t below = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += below;
    }
    return sum;
  };
  uint32_t mine = 0;
  for (int e = e0; e < e1; ++e) {
    const uint32_t t = (uint32_t)(count[e] + tile - 1) / (uint32_t)tile;
    mine += t;
    if (t >> 16) s_warp[kWarps] = 1;
  }
  const uint32_t sum = running(mine);
  if (lane == 31) s_warp[warp] = sum;
  int8_barrier<THREADS>();
  const uint32_t below = running(lane < kWarps ? s_warp[lane] : 0);
  const uint32_t total = __shfl_sync(0xffffffffu, below, 31), before = __shfl_sync(0xffffffffu, below, (warp + 31) & 31);
  uint32_t at = (warp ? before : 0) + sum - mine;
  long long whole = total;
  if (s_warp[kWarps]) {  // an expert of millions of rows: the sums may have wrapped
    whole = 0;
    for (int e = 0; e < p.E; ++e) whole += (count[e] + tile - 1) / tile;
  }
  for (int e = e0; e < e1; ++e) {
    pre[e] = (int)at;
    at += (uint32_t)(count[e] + tile - 1) / (uint32_t)tile;
  }
  if (threadIdx.x == 0) pre[p.E] = (int)total;
  int8_barrier<THREADS>();
  return whole <= (long long)p.W * p.A / tile + p.E;
}

// The expert whose tiles hold mt: the last one whose tiles begin at or before it.
__device__ __forceinline__ int int8_expert_of(const int* pre, int E, int mt) {
  int e = 0;
  for (int half = 512; half; half >>= 1)
    if (e + half < E && pre[e + half] <= mt) e += half;
  return e;
}

template <int YT>
__device__ __forceinline__ uint16_t int8_round(float v) {
  return YT == MOE_F16 ? __half_as_ushort(__float2half_rn(v)) : __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// ------------------------------------------------------------- the tensor cores

// Boxes of 16, 32, .. rows of x and of 128 rows of w, 128 elements of K: one copy of each a stage.
struct Int8Maps {
  CUtensorMap x[6], w;
};

constexpr int kWidenWarp = 2, kSets = 4, kSetWarps = 4;
constexpr int kInt8ProductThreads = 22 * 32, kInt8PlanThreads = 8 * 32;
constexpr int kInt8Stage = 128;    // elements of K a stage
constexpr int kInt8Half = 128, kInt8Width = 2 * kInt8Half;  // weight rows of a unit in each CTA, and in both
constexpr int kInt8MostRows = 192; // MMA N
constexpr int kInt8RawStages = 8;  // at most
// An epilogue warp turns 32 rows x 32 results of 2 bytes around in shared memory, rows 80 bytes apart.
constexpr uint32_t kInt8TurnRow = 80, kInt8TurnWarp = 32 * kInt8TurnRow;
constexpr size_t kInt8ProductSmem = 227 * 1024 - 1024;  // dynamic; the barriers and 1 KB of alignment aside

// Behind the ring: the epilogue warps' turning places and row scales, the experts' tiles.
__host__ __device__ constexpr uint32_t int8_fixed_smem(int E) {
  return 4 * (kInt8TurnWarp + kInt8MostRows * 4) + ((3u * E + 1) * 4 + 127) / 128 * 128;
}
// Halves of a stage in a set's slot, 32 columns of TMEM each, beside two accumulators of `tile` columns. (With half a
// stage a slot everywhere 4096 rows of 128 experts, 2048 -> 1024, took 56.7 us where whole stages take 50.4: twice the
// hand-overs. Six slots where TMEM holds them were no faster than four.)
__host__ __device__ constexpr int int8_halves(int tile) { return tile > 128 ? 1 : 2; }
static_assert(2 * 192 + kSets * 32 * int8_halves(192) <= 512 && 2 * 128 + kSets * 32 * int8_halves(128) <= 512, "TMEM");
static_assert(kInt8MostRows == 192, "six boxes of x");

struct Int8Wait {
  volatile int* flag;
  int* status;
  uint64_t limit;
};

// A barrier's phase, asleep until it comes or some microseconds have passed. (Without the hint the waiting warps' asking
// took two thirds of the issue slots.)
__device__ __forceinline__ bool int8_sleep(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(20000u)
      : "memory");
  return ok != 0;
}
// A wait of the pipeline, bounded by `limit` once it has lasted a while.
static __device__ __noinline__ bool int8_wait_long(uint32_t bar, uint32_t parity, volatile int* flag, int* status, uint64_t limit) {
  const uint64_t t0 = globaltimer_ns();
#pragma unroll 1
  for (;;) {
    if (int8_sleep(bar, parity)) return true;
    if (*flag) return false;
    if (globaltimer_ns() - t0 > limit) {
      set_error(status, MOE_ERR_TIMEOUT);
      *flag = 1;
      return false;
    }
  }
}
__device__ __forceinline__ bool int8_wait_one(uint32_t bar, uint32_t parity, const Int8Wait& a) {
  return int8_sleep(bar, parity) || int8_wait_long(bar, parity, a.flag, a.status, a.limit);
}
// All lanes of a warp ask, with one answer for all: nothing of it diverges when the phase is there. (One lane asking for
// the others cost 330 clocks for a phase that was there.)
__device__ __forceinline__ bool int8_wait(uint32_t bar, uint32_t parity, const Int8Wait& a) {
  if (__all_sync(0xffffffffu, int8_sleep(bar, parity))) return true;
  return __all_sync(0xffffffffu, int8_wait_long(bar, parity, a.flag, a.status, a.limit));
}

// Two barriers' phases at once.
__device__ __forceinline__ bool int8_wait2(uint32_t bar0, uint32_t parity0, uint32_t bar1, uint32_t parity1, const Int8Wait& a) {
  const bool one = int8_sleep(bar0, parity0), two = int8_sleep(bar1, parity1);
  if (__all_sync(0xffffffffu, one && two)) return true;
  return int8_wait(bar0, parity0, a) && int8_wait(bar1, parity1, a);
}

__device__ __forceinline__ void mbar_arrive_at(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ int4 lds_v4(uint32_t at) {
  int4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}

// Four int8 as two fp16 pairs, elements (0, 2) and (1, 3), exactly: 128 added to each, the bytes taken for the mantissas
// of 1024 + .., and 1152 subtracted. (By masks and a shift instead of byte permutes it took half as long again.)
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& even, uint32_t& odd) {
  const uint32_t biased = w ^ 0x80808080u;
  const uint32_t a = __byte_perm(biased, 0x64646464u, 0x4240), b = __byte_perm(biased, 0x64646464u, 0x4341);
  const __half2 less = __half2half2(__ushort_as_half(0xe480));  // -1152
  const __half2 x = __hadd2(*reinterpret_cast<const __half2*>(&a), less), y = __hadd2(*reinterpret_cast<const __half2*>(&b), less);
  even = *reinterpret_cast<const uint32_t*>(&x);
  odd = *reinterpret_cast<const uint32_t*>(&y);
}
__device__ __forceinline__ void widen16(int4 v, uint32_t* o) {
  widen4((uint32_t)v.x, o[0], o[1]);
  widen4((uint32_t)v.y, o[2], o[3]);
  widen4((uint32_t)v.z, o[4], o[5]);
  widen4((uint32_t)v.w, o[6], o[7]);
}

struct Int8Unit {
  int e, n0, rows, row0;
};

// A pair's units in turn: row tile mt and n-tile ni of unit u, u + pairs, ..
struct Int8Cursor {
  int u, mt, ni, m_step, n_step, n_tiles;
  __device__ Int8Cursor(int n_tiles_) : u(blockIdx.x >> 1), n_tiles(n_tiles_) {
    const int pairs = gridDim.x >> 1;
    const float one = 1.0f / (float)n_tiles;  // of numbers below 2^16, halves away from a whole quotient
    mt = (int)(((float)u + 0.5f) * one);
    ni = u - mt * n_tiles;
    m_step = (int)(((float)pairs + 0.5f) * one);
    n_step = pairs - m_step * n_tiles;
  }
  __device__ void next() {
    u += gridDim.x >> 1;
    mt += m_step;
    ni += n_step;
    if (ni >= n_tiles) {
      ni -= n_tiles;
      ++mt;
    }
  }
};

// Its expert and rows.
__device__ __forceinline__ Int8Unit int8_unit(const Int8ProductParams& p, const int* pre, const Int8Cursor& at, int tile) {
  // found by a whole warp: among every (E/32)th expert, then among those between
  const int lane = threadIdx.x & 31, step = (p.E + 31) >> 5;
  const int far = lane * step;
  const int block = (31 - __clz(__ballot_sync(0xffffffffu, far < p.E && pre[far] <= at.mt))) * step;
  const int near = block + lane;
  const int e = block + 31 - __clz(__ballot_sync(0xffffffffu, lane < step && near < p.E && pre[near] <= at.mt));
  const int* first = pre + p.E + 1;
  const int* count = first + p.E;
  const int before = (at.mt - pre[e]) * tile;
  return {e, at.ni * kInt8Width, min(tile, count[e] - before), first[e] + before};
}

// Stages of the copies' ring, as many as shared memory holds beside the sets' slots.
static uint8_t int8_raw_stages(int E, int tile) {
  const uint32_t room = (uint32_t)kInt8ProductSmem - 1024 - int8_fixed_smem(E) - kSets * int8_halves(tile) * tile * 64;
  const uint32_t stages = room / ((uint32_t)(kInt8Width + tile) * 64);
  return (uint8_t)(stages < kInt8RawStages ? stages : kInt8RawStages);
}
static_assert((kInt8ProductSmem - 1024 - int8_fixed_smem(1024) - kSets * int8_halves(kInt8MostRows) * kInt8MostRows * 64) /
                      ((kInt8Width + kInt8MostRows) * 64) >= 4, "four stages at least");

// 32 neighbouring columns (rows c0 .. of the tile) of the accumulator by 32 weight rows (a lane each): scaled,
// through the epilogue, turned around and stored. xs: where the rows' scales lie.
template <int YT, bool SWIGLU>
__device__ __forceinline__ void int8_store(const Int8ProductParams& p, uint32_t turn, const uint32_t (&v)[32], float wscale,
                                           uint32_t xs, int row0, int rows, int col) {
  const int lane = threadIdx.x & 31;
  // 16 columns at a time, their scales loaded first and their results stored last: in between nothing orders the
  // columns, whose chains of some 200 clocks overlap
#pragma unroll
  for (int c0 = 0; c0 < 32; c0 += 16) {
    f32x2 s[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int4 w = lds_v4(xs + (c0 + 4 * i) * 4);
      s[2 * i] = f2_pack(__int_as_float(w.x), __int_as_float(w.y));
      s[2 * i + 1] = f2_pack(__int_as_float(w.z), __int_as_float(w.w));
    }
    float x[16];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      f2_split(f2_mul(f2_mul(f2_pack(__uint_as_float(v[c0 + 2 * i]), __uint_as_float(v[c0 + 2 * i + 1])), s[i]),
                      f2_pack(wscale, wscale)), x[2 * i], x[2 * i + 1]);
    if (SWIGLU) {
      // gates lie in the even lanes, what they gate in the odd ones: of two columns the even lane takes the first, the
      // odd one the second
      uint16_t h[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float got = __shfl_xor_sync(0xffffffffu, lane & 1 ? x[2 * i] : x[2 * i + 1], 1);
        h[i] = int8_round<YT>(int8_swiglu(lane & 1 ? got : x[2 * i], lane & 1 ? x[2 * i + 1] : got));
      }
      const uint32_t to = turn + (c0 + (lane & 1)) * kInt8TurnRow + (lane >> 1) * 2;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        asm volatile("st.shared.u16 [%0], %1;" ::"r"(to + 2 * i * kInt8TurnRow), "h"(h[i]) : "memory");
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        asm volatile("st.shared.u16 [%0], %1;" ::"r"(turn + (c0 + i) * kInt8TurnRow + lane * 2), "h"(int8_round<YT>(x[i])) : "memory");
    }
  }
  __syncwarp();
  constexpr int kCols = SWIGLU ? 16 : 32;  // results of a row
  uint16_t* out = static_cast<uint16_t*>(p.y) + (size_t)row0 * p.C + col;
  if ((p.C & 7) == 0) {
    constexpr int kParts = kCols / 8;  // of 16 bytes
    const int part = lane % kParts, r0 = lane / kParts;
    const int last = col + part * 8 < p.C ? rows : 0;
#pragma unroll
    for (int r = r0; r < 32; r += 32 / kParts) {
      const int4 w = lds_v4(turn + r * kInt8TurnRow + part * 16);
      if (r < last) st_v4(out + (size_t)r * p.C + part * 8, w);
    }
  } else {
    const int c = lane % kCols, last = col + c < p.C ? rows : 0;
#pragma unroll 4
    for (int r = lane / kCols; r < last; r += 32 / kCols) {
      uint16_t w;
      asm volatile("ld.shared.u16 %0, [%1];" : "=h"(w) : "r"(turn + r * kInt8TurnRow + c * 2));
      out[(size_t)r * p.C + c] = w;
    }
  }
  __syncwarp();
}

template <int YT, bool SWIGLU>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kInt8ProductThreads, 1)
    int8_product_kernel(const __grid_constant__ Int8Maps maps, const __grid_constant__ Int8ProductParams p) {
  extern __shared__ __align__(1024) uint8_t psm_raw[];
  __shared__ __align__(8) uint64_t raw_full[kInt8RawStages], raw_empty[kInt8RawStages];
  __shared__ __align__(8) uint64_t wide_full[kSets], wide_empty[kSets];  // full: of the first CTA, for both
  __shared__ __align__(8) uint64_t acc_full[2], acc_empty[2], drained;              // empty: of the first CTA, for both
  __shared__ uint32_t tmem_slot;
  __shared__ uint32_t s_warp[kInt8PlanThreads / 32 + 1];
  __shared__ int s_most;
  __shared__ int s_units;
  __shared__ volatile int s_abort;

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  uint8_t* sm = psm_raw + ((1024u - (smem_u32(psm_raw) & 1023u)) & 1023u);
  uint8_t* turn = sm + kInt8ProductSmem - 1024 - int8_fixed_smem(p.E);
  int* pre = reinterpret_cast<int*>(turn + 4 * (kInt8TurnWarp + kInt8MostRows * 4));

  if (warp == 0) {  // a lane has a barrier of each kind
    if (lane < kInt8RawStages) {
      mbar_init(&raw_full[lane], 1);
      mbar_init(&raw_empty[lane], 2 * kSetWarps);  // two sets once, or one twice
    }
    if (lane < kSets) {
      mbar_init(&wide_full[lane], 2 * kSetWarps);  // a set's warps in each CTA
      mbar_init(&wide_empty[lane], 1);
    }
    if (lane < 2) {
      mbar_init(&acc_full[lane], 1);
      mbar_init(&acc_empty[lane], 8);
    }
    if (lane == 2) mbar_init(&drained, 1);
    if (lane == 3) s_abort = 0, s_most = 0, s_warp[kInt8PlanThreads / 32] = 0;
    mbar_fence_init();
    __syncwarp();
  }
  cluster_arrive();
  pdl_wait();
  pdl_launch_dependents();
  // Eight warps count the experts' tiles: all of them took twice as long over it, for their instructions.
  if (threadIdx.x < kInt8PlanThreads) {
    int8_barrier<kInt8PlanThreads>();  // s_most and the last of s_warp are 0
    const int most = __reduce_max_sync(0xffffffffu, int8_expert_rows<kInt8PlanThreads>(p, pre));
    if (lane == 0 && most) atomicMax(&s_most, most);
    int8_barrier<kInt8PlanThreads>();
    const int tile = min(kInt8MostRows, max(32, (s_most + 31) >> 5 << 5));
    // overlapping experts can have more row tiles than the units' numbers hold: then none is worked on
    const bool countable = int8_row_tiles<kInt8PlanThreads>(p, tile, pre, s_warp);
    if (threadIdx.x == 0) s_units = countable ? pre[p.E] * ((p.N + kInt8Width - 1) / kInt8Width) : 0;
  } else if (warp == kInt8PlanThreads / 32) {
    tmem_alloc_pair(&tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_slot, 0);
  const int tile = min(kInt8MostRows, max(32, (__shfl_sync(0xffffffffu, s_most, 0) + 31) >> 5 << 5));
  const int KB = (p.K + kInt8Stage - 1) / kInt8Stage, n_tiles = (p.N + kInt8Width - 1) / kInt8Width;
  const int units = __shfl_sync(0xffffffffu, s_units, 0);
  const uint32_t raw_stages = p.raw_stages[(tile >> 5) - 1], raw_bytes = (uint32_t)(kInt8Width + tile) * 64;
  const int halves = int8_halves(tile);
  const uint32_t panel = tile * 64, slot_bytes = panel * halves, slot_cols = 32 * halves;
  // shared memory: the widened rows, then the copies' ring; tensor memory: two accumulators, then the widened weights
  const uint32_t sm0 = smem_u32(sm), raw0 = sm0 + kSets * slot_bytes, tmem_a = tmem + 2 * tile;
  const uint32_t raw_full0 = smem_u32(raw_full), raw_empty0 = smem_u32(raw_empty);
  const uint32_t wide_full0 = smem_u32(wide_full), wide_empty0 = smem_u32(wide_empty);
  const Int8Wait ab{&s_abort, p.status, p.timeout_ns};
  cluster_wait();  // the other CTA's barriers are there before anything arrives on them

  // A unit's copies and its MMAs are one thread's each. (With a whole warp going along, the MMA predicated for one
  // lane, each MMA took 60 clocks to issue: 32 is its time with 64 rows.)
  if (warp == 0) {
    const bool leader = elect_one();
    uint32_t stage = 0, phase = 1;
    bool ok = true;
    for (Int8Cursor at(n_tiles); at.u < units && ok; at.next()) {
      const Int8Unit un = int8_unit(p, pre, at, tile);
      if (leader) {
        const int x_boxes = (un.rows + 31) / 32;  // of 16 rows, in each CTA
        const int n0 = un.n0 + (int)rank * kInt8Half, row = un.row0 + (int)rank * x_boxes * 16;
        const CUtensorMap* x_map = &maps.x[x_boxes - 1];
        const uint32_t bytes = (uint32_t)(kInt8Half + x_boxes * 16) * 128u;
        for (int kb = 0; kb < KB; ++kb) {
          ok = int8_wait_one(raw_empty0 + stage * 8, phase, ab);
          if (!ok) break;
          const uint32_t st = raw0 + stage * raw_bytes, bar = raw_full0 + stage * 8;
          mbar_expect_tx_if(true, bar, bytes);
          tma_load_3d_if(true, st, &maps.w, kb * kInt8Stage, n0, un.e, bar);
          tma_load_2d_if(true, st + kInt8Half * 128, x_map, kb * kInt8Stage, row, bar);
          if (++stage == raw_stages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      ok = __all_sync(0xffffffffu, ok);
    }
  } else if (warp == 1) {
    if (rank == 0) {
      const uint64_t bdesc0 = sw128_desc(sm);
      const bool leader = elect_one();
      uint32_t slot = 0, phase = 0, done = 0;
      bool ok = true;
      for (Int8Cursor at(n_tiles); at.u < units && ok; at.next(), ++done) {
        const Int8Unit un = int8_unit(p, pre, at, tile);
        if (leader) {
          const uint32_t idesc = idesc_f16_pair((un.rows + 31) / 32 * 32), buf = done & 1, acc = tmem + buf * tile;
          ok = int8_wait_one(smem_u32(&acc_empty[buf]), ((done >> 1) & 1) ^ 1, ab);
          const int parts = halves == 2 ? KB : 2 * KB;
          for (int kb = 0; kb < parts && ok; ++kb) {
            ok = int8_wait_one(wide_full0 + slot * 8, phase, ab);
            if (!ok) break;
            tc_fence_after();
            const uint64_t bdesc = bdesc0 + slot * (slot_bytes >> 4);
            const uint32_t a = tmem_a + slot * slot_cols, here = slot;
            if (++slot == kSets) {
              slot = 0;
              phase ^= 1;
            }
            const int left = p.K - kb * (64 * halves);
            if (left >= 64 * halves) {
              tc_mma4_f16_pair(acc, a, bdesc, idesc, kb > 0);
              if (halves == 2) tc_mma4_f16_pair(acc, a + 32, bdesc + (panel >> 4), idesc, true);
            } else {
#pragma unroll 1
              for (int kk = 0; kk * 16 < left; ++kk)
                tc_mma_f16_pair(acc, a + kk * 8, bdesc + (kk >> 2) * (panel >> 4) + (kk & 3) * 2, idesc, kk > 0 || kb > 0);
            }
            tc_commit_pair(wide_empty0 + here * 8);
            if (kb + 1 == parts) tc_commit_pair(smem_u32(&acc_full[buf]));
          }
        }
        ok = __all_sync(0xffffffffu, ok);
      }
      if (leader) tc_commit_pair(smem_u32(&drained));
      __syncwarp();
    }
  } else if (warp < kWidenWarp + kSets * kSetWarps) {
    // of half a stage a thread has the 64 elements of a weight row, a warp 16 rows x 32 elements of x at a time
    const uint32_t mine = warp - kWidenWarp, set = mine / kSetWarps, w = mine % kSetWarps, q = warp & 3;
    const uint32_t swz = lane & 7;  // a row's place in its group of 8, which the copies' and the MMA's swizzle go by
    const uint32_t first = halves == 2 ? 0 : set & 1;  // the first half that is this set's
    const uint32_t w_row = (q * 32 + lane) * 128 + ((first * 4 ^ swz) << 4);  // chunk c is 16 c away by exclusive or
    const uint32_t ta0 = tmem_a + ((q * 32) << 16);
    // x: block of 16 rows t >> 1, chunks (t & 1) * 2 and the next, of task t = w, w + 4, ..
    const uint32_t chunk = (w & 1) * 2 + (lane >> 4), x_row = (w >> 1) * 2048 + (lane & 15) * 128;
    const uint32_t x_from = kInt8Half * 128 + x_row + (((first * 4 + chunk) ^ swz) << 4);
    const uint32_t x_to0 = sm0 + x_row + (((2 * chunk) ^ swz) << 4), x_to1 = sm0 + x_row + (((2 * chunk + 1) ^ swz) << 4);
    const uint32_t full0 = cluster_addr(wide_full0, 0);
    const uint32_t step = 2 * halves, begin = halves == 2 ? set : set >> 1;  // stages
    uint32_t raw = begin, raw_phase = 0, slot_phase = 1;
    bool ok = true;
    Int8Cursor at(n_tiles);
    int kb = (int)begin;
    for (; kb >= KB && at.u < units; kb -= KB) at.next();
    while (at.u < units && ok) {
      const Int8Unit un = int8_unit(p, pre, at, tile);
      const int tasks = (__shfl_sync(0xffffffffu, un.rows, 0) + 31) / 32 * 2;
      for (; kb < KB; kb += step) {
        ok = int8_wait2(raw_full0 + raw * 8, raw_phase, wide_empty0 + set * 8, slot_phase, ab);
        if (!ok) break;
        tc_fence_after();
        const uint32_t st = raw0 + raw * raw_bytes;
        uint32_t off = set * slot_bytes, ta = ta0 + set * slot_cols;
        // the second half's chunks are 64 bytes away, up or down, in the swizzled rows
#pragma unroll 1
        for (uint32_t flip = 0; flip < 64u * halves; flip += 64, ta += 32, off += panel) {
          {
            const uint32_t from = st + (w_row ^ flip);
            const int4 c0 = lds_v4(from), c1 = lds_v4(from ^ 16), c2 = lds_v4(from ^ 32), c3 = lds_v4(from ^ 48);
            uint32_t v[16];
            widen16(c0, v);
            widen16(c1, v + 8);
            tc_st16(ta, v);
            widen16(c2, v);
            widen16(c3, v + 8);
            tc_st16(ta + 16, v);
          }
          const uint32_t from = st + (x_from ^ flip), to0 = x_to0 + off, to1 = x_to1 + off;
#pragma unroll
          for (int i = 0; i < (kInt8MostRows / 32 * 2 + kSetWarps - 1) / kSetWarps; ++i)
            if ((int)w + i * kSetWarps < tasks) {
              const uint32_t g = i * kSetWarps * 1024;
              uint32_t v[8];
              widen16(lds_v4(from + g), v);
              asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to0 + g), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
                           : "memory");
              asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to1 + g), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                           : "memory");
            }
        }
        tc_wait_st();
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive_at(raw_empty0 + raw * 8, halves);
          mbar_arrive_cluster(full0 + set * 8);
        }
        if ((raw += step) >= raw_stages) {
          raw -= raw_stages;
          raw_phase ^= 1;
        }
        slot_phase ^= 1;
      }
      if (!ok) break;
      for (; kb >= KB && at.u < units; kb -= KB) at.next();
    }
    // the commit of the set's last slot comes from the first CTA: it is there before this one may leave
    if (ok) int8_wait(wide_empty0 + set * 8, slot_phase, ab);
  } else {
    const uint32_t q = warp & 3;
    const uint32_t my_turn = smem_u32(turn) + q * kInt8TurnWarp, my_xs = smem_u32(turn) + 4 * kInt8TurnWarp + q * kInt8MostRows * 4;
    const uint32_t empty0 = cluster_addr(smem_u32(acc_empty), 0);
    uint32_t done = 0;
    for (Int8Cursor at(n_tiles); at.u < units; at.next(), ++done) {
      const Int8Unit un = int8_unit(p, pre, at, tile);
      const uint32_t buf = done & 1;
      // An accumulator goes back only to a later unit, whose MMAs wait for all eight arrivals: one that nobody waits
      // for could reach the first CTA when it has left.
      const bool taken_again = at.u + 2 * (int)(gridDim.x >> 1) < units;
      const int n = un.n0 + (int)rank * kInt8Half + 32 * (int)q;  // the warp's first weight row
      const int groups = n < p.N ? (un.rows + 31) / 32 : 0;
      const float wscale = n + lane < p.N && groups ? p.ws[(size_t)un.e * p.N + n + lane] : 0.f;
      for (int g = 0; g < groups; ++g) {
        const int r = 32 * g + lane;
        const float v = p.xs && r < un.rows ? p.xs[un.row0 + r] : 1.f;
        asm volatile("st.shared.f32 [%0], %1;" ::"r"(my_xs + r * 4), "f"(v) : "memory");
      }
      __syncwarp();
      if (!int8_wait(smem_u32(&acc_full[buf]), (done >> 1) & 1, ab)) break;
      tc_fence_after();
      const uint32_t acc = tmem + ((32 * q) << 16) + buf * tile;
#pragma unroll 1
      for (int g = 0; g < groups; ++g) {
        const int left = un.rows - 32 * g;
        uint32_t v[32];
        tc_ld32(acc + 32 * g, v);
        tc_wait_ld();
        if (g + 1 == groups) {
          // the last columns are in registers: the accumulator goes back before they are stored
          tc_fence_before();
          __syncwarp();
          if (lane == 0 && taken_again) mbar_arrive_cluster(empty0 + buf * 8);
        }
        int8_store<YT, SWIGLU>(p, my_turn, v, wscale, my_xs + g * 128, un.row0 + 32 * g, min(32, left), SWIGLU ? n / 2 : n);
      }
      if (groups == 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && taken_again) mbar_arrive_cluster(empty0 + buf * 8);
      }
    }
  }

  __syncthreads();
  if (threadIdx.x == 0) {
    // the pair's MMAs, and after an abort the copies in flight, end before their memory is given back
    if (!mbar_try_wait(&drained, 0) || s_abort) {
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(&drained, 0) && globaltimer_ns() - t0 < 1000000ull) {}
      if (s_abort)
        while (globaltimer_ns() - t0 < 1000000ull) {}
    }
  }
  tc_fence_before();
  __syncthreads();
  // Nor does a CTA leave while the other one may still arrive on its barriers. The barrier releases nothing, so it orders no
  // arrival: each one has been waited for, or (after an abort) a millisecond has passed.
  cluster_sync();
  if (warp == kInt8PlanThreads / 32) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// ------------------------------------------------------------- any k and alignment

// Rows whose length the tensor kernel's copies cannot take (k not a multiple of 16): 32 rows
// x 64 features a unit, by a warp's integer products (mma.sync, sums in 32-bit integers). A
// warp loads 128 bytes of a row as aligned words, which neighbouring lanes put together,
// while the stage before is worked on. 4096 rows of 128 experts, 2040 -> 1024: 372 us, where
// the tensor kernel takes 52 with 2032; bound by the words' loads and their putting together
// (a stage has 96 of these for 8 products a warp).
constexpr int kPlainThreads = 256, kPlainRows = 32, kPlainCols = 64, kPlainK = 128;

// A matrix's rows from one of them on, `left` of its bytes: 32-bit offsets from an aligned address, which `skip` bytes of
// other rows may follow.
struct PlainRows {
  const int8_t* base;
  uint32_t skip, left;
  __device__ PlainRows(const int8_t* m, long long total, long long at)
      : base(m + (at & ~3ll)), skip((uint32_t)at & 3), left((uint32_t)min(total - (at & ~3ll), 0x7fffffffll)) {}
  // a lane's aligned word of the `bytes` bytes at `at`, and the one behind lane 31's; the words that hold
  // the matrix's last bytes and others are left out
  __device__ __forceinline__ void load(uint32_t at, int bytes, uint32_t& word, uint32_t& behind) const {
    const uint32_t lane = threadIdx.x & 31, byte = (at & ~3u) + 4 * lane;
    const bool here = (int)(4 * lane) < bytes + (int)(at & 3);
    word = here && byte + 4 <= left ? __ldg(reinterpret_cast<const unsigned int*>(base + byte)) : 0u;
    behind = here && lane == 31 && (at & 3) && byte + 8 <= left ? __ldg(reinterpret_cast<const unsigned int*>(base + byte + 4)) : 0u;
  }
  // a lane's four of those bytes, zeros beyond them
  __device__ __forceinline__ uint32_t four(uint32_t at, int bytes, uint32_t word, uint32_t behind) const {
    const uint32_t lane = threadIdx.x & 31, byte = (at & ~3u) + 4 * lane;
    const auto last = [&](uint32_t from, uint32_t& v) {  // the matrix's last word, if bytes follow it that are not its own
      if (from < left && from + 4 > left)
        for (uint32_t q = 0; from + q < left; ++q) v |= (uint32_t)(uint8_t)base[from + q] << (8 * q);
    };
    last(byte, word);
    if (lane == 31) last(byte + 4, behind);
    uint32_t next = __shfl_down_sync(0xffffffffu, word, 1);
    if (lane == 31) next = behind;
    const uint32_t v = __funnelshift_r(word, next, 8 * (at & 3));
    const int mine = bytes - 4 * (int)lane;
    return mine >= 4 ? v : mine <= 0 ? 0 : v & (0xffffffffu >> (32 - 8 * mine));
  }
};

// 16 rows by 8 features, 32 products each: a lane (g, t) of 8 x 4 has row g's and row g + 8's words t and t + 4 of x, feature
// g's of w, and results (g, 2 t), (g, 2 t + 1) and those of row g + 8.
__device__ __forceinline__ void plain_mma(int (&d)[4], const int (&a)[4], int b0, int b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int YT, bool SWIGLU>
__global__ void __launch_bounds__(kPlainThreads, 2) int8_product_plain_kernel(Int8ProductParams p) {
  // 4 words beyond a row's: a fragment's eight rows of four words are in different banks
  __shared__ int s_x[kPlainRows][kPlainK / 4 + 4], s_w[kPlainCols][kPlainK / 4 + 4];
  __shared__ uint32_t s_warp[kPlainThreads / 32 + 1];
  extern __shared__ int pre[];
  if (threadIdx.x == 0) s_warp[kPlainThreads / 32] = 0;
  pdl_wait();
  pdl_launch_dependents();
  __syncthreads();
  int8_expert_rows<kPlainThreads>(p, pre);
  if (!int8_row_tiles<kPlainThreads>(p, kPlainRows, pre, s_warp)) return;
  const int* first = pre + p.E + 1;
  const int* count = first + p.E;
  const int n_tiles = (p.N + kPlainCols - 1) / kPlainCols;
  const long long units = (long long)pre[p.E] * n_tiles;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int m0 = 16 * (warp & 1), f0 = 16 * (warp >> 1);  // the warp's 16 rows and 16 features
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const int mt = (int)(u / n_tiles), n0 = (int)(u % n_tiles) * kPlainCols;
    const int e = int8_expert_of(pre, p.E, mt);
    const int before = (mt - pre[e]) * kPlainRows, rows = min(kPlainRows, count[e] - before);
    const long long row0 = first[e] + before;
    int acc[2][4] = {};  // of 16 x 8 each
    constexpr int kPitch = kPlainK / 4 + 4, kWarps = kPlainThreads / 32, kXLoads = kPlainRows / kWarps, kLoads = (kPlainRows + kPlainCols) / kWarps;
    const PlainRows xr(p.x, (long long)p.W * p.A * p.K, row0 * p.K);
    const PlainRows wr(p.w, (long long)p.E * p.N * p.K, ((long long)e * p.N + n0) * p.K);
    uint32_t next[kLoads], behind[kLoads];
    // all loads of a stage before anything waits for one of them
    const auto load = [&](int k0) {
      const int bytes = min(kPlainK, p.K - k0);
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int r = (i < kXLoads ? i : i - kXLoads) * kWarps + warp;
        const PlainRows& m = i < kXLoads ? xr : wr;
        m.load(m.skip + r * p.K + k0, r < (i < kXLoads ? rows : p.N - n0) ? bytes : -4, next[i], behind[i]);
      }
    };
    load(0);
    for (int k0 = 0; k0 < p.K; k0 += kPlainK) {
      const int bytes = min(kPlainK, p.K - k0);
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int r = (i < kXLoads ? i : i - kXLoads) * kWarps + warp;
        const PlainRows& m = i < kXLoads ? xr : wr;
        (i < kXLoads ? s_x[r] : s_w[r])[lane] =
            (int)m.four(m.skip + r * p.K + k0, r < (i < kXLoads ? rows : p.N - n0) ? bytes : -4, next[i], behind[i]);
      }
      __syncthreads();
      if (k0 + kPlainK < p.K) load(k0 + kPlainK);
#pragma unroll
      for (int k = 0; k < kPlainK / 4; k += 8) {
        const int* x = &s_x[m0 + g][k + t];
        const int a[4] = {x[0], x[8 * kPitch], x[4], x[8 * kPitch + 4]};
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const int* w = &s_w[f0 + 8 * b + g][k + t];
          plain_mma(acc[b], a, w[0], w[4]);
        }
      }
    }
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      const int r = m0 + g + 8 * a;
      if (r >= rows) continue;
      const float xs = p.xs ? p.xs[row0 + r] : 1.f;
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int j = n0 + f0 + 8 * b + 2 * t;  // and the next
        float z[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) z[i] = j + i < p.N ? (float)acc[b][2 * a + i] * xs * p.ws[(size_t)e * p.N + j + i] : 0.f;
        uint16_t* y = static_cast<uint16_t*>(p.y) + (size_t)(row0 + r) * p.C;
        if (SWIGLU) {
          if (j < p.N) y[j >> 1] = int8_round<YT>(int8_swiglu(z[0], z[1]));
        } else {
          if (j < p.N) y[j] = int8_round<YT>(z[0]);
          if (j + 1 < p.N) y[j + 1] = int8_round<YT>(z[1]);
        }
      }
    }
  }
}

// ------------------------------------------------------------- host side

static PFN_cuTensorMapEncodeTiled_v12000 int8_encode_fn() {
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

// Matrices [depth][rows][cols] of int8, boxes of 128 columns x box_rows rows; zeros beyond the ends.
static bool int8_map(CUtensorMap* m, const void* base, unsigned long long cols, unsigned long long rows, unsigned long long depth,
                     unsigned box_rows) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = int8_encode_fn();
  if (!enc) return false;
  cuuint64_t dims[3] = {cols, rows, depth};
  cuuint64_t strides[2] = {cols, cols * rows};
  cuuint32_t box[3] = {(cuuint32_t)kInt8Stage, box_rows, 1};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, depth ? 3 : 2, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

typedef void (*Int8PlainKernel)(Int8ProductParams);
typedef void (*Int8Kernel)(Int8Maps, Int8ProductParams);

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
  // units of a row tile x 64 weight rows are counted in 32 bits, and a CTA looks some of its units ahead
  const long long most_units = ((long long)W * A / 32 + E) * ((n + 63LL) / 64);
  if ((long long)E * n >= 2147483647LL || most_units >= 2147483647LL - 65536) return MOE_ERR_INVALID_ARG;
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
  p.timeout_ns = (uint64_t)cfg->wait_timeout_us * 1000ull;
  const bool sw = epilogue == MOE_EPI_SWIGLU;
  int per_sm = 0;
  if (k % 16 == 0) {
    Int8Maps maps;
    bool good = true;
    for (unsigned i = 0; i < 6; ++i)
      good = good && int8_map(&maps.x[i], x, (unsigned long long)k, (unsigned long long)W * A, 0, 16 * (i + 1));
    good = good && int8_map(&maps.w, w, (unsigned long long)k, (unsigned long long)n, (unsigned long long)E, kInt8Half);
    if (!good) return MOE_ERR_CUDA;
    for (int t = 0; t < 6; ++t) p.raw_stages[t] = int8_raw_stages(E, 32 * (t + 1));
    const Int8Kernel kernel = y_dtype == MOE_F16 ? (sw ? int8_product_kernel<MOE_F16, true> : int8_product_kernel<MOE_F16, false>)
                                                 : (sw ? int8_product_kernel<MOE_BF16, true> : int8_product_kernel<MOE_BF16, false>);
    if (resident_blocks((const void*)kernel, kInt8ProductThreads, kInt8ProductSmem, &per_sm) != cudaSuccess || per_sm < 1)
      return MOE_ERR_CUDA;
    const long long pairs = most_units < nsm / 2 ? most_units : nsm / 2;
    if (pairs < 1) return MOE_ERR_CUDA;
    PdlLaunch L(dim3((unsigned)(2 * pairs)), dim3(kInt8ProductThreads), kInt8ProductSmem,
                static_cast<cudaStream_t>(stream));
    if (cudaLaunchKernelEx(&L.cfg, kernel, maps, p) != cudaSuccess) return MOE_ERR_CUDA;
    note_launches(1);
    return MOE_OK;
  }
  const Int8PlainKernel plain =
      y_dtype == MOE_F16 ? (sw ? int8_product_plain_kernel<MOE_F16, true> : int8_product_plain_kernel<MOE_F16, false>)
                         : (sw ? int8_product_plain_kernel<MOE_BF16, true> : int8_product_plain_kernel<MOE_BF16, false>);
  const size_t smem = (3 * (size_t)E + 1) * 4;
  if (resident_blocks((const void*)plain, kPlainThreads, smem, &per_sm) != cudaSuccess || per_sm < 1) return MOE_ERR_CUDA;
  PdlLaunch L(dim3((unsigned)(nsm * per_sm)), dim3(kPlainThreads), smem, static_cast<cudaStream_t>(stream));
  if (cudaLaunchKernelEx(&L.cfg, plain, p) != cudaSuccess) return MOE_ERR_CUDA;
  note_launches(1);
  return MOE_OK;
}

// ebc_mx4_product.cu -- the experts' products on 4-bit microscaled operands:
// ys[r] = W[e(r)] x[r], block-scaled fp4 matrix instructions with the
// accumulator in tensor memory.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "ebc_mx4.cuh"

using namespace ebc;

namespace {

// ---- geometry ----
// A tile is 128 outputs of an expert (the M side: weights, one per tensor
// memory lane) by kTN of its rows (the N side).  The rows are on the N side
// because an expert's share of a batch is ragged and often small, and N may be
// as small as 16 where M is fixed.  A stage holds 256 values of K: 128 bytes a
// row, one span of the 128-byte swizzle, four matrix instructions of K = 64.
constexpr int kM = 128;
constexpr int kStageK = 256;
constexpr int kRowBytes = kStageK / 2;
constexpr int kScaleTile = 512;    // bytes of the scales of 128 rows x 4 blocks, as the matrix unit wants them
// warp 0 loads, warp 1 multiplies, warps 2-3 lay out scales, warps 4-11 store:
// three warps a scheduler, so that a storing thread can hold its share of a
// tile (64 words) in its 168 registers
constexpr int kThreads = 384;
// (in a pair's second CTA, which does not multiply, warp 1 announces the scales)
constexpr int kScaleWarp0 = 2, kScaleWarps = 2;
constexpr int kStoreWarp0 = 4, kStoreWarps = 8;
constexpr int kStoreRows = 16;     // rows that a storing warp reads at a time

// kCtas = 2: a pair of CTAs on one tile of 256 outputs.  Each brings in its own
// 128 outputs and half of the rows; the pair's matrix instructions read both
// halves, so a CTA moves and reads half as many of the rows' bytes.
template <int kTN, int kCtas>
struct Geom {
  static constexpr int kOuts = kM * kCtas;                                // outputs of a tile
  static constexpr int kScaleB = (kTN + 127) / 128;                       // scale tiles of the rows per 4 blocks
  static constexpr int kBRows = kTN / kCtas;                              // rows that a CTA brings in
  static constexpr int kBox = kBRows < 64 ? kBRows : 64;                  // rows of one copy
  static constexpr int kRound = 16 * kCtas;                               // N of the instructions is a multiple
  static constexpr int kABytes = kM * kRowBytes;
  static constexpr int kBBytes = kBRows * kRowBytes;
  static constexpr int kScaleBytes = 2 * (1 + kScaleB) * kScaleTile;      // per stage: 8 blocks a row
  // (256 rows a tile with 4 / 5 stages of codes: 329 / 320 us of 8192 x 8192, and
  // more do not fit; 16 rows with 5 / 6 / 8 / 10: 12.9 / 12.6 / 13.1 / 13.5 us of a
  // decode step)
  static constexpr int kStages = kTN == 256 ? 5 : kTN == 64 ? 7 : 6;
  // A pair's scales have a ring of their own, a longer one: the second CTA's are
  // known to the first only some 3600 cycles after they were laid out (see
  // below).  The barriers on which stages are given back are as many, so that one
  // instruction a stage gives back both.  8192 x 8192: 5 / 6 / 7 / 8 / 10 / 12 /
  // 14 / 16 stages 483 / 426 / 396 / 360 / 342 / 328 / 325 / 322 us.
  static constexpr int kScaleStages = kCtas == 2 ? 16 : kStages;
  static constexpr int kAcc = kTN == 256 ? 1 : 2;                         // accumulators
  static constexpr int kAccCols = kTN < 32 ? 32 : kTN;
  static constexpr int kScaleCols = 2 * (1 + kScaleB) * 4;                // tensor memory columns per stage
  static constexpr int kCols = 512;
  // Whether clusters of CTAs may share a tile's K.  They do where the tiles are
  // so few that twice as many would still run at once, and then the smallest
  // tiles, which the choice of a tile's rows falls on, are at most that many.
  static constexpr bool kShares = kTN == 16;
  static constexpr size_t kSmem =
      1024 + (size_t)kStages * (kABytes + kBBytes) + (size_t)kScaleStages * kScaleBytes;
  // A scale warp's next stages must not be two rounds of the ring past what it
  // knows to be given back: a barrier's phase is told by its parity alone.
  static_assert(2 * kScaleWarps <= kScaleStages + 1, "scale warps");
  static_assert(kAcc * kAccCols + kStages * kScaleCols <= kCols, "tensor memory");
  static_assert(kSmem <= 217 * 1024, "shared memory");
};

// ---- PTX ----
__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void mbar_init(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}
// The address of a shared variable of the pair's first CTA (kCtas = 1: of this
// one), as the pair's shared memory has it.
template <int kCtas>
__device__ __forceinline__ uint32_t in_first(const void* p) {
  uint32_t r = smem_u32(p);
  if constexpr (kCtas == 2) asm volatile("mapa.shared::cluster.u32 %0, %0, 0;" : "+r"(r));
  return r;
}
// An arrival at such a barrier that announces no memory of another CTA: this
// CTA's, or none (an accumulator given back).
template <int kCtas>
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  if constexpr (kCtas == 2)
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
  else
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// An arrival at a barrier of the pair's first CTA that makes this CTA's memory
// known to who waits there: a round trip to L2, 1200 cycles and more.  After it a
// relaxed one is enough, for who waits for both in that order.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_arrive_after(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// kCtas = 2: what the pair's other CTA has announced is known after the wait, too
template <int kCtas = 1>
__device__ __forceinline__ bool mbar_try_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  if constexpr (kCtas == 2)
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
  return ok != 0u;
}
// whether the phase is over now: does not wait
template <int kCtas = 1>
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  if constexpr (kCtas == 2)
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
  return ok != 0u;
}
// a box into this CTA's shared memory; its bytes are counted at `bar`, which
// may be the other CTA's of the pair
template <int kCtas>
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1) {
  if constexpr (kCtas == 2)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(dst),
        "l"(map), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            dst),
        "l"(map), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// an arrival at `bar` (of both CTAs of a pair) once what was issued is done
template <int kCtas>
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  if constexpr (kCtas == 2)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
  else
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}
// 32 rows x 16 bytes of scales to four columns of each quarter of tensor memory
// (in both CTAs of a pair, each from its own shared memory)
template <int kCtas>
__device__ __forceinline__ void tc_copy_scales(uint32_t taddr, uint64_t desc) {
  if constexpr (kCtas == 2)
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
template <int kCtas>
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                       uint32_t accumulate) {
  if constexpr (kCtas == 2)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
        : "memory");
}
template <int kCtas>
__device__ __forceinline__ void tc_alloc(uint32_t* where, uint32_t cols) {
  if constexpr (kCtas == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(where)), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(where)), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
}
template <int kCtas>
__device__ __forceinline__ void tc_free(uint32_t tmem, uint32_t cols) {
  if constexpr (kCtas == 2)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols) : "memory");
  else
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols) : "memory");
}
// 32 lanes x 16 columns, a lane a thread
__device__ __forceinline__ void tc_load16(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
}
// one thread of the warp, known to the compiler as such: what it issues has
// its operands in uniform registers
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0u;
}
__device__ __forceinline__ void tc_load_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// Shared-memory operand descriptor: rows of 128 bytes in the 128-byte swizzle,
// eight-row groups 1024 bytes apart.  Addresses count in 16 bytes.
constexpr uint64_t kOperandDesc = (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
// Scales: no swizzle, eight-row groups of 16-byte rows 128 bytes apart.
constexpr uint64_t kScaleDesc = (1ull << 16) | (8ull << 32) | (1ull << 46);
__device__ __forceinline__ uint32_t desc_addr(uint32_t addr) { return (addr >> 4) & 0x3FFFu; }
// Instruction descriptor: both operands E2M1 along K, scales UE8M0, M = m,
// N = n; `id` (0 or 2) is the byte of a scale word where the instruction's two
// blocks start.
__device__ __forceinline__ uint32_t instr_desc(int m, int n, int id) {
  return (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | (1u << 23) | ((uint32_t)(m >> 4) << 24) |
         ((uint32_t)id << 4) | ((uint32_t)id << 29);
}

// The tiles of a CTA, one after the other: a run of rows, and a place among the
// outputs.  Steps are additions; the run's expert is mostly the last tile's or
// the next, else searched for.
struct Walk {
  int step_run, step_out, run, out, e;
  __device__ __forceinline__ Walk(int out_tiles, unsigned first, unsigned step)
      : step_run((int)(step / (unsigned)out_tiles)),
        step_out((int)(step % (unsigned)out_tiles)),
        run((int)(first / (unsigned)out_tiles)),
        out((int)(first % (unsigned)out_tiles)),
        e(0) {}
  // Whether there is a tile; then its first row and row count (at most tn).
  // begin, tiles: per expert, its first row and the runs of the experts before.
  __device__ __forceinline__ bool at(const int* begin, const int* tiles, int experts, int tn, int* row0,
                                     int* count) {
    if (run >= tiles[experts]) return false;
    if (tiles[e + 1] <= run) ++e;
    if (tiles[e + 1] <= run) {
      int hi = experts;   // tiles[e] <= run < tiles[hi]
      while (hi - e > 1) {
        const int mid = (e + hi) >> 1;
        if (tiles[mid] <= run) e = mid; else hi = mid;
      }
    }
    *row0 = begin[e] + (run - tiles[e]) * tn;
    const int left = begin[e + 1] - *row0;
    *count = left < tn ? left : tn;
    return true;
  }
  __device__ __forceinline__ void next(int out_tiles) {
    run += step_run;
    out += step_out;
    if (out >= out_tiles) {
      out -= out_tiles;
      ++run;
    }
  }
};

struct Args {
  const uint8_t* xs;        // scales of the rows
  const uint8_t* ws;        // scales of the weights
  const int32_t* offsets;   // null: one expert takes every row
  void* ys;
  Glob* glob;
  int64_t rows, outs, scale_bytes;
  int out_type, blocks, experts;   // blocks: scale blocks a row
  int first_wait;                  // (normally the full limit) polls of the multiplying warp's first wait for a stage, and of a pair's first loading warp
  int split_log2;                  // CTAs (a cluster) that share a tile's K; more than one only with a tile a cluster
};

// A wait that gives up: after `limit` polls or kWaitCycles, or once another
// thread of the cluster did.  The first to give up records the time-out and
// tells the cluster's CTAs (which all stay until the last has ended).
constexpr long long kWaitCycles = 1ll << 32;   // about two seconds
template <int kCtas = 1>
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort, Glob* glob,
                                     int limit = kWaitLimit) {
  if (limit > 0 && mbar_try_wait<kCtas>(bar, parity)) return true;
  const long long begin = clock64();
  for (int i = 1; i < limit && clock64() - begin < kWaitCycles; ++i) {
    if (mbar_try_wait<kCtas>(bar, parity)) return true;
    if (*abort) return false;
  }
  record_error(glob, EBC_ERR_DEVICE_TIMEOUT);
  uint32_t ctas;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
  for (uint32_t q = 0; q < ctas; ++q) {
    uint32_t at = smem_u32(const_cast<int*>(abort));
    asm volatile("mapa.shared::cluster.u32 %0, %0, %1;\n st.shared::cluster.u32 [%0], %2;" : "+r"(at) : "r"(q), "r"(1)
                 : "memory");
  }
  return false;
}

// What the other CTA of a pair has asked for, told in both directions by the
// loading warps (stages + 1; 0 is what a CTA that has not told leaves).
__device__ __forceinline__ void tell_pair(volatile uint32_t* told, uint32_t rank, uint32_t stages) {
  uint32_t at = smem_u32(const_cast<uint32_t*>(told));
  asm volatile("mapa.shared::cluster.u32 %0, %0, %1;\n st.shared::cluster.u32 [%0], %2;" : "+r"(at)
               : "r"(rank ^ 1u), "r"(stages + 1)
               : "memory");
}
__device__ __forceinline__ uint32_t told_by_pair(volatile uint32_t* told) {
  for (int i = 0; i < kWaitLimit; ++i) {
    const uint32_t v = *told;
    if (v) return v - 1;
    __nanosleep(64);
  }
  return 0;
}

// A wait for what is in flight, with the same limits and nobody to tell.
__device__ __forceinline__ void drain(uint64_t* bar, uint32_t parity) {
  const long long begin = clock64();
  for (int i = 0; i < kWaitLimit && clock64() - begin < kWaitCycles; ++i)
    if (mbar_try_wait(bar, parity)) return;
}

// two sums as bf16 or fp16, `lo` in the low half
__device__ __forceinline__ uint32_t pack2(uint32_t lo, uint32_t hi, bool bf16) {
  if (bf16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(lo), __uint_as_float(hi));
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(__uint_as_float(lo), __uint_as_float(hi));
  return *reinterpret_cast<const uint32_t*>(&v);
}

// A storing warp's share of a tile, 16-bit results: 32 outputs, one a lane, of
// every other run of 16 rows.  All of it is read and rounded first and the
// accumulator given back, then it is stored while the next tile is multiplied.
// A store is 64 bytes of one row: turning the values over in shared memory to
// 16 bytes a lane took 2 to 3% longer in all (shared memory is what the
// multiplying waits for) and 30% with rows of odd length.
template <int kTN, int kCtas>
__device__ __forceinline__ void store_tile(uint32_t d, bool bf16, uint16_t* y, int64_t ld, bool mine, int odd,
                                           int count, int lane, uint32_t given_back) {
  constexpr int kRuns = kTN < 32 ? 1 : kTN / 32;
  constexpr int kBatch = kRuns < 2 ? kRuns : 2;   // runs whose loads are in flight
  uint32_t v[kRuns][8];
#pragma unroll
  for (int i0 = 0; i0 < kRuns; i0 += kBatch) {
    uint32_t f[kBatch][16];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (((i0 + i) * 2 + odd) * kStoreRows < count) tc_load16(d + ((i0 + i) * 2 + odd) * kStoreRows, f[i]);
    tc_load_wait();
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (((i0 + i) * 2 + odd) * kStoreRows < count)
#pragma unroll
        for (int c = 0; c < 8; ++c) v[i0 + i][c] = pack2(f[i][2 * c], f[i][2 * c + 1], bf16);
  }
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive<kCtas>(given_back);
  int left = count - odd * kStoreRows;
  y += odd * kStoreRows * ld + lane;
#pragma unroll
  for (int i = 0; i < kRuns; ++i) {
    uint16_t* p = y;
    if (left >= kStoreRows) {
      if (mine)
#pragma unroll
        for (int c = 0; c < kStoreRows; ++c) {
          *p = (uint16_t)(c & 1 ? v[i][c / 2] >> 16 : v[i][c / 2]);
          p += ld;
        }
    } else if (left > 0) {
#pragma unroll
      for (int c = 0; c < kStoreRows; ++c) {
        if (mine && c < left) *p = (uint16_t)(c & 1 ? v[i][c / 2] >> 16 : v[i][c / 2]);
        p += ld;
      }
    }
    y += 2 * kStoreRows * ld;
    left -= 2 * kStoreRows;
  }
}

// The same in fp32, 16 rows at a time.
__device__ __forceinline__ void store_full(uint32_t taddr, float* y, int64_t ld, bool mine, int n_row, int lane) {
  uint32_t v[16];
  tc_load16(taddr, v);
  tc_load_wait();
  y += lane;
#pragma unroll
  for (int c = 0; c < kStoreRows; ++c) {
    if (mine && c < n_row) *y = __uint_as_float(v[c]);
    y += ld;
  }
}

// One persistent CTA an SM walks tiles blockIdx.x, + gridDim.x, ...; outputs
// of a run of rows come one after the other, so that the CTAs working at the
// same time share both operands in L2.
//   warp 0      brings the codes of both operands in by TMA, a ring of stages
//   warps 2-3   lay the scales out: the matrix unit reads the scales of 128
//               rows x 4 blocks from tensor memory as 32 lanes x 4 words,
//               row r in lane r % 32, word r / 32, so a row's four scale bytes
//               are one 4-byte store.  Rows and blocks past the end get 1.
//   warp 1      copies a stage's scales to tensor memory and issues its matrix
//               instructions; each stage has its own scale columns, so they
//               are written again only after the stage was given back; in a
//               pair's second CTA it announces that CTA's scales to the first
//   warps 4-11  read the accumulator, round once, to the type that the caller
//               asked for, and store
// The N of the instructions is the tile's row count rounded up to 16, so a
// ragged segment's last tile costs what it holds.
// With few tiles a cluster of CTAs takes one: each the sum over its share
// of K, which it leaves in shared memory; then each adds up the cluster's sums
// of every split-th row, in the order of the CTAs.
// In a pair the first CTA multiplies for both; stages, scales and accumulators
// are announced at its barriers, and its instructions' ends at both CTAs'.
// Every wait is bounded (see wait()); a CTA that gives up waits for the copies
// and instructions it has in flight, frees its tensor memory and returns.  A
// pair's copies are counted together, at the first CTA's barriers, so there the
// loading warps first bring each other to the same stage.
// 17/32 of a byte is read a value of rows and weights, and outs * rows results
// are written; one expert, 16384 rows x 8192 x 8192: 320 us (6.9 PFLOP/s), where
// a pair's stage takes 550 cycles to 512 of its instructions; 32 experts of 4096
// x 4096: 120 us (4.6 PFLOP/s), a quarter of it the accumulator's reading, which
// the next tile's instructions wait for; one turn of small tiles: 7 to 9 us of
// latency, from the first stage's arrival to the last result's store.
template <int kTN, int kCtas>
__global__ void __launch_bounds__(kThreads, 1) k_mx4_product(const __grid_constant__ CUtensorMap wmap,
                                                             const __grid_constant__ CUtensorMap xmap, Args a) {
  using G = Geom<kTN, kCtas>;
  extern __shared__ uint8_t raw[];
  __shared__ uint64_t full[G::kStages], scaled[G::kScaleStages], empty[G::kScaleStages];
  __shared__ uint64_t laid[G::kScaleStages];   // of a pair's second CTA: scales laid out, not yet announced
  __shared__ uint64_t acc_full[G::kAcc], acc_empty[G::kAcc], drained;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ uint32_t s_told;   // see tell_pair()
  __shared__ int s_begin[EBC_MAX_EXPERTS + 1];   // first row of each expert
  __shared__ int s_tiles[EBC_MAX_EXPERTS + 1];   // runs of kTN rows of the experts before
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int rank = kCtas == 2 ? blockIdx.x & 1 : 0;   // in the pair
  uint8_t* base = raw + (1024 - (smem_u32(raw) & 1023)) % 1024;
  uint8_t* sA = base;
  uint8_t* sB = sA + G::kStages * G::kABytes;
  uint8_t* sS = sB + G::kStages * G::kBBytes;

  if (w == 0 && lane == 0) {
    for (int i = 0; i < G::kStages; ++i) mbar_init(&full[i], 1);
    for (int i = 0; i < G::kScaleStages; ++i) {
      mbar_init(&scaled[i], kCtas);
      mbar_init(&laid[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < G::kAcc; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], kStoreWarps * kCtas);
    }
    mbar_init(&drained, 1);
    s_abort = 0;
    s_told = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (w == 1) {
    tc_alloc<kCtas>(&s_tmem, G::kCols);
    tc_fence_before();
  }
  pdl_enter();
  if (w == 2) {
    // the experts' segments, made to ascend inside the rows, and their runs
    bool bad = a.offsets && lane == 0 && a.offsets[0] != 0;
    int before = 0, tiles = 0;
    if (lane == 0) s_begin[0] = s_tiles[0] = 0;
    for (int e0 = 0; e0 < a.experts; e0 += 32) {
      const int e = e0 + lane;
      int end = 0;
      if (e < a.experts) {
        const int v = a.offsets ? a.offsets[e + 1] : (int)a.rows;
        end = v < 0 ? 0 : v > a.rows ? (int)a.rows : v;
        bad |= end != v;
      }
      int top = end > before ? end : before;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, top, off);
        if (lane >= off && v > top) top = v;
      }
      bad |= e < a.experts && top != end;
      int prev = __shfl_up_sync(0xffffffffu, top, 1);
      if (lane == 0) prev = before;
      int run = (top - prev + kTN - 1) / kTN;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, run, off);
        if (lane >= off) run += v;
      }
      if (e < a.experts) {
        s_begin[e + 1] = top;
        s_tiles[e + 1] = tiles + run;
      }
      before = __shfl_sync(0xffffffffu, top, 31);
      tiles += __shfl_sync(0xffffffffu, run, 31);
    }
    if (bad && blockIdx.x == 0) record_error(a.glob, EBC_ERR_INVALID_ARG);
  }
  __syncthreads();
  if (kCtas == 2 || (G::kShares && a.split_log2 > 0)) cluster_sync();   // the cluster's CTAs have started and set up their barriers
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const uint32_t tmem_scales = tmem + G::kAcc * G::kAccCols;
  const int out_tiles = (int)((a.outs + G::kOuts - 1) / G::kOuts);
  const int stages = (a.blocks + 7) / 8;   // stages of a tile

  const int shift = G::kShares ? a.split_log2 : 0, split = 1 << shift, part = (int)blockIdx.x & (split - 1);
  // the groups of two stages, and the stages, that are this CTA's
  const int groups = (stages + 1) / 2, group0 = groups * part >> shift, group1 = groups * (part + 1) >> shift;
  const int k0 = 2 * group0, k1 = 2 * group1 < stages ? 2 * group1 : stages;
  const Walk start(out_tiles, blockIdx.x / kCtas >> shift, gridDim.x / kCtas >> shift);
  Walk walk = start;
  int row0, count;
  uint32_t issued = 0;   // stages that warp 0 has asked for
  if (w == 0) {
    int s = 0, back = G::kScaleStages - G::kStages;   // the barrier that a stage of kStages before was given back on
    uint32_t phase = 1;                               // of that barrier
    bool ok = true;
    uint32_t goal = ~0u;  // stages to ask for: all, until a wait gave up
    int limit = kCtas == 2 && rank == 0 ? a.first_wait : kWaitLimit;
    for (; issued < goal && walk.at(s_begin, s_tiles, a.experts, kTN, &row0, &count); walk.next(out_tiles)) {
      // a pair's first CTA has the first half of the instructions' N, the other the second
      const int mine = (count + G::kRound - 1) / G::kRound * 16;
      const int boxes = (mine + G::kBox - 1) / G::kBox, brow = row0 + rank * mine;
      const int wrow = (int)(walk.e * a.outs) + walk.out * G::kOuts + rank * kM;
      for (int k = k0; k < k1 && issued < goal; ++k) {
        if (ok) ok = __all_sync(0xffffffffu, wait(&empty[back], phase, &s_abort, a.glob, limit));
        limit = kWaitLimit;
        if (!ok && goal == ~0u) {
          // A stage that the other CTA has asked for has been given back to both
          // (by one commit), so this CTA can ask for it too without a wait; then
          // each stage's bytes are expected once and arrive in full.
          goal = issued;
          if constexpr (kCtas == 2) {
            if (lane == 0) tell_pair(&s_told, rank, issued);
            const uint32_t other = __shfl_sync(0xffffffffu, told_by_pair(&s_told), 0);
            if (other > goal) goal = other;
          }
          if (issued == goal) break;
        }
        if (elect_one()) {
          const uint32_t bar = in_first<kCtas>(&full[s]);
          if (rank == 0) mbar_expect_tx(&full[s], kCtas * (G::kABytes + boxes * G::kBox * kRowBytes));
          tma_load_2d<kCtas>(smem_u32(sA) + s * G::kABytes, &wmap, bar, k * kRowBytes, wrow);
          for (int i = 0; i < boxes; ++i)
            tma_load_2d<kCtas>(smem_u32(sB) + s * G::kBBytes + i * G::kBox * kRowBytes, &xmap, bar, k * kRowBytes,
                               brow + i * G::kBox);
        }
        __syncwarp();
        ++issued;
        if (++s == G::kStages) s = 0;
        if (++back == G::kScaleStages) {
          back = 0;
          phase ^= 1;
        }
      }
    }
    // every stage given back: no arrival is left on its way to this CTA's barriers
    for (uint32_t i = issued > G::kScaleStages ? issued - G::kScaleStages : 0; ok && i < issued; ++i)
      ok = __all_sync(0xffffffffu, wait(&empty[i % G::kScaleStages], (i / G::kScaleStages) & 1, &s_abort, a.glob));
    if (kCtas == 2 && goal == ~0u && lane == 0) tell_pair(&s_told, rank, issued);
  } else if (w == 1 && rank == 0) {
    // Two stages a step with single CTAs, so that the watching, which costs as
    // much as issuing a stage's instructions, is shared (16 rows x 32 experts x
    // 4096 x 2048: 11.9 -> 10.7 us); one with pairs, whose instructions take
    // longer to run.  The lanes watch the stages' codes and scales at the same
    // time, and the next step's before this one's instructions are issued, so
    // that a wait that is over costs nothing.
    const uint32_t desc_a = desc_addr(smem_u32(sA)), desc_b = desc_addr(smem_u32(sB)), desc_s = desc_addr(smem_u32(sS));
    const int full_stages = (a.blocks + 1) / 8;   // stages of four instructions
    uint64_t* const watch = lane & 1 ? scaled : full;
    const bool scales = kCtas == 2 && (lane & 1);   // the lane watches another ring
    auto after = [](int s) { return s + 1 == G::kStages ? 0 : s + 1; };
    auto after_r = [](int r) { return r + 1 == G::kScaleStages ? 0 : r + 1; };
    int s = 0, r = 0, buf = 0, limit = a.first_wait;   // r: a pair's place in the scales' ring
    uint32_t phase = 0, phase_r = 0, acc_phase = 1;
    bool ok = true, ready = false;
    for (; ok && walk.at(s_begin, s_tiles, a.experts, kTN, &row0, &count); walk.next(out_tiles)) {
      const int n = (count + G::kRound - 1) / G::kRound * G::kRound;
      const uint32_t id0 = instr_desc(G::kOuts, n, 0), id2 = instr_desc(G::kOuts, n, 2);
      ok = __all_sync(0xffffffffu, wait(&acc_empty[buf], acc_phase, &s_abort, a.glob));
      if (!ok) break;
      tc_fence_after();
      const uint32_t d = tmem + buf * G::kAccCols;
      // a stage's scales to its columns, then its instructions (by one thread)
      auto multiply = [&](int s, int r, int k) {
        const uint32_t ta = tmem_scales + s * G::kScaleCols, tb = ta + 8;
        const uint64_t ds = kScaleDesc + (desc_s + (kCtas == 2 ? r : s) * (G::kScaleBytes >> 4));
        const uint64_t da = kOperandDesc + (desc_a + s * (G::kABytes >> 4));
        const uint64_t db = kOperandDesc + (desc_b + s * (G::kBBytes >> 4));
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          tc_copy_scales<kCtas>(ta + 4 * q, ds + q * (kScaleTile >> 4));
#pragma unroll
          for (int j = 0; j < G::kScaleB; ++j)
            tc_copy_scales<kCtas>(tb + 4 * (q * G::kScaleB + j), ds + (2 + q * G::kScaleB + j) * (kScaleTile >> 4));
        }
        const int left = k < full_stages ? 8 : a.blocks - k * 8;   // scale blocks from here on
        tc_mma<kCtas>(d, da, db, id0, ta, tb, k > k0);
#pragma unroll
        for (int q = 1; q < 4; ++q)
          if (2 * q < left)
            tc_mma<kCtas>(d, da + 2 * q, db + 2 * q, q & 1 ? id2 : id0, ta + 4 * (q >> 1),
                          tb + 4 * G::kScaleB * (q >> 1), 1);
        tc_commit<kCtas>(&empty[kCtas == 2 ? r : s]);
      };
      for (int k = k0; k < k1;) {
        const bool two = kCtas == 1 && k + 1 < k1;
        const int s1 = after(s), r1 = after_r(r);
        const uint32_t phase1 = phase ^ (s1 == 0), phase_r1 = phase_r ^ (r1 == 0);
        if (!ready) {
          const bool second = two && (lane & 2);
          ok = __all_sync(0xffffffffu,
                          wait<kCtas>(&watch[scales ? r : second ? s1 : s], scales ? phase_r : second ? phase1 : phase,
                                      &s_abort, a.glob, limit));
          if (!ok) break;
        }
        limit = kWaitLimit;
        tc_fence_after();
        const int s2 = two ? after(s1) : s1, s3 = after(s2);
        const uint32_t phase2 = two ? phase1 ^ (s2 == 0) : phase1, phase3 = phase2 ^ (s3 == 0);
        const int next = kCtas == 2 ? (scales ? r1 : s1) : lane & 2 ? s3 : s2;
        const uint32_t next_phase = kCtas == 2 ? (scales ? phase_r1 : phase1) : lane & 2 ? phase3 : phase2;
        const bool over = mbar_test<kCtas>(&watch[next], next_phase);
        if (elect_one()) {
          multiply(s, r, k);
          if (two) multiply(s1, 0, k + 1);
          if (k + 1 + two >= k1) tc_commit<kCtas>(&acc_full[buf]);
        }
        ready = __all_sync(0xffffffffu, over);
        k += 1 + two;
        s = s2;
        phase = phase2;
        r = r1;
        phase_r = phase_r1;
      }
      if (++buf == G::kAcc) {
        buf = 0;
        acc_phase ^= 1;
      }
    }
  } else if (w == 1) {
    // A pair's second CTA: announces to the first the stages whose scales are
    // laid out, as many as there are at a time.  What the scale warps stored is
    // ordinary memory of this CTA: to be known in the other it has to be released
    // to the cluster, and a warp of its own does that, so that the next scales
    // are read and laid out meanwhile.  (Released by the scale warps, 8192 x 8192
    // takes 457 us, by three of them 352; single CTAs without any of this 484.)
    uint32_t n = 0;   // stages announced
    bool ok = true;
    for (; ok && walk.at(s_begin, s_tiles, a.experts, kTN, &row0, &count); walk.next(out_tiles)) {
      for (int left = k1 - k0; left > 0;) {
        ok = __all_sync(0xffffffffu, wait(&laid[n % G::kScaleStages], (n / G::kScaleStages) & 1, &s_abort, a.glob));
        if (!ok) break;
        int more = 1;
        while (more < left && more < G::kScaleStages &&
               __all_sync(0xffffffffu, mbar_test(&laid[(n + more) % G::kScaleStages], ((n + more) / G::kScaleStages) & 1)))
          ++more;
        if (lane == 0) {
          mbar_arrive_cluster(in_first<kCtas>(&scaled[n % G::kScaleStages]));
          for (int i = 1; i < more; ++i) mbar_arrive_after(in_first<kCtas>(&scaled[(n + i) % G::kScaleStages]));
        }
        __syncwarp();
        n += more;
        left -= more;
      }
    }
  } else if (w < kStoreWarp0) {
    // A warp takes every other group of 512 values (two stages), 16 scale bytes
    // a row.  A lane has rows lane, + 32, + 64 and + 96 of each 128, whose words
    // stand next to each other: one 16-byte store for 4 blocks of 4 rows.  The
    // loads of a group are over before its fence, which would wait for them.
    const int64_t weights = (int64_t)a.experts * a.outs;
    const uint32_t one = 0x7F7F7F7Fu;
    uint32_t before = 0, turn = w - kScaleWarp0;   // stages of the tiles before; groups until the warp's next
    bool ok = true;
    for (; ok && walk.at(s_begin, s_tiles, a.experts, kTN, &row0, &count); walk.next(out_tiles)) {
      constexpr int kTiles = 1 + G::kScaleB;
      const uint8_t* src[kTiles][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t wr = walk.e * a.outs + walk.out * G::kOuts + rank * kM + j * 32 + lane;
        src[0][j] = wr < weights ? a.ws + wr * a.scale_bytes : nullptr;
#pragma unroll
        for (int i = 1; i < kTiles; ++i) {
          const int r = (i - 1) * 128 + j * 32 + lane;
          src[i][j] = r < count ? a.xs + ((int64_t)row0 + r) * a.scale_bytes : nullptr;
        }
      }
      int g = turn;
      for (; ok && g < group1 - group0; g += kScaleWarps) {
        const int at = group0 + g;
        uint32_t word[kTiles][4][4];
#pragma unroll
        for (int i = 0; i < kTiles; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint4 v = make_uint4(one, one, one, one);
            if (src[i][j]) v = reinterpret_cast<const uint4*>(src[i][j])[at];
            word[i][j][0] = v.x;
            word[i][j][1] = v.y;
            word[i][j][2] = v.z;
            word[i][j][3] = v.w;
          }
        if (at == groups - 1) {   // blocks past the row's end
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int left = a.blocks - (at * 16 + q * 4);
            const uint32_t keep = left >= 4 ? ~0u : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
#pragma unroll
            for (int i = 0; i < kTiles; ++i)
#pragma unroll
              for (int j = 0; j < 4; ++j) word[i][j][q] = (word[i][j][q] & keep) | (one & ~keep);
          }
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (2 * at + half >= stages) break;
          const uint32_t n = before + 2 * g + half;
          const int s = n % G::kScaleStages;
          ok = __all_sync(0xffffffffu, wait(&empty[s], ((n / G::kScaleStages) & 1) ^ 1, &s_abort, a.glob));
          if (!ok) break;
          uint8_t* sc = sS + s * G::kScaleBytes + lane * 16;
#pragma unroll
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int i = 0; i < kTiles; ++i)
              *reinterpret_cast<uint4*>(sc + (i == 0 ? q : 2 + q * G::kScaleB + i - 1) * kScaleTile) =
                  make_uint4(word[i][0][2 * half + q], word[i][1][2 * half + q], word[i][2][2 * half + q],
                             word[i][3][2 * half + q]);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive<1>(smem_u32(rank == 1 ? &laid[s] : &scaled[s]));
        }
      }
      turn = g - (group1 - group0);
      before += k1 - k0;
    }
  } else {
    // a warp has the outputs of its quarter of the lanes, and every other run of 16 rows
    const int quarter = w & 3, odd = (w - kStoreWarp0) >> 2;
    int buf = 0;
    uint32_t phase = 0;
    for (; walk.at(s_begin, s_tiles, a.experts, kTN, &row0, &count); walk.next(out_tiles)) {
      if (!__all_sync(0xffffffffu, wait(&acc_full[buf], phase, &s_abort, a.glob))) break;
      tc_fence_after();
      const int64_t out = (int64_t)walk.out * G::kOuts + rank * kM + quarter * 32;
      const bool mine = out + lane < a.outs;
      const uint32_t d = tmem + buf * G::kAccCols + ((uint32_t)(quarter * 32) << 16);
      const int64_t at = (int64_t)row0 * a.outs + out;
      if (G::kShares && split > 1) {
        // the sums of the CTA's share, [row][output], where the stages were
        float* sums = reinterpret_cast<float*>(base) + quarter * 32 + lane;
        for (int c0 = odd * kStoreRows; c0 < count; c0 += 2 * kStoreRows) {
          uint32_t v[16];
          tc_load16(d + c0, v);
          tc_load_wait();
#pragma unroll
          for (int c = 0; c < 16; ++c) sums[(c0 + c) * kM] = __uint_as_float(v[c]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive<kCtas>(in_first<kCtas>(&acc_empty[buf]));
      } else if (a.out_type != EBC_F32) {
        store_tile<kTN, kCtas>(d, a.out_type == EBC_BF16, (uint16_t*)a.ys + at, a.outs, mine, odd, count, lane,
                               in_first<kCtas>(&acc_empty[buf]));
      } else {
        for (int c0 = odd * kStoreRows; c0 < count; c0 += 2 * kStoreRows)
          store_full(d + c0, (float*)a.ys + at + c0 * a.outs, a.outs, mine, count - c0, lane);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive<kCtas>(in_first<kCtas>(&acc_empty[buf]));
      }
      if (++buf == G::kAcc) {
        buf = 0;
        phase ^= 1;
      }
    }
    // rows that no expert has
    const int es = a.out_type == EBC_F32 ? 4 : 2;
    const int64_t words = (a.rows - s_begin[a.experts]) * a.outs;
    uint8_t* y0 = (uint8_t*)a.ys + (int64_t)s_begin[a.experts] * a.outs * es;
    for (int64_t i = (int64_t)blockIdx.x * (32 * kStoreWarps) + (tid - 32 * kStoreWarp0); i < words;
         i += (int64_t)gridDim.x * (32 * kStoreWarps)) {
      if (es == 4)
        reinterpret_cast<uint32_t*>(y0)[i] = 0u;
      else
        reinterpret_cast<uint16_t*>(y0)[i] = 0;
    }
  }

  tc_fence_before();
  bool gave_up = __syncthreads_or(s_abort) != 0;   // the same for all threads: another CTA may set it now
  if constexpr (kCtas == 2) {
    cluster_sync();   // no wait of the pair is left: the same for both CTAs
    gave_up = *const_cast<volatile int*>(&s_abort) != 0;
  }
  tc_fence_after();
  if (gave_up) {
    // nothing that was started may outlive the CTA (a pair's copies are counted
    // at its first CTA, its instructions' ends at both)
    if (rank == 0 && w == 0) {
      for (uint32_t i = issued > G::kStages ? issued - G::kStages : 0; i < issued; ++i)
        drain(&full[i % G::kStages], (i / G::kStages) & 1);
    }
    if (w == 1) {
      if (rank == 0 && elect_one()) tc_commit<kCtas>(&drained);
      __syncwarp();
      drain(&drained, 0);
    }
    __syncthreads();
  }
  if (G::kShares && split > 1) {
    cluster_sync();   // every CTA's sums are there
    Walk tile = start;
    if (tile.at(s_begin, s_tiles, a.experts, kTN, &row0, &count)) {
      const int out0 = tile.out * kM, n_out = a.outs - out0 < kM ? (int)(a.outs - out0) : kM;
      for (int i = tid; i < ((count - part + split - 1) >> shift) * kM; i += kThreads) {
        const int c = i / kM * split + part, n = i % kM;
        if (n >= n_out) continue;
        float sum = 0.f;
        for (int q = 0; q < split; ++q) {
          uint32_t from = smem_u32(base) + (c * kM + n) * 4;
          float v;
          asm volatile("mapa.shared::cluster.u32 %1, %1, %2;\n ld.shared::cluster.f32 %0, [%1];"
                       : "=f"(v), "+r"(from)
                       : "r"(q)
                       : "memory");
          sum += v;
        }
        const int64_t at = ((int64_t)row0 + c) * a.outs + out0 + n;
        if (a.out_type == EBC_BF16)
          ((__nv_bfloat16*)a.ys)[at] = from_f32<__nv_bfloat16>(sum);
        else if (a.out_type == EBC_F16)
          ((__half*)a.ys)[at] = from_f32<__half>(sum);
        else
          ((float*)a.ys)[at] = sum;
      }
    }
    __syncthreads();
    cluster_sync();   // and have been read
  }
  if (kCtas == 2) cluster_sync();   // neither CTA reads the other's memory any more
  if (w == 1) tc_free<kCtas>(tmem, G::kCols);
}

bool aligned(const void* p, int bytes) { return ((uintptr_t)p & (uintptr_t)(bytes - 1)) == 0; }

// codes [rows][code_bytes] in boxes of 128 bytes x box_rows
cudaError_t make_map(CUtensorMap* map, const uint8_t* codes, int64_t rows, int64_t code_bytes, int box_rows) {
  // found once, whichever host thread comes first
  static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
    cudaDriverEntryPointQueryResult q;
    void* fn = nullptr;
    const bool found = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                                        &q) == cudaSuccess && q == cudaDriverEntryPointSuccess;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(found ? fn : nullptr);
  }();
  if (!encode) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {(cuuint64_t)code_bytes, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)code_bytes};
  const cuuint32_t box[2] = {(cuuint32_t)kRowBytes, (cuuint32_t)box_rows};
  const cuuint32_t estr[2] = {1u, 1u};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(codes), dims, strides, box,
                            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int kTN, int kCtas>
cudaError_t product_t(const CallView& v, const uint8_t* xc, const uint8_t* wc, int64_t width, Args a,
                      cudaStream_t st) {
  using G = Geom<kTN, kCtas>;
  CUtensorMap wmap, xmap;
  const int64_t cb = EBC_MX4_CODE_BYTES(width);
  cudaError_t e = make_map(&wmap, wc, a.experts * a.outs, cb, kM);
  if (e == cudaSuccess) e = make_map(&xmap, xc, a.rows, cb, G::kBox);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(k_mx4_product<kTN, kCtas>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)G::kSmem);
  if (e != cudaSuccess) return e;
  const int64_t most = (a.rows / kTN + (a.experts < a.rows ? a.experts : a.rows)) *
                       ((a.outs + G::kOuts - 1) / G::kOuts), ctas = v.nsm / kCtas;
  // Share a tile's K among up to eight CTAs where all tiles still run at once
  // (a cluster's SMs come from one of the device's eight parts, each of which
  // may have up to split - 1 too few for another): one row x 1024 outputs x
  // 16384 takes 17.3 us in 8 CTAs and 8.2 in 64.
  int split = 1;
  a.split_log2 = 0;
  if (G::kShares)
    while (split < 8 && most * split * 2 <= v.nsm - 8 * (split * 2 - 1) && split * 2 <= (a.blocks + 15) / 16) {
      split *= 2;
      ++a.split_log2;
    }
  const unsigned cluster = kCtas * split;
  return launch_named(v, "k_mx4_product", st, k_mx4_product<kTN, kCtas>,
                      dim3((unsigned)(most < ctas ? most : ctas) * cluster), dim3(kThreads), G::kSmem, cluster, wmap,
                      xmap, a);
}

// The rows of a tile: what takes the fewest cycles, and the smaller of two that
// take as many.  Cycles are turns of the machine times a tile's: 450 a stage
// with single CTAs whatever the rows (the instructions take that to issue, less
// to run) and 550 with pairs, and about 2000 a tile for the results with single
// CTAs, 3800 with pairs, which have one accumulator.
// us with 16 / 32 / 64 / 128 / 256 rows a tile (the chosen one in brackets):
//      16 rows x 32 experts x 4096 x 2048   [10.4] 10.6  12.4  12.7   15.3
//     256 rows x  1 expert  x 4096 x 4096    18.9  11.7  [8.2]  9.2   13.5
//    2048 rows x 32 experts x 2048 x 2048    39.5  25.8  19.0 [15.4]  19.8
//    2228 rows x  5 experts x 2541 x  192    14.9  10.3   8.3  [8.8]  11.7
//   16384 rows x 32 experts x 4096 x 4096   841   463   240   155   [120]
int tile_rows(int64_t rows, int64_t outs, int64_t stages, int experts, int nsm) {
  const int64_t active = experts < rows ? experts : rows;
  int best = 16;
  int64_t least = INT64_MAX;
  for (int tn = 16; tn <= 256; tn *= 2) {
    const bool pair = tn == 256;
    const int64_t wide = pair ? 2 * kM : kM, units = pair ? nsm / 2 : nsm;
    // each expert's last run is half full on average, and a run at least
    const int64_t runs = rows / tn + active / 2 > active ? rows / tn + active / 2 : active;
    const int64_t turns = (runs * ((outs + wide - 1) / wide) + units - 1) / units;
    const int64_t cycles = turns * (pair ? 550 * stages + 3800 : 450 * stages + 2000);
    if (cycles < least) {
      least = cycles;
      best = tn;
    }
  }
  return best;
}

}  // namespace

extern "C" {

int ebc_mx4_product(ebc_ctx* ctx, const uint8_t* d_x_codes, const uint8_t* d_x_scales, int64_t rows, int64_t width,
                    const uint8_t* d_w_codes, const uint8_t* d_w_scales, int64_t outs, int n_experts,
                    const int32_t* d_offsets, int out_type, void* d_ys, void* stream) {
  const int b = type_bytes(out_type);
  // a tile that starts at the last row, or at the last output, still ends inside 31 bits
  constexpr int64_t kMost = (1ll << 31) - 256;
  if (!ctx || !b || rows < 0 || rows > kMost || width < 1 || width > (1 << 24) || outs < 1 || n_experts < 1 ||
      n_experts > EBC_MAX_EXPERTS || outs > kMost / n_experts || (!d_offsets && n_experts != 1) ||
      !aligned(d_offsets, 4))
    return EBC_ERR_INVALID_ARG;
  if (rows > 0 && (!d_x_codes || !aligned(d_x_codes, 16) || !d_x_scales || !aligned(d_x_scales, 16) || !d_w_codes ||
                   !aligned(d_w_codes, 16) || !d_w_scales || !aligned(d_w_scales, 16) || !d_ys || !aligned(d_ys, b)))
    return EBC_ERR_INVALID_ARG;
  CallView v;
  cudaStream_t st = (cudaStream_t)stream;
  const int rc = begin_call(ctx, st, &v);
  if (rc || rows == 0) return rc;
  Args a;
  a.xs = d_x_scales;
  a.ws = d_w_scales;
  a.offsets = d_offsets;
  a.ys = d_ys;
  a.glob = v.glob;
  a.rows = rows;
  a.outs = outs;
  a.scale_bytes = EBC_MX4_SCALE_BYTES(width);
  a.out_type = out_type;
  a.blocks = (int)((width + EBC_MX4_BLOCK - 1) / EBC_MX4_BLOCK);
  a.experts = n_experts;
  a.first_wait = v.first_wait;
  switch (tile_rows(rows, outs, (width + kStageK - 1) / kStageK, n_experts, v.nsm)) {
    case 16: return cuda_code(product_t<16, 1>(v, d_x_codes, d_w_codes, width, a, st));
    case 32: return cuda_code(product_t<32, 1>(v, d_x_codes, d_w_codes, width, a, st));
    case 64: return cuda_code(product_t<64, 1>(v, d_x_codes, d_w_codes, width, a, st));
    case 128: return cuda_code(product_t<128, 1>(v, d_x_codes, d_w_codes, width, a, st));
    default: return cuda_code(product_t<256, 2>(v, d_x_codes, d_w_codes, width, a, st));
  }
}

}  // extern "C"

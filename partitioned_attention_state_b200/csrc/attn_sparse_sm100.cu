// attn_sparse_sm100.cu -- attention of 128-row query blocks over lists of key
// blocks, for sm_100a (TMA + tcgen05 + TMEM).
//
//   S = Q K_list^T, P = exp2(S log2(e)/sqrt(D) - m), O = P V_list / l, L = ln2 (m + log2 l)
//
// with the running row maximum m and sum l of an online softmax over the list's
// 128-key tiles.  A tile is one listed block of 128 keys or two of 64, each
// fetched by its own TMA boxes of 64 rows, so the list costs the tile nothing:
// in shared memory the two halves lie where the halves of a contiguous tile
// would.  Rows past the last key are zero-filled by TMA and their logits set to
// -infinity; the second half of an odd list's last tile is left out of P V
// altogether, since shared memory there holds earlier keys.
//
// A work item is (head, query block), and the grid has a CTA per item.  With
// more items than SMs, a running CTA takes further items over from CTAs
// that have not started (cluster launch control), a few tiles ahead of its need: the
// lists may have any lengths, and this balances them without a counter in
// memory, keeps the items head-major, so that CTAs that run together read one
// head's K and V through L2, and overlaps one item's end with the next one's
// start.  With at most half as many, the `split` CTAs of a cluster take an equal
// run of the list's tiles each and join their states (m, l, unnormalised O) through
// distributed shared memory.
//
// Per CTA, 16 warps (4 warpgroups, registers rebalanced with setmaxnreg):
//   warps 0-7   softmax: two sets of four warps that take alternate tiles, a row
//               per thread; P is written back over S in TMEM as 16-bit values.
//               One set's exponentials (1,024 clk of the exponential unit per
//               tile) run while the other hands its tile on, loads the next S and
//               takes its maxima.  Both scale by one reference maximum per row,
//               handed from set to set in shared memory, so that O stays a single
//               accumulator; a row's sum is kept by each set and added at the end
//   warps 8-11  epilogue, under the next item's tiles: O (TMEM) normalised and
//               rounded into the item's own Q buffer, whence TMA stores it.  A
//               row per lane stored straight to memory put 32 sectors in 32
//               lines into every instruction and held up the SM's load/store
//               unit, which the softmax needs, for 2,000 clk per item
//   warp 12     tcgen05.mma S = Q K^T; TMEM alloc/free
//   warp 13     TMA: Q (two buffers), the K ring and the V ring
//   warp 14     scheduler: the next item, its list's length, and which of its
//               tiles need a mask, published to the other roles in shared memory
//   warp 15     tcgen05.mma O += P V (a second issuing thread: one thread
//               issues an MMA only every ~50 clk)
// Tensor memory: three S/P buffers [0,384), O [384,384+DP).
//
// P is rounded to the 16-bit type of V for the tensor cores (by at most 2^-8 of
// a weight in bf16, 2^-11 in fp16, with signs that average out over a row's keys);
// sums, maxima and O stay in fp32, and l sums the unrounded weights.  In fp16 the
// weights are scaled by 2^7, as far as the range allows with a reference that lags
// by 2^8: unscaled, weights below 2^-25 of the row's heaviest rounded to nothing,
// and with them up to 2^-25 of O per key of a long list.
//
// Every wait is bounded; one that runs out raises an abort flag shared by all
// roles and writes DT_ERR_TIMEOUT to *status, and every role drains its
// in-flight work before the CTA frees its tensor memory and exits.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/dt.h"
#include "attn_sparse.h"
#include "geometry.h"
#include "sm100_more.cuh"

namespace dt {
namespace {

using namespace sm100;

constexpr int kThreads = 512;
constexpr int kWarpEpi = 8, kWarpMma = 12, kWarpTma = 13, kWarpSched = 14, kWarpMmaPV = 15;
// Registers per thread at launch (the build checks that ptxas chose them) and
// the per-warpgroup split, which must fit the launch pool.
constexpr int kLaunchRegs = 128;
constexpr int kRegsSoftmax = 192, kRegsEpilogue = 80, kRegsOther = 48;
static_assert(128 * (2 * kRegsSoftmax + kRegsEpilogue + kRegsOther) <= kThreads * kLaunchRegs, "register split");
constexpr uint64_t kDrainLimitNs = 1000000000ull;
constexpr int kMaxDevices = 64;
constexpr int kMaxSplit = 16;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kLead = 8;                    // tiles of an item left to load when the next item is taken
constexpr float kRescaleThreshold = 8.0f;   // log2 units: rescale O only when the max grows by > 2^8
// log2 of the scale of P: the reference maximum stands this far below the row's.  2^(7 + 8) is in fp16's range; bf16
// has the exponents of fp32.
template <bool F16>
constexpr float kLift = F16 ? 7.0f : 0.0f;

__device__ __forceinline__ float neg_inf() { return -__int_as_float(0x7f800000); }
__device__ __forceinline__ float u2f(uint32_t u) { return __uint_as_float(u); }
__device__ __forceinline__ uint32_t f2u(float f) { return __float_as_uint(f); }

template <int DP>
struct Cfg {
  static constexpr int kN64 = DP / 64;                 // 64-column SW128 blocks
  static constexpr int kTail = (DP % 64) ? 1 : 0;      // one 16-column SW32 block
  static_assert(DP % 64 == 0 || DP % 64 == 16, "padded head dim must be 64k or 64k+16");
  static constexpr int kBlk = 128 * 64 * 2;            // bytes of a 128x64 16-bit block
  static constexpr int kTailBytes = 128 * 16 * 2;
  static constexpr int kTileBytes = kN64 * kBlk + kTail * kTailBytes;   // = 128 * DP * 2
  static constexpr int kNQ = 2;                        // Q buffers: the next item's Q loads under this one
  static constexpr int kNK = DP == 128 ? 2 : (DP == 80 ? 4 : 5);
  static constexpr int kNV = DP == 128 ? 3 : (DP == 80 ? 5 : 6);
  static constexpr int kNS = 3;                        // S/P buffers in tensor memory
  static constexpr int kColS = 0;
  static constexpr int kColO = 128 * kNS;
  static_assert(kColO + DP <= 512, "tensor memory budget");
  static constexpr int bQFull = 0, bQEmpty = bQFull + kNQ, bKFull = bQEmpty + kNQ, bVFull = bKFull + kNK,
                       bKEmpty = bVFull + kNV, bVEmpty = bKEmpty + kNK, bSFull = bVEmpty + kNV,
                       bPFull = bSFull + kNS, bPVDone = bPFull + kNS, bOFull = bPVDone + kNS, bOFree = bOFull + 1,
                       bStFull = bOFree + 1, bStFree = bStFull + 1, bTok = bStFree + 1, bInfoFull = bTok + 8,
                       bInfoFree = bInfoFull + 2, bNeed = bInfoFree + 2, bClc = bNeed + 1, bDrain = bClc + 1,
                       bDrainPV = bDrain + 1,
                       kNumBars = bDrainPV + 1 + (bDrainPV & 1 ? 0 : 1);      // even: what follows is 16-byte aligned
  // Arrivals that complete a phase.  Where a role of whole warps arrives, each of its threads does (no single-lane
  // branches); the rest are tensor-core commits and TMA's expected bytes.
  static __device__ __forceinline__ int arrivals(int i) {
    if (i >= bPFull && i < bPFull + kNS) return 4 * 32;            // a softmax set
    if (i >= bTok && i < bTok + 8) return 32;                      // a warp of it
    if (i == bStFull) return 8 * 32;
    if (i == bStFree || i == bOFree) return 4 * 32;                // the epilogue
    // a Q buffer is free when its last Q K^T is done and the 4 epilogue warps have stored O from it
    if (i >= bQEmpty && i < bQEmpty + kNQ) return 1 + 4;
    if (i == bNeed) return 32;                                     // the TMA warp
    // readers of an item: TMA and two MMA warps, softmax, epilogue
    if (i >= bInfoFree && i < bInfoFree + 2) return 3 * 32 + 8 * 32 + 4 * 32;
    return 1;
  }
  // per row: reference maximum, and each set's (maximum, sum) of the item
  static constexpr int kStatsBytes = 5 * 128 * 4;
  static constexpr int kSmem = kTileBytes * (kNQ + kNK + kNV) + kStatsBytes + kNumBars * 8 + 2 * 48 + 16 + 16;
  static_assert(kSmem <= 232448, "shared memory budget");
  // a split item's partial O ([128][DP] fp32) reuses the K ring, drained by then
  static_assert(kNK * kTileBytes >= 128 * DP * 4, "partial O fits the K ring");
};

// Bounded wait for a barrier's phase: one probe, then suspended waits of 200 us
// (under a shorter limit, probes) until the phase completes, another role aborts
// or the limit is over (recorded in *status, first error wins; then *abort is raised).
__device__ __forceinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile int* abort, int32_t* status,
                                       uint64_t limit) {
  const uint64_t t0 = globaltimer();
  while (true) {
    if (limit < 200000u ? mbar_test(bar, parity) : mbar_try_wait_hint(bar, parity, 200000u)) return true;
    if (*abort) return false;
    if (globaltimer() - t0 >= limit) {
      *abort = 1;
      atomicCAS(status, 0, DT_ERR_TIMEOUT);
      return false;
    }
  }
}
__device__ __forceinline__ bool thread_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int32_t* status,
                                            uint64_t limit) {
  return mbar_test(bar, parity) || wait_slow(bar, parity, abort, status, limit);
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int32_t* status,
                                          uint64_t limit) {
  return __all_sync(0xffffffffu, thread_wait(bar, parity, abort, status, limit));
}

template <bool F16>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  uint32_t r;
  if (F16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}

// kind::f16 instruction descriptor: the 16-bit format bits are 0 for f16, 1 for bf16
template <bool F16>
__host__ __device__ constexpr uint32_t idesc16(int M, int N, int b_mn) {
  const uint32_t d = idesc_bf16_f32(M, N, 0, b_mn);
  return F16 ? d & ~((1u << 7) | (1u << 10)) : d;
}

// One item, as the scheduler publishes it: entries [0, n) of list `item`, of
// which this CTA takes tiles [t0, t0 + nt); h < 0 ends the sequence.  Tiles from
// `masked` on may hold less than whole blocks (a short or bad one, or half a
// tile): the softmax looks at the entries of those alone.  first_a, first_b:
// the entries of tile t0.
struct __align__(16) Item { int h, q0, rows, item, n, t0, nt, masked, first_a, first_b, pad0, pad1; };
static_assert(sizeof(Item) == 48, "Item in shared memory");

// The entries of tile t of a list (b: -1 past its end).  Volatile, or the
// compiler moves a load that was issued a tile ahead down to the value's use.
__device__ __forceinline__ int ld_ahead(const int32_t* a) {
  int v;
  asm volatile("ld.global.nc.s32 %0, [%1];" : "=r"(v) : "l"(a));
  return v;
}
struct Entries { int a, b; };
__device__ __forceinline__ Entries load_entries(const SparseParams& p, const Item& it, int t) {
  Entries e = {-1, -1};
  const int i = t * p.per_tile;
  const int32_t* l = p.idx + (int64_t)it.item * p.cap + i;
  if (i < it.n) e.a = ld_ahead(l);
  if (p.per_tile == 2 && i + 1 < it.n) e.b = ld_ahead(l + 1);
  return e;
}
// First key rows of the two 64-row halves of tile t; Sk (nothing there) for an
// entry outside the sequence, -1 for the half that an odd list does not have.
struct Halves { int r0, r1; };
__device__ __forceinline__ Halves tile_halves(const SparseParams& p, const Item& it, int t, Entries e) {
  Halves v;
  if (p.per_tile == 1) {
    v.r0 = (unsigned)e.a < (unsigned)p.nkb ? e.a * 128 : p.Sk;
    v.r1 = v.r0 < p.Sk - 64 ? v.r0 + 64 : p.Sk;
  } else {
    v.r0 = (unsigned)e.a < (unsigned)p.nkb ? e.a * 64 : p.Sk;
    v.r1 = 2 * t + 1 >= it.n ? -1 : ((unsigned)e.b < (unsigned)p.nkb ? e.b * 64 : p.Sk);
  }
  return v;
}
// Item `item` (>= 0) for rank `rank` of its cluster, by all lanes of a warp:
// reads the whole list once, reports what is wrong with it.
__device__ __forceinline__ Item make_item(const SparseParams& p, int item, int rank, int lane) {
  Item it = {};
  it.item = item;
  it.h = (int)((unsigned)item / (unsigned)p.nqb);
  it.q0 = (item - it.h * p.nqb) * kTile;
  it.rows = imin(kTile, p.Sq - it.q0);
  const int32_t* list = p.idx + (int64_t)item * p.cap;
  const int count = p.count ? __ldg(p.count + item) : p.cap;
  it.n = imin(imax(count, 0), p.cap);
  const int nt = (it.n + p.per_tile - 1) / p.per_tile;
  it.t0 = (int)((int64_t)nt * rank / p.split);
  it.nt = (int)((int64_t)nt * (rank + 1) / p.split) - it.t0;
  const unsigned whole = (unsigned)p.Sk / (unsigned)(kTile / p.per_tile);     // blocks below this one are whole
  int at = p.per_tile == 2 && (it.n & 1) ? it.n - 1 : it.n;
  bool bad = count != it.n;
  for (int j = 0; j < it.n; j += 128) {
    int e[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) e[k] = j + 32 * k + lane < it.n ? __ldg(list + j + 32 * k + lane) : 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const bool in = j + 32 * k + lane < it.n;
      const uint32_t odd = __ballot_sync(0xffffffffu, in && (unsigned)e[k] >= whole);
      if (odd) at = imin(at, j + 32 * k + __ffs(odd) - 1);
      bad |= in && (unsigned)e[k] >= (unsigned)p.nkb;
    }
  }
  it.masked = at / p.per_tile;
  if (__any_sync(0xffffffffu, bad) && lane == 0 && rank == 0) atomicCAS(p.status, 0, DT_ERR_INVALID);
  const Entries f = load_entries(p, it, it.t0);
  it.first_a = f.a;
  it.first_b = f.b;
  return it;
}

// Cluster launch control: ask for a CTA of the grid that has not started, to be
// run here instead; the 16-byte answer lands in shared memory and completes on
// `bar`.  Returns its index, or -1 where none was left.
__device__ __forceinline__ void clc_ask(uint32_t answer, uint64_t* bar) {
  mbar_arrive_expect_tx(bar, 16);
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                   answer),
               "r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ int clc_answer(uint32_t answer) {
  uint32_t ok, x = 0;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 a;\n\t"
      "ld.shared.b128 a, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, a;\n\t}"
      : "=r"(ok), "=r"(x)
      : "r"(answer)
      : "memory");
  return ok ? (int)x : -1;
}

// Partial O of a split item in shared memory: row-major [128][DP] fp32, 16-byte
// chunks XOR-swizzled by (row & 7) inside each full group of 8 chunks, so that
// a warp writing one chunk of 32 rows hits every bank once per 8 lanes.
template <int DP>
__device__ __forceinline__ int part_chunk(int row, int cc) {
  return row * DP + 4 * (((cc | 7) < DP / 4) ? (cc ^ (row & 7)) : cc);
}

__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// shared::cluster address of this CTA's shared address `a` in CTA `rank`
__device__ __forceinline__ uint32_t map_rank(uint32_t a, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  return r;
}
__device__ __forceinline__ float ld_cluster(uint32_t a) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
  return v;
}

// Ties values loaded from tensor memory to the wait that precedes this: no use of theirs moves above it.
template <int N>
__device__ __forceinline__ void after_wait(uint32_t* r) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

// 8 columns of an output row
template <bool F16>
__device__ __forceinline__ void store_out8(const SparseParams& p, int64_t off, const float* x) {
  if (p.out_f32) {
    float* dst = static_cast<float*>(p.O) + off;
    *reinterpret_cast<float4*>(dst) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(dst + 4) = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.O) + off) =
        make_uint4(pack16<F16>(x[0], x[1]), pack16<F16>(x[2], x[3]), pack16<F16>(x[4], x[5]), pack16<F16>(x[6], x[7]));
  }
}

template <int DP, bool F16>
__global__ void __launch_bounds__(kThreads, 1) attn_block_sparse_kernel(const __grid_constant__ SparseParams p) {
  using C = Cfg<DP>;
  constexpr int D = DP == 80 ? 72 : DP;
  extern __shared__ __align__(1024) uint8_t smem[];
  // the swizzled layouts need 1024-byte alignment; the same in every CTA of a launch
  if (smem_u32(smem) & 1023u) {
    if (threadIdx.x == 0) atomicCAS(p.status, 0, DT_ERR_UNSUPPORTED);
    return;
  }
  uint8_t* sQ = smem;
  uint8_t* sK = sQ + C::kNQ * C::kTileBytes;
  uint8_t* sV = sK + C::kNK * C::kTileBytes;
  float* stat_m = reinterpret_cast<float*>(sV + C::kNV * C::kTileBytes);      // [2 sets][128]
  float* stat_l = stat_m + 256;                                              // [2 sets][128]
  float* s_ref = stat_l + 256;                                               // [128]
  uint64_t* bars = reinterpret_cast<uint64_t*>(s_ref + 128);
  Item* info = reinterpret_cast<Item*>(bars + C::kNumBars);                  // [2]
  uint32_t* clc = reinterpret_cast<uint32_t*>(info + 2);                     // [4]
  uint32_t* tmem_holder = clc + 4;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t lim = p.wait_limit_ns;
  const int rank = p.split > 1 ? (int)cluster_rank() : 0;

  // Unrolled, so that each count is a constant: 0.3 us of every call less than a
  // lane per barrier, whose counts are then computed (16 heads x 1,024 queries: 11.4, was 11.7 us).
  if (warp == kWarpTma && lane == 0) {
#pragma unroll
    for (int i = 0; i < C::kNumBars; ++i) mbar_init(&bars[i], C::arrivals(i));
    *abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async();
  }
  if (warp == kWarpMma) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  // The seq-th item for this role (warp-wide); false at the end or after an abort.
  auto next_item = [&](uint32_t seq, Item& it) {
    if (!warp_wait(&bars[C::bInfoFull + (seq & 1)], (seq >> 1) & 1, abort_flag, p.status, lim)) return false;
    it = info[seq & 1];
    mbar_arrive(&bars[C::bInfoFree + (seq & 1)]);
    return it.h >= 0;
  };

  if (warp >= kWarpMma) {
    regs_set<kLaunchRegs, kRegsOther>();
    if (warp == kWarpSched) {
      // ---------------------------------------------------------- scheduler
      // An item is taken when the TMA warp has kLead tiles of the one before left to issue: late enough that a CTA
      // hoards nothing (taken two items ahead, ragged lists of 3.5 items a CTA ended 20 % later), early enough for
      // the answer and the list's two memory latencies.
      const uint32_t answer = smem_u32(clc);
      int item = blockIdx.x / p.split;
      bool ok = true;
      for (uint32_t seq = 0; ok; ++seq) {
        if (seq > 0 && p.split > 1) item = -1;
        if (seq > 0 && p.split == 1) {
          ok = warp_wait(&bars[C::bNeed], (seq - 1) & 1, abort_flag, p.status, lim);
          if (!ok) break;
          if (lane == 0) clc_ask(answer, &bars[C::bClc]);
          __syncwarp();
          volatile int never = 0;                         // waited for whatever happens: the answer is in flight
          ok = warp_wait(&bars[C::bClc], (seq - 1) & 1, &never, p.status, kDrainLimitNs);
          if (!ok) break;
          item = clc_answer(answer);
          fence_proxy_async();                            // the answer is read before the next one overwrites it
        }
        Item it = {};
        it.h = -1;
        if (item >= 0) it = make_item(p, item, rank, lane);
        ok = seq < 2 || warp_wait(&bars[C::bInfoFree + (seq & 1)], ((seq >> 1) - 1) & 1, abort_flag, p.status, lim);
        if (!ok) break;
        if (lane == 0) {
          info[seq & 1] = it;
          mbar_arrive(&bars[C::bInfoFull + (seq & 1)]);
        }
        __syncwarp();
        if (it.h < 0) break;
      }
    } else if (warp == kWarpTma) {
      // ---------------------------------------------------------- TMA producer
      // Whole-warp loops with an elected lane for the copies, as in the MMA warps: issued by one lane of a divergent
      // loop, a tile's 8 copies took ~850 clk, and the loads ran no tile ahead of the tensor cores.
      if (elect_one()) {
        prefetch_tmap(&p.tmQ);
        prefetch_tmap(&p.tmK);
        prefetch_tmap(&p.tmV);
        if (C::kTail) {
          prefetch_tmap(&p.tmQt);
          prefetch_tmap(&p.tmKt);
          prefetch_tmap(&p.tmVt);
        }
      }
      __syncwarp();
      // K/V blocks are read by many query blocks of the head; a Q tile once
      const uint64_t pol_keep = l2_policy_evict_last(), pol_once = l2_policy_evict_first();
      uint32_t gk = 0, gv = 0, nq = 0;                    // K tiles, V tiles, Q tiles issued
      // 64 rows from row0 of a K, V or Q head, into half `half` of a tile
      auto load_half = [&](const CUtensorMap* t64, const CUtensorMap* t16, uint8_t* tile, uint64_t* bar, int half,
                           int row0, int h, uint64_t pol) {
#pragma unroll
        for (int c = 0; c < C::kN64; ++c)
          tma_load_3d_hint(tile + c * C::kBlk + half * (C::kBlk / 2), t64, bar, 64 * c, row0, h, pol);
        if (C::kTail)
          tma_load_3d_hint(tile + C::kN64 * C::kBlk + half * (C::kTailBytes / 2), t16, bar, 64 * C::kN64, row0, h, pol);
      };
      Halves vp = {0, 0};                                 // the tile whose V is still to be issued
      int vh = -1;
      auto issue_v = [&]() {
        if (vh < 0) return true;
        const uint32_t st = gv % C::kNV;
        if (gv >= (uint32_t)C::kNV && !warp_wait(&bars[C::bVEmpty + st], ((gv / C::kNV) - 1) & 1, abort_flag, p.status, lim))
          return false;
        if (elect_one()) {
          uint8_t* dst = sV + st * C::kTileBytes;
          uint64_t* full = &bars[C::bVFull + st];
          mbar_arrive_expect_tx(full, vp.r1 < 0 ? C::kTileBytes / 2 : C::kTileBytes);
          load_half(&p.tmV, &p.tmVt, dst, full, 0, vp.r0, vh, pol_keep);
          if (vp.r1 >= 0) load_half(&p.tmV, &p.tmVt, dst, full, 1, vp.r1, vh, pol_keep);
        }
        __syncwarp();
        vh = -1;
        ++gv;
        return true;
      };
      // V(g) goes out after K(g+1): the order in which their stages fall free
      bool ok = true;
      Item it;
      for (uint32_t seq = 0; ok; ++seq) {
        // the last V of an item goes first if the next item is not there yet
        if (!__all_sync(0xffffffffu, mbar_test(&bars[C::bInfoFull + (seq & 1)], (seq >> 1) & 1))) ok = issue_v();
        if (!ok || !next_item(seq, it)) break;
        if (it.nt <= kLead) mbar_arrive(&bars[C::bNeed]);
        if (it.nt == 0) continue;
        const uint32_t b = nq % C::kNQ;
        ok = nq < (uint32_t)C::kNQ ||
             warp_wait(&bars[C::bQEmpty + b], (nq / C::kNQ - 1) & 1, abort_flag, p.status, lim);
        if (!ok) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(&bars[C::bQFull + b], C::kTileBytes);
          load_half(&p.tmQ, &p.tmQt, sQ + b * C::kTileBytes, &bars[C::bQFull + b], 0, it.q0, it.h, pol_once);
          load_half(&p.tmQ, &p.tmQt, sQ + b * C::kTileBytes, &bars[C::bQFull + b], 1, it.q0 + 64, it.h, pol_once);
        }
        __syncwarp();
        ++nq;
        const int hk = (int)((unsigned)it.h / (unsigned)p.per_kv);
        Entries nxt = {it.first_a, it.first_b};
        for (int t = it.t0; ok && t < it.t0 + it.nt; ++t) {
          const Halves v = tile_halves(p, it, t, nxt);
          if (t + 1 < it.t0 + it.nt) nxt = load_entries(p, it, t + 1);
          const uint32_t st = gk % C::kNK;
          ok = gk < (uint32_t)C::kNK ||
               warp_wait(&bars[C::bKEmpty + st], ((gk / C::kNK) - 1) & 1, abort_flag, p.status, lim);
          if (!ok) break;
          if (elect_one()) {
            uint8_t* dst = sK + st * C::kTileBytes;
            uint64_t* full = &bars[C::bKFull + st];
            mbar_arrive_expect_tx(full, v.r1 < 0 ? C::kTileBytes / 2 : C::kTileBytes);
            load_half(&p.tmK, &p.tmKt, dst, full, 0, v.r0, hk, pol_keep);
            if (v.r1 >= 0) load_half(&p.tmK, &p.tmKt, dst, full, 1, v.r1, hk, pol_keep);
          }
          __syncwarp();
          ++gk;
          if (it.t0 + it.nt - t == kLead + 1) mbar_arrive(&bars[C::bNeed]);
          ok = issue_v();
          vp = v;
          vh = hk;
        }
      }
      if (ok) issue_v();
      // let every copy this warp started land before shared memory goes away
      volatile int never = 0;
      auto drain = [&](int bar, uint32_t stages, uint32_t n) {
        for (uint32_t s = 0; s < stages; ++s)
          if (s < n)                                      // the latest tile that used stage s
            warp_wait(&bars[bar + s], ((n - 1 - ((n - 1 - s) % stages)) / stages) & 1, &never, p.status, kDrainLimitNs);
      };
      drain(C::bKFull, C::kNK, gk);
      drain(C::bVFull, C::kNV, gv);
      drain(C::bQFull, C::kNQ, nq);
      __syncwarp();
    } else if (warp == kWarpMma) {
      // ---------------------------------------------------------- S = Q K^T
      // The MMA warps run their loops whole and elect a lane for each tile's
      // instructions, so that descriptors stay in uniform registers: issued by
      // one lane of a divergent loop an MMA took ~115 clk, and 8 of them nearly a
      // whole tile's time.
      constexpr uint32_t idesc = idesc16<F16>(128, 128, 0);
      const uint64_t qd0 = smem_desc(smem_u32(sQ), 16, 1024, kSwizzle128B);
      const uint64_t kd0 = smem_desc(smem_u32(sK), 16, 1024, kSwizzle128B);
      const uint64_t qt0 = smem_desc(smem_u32(sQ) + C::kN64 * C::kBlk, 16, 256, kSwizzle32B);
      const uint64_t kt0 = smem_desc(smem_u32(sK) + C::kN64 * C::kBlk, 16, 256, kSwizzle32B);
      uint32_t g = 0, nq = 0;
      bool ok = true;
      Item it;
      for (uint32_t seq = 0; ok && next_item(seq, it); ++seq) {
        if (it.nt == 0) continue;
        const uint32_t qb = nq % C::kNQ;
        ok = warp_wait(&bars[C::bQFull + qb], (nq / C::kNQ) & 1, abort_flag, p.status, lim);
        ++nq;
        for (int t = 0; t < it.nt && ok; ++t, ++g) {
          const uint32_t st = g % C::kNK, sb = g % C::kNS;
          // K has arrived, and S buffer sb, which held P(g-3), is free: its P V (issued by warp 15) is done
          ok = warp_wait(&bars[C::bKFull + st], (g / C::kNK) & 1, abort_flag, p.status, lim) &&
               (g < (uint32_t)C::kNS ||
                warp_wait(&bars[C::bPVDone + sb], (g / C::kNS - 1) & 1, abort_flag, p.status, lim));
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const uint32_t dS = tmem + C::kColS + sb * 128;
            const uint64_t qd = qd0 + qb * (C::kTileBytes >> 4), kd = kd0 + st * (C::kTileBytes >> 4);
#pragma unroll
            for (int blk = 0; blk < C::kN64; ++blk)
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)               // 16 head-dim columns (32 bytes of a row) per MMA
                mma_ss(dS, qd + (blk * C::kBlk + kk * 32 >> 4), kd + (blk * C::kBlk + kk * 32 >> 4), idesc,
                       blk + kk > 0 ? 1u : 0u);
            if (C::kTail)
              mma_ss(dS, qt0 + qb * (C::kTileBytes >> 4), kt0 + st * (C::kTileBytes >> 4), idesc, 1u);
            mma_commit(&bars[C::bSFull + sb]);
            mma_commit(&bars[C::bKEmpty + st]);
            if (t == it.nt - 1) mma_commit(&bars[C::bQEmpty + qb]);
          }
          __syncwarp();
        }
      }
      // all MMAs that this warp issued complete before tensor memory is freed
      if (elect_one()) {
        mma_commit(&bars[C::bDrain]);
        volatile int never = 0;
        thread_wait(&bars[C::bDrain], 0, &never, p.status, kDrainLimitNs);
      }
      __syncwarp();
    } else if (warp == kWarpMmaPV) {
      // ---------------------------------------------------------- O += P V
      constexpr uint32_t idesc_pv = idesc16<F16>(128, 64 * C::kN64, 1);
      constexpr uint32_t idesc_pvt = idesc16<F16>(128, 16, 1);
      const uint64_t vd0 = smem_desc(smem_u32(sV), C::kBlk, 1024, kSwizzle128B);
      const uint64_t vt0 = smem_desc(smem_u32(sV) + C::kN64 * C::kBlk, C::kTailBytes, 256, kSwizzle32B);
      uint32_t g = 0, nq = 0;
      bool ok = true;
      Item it;
      for (uint32_t seq = 0; ok && next_item(seq, it); ++seq) {
        if (it.nt == 0) continue;
        for (int t = 0; t < it.nt && ok; ++t, ++g) {
          const uint32_t sb = g % C::kNS, st = g % C::kNV;
          ok = warp_wait(&bars[C::bVFull + st], (g / C::kNV) & 1, abort_flag, p.status, lim) &&
               (t > 0 || nq == 0 || warp_wait(&bars[C::bOFree], (nq - 1) & 1, abort_flag, p.status, lim)) &&
               warp_wait(&bars[C::bPFull + sb], (g / C::kNS) & 1, abort_flag, p.status, lim);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const uint32_t aP = tmem + C::kColS + sb * 128;
            const uint64_t vd = vd0 + st * (C::kTileBytes >> 4), vdt = vt0 + st * (C::kTileBytes >> 4);
            const uint32_t acc = t > 0 ? 1u : 0u;
            // 16 keys per MMA: descriptors advance by 16 V rows
            auto pv = [&](int kk) {
              mma_ts(tmem + C::kColO, aP + 8 * kk, vd + kk * (2048 >> 4), idesc_pv, kk > 0 ? 1u : acc);
              if (C::kTail)
                mma_ts(tmem + C::kColO + 64 * C::kN64, aP + 8 * kk, vdt + kk * (512 >> 4), idesc_pvt, kk > 0 ? 1u : acc);
            };
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) pv(kk);
            if (p.per_tile == 1 || 2 * (it.t0 + t) + 1 < it.n) {      // a tile that holds one 64-key block ends here
#pragma unroll
              for (int kk = 4; kk < 8; ++kk) pv(kk);
            }
            mma_commit(&bars[C::bVEmpty + st]);
            mma_commit(&bars[C::bPVDone + sb]);
            if (t == it.nt - 1) mma_commit(&bars[C::bOFull]);
          }
          __syncwarp();
        }
        ++nq;
      }
      if (elect_one()) {
        mma_commit(&bars[C::bDrainPV]);
        volatile int never = 0;
        thread_wait(&bars[C::bDrainPV], 0, &never, p.status, kDrainLimitNs);
      }
      __syncwarp();
    }
    if (p.split > 1) cluster_sync_all();
  } else if (warp < kWarpEpi) {
    regs_set<kLaunchRegs, kRegsSoftmax>();
    // ------------------------------------------------------------ softmax
    // Set `set` takes the tiles g = set, set + 2, ... (counted over the CTA's
    // items); thread = tile row.  Tile g's reference maximum follows from tile
    // g-1's, which the other set's warp of the same rows hands over through
    // s_ref and the token barrier: the order of the tiles, and with it the
    // result, is that of one set.
    const int set = warp >> 2, pair = warp & 3;
    const int r = pair * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(pair * 32) << 16;
    const float sl2 = p.scale_log2;
    uint64_t* tok_in = &bars[C::bTok + 2 * pair + (set ^ 1)];
    uint64_t* tok_out = &bars[C::bTok + 2 * pair + set];
    uint32_t g0 = 0, nq = 0;                       // first tile of the item, items done
    Item it;
    for (uint32_t seq = 0; next_item(seq, it); ++seq) {
      const int nt = it.nt, masked = it.masked - it.t0;  // tiles from `masked` on may need a mask
      if (nt == 0) continue;
      const bool idle = pair * 32 >= it.rows;      // none of this warp's rows exist: hand the tiles on
      float m = neg_inf();                          // reference (log2 units) that l stands on
      uint64_t l2[4] = {0ull, 0ull, 0ull, 0ull};    // packed pairs of partial row sums
      for (int i = (g0 ^ set) & 1; i < nt; i += 2) {
        const uint32_t g = g0 + i, sb = g % C::kNS;
        if (!warp_wait(&bars[C::bSFull + sb], (g / C::kNS) & 1, abort_flag, p.status, lim)) goto sm_done;
        if (idle) {
          if (g > 0 && !warp_wait(tok_in, ((g - 1) >> 1) & 1, abort_flag, p.status, lim)) goto sm_done;
          mbar_arrive(tok_out);
          mbar_arrive(&bars[C::bPFull + sb]);
          continue;
        }
        tc_fence_after();
        const uint32_t sc = tmem + lane_base + C::kColS + sb * 128;
        uint32_t sr[128];
        tmem_ld32(sc, sr);
        tmem_ld32(sc + 32, sr + 32);
        // the reference after the previous tile: usually long there, so it is waited for under the loads
        if (g > 0 && !warp_wait(tok_in, ((g - 1) >> 1) & 1, abort_flag, p.status, lim)) goto sm_done;
        const float old = i == 0 ? neg_inf() : s_ref[r];
        tmem_wait_ld();
        after_wait<64>(sr);
        tmem_ld32(sc + 64, sr + 64);
        tmem_ld32(sc + 96, sr + 96);
        // maxima in four chains; the first half's under the second half's loads
        float x[4];
        auto chain = [&](int e0) {
#pragma unroll
          for (int e = e0; e < e0 + 64; e += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              x[k] = e == 0 ? fmaxf(u2f(sr[2 * k]), u2f(sr[2 * k + 1]))
                            : max3f(x[k], u2f(sr[e + 2 * k]), u2f(sr[e + 2 * k + 1]));
        };
        const bool mask = i >= masked;
        if (!mask) chain(0);
        tmem_wait_ld();
        after_wait<64>(sr + 64);
        if (mask) {
          const Halves hv = tile_halves(p, it, it.t0 + i, load_entries(p, it, it.t0 + i));
          const int v0 = p.Sk - hv.r0, v1 = hv.r1 < 0 ? 0 : p.Sk - hv.r1;    // keys of each half
          // assigned, not added: the logits there may be anything
#pragma unroll
          for (int e = 0; e < 128; ++e)
            if (!((e & 63) < (e < 64 ? v0 : v1))) sr[e] = f2u(neg_inf());
        }
        if (mask) chain(0);
        chain(64);
        const float top = fmaf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), sl2, -kLift<F16>);
        const float ref = i == 0 ? top : (top > old + kRescaleThreshold ? top : old);
        // a row that has seen only masked keys (reference -inf) has O = 0: it takes the new one without a rescale
        const bool res = ref != old && old != neg_inf();
        if (__any_sync(0xffffffffu, res)) {
          // O holds the previous tiles' sum: wait for its last P V, then rescale
          if (!warp_wait(&bars[C::bPVDone + (g - 1) % C::kNS], ((g - 1) / C::kNS) & 1, abort_flag, p.status, lim))
            goto sm_done;
          tc_fence_after();
          const float alpha = res ? ex2(old - ref) : 1.f;
          const uint32_t oc = tmem + lane_base + C::kColO;
#pragma unroll 1
          for (int c0 = 0; c0 < DP; c0 += 16) {
            uint32_t o[16];
            tmem_ld16(oc + c0, o);
            tmem_wait_ld();
            after_wait<16>(o);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = f2u(u2f(o[e]) * alpha);
            tmem_st16(oc + c0, o);
          }
          tmem_wait_st();
        }
        s_ref[r] = ref;
        mbar_arrive(tok_out);
        if (m != ref) {                             // l onto the new reference (0 while m is -inf)
          const float beta = ex2(m - ref);
          const uint64_t b2 = pk2(beta, beta);
#pragma unroll
          for (int k = 0; k < 4; ++k) l2[k] = mul2(l2[k], b2);
          m = ref;
        }
        const float mr = ref == neg_inf() ? 0.f : ref;
        const uint64_t sl2x2 = pk2(sl2, sl2), nm = pk2(-mr, -mr);
        // exponentials, 32 columns (16 P columns) per TMEM store
#pragma unroll
        for (int c = 0; c < 128; c += 32) {
          uint32_t ph[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float a, b;
            upk2(fma2(pk2(u2f(sr[c + e]), u2f(sr[c + e + 1])), sl2x2, nm), a, b);
            a = ex2(a);
            b = ex2(b);
            l2[(e >> 1) & 3] = add2(l2[(e >> 1) & 3], pk2(a, b));
            ph[e >> 1] = pack16<F16>(a, b);
          }
          tmem_st16(sc + c / 2, ph);
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&bars[C::bPFull + sb]);
      }
      float u0, u1;
      upk2(add2(add2(l2[0], l2[1]), add2(l2[2], l2[3])), u0, u1);
      if (nq >= 1 && !warp_wait(&bars[C::bStFree], (nq - 1) & 1, abort_flag, p.status, lim)) goto sm_done;
      stat_m[set * 128 + r] = m;
      stat_l[set * 128 + r] = u0 + u1;
      mbar_arrive(&bars[C::bStFull]);
      ++nq;
      g0 += nt;
    }
  sm_done:;
    __syncwarp();
    if (p.split > 1) cluster_sync_all();
  } else {
    regs_set<kLaunchRegs, kRegsEpilogue>();
    // ------------------------------------------------------------ epilogue
    const int r = (warp - kWarpEpi) * 32 + lane;          // tile row of this thread
    const uint32_t oaddr = tmem + (static_cast<uint32_t>((warp - kWarpEpi) * 32) << 16) + C::kColO;
    uint32_t nq = 0;
    Item it;
    for (uint32_t seq = 0; next_item(seq, it); ++seq) {
      const bool valid = r < it.rows;
      const int64_t orow = it.h * p.o_head + (int64_t)(it.q0 + r) * p.o_row;
      float* lrow = p.L + (int64_t)it.h * p.Sq + it.q0 + r;
      if (it.nt == 0) {
        if (p.split > 1) {                                // an empty state for the join
          stat_m[r] = neg_inf();
          stat_l[r] = 0.f;
        } else if (valid) {
          const float z[8] = {};
          for (int c = 0; c < D; c += 8) store_out8<F16>(p, orow + c, z);
          *lrow = neg_inf();
        }
        continue;
      }
      if (!warp_wait(&bars[C::bStFull], nq & 1, abort_flag, p.status, lim)) goto ep_done;
      // references only rise, so O stands on the higher of the sets'; a set that had no tile has (-inf, 0)
      const float ma = stat_m[r], mb = stat_m[128 + r], la = stat_l[r], lb = stat_l[128 + r];
      const float m = ma != ma || mb != mb ? ma + mb : fmaxf(ma, mb);
      const float l = (ma == m ? la : la * ex2(ma - m)) + (mb == m ? lb : lb * ex2(mb - m));
      if (p.split > 1) {
        stat_m[r] = m;
        stat_l[r] = l;
      }
      mbar_arrive(&bars[C::bStFree]);
      if (!warp_wait(&bars[C::bOFull], nq & 1, abort_flag, p.status, lim)) goto ep_done;
      tc_fence_after();
      // l > 0 unless every listed key is past the end or has a logit of -inf; NaN stays
      const float inv = l == 0.f ? 0.f : 1.f / l;
      float* part = reinterpret_cast<float*>(sK);
      // 16-bit rows in the layout of the TMA store's boxes: [64-column block][row], 16-byte chunks XOR-swizzled by
      // (row & 7); the 8 tail columns of D = 72 as plain 16-byte rows
      const bool pack = p.split == 1 && !p.out_f32;
      uint8_t* tile = sQ + (nq % C::kNQ) * C::kTileBytes;
      // Rolled loops, 16 columns a time: this code runs once an item, and unrolled its instruction misses held up
      // every warp of the SM for longer than the work takes (5,000 clk, against 2,000 here, at D = 128).
      auto load16 = [&](int c0, uint32_t (&op)[16]) {
        tmem_ld16(oaddr + c0, op);
        tmem_wait_ld();
        after_wait<16>(op);
        if (c0 + 16 >= DP) {
          tc_fence_before();
          mbar_arrive(&bars[C::bOFree]);                  // all of O is read: the next item's first P V may go
        }
      };
      if (pack) {
        const bool some = __any_sync(0xffffffffu, l == 0.f);
#pragma unroll 1
        for (int c0 = 0; c0 < DP; c0 += 16) {
          uint32_t op[16], pk[8];
          load16(c0, op);
          if (some && l == 0.f)
#pragma unroll
            for (int e = 0; e < 16; ++e) op[e] = 0u;
#pragma unroll
          for (int e = 0; e < 16; e += 2) pk[e / 2] = pack16<F16>(u2f(op[e]) * inv, u2f(op[e + 1]) * inv);
          uint8_t* at = tile + (c0 >> 6) * C::kBlk;
          if (c0 < 64 * C::kN64) {
            at += r * 128;
            const int ch = (c0 >> 3) & 7;
            *reinterpret_cast<uint4*>(at + ((ch ^ (r & 7)) << 4)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
            *reinterpret_cast<uint4*>(at + (((ch + 1) ^ (r & 7)) << 4)) = make_uint4(pk[4], pk[5], pk[6], pk[7]);
          } else {
            *reinterpret_cast<uint4*>(at + r * 16) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
          }
        }
      } else if (p.split > 1) {
        // (a warp without rows has nothing to hand over)
        constexpr int kStep = DP % 32 ? 16 : 32;
        if (r - lane < it.rows)
#pragma unroll 1
          for (int c0 = 0; c0 < DP; c0 += kStep) {
            uint32_t op[kStep];
#pragma unroll
            for (int c = 0; c < kStep; c += 16) tmem_ld16p(oaddr + c0 + c, op + c);
            tmem_wait_ld();
            after_wait<kStep>(op);
#pragma unroll
            for (int c = 0; c < kStep; c += 4)
              if (valid && c0 + c < D)
                *reinterpret_cast<float4*>(part + part_chunk<DP>(r, (c0 + c) / 4)) =
                    make_float4(u2f(op[c]), u2f(op[c + 1]), u2f(op[c + 2]), u2f(op[c + 3]));
          }
        tc_fence_before();
        mbar_arrive(&bars[C::bOFree]);
      } else {
#pragma unroll 1
        for (int c0 = 0; c0 < DP; c0 += 16) {
          uint32_t op[16];
          load16(c0, op);
#pragma unroll
          for (int c = 0; c < 16; c += 8) {
            if (c0 + c >= D) break;
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = l == 0.f ? 0.f : u2f(op[c + e]) * inv;
            if (valid) store_out8<F16>(p, orow + c0 + c, x);
          }
        }
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) {
        const int r0 = r;                                 // the warp's first row; rows past Sq are not written
        if (pack && r0 < it.rows) {
          for (int c = 0; c < C::kN64; ++c)
            tma_store_3d(&p.tmO, tile + c * C::kBlk + r0 * 128, 64 * c, it.q0 + r0, it.h);
          if (C::kTail) tma_store_3d(&p.tmOt, tile + C::kN64 * C::kBlk + r0 * 16, 64 * C::kN64, it.q0 + r0, it.h);
          bulk_commit();
          bulk_wait_read();
        }
        mbar_arrive(&bars[C::bQEmpty + nq % C::kNQ]);
      }
      __syncwarp();
      if (p.split == 1 && valid) *lrow = l == 0.f ? neg_inf() : (m + lg2(l)) * kLn2;
      ++nq;
    }
  ep_done:;
    __syncwarp();
    if (p.split > 1) {
      // Join of the cluster's states of its one item: M = max m_i, w_i =
      // 2^(m_i - M), O = sum w_i O_i / sum w_i l_i.  CTA `rank` joins 8-column
      // chunks rank, rank + split, ... of the item's rows.  Four CTAs' values are
      // loaded together: one by one their latencies were most of a short call's
      // end.  Every warp reaches both barriers whatever its role met before.
      cluster_sync_all();
      if (!*abort_flag) {
        const Item it0 = info[0];                         // the one item, untouched since
        const uint32_t a_m = smem_u32(stat_m), a_l = smem_u32(stat_l), a_o = smem_u32(sK);
        const int nchunk = it0.rows * (D / 8);
        // each CTA starts at its own state, so that they do not all read one CTA's at once
        auto peer = [&](int k) { return rank + k < p.split ? rank + k : rank + k - p.split; };
        for (int i = r * p.split + rank; i < nchunk; i += 128 * p.split) {
          const int row = i / (D / 8), c = 8 * (i - row * (D / 8));
          float M = neg_inf();
          for (int k0 = 0; k0 < p.split; k0 += 4) {
            float m[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              m[k] = neg_inf();
              if (k0 + k < p.split) m[k] = ld_cluster(map_rank(a_m + 4 * row, peer(k0 + k)));
            }
            M = fmaxf(M, fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])));
          }
          const float Mr = M == neg_inf() ? 0.f : M;
          float x[8] = {}, l = 0.f;
          for (int k0 = 0; k0 < p.split; k0 += 4) {
            float m[4], lk[4];
            float4 u[4], v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              lk[k] = 0.f;
              if (k0 + k >= p.split) continue;
              const int from = peer(k0 + k);
              m[k] = ld_cluster(map_rank(a_m + 4 * row, from));
              lk[k] = ld_cluster(map_rank(a_l + 4 * row, from));
              u[k] = ld_cluster4(map_rank(a_o + 4 * part_chunk<DP>(row, c / 4), from));
              v[k] = ld_cluster4(map_rank(a_o + 4 * part_chunk<DP>(row, c / 4 + 1), from));
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if (lk[k] == 0.f) continue;                 // an empty state's O was never written
              const float w = ex2(m[k] - Mr);
              l = fmaf(w, lk[k], l);
              x[0] = fmaf(w, u[k].x, x[0]); x[1] = fmaf(w, u[k].y, x[1]);
              x[2] = fmaf(w, u[k].z, x[2]); x[3] = fmaf(w, u[k].w, x[3]);
              x[4] = fmaf(w, v[k].x, x[4]); x[5] = fmaf(w, v[k].y, x[5]);
              x[6] = fmaf(w, v[k].z, x[6]); x[7] = fmaf(w, v[k].w, x[7]);
            }
          }
          const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] *= inv;
          store_out8<F16>(p, it0.h * p.o_head + (int64_t)(it0.q0 + row) * p.o_row + c, x);
          if (c == 0) p.L[(int64_t)it0.h * p.Sq + it0.q0 + row] = l == 0.f ? neg_inf() : (M + lg2(l)) * kLn2;
        }
      }
      __syncwarp();
    }
  }

  if (p.split > 1) cluster_sync_all();                    // no CTA leaves while another reads its state
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int DP, bool F16>
int launch_dp(SparseParams& p, int sms, cudaStream_t stream) {
  using C = Cfg<DP>;
  auto kernel = attn_block_sparse_kernel<DP, F16>;
  // Per device: the function's attributes, and how many clusters of each size
  // run at once (a repeated set from racing threads is harmless).
  static std::atomic<bool> ready[kMaxDevices];
  static std::atomic<int> clusters[kMaxDevices][kMaxSplit + 1];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return DT_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  if (!ready[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess ||
        cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
      return DT_ERR_CUDA;
    for (int s = 2; s <= kMaxSplit; ++s) {
      int n = 0;
      attr.val.clusterDim.x = s;
      cfg.numAttrs = 1;
      cfg.gridDim = dim3(s);
      if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
        cudaGetLastError();                       // a size the device does not run
        n = 0;
      }
      clusters[dev][s].store(n, std::memory_order_relaxed);
    }
    ready[dev].store(true, std::memory_order_release);
  }
  const int64_t items = (int64_t)p.H * p.nqb;
  // Split the lists where whole lists would leave half the SMs idle: the
  // largest cluster of which all run at once, at no less than two tiles a CTA.
  // One row a head over 512 blocks of 64, D = 128, 148 SMs: 40 heads 108 us in
  // three, 129 in two, 148 in four (whose clusters do not all run at once), 219
  // whole; 74 heads 182 in two, 203 in three, 237 whole.  With more lists than
  // half the SMs the clusters come in waves: 75 heads 238 whole, 284 in two, 204
  // in three; 100 heads 257, 292, 302; 148 heads 348, 357, 412.
  p.split = 1;
  const int tiles = ceil_div(p.cap, p.per_tile);
  if (2 * items <= sms)
    for (int s = 2; s <= kMaxSplit && 2 * s <= tiles; ++s)
      if (items <= clusters[dev][s].load(std::memory_order_relaxed)) p.split = s;
  attr.val.clusterDim.x = p.split;
  cfg.numAttrs = p.split > 1 ? 1 : 0;
  cfg.gridDim = dim3((unsigned)(items * p.split));
  return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? DT_OK : DT_ERR_CUDA;
}

}  // namespace

int launch_attn_sparse(SparseParams& p, int dp, bool f16, int sms, cudaStream_t stream) {
  switch (dp) {
    case 64: return f16 ? launch_dp<64, true>(p, sms, stream) : launch_dp<64, false>(p, sms, stream);
    case 80: return f16 ? launch_dp<80, true>(p, sms, stream) : launch_dp<80, false>(p, sms, stream);
    case 128: return f16 ? launch_dp<128, true>(p, sms, stream) : launch_dp<128, false>(p, sms, stream);
  }
  return DT_ERR_UNSUPPORTED;
}

}  // namespace dt

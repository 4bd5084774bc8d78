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
// A work item is (head, query block).  With at least as many items as SMs the
// grid is persistent, one CTA per SM striding over the items head-major, so the
// CTAs that run together read one head's K and V through L2.  With fewer, the
// `split` CTAs of a cluster take an equal run of the list's tiles each and join
// their states (m, l, unnormalised O) through distributed shared memory.
//
// Per CTA, 16 warps (4 warpgroups, registers rebalanced with setmaxnreg):
//   warps 0-7   softmax: two warps per SM sub-partition, each owning 16 rows of
//               the tile (16-lane TMEM accesses; a thread holds 2 rows x 32
//               columns); P is written back over S in TMEM as 16-bit values
//   warps 8-11  epilogue: O (TMEM) -> registers, TMEM released, normalised rows
//               and LSEs to memory, under the next item's tiles
//   warp 12     tcgen05.mma S = Q K^T; TMEM alloc/free
//   warp 13     TMA: Q (two buffers) and the K ring
//   warp 14     TMA: the V ring
//   warp 15     tcgen05.mma O += P V (a second issuing thread: one thread
//               issues an MMA only every ~50 clk)
// Tensor memory: three S/P buffers [0,384), O [384,384+DP).
//
// P is rounded to the 16-bit type of V for the tensor cores (relative 2^-9
// bf16, 2^-12 fp16 per weight, averaged over a row's keys); sums, maxima and O
// stay in fp32, and l sums the unrounded weights.
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
#include "sm100.cuh"

namespace dt {
namespace {

using namespace sm100;

constexpr int kThreads = 512;
constexpr int kWarpEpi = 8, kWarpMma = 12, kWarpTmaK = 13, kWarpTmaV = 14, kWarpMmaPV = 15;
// Registers per thread at launch (the build checks that ptxas chose them) and
// the per-warpgroup split, which must fit the launch pool.
constexpr int kLaunchRegs = 128;
constexpr int kRegsSoftmax = 128, kRegsEpilogue = 192, kRegsOther = 64;
static_assert(128 * (2 * kRegsSoftmax + kRegsEpilogue + kRegsOther) <= kThreads * kLaunchRegs, "register split");
constexpr uint64_t kDrainLimitNs = 1000000000ull;
constexpr int kMaxDevices = 64;
constexpr int kMaxSplit = 16;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleThreshold = 8.0f;   // log2 units: rescale O only when the max grows by > 2^8

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
                       bStFull = bOFree + 1, bStFree = bStFull + 2, bDrain = bStFree + 2, bDrainPV = bDrain + 1,
                       kNumBars = bDrainPV + 1;
  static constexpr int kStatsBytes = 2 * 2 * 128 * 4;
  static constexpr int kSmem = kTileBytes * (kNQ + kNK + kNV) + kStatsBytes + kNumBars * 8 + 16;
  static_assert(kSmem <= 232448, "shared memory budget");
  // a split item's partial O ([128][DP] fp32) reuses the K ring, drained by then
  static_assert(kNK * kTileBytes >= 128 * DP * 4, "partial O fits the K ring");
};

// Columns c_j = 8*(j/2) + cq + (j%2), j = 0..31, that a softmax thread holds:
// how many of them are below x (they increase in j).
__device__ __forceinline__ int cols_below(int x, int cq) {
  const int y = x - cq;
  return imin(imax((y + 7) >> 3, 0), 16) + imin(imax((y + 6) >> 3, 0), 16);
}
__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? 0xffffffffu : ((1u << n) - 1u); }

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int32_t* status,
                                          uint64_t limit) {
  const bool ok = mbar_wait(bar, parity, abort, status, DT_ERR_TIMEOUT, limit);
  return __all_sync(0xffffffffu, ok);
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

// One item's list: entries [0, n), of which this CTA takes tiles [t0, t1).
// The list's length and its first entries are loaded an item ahead, and every
// other entry a tile ahead: a load from L2 costs as much as a third of a tile,
// and two one after another at every item cost each role 1-2 us.
struct Item { int h, q0, rows, n, t0, t1; };
__device__ __forceinline__ int load_count(const SparseParams& p, int item) {
  return p.count && item < p.H * p.nqb ? __ldg(p.count + item) : p.cap;
}
__device__ __forceinline__ Item make_item(const SparseParams& p, int item, int rank, int count) {
  Item it;
  it.h = item / p.nqb;
  it.q0 = (item - it.h * p.nqb) * kTile;
  it.rows = imin(kTile, p.Sq - it.q0);
  it.n = imin(imax(count, 0), p.cap);
  const int nt = (it.n + p.per_tile - 1) / p.per_tile;
  it.t0 = p.split == 1 ? 0 : (int)((int64_t)nt * rank / p.split);
  it.t1 = p.split == 1 ? nt : (int)((int64_t)nt * (rank + 1) / p.split);
  return it;
}
// The entries of tile t of an item's list, as loaded (none past the list's allocation).
struct Entries { int a, b; };
__device__ __forceinline__ Entries load_entries(const SparseParams& p, int item, int t) {
  Entries e = {-1, -1};
  const int i = t * p.per_tile;
  if (item < p.H * p.nqb && i < p.cap) {
    const int32_t* l = p.idx + (int64_t)item * p.cap + i;
    e.a = __ldg(l);
    if (p.per_tile == 2 && i + 1 < p.cap) e.b = __ldg(l + 1);
  }
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
  float* stat_m = reinterpret_cast<float*>(sV + C::kNV * C::kTileBytes);      // [2][128]
  float* stat_l = stat_m + 256;                                              // [2][128]
  uint64_t* bars = reinterpret_cast<uint64_t*>(stat_l + 256);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + C::kNumBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t lim = p.wait_limit_ns;
  const int rank = p.split > 1 ? (int)cluster_rank() : 0;
  const int items = p.H * p.nqb;
  const int item0 = blockIdx.x / p.split, istep = gridDim.x / p.split;

  if (warp == kWarpTmaK && lane == 0) {
    for (int i = 0; i < C::kNumBars; ++i) mbar_init(&bars[i], 1);
    // every thread of the arriving role arrives (no single-lane branches)
    for (int i = 0; i < C::kNS; ++i) mbar_init(&bars[C::bPFull + i], 8 * 32);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars[C::bStFull + i], 8 * 32);
      mbar_init(&bars[C::bStFree + i], 4 * 32);
    }
    mbar_init(&bars[C::bOFree], 4 * 32);
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

  if (warp >= kWarpMma) {
    regs_set<kLaunchRegs, kRegsOther>();
    if (warp == kWarpTmaK || warp == kWarpTmaV) {
      // ---------------------------------------------------------- TMA producers
      if (lane == 0) {
        const bool is_k = warp == kWarpTmaK;
        const CUtensorMap* tm = is_k ? &p.tmK : &p.tmV;
        const CUtensorMap* tmt = is_k ? &p.tmKt : &p.tmVt;
        uint8_t* ring = is_k ? sK : sV;
        const uint32_t ns = is_k ? C::kNK : C::kNV;
        uint64_t* full = &bars[is_k ? C::bKFull : C::bVFull];
        uint64_t* empty = &bars[is_k ? C::bKEmpty : C::bVEmpty];
        prefetch_tmap(tm);
        if (C::kTail) prefetch_tmap(tmt);
        if (is_k) { prefetch_tmap(&p.tmQ); if (C::kTail) prefetch_tmap(&p.tmQt); }
        // K/V blocks are read by many query blocks of the head; a Q tile once
        const uint64_t pol_keep = l2_policy_evict_last(), pol_once = l2_policy_evict_first();
        uint32_t g = 0, nq = 0;
        // 64 rows from row0 of a K, V or Q head, into half `half` of a tile
        auto load_half = [&](const CUtensorMap* t64, const CUtensorMap* t16, uint8_t* tile, uint64_t* bar, int half,
                             int row0, int h, uint64_t pol) {
#pragma unroll
          for (int c = 0; c < C::kN64; ++c)
            tma_load_3d_hint(tile + c * C::kBlk + half * (C::kBlk / 2), t64, bar, 64 * c, row0, h, pol);
          if (C::kTail)
            tma_load_3d_hint(tile + C::kN64 * C::kBlk + half * (C::kTailBytes / 2), t16, bar, 64 * C::kN64, row0, h, pol);
        };
        int count = load_count(p, item0);
        Entries first = load_entries(p, item0, make_item(p, item0, rank, count).t0);
        for (int item = item0; item < items; item += istep) {
          const Item it = make_item(p, item, rank, count);
          if (is_k && rank == 0 && count != it.n) atomicCAS(p.status, 0, DT_ERR_INVALID);
          Entries nxt = first;
          count = load_count(p, item + istep);
          first = load_entries(p, item + istep, 0);
          if (it.t0 == it.t1) continue;
          if (is_k) {
            const uint32_t b = nq % C::kNQ;
            if (nq >= (uint32_t)C::kNQ &&
                !mbar_wait(&bars[C::bQEmpty + b], (nq / C::kNQ - 1) & 1, abort_flag, p.status, DT_ERR_TIMEOUT, lim))
              goto tma_done;
            uint8_t* dst = sQ + b * C::kTileBytes;
            mbar_arrive_expect_tx(&bars[C::bQFull + b], C::kTileBytes);
            load_half(&p.tmQ, &p.tmQt, dst, &bars[C::bQFull + b], 0, it.q0, it.h, pol_once);
            load_half(&p.tmQ, &p.tmQt, dst, &bars[C::bQFull + b], 1, it.q0 + 64, it.h, pol_once);
            ++nq;
          }
          const int hk = it.h / p.per_kv;
          for (int t = it.t0; t < it.t1; ++t, ++g) {
            const Halves v = tile_halves(p, it, t, nxt);
            if (t + 1 < it.t1) nxt = load_entries(p, item, t + 1);
            if (is_k && (v.r0 >= p.Sk || (p.per_tile == 2 && v.r1 >= p.Sk))) atomicCAS(p.status, 0, DT_ERR_INVALID);
            const uint32_t st = g % ns;
            if (g >= ns && !mbar_wait(&empty[st], ((g / ns) - 1) & 1, abort_flag, p.status, DT_ERR_TIMEOUT, lim))
              goto tma_done;
            uint8_t* dst = ring + st * C::kTileBytes;
            mbar_arrive_expect_tx(&full[st], v.r1 < 0 ? C::kTileBytes / 2 : C::kTileBytes);
            load_half(tm, tmt, dst, &full[st], 0, v.r0, hk, pol_keep);
            if (v.r1 >= 0) load_half(tm, tmt, dst, &full[st], 1, v.r1, hk, pol_keep);
          }
        }
      tma_done:
        // let every copy this warp started land before shared memory goes away
        volatile int never = 0;
        for (uint32_t s = 0; s < ns; ++s)
          if (s < g) {
            const uint32_t last = g - 1 - ((g - 1 - s) % ns);             // latest tile that used stage s
            mbar_wait(&full[s], (last / ns) & 1, &never, p.status, DT_ERR_TIMEOUT, kDrainLimitNs);
          }
        if (is_k)
          for (uint32_t b = 0; b < (uint32_t)C::kNQ; ++b)
            if (b < nq) {
              const uint32_t last = nq - 1 - ((nq - 1 - b) % C::kNQ);
              mbar_wait(&bars[C::bQFull + b], (last / C::kNQ) & 1, &never, p.status, DT_ERR_TIMEOUT, kDrainLimitNs);
            }
      }
      __syncwarp();
    } else if (warp == kWarpMma) {
      // ---------------------------------------------------------- S = Q K^T
      if (lane == 0) {
        constexpr uint32_t idesc = idesc16<F16>(128, 128, 0);
        const uint32_t aK = smem_u32(sK);
        uint32_t g = 0, nq = 0;
        bool ok = true;
        int count = load_count(p, item0);
        for (int item = item0; item < items && ok; item += istep) {
          const Item it = make_item(p, item, rank, count);
          count = load_count(p, item + istep);
          if (it.t0 == it.t1) continue;
          const uint32_t qb = nq % C::kNQ;
          const uint32_t aQ = smem_u32(sQ) + qb * C::kTileBytes;
          if (!mbar_wait(&bars[C::bQFull + qb], (nq / C::kNQ) & 1, abort_flag, p.status, DT_ERR_TIMEOUT, lim)) break;
          ++nq;
          for (int t = it.t0; t < it.t1; ++t, ++g) {
            const uint32_t st = g % C::kNK, sb = g % C::kNS;
            if (!mbar_wait(&bars[C::bKFull + st], (g / C::kNK) & 1, abort_flag, p.status, DT_ERR_TIMEOUT, lim)) {
              ok = false;
              break;
            }
            // S buffer sb held P(g-3): its P V (issued by warp 15) must be done
            if (g >= (uint32_t)C::kNS &&
                !mbar_wait(&bars[C::bPVDone + sb], (g / C::kNS - 1) & 1, abort_flag, p.status, DT_ERR_TIMEOUT, lim)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t dS = tmem + C::kColS + sb * 128;
            const uint32_t kb = aK + st * C::kTileBytes;
            uint32_t acc = 0u;
#pragma unroll 1
            for (int blk = 0; blk < C::kN64; ++blk) {
              uint64_t qd = smem_desc(aQ + blk * C::kBlk, 16, 1024, kSwizzle128B);
              uint64_t kd = smem_desc(kb + blk * C::kBlk, 16, 1024, kSwizzle128B);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) {             // 16 head-dim columns (32 bytes of a row) per MMA
                mma_ss(dS, qd, kd, idesc, acc);
                acc = 1u;
                qd += 32 >> 4;
                kd += 32 >> 4;
              }
            }
            if (C::kTail) {
              const uint32_t off = C::kN64 * C::kBlk;
              mma_ss(dS, smem_desc(aQ + off, 16, 256, kSwizzle32B), smem_desc(kb + off, 16, 256, kSwizzle32B), idesc, 1u);
            }
            mma_commit(&bars[C::bSFull + sb]);
            mma_commit(&bars[C::bKEmpty + st]);
          }
          mma_commit(&bars[C::bQEmpty + qb]);
        }
        // all MMAs this thread issued complete before tensor memory is freed
        mma_commit(&bars[C::bDrain]);
        volatile int never = 0;
        mbar_wait(&bars[C::bDrain], 0, &never, p.status, DT_ERR_TIMEOUT, kDrainLimitNs);
      }
      __syncwarp();
    } else if (warp == kWarpMmaPV) {
      // ---------------------------------------------------------- O += P V
      if (lane == 0) {
        constexpr uint32_t idesc_pv = idesc16<F16>(128, 64 * C::kN64, 1);
        constexpr uint32_t idesc_pvt = idesc16<F16>(128, 16, 1);
        const uint32_t aV = smem_u32(sV);
        uint32_t g = 0, nq = 0;
        bool ok = true;
        int count = load_count(p, item0);
        for (int item = item0; item < items && ok; item += istep) {
          const Item it = make_item(p, item, rank, count);
          count = load_count(p, item + istep);
          if (it.t0 == it.t1) continue;
          for (int t = it.t0; t < it.t1 && ok; ++t, ++g) {
            const uint32_t sb = g % C::kNS, st = g % C::kNV;
            ok = mbar_wait(&bars[C::bPFull + sb], (g / C::kNS) & 1, abort_flag, p.status, DT_ERR_TIMEOUT, lim) &&
                 (t > it.t0 || nq == 0 ||
                  mbar_wait(&bars[C::bOFree], (nq - 1) & 1, abort_flag, p.status, DT_ERR_TIMEOUT, lim)) &&
                 mbar_wait(&bars[C::bVFull + st], (g / C::kNV) & 1, abort_flag, p.status, DT_ERR_TIMEOUT, lim);
            if (!ok) break;
            tc_fence_after();
            uint32_t aP = tmem + C::kColS + sb * 128;
            const uint32_t vb = aV + st * C::kTileBytes;
            // 16 keys per MMA: descriptors advance by 16 V rows.  A tile that
            // holds one 64-key block ends after 4.
            const int kn = p.per_tile == 2 && 2 * t + 1 >= it.n ? 4 : 8;
            uint64_t vd = smem_desc(vb, C::kBlk, 1024, kSwizzle128B);
            uint64_t vdt = smem_desc(vb + C::kN64 * C::kBlk, C::kTailBytes, 256, kSwizzle32B);
            uint32_t acc = t > it.t0 ? 1u : 0u;
#pragma unroll 1
            for (int kk = 0; kk < kn; ++kk) {
              mma_ts(tmem + C::kColO, aP, vd, idesc_pv, acc);
              if (C::kTail) mma_ts(tmem + C::kColO + 64 * C::kN64, aP, vdt, idesc_pvt, acc);
              acc = 1u;
              aP += 8;
              vd += 2048 >> 4;
              vdt += 512 >> 4;
            }
            mma_commit(&bars[C::bVEmpty + st]);
            mma_commit(&bars[C::bPVDone + sb]);
            if (t == it.t1 - 1) mma_commit(&bars[C::bOFull]);
          }
          ++nq;
        }
        mma_commit(&bars[C::bDrainPV]);
        volatile int never = 0;
        mbar_wait(&bars[C::bDrainPV], 0, &never, p.status, DT_ERR_TIMEOUT, kDrainLimitNs);
      }
      __syncwarp();
    }
  } else if (warp < kWarpEpi) {
    regs_set<kLaunchRegs, kRegsSoftmax>();
    // ------------------------------------------------------------ softmax
    // Warp w owns tile rows rbase .. rbase+15; thread t holds rows ra = rbase +
    // t/4 and rb = ra + 8 at columns 8i + 2(t%4) + {0,1}, i = 0..15.
    const int rbase = (warp & 3) * 32 + (warp >> 2) * 16;
    const int ra = rbase + (lane >> 2), rb = ra + 8;
    const int cq = 2 * (lane & 3);
    const uint32_t lane_base = static_cast<uint32_t>(rbase) << 16;
    const float sl2 = p.scale_log2;
    uint32_t g = 0, nq = 0;
    int count = load_count(p, item0);
    Entries first = load_entries(p, item0, make_item(p, item0, rank, count).t0);
    for (int item = item0; item < items; item += istep) {
      const Item it = make_item(p, item, rank, count);
      Entries nxt = first;
      count = load_count(p, item + istep);
      first = load_entries(p, item + istep, 0);
      if (it.t0 == it.t1) continue;
      const bool idle = rbase >= it.rows;          // none of this warp's rows exist: hand the tiles on
      float ma = neg_inf(), mb = neg_inf();         // running max (log2 units)
      uint64_t la[2] = {0ull, 0ull}, lb[2] = {0ull, 0ull};      // packed pairs of partial row sums
      for (int t = it.t0; t < it.t1; ++t, ++g) {
        const uint32_t sb = g % C::kNS;
        const Halves hv = tile_halves(p, it, t, nxt);
        if (t + 1 < it.t1) nxt = load_entries(p, item, t + 1);
        if (!warp_wait(&bars[C::bSFull + sb], (g / C::kNS) & 1, abort_flag, p.status, lim)) goto sm_done;
        if (idle) {
          mbar_arrive(&bars[C::bPFull + sb]);
          continue;
        }
        tc_fence_after();
        const uint32_t sc = tmem + lane_base + C::kColS + sb * 128;
        uint32_t sr[64];
        tmem_ld_16x256b_x8(sc, sr);
        tmem_ld_16x256b_x8(sc + 64, sr + 32);
        tmem_wait_ld();
        const int v0 = p.Sk - hv.r0, v1 = hv.r1 < 0 ? 0 : p.Sk - hv.r1;      // keys of each half
        if (v0 < 64 || v1 < 64) {
          // kept columns as a bit mask over this thread's 32, one test per
          // element: compact code for the rare tile.  Assigned, not added: the
          // logits there may be anything.
          const uint32_t keep = low_bits(cols_below(imin(v0, 64), cq)) |
                                (low_bits(cols_below(64 + imin(v1, 64), cq)) & ~low_bits(cols_below(64, cq)));
#pragma unroll
          for (int e = 0; e < 64; ++e)
            if (!(keep & (1u << (2 * (e >> 2) + (e & 1))))) sr[e] = f2u(neg_inf());
        }
        // row maxima: two chains per row, then across the 4 threads of a row
        float xa0 = fmaxf(u2f(sr[0]), u2f(sr[1])), xa1 = fmaxf(u2f(sr[4]), u2f(sr[5]));
        float xb0 = fmaxf(u2f(sr[2]), u2f(sr[3])), xb1 = fmaxf(u2f(sr[6]), u2f(sr[7]));
#pragma unroll
        for (int r4 = 2; r4 < 16; r4 += 2) {
          xa0 = max3f(xa0, u2f(sr[4 * r4]), u2f(sr[4 * r4 + 1]));
          xa1 = max3f(xa1, u2f(sr[4 * r4 + 4]), u2f(sr[4 * r4 + 5]));
          xb0 = max3f(xb0, u2f(sr[4 * r4 + 2]), u2f(sr[4 * r4 + 3]));
          xb1 = max3f(xb1, u2f(sr[4 * r4 + 6]), u2f(sr[4 * r4 + 7]));
        }
        float mxa = fmaxf(xa0, xa1), mxb = fmaxf(xb0, xb1);
        mxa = fmaxf(mxa, __shfl_xor_sync(0xffffffffu, mxa, 1));
        mxb = fmaxf(mxb, __shfl_xor_sync(0xffffffffu, mxb, 1));
        mxa = fmaxf(mxa, __shfl_xor_sync(0xffffffffu, mxa, 2));
        mxb = fmaxf(mxb, __shfl_xor_sync(0xffffffffu, mxb, 2));
        const float mxa2 = mxa * sl2, mxb2 = mxb * sl2;
        const bool first = t == it.t0;
        const float na = first ? mxa2 : ((mxa2 > ma + kRescaleThreshold) ? mxa2 : ma);
        const float nb = first ? mxb2 : ((mxb2 > mb + kRescaleThreshold) ? mxb2 : mb);
        // a row that has seen only masked keys (max -inf) has O = 0 and l = 0:
        // it takes the new reference without a rescale
        const bool resa = !first && (na != ma) && (ma != neg_inf());
        const bool resb = !first && (nb != mb) && (mb != neg_inf());
        if (__any_sync(0xffffffffu, resa || resb)) {
          // O holds the previous tiles' sum: wait for its last P V, then rescale
          if (!warp_wait(&bars[C::bPVDone + (g - 1) % C::kNS], ((g - 1) / C::kNS) & 1, abort_flag, p.status, lim))
            goto sm_done;
          tc_fence_after();
          const float alpha_a = resa ? ex2(ma - na) : 1.f, alpha_b = resb ? ex2(mb - nb) : 1.f;
          const uint32_t oc = tmem + lane_base + C::kColO;
#pragma unroll 1
          for (int c0 = 0; c0 < DP; c0 += 16) {
            uint32_t o[8];
            tmem_ld_16x256b_x2(oc + c0, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = f2u(u2f(o[e]) * ((e & 2) ? alpha_b : alpha_a));
            tmem_st_16x256b_x2(oc + c0, o);
          }
          tmem_wait_st();
          const uint64_t aa = pk2(alpha_a, alpha_a), ab = pk2(alpha_b, alpha_b);
#pragma unroll
          for (int k = 0; k < 2; ++k) { la[k] = fma2(la[k], aa, 0ull); lb[k] = fma2(lb[k], ab, 0ull); }
        }
        ma = na; mb = nb;
        const float mra = (ma == neg_inf()) ? 0.f : ma, mrb = (mb == neg_inf()) ? 0.f : mb;
        const uint64_t sl2x2 = pk2(sl2, sl2), nma = pk2(-mra, -mra), nmb = pk2(-mrb, -mrb);
        // exponentials, 8 repetitions (32 P columns) per TMEM store
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t ph[16];
#pragma unroll
          for (int r4 = 0; r4 < 8; ++r4) {
            const int e = 4 * (8 * hf + r4);
            float x0, x1, x2, x3;
            upk2(fma2(pk2(u2f(sr[e]), u2f(sr[e + 1])), sl2x2, nma), x0, x1);
            upk2(fma2(pk2(u2f(sr[e + 2]), u2f(sr[e + 3])), sl2x2, nmb), x2, x3);
            const float p0 = ex2(x0), p1 = ex2(x1), p2 = ex2(x2), p3 = ex2(x3);
            la[r4 & 1] = add2(la[r4 & 1], pk2(p0, p1));
            lb[r4 & 1] = add2(lb[r4 & 1], pk2(p2, p3));
            ph[2 * r4] = pack16<F16>(p0, p1);
            ph[2 * r4 + 1] = pack16<F16>(p2, p3);
          }
          tmem_st_16x128b_x8(sc + 32 * hf, ph);
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&bars[C::bPFull + sb]);
      }
      float sa, sbm;
      {
        float u0, u1, w0, w1;
        upk2(add2(la[0], la[1]), u0, u1);
        upk2(add2(lb[0], lb[1]), w0, w1);
        sa = u0 + u1;
        sbm = w0 + w1;
      }
      sa += __shfl_xor_sync(0xffffffffu, sa, 1);
      sbm += __shfl_xor_sync(0xffffffffu, sbm, 1);
      sa += __shfl_xor_sync(0xffffffffu, sa, 2);
      sbm += __shfl_xor_sync(0xffffffffu, sbm, 2);
      const uint32_t st = nq & 1;
      if (nq >= 2 && !warp_wait(&bars[C::bStFree + st], ((nq >> 1) - 1) & 1, abort_flag, p.status, lim)) goto sm_done;
      // the 4 threads of a row hold the same values: all of them write
      stat_m[st * 128 + ra] = ma;
      stat_l[st * 128 + ra] = sa;
      stat_m[st * 128 + rb] = mb;
      stat_l[st * 128 + rb] = sbm;
      mbar_arrive(&bars[C::bStFull + st]);
      ++nq;
    }
  sm_done:;
  } else {
    regs_set<kLaunchRegs, kRegsEpilogue>();
    // ------------------------------------------------------------ epilogue
    const int r = (warp - kWarpEpi) * 32 + lane;          // tile row of this thread
    const uint32_t oaddr = tmem + (static_cast<uint32_t>((warp - kWarpEpi) * 32) << 16) + C::kColO;
    uint32_t nq = 0;
    int count = load_count(p, item0);
    for (int item = item0; item < items; item += istep) {
      const Item it = make_item(p, item, rank, count);
      count = load_count(p, item + istep);
      const bool valid = r < it.rows;
      const int64_t orow = it.h * p.o_head + (int64_t)(it.q0 + r) * p.o_row;
      float* lrow = p.L + (int64_t)it.h * p.Sq + it.q0 + r;
      if (it.t0 == it.t1) {
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
      const uint32_t st = nq & 1;
      if (!warp_wait(&bars[C::bStFull + st], (nq >> 1) & 1, abort_flag, p.status, lim)) goto ep_done;
      const float m = stat_m[st * 128 + r], l = stat_l[st * 128 + r];
      mbar_arrive(&bars[C::bStFree + st]);
      if (!warp_wait(&bars[C::bOFull], nq & 1, abort_flag, p.status, lim)) goto ep_done;
      tc_fence_after();
      uint32_t op[DP];
#pragma unroll
      for (int c0 = 0; c0 < DP; c0 += 16) tmem_ld16p(oaddr + c0, op + c0);
      tmem_wait_ld();
      tc_fence_before();
      mbar_arrive(&bars[C::bOFree]);
      if (p.split > 1) {
        float* part = reinterpret_cast<float*>(sK);
        if (valid)
#pragma unroll
          for (int c = 0; c < D; c += 4)
            *reinterpret_cast<float4*>(part + part_chunk<DP>(r, c / 4)) =
                make_float4(u2f(op[c]), u2f(op[c + 1]), u2f(op[c + 2]), u2f(op[c + 3]));
      } else if (valid) {
        // l > 0 unless every listed key is past the end or has a logit of -inf; NaN stays
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int c = 0; c < D; c += 8) {
          float x[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = l == 0.f ? 0.f : u2f(op[c + e]) * inv;
          store_out8<F16>(p, orow + c, x);
        }
        *lrow = l == 0.f ? neg_inf() : (m + lg2(l)) * kLn2;
      }
      ++nq;
    }
  ep_done:;
  }

  if (p.split > 1) {
    // Join of the cluster's states of its one item: M = max m_i, w_i =
    // 2^(m_i - M), O = sum w_i O_i / sum w_i l_i.  CTA `rank` joins 8-column
    // chunks rank, rank + split, ... of the item's rows; every thread reaches
    // both barriers whatever its role met before.
    __syncwarp();
    cluster_sync_all();
    if (warp >= kWarpEpi && warp < kWarpMma && !*abort_flag) {
      const Item it = make_item(p, item0, rank, load_count(p, item0));
      const uint32_t a_m = smem_u32(stat_m), a_l = smem_u32(stat_l), a_o = smem_u32(sK);
      const int nchunk = it.rows * (D / 8);
      for (int i = (threadIdx.x - kWarpEpi * 32) * p.split + rank; i < nchunk; i += 128 * p.split) {
        const int row = i / (D / 8), c = 8 * (i - row * (D / 8));
        float M = neg_inf();
        for (int k = 0; k < p.split; ++k) M = fmaxf(M, ld_cluster(map_rank(a_m + 4 * row, k)));
        const float Mr = M == neg_inf() ? 0.f : M;
        float x[8] = {}, l = 0.f;
        for (int k = 0; k < p.split; ++k) {
          const float lk = ld_cluster(map_rank(a_l + 4 * row, k));
          if (lk == 0.f) continue;                        // an empty state, and its O was never written
          const float w = ex2(ld_cluster(map_rank(a_m + 4 * row, k)) - Mr);
          const float4 u = ld_cluster4(map_rank(a_o + 4 * part_chunk<DP>(row, c / 4), k));
          const float4 v = ld_cluster4(map_rank(a_o + 4 * part_chunk<DP>(row, c / 4 + 1), k));
          l = fmaf(w, lk, l);
          x[0] = fmaf(w, u.x, x[0]); x[1] = fmaf(w, u.y, x[1]); x[2] = fmaf(w, u.z, x[2]); x[3] = fmaf(w, u.w, x[3]);
          x[4] = fmaf(w, v.x, x[4]); x[5] = fmaf(w, v.y, x[5]); x[6] = fmaf(w, v.z, x[6]); x[7] = fmaf(w, v.w, x[7]);
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= inv;
        store_out8<F16>(p, it.h * p.o_head + (int64_t)(it.q0 + row) * p.o_row + c, x);
        if (c == 0) p.L[(int64_t)it.h * p.Sq + it.q0 + row] = l == 0.f ? neg_inf() : (M + lg2(l)) * kLn2;
      }
    }
    __syncwarp();
    cluster_sync_all();                                   // no CTA leaves while another reads its state
  }
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
  // Split the lists where whole lists would leave SMs idle: the largest
  // cluster of which all run at once, at no less than two tiles a CTA.
  p.split = 1;
  const int tiles = ceil_div(p.cap, p.per_tile);
  if (2 * items <= sms)
    for (int s = 2; s <= kMaxSplit && 2 * s <= tiles; ++s)
      if (items <= clusters[dev][s].load(std::memory_order_relaxed)) p.split = s;
  attr.val.clusterDim.x = p.split;
  cfg.numAttrs = p.split > 1 ? 1 : 0;
  cfg.gridDim = dim3((unsigned)(p.split > 1 ? items * p.split : (items < sms ? items : sms)));
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

// token_ops.cu -- the passes in front of block-sparse attention (sm_100a):
//   rope_table_kernel     cos/sin of token positions;
//   qk_norm_rope_kernel   per-head RMS norm, rotation, layout change and block
//                         means of queries and keys (values pass through);
//   block_select_kernel   top-k key blocks of every query block by the 64-bit
//                         scores of block means.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "../../include/dt.h"
#include "sm100_more.cuh"
#include "token_ops.h"

namespace dt {
namespace {

using namespace sm100;

int launched() { return cudaGetLastError() == cudaSuccess ? DT_OK : DT_ERR_CUDA; }
int cdiv(int a, int b) { return (a + b - 1) / b; }

// ------------------------------------------------------------------ rotation table
// cos and sin of 2 pi t, t = pos * turns, where only t's fraction counts: with
// turns as a 64-bit binary fraction T, pos * T mod 2^64 is that fraction
// without any reduction, and needs no 64-bit floating point.  T is off by less
// than 2^-58 (truncation 2^-64; at most 127 extended-precision products of one
// power: 0.16 e^-z (3 * 127 + z + 2) 2^-64, z = -ln of the frequency), so the
// farthest position by less than 2^-27 turns.  Its upper 32 bits split into the nearest quarter turn and a
// rest |x| <= 1/8 turn, on which sin(2 pi x) / x and cos(2 pi x) are
// polynomials in x^2 (minimax by Remez exchange: 1.3e-9 and 5e-11), two pairs in
// each packed operation.  The roundings of x (2 pi 2^-28) and of the polynomials
// leave the results within 2^-22 by bound, 2^-23.2 as measured, near and far.
// A CTA owns kRopeTokens tokens, a thread two pairs of a token (16 bytes of the
// table) at a time; T and the axes lie in shared memory, since lanes with
// different pairs would serialise on the parameter bank.  The library's sincospif and
// a division per element took 10.2 us for 32,760 tokens of 64 pairs.
constexpr int kRopeThreads = 256, kRopeTokens = 32;

__device__ __forceinline__ uint64_t both(float x) { return pk2(x, x); }

__global__ void __launch_bounds__(kRopeThreads) rope_table_kernel(const __grid_constant__ RopeTableArgs a) {
  __shared__ uint64_t turns[kMaxPairs];
  __shared__ int axis[kMaxPairs];
  for (int i = threadIdx.x; i < a.pairs; i += kRopeThreads) {
    turns[i] = a.turns[i];
    axis[i] = a.axis[i];
  }
  __syncthreads();
  const int halfp = (a.pairs + 1) / 2;
  const uint32_t inv = 0xffffffffu / halfp + 1u;    // i / halfp = i * inv >> 32 for i < 2^12, halfp <= 64 (0: halfp = 1)
  const int s0 = blockIdx.x * kRopeTokens, n = min(kRopeTokens, a.S - s0) * halfp;
#pragma unroll 4
  for (int i = threadIdx.x; i < n; i += kRopeThreads) {
    const int ds = halfp > 1 ? (int)__umulhi(i, inv) : i, p0 = 2 * (i - ds * halfp), s = s0 + ds;
    uint32_t q[2];
    float x[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int pr = min(p0 + e, a.pairs - 1);
      const int64_t pos = __ldg(a.pos + (int64_t)axis[pr] * a.S + s);
      const uint32_t u = (uint32_t)(((uint64_t)pos * turns[pr]) >> 32);       // 2^-32 turns
      q[e] = (u + 0x20000000u) >> 30;
      x[e] = (float)(int)(u - (q[e] << 30)) * 0x1p-32f;
    }
    const uint64_t x2 = pk2(x[0], x[1]), z = mul2(x2, x2);
    uint64_t sp = fma2(both(-0x1.2cf8aap+6f), z, both(0x1.465a52p+6f));
    sp = fma2(sp, z, both(-0x1.4abba8p+5f));
    sp = mul2(fma2(sp, z, both(0x1.921fb4p+2f)), x2);
    uint64_t cp = fma2(both(0x1.d9c364p+5f), z, both(-0x1.55c57cp+6f));
    cp = fma2(cp, z, both(0x1.03c1dcp+6f));
    cp = fma2(cp, z, both(-0x1.3bd3ccp+4f));
    cp = fma2(cp, z, both(1.f));
    float sn[2], cs[2], out[4];
    upk2(sp, sn[0], sn[1]);
    upk2(cp, cs[0], cs[1]);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      // a quarter turn on: (c, s) -> (-s, c)
      const float c = q[e] & 1 ? sn[e] : cs[e], sv = q[e] & 1 ? cs[e] : sn[e];
      out[2 * e] = __uint_as_float(__float_as_uint(c) ^ (((q[e] + 1) & 2) << 30));
      out[2 * e + 1] = __uint_as_float(__float_as_uint(sv) ^ ((q[e] & 2) << 30));
    }
    float* dst = a.table + ((int64_t)s * a.pairs + p0) * 2;
    if ((a.pairs & 1) == 0) {
      *reinterpret_cast<float4*>(dst) = make_float4(out[0], out[1], out[2], out[3]);
    } else {                                       // rows of an odd number of pairs are 8-byte aligned only
      *reinterpret_cast<float2*>(dst) = make_float2(out[0], out[1]);
      if (p0 + 1 < a.pairs) *reinterpret_cast<float2*>(dst + 2) = make_float2(out[2], out[3]);
    }
  }
}

// ------------------------------------------------------------------ norm + rotation
template <typename T> struct Vec4;                 // 4 elements of T as one access
template <> struct Vec4<float> { using type = float4; };
template <> struct Vec4<__nv_bfloat16> { using type = uint2; };
template <> struct Vec4<__half> { using type = uint2; };

__device__ __forceinline__ void widen(const float4& v, float* x) { x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w; }
template <typename T>
__device__ __forceinline__ void widen4(const typename Vec4<T>::type& v, float* x);
template <>
__device__ __forceinline__ void widen4<float>(const float4& v, float* x) { widen(v, x); }
template <>
__device__ __forceinline__ void widen4<__nv_bfloat16>(const uint2& v, float* x) {
  x[0] = __uint_as_float(v.x << 16); x[1] = __uint_as_float(v.x & 0xffff0000u);
  x[2] = __uint_as_float(v.y << 16); x[3] = __uint_as_float(v.y & 0xffff0000u);
}
template <>
__device__ __forceinline__ void widen4<__half>(const uint2& v, float* x) {
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&v.x));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&v.y));
  x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
}
template <typename T>
__device__ __forceinline__ typename Vec4<T>::type narrow4(const float* x);
template <>
__device__ __forceinline__ float4 narrow4<float>(const float* x) { return make_float4(x[0], x[1], x[2], x[3]); }
template <>
__device__ __forceinline__ uint2 narrow4<__nv_bfloat16>(const float* x) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
template <>
__device__ __forceinline__ uint2 narrow4<__half>(const float* x) {
  const __half2 a = __floats2half2_rn(x[0], x[1]), b = __floats2half2_rn(x[2], x[3]);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
// 8 elements as two groups of 4; one 16-byte access where they are adjacent 16-bit elements.
// copy8 starts their copy into this lane's shared-memory slot, read8 takes them from there.
template <int N>
__device__ __forceinline__ void async_copy(void* smem, const void* at) {
  if (N == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(smem)), "l"(at) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(smem)), "l"(at) : "memory");
}
__device__ __forceinline__ void async_copy_l1(void* smem, const void* at) {      // 16 bytes, kept in L1
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(smem_u32(smem)), "l"(at) : "memory");
}
template <typename T, bool SPLIT>
__device__ __forceinline__ void copy8(uint8_t* slot, const T* at, int gap) {
  if (sizeof(T) == 2 && !SPLIT) {
    async_copy<16>(slot, at);
  } else {
    async_copy<4 * sizeof(T)>(slot, at);
    async_copy<4 * sizeof(T)>(slot + 4 * sizeof(T), at + gap);
  }
}
template <typename T>
__device__ __forceinline__ void read8(const uint8_t* slot, float* x) {
  using V = typename Vec4<T>::type;
  V v[2];
  if (sizeof(T) == 2) {
    *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(slot);
  } else {
    v[0] = reinterpret_cast<const V*>(slot)[0];
    v[1] = reinterpret_cast<const V*>(slot)[1];
  }
  widen4<T>(v[0], x);
  widen4<T>(v[1], x + 4);
}
template <typename T, bool SPLIT>
__device__ __forceinline__ void store8(T* at, int gap, const float* x) {
  using V = typename Vec4<T>::type;
  V v[2] = {narrow4<T>(x), narrow4<T>(x + 4)};
  if (sizeof(T) == 2 && !SPLIT) {
    *reinterpret_cast<uint4*>(at) = *reinterpret_cast<const uint4*>(v);
  } else {
    *reinterpret_cast<V*>(at) = v[0];
    *reinterpret_cast<V*>(at + gap) = v[1];
  }
}

// A warp owns neighbouring heads, 32/LPR of them (LPR lanes hold a row, 8 elements
// each), and a run of consecutive tokens, which it walks one by one: all 128 of a
// tile, or, when that would leave SMs idle, 1/wt of them (wt = 2, 4, 8 warps
// per run of heads).  A step's rows lie side by side in a token-major input, and
// share the token's rotation.  The warps of a CTA take neighbouring heads too, so
// the rotation comes from L2 once per CTA and from L1 for its other warps.  Rows and
// rotations come through rings of asynchronous copies, kDepth steps deep: with
// two or four rows in registers the pass waited on memory at 4.6-4.8 TB/s,
// whatever it computed, and with the rotation loaded one step ahead its latency,
// which the CTA's warps meet together, cost 80 us of 400 on 40 heads of 128.
// An element's partner in its pair is always in the same lane (HALVES: 4
// elements from each half), so the row's sum of squares is the only exchange, by
// shuffles.  A row is read before it is stored, by the lanes that store it
// (in-place calls).  Block means: sums over a lane's tokens, then over the
// warps of the head through shared memory, in a fixed order.
constexpr int kNormThreads = 256, kNormWarps = kNormThreads / 32;

template <typename TI, int LPR>
struct NormSmem {
  static constexpr int kDepth = sizeof(TI) == 4 ? 4 : 8;
  static constexpr int kSlot = 8 * sizeof(TI);      // bytes of a lane's 8 elements
  static constexpr int kRing = kDepth * 32 * kSlot; // a warp's rows
  static constexpr int kTurn = kDepth * LPR * 32;   // a warp's rotations (32 bytes per lane of a row)
  static constexpr int kPart = kNormWarps * 32 * 8 * 4;
  static constexpr int kBytes = kPart + kNormWarps * (kRing + kTurn);
  static_assert(kRing >= 32 * 8 * 4, "a ring holds a warp's sums");
};

template <typename TI, typename TO, int LPR, bool HALVES>
__global__ void __launch_bounds__(kNormThreads, 3) qk_norm_rope_kernel(const __grid_constant__ NormRopeArgs a) {
  constexpr int kHeads = 32 / LPR;                  // heads of a warp
  using M = NormSmem<TI, LPR>;
  constexpr int kDepth = M::kDepth, kSlot = M::kSlot;
  extern __shared__ __align__(16) uint8_t norm_smem[];
  // Sums over each warp's first segment (64 tokens, or its run if shorter), then the rings; the sums over a second
  // segment take the place of the warp's rows when all of those are read.
  float* part = reinterpret_cast<float*>(norm_smem);
  uint8_t* rings = norm_smem + M::kPart;
  const dt_norm_rope_params& p = a.p;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % LPR, sub = (threadIdx.x % 32) / LPR;
  const int wh = kNormWarps / a.wt;                 // runs of heads of the CTA
  const int tile = blockIdx.x / a.groups, group = blockIdx.x - tile * a.groups;
  const int hw = warp / a.wt, ws = warp - hw * a.wt;
  const int run = 128 / a.wt, seg = min(run, 64);
  const int hh = (group * wh + hw) * kHeads + sub;  // this lane's head, counted over queries, keys, values
  const int s0 = tile * 128 + ws * run;
  const bool turned = 8 * lane < p.rot;
  const int c0 = HALVES && turned ? 4 * lane : 8 * lane;
  const int gap = HALVES && turned ? p.rot / 2 : 4; // from the first 4 elements to the others

  const int kind = hh < p.H ? 0 : (hh < p.H + p.Hkv ? 1 : 2);
  const int h = kind == 0 ? hh : (kind == 1 ? hh - p.H : hh - p.H - p.Hkv);
  const TI* in = static_cast<const TI*>(kind == 0 ? a.q : (kind == 1 ? a.k : a.v));
  TO* out = static_cast<TO*>(kind == 0 ? a.Q : (kind == 1 ? a.K : a.V));
  const bool on = 8 * lane < p.D && hh < p.H + 2 * p.Hkv && in;
  int left = on ? min(p.S - s0, run) : 0;           // rows from this lane's next to the end of the run
  const int steps = min(run, max(0, p.S - s0));     // tokens of this warp's run
  const bool store = on && out != nullptr;
  const dt_strides si = kind == 0 ? p.q_in : (kind == 1 ? p.k_in : p.v_in);
  const dt_strides so = kind == 0 ? p.q_out : (kind == 1 ? p.k_out : p.v_out);
  if (on) in += h * si.head + s0 * si.row + c0;
  if (store) out += h * so.head + s0 * so.row + c0;
  const bool turn = on && kind < 2 && turned;
  const bool norm = p.norm && __any_sync(0xffffffffu, on && kind < 2);
  const float* w = kind == 0 ? a.wq : a.wk;
  float wv[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
  if (norm && w && on && kind < 2) {
    widen(__ldg(reinterpret_cast<const float4*>(w + c0)), wv);
    widen(__ldg(reinterpret_cast<const float4*>(w + c0 + gap)), wv + 4);
  }
  const uint64_t w2[4] = {pk2(wv[0], wv[1]), pk2(wv[2], wv[3]), pk2(wv[4], wv[5]), pk2(wv[6], wv[7])};
  uint8_t* slot = rings + warp * M::kRing + (threadIdx.x % 32) * kSlot;       // a lane reads back what it copied
  // A rotation row: lanes copy 16 bytes (two pairs) each; the two pieces of a reader's 4 pairs lie half a row apart,
  // so that a read touches every bank once.
  uint8_t* turns = rings + kNormWarps * M::kRing + warp * M::kTurn;
  const int l32 = threadIdx.x % 32, tdst = ((l32 >> 1) + (l32 & 1) * LPR) * 16;
  const bool any_turn = __any_sync(0xffffffffu, turn);
  const float* tr = a.table + (int64_t)s0 * p.rot + 4 * l32;
  int tleft = any_turn && 4 * l32 < p.rot ? min(p.S - s0, run) : 0;           // rotation rows left for this lane
  // Lanes past D (or of no head) copy nothing: their slots are zero throughout, and add nothing to a row's sum.
  // What a slot holds past the run's end is not stored and not summed.
  if (!on)
    for (int i = 0; i < kDepth; ++i)
      for (int e = 0; e < kSlot; e += 16) *reinterpret_cast<uint4*>(slot + i * 32 * kSlot + e) = make_uint4(0, 0, 0, 0);
  auto fetch = [&](int i, int ahead) {              // the row `ahead` tokens from this lane's next, into ring position i
    if (ahead < left) copy8<TI, HALVES>(slot + i * 32 * kSlot, in, gap);
    if (ahead < tleft) async_copy_l1(turns + i * LPR * 32 + tdst, tr);
    asm volatile("cp.async.commit_group;" ::: "memory");
    in += si.row;
    tr += p.rot;
  };
#pragma unroll
  for (int i = 0; i < kDepth - 1; ++i) fetch(i, i);
  if (__all_sync(0xffffffffu, kind == 2)) {
    // values: layout and type alone
#pragma unroll 1
    for (int t = 0; t < steps; t += kDepth)
#pragma unroll
      for (int i = 0; i < kDepth; ++i) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 2) : "memory");
        float x[8];
        read8<TI>(slot + i * 32 * kSlot, x);
        fetch((i + kDepth - 1) % kDepth, kDepth - 1);
        if (left > 0 && store) store8<TO, HALVES>(out, gap, x);
        out += so.row;
        --left;
      }
  } else {
    const bool sums = a.q_mean || a.k_mean;
#pragma unroll 1
    for (int t0 = 0; t0 < run; t0 += seg) {
      uint64_t sum[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll 1
      for (int t = t0; t < t0 + seg && t < steps; t += kDepth)
#pragma unroll
        for (int i = 0; i < kDepth; ++i) {
          asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 2) : "memory");
          __syncwarp();                             // every lane's copies have landed, and the slot refilled below is read
          float x[8];
          read8<TI>(slot + i * 32 * kSlot, x);
          float4 c0v, c1v;                          // (cos, sin) of the lane's 4 pairs
          if (turn) {
            c0v = *reinterpret_cast<const float4*>(turns + i * LPR * 32 + lane * 16);
            c1v = *reinterpret_cast<const float4*>(turns + i * LPR * 32 + LPR * 16 + lane * 16);
          }
          fetch((i + kDepth - 1) % kDepth, kDepth - 1);
          if (norm) {
            uint64_t x2[4] = {pk2(x[0], x[1]), pk2(x[2], x[3]), pk2(x[4], x[5]), pk2(x[6], x[7])};
            uint64_t ss2 = mul2(x2[0], x2[0]);
#pragma unroll
            for (int e = 1; e < 4; ++e) ss2 = fma2(x2[e], x2[e], ss2);
            float sa, sb;
            upk2(ss2, sa, sb);
            float ss = sa + sb;
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            // a value head beside key heads keeps its scale
            const float r = kind < 2 ? rsqrtf(fmaf(ss, a.inv_d, p.eps)) : 1.f;
            const uint64_t r2 = pk2(r, r);
#pragma unroll
            for (int e = 0; e < 4; ++e) upk2(mul2(mul2(x2[e], r2), w2[e]), x[2 * e], x[2 * e + 1]);
          }
          if (turn) {
            const float c[8] = {c0v.x, c0v.y, c0v.z, c0v.w, c1v.x, c1v.y, c1v.z, c1v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int ia = HALVES ? e : 2 * e, ib = HALVES ? e + 4 : 2 * e + 1;
              const float xa = x[ia], xb = x[ib];
              x[ia] = fmaf(xa, c[2 * e], -(xb * c[2 * e + 1]));
              x[ib] = fmaf(xa, c[2 * e + 1], xb * c[2 * e]);
            }
          }
          if (left > 0) {
            if (store) store8<TO, HALVES>(out, gap, x);
            if (sums)
#pragma unroll
              for (int e = 0; e < 4; ++e) sum[e] = add2(sum[e], pk2(x[2 * e], x[2 * e + 1]));
          }
          out += so.row;
          --left;
          --tleft;
        }
      if (sums) {
        // The second sums take the place of the rows.  A lane's 32 bytes lie over other lanes' 16-byte slots too: every
        // lane waits for its own copies and all lanes meet before any writes.
        if (t0 > 0) asm volatile("cp.async.wait_group 0;" ::: "memory");
        if (t0 > 0) __syncwarp();
        float* dst = (t0 > 0 ? reinterpret_cast<float*>(rings + warp * M::kRing) : part + warp * 256) + 8 * l32;
        float v[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) upk2(sum[e], v[2 * e], v[2 * e + 1]);
        *reinterpret_cast<float4*>(dst) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4*>(dst + 4) = make_float4(v[4], v[5], v[6], v[7]);
      }
    }
  }
  if (!a.q_mean && !a.k_mean) return;
  __syncthreads();
  // one thread per (head of the CTA, 64-token half, column); a 128-row block is written by its first half
  for (int i = threadIdx.x; i < wh * kHeads * 2 * LPR * 8; i += kNormThreads) {
    const int hi = i / (2 * LPR * 8), b = (i / (LPR * 8)) & 1, c = i % (LPR * 8);   // c: lane-major position
    const int hq = group * wh * kHeads + hi, hr = hi / kHeads;
    float* m = hq < p.H ? a.q_mean : (hq < p.H + p.Hkv ? a.k_mean : nullptr);
    if (!m || !(hq < p.H ? a.q : a.k)) continue;
    const int blk = hq < p.H ? p.q_block : p.k_block, nblk = (p.S + blk - 1) / blk;
    const int r0 = tile * 128 + 64 * b, n = min(blk, p.S - r0);
    const int l8 = c / 8, e = c & 7;
    if ((blk == 128 && b == 1) || n <= 0 || 8 * l8 >= p.D) continue;
    // the slots of half b: with one warp per run of heads its segments, else the warps of that half, segment 0 of each
    const int at = (hi % kHeads) * LPR * 8 + c;
    float v = 0.f;
    for (int hb = b; hb < (blk == 128 ? 2 : b + 1); ++hb) {
      if (a.wt == 1) v += hb ? reinterpret_cast<const float*>(rings + hr * M::kRing)[at] : part[hr * 256 + at];
      else
        for (int k = 0; k < a.wt / 2; ++k) v += part[(hr * a.wt + hb * (a.wt / 2) + k) * 256 + at];
    }
    const bool tl = HALVES && 8 * l8 < p.rot;
    const int col = tl ? (e < 4 ? 4 * l8 + e : p.rot / 2 + 4 * l8 + e - 4) : 8 * l8 + e;
    m[((int64_t)(hq < p.H ? hq : hq - p.H) * nblk + r0 / blk) * p.D + col] = v / (float)n;
  }
}

// Raises a kernel's shared-memory limit to `bytes`, once per device and size (racing threads repeat it harmlessly).
template <typename K>
bool allow_smem(K kernel, std::atomic<int> (&allowed)[64], int bytes) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  if (allowed[dev].load(std::memory_order_acquire) >= bytes) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
  allowed[dev].store(bytes, std::memory_order_release);
  return true;
}

template <typename TI, typename TO, int LPR, bool HALVES>
int norm_rope_launch(const NormRopeArgs& a, unsigned grid, cudaStream_t st) {
  constexpr int kBytes = NormSmem<TI, LPR>::kBytes;
  static std::atomic<int> allowed[64];
  if (!allow_smem(qk_norm_rope_kernel<TI, TO, LPR, HALVES>, allowed, kBytes)) return DT_ERR_CUDA;
  qk_norm_rope_kernel<TI, TO, LPR, HALVES><<<grid, kNormThreads, kBytes, st>>>(a);
  return launched();
}
template <typename TI, typename TO>
int norm_rope_dispatch(const NormRopeArgs& a, unsigned grid, cudaStream_t st) {
  const bool hv = a.p.pairing == DT_ROPE_HALVES;
  if (a.p.D <= 64) return hv ? norm_rope_launch<TI, TO, 8, true>(a, grid, st) : norm_rope_launch<TI, TO, 8, false>(a, grid, st);
  return hv ? norm_rope_launch<TI, TO, 16, true>(a, grid, st) : norm_rope_launch<TI, TO, 16, false>(a, grid, st);
}

// ------------------------------------------------------------------ block selection
// One CTA: R query blocks of one head against all its key blocks.
//
// Scores on the 64-bit tensor cores (m8n8k4): fp32 operands widen exactly, a
// product of two is exact, and only the sum rounds, at 2^-53.  A warp owns 16
// key blocks at a time and the CTA's R query blocks (padded to 8 with zero rows); the
// queries lie in shared memory as doubles, the keys come from L2 straight into
// the fragments.  The order of a dot product's terms is free, so lane j of a
// quad takes the consecutive columns 4j .. 4j+3 of each 16 for its 4 k-steps:
// 16-byte loads on both sides instead of one element per step.
//
// Then a warp per row finds the topk-th score and writes the chosen blocks in
// increasing order by ballots.  It bins the scores evenly over the row's range and
// ranks the few in the bin that holds the topk-th: digits of the scores' bit
// patterns, which a radix selection bins by, need three passes over the row and put
// most of it into two or three counters in the first (96 us in all on the case
// below, 75 this way; the scores alone are 37 us of the 64-bit pipe).
constexpr int kSelThreads = 256, kSelWarps = kSelThreads / 32;

// order-preserving key of a score; NaN counts as -infinity
__device__ __forceinline__ uint64_t order_key(double x) {
  if (isnan(x)) x = -INFINITY;
  x += 0.0;                                         // -0 and +0 are equal
  const int64_t b = __double_as_longlong(x);
  return (uint64_t)(b < 0 ? ~b : (b | (int64_t)0x8000000000000000ull));
}
// the score of an order key
__device__ __forceinline__ double key_score(uint64_t k) {
  return __longlong_as_double((k >> 63) ? (int64_t)(k & 0x7fffffffffffffffull) : (int64_t)~k);
}
// The bin, counted from the highest, in which the running count of a warp's 256-bin histogram reaches `want` (>= 1, at
// most the total); want becomes the rank inside it, size its count.  Lane l sums bins 255-8l .. 248-8l.
__device__ __forceinline__ int find_bin(const uint32_t* hs, int lane, int& want, uint32_t& size) {
  uint32_t c[8], mine = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) mine += c[e] = hs[255 - 8 * lane - e];
  uint32_t run = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, run, o);
    if (lane >= o) run += u;
  }
  const int src = __ffs(__ballot_sync(0xffffffffu, run >= (uint32_t)want)) - 1;
  uint32_t before = run - mine, n = 0;
  int bin = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if (n == 0 && before + c[e] >= (uint32_t)want) { bin = 255 - 8 * lane - e; n = c[e]; }
    else if (n == 0) before += c[e];
  }
  size = __shfl_sync(0xffffffffu, n, src);
  want -= (int)__shfl_sync(0xffffffffu, before, src);
  return __shfl_sync(0xffffffffu, bin, src);
}
__device__ __forceinline__ void mma_f64(double (&c)[2], double a, double b) {
  asm volatile("mma.sync.aligned.m8n8k4.row.col.f64.f64.f64.f64 {%0, %1}, {%2}, {%3}, {%0, %1};"
               : "+d"(c[0]), "+d"(c[1]) : "d"(a), "d"(b));
}

__host__ __device__ inline int select_ldq(int D) { return (D + 15) / 16 * 16 + 2; }   // doubles; +2 spreads the banks

constexpr int kSelRows = 8;                         // query blocks of a CTA at most: one MMA row tile

__global__ void __launch_bounds__(kSelThreads, 4) block_select_kernel(const dt_select_params p, const float* q_mean,
                                                                      const float* k_mean, int32_t* idx,
                                                                      int32_t* count, int qtiles, int R) {
  extern __shared__ double sm[];
  __shared__ uint32_t hist[kSelWarps][256];
  const int D = p.D, nk = p.nk, ldq = select_ldq(D);
  double* sQ = sm;                                  // [kSelRows][ldq], zeros past the rows and columns
  uint64_t* keys = reinterpret_cast<uint64_t*>(sQ + kSelRows * ldq);     // [R][nk]
  uint8_t* bins = reinterpret_cast<uint8_t*>(keys + (int64_t)R * nk);    // [R][nk], see below
  const int h = blockIdx.x / qtiles, q0 = (blockIdx.x - h * qtiles) * R;
  const int rows = min(R, p.nq - q0);
  const float* km = k_mean + (int64_t)(h / (p.H / p.Hkv)) * nk * D;
  const float* qm = q_mean + ((int64_t)h * p.nq + q0) * D;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, j = lane & 3;            // a fragment's row (query or key) and quad lane
  const double scale = 1.0 / sqrt((double)D);

  for (int i = tid; i < kSelRows * ldq; i += kSelThreads) {
    const int r = i / ldq, c = i - r * ldq;
    sQ[i] = r < rows && c < D ? (double)qm[(int64_t)r * D + c] : 0.0;
  }
  __syncthreads();
  for (int n0 = 16 * warp; n0 < nk; n0 += 16 * kSelWarps) {
    double acc[2][2] = {};
    const float* kr[2];
#pragma unroll
    for (int n = 0; n < 2; ++n) kr[n] = km + (int64_t)min(n0 + 8 * n + g, nk - 1) * D;
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
    for (int k0 = 4 * j; k0 - 4 * j < D; k0 += 16) {
      float4 kb[2];
#pragma unroll
      for (int n = 0; n < 2; ++n) kb[n] = k0 < D ? __ldg(reinterpret_cast<const float4*>(kr[n] + k0)) : zero;
      const double2* src = reinterpret_cast<const double2*>(sQ + g * ldq + k0);
      const double2 u = src[0], v = src[1];
      const double qa[4] = {u.x, u.y, v.x, v.y};
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int n = 0; n < 2; ++n)
          mma_f64(acc[n], qa[t], t == 0 ? kb[n].x : (t == 1 ? kb[n].y : (t == 2 ? kb[n].z : kb[n].w)));
    }
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int c = n0 + 8 * n + 2 * j + e;
        if (g < rows && c < nk) keys[(int64_t)g * nk + c] = order_key(acc[n][e] * scale);
      }
  }
  __syncthreads();

  const int topk = min(p.topk, nk), lo_keep = p.keep_first, hi_keep = nk - p.keep_last;
  const uint32_t below = (1u << lane) - 1u;
  for (int r = warp; r < rows; r += kSelWarps) {
    uint64_t* kr = keys + (int64_t)r * nk;
    uint32_t* hs = hist[warp];
    // Keys kept by position get the highest key; under a margin, keys below the floor the lowest (0, which no
    // score has), and are never chosen.
    const uint64_t forced = ~0ull;
    uint64_t kmax = 0, kmin = ~0ull;
#pragma unroll 4
    for (int i = lane; i < nk; i += 32) {
      kmax = max(kmax, kr[i]);
      kmin = min(kmin, kr[i]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      kmax = max(kmax, (uint64_t)__shfl_xor_sync(0xffffffffu, kmax, o));
      kmin = min(kmin, (uint64_t)__shfl_xor_sync(0xffffffffu, kmin, o));
    }
    const uint64_t floor_key = p.margin < INFINITY && nk > 0 ? order_key(key_score(kmax) - p.margin) : 0;
    // The last key to be taken: (kt, it), the topk-th in the order of scores (highest first) and indices.  First by
    // bins 1 .. 254 over the row's range (0: below the floor, 255: kept by position): a bin is a monotone function of
    // the score (conversion, difference, product and truncation all are), so the bins above the topk-th key's are
    // taken whole, and its own usually holds a few keys.
    const float fmin = (float)key_score(kmin), per = 253.f / ((float)key_score(kmax) - fmin);
    const bool binned = topk > 0 && per < INFINITY && per > 0.f;   // finite and not all equal
    uint8_t* br = bins + (int64_t)r * nk;
    int want = topk;                                // 1-based rank of that key among those still in question
    for (int i = lane; i < 256; i += 32) hs[i] = 0;
    __syncwarp();
    int held = 0, live = 0;                         // keys kept by position, and other keys above the floor
#pragma unroll 4
    for (int i = lane; i < nk; i += 32) {
      const uint64_t k = kr[i];
      int b = 0;
      if (i < lo_keep || i >= hi_keep) {
        kr[i] = forced;
        b = 255;
        ++held;
      } else if (k < floor_key) {
        kr[i] = 0;
      } else {
        ++live;
        if (binned) {
          b = 1 + min(253, (int)(((float)key_score(k) - fmin) * per));
          atomicAdd(&hs[b], 1u);
        }
      }
      br[i] = (uint8_t)b;
    }
    held = __reduce_add_sync(0xffffffffu, held);
    live = __reduce_add_sync(0xffffffffu, live);
    __syncwarp();
    want -= held;
    uint64_t kt = 0;
    int it = nk, tb = 0;                            // tb > 0: only the keys of bin tb need comparing
    bool done = false;
    if (topk == 0 || live <= want) {
      kt = 1;                                       // everything above the floor
      done = true;
    } else if (want <= 0) {
      kt = forced;                                  // the kept ones alone
      done = true;
    } else if (binned) {
      uint32_t size;
      tb = find_bin(hs, lane, want, size);
      done = size <= 32;
      if (done) {
        // the bin's keys, in order of index, one per lane (the histogram is done with)
        __syncwarp();
        int n = 0;
        for (int i0 = 0; i0 < nk; i0 += 32) {
          const bool in = i0 + lane < nk && br[i0 + lane] == tb;
          const uint32_t m = __ballot_sync(0xffffffffu, in);
          if (in) hs[n + __popc(m & below)] = i0 + lane;
          n += __popc(m);
        }
        __syncwarp();
        const int at = lane < n ? (int)hs[lane] : 0;
        const uint64_t mine = lane < n ? kr[at] : 0;
        int rank = 1;                               // place among them
        for (int o = 0; o < n; ++o) {
          const uint64_t v = __shfl_sync(0xffffffffu, mine, o);
          rank += v > mine || (v == mine && o < lane);
        }
        const int src = __ffs(__ballot_sync(0xffffffffu, lane < n && rank == want)) - 1;
        kt = __shfl_sync(0xffffffffu, mine, src);
        it = __shfl_sync(0xffffffffu, at, src);
      } else {
        tb = 0;
      }
    }
    if (!done) {
      // Many equal or nearly equal keys, or infinities: 8 bits of the key a pass from the highest bit in which the
      // row's keys differ, ending as soon as all keys of a digit are wanted.  Where keys equal to the last are left
      // over, the lowest indices take them.
      uint64_t all_and = ~0ull, all_or = 0;
      for (int i = lane; i < nk; i += 32) {
        all_and &= kr[i];
        all_or |= kr[i];
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        all_and &= __shfl_xor_sync(0xffffffffu, all_and, o);
        all_or |= __shfl_xor_sync(0xffffffffu, all_or, o);
      }
      want = topk;                                  // the kept keys count here: they are the highest
      const uint64_t differ = all_and ^ all_or;
      int shift = differ ? 64 - __clzll(differ) : 0;        // bits below `shift` are still open
      uint64_t prefix = shift == 64 ? 0ull : all_and >> shift << shift;
      uint32_t size = nk;
      while (shift > 0 && size != (uint32_t)want) {
        const int bits = min(8, shift);
        const uint64_t hi = shift == 64 ? 0ull : ~0ull << shift;
        shift -= bits;
        __syncwarp();
        for (int i = lane; i < 256; i += 32) hs[i] = 0;
        __syncwarp();
        for (int i = lane; i < nk; i += 32) {
          const uint64_t k = kr[i];
          if ((k & hi) == prefix) atomicAdd(&hs[(uint32_t)(k >> shift) & ((1u << bits) - 1u)], 1u);
        }
        __syncwarp();
        prefix |= (uint64_t)find_bin(hs, lane, want, size) << shift;
      }
      kt = prefix;                                  // with bits open, every key above it is wanted too
      if (shift == 0) {
        int left = want;                            // of the keys equal to kt
        for (int i0 = 0; i0 < nk && left > 0; i0 += 32) {
          const uint32_t m = __ballot_sync(0xffffffffu, i0 + lane < nk && kr[i0 + lane] == kt);
          if (__popc(m) >= left) it = i0 + (int)__fns(m, 0, left);
          left -= __popc(m);
        }
      }
    }
    int32_t* out = idx + ((int64_t)h * p.nq + q0 + r) * p.topk;
    int n = 0;
    if (tb > 0) {
#pragma unroll 4
      for (int i0 = 0; i0 < nk; i0 += 32) {
        const int i = i0 + lane, b = i < nk ? br[i] : 0;
        bool take = b > tb;
        if (b == tb) {
          const uint64_t k = kr[i];
          take = k > kt || (k == kt && i <= it);
        }
        const uint32_t m = __ballot_sync(0xffffffffu, take);
        if (take) out[n + __popc(m & below)] = i;
        n += __popc(m);
      }
    } else {
#pragma unroll 2
      for (int i0 = 0; i0 < nk; i0 += 32) {
        const int i = i0 + lane;
        const uint64_t k = i < nk && topk > 0 ? kr[i] : 0;
        const bool take = k != 0 && (k > kt || (k == kt && i <= it));
        const uint32_t m = __ballot_sync(0xffffffffu, take);
        if (take) out[n + __popc(m & below)] = i;
        n += __popc(m);
      }
    }
    for (int i = n + lane; i < p.topk; i += 32) out[i] = -1;
    if (lane == 0) count[(int64_t)h * p.nq + q0 + r] = n;
    __syncwarp();                                   // the histogram is cleared for the next row
  }
}

constexpr int kSelSmemMax = 160 * 1024;            // one row of DT_SELECT_MAX_BLOCKS keys and bins, queries of D = 128

size_t select_smem(int R, int D, int nk) {
  return (size_t)kSelRows * select_ldq(D) * 8 + (size_t)R * nk * 9;
}

}  // namespace

int launch_rope_table(const RopeTableArgs& a, cudaStream_t stream) {
  rope_table_kernel<<<(unsigned)cdiv(a.S, kRopeTokens), kRopeThreads, 0, stream>>>(a);
  return launched();
}

int launch_qk_norm_rope(NormRopeArgs a, int sms, cudaStream_t stream) {
  const dt_norm_rope_params& p = a.p;
  const int64_t tiles = cdiv(p.S, 128);
  const int heads = p.H + 2 * p.Hkv;
  const int runs = cdiv(heads, p.D <= 64 ? 4 : 2);           // a warp's heads: 32 lanes / lanes per row
  // warps per run of heads: one, or more while the CTAs are fewer than two per SM
  a.wt = 1;
  while (a.wt < kNormWarps && tiles * cdiv(runs * a.wt, kNormWarps) < 2 * sms) a.wt *= 2;
  a.groups = cdiv(runs * a.wt, kNormWarps);
  a.inv_d = 1.f / (float)p.D;
  if (tiles * a.groups >= (int64_t)1 << 31) return DT_ERR_INVALID;
  const unsigned grid = (unsigned)(tiles * a.groups);
  if (p.in_type == DT_TYPE_BF16) return norm_rope_dispatch<__nv_bfloat16, __nv_bfloat16>(a, grid, stream);
  if (p.in_type == DT_TYPE_F16)
    return p.out_type == DT_TYPE_F16 ? norm_rope_dispatch<__half, __half>(a, grid, stream)
                                     : norm_rope_dispatch<__half, __nv_bfloat16>(a, grid, stream);
  return p.out_type == DT_TYPE_F32 ? norm_rope_dispatch<float, float>(a, grid, stream)
                                   : norm_rope_dispatch<float, __nv_bfloat16>(a, grid, stream);
}

int launch_block_select(const dt_select_params& p, const float* q_mean, const float* k_mean, int32_t* idx,
                        int32_t* count, cudaStream_t stream) {
  // Query blocks per CTA: as many as there are, up to 8, while the keys of the rows leave room for four CTAs on an SM
  // (some score while others select), and one at the least.  Measured at D = 128: 40 heads of 256 x 512 blocks 76 us
  // with 8 rows, 124 with 4, 217 with 2, and 79 with 16 rows on two CTAs an SM.  Rows of a thousand blocks and more
  // get fewer than is best: 16 x 1,024 blocks 39 us with the 4 of this rule, 31 with 8; 16 x 3,000 206 with 1, 130
  // with 2; 32 x 4,096 475 with 1, 341 with 4; 16 heads of 128 x 8,192 1,729 with 1, 1,517 with 2.
  int R = kSelRows;
  while (R > 1 && (R / 2 >= p.nq || select_smem(R, p.D, p.nk) > 46 * 1024)) R /= 2;
  const size_t smem = select_smem(R, p.D, p.nk);
  // the most that any call asks for, so that calls of other sizes never lower it under a call in flight
  static std::atomic<int> allowed[64];
  if (!allow_smem(block_select_kernel, allowed, kSelSmemMax)) return DT_ERR_CUDA;
  const int qtiles = cdiv(p.nq, R);
  block_select_kernel<<<(unsigned)(p.H * qtiles), kSelThreads, smem, stream>>>(p, q_mean, k_mean, idx, count, qtiles, R);
  return launched();
}

}  // namespace dt

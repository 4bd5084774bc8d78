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

#include "../../include/dt.h"
#include "token_ops.h"

namespace dt {
namespace {

int launched() { return cudaGetLastError() == cudaSuccess ? DT_OK : DT_ERR_CUDA; }
int cdiv(int a, int b) { return (a + b - 1) / b; }

// ------------------------------------------------------------------ rotation table
// cos and sin of 2 pi t, t = pos * turns.  The product and its reduction to
// the nearest whole turn are in 64 bits (t - rint(t) is exact), so the angle of
// a position of 2^31 still has 2^-22 turns of error or less.  The fraction is
// split into two floats: sincospif of the high part, then the angle-sum
// formula to first order for the low one (|low| <= 2^-25 turns, so the
// second-order term is below 2^-46): full fp32 accuracy without the 64-bit
// sincos, which alone would cost four times the table's HBM time.
// One thread per two pairs of a token (16 bytes of the table).
__global__ void __launch_bounds__(256) rope_table_kernel(const __grid_constant__ RopeTableArgs a) {
  const int halfp = (a.pairs + 1) / 2;
  const int64_t n = (int64_t)a.S * halfp;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
    const int s = (int)(i / halfp), p0 = 2 * (int)(i - (int64_t)s * halfp);
    float out[4];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int pr = p0 + e < a.pairs ? p0 + e : p0;
      const double t = (double)__ldg(a.pos + (int64_t)a.axis[pr] * a.S + s) * a.turns[pr];
      const double f = t - rint(t);
      const float hi = (float)f, lo = (float)(f - (double)hi);
      float sn, cs;
      sincospif(2.f * hi, &sn, &cs);
      const float d = 6.2831853071795865f * lo;
      out[2 * e] = fmaf(-d, sn, cs);
      out[2 * e + 1] = fmaf(d, cs, sn);
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
// 8 elements as two groups of 4; one 16-byte access where they are adjacent 16-bit elements
template <typename T, bool SPLIT>
__device__ __forceinline__ void load8(const T* row, int c0, int c1, typename Vec4<T>::type (&v)[2]) {
  using V = typename Vec4<T>::type;
  if (sizeof(T) == 2 && !SPLIT) {
    const uint4 u = __ldcs(reinterpret_cast<const uint4*>(row + c0));
    *reinterpret_cast<uint4*>(v) = u;
  } else {
    v[0] = __ldcs(reinterpret_cast<const V*>(row + c0));
    v[1] = __ldcs(reinterpret_cast<const V*>(row + c1));
  }
}
template <typename T, bool SPLIT>
__device__ __forceinline__ void store8(T* row, int c0, int c1, const float* x) {
  using V = typename Vec4<T>::type;
  V v[2] = {narrow4<T>(x), narrow4<T>(x + 4)};
  if (sizeof(T) == 2 && !SPLIT) {
    *reinterpret_cast<uint4*>(row + c0) = *reinterpret_cast<const uint4*>(v);
  } else {
    *reinterpret_cast<V*>(row + c0) = v[0];
    *reinterpret_cast<V*>(row + c1) = v[1];
  }
}

// A CTA owns 128 consecutive tokens and walks a run of heads (of all parts:
// queries, then keys, then values), so the tokens' 64 KB of rotation (D = 128)
// come from L2 once per CTA and from L1 for its other heads: read per head from
// L2 they would be twice the bytes of the 16-bit rows.  LPR lanes hold a row, 8
// elements each.  An element's partner in its pair is always in the same
// thread (HALVES: 4 elements from each half), so the row's sum of squares is
// the only exchange, by shuffles.  A head's rows are loaded before they are
// stored and by the thread that stores them (in-place calls).  Block means:
// sums over a thread's rows, then over the lanes of the same columns, then
// over the warps through shared memory, in a fixed order.
constexpr int kNormThreads = 512;

template <typename TI, typename TO, int LPR, bool HALVES>
__global__ void __launch_bounds__(kNormThreads, 2) qk_norm_rope_kernel(const __grid_constant__ NormRopeArgs a) {
  constexpr int kRowsPerPass = kNormThreads / LPR;
  constexpr int R = 64 / kRowsPerPass;              // rows of a 64-row half a thread owns: 1 for LPR 8, 2 for 16
  constexpr int kWarps = kNormThreads / 32;
  __shared__ float part[2][kWarps][LPR * 8];        // block sums per warp, halves of the tile apart
  const dt_norm_rope_params& p = a.p;
  const int s0 = blockIdx.x * 128;
  const int lane = threadIdx.x % LPR, rbase = threadIdx.x / LPR, warp = threadIdx.x / 32;
  const bool on = 8 * lane < p.D;
  const bool turned = 8 * lane < p.rot;
  const int c0 = HALVES && turned ? 4 * lane : 8 * lane;
  const int c1 = HALVES && turned ? p.rot / 2 + 4 * lane : 8 * lane + 4;
  const int heads = p.H + 2 * p.Hkv;
  const int h_end = min(heads, (int)(blockIdx.y + 1) * a.heads_per_cta);

  for (int hh = blockIdx.y * a.heads_per_cta; hh < h_end; ++hh) {
    const int kind = hh < p.H ? 0 : (hh < p.H + p.Hkv ? 1 : 2);
    const int h = kind == 0 ? hh : (kind == 1 ? hh - p.H : hh - p.H - p.Hkv);
    const TI* in = static_cast<const TI*>(kind == 0 ? a.q : (kind == 1 ? a.k : a.v));
    TO* out = static_cast<TO*>(kind == 0 ? a.Q : (kind == 1 ? a.K : a.V));
    float* mean = kind == 0 ? a.q_mean : (kind == 1 ? a.k_mean : nullptr);
    if (!in) continue;
    const dt_strides si = kind == 0 ? p.q_in : (kind == 1 ? p.k_in : p.v_in);
    const dt_strides so = kind == 0 ? p.q_out : (kind == 1 ? p.k_out : p.v_out);
    const float* w = kind == 0 ? a.wq : a.wk;
    in += h * si.head;
    out += h * so.head;

    float wv[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
    if (kind < 2 && p.norm && w && on) {
      widen(__ldg(reinterpret_cast<const float4*>(w + c0)), wv);
      widen(__ldg(reinterpret_cast<const float4*>(w + c1)), wv + 4);
    }
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      typename Vec4<TI>::type raw[R][2];
      float4 cs[R][2];                              // (cos, sin) of the thread's 4 pairs
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const int s = s0 + 64 * b + rbase + j * kRowsPerPass;
        if (on && s < p.S) load8<TI, HALVES>(in + s * si.row, c0, c1, raw[j]);
        else { raw[j][0] = {}; raw[j][1] = {}; }
        if (kind < 2 && turned && s < p.S) {
          const float4* t = reinterpret_cast<const float4*>(a.table + ((int64_t)s * (p.rot / 2) + 4 * lane) * 2);
          cs[j][0] = __ldg(t);
          cs[j][1] = __ldg(t + 1);
        } else {
          cs[j][0] = cs[j][1] = make_float4(1.f, 0.f, 1.f, 0.f);
        }
      }
      float sum[8] = {};
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const int s = s0 + 64 * b + rbase + j * kRowsPerPass;
        float x[8];
        widen4<TI>(raw[j][0], x);
        widen4<TI>(raw[j][1], x + 4);
        if (kind < 2) {
          if (p.norm) {
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            const float r = rsqrtf(ss / (float)p.D + p.eps);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = x[e] * r * wv[e];
          }
          if (turned) {
            const float t[8] = {cs[j][0].x, cs[j][0].y, cs[j][0].z, cs[j][0].w,
                                cs[j][1].x, cs[j][1].y, cs[j][1].z, cs[j][1].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int ia = HALVES ? e : 2 * e, ib = HALVES ? e + 4 : 2 * e + 1;
              const float xa = x[ia], xb = x[ib];
              x[ia] = fmaf(xa, t[2 * e], -(xb * t[2 * e + 1]));
              x[ib] = fmaf(xa, t[2 * e + 1], xb * t[2 * e]);
            }
          }
        }
        if (on && s < p.S) {
          if (a.store[kind]) store8<TO, HALVES>(out + s * so.row, c0, c1, x);
#pragma unroll
          for (int e = 0; e < 8; ++e) sum[e] += x[e];
        }
      }
      if (mean) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
#pragma unroll
          for (int o = LPR; o < 32; o <<= 1) sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], o);
        }
        if ((threadIdx.x & 31) < LPR) {
          *reinterpret_cast<float4*>(&part[b][warp][8 * lane]) = make_float4(sum[0], sum[1], sum[2], sum[3]);
          *reinterpret_cast<float4*>(&part[b][warp][8 * lane + 4]) = make_float4(sum[4], sum[5], sum[6], sum[7]);
        }
      }
    }
    if (mean) {
      __syncthreads();
      const int blk = kind == 0 ? p.q_block : p.k_block;
      const int nblk = (p.S + blk - 1) / blk;
      for (int i = threadIdx.x; i < 2 * LPR * 8; i += kNormThreads) {
        const int b = i / (LPR * 8), c = i - b * (LPR * 8);      // c: lane-major position
        const int r0 = s0 + 64 * b, n = min(blk, p.S - r0);
        const int l8 = c / 8, e = c & 7;
        if ((blk == 128 && b == 1) || n <= 0 || 8 * l8 >= p.D) continue;
        float v = 0.f;
        for (int k = 0; k < kWarps; ++k) v += part[b][k][c];
        if (blk == 128)
          for (int k = 0; k < kWarps; ++k) v += part[1][k][c];
        const bool tl = HALVES && 8 * l8 < p.rot;
        const int col = tl ? (e < 4 ? 4 * l8 + e : p.rot / 2 + 4 * l8 + e - 4) : 8 * l8 + e;
        mean[((int64_t)h * nblk + r0 / blk) * p.D + col] = v / (float)n;
      }
      __syncthreads();
    }
  }
}

template <typename TI, typename TO>
void norm_rope_dispatch(const NormRopeArgs& a, dim3 grid, cudaStream_t st) {
  const bool hv = a.p.pairing == DT_ROPE_HALVES;
#define DT_NR(LPR)                                                                                   \
  (hv ? qk_norm_rope_kernel<TI, TO, LPR, true><<<grid, kNormThreads, 0, st>>>(a)                      \
      : qk_norm_rope_kernel<TI, TO, LPR, false><<<grid, kNormThreads, 0, st>>>(a))
  if (a.p.D <= 64) DT_NR(8);
  else DT_NR(16);
#undef DT_NR
}

// ------------------------------------------------------------------ block selection
// One CTA: kRows query blocks of one head against all its key blocks.
// Scores: 64-bit FMAs (B200 issues half as many as fp32 ones) over tiles of 64
// key blocks staged in shared memory as doubles, one key block and a quarter of
// the rows per thread; then a warp per row finds the topk-th largest by a
// radix selection over order-preserving 64-bit keys, and writes the chosen
// blocks in increasing order by ballots.
constexpr int kSelThreads = 256;
constexpr int kSelTile = 64;                        // key blocks per staged tile
constexpr int kSelPad = 1;                          // doubles between staged rows (bank spread)

// order-preserving key of a score; NaN counts as -infinity
__device__ __forceinline__ uint64_t order_key(double x) {
  if (isnan(x)) x = -INFINITY;
  x += 0.0;                                         // -0 and +0 are equal
  const int64_t b = __double_as_longlong(x);
  return (uint64_t)(b < 0 ? ~b : (b | (int64_t)0x8000000000000000ull));
}

template <int ROWS>
__global__ void __launch_bounds__(kSelThreads) block_select_kernel(const dt_select_params p, const float* q_mean,
                                                                   const float* k_mean, int32_t* idx,
                                                                   int32_t* count, int qtiles) {
  extern __shared__ double sm[];
  const int D = p.D, ld = D + kSelPad;
  double* sQ = sm;                                  // [ROWS][D]
  double* sK = sQ + ROWS * D;                       // [kSelTile][ld]
  uint64_t* keys = reinterpret_cast<uint64_t*>(sK + kSelTile * ld);      // [ROWS][nk]
  __shared__ uint32_t hist[kSelThreads / 32][256];
  const int h = blockIdx.x / qtiles, q0 = (blockIdx.x - h * qtiles) * ROWS;
  const int rows = min(ROWS, p.nq - q0);
  const float* km = k_mean + (int64_t)(h / (p.H / p.Hkv)) * p.nk * D;
  const float* qm = q_mean + ((int64_t)h * p.nq + q0) * D;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const double scale = 1.0 / sqrt((double)D);

  for (int i = tid; i < ROWS * D; i += kSelThreads) sQ[i] = i < rows * D ? (double)qm[i] : 0.0;
  for (int k0 = 0; k0 < p.nk; k0 += kSelTile) {
    const int nt = min(kSelTile, p.nk - k0);
    __syncthreads();
    for (int i = tid; i < kSelTile * (D / 4); i += kSelThreads) {
      const int r = i / (D / 4), c = 4 * (i - r * (D / 4));
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < nt) v = __ldg(reinterpret_cast<const float4*>(km + (int64_t)(k0 + r) * D + c));
      double* d = sK + r * ld + c;
      d[0] = v.x; d[1] = v.y; d[2] = v.z; d[3] = v.w;
    }
    __syncthreads();
    // thread: key column tid % 64, rows tid/64, tid/64 + 4, ...
    constexpr int RT = ROWS >= 4 ? ROWS / 4 : 1;
    const int col = tid & 63, rg = tid >> 6;
    if (rg < ROWS) {
      double acc[RT] = {};
      const double* kr = sK + col * ld;
#pragma unroll 4
      for (int d = 0; d < D; ++d) {
        const double kv = kr[d];
#pragma unroll
        for (int j = 0; j < RT; ++j) acc[j] = fma(sQ[(rg + 4 * j) * D + d], kv, acc[j]);
      }
      if (col < nt)
#pragma unroll
        for (int j = 0; j < RT; ++j) keys[(int64_t)(rg + 4 * j) * p.nk + k0 + col] = order_key(acc[j] * scale);
    }
  }
  __syncthreads();

  for (int r = warp; r < rows; r += kSelThreads / 32) {
    uint64_t* kr = keys + (int64_t)r * p.nk;
    const uint64_t forced = ~0ull;                  // above every score's key
    const int lo_keep = p.keep_first, hi_keep = p.nk - p.keep_last;
    uint64_t best = 0;
    for (int i = lane; i < p.nk; i += 32) best = max(best, kr[i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) best = max(best, (uint64_t)__shfl_xor_sync(0xffffffffu, best, o));
    uint64_t floor_key = 0;
    if (p.margin < INFINITY && p.nk > 0) {
      const int64_t b = (best >> 63) ? (int64_t)(best & 0x7fffffffffffffffull) : (int64_t)~best;
      floor_key = order_key(__longlong_as_double(b) - p.margin);
    }
    __syncwarp();
    for (int i = lane; i < p.nk; i += 32) {
      if (i < lo_keep || i >= hi_keep) kr[i] = forced;
      else if (kr[i] < floor_key) kr[i] = 0;         // dropped: below every key that stays
    }
    __syncwarp();
    // the topk-th largest key, 8 bits at a time: `prefix` holds the bits found, `want` the rank inside them
    const int topk = min(p.topk, p.nk);
    uint64_t prefix = 0;
    int want = topk;                                // 1-based rank among keys that match the prefix
    for (int shift = 56; shift >= 0 && topk > 0; shift -= 8) {
      for (int i = lane; i < 256; i += 32) hist[warp][i] = 0;
      __syncwarp();
      const uint64_t himask = shift == 56 ? 0ull : (~0ull << (shift + 8));
      for (int i = lane; i < p.nk; i += 32)
        if ((kr[i] & himask) == (prefix & himask)) atomicAdd(&hist[warp][(kr[i] >> shift) & 255], 1u);
      __syncwarp();
      // lane l holds bins 255-8l .. 248-8l (descending); find the bin where the running count reaches want
      uint32_t mine = 0;
      for (int e = 0; e < 8; ++e) mine += hist[warp][255 - 8 * lane - e];
      uint32_t run = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += u;
      }
      const uint32_t hit = __ballot_sync(0xffffffffu, run >= (uint32_t)want);
      const int src = __ffs(hit) - 1;
      uint32_t before = run - mine;
      int bin = 0, left = 0;
      if (lane == src) {
        for (int e = 0; e < 8; ++e) {
          const uint32_t c = hist[warp][255 - 8 * lane - e];
          if (before + c >= (uint32_t)want) { bin = 255 - 8 * lane - e; left = want - (int)before; break; }
          before += c;
        }
      }
      bin = __shfl_sync(0xffffffffu, bin, src);
      want = __shfl_sync(0xffffffffu, left, src);
      prefix |= (uint64_t)bin << shift;
      __syncwarp();
    }
    // chosen: key > prefix, or the first `want` equal to it; key 0 is never chosen (dropped by the margin)
    int32_t* out = idx + ((int64_t)h * p.nq + q0 + r) * p.topk;
    int n = 0, eq = 0;
    for (int i0 = 0; i0 < p.nk && topk > 0; i0 += 32) {
      const int i = i0 + lane;
      const uint64_t k = i < p.nk ? kr[i] : 0;
      const bool same = i < p.nk && k == prefix;
      const uint32_t below = (1u << lane) - 1u;
      const uint32_t em = __ballot_sync(0xffffffffu, same);
      const bool take = i < p.nk && k != 0 && (k > prefix || (same && eq + __popc(em & below) < want));
      const uint32_t tm = __ballot_sync(0xffffffffu, take);
      if (take) out[n + __popc(tm & below)] = i;
      n += __popc(tm);
      eq += __popc(em);
    }
    for (int i = n + lane; i < p.topk; i += 32) out[i] = -1;
    if (lane == 0) count[(int64_t)h * p.nq + q0 + r] = n;
  }
}

size_t select_smem(int rows, int D, int nk) {
  return ((size_t)rows * D + (size_t)kSelTile * (D + kSelPad) + (size_t)rows * nk) * 8;
}

template <int ROWS>
int select_launch(const dt_select_params& p, const float* qm, const float* km, int32_t* idx, int32_t* count,
                  cudaStream_t st) {
  const size_t smem = select_smem(ROWS, p.D, p.nk);
  if (cudaFuncSetAttribute(block_select_kernel<ROWS>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
      cudaSuccess)
    return DT_ERR_CUDA;
  const int qtiles = cdiv(p.nq, ROWS);
  block_select_kernel<ROWS><<<(unsigned)(p.H * qtiles), kSelThreads, smem, st>>>(p, qm, km, idx, count, qtiles);
  return launched();
}

}  // namespace

int launch_rope_table(const RopeTableArgs& a, cudaStream_t stream) {
  const int64_t n = (int64_t)a.S * ((a.pairs + 1) / 2);
  const int64_t grid = (n + 255) / 256;
  rope_table_kernel<<<(unsigned)(grid < (1 << 30) ? grid : (1 << 30)), 256, 0, stream>>>(a);
  return launched();
}

int launch_qk_norm_rope(NormRopeArgs a, int sms, cudaStream_t stream) {
  const dt_norm_rope_params& p = a.p;
  const int tiles = cdiv(p.S, 128), heads = p.H + 2 * p.Hkv;
  // heads a CTA walks with one read of the rotation: as many as still leave every SM a few CTAs
  int64_t per = (int64_t)tiles * heads / (4 * sms);
  a.heads_per_cta = (int)(per < 1 ? 1 : (per > 8 ? 8 : per));
  const dim3 grid(tiles, cdiv(heads, a.heads_per_cta));
  a.store[0] = a.Q != nullptr;
  a.store[1] = a.K != nullptr;
  a.store[2] = a.V != nullptr;
  if (p.in_type == DT_TYPE_BF16) norm_rope_dispatch<__nv_bfloat16, __nv_bfloat16>(a, grid, stream);
  else if (p.in_type == DT_TYPE_F16 && p.out_type == DT_TYPE_F16) norm_rope_dispatch<__half, __half>(a, grid, stream);
  else if (p.in_type == DT_TYPE_F16) norm_rope_dispatch<__half, __nv_bfloat16>(a, grid, stream);
  else if (p.out_type == DT_TYPE_F32) norm_rope_dispatch<float, float>(a, grid, stream);
  else norm_rope_dispatch<float, __nv_bfloat16>(a, grid, stream);
  return launched();
}

int launch_block_select(const dt_select_params& p, const float* q_mean, const float* k_mean, int32_t* idx,
                        int32_t* count, cudaStream_t stream) {
  // rows per CTA: as many as their keys fit in shared memory (the K tile is then staged for more rows)
  constexpr size_t kMax = 200 * 1024;
  if (p.nq > 8 && select_smem(16, p.D, p.nk) <= kMax) return select_launch<16>(p, q_mean, k_mean, idx, count, stream);
  if (p.nq > 2 && select_smem(8, p.D, p.nk) <= kMax) return select_launch<8>(p, q_mean, k_mean, idx, count, stream);
  return select_launch<1>(p, q_mean, k_mean, idx, count, stream);
}

}  // namespace dt

// api.cu -- extern "C" device entry points of libdt: argument validation,
// TMA descriptor encoding and kernel launches.  No allocation happens here.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>
#include <cmath>
#include <cstring>

#include "../../include/dt.h"
#include "attn_fused.h"
#include "attn_sparse.h"
#include "geometry.h"
#include "state_ops.h"
#include "token_ops.h"

namespace {

std::atomic<long long> g_wait_limit_ns{2000000000ll};

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int sm_count(int* out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DT_ERR_CUDA;
  static int cached[64] = {0};
  if (dev >= 0 && dev < 64 && cached[dev] > 0) { *out = cached[dev]; return DT_OK; }
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return DT_ERR_CUDA;
  if (dev >= 0 && dev < 64) cached[dev] = n;
  *out = n;
  return DT_OK;
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  if (!fn) {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(f);
  }
  return fn;
}

// bf16 [H][S][D] viewed as a 3-D tensor (D, S, H); box (bw, 128, 1).
bool encode_qkv(CUtensorMap* m, const void* base, int H, int S, int D, int bw, CUtensorMapSwizzle sw) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)S, (cuuint64_t)H};
  cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)S * D * 2};
  cuuint32_t box[3] = {(cuuint32_t)bw, 128u, 1u};
  cuuint32_t estr[3] = {1u, 1u, 1u};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool shape_ok(int H, int S, int D) {
  if (H < 0 || S < 0) return false;
  // int32 row indexing inside the kernels: H*S*D and rows of the cache fit
  if ((int64_t)H * S * (int64_t)D >= (int64_t)1 << 31) return false;
  return true;
}

}  // namespace

extern "C" int dt_set_wait_limit_ns(int64_t ns) {
  g_wait_limit_ns.store(ns < 0 ? 0 : ns);
  return DT_OK;
}

namespace {
int fused_step(const dt_plan_params* p, int32_t head_begin, int32_t head_count, const uint8_t* d_plan, const void* Q,
               const void* K, const void* V, float* cache_O, float* cache_L, float* R, void* O, float* L,
               int64_t* d_counters, int32_t* d_status, float* d_err, int err_all, void* stream);
}  // namespace

extern "C" int dt_attn_partial_fused_heads(const dt_plan_params* p, int32_t head_begin, int32_t head_count,
                                           const uint8_t* d_plan, const void* Q, const void* K, const void* V,
                                           float* cache_O, float* cache_L, float* R, void* O, float* L,
                                           int64_t* d_counters, int32_t* d_status, void* stream) {
  return fused_step(p, head_begin, head_count, d_plan, Q, K, V, cache_O, cache_L, R, O, L, d_counters, d_status,
                    nullptr, 0, stream);
}

extern "C" int dt_attn_partial_fused_tracked(const dt_plan_params* p, const uint8_t* d_plan, const void* Q,
                                             const void* K, const void* V, float* cache_O, float* cache_L, void* O,
                                             float* L, int64_t* d_counters, int32_t* d_status, float* d_err,
                                             int32_t err_all, void* stream) {
  if (!p || p->mode == DT_MODE_WINDOW || !d_err) return DT_ERR_INVALID;
  return fused_step(p, 0, p->H, d_plan, Q, K, V, cache_O, cache_L, nullptr, O, L, d_counters, d_status, d_err,
                    err_all, stream);
}

namespace {
int fused_step(const dt_plan_params* p, int32_t head_begin, int32_t head_count, const uint8_t* d_plan, const void* Q,
               const void* K, const void* V, float* cache_O, float* cache_L, float* R, void* O, float* L,
               int64_t* d_counters, int32_t* d_status, float* d_err, int err_all, void* stream) {
  if (!p || p->mode < DT_MODE_ALL_COMPUTE || p->mode > DT_MODE_ANCHOR) return DT_ERR_INVALID;
  const bool win = p->mode == DT_MODE_WINDOW;
  if (!shape_ok(p->H, p->S, p->D)) return DT_ERR_INVALID;
  if (win ? p->window < 1 : p->P < 1) return DT_ERR_INVALID;
  if (p->group < 0 || (win && p->group != 0)) return DT_ERR_INVALID;
  if (p->state_dtype != DT_STATE_F32 && p->state_dtype != DT_STATE_BF16) return DT_ERR_INVALID;
  if (win && p->state_dtype != DT_STATE_F32) return DT_ERR_INVALID;
  if (head_begin < 0 || head_count < 0 || head_begin > p->H - head_count) return DT_ERR_INVALID;
  if (p->D != 64 && p->D != 72 && p->D != 128) return DT_ERR_UNSUPPORTED;
  const int nseg = win ? 2 : (p->group > 0 ? 1 + dt::ceil_div(p->P, p->group) : p->P);
  if (nseg > 64) return DT_ERR_UNSUPPORTED;              // the kernel keeps a plan row as a 64-bit mask
  if (head_count == 0 || p->S == 0) return DT_OK;
  if (!d_plan || !Q || !K || !V || !O || !L || !d_status) return DT_ERR_INVALID;
  if (win ? !R : (!cache_O || !cache_L)) return DT_ERR_INVALID;
  const void* ptrs[] = {d_plan, Q, K, V, O, L, d_status};
  for (const void* q : ptrs)
    if (!aligned16(q)) return DT_ERR_UNSUPPORTED;
  if ((cache_O && !aligned16(cache_O)) || (cache_L && !aligned16(cache_L)) || (R && !aligned16(R)) ||
      (d_counters && !aligned16(d_counters)) || (d_err && !aligned16(d_err)))
    return DT_ERR_UNSUPPORTED;

  dt::Geom G = dt::make_geom(p->H, p->S, p->D, win ? 1 : p->P, win ? p->window : 0, win ? 0 : p->group);
  const int dp = p->D == 72 ? 80 : p->D;
  dt::AttnParams kp;
  memset(&kp, 0, sizeof(kp));
  const CUtensorMapSwizzle sw128 = CU_TENSOR_MAP_SWIZZLE_128B, sw32 = CU_TENSOR_MAP_SWIZZLE_32B;
  if (!encode_qkv(&kp.tmQ, Q, p->H, p->S, p->D, 64, sw128) || !encode_qkv(&kp.tmK, K, p->H, p->S, p->D, 64, sw128) ||
      !encode_qkv(&kp.tmV, V, p->H, p->S, p->D, 64, sw128))
    return DT_ERR_CUDA;
  if (p->D == 72) {
    if (!encode_qkv(&kp.tmQt, Q, p->H, p->S, p->D, 16, sw32) || !encode_qkv(&kp.tmKt, K, p->H, p->S, p->D, 16, sw32) ||
        !encode_qkv(&kp.tmVt, V, p->H, p->S, p->D, 16, sw32))
      return DT_ERR_CUDA;
  }
  kp.plan = d_plan;
  kp.cache_O = cache_O;
  kp.cache_L = cache_L;
  kp.R = R;
  kp.O = O;
  kp.L = L;
  kp.counters = d_counters;
  kp.status = d_status;
  kp.H = p->H; kp.S = p->S; kp.D = p->D; kp.P = win ? 1 : p->P; kp.window = win ? p->window : 0;
  kp.geom = G;
  kp.state_bf16 = p->state_dtype == DT_STATE_BF16;
  kp.cache_v8 = (reinterpret_cast<uintptr_t>(cache_O) & 31u) == 0;
  // items are numbered over all heads, so a head range computes exactly what
  // the whole launch computes for those heads
  kp.item0 = head_begin * G.nqt;
  kp.item_end = (head_begin + head_count) * G.nqt;
  kp.scale_log2 = (float)(1.4426950408889634 / sqrt((double)p->D));
  kp.wait_limit_ns = (uint64_t)g_wait_limit_ns.load();
  kp.err = d_err;
  kp.err_all = err_all ? 1 : 0;
  int sms = 0;
  if (int e = sm_count(&sms)) return e;
  const int n_items = kp.item_end - kp.item0;
  if (n_items == 0) return DT_OK;
  int grid = n_items < sms ? n_items : sms;
  return dt::launch_attn_fused(kp, dp, grid, reinterpret_cast<cudaStream_t>(stream));
}
}  // namespace

extern "C" int dt_attn_partial_fused(const dt_plan_params* p, const uint8_t* d_plan, const void* Q, const void* K,
                                     const void* V, float* cache_O, float* cache_L, float* R, void* O, float* L,
                                     int64_t* d_counters, int32_t* d_status, void* stream) {
  if (!p) return DT_ERR_INVALID;
  return dt_attn_partial_fused_heads(p, 0, p->H, d_plan, Q, K, V, cache_O, cache_L, R, O, L, d_counters, d_status,
                                     stream);
}

extern "C" int dt_state_merge(int32_t N, int32_t H, int32_t S, int32_t D, const float* O_in, const float* L_in,
                              float* O_out, float* L_out, int32_t* d_status, void* stream) {
  if (N < 1 || D < 4 || D % 4 != 0 || !shape_ok(H, S, D)) return DT_ERR_INVALID;
  if ((int64_t)N * H * S * (int64_t)D >= ((int64_t)1 << 40)) return DT_ERR_INVALID;
  if ((int64_t)H * S == 0) return DT_OK;
  if (!O_in || !L_in || !O_out || !L_out) return DT_ERR_INVALID;
  if (!aligned16(O_in) || !aligned16(O_out) || !aligned16(L_in) || !aligned16(L_out)) return DT_ERR_UNSUPPORTED;
  (void)d_status;
  int sms = 0;
  if (int e = sm_count(&sms)) return e;
  return dt::launch_state_merge(N, H, S, D, O_in, L_in, O_out, L_out, sms, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int dt_state_cache_update(const dt_plan_params* p, const uint8_t* d_plan, const float* fresh_O,
                                     const float* fresh_L, float* cache_O, float* cache_L, int32_t* d_status,
                                     void* stream) {
  if (!p || p->mode == DT_MODE_WINDOW || p->mode < DT_MODE_ALL_COMPUTE || p->mode > DT_MODE_ANCHOR)
    return DT_ERR_INVALID;
  if (p->P < 1 || p->group < 0 || p->D < 4 || p->D % 4 != 0 || !shape_ok(p->H, p->S, p->D)) return DT_ERR_INVALID;
  if (p->state_dtype != DT_STATE_F32) return DT_ERR_UNSUPPORTED;
  if (p->H == 0 || p->S == 0) return DT_OK;
  if (!d_plan || !fresh_O || !fresh_L || !cache_O || !cache_L) return DT_ERR_INVALID;
  if (!aligned16(fresh_O) || !aligned16(cache_O) || !aligned16(fresh_L) || !aligned16(cache_L))
    return DT_ERR_UNSUPPORTED;
  (void)d_status;
  dt::Geom G = dt::make_geom(p->H, p->S, p->D, p->P, 0, p->group);
  int sms = 0;
  if (int e = sm_count(&sms)) return e;
  return dt::launch_cache_update(G, d_plan, fresh_O, fresh_L, cache_O, cache_L, sms,
                                 reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int dt_group_compose(const dt_plan_params* p, int32_t factor, int32_t* stamps, float* cache_O,
                                float* cache_L, int32_t* d_status, void* stream) {
  if (!p || p->mode == DT_MODE_WINDOW || p->mode < DT_MODE_ALL_COMPUTE || p->mode > DT_MODE_ANCHOR)
    return DT_ERR_INVALID;
  if (p->P < 1 || p->group < 1 || factor < 2 || factor > 8) return DT_ERR_INVALID;
  if (p->state_dtype != DT_STATE_F32) return DT_ERR_UNSUPPORTED;
  if (p->D < 4 || p->D % 4 != 0 || !shape_ok(p->H, p->S, p->D)) return DT_ERR_INVALID;
  if ((int64_t)p->group * factor > (int64_t)1 << 30) return DT_ERR_INVALID;
  const dt::Geom G = dt::make_geom(p->H, p->S, p->D, p->P, 0, p->group);
  const int m = G.P - 1, m2 = dt::ceil_div(m, factor);
  if ((int64_t)p->H * p->S > 0) {
    if (!cache_O || !cache_L) return DT_ERR_INVALID;
    if (!aligned16(cache_O) || !aligned16(cache_L)) return DT_ERR_UNSUPPORTED;
  }
  (void)d_status;
  if (stamps) {
    // [nqt][1+m] -> [nqt][1+m2] in place, rows and entries in increasing
    // order with no buffer: new entry i of row qt lands at qt*(1+m2)+i, which
    // is never after old entry i of that row, and every old entry it could
    // cover (row < qt, or entry <= i of row qt) has already been consumed,
    // since new entry i reads old entries factor*i+1 .. > i.
    for (int qt = 0; qt < G.nqt; ++qt) {
      const int32_t* old_row = stamps + (size_t)qt * (1 + m);
      int32_t* new_row = stamps + (size_t)qt * (1 + m2);
      new_row[0] = old_row[0];
      for (int i = 0; i < m2; ++i) {
        int32_t s = old_row[1 + factor * i];
        for (int j = factor * i + 1; j < factor * i + factor && j < m; ++j) s = old_row[1 + j] < s ? old_row[1 + j] : s;
        new_row[1 + i] = s;
      }
    }
  }
  if ((int64_t)p->H * p->S == 0) return DT_OK;
  int sms = 0;
  if (int e = sm_count(&sms)) return e;
  return dt::launch_group_compose(m, factor, p->H, p->S, p->D, cache_O, cache_L, sms,
                                  reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int dt_state_importance(const dt_plan_params* p, const float* cache_L, const float* L, float* d_weights,
                                   int32_t* d_status, void* stream) {
  if (!p || p->mode == DT_MODE_WINDOW || p->mode < DT_MODE_ALL_COMPUTE || p->mode > DT_MODE_ANCHOR)
    return DT_ERR_INVALID;
  if (p->P < 1 || p->group < 0 || p->D < 1 || !shape_ok(p->H, p->S, p->D)) return DT_ERR_INVALID;
  const dt::Geom G = dt::make_geom(p->H, p->S, p->D, p->P, 0, p->group);
  if ((int64_t)G.nqt * G.P == 0) return DT_OK;
  if (!d_weights) return DT_ERR_INVALID;
  if (p->H == 0) return dt::launch_fill_zero(d_weights, (int64_t)G.nqt * G.P, reinterpret_cast<cudaStream_t>(stream));
  if (!cache_L || !L) return DT_ERR_INVALID;
  if (!aligned16(cache_L) || !aligned16(L) || !aligned16(d_weights)) return DT_ERR_UNSUPPORTED;
  (void)d_status;
  return dt::launch_state_importance(G, cache_L, L, d_weights, reinterpret_cast<cudaStream_t>(stream));
}

namespace {
bool overlap(const void* a, const void* b, size_t n) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + n && y < x + n;
}
}  // namespace

extern "C" int dt_share_output(int32_t n_heads, int32_t S, int32_t D, const void* src_O, const float* src_L,
                               void* dst_O, float* dst_L, void* stream) {
  if (n_heads < 0 || S < 0 || D < 1 || !shape_ok(n_heads, S, D)) return DT_ERR_INVALID;
  const size_t nO = (size_t)n_heads * S * D * 2, nL = (size_t)n_heads * S * 4;
  if (nO == 0) return DT_OK;
  if (!src_O || !src_L || !dst_O || !dst_L) return DT_ERR_INVALID;
  const bool sameO = src_O == dst_O, sameL = src_L == dst_L;
  if ((!sameO && overlap(src_O, dst_O, nO)) || (!sameL && overlap(src_L, dst_L, nL))) return DT_ERR_INVALID;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (!sameO && cudaMemcpyAsync(dst_O, src_O, nO, cudaMemcpyDeviceToDevice, st) != cudaSuccess) return DT_ERR_CUDA;
  if (!sameL && cudaMemcpyAsync(dst_L, src_L, nL, cudaMemcpyDeviceToDevice, st) != cudaSuccess) return DT_ERR_CUDA;
  return DT_OK;
}

extern "C" int dt_attn_cfg_shared(const dt_plan_params* p, const uint8_t* d_plan, const void* Q, const void* K,
                                  const void* V, float* cache_O, float* cache_L, float* R, void* O, float* L,
                                  int64_t* d_counters, int32_t* d_status, void* stream) {
  if (!p || p->H % 2 != 0) return DT_ERR_INVALID;
  const int hb = p->H / 2;
  if (int e = dt_attn_partial_fused_heads(p, 0, hb, d_plan, Q, K, V, cache_O, cache_L, R, O, L, d_counters, d_status,
                                          stream))
    return e;
  if (hb == 0 || p->S == 0) return DT_OK;
  const size_t half = (size_t)hb * p->S;
  if (int e = dt_share_output(hb, p->S, p->D, O, L, static_cast<uint16_t*>(O) + half * p->D, L + half, stream))
    return e;
  const bool win = p->mode == DT_MODE_WINDOW;
  const dt::Geom G = dt::make_geom(p->H, p->S, p->D, win ? 1 : p->P, win ? p->window : 0, win ? 0 : p->group);
  int sms = 0;
  if (int e = sm_count(&sms)) return e;
  const int elem = win ? 4 : (p->state_dtype == DT_STATE_BF16 ? 2 : 4);
  return dt::launch_share_states(G, d_plan, hb, elem, cache_O, cache_L, R, sms,
                                 reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int dt_window_residual(int32_t op, int32_t H, int32_t S, int32_t D, const float* O_full,
                                  const float* O_win, float* R, void* O, int32_t* d_status, void* stream) {
  if (op != DT_WR_MAKE && op != DT_WR_APPLY) return DT_ERR_INVALID;
  if (D < 4 || D % 4 != 0 || !shape_ok(H, S, D)) return DT_ERR_INVALID;
  const int64_t n = (int64_t)H * S * D;
  if (n == 0) return DT_OK;
  if (!O_win || !R || (op == DT_WR_MAKE && !O_full) || (op == DT_WR_APPLY && !O)) return DT_ERR_INVALID;
  if (!aligned16(O_win) || !aligned16(R) || (O_full && !aligned16(O_full)) || (O && !aligned16(O)))
    return DT_ERR_UNSUPPORTED;
  (void)d_status;
  int sms = 0;
  if (int e = sm_count(&sms)) return e;
  return dt::launch_window_residual(op, n, O_full, O_win, R, O, sms, reinterpret_cast<cudaStream_t>(stream));
}

// ---- block-sparse attention and the passes in front of it -------------------
namespace {

int type_size(int t) { return t == DT_TYPE_F32 ? 4 : 2; }
bool type_ok(int t) { return t == DT_TYPE_BF16 || t == DT_TYPE_F16 || t == DT_TYPE_F32; }
// rows that start on 16-byte boundaries: strides of n > 1 heads / rows must be
// multiples of 16 bytes (a stride that no element uses is not looked at)
bool strides_aligned(const dt_strides& s, int heads, int rows, int size) {
  return (heads <= 1 || s.head * size % 16 == 0) && (rows <= 1 || s.row * size % 16 == 0);
}
bool strides_from(int64_t least, const dt_strides& s, int heads, int rows) {
  return (heads <= 1 || s.head >= least) && (rows <= 1 || s.row >= least);
}

// 16-bit [heads][S][D] with element strides as a 3-D tensor (D, S, heads); box (bw, rows, 1)
bool encode_strided(CUtensorMap* m, const void* base, int heads, int S, int D, dt_strides st, bool f16, int bw,
                    CUtensorMapSwizzle sw, int rows = 64) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)S, (cuuint64_t)heads};
  // an extent of 1 never uses its stride: any legal one will do
  const cuuint64_t row = S > 1 ? (cuuint64_t)st.row * 2 : (cuuint64_t)((D * 2 + 15) / 16 * 16);
  const cuuint64_t head = heads > 1 ? (cuuint64_t)st.head * 2 : row;
  cuuint64_t strides[2] = {row, head};
  cuuint32_t box[3] = {(cuuint32_t)bw, (cuuint32_t)rows, 1u};
  cuuint32_t estr[3] = {1u, 1u, 1u};
  return fn(m, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base),
            dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

extern "C" int dt_rope_table(const dt_rope_params* p, const int32_t* pos, float* table, void* stream) {
  if (!p || p->S < 0 || p->S > 1 << 30 || p->n_axes < 1 || p->n_axes > DT_ROPE_MAX_AXES) return DT_ERR_INVALID;
  if (!(p->base >= 1.0) || !std::isfinite(p->base)) return DT_ERR_INVALID;
  int64_t rot = 0;
  for (int a = 0; a < p->n_axes; ++a) {
    if (p->dim[a] < 2 || p->dim[a] % 2 != 0) return DT_ERR_INVALID;
    rot += p->dim[a];
  }
  if (rot > 2 * dt::kMaxPairs) return DT_ERR_INVALID;
  if (p->S == 0) return DT_OK;
  if (!pos || !table) return DT_ERR_INVALID;
  if (!aligned16(pos) || !aligned16(table)) return DT_ERR_UNSUPPORTED;
  dt::RopeTableArgs a;
  memset(&a, 0, sizeof(a));
  a.pos = pos;
  a.table = table;
  a.S = p->S;
  for (int x = 0; x < p->n_axes; ++x) {
    // powers of one ratio: at most 127 extended-precision products, and the truncation, stay below 2^-58
    const long double ratio = powl((long double)p->base, -2.0L / p->dim[x]);
    long double t = 1.0L / 6.283185307179586476925L;
    for (int j = 0; j < p->dim[x] / 2; ++j, t *= ratio) {
      a.turns[a.pairs] = (uint64_t)ldexpl(t - floorl(t), 64);       // whole turns do not matter
      a.axis[a.pairs++] = (uint8_t)x;
    }
  }
  return dt::launch_rope_table(a, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int dt_qk_norm_rope(const dt_norm_rope_params* p, const void* q, const void* k, const void* v,
                               const float* wq, const float* wk, const float* table, void* Q, void* K, void* V,
                               float* q_mean, float* k_mean, void* stream) {
  if (!p || p->S < 0 || p->S > 1 << 30 || p->D < 8 || p->D > 128 || p->D % 8 != 0) return DT_ERR_INVALID;
  if (p->H < 0 || p->Hkv < 0 || p->H > 1 << 14 || p->Hkv > 1 << 14) return DT_ERR_INVALID;
  if (p->rot < 0 || p->rot > p->D || p->rot % 8 != 0) return DT_ERR_INVALID;
  if (p->pairing != DT_ROPE_INTERLEAVED && p->pairing != DT_ROPE_HALVES) return DT_ERR_INVALID;
  if (!type_ok(p->in_type) || !type_ok(p->out_type)) return DT_ERR_INVALID;
  if (p->out_type != p->in_type && p->out_type != DT_TYPE_BF16) return DT_ERR_UNSUPPORTED;
  if (p->norm != 0 && p->norm != 1) return DT_ERR_INVALID;
  if (p->norm && !(p->eps >= 0.f && p->eps < INFINITY)) return DT_ERR_INVALID;
  if ((q_mean && p->q_block != 64 && p->q_block != 128) || (k_mean && p->k_block != 64 && p->k_block != 128))
    return DT_ERR_INVALID;
  // a part without an input has no outputs; a part with one has something to write
  if (q ? (!Q && !q_mean) : (Q || q_mean)) return DT_ERR_INVALID;
  if (k ? (!K && !k_mean) : (K || k_mean)) return DT_ERR_INVALID;
  if ((v != nullptr) != (V != nullptr)) return DT_ERR_INVALID;
  if (p->rot > 0 && (q || k) && !table && p->S > 0) return DT_ERR_INVALID;
  struct { const void* p; dt_strides s; int heads, size; } t[] = {
      {q, p->q_in, p->H, type_size(p->in_type)},    {k, p->k_in, p->Hkv, type_size(p->in_type)},
      {v, p->v_in, p->Hkv, type_size(p->in_type)},  {Q, p->q_out, p->H, type_size(p->out_type)},
      {K, p->k_out, p->Hkv, type_size(p->out_type)}, {V, p->v_out, p->Hkv, type_size(p->out_type)}};
  for (const auto& x : t)
    if (x.p) {
      // a stride of 0 broadcasts an input; rows of an output would overwrite one another
      if (!strides_from(&x < t + 3 || p->S == 0 ? 0 : 1, x.s, x.heads, p->S)) return DT_ERR_INVALID;
      if (!aligned16(x.p) || !strides_aligned(x.s, x.heads, p->S, x.size)) return DT_ERR_UNSUPPORTED;
    }
  // in place: each element is read and written by one thread only if both sides are laid out alike
  for (int i = 0; i < 3; ++i)
    if (t[i].p && t[i].p == t[i + 3].p &&
        (p->in_type != p->out_type || (p->S > 1 && t[i].s.row != t[i + 3].s.row) ||
         (t[i].heads > 1 && t[i].s.head != t[i + 3].s.head)))
      return DT_ERR_INVALID;
  for (const void* x : {(const void*)wq, (const void*)wk, (const void*)table, (const void*)q_mean, (const void*)k_mean})
    if (x && !aligned16(x)) return DT_ERR_UNSUPPORTED;
  if (p->S == 0 || p->H + p->Hkv == 0) return DT_OK;
  if (!q && !k && !v) return DT_OK;
  int sms = 0;
  if (int e = sm_count(&sms)) return e;
  dt::NormRopeArgs a;
  memset(&a, 0, sizeof(a));
  a.q = q; a.k = k; a.v = v;
  a.Q = Q; a.K = K; a.V = V;
  a.wq = wq; a.wk = wk; a.table = table;
  a.q_mean = q_mean; a.k_mean = k_mean;
  a.p = *p;
  return dt::launch_qk_norm_rope(a, sms, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int dt_block_select(const dt_select_params* p, const float* q_mean, const float* k_mean, int32_t* idx,
                               int32_t* count, void* stream) {
  if (!p || p->H < 0 || p->nq < 0 || p->nk < 0) return DT_ERR_INVALID;
  if (p->D < 4 || p->D > 128 || p->D % 4 != 0 || p->topk < 1) return DT_ERR_INVALID;
  if (p->keep_first < 0 || p->keep_last < 0 || (int64_t)p->keep_first + p->keep_last > p->topk) return DT_ERR_INVALID;
  if (!(p->margin >= 0.0)) return DT_ERR_INVALID;
  // the kernel's 32-bit list and row counters run up to a warp past these
  if (p->topk > 1 << 30 || p->nq > 1 << 30) return DT_ERR_INVALID;
  if (p->H > 0 && (p->Hkv < 1 || p->H % p->Hkv != 0)) return DT_ERR_INVALID;
  if ((int64_t)p->H * p->nq >= (int64_t)1 << 31) return DT_ERR_INVALID;
  if (p->nk > DT_SELECT_MAX_BLOCKS) return DT_ERR_UNSUPPORTED;
  if (p->H == 0 || p->nq == 0) return DT_OK;
  if (!q_mean || (!k_mean && p->nk > 0) || !idx || !count) return DT_ERR_INVALID;
  if (!aligned16(q_mean) || !aligned16(k_mean) || !aligned16(idx) || !aligned16(count)) return DT_ERR_UNSUPPORTED;
  return dt::launch_block_select(*p, q_mean, k_mean, idx, count, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int dt_attn_block_sparse(const dt_sparse_params* p, const void* Q, const void* K, const void* V,
                                    const int32_t* idx, const int32_t* count, void* O, float* L, int32_t* d_status,
                                    void* stream) {
  if (!p || p->H < 0 || p->Sq < 0 || p->Sk < 0 || p->cap < 0) return DT_ERR_INVALID;
  if (p->H > 0 && (p->Hkv < 1 || p->H % p->Hkv != 0)) return DT_ERR_INVALID;
  if (p->k_block != 64 && p->k_block != 128) return DT_ERR_INVALID;
  if (!type_ok(p->type) || !type_ok(p->out_type)) return DT_ERR_INVALID;
  if (p->type == DT_TYPE_F32 || (p->out_type != p->type && p->out_type != DT_TYPE_F32)) return DT_ERR_UNSUPPORTED;
  if (p->D != 64 && p->D != 72 && p->D != 128) return DT_ERR_UNSUPPORTED;
  // 32-bit row and list counters run up to a tile (lists: 128 entries) past these
  if (p->Sq > 1 << 30 || p->Sk > 1 << 30 || p->cap > 1 << 30) return DT_ERR_INVALID;
  const int nqb = dt::ceil_div(p->Sq, DT_TILE);
  if ((int64_t)p->H * nqb * 16 >= (int64_t)1 << 31) return DT_ERR_INVALID;
  if (p->H == 0 || p->Sq == 0) return DT_OK;
  if (!Q || !O || !L || !d_status || (p->Sk > 0 && (!K || !V)) || (p->cap > 0 && !idx)) return DT_ERR_INVALID;
  if (p->Sk == 0 && p->cap > 0 && !count) return DT_ERR_INVALID;       // lists of nothing but bad entries
  const int osize = type_size(p->out_type);
  const struct { const void* p; dt_strides s; int heads, rows, size; } t[] = {{Q, p->q, p->H, p->Sq, 2},
                                                                             {K, p->k, p->Hkv, p->Sk, 2},
                                                                             {V, p->v, p->Hkv, p->Sk, 2},
                                                                             {O, p->o, p->H, p->Sq, osize}};
  for (const auto& x : t) {
    if (x.rows == 0) continue;                                          // no keys: dense strides are {0, D}
    if ((x.heads > 1 && (x.s.head <= 0 || x.s.head >= (int64_t)1 << 39)) ||
        (x.rows > 1 && (x.s.row <= 0 || x.s.row >= (int64_t)1 << 39)))
      return DT_ERR_INVALID;
    if (!aligned16(x.p) || !strides_aligned(x.s, x.heads, x.rows, x.size)) return DT_ERR_UNSUPPORTED;
  }
  if (!aligned16(idx) || !aligned16(count) || !aligned16(L) || !aligned16(d_status)) return DT_ERR_UNSUPPORTED;

  dt::SparseParams kp;
  memset(&kp, 0, sizeof(kp));
  const bool f16 = p->type == DT_TYPE_F16;
  const CUtensorMapSwizzle sw128 = CU_TENSOR_MAP_SWIZZLE_128B, sw32 = CU_TENSOR_MAP_SWIZZLE_32B;
  // no keys: every list counts as empty (cap 0 below), so no box is ever
  // loaded from K and V and their maps may stand on Q's memory
  const bool keys = p->Sk > 0;
  const void* Kb = keys ? K : Q;
  const void* Vb = keys ? V : Q;
  const int kr = keys ? p->Sk : 1, kh = keys ? p->Hkv : 1;
  bool ok = encode_strided(&kp.tmQ, Q, p->H, p->Sq, p->D, p->q, f16, 64, sw128) &&
            encode_strided(&kp.tmK, Kb, kh, kr, p->D, p->k, f16, 64, sw128) &&
            encode_strided(&kp.tmV, Vb, kh, kr, p->D, p->v, f16, 64, sw128);
  if (ok && p->D == 72)
    ok = encode_strided(&kp.tmQt, Q, p->H, p->Sq, p->D, p->q, f16, 16, sw32) &&
         encode_strided(&kp.tmKt, Kb, kh, kr, p->D, p->k, f16, 16, sw32) &&
         encode_strided(&kp.tmVt, Vb, kh, kr, p->D, p->v, f16, 16, sw32);
  if (ok && p->out_type != DT_TYPE_F32)
    ok = encode_strided(&kp.tmO, O, p->H, p->Sq, p->D, p->o, f16, 64, sw128, 32) &&
         (p->D != 72 || encode_strided(&kp.tmOt, O, p->H, p->Sq, p->D, p->o, f16, 8, CU_TENSOR_MAP_SWIZZLE_NONE, 32));
  if (!ok) return DT_ERR_CUDA;
  kp.idx = idx;
  kp.count = count;
  kp.O = O;
  kp.L = L;
  kp.status = d_status;
  kp.o_head = p->o.head;
  kp.o_row = p->o.row;
  kp.H = p->H;
  kp.per_kv = p->H / p->Hkv;
  kp.Sq = p->Sq;
  kp.Sk = p->Sk;
  kp.nqb = nqb;
  kp.nkb = dt::ceil_div(p->Sk, p->k_block);
  kp.cap = keys ? p->cap : 0;
  kp.per_tile = DT_TILE / p->k_block;
  kp.out_f32 = p->out_type == DT_TYPE_F32;
  kp.scale_log2 = (float)(1.4426950408889634 / sqrt((double)p->D));
  kp.wait_limit_ns = (uint64_t)g_wait_limit_ns.load();
  int sms = 0;
  if (int e = sm_count(&sms)) return e;
  return dt::launch_attn_sparse(kp, p->D == 72 ? 80 : p->D, f16, sms, reinterpret_cast<cudaStream_t>(stream));
}

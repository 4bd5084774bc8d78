// attn_sparse.h -- kernel parameter block and launcher of block-sparse attention.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace dt {

struct SparseParams {
  CUtensorMap tmQ, tmK, tmV;        // 64-column blocks of 64 rows, 128-byte swizzle
  CUtensorMap tmQt, tmKt, tmVt;     // 16-column tail block (D = 72), 32-byte swizzle
  CUtensorMap tmO, tmOt;            // 16-bit output: boxes of 32 rows, 64 columns (128-byte swizzle) and the 8 of the tail
  const int32_t* idx;               // [H][nqb][cap]
  const int32_t* count;             // [H][nqb] or null (cap each)
  void* O;
  float* L;
  int32_t* status;
  int64_t o_head, o_row;            // element strides of O
  int H, per_kv;                    // query heads; query heads per key head
  int Sq, Sk, nqb, nkb, cap;
  int per_tile;                     // list entries per 128-key tile: 1 (k_block 128) or 2 (64)
  int split;                        // CTAs of a cluster that share a list (1: persistent, no cluster)
  int out_f32;
  float scale_log2;                 // log2(e) / sqrt(D)
  uint64_t wait_limit_ns;
};

// Launches the instance for padded head dim dp (64, 80, 128) and 16-bit type;
// chooses p.split from the number of lists, their length and the SMs.
int launch_attn_sparse(SparseParams& p, int dp, bool f16, int sms, cudaStream_t stream);

}  // namespace dt

// Device helpers of the ops on a cache with drafted tokens (tree_attention.cu, attention_weights.cu,
// cache_moves.cu).
#pragma once

#include <climits>

#include "cache_ops.h"
#include "tc_device.h"

namespace fr {
namespace tc {

constexpr int TREE_KEYS = 128;   // slots per tile

__device__ __forceinline__ void report_sample(unsigned* status, uint32_t where, int sample) {
  if (!(atomicOr(status, ST_BOUNDS_BIT) & ST_BOUNDS_BIT)) {   // the first refused sample reports
    atomicExch(status + 1, where);
    atomicExch(status + 2, static_cast<unsigned>(sample));
  }
}

// Key tiles of one (sample, KV head): 0 for a padded sample and for one whose length is out of range.
__device__ __forceinline__ int sample_tiles(const TreeArgs& a, int b) {
  const int len = a.lens[b];
  return len < 0 || len > a.S_max - a.N ? 0 : (len + a.N + TREE_KEYS - 1) / TREE_KEYS;
}

// Word i of the drafted tokens that token n sees, from its mask row (nullptr: tokens 0..n).
__device__ __forceinline__ uint32_t seen_word(const uint32_t* row, int n, int N, int i) {
  if (32 * i >= N || i < 0) return 0u;
  const uint32_t last = 32 * i + 32 > N ? (1u << (N - 32 * i)) - 1u : 0xffffffffu;
  if (row) return row[i] & last;
  return n >= 32 * i + 31 ? last : n < 32 * i ? 0u : ((2u << (n - 32 * i)) - 1u) & last;
}

// Bits t = 0..31: token n sees the slot of drafted index j0 + t (negative: committed, seen).
__device__ __forceinline__ uint32_t seen_slots(const uint32_t* row, int n, int N, int j0) {
  if (j0 <= -32) return 0xffffffffu;
  if (j0 >= N) return 0u;
  if (j0 < 0) return ((1u << -j0) - 1u) | (seen_word(row, n, N, 0) << -j0);
  const uint32_t lo = seen_word(row, n, N, j0 >> 5), hi = seen_word(row, n, N, (j0 >> 5) + 1);
  return __funnelshift_r(lo, hi, j0 & 31);
}

// Tensor map of [planes][rows][dh] bf16 (rows contiguous, planes plane_rows apart) for one copy of
// `box_rows` rows x `blocks` 64-feature blocks into [block][row][128 B], 128-byte swizzle; rows past
// `rows` read as zeros.
inline bool encode_rows_map(CUtensorMap* m, const void* base, uint64_t dh, uint64_t rows, uint64_t plane_rows,
                            uint64_t planes, uint32_t box_rows, uint32_t blocks) {
  const PFN_cuTensorMapEncodeTiled_v12000 fn = tensor_map_encoder();
  if (!fn) return false;
  const cuuint32_t es[4] = {1u, 1u, 1u, 1u};
  const cuuint64_t dims[4] = {64, rows, dh / 64, planes};
  const cuuint64_t strides[3] = {dh * 2, 128, plane_rows * dh * 2};
  const cuuint32_t box[4] = {64u, box_rows, blocks, 1u};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4u, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace tc
}  // namespace fr

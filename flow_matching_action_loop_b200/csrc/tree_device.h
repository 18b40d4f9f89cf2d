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

// The line of tiles: the samples' U units each (attention: KV head major, row tile minor; weights: KV
// heads), a unit's tiles in a row.
struct TileRange {
  long long t0, t1, cum;   // this CTA's tiles; first tile of sample b
  int b;                   // sample of t0
};

struct TileIter {
  long long t, t1, cum;
  int b, nb, U;
  // segment
  int len, hk, rt, tile0, tile1, first;
  __device__ __forceinline__ void start(const TreeArgs& a, const TileRange& r, int U_) {
    t = r.t0;
    t1 = r.t1;
    cum = r.cum;
    b = r.b;
    U = U_;
    first = 1;
    nb = t < t1 ? sample_tiles(a, b) : 0;
  }
  __device__ __forceinline__ bool next(const TreeArgs& a, int RT) {
    if (t >= t1) return false;
    while (t - cum >= static_cast<long long>(U) * nb) {
      cum += static_cast<long long>(U) * nb;
      nb = sample_tiles(a, ++b);
    }
    const int rel = static_cast<int>(t - cum), u = rel / nb;
    len = a.lens[b];
    hk = u / RT;
    rt = u - hk * RT;
    tile0 = rel - u * nb;
    tile1 = static_cast<int>(min(static_cast<long long>(nb), tile0 + (t1 - t)));
    t += tile1 - tile0;
    return true;
  }
};

// One warp: the tiles of the samples before b_end; with `status`, samples of a bad length are reported.
__device__ __forceinline__ long long tiles_before(const TreeArgs& a, int U, int b_end, unsigned* status) {
  const int lane = threadIdx.x & 31;
  long long sum = 0;
  for (int b0 = 0; b0 < b_end; b0 += 32) {
    const int b = b0 + lane;
    int n = 0;
    if (b < b_end) {
      n = sample_tiles(a, b);
      if (status && n == 0 && a.lens[b] >= 0) report_sample(status, CACHE_BAD_LEN, b);
    }
    sum += n;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum * U;
}

// One warp: the sample that holds tile `at`, and the tiles before it.
__device__ __forceinline__ void find_tile(const TreeArgs& a, int U, long long at, int& b_at, long long& cum_at) {
  const int lane = threadIdx.x & 31;
  long long cum = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const long long n = b0 + lane < a.B ? static_cast<long long>(sample_tiles(a, b0 + lane)) * U : 0;
    long long incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, cum + incl > at);
    if (hit) {
      const int l = __ffs(hit) - 1;
      b_at = b0 + l;
      cum_at = cum + __shfl_sync(0xffffffffu, incl - n, l);
      return;
    }
    cum += __shfl_sync(0xffffffffu, incl, 31);
  }
}

// One warp: this CTA's share of the line.  The first min(T, CTAs) CTAs have at least one tile each.
__device__ __forceinline__ TileRange tile_range(const TreeArgs& a, int U) {
  const long long T = tiles_before(a, U, a.B, blockIdx.x == 0 ? a.status : nullptr);
  const long long n = min(T, static_cast<long long>(gridDim.x)), c = blockIdx.x;
  TileRange r;
  r.t0 = c < n ? T * c / n : 0;
  r.t1 = c < n ? T * (c + 1) / n : 0;
  r.b = 0;
  r.cum = 0;
  if (r.t0 < r.t1) find_tile(a, U, r.t0, r.b, r.cum);
  return r;
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

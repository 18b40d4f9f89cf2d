// Device helpers of the ops on a cache with drafted tokens (tree_attention.cu, attention_weights.cu,
// cache_moves.cu).
#pragma once

#include <climits>

#include "cache_ops.h"
#include "tc_device.h"

namespace fr {
namespace tc {

constexpr int TREE_KEYS = 128;   // slots per tile
constexpr int TREE_WHOLE = 4;    // units of up to so many tiles are not cut (tree_attention.cu)

__device__ __forceinline__ void report_sample(unsigned* status, uint32_t where, int sample) {
  if (!(atomicOr(status, ST_BOUNDS_BIT) & ST_BOUNDS_BIT)) {   // the first refused sample reports
    atomicExch(status + 1, where);
    atomicExch(status + 2, static_cast<unsigned>(sample));
  }
}

// The line of tiles: the samples' units one after the other, a unit's tiles in a row.  A unit is a KV head
// and a batch of up to a.rtg row tiles (the weights kernel: all rows).  The line is cut into equal ranges,
// one per group of a.rtg CTAs; CTA r of a group runs row tile r of each batch, so that a group reads a key
// tile from HBM once and from the L2 after that.  (The entry points refuse sizes whose line is longer than an
// int.)
struct TileRange {
  int t0, t1, cum;   // this group's tiles; first tile of sample b
  int b, len;        // sample of the unit that t0 lies in or follows
};

__device__ __forceinline__ int tiles_of(const TreeArgs& a, int len) {
  return len < 0 || len > a.S_max - a.N ? 0 : (len + a.N + TREE_KEYS - 1) / TREE_KEYS;
}

// Key tiles of one (sample, KV head): 0 for a padded sample and for one whose length is out of range.
__device__ __forceinline__ int sample_tiles(const TreeArgs& a, int b) { return tiles_of(a, a.lens[b]); }

struct TileIter {
  int t, t1, cum;
  int b, len, nb, U;
  int hk, rt, tile0, tile1;   // segment: tiles [tile0, tile1) of the nb of unit (b, hk), row tile rt
  __device__ __forceinline__ void start(const TreeArgs& a, const TileRange& r, int U_) {
    t = r.t0;
    t1 = r.t1;
    cum = r.cum;
    b = r.b;
    len = r.len;
    U = U_;
    nb = tiles_of(a, len);
  }
  // The next segment, of CTA r of a group whose units have NB batches of the RT row tiles.
  __device__ __forceinline__ bool next(const TreeArgs& a, int RT, int NB, int r) {
    do {
      if (t >= t1) return false;
      while (t - cum >= U * nb) {
        cum += U * nb;
        len = a.lens[++b];
        nb = tiles_of(a, len);
      }
      const int rel = t - cum, u = rel / nb;
      hk = NB == 1 ? u : u / NB;
      rt = (u - hk * NB) * a.rtg + r;
      tile0 = rel - u * nb;
      tile1 = min(nb, tile0 + (t1 - t));
      t += tile1 - tile0;
    } while (rt >= RT);   // the last batch has fewer row tiles
    return true;
  }
};

// First tile of CTA c of n: floor(T c / n).
__device__ __forceinline__ int share_begin(int T, int c, int n) {
  const int q = T / n;
  return q * c + (T - q * n) * c / n;
}

// One warp: the tiles of the samples before b_end.
__device__ __forceinline__ int tiles_before(const TreeArgs& a, int U, int b_end) {
  int sum = 0;
  for (int b = threadIdx.x & 31; b < b_end; b += 32) sum += sample_tiles(a, b);
  return __reduce_add_sync(0xffffffffu, sum) * U;
}

// One warp: the sample that holds tile t < T, in r (b, len, cum).
__device__ __forceinline__ void locate(const TreeArgs& a, int U, int t, TileRange& r) {
  const int lane = threadIdx.x & 31;
  r.cum = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const int len = b0 + lane < a.B ? a.lens[b0 + lane] : -1, own = tiles_of(a, len) * U;
    int incl = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, r.cum + incl > t);
    if (hit) {
      const int l = __ffs(hit) - 1;
      r.b = b0 + l;
      r.cum += __shfl_sync(0xffffffffu, incl - own, l);
      r.len = __shfl_sync(0xffffffffu, len, l);
      break;
    }
    r.cum += __shfl_sync(0xffffffffu, incl, 31);
  }
}

// The line's length, its units, the groups that have tiles.
struct Line {
  int T, units, n;
};

// One warp: the line of all samples.
__device__ __forceinline__ Line measure_line(const TreeArgs& a, int U, bool report) {
  int T = 0, active = 0;
  for (int b = threadIdx.x & 31; b < a.B; b += 32) {
    const int len = a.lens[b], n = tiles_of(a, len);
    if (report && n == 0 && len >= 0) report_sample(a.status, CACHE_BAD_LEN, b);
    T += n;
    active += n > 0;
  }
  Line l;
  l.T = __reduce_add_sync(0xffffffffu, T) * U;
  l.units = __reduce_add_sync(0xffffffffu, active) * U;
  l.n = min(l.T, a.groups);
  return l;
}

// A unit of nb tiles is not cut if it is short (a bound moves by half of it), and the groups, with whole units of this
// length, have at most a.whole_extra tiles more than their share of the line; see tree_attention.cu.
__device__ __forceinline__ bool kept_whole(const TreeArgs& a, const Line& l, int nb) {
  return nb <= TREE_WHOLE || (nb <= a.whole_extra && nb * ((l.units + l.n - 1) / l.n) <= l.T / l.n + a.whole_extra);
}

// A bound between two groups that lies in a unit that is kept whole goes to the unit's nearer end.
__device__ __forceinline__ int move_bound(const TreeArgs& a, const Line& l, const TileRange& r, int t) {
  const int nb = tiles_of(a, r.len);
  if (!kept_whole(a, l, nb)) return t;
  const int in = (t - r.cum) % nb;
  return 2 * in > nb ? t + nb - in : t - in;
}

// One warp: group c's share of the line.  CUT: at any tile, and the first min(T, groups) groups have at least one
// tile each.  CTA 0 reports the samples of a bad length.
template <bool CUT>
__device__ __forceinline__ TileRange tile_range(const TreeArgs& a, int U, int c) {
  const Line l = measure_line(a, U, blockIdx.x == 0);
  TileRange r = {0, 0, 0, 0, -1};
  if (c >= l.n) return r;
  const int t0 = share_begin(l.T, c, l.n), t1 = share_begin(l.T, c + 1, l.n);
  locate(a, U, t0, r);
  r.t0 = t0;
  r.t1 = t1;
  if constexpr (!CUT) {
    r.t0 = move_bound(a, l, r, t0);
    if (t1 - r.cum < U * tiles_of(a, r.len)) {   // in the same sample
      r.t1 = move_bound(a, l, r, t1);
    } else if (t1 < l.T) {
      TileRange next;
      locate(a, U, t1, next);
      r.t1 = move_bound(a, l, next, t1);
    }
  }
  return r;
}

// A wait of at most limit_ns; at 1 ns the one test that it begins with (mbar_wait's own first test may suspend the
// thread for longer).
__device__ __forceinline__ bool tree_wait(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
  if (limit_ns == 1) return sm100::mbar_test(bar, parity);
  const uint64_t t0 = sm100::globaltimer();
  while (!sm100::mbar_try_wait(bar, parity))
    if (sm100::globaltimer() - t0 > limit_ns) return false;
  return true;
}

// Two float32 operations per instruction (sm_100), each rounded to nearest.
__device__ __forceinline__ uint64_t pack_f32x2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack_f32x2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Word i of what token n sees of the slots from the first drafted one on, from its mask row of W words
// (nullptr: tokens 0..n); before it committed slots, after the N drafted ones nothing.  The load has no
// branch before it, so that several calls' loads are on their way together.
__device__ __forceinline__ uint32_t seen_word(const uint32_t* row, int n, int N, int W, int i) {
  uint32_t w = row ? row[min(max(i, 0), W - 1)] : 0xffffffffu;
  if (!row) w = n >= 32 * i + 31 ? 0xffffffffu : n < 32 * i ? 0u : (2u << (n & 31)) - 1u;
  const uint32_t in = 32 * i + 32 <= N ? 0xffffffffu : 32 * i >= N ? 0u : (1u << (N & 31)) - 1u;
  return i < 0 ? 0xffffffffu : w & in;
}

// Bits t = 0..31: token n sees the slot of drafted index j0 + t (negative: committed, seen).
__device__ __forceinline__ uint32_t seen_slots(const uint32_t* row, int n, int N, int W, int j0) {
  return __funnelshift_r(seen_word(row, n, N, W, j0 >> 5), seen_word(row, n, N, W, (j0 >> 5) + 1), j0 & 31);
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

// Row moves inside a static KV cache: commit of accepted drafted tokens, eviction by accumulated
// attention weight.
#include <algorithm>
#include <cooperative_groups.h>

#include "fr.h"
#include "tree_device.h"

namespace fr {
namespace tc {
namespace {

namespace cg = cooperative_groups;

// ------------------------------------------------------------------ commit
// One CTA per (K or V, KV head, sample).  path ascends, so row i moves down (path[i] >= i) and no later
// source lies below a written row: rows go in rounds of what the CTA holds in registers, every load of a
// round before its stores, one barrier between them.
constexpr int CM_THREADS = 256;
constexpr int CM_VECS = 8;   // 16-byte words a thread holds per round

__global__ void __launch_bounds__(CM_THREADS) k_cache_commit(const __grid_constant__ MoveArgs a) {
  __shared__ int path[CM_THREADS];   // N <= FR_TREE_MAX_NODES
  const int part = blockIdx.x, h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  const int len = a.lens[b], np = a.npath[b];
  const bool writer = part == 0 && h == 0 && tid == 0;
  if (len < 0) {
    if (writer) a.lens_out[b] = len;
    return;
  }
  bool bad = len > a.S_max - a.N, bad_path = np < 0 || np > a.N;
  if (!bad_path && tid < np) {
    const int32_t* p = a.path + static_cast<size_t>(b) * a.N;
    const int v = p[tid];
    path[tid] = v;
    bad_path = v < 0 || v >= a.N || (tid > 0 && v <= p[tid - 1]);
  }
  bad_path = __syncthreads_or(bad_path);
  if (bad || bad_path) {
    if (writer) {
      report_sample(a.status, bad ? CACHE_BAD_LEN : CACHE_BAD_PATH, b);
      a.lens_out[b] = len;
    }
    return;
  }
  if (writer) a.lens_out[b] = len + np;
  const size_t slot0 = (static_cast<size_t>(b) * a.Hkv + h) * a.S_max + len;
  uint32_t* word = part == 0 ? reinterpret_cast<uint32_t*>(a.acc) : reinterpret_cast<uint32_t*>(a.pos);
  uint32_t w = 0;
  if (word && tid < np) w = word[slot0 + path[tid]];
  __syncthreads();
  if (word && tid < np) word[slot0 + tid] = w;
  const int nv = a.row_bytes / 16;
  uint4* rows = reinterpret_cast<uint4*>(part == 0 ? a.k : a.v) + slot0 * nv;
  const int per = CM_THREADS * CM_VECS / nv;   // rows per round
  for (int i0 = 0; i0 < np; i0 += per) {
    const int items = min(per, np - i0) * nv;
    uint4 x[CM_VECS];
#pragma unroll
    for (int u = 0; u < CM_VECS; ++u) {
      const int it = tid + u * CM_THREADS;
      if (it < items) x[u] = rows[static_cast<size_t>(path[i0 + it / nv]) * nv + it % nv];
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < CM_VECS; ++u) {
      const int it = tid + u * CM_THREADS;
      if (it < items) rows[static_cast<size_t>(i0) * nv + it] = x[u];
    }
  }
}

// ------------------------------------------------------------------ eviction
// One cluster per (KV head, sample); its CTAs share the sample's slots in contiguous slices.  The order
// is that of a 32-bit key (protected slots above all, then acc, NaN lowest; equal keys by slot), held in
// shared memory.  The keep-th largest key is found by a radix select over 8-bit digits from the top, the
// histograms summed over the cluster through distributed shared memory; each CTA then lists, in slot
// order, its freed slots below `keep` (holes) and its kept slots at or past it (movers), both of which
// have the same number over the cluster.  The r-th hole takes the r-th mover: only those rows of K and V
// move, and as no hole is a mover the copies need no order.
constexpr int EV_THREADS = 512, EV_WARPS = EV_THREADS / 32;
constexpr int EV_MAX_CLUSTER = 16;
constexpr int EV_SLICE_BYTES = 6;   // per slot of a slice: key (4) + list entry (2)

// Monotonic in the float order; NaN below everything, 0xFFFFFFFF above everything.
__device__ __forceinline__ uint32_t rank_key(float f) {
  if (f != f) return 0u;
  const uint32_t u = __float_as_uint(f + 0.f);   // -0 counts as 0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(EV_THREADS) k_cache_evict(const __grid_constant__ MoveArgs a) {
  extern __shared__ __align__(16) uint8_t ev_dyn[];
  __shared__ uint32_t hist[2][256], tot[256];
  __shared__ int pmax, n_hole, n_move, s_digit, s_left, s_eq0;
  __shared__ int w_eq[EV_WARPS], w_hole[EV_WARPS], w_move[EV_WARPS];
  __shared__ int hole_base[EV_MAX_CLUSTER + 1], move_base[EV_MAX_CLUSTER + 1];
  __shared__ int mv_dst[EV_THREADS], mv_src[EV_THREADS];
  cg::cluster_group cl = cg::this_cluster();
  const int C = static_cast<int>(cl.num_blocks()), c = static_cast<int>(cl.block_rank());
  const int h = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int len = a.lens[b], keep = a.keep;
  const size_t row0 = (static_cast<size_t>(b) * a.Hkv + h) * a.S_max;
  const float* acc = a.acc_in + row0;
  const int32_t* pos = a.pos_in + row0;
  float* acc_out = a.acc_out + row0;
  int32_t* pos_out = a.pos_out + row0;
  int32_t* src = a.src + (static_cast<size_t>(b) * a.Hkv + h) * keep;
  const bool writer = h == 0 && c == 0 && tid == 0;
  if (len < 0 || len > a.S_max) {   // the whole cluster leaves
    if (writer) {
      if (len > a.S_max) report_sample(a.status, CACHE_BAD_LEN, b);
      a.lens_out[b] = len;
    }
    return;
  }
  if (writer) a.lens_out[b] = min(len, keep);
  if (len <= keep) {   // nothing to free
    for (int j = c * EV_THREADS + tid; j < keep; j += C * EV_THREADS) {
      src[j] = j < len ? j : -1;
      if (j < len) {
        acc_out[j] = acc[j];
        pos_out[j] = pos[j];
      }
    }
    return;
  }

  const int per = ((len + C - 1) / C + 31) & ~31;
  const int lo = min(c * per, len), n = min(per, len - lo);
  uint32_t* key = reinterpret_cast<uint32_t*>(ev_dyn);
  uint16_t* list = reinterpret_cast<uint16_t*>(key + per);
  if (tid == 0) pmax = INT32_MIN;
  if (tid < 256) hist[0][tid] = 0;
  __syncthreads();
  int pm = INT32_MIN;
#pragma unroll 4
  for (int i = tid; i < n; i += EV_THREADS) {
    const float w = acc[lo + i];
    const int q = pos[lo + i];
    key[i] = rank_key(w);
    pm = max(pm, q);
    if (lo + i < keep) {   // as if it stayed; a freed slot's new token overwrites this
      src[lo + i] = lo + i;
      acc_out[lo + i] = w;
      pos_out[lo + i] = q;
    }
  }
  pm = __reduce_max_sync(0xffffffffu, pm);
  if (lane == 0) atomicMax(&pmax, pm);
  cl.sync();
  if (a.recent > 0) {
    const int last = __reduce_max_sync(0xffffffffu, lane < C ? *cl.map_shared_rank(&pmax, lane) : INT32_MIN);
    const long long bound = static_cast<long long>(last) - a.recent;
#pragma unroll 4
    for (int i = tid; i < n; i += EV_THREADS)
      if (pos[lo + i] > bound) key[i] = 0xffffffffu;
  }
  __syncthreads();

  // radix select: after each digit, `left` of the keys that share the digits so far belong to the kept;
  // when those are all of them, the digits that follow do not matter
  uint32_t prefix = 0;
  int left = keep, shift = 32, last = 0;
  const int n32 = (n + 31) & ~31;
  for (bool all = false; !all && shift > 0; last ^= 1) {
    shift -= 8;
    uint32_t* hp = hist[last];
    for (int i = tid; i < n32; i += EV_THREADS) {   // whole warps
      const uint32_t k = i < n ? key[i] : 0u;
      const bool in = i < n && (shift == 24 || (k >> (shift + 8)) == prefix);
      const uint32_t d = in ? (k >> shift) & 255u : 256u;
      if (shift == 24) {   // few digits (signs and exponents): one addition per digit and warp
        const unsigned same = __match_any_sync(0xffffffffu, d);
        if (in && lane == __ffs(same) - 1) atomicAdd(&hp[d], static_cast<uint32_t>(__popc(same)));
      } else if (in) {
        atomicAdd(&hp[d], 1u);
      }
    }
    cl.sync();
    if (tid < 256) {
      uint32_t t = 0;
#pragma unroll 4
      for (int r = 0; r < C; ++r) t += cl.map_shared_rank(hp, r)[tid];
      tot[tid] = t;
      hist[last ^ 1][tid] = 0;   // last read before this barrier, by every CTA
    }
    __syncthreads();
    if (warp == 0) {   // lane l holds digits 255 - 8l .. 248 - 8l
      uint32_t v[8], sum = 0;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        v[u] = tot[255 - 8 * lane - u];
        sum += v[u];
      }
      uint32_t incl = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
      }
      uint32_t above = incl - sum;
      if (above < static_cast<uint32_t>(left) && static_cast<uint32_t>(left) <= incl) {
        int u = 0;
        while (u < 7 && above + v[u] < static_cast<uint32_t>(left)) above += v[u++];
        s_digit = 255 - 8 * lane - u;
        s_left = left - static_cast<int>(above);
      }
    }
    __syncthreads();
    prefix = (prefix << 8) | static_cast<uint32_t>(s_digit);
    left = s_left;
    all = tot[s_digit] == static_cast<uint32_t>(left);
  }
  last ^= 1;   // the last digit's histogram
  // keys whose first digits are above `prefix` are kept, and the first `left` of those equal to it, in slot
  // order
  if (warp == 0) {
    const uint32_t e = lane < c ? cl.map_shared_rank(hist[last], lane)[prefix & 255u] : 0u;
    s_eq0 = static_cast<int>(__reduce_add_sync(0xffffffffu, e));
  }
  // each warp walks a contiguous part of the slice, so that ranks follow from ballots
  const int part = ((n + EV_WARPS - 1) / EV_WARPS + 31) & ~31;
  const int wlo = min(warp * part, n), whi = min(wlo + part, n);
  const unsigned below = (1u << lane) - 1u;
  int cnt = 0;
  for (int i0 = wlo; i0 < whi; i0 += 32) {
    const int i = i0 + lane;
    cnt += __popc(__ballot_sync(0xffffffffu, i < whi && key[i] >> shift == prefix));
  }
  if (lane == 0) w_eq[warp] = cnt;
  __syncthreads();
  int eq0 = s_eq0;
  for (int w = 0; w < warp; ++w) eq0 += w_eq[w];
  // twice over the part: count holes and movers, then (their places known) list them
  int holes = 0, moves = 0;
  for (int round = 0; round < 2; ++round) {
    int eq = eq0, nh = holes, nm = moves;
    for (int i0 = wlo; i0 < whi; i0 += 32) {
      const int i = i0 + lane, slot = lo + i;
      const bool in = i < whi;
      const uint32_t k = in ? key[i] >> shift : 0u;
      const unsigned be = __ballot_sync(0xffffffffu, in && k == prefix);
      const bool kept = in && (k > prefix || (k == prefix && eq + __popc(be & below) < left));
      const bool hole = in && !kept && slot < keep, mover = kept && slot >= keep;
      const unsigned bh = __ballot_sync(0xffffffffu, hole), bm = __ballot_sync(0xffffffffu, mover);
      if (round == 1) {
        if (hole) list[nh + __popc(bh & below)] = static_cast<uint16_t>(i);
        if (mover) list[per - 1 - nm - __popc(bm & below)] = static_cast<uint16_t>(i);
      }
      eq += __popc(be);
      nh += __popc(bh);
      nm += __popc(bm);
    }
    if (round == 0) {
      if (lane == 0) {
        w_hole[warp] = nh;
        w_move[warp] = nm;
      }
      __syncthreads();
      int th = 0, tm = 0;
      for (int w = 0; w < EV_WARPS; ++w) {
        if (w == warp) holes = th, moves = tm;
        th += w_hole[w];
        tm += w_move[w];
      }
      if (tid == 0) n_hole = th, n_move = tm;
    }
  }
  cl.sync();   // every CTA's lists and counts
  if (warp == 0) {   // C <= 16: sums over the CTAs before each
    int th = lane < C ? *cl.map_shared_rank(&n_hole, lane) : 0;
    int tm = lane < C ? *cl.map_shared_rank(&n_move, lane) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, th, o), z = __shfl_up_sync(0xffffffffu, tm, o);
      if (lane >= o) th += y, tm += z;
    }
    if (lane < C) {
      hole_base[lane + 1] = th;
      move_base[lane + 1] = tm;
    }
    if (lane == 0) hole_base[0] = move_base[0] = 0;
  }
  __syncthreads();
  const long long M = hole_base[C];
  const int r_lo = static_cast<int>(c * M / C), r_hi = static_cast<int>((c + 1) * M / C);
  const int nv = a.row_bytes / 16;
  uint4* kr = reinterpret_cast<uint4*>(a.k) + row0 * nv;
  uint4* vr = reinterpret_cast<uint4*>(a.v) + row0 * nv;
  for (int r0 = r_lo; r0 < r_hi; r0 += EV_THREADS) {
    const int nb = min(EV_THREADS, r_hi - r0);
    if (tid < nb) {
      const int r = r0 + tid;
      int ch = 0, cm = 0;
      while (r >= hole_base[ch + 1]) ++ch;
      while (r >= move_base[cm + 1]) ++cm;
      const int dst = ch * per + cl.map_shared_rank(list, ch)[r - hole_base[ch]];
      const int s = cm * per + cl.map_shared_rank(list, cm)[per - 1 - (r - move_base[cm])];
      src[dst] = s;
      acc_out[dst] = acc[s];
      pos_out[dst] = pos[s];
      mv_dst[tid] = dst;
      mv_src[tid] = s;
    }
    __syncthreads();
    // a warp moves U rows of K and V at a time, every load before the stores
    constexpr int U = 8;
    for (int m0 = warp; m0 < nb; m0 += EV_WARPS * U) {
      for (int e = lane; e < 2 * nv; e += 32) {
        uint4* base = e < nv ? kr + e : vr + (e - nv);
        uint4 x[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (m0 + u * EV_WARPS < nb) x[u] = base[static_cast<size_t>(mv_src[m0 + u * EV_WARPS]) * nv];
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (m0 + u * EV_WARPS < nb) base[static_cast<size_t>(mv_dst[m0 + u * EV_WARPS]) * nv] = x[u];
      }
    }
    __syncthreads();
  }
  cl.sync();   // no CTA leaves while another reads its lists
}

// CTAs per cluster: as many as give the GPU two CTAs per SM, of at least 128 slots, and what shared memory
// asks for.
int evict_cluster(int units, int S_max) {
  int C = 1;
  while (C < EV_MAX_CLUSTER && ((2 * C * units <= 296 && S_max >= 2 * C * 128) || S_max > C * 32768)) C *= 2;
  return C;
}

}  // namespace

cudaError_t cache_moves_init() {
  const void* f = reinterpret_cast<const void*>(k_cache_evict);
  cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  const int slice = ((FR_EVICT_MAX_SLOTS + EV_MAX_CLUSTER - 1) / EV_MAX_CLUSTER + 31) & ~31;
  return cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, slice * EV_SLICE_BYTES);
}

cudaError_t launch_cache_commit(const MoveArgs& a, cudaStream_t s) {
  k_cache_commit<<<dim3(2, a.Hkv, a.B), CM_THREADS, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_cache_evict(const MoveArgs& a, cudaStream_t s) {
  const int C = evict_cluster(a.B * a.Hkv, a.S_max);
  const int slice = ((a.S_max + C - 1) / C + 31) & ~31;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(C, a.Hkv, a.B);
  cfg.blockDim = dim3(EV_THREADS);
  cfg.dynamicSmemBytes = static_cast<size_t>(slice) * EV_SLICE_BYTES;
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = C;
  at.val.clusterDim.y = 1;
  at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_cache_evict, a);
}

}  // namespace tc
}  // namespace fr

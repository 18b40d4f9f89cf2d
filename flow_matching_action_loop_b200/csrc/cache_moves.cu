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
// round before its stores, one barrier between them.  64 samples, 8 heads of 128 features, up to 63 rows each: 5.5 us
// on the device for 16 MB (2.9 TB/s, mostly launch and two dependent loads); a call's host time is twice that.
constexpr int CM_THREADS = 256;
constexpr int CM_VECS = 8;   // 16-byte words a thread holds per round

__global__ void __launch_bounds__(CM_THREADS) k_cache_commit(const __grid_constant__ MoveArgs a) {
  __shared__ int path[CM_THREADS];   // N <= FR_TREE_MAX_NODES
  const int part = blockIdx.x, h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  const int len = a.lens[b], np = a.npath[b];
  const bool writer = part == 0 && h == 0 && tid == 0 && in_bounds(a.status, b, a.ext.lens, CHK_COMMIT_LENS);
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
  if (word && tid < np && in_bounds(a.status, slot0 + tid, part == 0 ? a.ext.acc : a.ext.pos, CHK_COMMIT_SLOTS))
    word[slot0 + tid] = w;
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
      const size_t to = static_cast<size_t>(i0) * nv + it;
      if (it < items && in_bounds(a.status, slot0 * nv + to, a.ext.rows, CHK_COMMIT_ROWS)) rows[to] = x[u];
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
//
// At 16 samples of up to 16384 slots, 8 heads of 128 bf16 features, trimmed to 12001: 81 us.  Keys are made after 13.5
// us, digits found after 21.5, lists joined after 26; the median CTA has moved its rows after 68 (119 MB written, as
// many read, 5.3 TB/s) and those of the longest samples after 82: HBM idles during the selection and partly at the end.
// Two CTAs of 512 threads per KV head and sample there; four took 87 us, four of 256 threads 84 us, two of 1024
// 100 us, one 133 us.  One head of 866 slots trimmed to 512: 10.4 us, of it 1.2 keys, 3.3 digits and 1.8 lists (a
// cluster barrier of 1 us each with the reads behind it), 2.4 moves, 0.6 the last barrier: what four CTAs cost each other;
// one CTA with all keys would need none.  float32 rows of 128 features, 8 x 8192 slots of 4 heads to 6001: 29 us for
// 12.6 at the rate of a copy.
constexpr int EV_THREADS = 512, EV_WARPS = EV_THREADS / 32;
constexpr int EV_MAX_CLUSTER = 16;
constexpr int EV_SLICE_BYTES = 6;   // per slot of a slice: key (4) + list entry (2)

// Monotonic in the float order; NaN below everything, 0xFFFFFFFF above everything.
__device__ __forceinline__ uint32_t rank_key(float f) {
  if (f != f) return 0u;
  const uint32_t u = __float_as_uint(f + 0.f);   // -0 counts as 0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(EV_THREADS, 2) k_cache_evict(const __grid_constant__ MoveArgs a) {
  extern __shared__ __align__(16) uint8_t ev_dyn[];
  __shared__ uint32_t hist[2][256], tot[256];
  __shared__ int pmax, n_hole, n_move, s_digit, s_left, s_tied;
  __shared__ int w_eq[EV_WARPS], w_events[EV_WARPS];
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
  const bool writer = h == 0 && c == 0 && tid == 0 && in_bounds(a.status, b, a.ext.lens, CHK_EVICT_LENS);
  auto put_src = [&](int j, int v) {
    if (in_bounds(a.status, src - a.src + j, a.ext.src, CHK_EVICT_SRC)) src[j] = v;
  };
  auto put_slot = [&](int j, float w, int32_t q) {
    if (in_bounds(a.status, row0 + j, a.ext.acc, CHK_EVICT_SLOTS)) acc_out[j] = w;
    if (in_bounds(a.status, row0 + j, a.ext.pos, CHK_EVICT_SLOTS)) pos_out[j] = q;
  };
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
      put_src(j, j < len ? j : -1);
      if (j < len) put_slot(j, acc[j], pos[j]);
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
  const int n32 = (n + 31) & ~31;
#pragma unroll 4
  for (int i = tid; i < n32; i += EV_THREADS) {   // whole warps
    const bool in = i < n;
    const float w = in ? acc[lo + i] : 0.f;
    const int q = in ? pos[lo + i] : INT32_MIN;
    const uint32_t k = rank_key(w), d = in ? k >> 24 : 256u;
    // the first digit's histogram: few digits (signs and exponents), one addition per digit and warp
    const unsigned same = __match_any_sync(0xffffffffu, d);
    if (in && lane == __ffs(same) - 1) atomicAdd(&hist[0][d], static_cast<uint32_t>(__popc(same)));
    pm = max(pm, q);
    if (in) key[i] = k;
    if (in && lo + i < keep) {   // as if it stayed; a freed slot's new token overwrites this
      put_src(lo + i, lo + i);
      put_slot(lo + i, w, q);
    }
  }
  if (a.recent > 0) {
    const int wm = __reduce_max_sync(0xffffffffu, pm);
    if (lane == 0) atomicMax(&pmax, wm);
    cl.sync();
    const int newest = __reduce_max_sync(0xffffffffu, lane < C ? *cl.map_shared_rank(&pmax, lane) : INT32_MIN);
    const long long bound = static_cast<long long>(newest) - a.recent;
    if (pm > bound) {   // this thread has protected slots: the largest key
#pragma unroll 4
      for (int i = tid; i < n; i += EV_THREADS)
        if (pos[lo + i] > bound) {
          atomicSub(&hist[0][key[i] >> 24], 1u);
          atomicAdd(&hist[0][255], 1u);
          key[i] = 0xffffffffu;
        }
    }
  }

  // radix select: after each digit, `left` of the keys that share the digits so far belong to the kept;
  // when those are all of them, the digits that follow do not matter
  uint32_t prefix = 0;
  int left = keep, shift = 32, last = 0;
  bool all = false;
  for (; !all && shift > 0; last ^= 1) {
    shift -= 8;
    uint32_t* hp = hist[last];
    if (shift < 24)
      for (int i = 4 * tid; i < n; i += 4 * EV_THREADS) {
        const uint4 k4 = *reinterpret_cast<const uint4*>(key + i);
        const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (i + e < n && (k[e] >> (shift + 8)) == prefix) atomicAdd(&hp[(k[e] >> shift) & 255u], 1u);
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
  // Kept are the keys whose first digits are above `prefix`, and those that equal it in slots below `tie`: all
  // of them or, where whole keys are equal, the first `left` in slot order.
  const int part = ((n + EV_WARPS - 1) / EV_WARPS + 127) & ~127;   // a warp's contiguous part, four slots a lane
  const int wlo = min(warp * part, n), whi = min(wlo + part, n);
  int tie = INT32_MAX;   // of this warp's part
  if (!all) {
    if (warp == 0) {
      const uint32_t e = lane < c ? cl.map_shared_rank(hist[last], lane)[prefix & 255u] : 0u;
      const int before = static_cast<int>(__reduce_add_sync(0xffffffffu, e));   // in the CTAs before this one
      if (lane == 0) s_tied = left - before;
    }
    int cnt = 0;
    for (int i = wlo + lane; i < whi; i += 32) cnt += key[i] == prefix;
    cnt = __reduce_add_sync(0xffffffffu, cnt);
    if (lane == 0) w_eq[warp] = cnt;
    __syncthreads();
    int want = s_tied;   // in this part
    for (int w = 0; w < warp; ++w) want -= w_eq[w];
    if (want <= 0) tie = 0;
    for (int i0 = wlo; want > 0 && want < cnt; i0 += 32) {   // ends at the want-th
      const bool eq = i0 + lane < whi && key[i0 + lane] == prefix;
      const unsigned be = __ballot_sync(0xffffffffu, eq);
      const unsigned hit = __ballot_sync(0xffffffffu, eq && __popc(be & ((1u << lane) - 1u)) == want - 1);
      if (hit) tie = lo + i0 + __ffs(hit), cnt = 0;
      want -= __popc(be);
    }
  }
  // bits 0-3: of slots i..i+3, those to be freed below `keep`; bits 4-7: those kept at or past it
  auto events = [&](int i) {
    const uint4 k4 = *reinterpret_cast<const uint4*>(key + i);
    const uint32_t k[4] = {k4.x >> shift, k4.y >> shift, k4.z >> shift, k4.w >> shift};
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int slot = lo + i + e;
      const bool kept = k[e] > prefix || (k[e] == prefix && slot < tie);
      if (i + e < n && kept == (slot >= keep)) m |= (kept ? 16u : 1u) << e;
    }
    return m;
  };
  // twice over the part: count holes and movers (its low and high half), then (their places known) list them
  uint32_t mine = 0;
  for (int i = wlo + 4 * lane; i < whi; i += 128) {
    const uint32_t m = events(i);
    mine += __popc(m & 15u) + (__popc(m >> 4) << 16);
  }
  mine = __reduce_add_sync(0xffffffffu, mine);
  if (lane == 0) w_events[warp] = static_cast<int>(mine);
  __syncthreads();
  int holes = 0, moves = 0, th = 0, tm = 0;
  for (int w = 0; w < EV_WARPS; ++w) {
    if (w == warp) holes = th, moves = tm;
    th += w_events[w] & 0xffff;
    tm += w_events[w] >> 16;
  }
  if (tid == 0) n_hole = th, n_move = tm;
  if (mine)
    for (int i0 = wlo; i0 < whi; i0 += 128) {
      const int i = i0 + 4 * lane;
      const uint32_t m = i < whi ? events(i) : 0u;
      if (!__any_sync(0xffffffffu, m != 0)) continue;
      const uint32_t own = __popc(m & 15u) | (__popc(m >> 4) << 8);
      uint32_t incl = own;   // at most 128 of either
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      int nh = holes + static_cast<int>((incl - own) & 255u), nm = moves + static_cast<int>((incl - own) >> 8);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if ((m >> e) & 1u) list[nh++] = static_cast<uint16_t>(i + e);
        if ((m >> (4 + e)) & 1u) list[per - 1 - nm++] = static_cast<uint16_t>(i + e);
      }
      const uint32_t sum = __shfl_sync(0xffffffffu, incl, 31);
      holes += static_cast<int>(sum & 255u);
      moves += static_cast<int>(sum >> 8);
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
    float w = 0.f;
    int q = 0, dst = 0;
    if (tid < nb) {
      const int r = r0 + tid;
      int ch = 0, cm = 0;
      while (r >= hole_base[ch + 1]) ++ch;
      while (r >= move_base[cm + 1]) ++cm;
      dst = ch * per + cl.map_shared_rank(list, ch)[r - hole_base[ch]];
      const int s = cm * per + cl.map_shared_rank(list, cm)[per - 1 - (r - move_base[cm])];
      mv_dst[tid] = dst;
      mv_src[tid] = s;
      put_src(dst, s);
      w = acc[s];   // stored behind the rows
      q = pos[s];
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
          if (m0 + u * EV_WARPS < nb) {
            const size_t to = static_cast<size_t>(mv_dst[m0 + u * EV_WARPS]) * nv;
            if (in_bounds(a.status, row0 * nv + to + (e < nv ? e : e - nv), a.ext.rows, CHK_EVICT_ROWS)) base[to] = x[u];
          }
      }
    }
    if (tid < nb) put_slot(dst, w, q);
    __syncthreads();
  }
  cl.sync();   // no CTA leaves while another reads its lists
}

// CTAs per cluster: as many as give the GPU two CTAs per SM (figures above), of at least 128 slots, and what
// shared memory asks for.
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

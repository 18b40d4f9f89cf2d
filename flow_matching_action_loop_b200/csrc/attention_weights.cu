// The attention weight that each slot of a static KV cache received (fr_attention_weights).
//
// With the log-sum-exp of every row known, slot s's weight is a sum over rows of independent terms,
// exp(q k_s / sqrt(dh) - lse).  The scores are computed transposed, K Q^T: a lane of tensor memory is a
// slot and a column a row, so that each thread sums the terms of one slot in registers and nothing is
// exchanged; there are no atomics.
//
// The 128-slot tiles of all (sample, KV head) pairs form one line, cut into equal ranges over the CTAs (one
// per SM).  A CTA keeps up to 256 of the pair's rows in shared memory and streams its K tiles past them, from
// the second 256 rows on (the next pass) out of the L2.  With several passes it does so for a block of up to 128
// tiles at a time, and its threads hold their slots' sums from pass to pass: acc receives each slot's whole sum in
// one addition, by one thread (added pass by pass, terms far below acc would be lost one pass at a time).
//   copy warp      query rows, K tiles by tensor map (128-byte swizzle) into a ring
//   MMA warp       K(t) Q^T, 128 rows at a time, into one of a sum group's two score buffers in tensor memory
//   sum warps      two groups of four take the tiles in turn, a thread a slot: 2^(s - lse) in fp32.  (With
//                  both groups on one tile, half of the columns each, a tile's exponentials had nothing to
//                  overlap with: 1870 cycles for 128 x 128 scores against 1024 of the exponentials.)
//
// Single tokens of 32 samples with up to 8191 slots, 8 KV heads of 128: 59 us, 338 MB at 5.7 TB/s (memory).  Trees of
// 63 tokens over 6 x 32767 slots, 8 query heads of 256: 51 us, 965 TFLOP/s, the multi-function unit and the tensor
// pipe each half busy; with a cold L2 55 us.  Holding the sums between the passes costs there 0.7 us; in blocks of 64
// tiles 300 rows of 64 features over 8 x 159900 slots took 172 us instead of 156 (a pass begins with new query rows).
#include <algorithm>
#include <type_traits>

#include "fr.h"
#include "tree_device.h"

namespace fr {
namespace tc {
namespace {

using namespace fr::sm100;

constexpr int AW_SUM = 256;
constexpr int AW_THREADS = AW_SUM + 64;
constexpr int AW_CHUNK = 128;               // rows per score buffer
constexpr int AW_PASS = 2 * AW_CHUNK;       // rows held in shared memory
constexpr int AW_SLOTS = 10;                // ring slots at most
constexpr int AW_SMEM = 224 * 1024;
constexpr int AW_HELD = 64;                 // sums that a thread holds (in local memory): its group's tiles of a block
constexpr int AW_BLOCK = 2 * AW_HELD;       // tiles

// Tile of a block of n at place i of a pass.  The groups take the places in turn, throughout.  After an odd number
// of tiles the next pass begins with the second group (flip): the tiles change places in pairs, so that each stays
// with its group.  Only the last one, without a partner, goes to the two groups in turn.
__device__ __forceinline__ int tile_at(int i, int n, int flip) { return (i ^ flip) < n ? i ^ flip : i; }

template <int DH>
struct WeightGeom {
  static constexpr int pieces = DH == 256 ? 2 : 1;                // per K tile, 64 or 128 features and more
  static constexpr int piece = TREE_KEYS * DH * 2 / pieces;
  static constexpr int blocks = DH / 64 / pieces;
  static constexpr int q_bytes = AW_CHUNK * DH * 2;               // one chunk of rows
};

// MANY: more than one pass.
template <int DH, bool MANY>
__global__ void __launch_bounds__(AW_THREADS, 1) k_attn_weights(const __grid_constant__ TreeArgs a) {
  using G = WeightGeom<DH>;
  extern __shared__ __align__(1024) uint8_t dsm[];
  __shared__ uint64_t full[AW_SLOTS], empty[AW_SLOTS], q_full, q_empty, bar_s[4], bar_e[4], fin_bar;   // [2 x group + buffer]
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  __shared__ TileRange range;
  __shared__ __align__(16) float lse_sh[AW_PASS];   // -lse in log2 units, -inf: a row that gives nothing
  __shared__ uint32_t live_sh[AW_PASS / 32];        // 0 bits: such rows of the pass, whose q may hold anything
  __shared__ float odd_sh[TREE_KEYS];               // sums of the tile that goes from group to group
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int g = a.Hq / a.Hkv, R = g * a.N;
  const int passes = MANY ? (R + AW_PASS - 1) / AW_PASS : 1;
  // the query rows of a pass take as many chunks as the largest pass has; the ring has the rest
  const int q_chunks = R > AW_CHUNK ? 2 : 1;
  const int NS = min(AW_SLOTS, (AW_SMEM - q_chunks * G::q_bytes) / G::piece);
  uint8_t* ring = dsm + q_chunks * G::q_bytes;

  if (tid == 0) {
    tma_prefetch_map(&a.tm_q);
    tma_prefetch_map(&a.tm_k);
    for (int i = 0; i < AW_SLOTS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&bar_s[i], 1);
      mbar_init(&bar_e[i], 4);
    }
    mbar_init(&q_full, 1);
    mbar_init(&q_empty, 1);
    mbar_init(&fin_bar, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(&tmem_base, 512);
    tmem_relinquish();
  }
  if (warp == 1) {
    const TileRange r = tile_range<true>(a, a.Hkv, blockIdx.x);
    if ((tid & 31) == 0) range = r;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tS = __shfl_sync(0xffffffffu, tmem_base, 0);
  volatile int* abort_v = &abort_flag;
  const TileRange rg = range;
  TileIter it;
  it.start(a, rg, a.Hkv);
  bool ok = true;
  auto pass_rows = [&](int p) { return min(AW_PASS, R - p * AW_PASS); };
  constexpr int block = MANY ? AW_BLOCK : INT_MAX;

  if (warp == AW_SUM / 32) {
    // ---------------- copies
    if ((tid & 31) == 0) {
      int slot = 0, use = 0, q_use = 0, issued = 0, turn = 0;
      bool more = it.next(a, 1, 1, 0);
      for (int b0 = it.tile0; ok && more;) {
        const int plane = it.b * a.Hkv + it.hk, n = min(block, it.tile1 - b0);
        for (int p = 0; ok && p < passes; ++p) {
          if (q_use > 0 && !tree_wait(&q_empty, (q_use - 1) & 1, a.wait_ns)) {
            ok = false;
            break;
          }
          ++q_use;
          const int nc = (pass_rows(p) + AW_CHUNK - 1) / AW_CHUNK;
          mbar_arrive_expect_tx(&q_full, nc * G::q_bytes);
          for (int c = 0; c < nc; ++c)
            tma_load_4d(dsm + c * G::q_bytes, &a.tm_q, 0, p * AW_PASS + c * AW_CHUNK, 0, plane, &q_full);
          for (int at = 0; ok && at < n; ++at) {
            const int tile = b0 + tile_at(at, n, MANY ? turn : 0);
            for (int i = 0; i < G::pieces; ++i) {
              if ((use > 0 && !tree_wait(&empty[slot], (use - 1) & 1, a.wait_ns)) || *abort_v) {
                ok = false;
                break;
              }
              mbar_arrive_expect_tx(&full[slot], G::piece);
              tma_load_4d(ring + slot * G::piece, &a.tm_k, 0, tile * TREE_KEYS, i * G::blocks, plane, &full[slot]);
              ++issued;
              if (++slot == NS) slot = 0, ++use;
            }
          }
          turn ^= n & 1;
        }
        b0 += n;
        if (b0 >= it.tile1) {
          more = it.next(a, 1, 1, 0);
          b0 = it.tile0;
        }
      }
      if (!ok) {
        *abort_v = 1;
        report_timeout(a.status, 0x720);
      }
      // no copy is in flight when the CTA leaves
      for (int i = max(0, issued - NS); i < issued; ++i) mbar_wait(&full[i % NS], (i / NS) & 1, WAIT_LIMIT_NS);
      if (q_use > 0) mbar_wait(&q_full, (q_use - 1) & 1, WAIT_LIMIT_NS);
    }
  } else if (warp == AW_SUM / 32 + 1) {
    // ---------------- MMAs, the whole warp in step.  The waits go in a fixed order (bounded, in ok_wait).
    const bool leader = elect_one();
    auto ok_wait = [&](uint64_t* bar, int phase) {
      if (__all_sync(0xffffffffu, mbar_test(bar, phase & 1))) return true;
      return __all_sync(0xffffffffu, tree_wait(bar, phase & 1, a.wait_ns) && !*abort_v) != 0;
    };
    auto same = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };   // known to be uniform
    const uint64_t dq = smem_desc_sw128(smem_u32(dsm), 16, 1024), dk = smem_desc_sw128(smem_u32(ring), 16, 1024);
    int slot = 0, use = 0, q_use = 0, grp = 0, items[2] = {0, 0};   // group of the next tile, items of each group
    for (int to_go = 0; ok;) {   // tiles of the segment
      if (to_go == 0) {
        if (!same(it.next(a, 1, 1, 0))) break;
        to_go = same(it.tile1 - it.tile0);
      }
      const int tiles = min(block, to_go);
      to_go -= tiles;
      for (int p = 0; ok && p < passes; ++p) {
        ok = ok_wait(&q_full, q_use);
        ++q_use;
        const int rows = pass_rows(p), nc = (rows + AW_CHUNK - 1) / AW_CHUNK;
        for (int tile = 0; ok && tile < tiles; ++tile, grp ^= 1) {
          int item = grp ? items[1] : items[0];
          for (int c = 0; ok && c < nc; ++c, ++item) {
            const int buf = 2 * grp + (item & 1), nth = item >> 1;
            if (nth > 0) ok = ok_wait(&bar_e[buf], nth - 1);   // its scores before these have been read
            const int cols = (min(AW_CHUNK, rows - c * AW_CHUNK) + 31) & ~31;
            const uint32_t idesc = idesc_f32acc(FMT_BF16, 128, cols), d = tS + buf * AW_CHUNK;
            const uint64_t qd = dq + c * (G::q_bytes / 16);
            int sl = slot, u = use;
#pragma unroll
            for (int i = 0; i < G::pieces; ++i) {
              if (ok && c == 0) ok = ok_wait(&full[sl], u);
              if (ok) {
                tc_fence_after();
                const uint64_t kd = dk + sl * (G::piece / 16);
#pragma unroll
                for (int k = 0; k < G::blocks * 4; ++k)
                  mma_bf16_warp(leader, d, kd + ((k >> 2) * (TREE_KEYS * 128) + (k & 3) * 32) / 16,
                                qd + ((i * G::blocks + (k >> 2)) * (AW_CHUNK * 128) + (k & 3) * 32) / 16, idesc,
                                i > 0 || k > 0);
                if (c == nc - 1) mma_commit_warp(leader, &empty[sl]);   // the tile's last rows
              }
              if (++sl == NS) sl = 0, ++u;
            }
            if (ok) mma_commit_warp(leader, &bar_s[buf]);
          }
          (grp ? items[1] : items[0]) = item;
#pragma unroll
          for (int i = 0; i < G::pieces; ++i)
            if (++slot == NS) slot = 0, ++use;
        }
        if (ok) mma_commit_warp(leader, &q_empty);
      }
    }
    if (!ok) {
      *abort_v = 1;
      if (leader) report_timeout(a.status, 0x721);
    }
    // every MMA issued has completed before tensor memory is freed
    mma_commit_warp(leader, &fin_bar);
    if (!mbar_wait(&fin_bar, 0, WAIT_LIMIT_NS) && leader) report_timeout(a.status, 0x722);
  } else {
    // ---------------- sums.  A warp whose wait gave up goes on without waiting (the named barrier needs every
    // warp).  Its arrivals come too early from then on: it sets the abort word before them, and no sum is stored
    // that was read after that.
    const int key = tid & 127, grp = tid >> 7, pw = warp & 3, lane = tid & 31;   // slot of the tile, group
    const uint32_t lanes = static_cast<uint32_t>(pw * 32) << 16;
    const float sl2 = a.scale * 1.4426950408889634f;   // scores in log2 units
    const uint64_t sl22 = pack_f32x2(sl2, sl2);
    int item = 0, turn = 0;                            // of this group; group of the next tile
    float held[MANY ? AW_HELD : 1];                    // sums of this thread's slots over the passes so far
    bool more = it.next(a, 1, 1, 0);
    for (int b0 = it.tile0; more;) {
      const int len = it.len, keys = len + a.N, n = min(block, it.tile1 - b0);
      float* acc = a.acc + (static_cast<size_t>(it.b) * a.Hkv + it.hk) * a.S_max;
      const float* lse = a.lse + (static_cast<size_t>(it.b) * a.Hq + static_cast<size_t>(it.hk) * g) * a.N;
      for (int p = 0; p < passes; ++p) {
        const int rows = pass_rows(p), nc = (rows + AW_CHUNK - 1) / AW_CHUNK, r0 = p * AW_PASS;
        asm volatile("bar.sync 5, 256;" ::: "memory");   // the last pass has read its lse
        {
          float x = -INFINITY;
          if (tid < rows) {
            const int tok = (r0 + tid) % a.N;
            const bool counts = !a.use || ((a.use[static_cast<size_t>(it.b) * a.W + (tok >> 5)] >> (tok & 31)) & 1u);
            const float v = lse[r0 + tid];
            // (one float32 rounding of the exponent: no more than half a step of lse itself gives the weight)
            if (counts && v != -INFINITY) x = -v * 1.4426950408889634f;
          }
          lse_sh[tid] = x;
          const unsigned live = __ballot_sync(0xffffffffu, x != -INFINITY || tid >= rows);   // (q reads as 0 past the rows)
          if (lane == 0) live_sh[warp] = live;
        }
        asm volatile("bar.sync 5, 256;" ::: "memory");
        // a committed slot adds to its sum, a drafted one begins with these rows; fetched a tile ahead
        const bool last = p == passes - 1;
        const int flip = MANY ? turn : 0;
        auto sum_before = [&](int at) {
          return last ? acc[min((b0 + tile_at(at, n, flip)) * TREE_KEYS + key, keys - 1)] : 0.f;
        };
        const int first = turn ^ grp;   // this group's places: every other one
        turn ^= n & 1;
        float before = sum_before(first);
        for (int at = first; at < n; at += 2) {
          const int in_block = tile_at(at, n, flip), tile = b0 + in_block, slot = tile * TREE_KEYS + key;
          const bool boundary = (tile + 1) * TREE_KEYS > len;
          const float next = sum_before(at + 2);
          float* part = !MANY ? nullptr : (n & 1) && in_block == n - 1 ? &odd_sh[key] : &held[in_block >> 1];
          const float so_far = MANY && p > 0 ? *part : 0.f;
          uint64_t w2[2] = {0, 0};
          for (int c = 0; c < nc; ++c, ++item) {
            const int buf = 2 * grp + (item & 1);
            const int cols = (min(AW_CHUNK, rows - c * AW_CHUNK) + 31) & ~31;
            const float* ls = lse_sh + c * AW_CHUNK;
            // columns (rows) that see this thread's slot: a lane finds the 32 slots of its warp that its
            // column sees, a transposition of the 32 x 32 bits gives each slot its columns
            uint32_t vis[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};
            if (boundary) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int tok = (r0 + c * AW_CHUNK + 32 * i + lane) % a.N;
                const uint32_t* words = a.mask ? a.mask + (static_cast<size_t>(it.b) * a.N + tok) * a.W : nullptr;
                vis[i] = seen_slots(words, tok, a.N, a.W, tile * TREE_KEYS + 32 * pw - len);
              }
              auto stage = [&](int st, uint32_t m) {   // the four words side by side: a shuffle waits long
                uint32_t y[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) y[i] = __shfl_xor_sync(0xffffffffu, vis[i], st);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  vis[i] = lane & st ? (vis[i] & ~m) | ((y[i] >> st) & m) : (vis[i] & m) | ((y[i] & m) << st);
              };
              stage(16, 0x0000ffffu);
              stage(8, 0x00ff00ffu);
              stage(4, 0x0f0f0f0fu);
              stage(2, 0x33333333u);
              stage(1, 0x55555555u);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) vis[i] &= live_sh[4 * c + i];
            if (!__all_sync(0xffffffffu, mbar_test(&bar_s[buf], (item >> 1) & 1)) && ok) {
              ok = __all_sync(0xffffffffu, tree_wait(&bar_s[buf], (item >> 1) & 1, a.wait_ns) && !*abort_v);
              if (!ok) *abort_v = 1;
            }
            tc_fence_after();
            const uint32_t ts = tS + buf * AW_CHUNK + lanes;
            // all: every column counts, for every slot
            auto terms = [&](const uint32_t* s, int col, uint32_t v, auto all) {
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                const float4 l4 = *reinterpret_cast<const float4*>(ls + col + e);
                float2 x = unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), sl22,
                                                  pack_f32x2(l4.x, l4.y)));
                float2 y = unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(s[e + 2]), __uint_as_float(s[e + 3])), sl22,
                                                  pack_f32x2(l4.z, l4.w)));
                if constexpr (!decltype(all)::value) {   // whatever score and lse are
                  if (!((v >> e) & 1u)) x.x = -INFINITY;
                  if (!((v >> (e + 1)) & 1u)) x.y = -INFINITY;
                  if (!((v >> (e + 2)) & 1u)) y.x = -INFINITY;
                  if (!((v >> (e + 3)) & 1u)) y.y = -INFINITY;
                }
                w2[0] = add_f32x2(w2[0], pack_f32x2(ex2_approx(x.x), ex2_approx(x.y)));
                w2[1] = add_f32x2(w2[1], pack_f32x2(ex2_approx(y.x), ex2_approx(y.y)));
              }
            };
            auto sum32 = [&](const uint32_t* s, int col, uint32_t v) {
              if (__all_sync(0xffffffffu, v == 0xffffffffu))
                terms(s, col, v, std::true_type());
              else
                terms(s, col, v, std::false_type());
            };
#pragma unroll
            for (int i = 0; i < 2; ++i) {   // 64 columns at a time
              if (64 * i < cols) {
                uint32_t sc[64];
                tmem_ld32_nowait(ts + 64 * i, sc);
                if (64 * i + 32 < cols) tmem_ld32_nowait(ts + 64 * i + 32, sc + 32);
                tmem_wait_ld();
                sum32(sc, 64 * i, vis[2 * i]);
                if (64 * i + 32 < cols) sum32(sc + 32, 64 * i + 32, vis[2 * i + 1]);
              }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar_e[buf]);
          }
          const float2 wp = unpack_f32x2(add_f32x2(w2[0], w2[1]));
          const float w = so_far + (wp.x + wp.y);
          if (MANY && !last) *part = w;
          if (last && slot < keys && !*abort_v && in_bounds(a.status, acc - a.acc + slot, a.ext.acc, CHK_WEIGHTS_ACC))
            acc[slot] = (slot < len ? before : 0.f) + w;
          before = next;
        }
      }
      b0 += n;
      if (b0 >= it.tile1) {
        more = it.next(a, 1, 1, 0);
        b0 = it.tile0;
      }
    }
    if (!ok) {
      *abort_v = 1;
      if ((tid & 31) == 0) report_timeout(a.status, 0x723);
    }
  }
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

template <int DH>
cudaError_t launch_weights(TreeArgs& a, cudaStream_t s) {
  using G = WeightGeom<DH>;
  const int R = a.Hq / a.Hkv * a.N;
  const uint64_t planes = static_cast<uint64_t>(a.B) * a.Hkv;
  if (!encode_rows_map(&a.tm_q, a.q, DH, R, R, planes, AW_CHUNK, DH / 64) ||
      !encode_rows_map(&a.tm_k, a.k, DH, a.S_max, a.S_max, planes, TREE_KEYS, G::blocks))
    return cudaErrorInvalidValue;
  (R > AW_PASS ? k_attn_weights<DH, true> : k_attn_weights<DH, false>)<<<a.groups, AW_THREADS, AW_SMEM, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t weights_init() {
  for (auto f : {k_attn_weights<64, false>, k_attn_weights<128, false>, k_attn_weights<256, false>,
                 k_attn_weights<64, true>, k_attn_weights<128, true>, k_attn_weights<256, true>}) {
    const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, AW_SMEM);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_attention_weights(const TreeArgs& args, cudaStream_t s) {
  TreeArgs a = args;
  a.rtg = 1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&a.groups, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  return a.dh == 64 ? launch_weights<64>(a, s) : a.dh == 128 ? launch_weights<128>(a, s) : launch_weights<256>(a, s);
}

}  // namespace tc
}  // namespace fr

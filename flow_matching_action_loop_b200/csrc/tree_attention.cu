// Attention of drafted tokens over a static KV cache (fr_attention_tree).
//
// The rows of a unit (sample, KV head, row tile) are up to 128 of the (query head, token) pairs that read
// the KV head, so that its K and V are read once for the whole group; its keys come in tiles of 128 slots.
// All units' tiles form one line that the CTAs (one per SM) cut into equal ranges, whatever the samples'
// lengths: a CTA runs the segments of units that lie in its range one after the other.  A segment that is
// its whole unit writes o and lse; one that is part of a unit writes its rows (O, reference, sum) to the
// scratch, and k_tree_merge, chained behind, joins them.  The CTAs that run the row tiles of one KV head do
// so side by side over the same range of keys (with a range of its own for each, the tiles came from HBM
// 2.6 times at 6 x 33000 slots and four row tiles).
//
// A cut costs a segment's end (3 us) and, by its rows, the merge.  So units are cut only where the groups would
// otherwise have many tiles more than their share: more than a sixteenth of the rows (kept_whole); up to four tiles
// never, above a sixteenth of the rows always (single tokens of 32 ragged samples over up to 64 tiles: 111 us cut, 129
// with the shorter ones whole).  60 x 8/1 heads of 256, 24 tokens: 5 tiles 35.5 us cut, 20.2 whole; 80 of them: 6 tiles 45.0 and 44.1, 10 tiles
// 55.5 and 61.3.  40 x 4/4 heads of 128, 8 tokens (8 rows): 4 tiles 20.3 and 19.8, 6 tiles 23.0 and 25.5.
//
// Where it costs few tiles more (tree_cluster), a unit has a cluster of up to 16 CTAs instead, its tiles in
// equal ranges, and the cluster joins its rows over distributed shared memory: no scratch, no second kernel.
// (First every CTA finds what each CTA counts in each row, then all threads sum four features each.  16
// features a thread, references joined on the way, took 10000 cycles instead of 7500 at 192 rows x 128
// features of six CTAs; partial rows through the L2 instead 8000.)
//
// Inside a CTA, per tile t:
//   copy warp     K(t+LA), V(t) by tensor map (128-byte swizzle) into a ring of shared-memory slots
//   MMA warp      S(t+LA) = Q K^T, then O += P(t) V(t): tcgen05, fp32 in tensor memory; P is the A operand
//                 from tensor memory
//   softmax warps two groups of four take the tiles in turn, a thread a row: maximum and sum in fp32,
//                 P = 2^(s - ref)
// One group's loads, maxima and stores thus overlap the other's exponentials (with both groups on one tile,
// half a row each, the multi-function unit idled more than half of a tile's 2500 cycles).  The groups hand the row's
// reference on from tile to tile.  Two score buffers (LA = 2) let both groups have a tile; at dh = 256
// tensor memory has room for one of 128 slots (LA = 1), and S(t+1) is issued once the scores of tile t are in
// registers.  (Buffers of 64 slots would leave room for two; not tried.)
// P has columns of its own: with P in those of the scores, S(t+1) waited for P(t-1) V(t-1) as well (1.97 us a
// tile at dh = 256 instead of 1.6).
// The reference of a row's exponentials moves only when its maximum has grown by more than 2^8 (P stays
// below 2^8, O and the sum keep one reference, O / sum is unchanged): O is rescaled rarely.
// P is rounded to bf16, the tensor core's operand type: half a bf16 step per weight, as much as the
// rounding of o itself.
//
// Single tokens of 32 samples with up to 8191 slots, 8 KV heads of 128: 113 us, 665 MB at 5.9 TB/s (memory); CTAs end
// between 97 and 108 us.  Trees of 63 tokens over 6 x 32767 slots, 8 query heads of 256: 104 us, 940 TFLOP/s, the
// tensor pipe 62 % active (one score buffer); CTAs end between 81 and 91 us, the merge follows.
// Short cases, us from the launch (median CTA; the last one in brackets):
//                                                  set-up  scores  tiles       O    all rows  weights  joined
//   one token over 816 slots, 8/1 heads of 256        1.0    2.3    3.8 (4.7)  5.2    6.5       7.5     8.3, of 9.8
//   4 trees of 24 over 2048, 16/2 heads of 128        1.0    2.2    5.5 (7.1)  6 (8)  8.0 (8.6) 9.2    10.7 (12.5), of 13.8
//   2 x 128 tokens over 4095, 16/16 heads of 64       1.2    2.0   10.6 (14.3) 12 (15) 15 (16)  16     17.6 (18.7), of 22
// so a CTA that runs few tiles of 128 rows takes about 1.3 us for each (S, softmax and P V of one row tile one after
// the other), and the join 4 us: the cluster's barrier, then two trips to the other CTAs' memory.
// k_tree_attn spills: 152 to 160 bytes of stores and 288 to 296 of loads in its shared-line form, 52 and 40 with a
// cluster, none in the merge.
#include <algorithm>
#include <cooperative_groups.h>
#include <type_traits>

#include "fr.h"
#include "tree_device.h"

namespace fr {
namespace tc {
namespace {

using namespace fr::sm100;

constexpr int TA_SOFTMAX = 256;                // softmax threads
constexpr int TA_THREADS = TA_SOFTMAX + 128;   // + a warpgroup of the copy warp and the MMA warp
// Registers: 384 threads are launched with 168 each; a softmax thread holds a row's 128 scores, so that the
// score buffer is free as soon as they are loaded.  (setmaxnreg draws on what the block was launched with: compiled to
// fewer registers, the growing warpgroups would wait for good.  tree_init refuses such a build.)
constexpr int TA_REGS = 168, TA_REGS_SOFTMAX = 208, TA_REGS_OTHER = 88;
static_assert(2 * TA_REGS_SOFTMAX + TA_REGS_OTHER == 3 * TA_REGS, "registers are only moved");
constexpr int TA_CTAS = 148;                   // at most (the SMs of a B200): the scratch holds two segments' rows for each
constexpr float TA_RESCALE = 8.f;
constexpr int TA_CLUSTER = 16;                 // CTAs of a cluster at most

// Shared memory: QB query tiles, then NS ring slots of `piece` bytes.  At dh = 256 a K tile comes as two
// pieces of 128 features, a V tile as two of 64 slots, so that the ring has five slots instead of two.
template <int DH>
struct TreeGeom {
  static constexpr int pieces = DH == 256 ? 2 : 1;              // per K or V tile
  static constexpr int piece = TREE_KEYS * DH * 2 / pieces;     // bytes
  static constexpr int LA = DH == 256 ? 1 : 2;                  // score buffers, tiles that S runs ahead
  static constexpr int QB = LA;                                 // query tiles
  static constexpr int NS = DH == 64 ? 10 : 5;
  static constexpr int q_bytes = 128 * DH * 2;
  static constexpr int smem = QB * q_bytes + NS * piece;
  static constexpr int v_keys = TREE_KEYS / pieces;             // slots per V piece
  static constexpr int k_blocks = DH / 64 / pieces;             // feature blocks per K piece
};

// 32 bytes, a whole sector, to a 32-byte aligned address.
__device__ __forceinline__ void st_global_32(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// Named barriers: 1..4 the two warps of a lane quadrant, 5 and 6 a softmax group, 7..14 the reference of
// (quadrant, group) on its way to the other group.
__device__ __forceinline__ void pair_barrier(int w) { asm volatile("bar.sync %0, 64;" ::"r"(1 + w) : "memory"); }
__device__ __forceinline__ void group_barrier(int g) { asm volatile("bar.sync %0, 128;" ::"r"(5 + g) : "memory"); }
__device__ __forceinline__ void ref_send(int w, int g) { asm volatile("bar.arrive %0, 64;" ::"r"(7 + 2 * w + g) : "memory"); }
__device__ __forceinline__ void ref_wait(int w, int g) { asm volatile("bar.sync %0, 64;" ::"r"(7 + 2 * w + g) : "memory"); }

// The cluster's barrier, in two steps; what the CTAs wrote before the arrival is seen after the wait.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

__device__ __forceinline__ float row_lse(float m, float l) {
  return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// 16 features of a row joined over segments: O and the sum brought to the largest reference.
struct MergedRow {
  float m = -INFINITY, l = 0.f, x = 0.f, o[16] = {};
  bool lost = false;   // a segment whose CTA gave up: its reference is NaN (that of scores never is)
  __device__ __forceinline__ void add(float m2, float l2, float x2, const float* v) {
    const float mn = fmaxf(m, m2);
    lost |= m2 != m2;
    x += x2;   // NaN where a drafted value row was not finite
    if (mn == -INFINITY) {   // no score above -inf: the sums are 0, or NaN with the scores
      l += l2;
      return;
    }
    const float w0 = exp2f(m - mn), w1 = exp2f(m2 - mn);
    m = mn;
    l = l * w0 + l2 * w1;
#pragma unroll
    for (int e = 0; e < 16; ++e) o[e] = o[e] * w0 + v[e] * w1;
  }
  // Row rr of the group (head, token), features 16 fg on.
  __device__ __forceinline__ void store(const TreeArgs& a, int b, int hk, int rr, int fg, int dh) const {
    const int tok = rr % a.N, hq = hk * (a.Hq / a.Hkv) + rr / a.N;
    const float inv = (l == 0.f ? 0.f : 1.f / l) + x;
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = pack_bf16x2(o[2 * i] * inv, o[2 * i + 1] * inv);
    const size_t at = ((static_cast<size_t>(b) * a.N + tok) * a.Hq + hq) * dh + fg * 16;
    if (in_bounds(a.status, at + 15, a.ext.o, CHK_TREE_O)) st_global_32(a.o + at, w);
    const size_t at_lse = (static_cast<size_t>(b) * a.Hq + hq) * a.N + tok;
    if (a.lse && fg == 0 && in_bounds(a.status, at_lse, a.ext.lse, CHK_TREE_LSE)) a.lse[at_lse] = row_lse(m, l);
  }
};

// CL: one cluster per unit.
template <int DH, bool CL>
__global__ void __launch_bounds__(TA_THREADS, 1) k_tree_attn(const __grid_constant__ TreeArgs a) {
  using G = TreeGeom<DH>;
  extern __shared__ __align__(1024) uint8_t dsm[];
  // bar_s, bar_l, bar_p, bar_o [tile parity]: scores written, scores read, P written, O updated.  Each is
  // waited for by one group (or the MMA warp) in every phase: none is passed on an older phase's parity.
  __shared__ uint64_t full[G::NS], empty[G::NS], q_full[2], q_empty[2], bar_s[2], bar_l[2], bar_o[2], bar_p[2], fin_bar;
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  __shared__ TileIter first_seg;           // its segment: the first
  __shared__ int any_seg;
  __shared__ float ref_sh[2][128], sum_sh[2][128];   // of the groups' last tiles
  __shared__ uint32_t bad[2][3][4];        // [group]: drafted value rows of a tile that are not finite
  constexpr uint32_t IDESC_S = idesc_f32acc(FMT_BF16, 128, TREE_KEYS);
  constexpr uint32_t IDESC_O = idesc_f32acc(FMT_BF16, 128, DH) | IDESC_B_MN_MAJOR;
  constexpr int OLD = DH + 4;              // floats per partial row: O, reference, sum, NaN if spoilt
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int g = a.Hq / a.Hkv, R = g * a.N, RT = (R + 127) >> 7, NB = (RT + a.rtg - 1) / a.rtg;
  const int grp = blockIdx.x / a.rtg, r_in = blockIdx.x - grp * a.rtg;
  uint8_t* ring = dsm + G::QB * G::q_bytes;
  volatile int* abort_v = &abort_flag;
  bool ok = true;

  // the copies' state: next ring position, segments whose queries have been fetched
  int pos = 0, segs = 0;
  auto load_q = [&](const TileIter& it) {
    const int qb = segs % G::QB, use = segs / G::QB;
    if (use > 0 && !tree_wait(&q_empty[qb], (use - 1) & 1, a.wait_ns)) return false;
    ++segs;
    mbar_arrive_expect_tx(&q_full[qb], G::q_bytes);
    tma_load_4d(dsm + qb * G::q_bytes, &a.tm_q, 0, it.rt * 128, 0, it.b * a.Hkv + it.hk, &q_full[qb]);
    return true;
  };
  auto load_piece = [&](const CUtensorMap* tm, int key, int block, int plane) {
    const int s = pos % G::NS, use = pos / G::NS;
    if ((use > 0 && !tree_wait(&empty[s], (use - 1) & 1, a.wait_ns)) || *abort_v) return false;
    mbar_arrive_expect_tx(&full[s], G::piece);
    tma_load_4d(ring + s * G::piece, tm, 0, key, block, plane, &full[s]);
    ++pos;
    return true;
  };
  auto load_k = [&](const TileIter& it, int tile) {
    for (int p = 0; p < G::pieces; ++p)
      if (!load_piece(&a.tm_k, tile * TREE_KEYS, p * G::k_blocks, it.b * a.Hkv + it.hk)) return false;
    return true;
  };

  // The copy warp finds the CTA's tiles and starts the first copies while warp 0 allocates tensor memory.
  if (warp == TA_SOFTMAX / 32) {
    if ((tid & 31) == 0) {
      tma_prefetch_map(&a.tm_q);
      tma_prefetch_map(&a.tm_k);
      tma_prefetch_map(&a.tm_v);
      for (int i = 0; i < G::NS; ++i) {
        mbar_init(&full[i], 1);
        mbar_init(&empty[i], 1);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(&q_full[i], 1);
        mbar_init(&q_empty[i], 1);
        mbar_init(&bar_o[i], 1);
        mbar_init(&bar_p[i], 4);
        mbar_init(&bar_s[i], 1);
        mbar_init(&bar_l[i], 4);
      }
      mbar_init(&fin_bar, 1);
      abort_flag = 0;
      fence_mbar_init();
    }
    __syncwarp();
    TileRange r = {};
    if constexpr (!CL) r = tile_range<false>(a, a.Hkv * NB, grp);
    if ((tid & 31) == 0) {
      TileIter it;
      if constexpr (CL) {   // the unit's tiles in equal ranges; no further segment
        const int unit = blockIdx.x / a.cluster, c = blockIdx.x - unit * a.cluster;
        it = {};
        it.rt = unit % RT;
        it.hk = unit / RT % a.Hkv;
        it.b = unit / (RT * a.Hkv);
        it.len = a.lens[it.b];
        it.nb = tiles_of(a, it.len);
        it.tile0 = it.nb * c / a.cluster;
        it.tile1 = it.nb * (c + 1) / a.cluster;
        any_seg = it.tile0 < it.tile1;
        if (it.nb == 0 && it.len >= 0 && c + it.rt + it.hk == 0) report_sample(a.status, CACHE_BAD_LEN, it.b);
      } else {
        it.start(a, r, a.Hkv * NB);
        any_seg = it.next(a, RT, NB, r_in);
      }
      if (any_seg) {
        load_q(it);
        load_k(it, it.tile0);
      }
      first_seg = it;
    }
  }
  if (tid < 24) (&bad[0][0][0])[tid] = 0;
  if (warp == 0) {
    tmem_alloc(&tmem_base, 512);
    tmem_relinquish();
  }
  if constexpr (!CL) grid_dep_launch();   // the merge kernel waits for this whole grid before it reads
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // tensor memory: LA score buffers (128 columns each), two P tiles (64 each), O (dh)
  const uint32_t tS = __shfl_sync(0xffffffffu, tmem_base, 0), tP = tS + 128 * G::LA, tO = tP + 128;
  TileIter it = first_seg;
  bool more = any_seg != 0;

  if (warp >= TA_SOFTMAX / 32) {
    regs_shrink<TA_REGS_OTHER>();
  if (warp == TA_SOFTMAX / 32) {
    // ---------------- copies: pieces in the order the MMA warp takes them, K(0) .. K(LA-1), then K(t+LA), V(t).
    // The places of K tiles past the last are left out, so that V(t) is always at pieces * (2 t + LA + 1).
    if ((tid & 31) == 0 && more) {
      TileIter vi = it;
      int tile = it.tile0, nk = 1;   // K side: K(nk - 1) has been issued
      auto next_k = [&]() {
        if (more && ++tile == it.tile1) {
          more = it.next(a, RT, NB, r_in);
          tile = it.tile0;
          if (more && !load_q(it)) return false;
        }
        if (!more) {
          pos += G::pieces;
          return true;
        }
        ++nk;
        return load_k(it, tile);
      };
      if (G::LA == 2) ok = next_k();
      bool more_v = true;
      for (int vt = vi.tile0; ok && more_v;) {
        ok = next_k();
        const int plane = vi.b * a.Hkv + vi.hk;
        for (int p = 0; ok && p < G::pieces; ++p) ok = load_piece(&a.tm_v, vt * TREE_KEYS + p * G::v_keys, 0, plane);
        if (++vt == vi.tile1) {
          more_v = vi.next(a, RT, NB, r_in);
          vt = vi.tile0;
        }
      }
      if (!ok) {
        *abort_v = 1;
        report_timeout(a.status, 0x710);
      }
      // no copy is in flight when the CTA leaves
      for (int p = max(0, pos - G::NS); p < pos; ++p) {
        const int i = p / G::pieces - G::LA;
        if (i >= 0 ? i % 2 != 0 || i / 2 + G::LA < nk : i + G::LA < nk)   // not a place left out
          mbar_wait(&full[p % G::NS], (p / G::NS) & 1, WAIT_LIMIT_NS);
      }
      for (int s = max(0, segs - G::QB); s < segs; ++s)
        mbar_wait(&q_full[s % G::QB], (s / G::QB) & 1, WAIT_LIMIT_NS);
    }
  } else if (warp == TA_SOFTMAX / 32 + 1) {
    // ---------------- MMAs, the whole warp in step
    if (more) {
      // S runs ahead of P V.  Whichever has what it waits for is issued next, S first (a softmax group may
      // wait for it); in a fixed order S(t+LA) waited for the softmax of tile t-1.  A barrier tells a phase
      // from the one two before it only if the phase between is known to have completed.  The place of
      // K(ts) in the ring held, NS places before, V(tv - 2) or an earlier tile as long as ts <= tv + LA + 1,
      // and P V has been issued up to tv - 1: so S runs at most that far ahead.
      const bool leader = elect_one();
      auto same = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };   // known to be uniform
      TileIter vi = it;
      int ts = 0, tv = 0, seg_s = 0;                        // next S and P V, query tile
      int st = same(it.tile1 - it.tile0), vt = st;          // tiles left of their segments
      bool more_s = true, s_begins = true, v_begins = true; // a segment begins with the tile
      auto test = [](uint64_t* bar, int phase) { return static_cast<unsigned>(mbar_test(bar, phase & 1)); };
      auto landed = [&](int p) {   // a tile's pieces, from ring position p on
        unsigned r = 1u;
#pragma unroll
        for (int i = 0; i < G::pieces; ++i) r &= test(&full[(p + i) % G::NS], (p + i) / G::NS);
        return r;
      };
      const uint64_t dq = smem_desc_sw128(smem_u32(dsm), 16, 1024), dk = smem_desc_sw128(smem_u32(ring), 16, 1024),
                     dv = smem_desc_sw128(smem_u32(ring), G::v_keys * 128, 1024);   // + byte offset / 16
      uint64_t idle = 0;
      const uint64_t limit = a.wait_ns - 1;
      for (;;) {
        const int pk = G::pieces * (ts < G::LA ? ts : 2 * ts - G::LA), pv = G::pieces * (2 * tv + G::LA + 1);
        // every test is on its way before the first answer is used: one after the other they took 700 cycles
        unsigned s_ok = more_s && ts <= tv + G::LA + 1, v_ok = tv < ts;
        if (s_ok) {
          s_ok = landed(pk);
          if (ts >= G::LA) s_ok &= test(&bar_l[(ts - G::LA) & 1], (ts - G::LA) >> 1);
          if (s_begins) s_ok &= test(&q_full[seg_s % G::QB], seg_s / G::QB);
        }
        if (v_ok) v_ok = landed(pv) & test(&bar_p[tv & 1], tv >> 1);
        const bool s_go = __all_sync(0xffffffffu, s_ok), v_go = __all_sync(0xffffffffu, v_ok);
        if (s_go) {
          tc_fence_after();
          const uint64_t qd = dq + (seg_s % G::QB) * (G::q_bytes / 16);
          const uint32_t d = tS + (ts % G::LA) * TREE_KEYS;
#pragma unroll
          for (int p = 0; p < G::pieces; ++p) {
            const uint64_t kd = dk + ((pk + p) % G::NS) * (G::piece / 16);
#pragma unroll
            for (int k = 0; k < G::k_blocks * 4; ++k)
              mma_bf16_warp(leader, d, qd + ((p * G::k_blocks + (k >> 2)) * (128 * 128) + (k & 3) * 32) / 16,
                            kd + ((k >> 2) * (TREE_KEYS * 128) + (k & 3) * 32) / 16, IDESC_S, p > 0 || k > 0);
            mma_commit_warp(leader, &empty[(pk + p) % G::NS]);
          }
          mma_commit_warp(leader, &bar_s[ts & 1]);
          ++ts;
          s_begins = false;
          if (--st == 0) {
            mma_commit_warp(leader, &q_empty[seg_s % G::QB]);
            more_s = same(it.next(a, RT, NB, r_in)) != 0;
            st = same(it.tile1 - it.tile0);
            s_begins = true;
            ++seg_s;
          }
        } else if (v_go) {
          tc_fence_after();
          // steps of 16 slots: those that hold slots in use
          const int steps = same(min(TREE_KEYS, vi.len + a.N - (vi.tile1 - vt) * TREE_KEYS + 15) / 16);
          const uint32_t p_tm = tP + (tv & 1) * 64;
#pragma unroll
          for (int p = 0; p < G::pieces; ++p) {
            const uint64_t vd = dv + ((pv + p) % G::NS) * (G::piece / 16);
#pragma unroll
            for (int k = 0; k < G::v_keys / 16; ++k) {
              const int step = p * (G::v_keys / 16) + k;
              if (step < steps)
                mma_bf16_ta_warp(leader, tO, p_tm + step * 8, vd + k * 128, IDESC_O, (!v_begins || step > 0) ? 1u : 0u);
            }
            mma_commit_warp(leader, &empty[(pv + p) % G::NS]);
          }
          mma_commit_warp(leader, &bar_o[tv & 1]);
          ++tv;
          v_begins = false;
          if (--vt == 0) {
            if (same(vi.next(a, RT, NB, r_in)) == 0) break;
            vt = same(vi.tile1 - vi.tile0);
            v_begins = true;
          }
        } else {
          const uint64_t now = globaltimer();
          if (idle == 0) idle = now;
          if (__any_sync(0xffffffffu, now - idle >= limit || *abort_v)) {
            ok = false;
            break;
          }
          continue;
        }
        idle = 0;
      }
      if (!ok) {
        *abort_v = 1;
        if (leader) report_timeout(a.status, 0x711);
      }
      // every MMA issued has completed before tensor memory is freed
      mma_commit_warp(leader, &fin_bar);
      if (!mbar_wait(&fin_bar, 0, WAIT_LIMIT_NS) && leader) report_timeout(a.status, 0x712);
    }
  }
  } else {
    regs_grow<TA_REGS_SOFTMAX>();
    // ---------------- softmax.  A warp whose wait gave up goes on without waiting (the named barriers need every
    // warp).  Its arrivals come too early from then on, so that no row of the CTA can be trusted: it sets the abort
    // word before them, and nothing is stored, and no partial row counts, that was read after that.
    const int row = tid & 127, hh = tid >> 7, pw = warp & 3;   // row of the tile, group, lane quadrant
    const uint32_t lanes = static_cast<uint32_t>(pw * 32) << 16;
    const float sl2 = a.scale * 1.4426950408889634f;   // scores in log2 units
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (!__all_sync(0xffffffffu, mbar_test(bar, parity)) && ok) {
        ok = __all_sync(0xffffffffu, tree_wait(bar, parity, a.wait_ns) && !*abort_v);
        if (!ok) *abort_v = 1;
      }
      tc_fence_after();
    };
    int t = 0, nbound = 0;
    for (; more; more = it.next(a, RT, NB, r_in)) {
      const int Rv = min(128, R - it.rt * 128);
      const bool work = pw * 32 < Rv;                  // this warp's rows are rows of the unit
      const int rr = it.rt * 128 + row;                // row of the group: (head, token)
      const int tok = rr % a.N, hq = it.hk * g + rr / a.N;
      const uint32_t* words = a.mask ? a.mask + (static_cast<size_t>(it.b) * a.N + min(tok, a.N - 1)) * a.W : nullptr;
      const int len = it.len, keys = len + a.N;
      float ref = -INFINITY, l = 0.f;                  // of this group's tiles so far
      bool spoilt = false;                             // a drafted value row that this row sees is not finite
      for (int tile = it.tile0; tile < it.tile1; ++tile, ++t) {
        if ((t & 1) != hh) continue;
        const int key0 = tile * TREE_KEYS;
        const bool boundary = key0 + TREE_KEYS > len;  // holds drafted slots or slots past them
        uint32_t vis[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};
        if (boundary) {
#pragma unroll
          for (int i = 0; i < 4; ++i) vis[i] = seen_slots(words, tok, a.N, a.W, key0 + 32 * i - len);
        }
        wait(&bar_s[t & 1], (t >> 1) & 1);
        const uint32_t ts = tS + (t % G::LA) * TREE_KEYS + lanes, tp = tP + (t & 1) * 64 + lanes;
        float corr = 1.f, off = 0.f;
        const uint64_t sl22 = pack_f32x2(sl2, sl2);
        uint64_t ps[2] = {0, 0};
        uint32_t s[128];
        if (work) {
#pragma unroll
          for (int i = 0; i < 4; ++i) tmem_ld32_nowait(ts + 32 * i, s + 32 * i);
          tmem_wait_ld();
          tc_fence_before();
        }
        __syncwarp();
        if ((tid & 31) == 0) mbar_arrive(&bar_l[t & 1]);
        auto weights = [&](auto which) {   // P of a quarter of a row
          constexpr int q = decltype(which)::value;
          const uint64_t off2 = pack_f32x2(-off, -off);
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float2 x = unpack_f32x2(fma_f32x2(
                pack_f32x2(__uint_as_float(s[32 * q + e]), __uint_as_float(s[32 * q + e + 1])), sl22, off2));
            const float p0 = ex2_approx(x.x), p1 = ex2_approx(x.y);
            ps[(e >> 1) & 1] = add_f32x2(ps[(e >> 1) & 1], pack_f32x2(p0, p1));
            pk[e >> 1] = pack_bf16x2(p0, p1);
          }
          tmem_st16(tp + 16 * q, pk);
        };
        if (work) {
          if (boundary) {
#pragma unroll
            for (int e = 0; e < 128; ++e)
              if (!((vis[e >> 5] >> (e & 31)) & 1u)) s[e] = 0xff800000u;   // -inf
          }
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int e = 0; e < 128; e += 2) {
            float& m = m4[(e >> 1) & 3];
            m = max3(m, __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
          }
          const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * sl2;
          // the reference after the tile before this one: the other group's
          float before = -INFINITY;
          if (tile > it.tile0) {
            ref_wait(pw, hh ^ 1);
            before = ref_sh[hh ^ 1][row];
          }
          const float nref = mx > before + TA_RESCALE || before == -INFINITY ? fmaxf(mx, before) : before;
          if (tile + 1 < it.tile1) {
            ref_sh[hh][row] = nref;
            ref_send(pw, hh);
          }
          if (nref != -INFINITY) {
            corr = exp2f(before - nref);   // first visible slot: 0
            l *= exp2f(ref - nref);
            off = nref;
          }
          ref = nref;
        }
        wait(&bar_o[t & 1], ((t >> 1) - 1) & 1);   // P(t - 2) has been read
        if (work) {
          weights(std::integral_constant<int, 0>{});
          weights(std::integral_constant<int, 1>{});
          weights(std::integral_constant<int, 2>{});
          weights(std::integral_constant<int, 3>{});
          const float2 pt = unpack_f32x2(add_f32x2(ps[0], ps[1]));
          l += pt.x + pt.y;
          if (tile > it.tile0 && __any_sync(0xffffffffu, corr != 1.f)) {
            wait(&bar_o[(t - 1) & 1], ((t - 1) >> 1) & 1);   // O holds the tiles before this one
#pragma unroll 1
            for (int c0 = 0; c0 < DH; c0 += 32) {
              tmem_ld32_nowait(tO + lanes + c0, s);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) s[e] = __float_as_uint(__uint_as_float(s[e]) * corr);
              tmem_st32(tO + lanes + c0, s);
            }
          }
          tmem_wait_st();
        }
        if (boundary) {
          // Values that a row does not see must not reach it through 0 * NaN: drafted rows that are not
          // finite, and the rows past the drafts in the last step of 16 slots that the product takes, are
          // zeroed where they landed.
          const int pv = G::pieces * (2 * t + G::LA + 1);    // ring position of V(t)
          // (its slots' uses before have landed once P(t - 1) V(t - 1) is done: only then do their phases tell)
          if (G::pieces == 2 && t > 0) wait(&bar_o[(t - 1) & 1], ((t - 1) >> 1) & 1);
          for (int p = 0; p < G::pieces; ++p) wait(&full[(pv + p) % G::NS], ((pv + p) / G::NS) & 1);
          // a thread has one 16-byte column of every 128 / (dh / 8)-th row
          constexpr int CPR = DH / 8, step = 128 / CPR;
          const int c16 = row % CPR;
          uint8_t* vp[G::pieces];
#pragma unroll
          for (int p = 0; p < G::pieces; ++p)
            vp[p] = ring + ((pv + p) % G::NS) * G::piece + (c16 >> 3) * (G::v_keys * 128) + (c16 & 7) * 16;
          auto word = [&](int r) {
            return reinterpret_cast<uint4*>(r < G::v_keys ? vp[0] + r * 128 : vp[G::pieces - 1] + (r - G::v_keys) * 128);
          };
          uint32_t(&bd)[4] = bad[hh][nbound % 3];
          const int r_first = max(0, len - key0) + row / CPR, r_end = min(TREE_KEYS, (keys - key0 + 15) & ~15);
          if (ok)
#pragma unroll 4
            for (int r = r_first; r < r_end; r += step) {
              uint4* x = word(r);
              const uint4 y = *x;
              if (key0 + r >= keys) {
                *x = make_uint4(0, 0, 0, 0);
              } else {
                // a bf16 is not finite if its exponent's bits are all ones
                const uint32_t w[4] = {y.x, y.y, y.z, y.w};
                bool odd = false;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  odd |= (w[e] & 0x7f80u) == 0x7f80u || (w[e] & 0x7f800000u) == 0x7f800000u;
                if (odd) atomicOr(&bd[r >> 5], 1u << (r & 31));
              }
            }
          group_barrier(hh);
          uint32_t odd4[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) odd4[i] = bd[i];
          if (odd4[0] | odd4[1] | odd4[2] | odd4[3]) {
            if (ok)
              for (int r = r_first; r < r_end; r += step)
                if ((bd[r >> 5] >> (r & 31)) & 1u) *word(r) = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 4; ++i) spoilt |= (vis[i] & odd4[i]) != 0;
          }
          fence_proxy_async_smem();
          if (row < 4) bad[hh][(nbound + 2) % 3][row] = 0;
          ++nbound;
        }
        tc_fence_before();
        __syncwarp();
        if ((tid & 31) == 0) mbar_arrive(&bar_p[t & 1]);
      }
      // ---------------- the segment's rows
      wait(&bar_o[(t - 1) & 1], ((t - 1) >> 1) & 1);
      {
        // the groups' sums, brought to the last tile's reference; the sign says that a value row was not finite
        sum_sh[hh][row] = spoilt ? -l : l;
        ref_sh[hh][row] = ref;
        pair_barrier(pw);
        tc_fence_after();   // (the other group's wait for the last product may be the one that counts)
        const float l0 = sum_sh[0][row], l1 = sum_sh[1][row], r0 = ref_sh[0][row], r1 = ref_sh[1][row];
        ref = fmaxf(r0, r1);
        const float at = ref == -INFINITY ? 0.f : ref;
        const float lt = fabsf(l0) * exp2f(r0 - at) + fabsf(l1) * exp2f(r1 - at);
        const float bad_v = signbit(l0) || signbit(l1) ? NAN : 0.f;
        const bool whole = !CL && it.tile1 - it.tile0 == it.nb;
        const bool mine = row < Rv;
        const float inv = whole ? (lt == 0.f ? 0.f : 1.f / lt) + bad_v : 1.f;
        __nv_bfloat16* orow = a.o + (static_cast<size_t>(it.b) * a.N + tok) * a.Hq * DH + static_cast<size_t>(hq) * DH;
        // a partial segment's rows: [dh / 4][rows][4] floats, then (reference, sum, spoilt) [rows][4], so
        // that a warp's rows leave side by side
        // (a cluster's in this CTA's shared memory, whose tiles have all been used)
        const int RW = CL ? 128 : min(128, R);
        float* part = CL ? reinterpret_cast<float*>(dsm) + 4 * row
                         : a.scratch + static_cast<size_t>(2 * blockIdx.x + (it.tile0 > 0 ? 0 : 1)) * RW * OLD + 4 * row;
#pragma unroll 1
        for (int c0 = hh * (DH / 2); c0 < (hh + 1) * (DH / 2); c0 += 32) {
          uint32_t ov[32];
          __syncwarp();   // (rows that store nothing)
          tmem_ld32_nowait(tO + lanes + c0, ov);
          tmem_wait_ld();
          if (!mine || (!CL && whole && *abort_v)) continue;
          if (whole) {
#pragma unroll
            for (int e = 0; e < 32; e += 16) {
              uint32_t w[8];
#pragma unroll
              for (int i = 0; i < 8; ++i)
                w[i] = pack_bf16x2(__uint_as_float(ov[e + 2 * i]) * inv, __uint_as_float(ov[e + 2 * i + 1]) * inv);
              if (in_bounds(a.status, orow - a.o + c0 + e + 15, a.ext.o, CHK_TREE_O)) st_global_32(orow + c0 + e, w);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              float* at = part + static_cast<size_t>((c0 + e) / 4) * RW * 4;
              if (CL || in_bounds(a.status, at - a.scratch + 3, a.ext.scratch, CHK_TREE_SCRATCH))
                *reinterpret_cast<uint4*>(at) = make_uint4(ov[e], ov[e + 1], ov[e + 2], ov[e + 3]);
            }
          }
        }
        tc_fence_before();
        pair_barrier(pw);   // both groups have read O and the sums before either goes on
        if (mine && hh == 0) {
          const bool lost = *abort_v != 0;   // then what either group has read may be wrong, or was left out
          const size_t at_lse = (static_cast<size_t>(it.b) * a.Hq + hq) * a.N + tok;
          if (!whole) {
            float* at = part + static_cast<size_t>(DH / 4) * RW * 4;
            if (CL || in_bounds(a.status, at - a.scratch + 3, a.ext.scratch, CHK_TREE_SCRATCH))
              *reinterpret_cast<float4*>(at) =
                  make_float4(!CL && lost ? NAN : ref, CL ? copysignf(lt, bad_v != bad_v ? -1.f : 1.f) : lt, bad_v, 0.f);
          } else if (a.lse && !lost && in_bounds(a.status, at_lse, a.ext.lse, CHK_TREE_LSE)) {
            a.lse[at_lse] = row_lse(ref, lt);
          }
        }
      }
    }
    if (!ok) {
      *abort_v = 1;
      if ((tid & 31) == 0) report_timeout(a.status, 0x713);
    }
  }
  __syncthreads();
  if constexpr (CL) {
    // A CTA that gave up says so in its rows' references, now that no copy of its own can land on them any more.
    if (*abort_v && tid < 128) reinterpret_cast<float*>(dsm)[(DH / 4 * 128 + tid) * 4] = NAN;
    __syncwarp();
    cluster_arrive();
    // What follows is every warp's.  (Behind the block's barrier: a warp that took its registers back before the
    // softmax warps had theirs would leave them waiting for good.)
    if (warp >= TA_SOFTMAX / 32)
      regs_grow<TA_REGS>();
    else
      regs_shrink<TA_REGS>();
  }
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
  if constexpr (CL) {
    // ---------------- the cluster's rows, over the CTAs that had tiles
    namespace cg = cooperative_groups;
    cg::cluster_group cl = cg::this_cluster();
    cluster_wait();
    const TileIter u = first_seg;
    const int C = a.cluster, Rv = min(128, R - u.rt * 128), n = min(C, u.nb);
    const int me = static_cast<int>(cl.block_rank());
    // the k-th CTA that had tiles: that of tile floor(nb k / n) (with nb < C some have none)
    auto rows_of = [&](int k) {
      const int c = u.nb >= C ? k : ((k + 1) * C - 1) / u.nb;
      return cl.map_shared_rank(reinterpret_cast<const float*>(dsm), c);
    };
    // every CTA: what each of them counts in each row, 2^(reference - largest) / sum
    float* weight = reinterpret_cast<float*>(dsm) + (DH / 4 + 1) * 128 * 4;   // [CTA][row]
    bool lost = false;   // a CTA gave up
    if (tid < Rv) {
      float2 st[TA_CLUSTER];   // reference, sum
#pragma unroll
      for (int k = 0; k < TA_CLUSTER; ++k) {
        st[k] = make_float2(-INFINITY, 0.f);
        if (k < n) st[k] = *reinterpret_cast<const float2*>(rows_of(k) + (DH / 4 * 128 + tid) * 4);
      }
      float m = -INFINITY, l = 0.f;
      bool spoilt = false;
#pragma unroll
      for (int k = 0; k < TA_CLUSTER; ++k) {
        m = fmaxf(m, st[k].x);
        lost |= st[k].x != st[k].x;
        spoilt |= signbit(st[k].y);
      }
      const float at = m == -INFINITY ? 0.f : m;
#pragma unroll
      for (int k = 0; k < TA_CLUSTER; ++k)
        if (k < n) {
          st[k].x = ex2_approx(st[k].x - at);
          l += fabsf(st[k].y) * st[k].x;
        }
      const float inv = spoilt ? NAN : l == 0.f ? 0.f : 1.f / l;
#pragma unroll
      for (int k = 0; k < TA_CLUSTER; ++k)
        if (k < n) weight[k * 128 + tid] = st[k].x * inv;
      if (a.lse && me == 0 && n > 0 && !lost) {
        const int rr = u.rt * 128 + tid, hq = u.hk * g + rr / a.N;
        const size_t at = (static_cast<size_t>(u.b) * a.Hq + hq) * a.N + rr % a.N;
        if (in_bounds(a.status, at, a.ext.lse, CHK_TREE_LSE)) a.lse[at] = row_lse(m, l);
      }
    }
    lost = __syncthreads_or(lost) != 0;
    // four features of a row a thread, the warps' items in turn over the CTAs
    const int items = n > 0 && !lost ? Rv * (DH / 4) : 0;
    for (int i = ((tid >> 5) * C + me) * 32 + (tid & 31); i < items; i += C * TA_THREADS) {
      const int f4 = i / Rv, row = i - f4 * Rv, rr = u.rt * 128 + row;
      float o[4] = {};
      constexpr int UN = 8;   // CTAs in flight: a read of another CTA's memory takes 1000 cycles
      for (int k0 = 0; k0 < n; k0 += UN) {
        float4 v[UN];
#pragma unroll
        for (int k = 0; k < UN; ++k)
          if (k0 + k < n) v[k] = *reinterpret_cast<const float4*>(rows_of(k0 + k) + (f4 * 128 + row) * 4);
#pragma unroll
        for (int k = 0; k < UN; ++k)
          if (k0 + k < n) {
            const float w = weight[(k0 + k) * 128 + row];
            o[0] += v[k].x * w;
            o[1] += v[k].y * w;
            o[2] += v[k].z * w;
            o[3] += v[k].w * w;
          }
      }
      const int hq = u.hk * g + rr / a.N;
      const size_t at = ((static_cast<size_t>(u.b) * a.N + rr % a.N) * a.Hq + hq) * DH + f4 * 4;
      if (in_bounds(a.status, at + 3, a.ext.o, CHK_TREE_O))
        *reinterpret_cast<uint2*>(a.o + at) = make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
    }
    // no CTA leaves while another reads its rows (the loads have returned: o has been stored)
    cluster_arrive_relaxed();
    cluster_wait();
  }
}

// ------------------------------------------------------------------ merge
// Joins the segments of units that lie on several CTAs.  A thread has 16 features of a row and every
// `split`-th segment; grid (row groups, row tiles x KV heads, samples).
constexpr int TM_THREADS = 256;

template <int DH>
__global__ void __launch_bounds__(TM_THREADS) k_tree_merge(const __grid_constant__ TreeArgs a, int split) {
  constexpr int OLD = DH + 4, FG = DH / 16;   // feature groups
  __shared__ Line sh_line;
  __shared__ int sh_cum;
  __shared__ float red[TM_THREADS][17];       // reference, 16 features (one split's threads after the other's)
  __shared__ float red_l[TM_THREADS], red_x[TM_THREADS];
  const int g = a.Hq / a.Hkv, R = g * a.N, RT = (R + 127) >> 7, NB = (RT + a.rtg - 1) / a.rtg;
  const int U = a.Hkv * NB;
  const int b = blockIdx.z, rt = blockIdx.y % RT, hk = blockIdx.y / RT;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rows = TM_THREADS / FG / split;   // rows per CTA, side by side in a warp
  const int Rv = min(128, R - rt * 128), RW = min(128, R);
  const int sub = tid / (rows * FG), fg = tid / rows % FG, row = blockIdx.x * rows + tid % rows;
  const int nb = sample_tiles(a, b);
  if (nb <= TREE_WHOLE || blockIdx.x * rows >= Rv) {   // (leaves when k_tree_attn has, as what follows relies on it)
    grid_dep_wait();
    return;
  }
  if (warp == 0) {
    const Line l = measure_line(a, U, false);
    if (lane == 0) sh_line = l;
  } else if (warp == 1) {
    const int c = tiles_before(a, U, b);
    if (lane == 0) sh_cum = c;
  }
  __syncthreads();
  grid_dep_wait();
  if (kept_whole(a, sh_line, nb)) return;
  const int T = sh_line.T, n = sh_line.n, t0 = sh_cum + (hk * NB + rt / a.rtg) * nb;
  // group c < n holds tiles [T c / n, T (c + 1) / n) of the units that are cut, at least one
  auto holder = [&](int t) { return static_cast<int>((static_cast<long long>(t + 1) * n - 1) / T); };
  const int c0 = holder(t0), c1 = holder(t0 + nb - 1);
  if (c0 == c1) return;   // one segment: written by k_tree_attn
  // a CTA's rows that begin a unit are in its second slot, those that go on with one in its first
  auto slot_of = [&](int c) { return 2 * (c * a.rtg + rt % a.rtg) + (c == c0 ? 1 : 0); };
  MergedRow m;
  if (row < Rv) {
    constexpr int UN = 4;   // segments in flight
    for (int cb = c0 + sub; cb <= c1; cb += UN * split) {
      float4 v[UN][4], st[UN];
#pragma unroll
      for (int i = 0; i < UN; ++i) {
        const int c = cb + i * split;
        if (c <= c1) {
          const float* p = a.scratch + static_cast<size_t>(slot_of(c)) * RW * OLD + 4 * row;
          st[i] = *reinterpret_cast<const float4*>(p + static_cast<size_t>(DH / 4) * RW * 4);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[i][e] = *reinterpret_cast<const float4*>(p + static_cast<size_t>(fg * 4 + e) * RW * 4);
        }
      }
#pragma unroll
      for (int i = 0; i < UN; ++i)
        if (cb + i * split <= c1) m.add(st[i].x, st[i].y, st[i].z, reinterpret_cast<const float*>(v[i]));
    }
  }
  if (split > 1) {
    red[tid][0] = m.lost ? NAN : m.m;
#pragma unroll
    for (int e = 0; e < 16; ++e) red[tid][e + 1] = m.o[e];
    red_l[tid] = m.l;
    red_x[tid] = m.x;
    __syncthreads();
    if (sub == 0)
      for (int w = tid + rows * FG; w < TM_THREADS; w += rows * FG) m.add(red[w][0], red_l[w], red_x[w], &red[w][1]);
  }
  if (row >= Rv || sub != 0 || m.lost) return;
  m.store(a, b, hk, rt * 128 + row, fg, DH);
}

// CTAs per group: all of a unit's row tiles up to 16; of more, the batch size from 8 to 16 that leaves the
// fewest CTAs and row tiles of the last batch idle.
void tree_groups(int ctas, int RT, int& rtg, int& groups) {
  rtg = std::min(RT, 16);
  if (RT > 16) {
    auto busy = [&](int r) { return (ctas / r * r) * static_cast<double>(RT) / ((RT + r - 1) / r * r); };
    for (int r = 15; r >= 8; --r)
      if (busy(r) > busy(rtg)) rtg = r;
  }
  groups = ctas / rtg;
}

template <int DH>
cudaError_t launch_tree(TreeArgs& a, cudaStream_t s) {
  using G = TreeGeom<DH>;
  const int g = a.Hq / a.Hkv, R = g * a.N, RT = (R + 127) / 128;
  const uint64_t planes = static_cast<uint64_t>(a.B) * a.Hkv;
  if (!encode_rows_map(&a.tm_q, a.q, DH, R, R, planes, 128, DH / 64) ||
      !encode_rows_map(&a.tm_k, a.k, DH, a.S_max, a.S_max, planes, TREE_KEYS, G::k_blocks) ||
      !encode_rows_map(&a.tm_v, a.v, DH, a.S_max, a.S_max, planes, G::v_keys, DH / 64))
    return cudaErrorInvalidValue;
  if (a.cluster > 1) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(planes) * RT * a.cluster);
    cfg.blockDim = dim3(TA_THREADS);
    cfg.dynamicSmemBytes = G::smem;
    cfg.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = a.cluster;
    at.val.clusterDim.y = 1;
    at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_tree_attn<DH, true>, a);
  }
  k_tree_attn<DH, false><<<a.groups * a.rtg, TA_THREADS, G::smem, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.S_max <= TREE_WHOLE * TREE_KEYS) return e;   // no unit is cut
  const int64_t units = static_cast<int64_t>(planes) * ((RT + a.rtg - 1) / a.rtg);
  if (units <= a.groups && a.S_max <= a.whole_extra * TREE_KEYS) return e;   // nor here: kept_whole at any lengths
  // segments per unit if every sample is as long as can be
  const int per = static_cast<int>(a.groups / std::min<int64_t>(units, a.groups)) + 1;
  const int split = per > 16 ? 8 : per > 8 ? 4 : per > 4 ? 2 : 1;
  const int rows = TM_THREADS / (DH / 16) / split;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((std::min(R, 128) + rows - 1) / rows, a.Hkv * RT, a.B);
  cfg.blockDim = dim3(TM_THREADS);
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_tree_merge<DH>, a, split);
}

// Clusters of c CTAs that can be resident together, per head dim (64, 128, 256), on each device.
constexpr int MAX_DEVICES = 64;
int g_clusters[MAX_DEVICES][3][TA_CLUSTER + 1];

template <int DH>
cudaError_t tree_init(int* clusters, int* regs) {
  const auto smem = cudaFuncAttributeMaxDynamicSharedMemorySize;
  cudaError_t e = cudaSuccess;
  for (auto f : {k_tree_attn<DH, false>, k_tree_attn<DH, true>}) {
    cudaFuncAttributes fa;
    if ((e = cudaFuncGetAttributes(&fa, f)) != cudaSuccess) return e;
    if (fa.numRegs != TA_REGS) *regs = fa.numRegs;
  }
  e = cudaFuncSetAttribute(k_tree_attn<DH, false>, smem, TreeGeom<DH>::smem);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(k_tree_attn<DH, true>, smem, TreeGeom<DH>::smem);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(k_tree_attn<DH, true>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  for (int c = 2; e == cudaSuccess && c <= TA_CLUSTER; ++c) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(c);
    cfg.blockDim = dim3(TA_THREADS);
    cfg.dynamicSmemBytes = TreeGeom<DH>::smem;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = c;
    at.val.clusterDim.y = 1;
    at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&clusters[c], k_tree_attn<DH, true>, &cfg);
  }
  return e;
}

// CTAs of a unit's cluster, or 1: tiles shared over the whole GPU.  A cluster is taken if all of them are
// resident together and a CTA's tiles, with every sample as long as the cache, are at most CLUSTER_EXTRA above an
// equal share of all tiles over the GPU: a tile takes 0.6 to 1.3 us there, the merge kernel and a CTA's second
// segment 4 us and more.  The lengths are not known here: of one long sample among short ones a cluster's CTAs run
// the same tiles, and the others idle.  So a CTA has at most CLUSTER_TILES.  Single tokens, 72 units of 256
// features, us for clusters / shared tiles: 33 tiles (17 a CTA) 54 / 62 with all samples long, 36 / 26 with one, 44 /
// 45 with lengths from an eighth on; 65 tiles 97 / 103, 62 / 38, 77 / 68; 258 tiles 353 / 356, 249 / 100, 264 / 230.
constexpr int CLUSTER_EXTRA = 5, CLUSTER_TILES = 17;
int tree_cluster(const int* resident, int ctas, int64_t units, int tiles) {
  int best = 1;
  for (int c = 2; c <= TA_CLUSTER && c <= tiles; ++c)
    if (units <= resident[c] && ((tiles + c - 1) / c < (tiles + best - 1) / best)) best = c;
  const int64_t share = units * tiles / ctas;
  return best > 1 && (tiles + best - 1) / best <= std::min<int64_t>(share + CLUSTER_EXTRA, CLUSTER_TILES) ? best : 1;
}

}  // namespace

size_t tree_scratch_bytes(int, int Hq, int Hkv, int N, int S_max, int dh) {
  if (S_max <= TREE_WHOLE * TREE_KEYS) return 0;
  return static_cast<size_t>(2) * TA_CTAS * std::min(128, Hq / Hkv * N) * (dh + 4) * 4;
}

cudaError_t launch_tree_attention(const TreeArgs& args, cudaStream_t s) {
  TreeArgs a = args;
  int dev = 0, nsm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int RT = (a.Hq / a.Hkv * a.N + 127) / 128, ctas = std::min(nsm, TA_CTAS);
  tree_groups(ctas, RT, a.rtg, a.groups);
  a.whole_extra = std::min(128, a.Hq / a.Hkv * a.N) / 16;
  a.cluster = 1;
  if (dev < MAX_DEVICES)
    a.cluster = tree_cluster(g_clusters[dev][a.dh == 64 ? 0 : a.dh == 128 ? 1 : 2], ctas,
                             static_cast<int64_t>(a.B) * a.Hkv * RT, (a.S_max + TREE_KEYS - 1) / TREE_KEYS);
  return a.dh == 64 ? launch_tree<64>(a, s) : a.dh == 128 ? launch_tree<128>(a, s) : launch_tree<256>(a, s);
}

cudaError_t cache_ops_init(int* regs) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || dev >= MAX_DEVICES) return e;
  if ((e = tree_init<64>(g_clusters[dev][0], regs)) != cudaSuccess ||
      (e = tree_init<128>(g_clusters[dev][1], regs)) != cudaSuccess ||
      (e = tree_init<256>(g_clusters[dev][2], regs)) != cudaSuccess)
    return e;
  if ((e = weights_init()) != cudaSuccess) return e;
  return cache_moves_init();
}

}  // namespace tc
}  // namespace fr

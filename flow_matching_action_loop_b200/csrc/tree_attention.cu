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
// Inside a CTA, per tile t:
//   copy warp     K(t+1), V(t) by tensor map (128-byte swizzle) into a ring of shared-memory slots
//   MMA warp      S(t+1) = Q K(t+1)^T, then O += P(t) V(t): tcgen05, fp32 in tensor memory; P is the A
//                 operand from tensor memory
//   softmax warps (8) two threads per row, 64 slots each: running maximum and sum in fp32, P = 2^(s - ref)
// The scores leave their columns for registers at the start of a tile's softmax, so the tensor core works on
// P(t-1) V(t-1) and S(t+1) while the softmax of tile t runs: it waits for neither the other's end (with P
// in the columns of the scores, S(t+1) waited for P(t-1) V(t-1): 1.97 us a tile at dh = 256 instead of
// the 1.54 us of the products).  The reference
// of a row's exponentials moves only when its maximum has grown by more than 2^8 (P stays below 2^8, O and
// the sum keep one reference, O / sum is unchanged): O is rescaled rarely.
// P is rounded to bf16, the tensor core's operand type: half a bf16 step per weight, as much as the
// rounding of o itself.
#include <algorithm>
#include <type_traits>

#include "fr.h"
#include "tree_device.h"

namespace fr {
namespace tc {
namespace {

using namespace fr::sm100;

constexpr int TA_SOFTMAX = 256;                // softmax threads
constexpr int TA_THREADS = TA_SOFTMAX + 64;    // + the copy warp and the MMA warp
constexpr int TA_CTAS = 148;                   // at most: the scratch holds two segments' rows for each
constexpr float TA_RESCALE = 8.f;

// Shared memory: QB query tiles, then NS ring slots of `piece` bytes.  At dh = 256 a K tile comes as two
// pieces of 128 features, a V tile as two of 64 slots, so that the ring has five slots instead of two.
template <int DH>
struct TreeGeom {
  static constexpr int pieces = DH == 256 ? 2 : 1;              // per K or V tile
  static constexpr int piece = TREE_KEYS * DH * 2 / pieces;     // bytes
  static constexpr int QB = DH == 256 ? 1 : 2;
  static constexpr int NS = DH == 64 ? 10 : 5;
  static constexpr int q_bytes = 128 * DH * 2;
  static constexpr int smem = QB * q_bytes + NS * piece;
  static constexpr int v_keys = TREE_KEYS / pieces;             // slots per V piece
  static constexpr int k_blocks = DH / 64 / pieces;             // feature blocks per K piece
};

// 32 bytes, a whole sector, to a 16-byte aligned address that is a multiple of 32 past o's rows.
__device__ __forceinline__ void st_global_32(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

__device__ __forceinline__ void pair_barrier(int w) { asm volatile("bar.sync %0, 64;" ::"r"(1 + w) : "memory"); }
__device__ __forceinline__ void softmax_barrier() { asm volatile("bar.sync 5, 256;" ::: "memory"); }

template <int DH>
__global__ void __launch_bounds__(TA_THREADS, 1) k_tree_attn(const __grid_constant__ TreeArgs a) {
  using G = TreeGeom<DH>;
  extern __shared__ __align__(1024) uint8_t dsm[];
  __shared__ uint64_t full[G::NS], empty[G::NS], q_full[2], q_empty[2], bar_s, bar_l, bar_o[2], bar_p[2], fin_bar;
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  __shared__ TileIter first_seg;           // its segment: the first
  __shared__ int any_seg;
  __shared__ float mx_sh[2][2][128];       // [tile parity][half][row]; a segment's sums at its end
  __shared__ uint32_t bad[3][4];           // drafted value rows of a tile that are not finite
  constexpr uint32_t IDESC_S = idesc_f32acc(FMT_BF16, 128, TREE_KEYS);
  constexpr uint32_t IDESC_O = idesc_f32acc(FMT_BF16, 128, DH) | IDESC_B_MN_MAJOR;
  constexpr int OLD = DH + 4;              // floats per partial row: O, reference, sum, NaN if spoilt
  const int tid = threadIdx.x, warp = tid >> 5;
  const int g = a.Hq / a.Hkv, R = g * a.N, RT = (R + 127) >> 7, NB = (RT + a.rtg - 1) / a.rtg;
  const int grp = blockIdx.x / a.rtg, r_in = blockIdx.x - grp * a.rtg;
  uint8_t* ring = dsm + G::QB * G::q_bytes;
  volatile int* abort_v = &abort_flag;
  bool ok = true;

  // the copies' state: next ring position, segments begun
  int pos = 0, seg = -1;
  auto load_q = [&](const TileIter& it) {
    ++seg;
    const int qb = seg % G::QB, use = seg / G::QB;
    if (use > 0 && !mbar_wait(&q_empty[qb], (use - 1) & 1, WAIT_LIMIT_NS)) return false;
    mbar_arrive_expect_tx(&q_full[qb], G::q_bytes);
    tma_load_4d(dsm + qb * G::q_bytes, &a.tm_q, 0, it.rt * 128, 0, it.b * a.Hkv + it.hk, &q_full[qb]);
    return true;
  };
  auto load_piece = [&](const CUtensorMap* tm, int key, int block, int plane) {
    const int s = pos % G::NS, use = pos / G::NS;
    if ((use > 0 && !mbar_wait(&empty[s], (use - 1) & 1, WAIT_LIMIT_NS)) || *abort_v) return false;
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
      for (int i = 0; i < G::NS; ++i) {
        mbar_init(&full[i], 1);
        mbar_init(&empty[i], 1);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(&q_full[i], 1);
        mbar_init(&q_empty[i], 1);
        mbar_init(&bar_o[i], 1);
        mbar_init(&bar_p[i], TA_SOFTMAX / 32);
      }
      mbar_init(&bar_s, 1);
      mbar_init(&bar_l, TA_SOFTMAX / 32);
      mbar_init(&fin_bar, 1);
      abort_flag = 0;
      fence_mbar_init();
    }
    __syncwarp();
    const TileRange r = tile_range(a, a.Hkv * NB, grp);
    if ((tid & 31) == 0) {
      TileIter it;
      it.start(a, r, a.Hkv * NB);
      any_seg = it.next(a, RT, NB, r_in);
      if (any_seg) {
        load_q(it);
        load_k(it, it.tile0);
      }
      first_seg = it;
    }
  }
  if (tid < 12) bad[tid >> 2][tid & 3] = 0;
  if (warp == 0) {
    tmem_alloc(&tmem_base, 512);
    tmem_relinquish();
  }
  grid_dep_launch();   // the merge kernel waits for this whole grid before it reads
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // tensor memory: scores (128 columns), two P tiles (64 each), O (dh)
  const uint32_t tS = tmem_base, tP = tmem_base + 128, tO = tmem_base + 256;
  TileIter it = first_seg;
  bool more = any_seg != 0;

  if (warp == TA_SOFTMAX / 32) {
    // ---------------- copies: pieces in the order the MMA warp takes them, K(0), then K(t+1), V(t)
    if ((tid & 31) == 0 && more) {
      int tile = it.tile0;   // K(t) has been issued
      for (;;) {
        const int v_plane = it.b * a.Hkv + it.hk, v_key = tile * TREE_KEYS;
        if (++tile == it.tile1) {
          more = it.next(a, RT, NB, r_in);
          tile = it.tile0;
          if (more) ok = load_q(it);
        }
        if (more) ok = ok && load_k(it, tile);
        else pos += G::pieces;   // V(t) is at position pieces * (2 t + 2) for the last tile too
        for (int p = 0; ok && p < G::pieces; ++p) ok = load_piece(&a.tm_v, v_key + p * G::v_keys, 0, v_plane);
        if (!ok || !more) break;
      }
      if (!ok) {
        *abort_v = 1;
        report_timeout(a.status, 0x710);
      }
      // no copy is in flight when the CTA leaves (a position that was left out waits for the slot's last use)
      for (int p = max(0, pos - G::NS); p < pos; ++p) {
        const bool skipped = !more && p >= pos - 2 * G::pieces && p < pos - G::pieces && ok;
        if (!skipped) mbar_wait(&full[p % G::NS], (p / G::NS) & 1, WAIT_LIMIT_NS);
      }
      for (int s = max(0, seg - G::QB + 1); s <= seg; ++s)
        mbar_wait(&q_full[s % G::QB], (s / G::QB) & 1, WAIT_LIMIT_NS);
    }
  } else if (warp == TA_SOFTMAX / 32 + 1) {
    // ---------------- MMAs
    if ((tid & 31) == 0 && more) {
      // The products of S(t+1) and of P(t) V(t) alternate.  What the next ones wait for is tested before the
      // last of the present ones are issued, so that no barrier's latency lies between them.
      int mpos = 0, mseg = -1, tile = it.tile0;   // ring position; S side: segment, tile of segment `it`
      auto landed = [&](int p) { return mbar_test(&full[(mpos + p) % G::NS], ((mpos + p) / G::NS) & 1); };
      auto wait_pieces = [&]() {
        for (int p = 0; p < G::pieces; ++p)
          if (!mbar_wait(&full[(mpos + p) % G::NS], ((mpos + p) / G::NS) & 1, WAIT_LIMIT_NS)) return false;
        return !*abort_v;
      };
      bool more_s = true, s_begins = true;
      auto advance_s = [&]() {   // the next tile of the S side
        s_begins = false;
        if (++tile == it.tile1) {
          more_s = it.next(a, RT, NB, r_in);
          tile = it.tile0;
          s_begins = true;
        }
      };
      auto s_wait = [&](int t) {
        if (s_begins && !mbar_wait(&q_full[(mseg + 1) % G::QB], ((mseg + 1) / G::QB) & 1, WAIT_LIMIT_NS)) return false;
        if (t > 0 && !mbar_wait(&bar_l, (t - 1) & 1, WAIT_LIMIT_NS)) return false;   // S(t - 1) has been read
        return wait_pieces();
      };
      // Returns whether P(t - 1) and V(t - 1) are there.
      auto issue_s = [&](int t) {
        if (s_begins) ++mseg;
        tc_fence_after();
        const uint32_t qa = smem_u32(dsm + (mseg % G::QB) * G::q_bytes);
        bool r = false;
#pragma unroll
        for (int p = 0; p < G::pieces; ++p) {
          const uint32_t ka = smem_u32(ring + ((mpos + p) % G::NS) * G::piece);
#pragma unroll
          for (int k = 0; k < G::k_blocks * 4; ++k) {
            if (p == G::pieces - 1 && k == G::k_blocks * 4 - 2 && t > 0) {
              r = mbar_test(&bar_p[(t - 1) & 1], ((t - 1) >> 1) & 1);
              for (int i = 0; i < G::pieces; ++i) r &= landed(G::pieces + i);
            }
            mma_bf16(tS, smem_desc_sw128(qa + (p * G::k_blocks + (k >> 2)) * (128 * 128) + (k & 3) * 32, 16, 1024),
                     smem_desc_sw128(ka + (k >> 2) * (TREE_KEYS * 128) + (k & 3) * 32, 16, 1024), IDESC_S,
                     p > 0 || k > 0);
          }
          mma_commit(&empty[(mpos + p) % G::NS]);
        }
        mma_commit(&bar_s);
        if (tile + 1 == it.tile1) mma_commit(&q_empty[mseg % G::QB]);
        mpos += G::pieces;
        return r;
      };
      bool v_begins = true, s_ok = false;   // V(t) is a segment's first; S(t + 1) can be issued
      int keys_v = it.len + a.N - tile * TREE_KEYS;
      ok = s_wait(0);
      if (ok) issue_s(0);
      for (int t = 0; ok; ++t) {
        advance_s();
        bool pv_ok = false;
        const int keys_s = more_s ? it.len + a.N - tile * TREE_KEYS : 0;
        if (more_s) {
          ok = s_ok || s_wait(t + 1);
          if (!ok) break;
          pv_ok = issue_s(t + 1);
        } else {
          mpos += G::pieces;
        }
        if (!pv_ok) ok = mbar_wait(&bar_p[t & 1], (t >> 1) & 1, WAIT_LIMIT_NS) && wait_pieces();
        if (!ok) break;
        tc_fence_after();
        const int steps = min(TREE_KEYS, keys_v + 15) / 16;   // of 16 slots: those that hold slots in use
        s_ok = false;
#pragma unroll
        for (int p = 0; p < G::pieces; ++p) {
          const uint32_t va = smem_u32(ring + ((mpos + p) % G::NS) * G::piece);
#pragma unroll
          for (int k = 0; k < G::v_keys / 16; ++k) {
            const int step = p * (G::v_keys / 16) + k;
            if (step == TREE_KEYS / 16 - 1 && more_s && tile + 1 < it.tile1) {
              // S(t + 2) follows in the same segment
              s_ok = mbar_test(&bar_l, (t + 1) & 1);
              for (int i = 0; i < G::pieces; ++i) s_ok &= landed(G::pieces + i);
            }
            if (step < steps)
              mma_bf16_ta(tO, tP + (t & 1) * 64 + step * 8, smem_desc_sw128(va + k * 2048, G::v_keys * 128, 1024), IDESC_O,
                          (!v_begins || step > 0) ? 1u : 0u);
          }
          mma_commit(&empty[(mpos + p) % G::NS]);
        }
        mma_commit(&bar_o[t & 1]);
        mpos += G::pieces;
        if (!more_s) break;
        v_begins = s_begins;
        keys_v = keys_s;
      }
      if (!ok) {
        *abort_v = 1;
        report_timeout(a.status, 0x711);
      }
      // every MMA issued has completed before tensor memory is freed
      mma_commit(&fin_bar);
      if (!mbar_wait(&fin_bar, 0, WAIT_LIMIT_NS)) report_timeout(a.status, 0x712);
    }
  } else {
    // ---------------- softmax.  A warp whose wait gave up goes on without waiting (the named barriers
    // need every warp) and stores nothing.
    const int row = tid & 127, hh = tid >> 7, pw = warp & 3;
    const uint32_t lanes = static_cast<uint32_t>(pw * 32) << 16;
    const float sl2 = a.scale * 1.4426950408889634f;   // scores in log2 units
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (!__all_sync(0xffffffffu, mbar_test(bar, parity)) && ok)
        ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, WAIT_LIMIT_NS) && !*abort_v);
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
      float ref = -INFINITY, l = 0.f;
      bool spoilt = false;                             // a drafted value row that this row sees is not finite
      for (int tile = it.tile0; tile < it.tile1; ++tile, ++t) {
        const int key0 = tile * TREE_KEYS;
        const bool boundary = key0 + TREE_KEYS > len;  // holds drafted slots or slots past them
        uint32_t vis[2] = {0xffffffffu, 0xffffffffu};
        if (boundary) {
          const int j0 = key0 + 64 * hh - len;
          vis[0] = seen_slots(words, tok, a.N, j0);
          vis[1] = seen_slots(words, tok, a.N, j0 + 32);
        }
        wait(&bar_s, t & 1);
        uint32_t s[64];
        if (work) {
          tmem_ld32_nowait(tS + lanes + 64 * hh, s);
          tmem_ld32_nowait(tS + lanes + 64 * hh + 32, s + 32);
          tmem_wait_ld();
          tc_fence_before();
        }
        __syncwarp();
        if ((tid & 31) == 0) mbar_arrive(&bar_l);
        if (work) {
          if (boundary) {
#pragma unroll
            for (int e = 0; e < 64; ++e)
              if (!((vis[e >> 5] >> (e & 31)) & 1u)) s[e] = 0xff800000u;   // -inf
          }
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int e = 0; e < 64; e += 2) {
            float& m = m4[(e >> 1) & 3];
            m = max3(m, __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
          }
          const float mine = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
          mx_sh[t & 1][hh][row] = mine;
          pair_barrier(pw);
          const float mx = fmaxf(mine, mx_sh[t & 1][hh ^ 1][row]) * sl2;
          const float nref = mx > ref + TA_RESCALE || ref == -INFINITY ? fmaxf(mx, ref) : ref;
          const float corr = nref == -INFINITY ? 1.f : exp2f(ref - nref);   // first visible slot: 0
          const float off = nref == -INFINITY ? 0.f : nref;
          const uint64_t sl22 = pack_f32x2(sl2, sl2), off2 = pack_f32x2(-off, -off);
          uint64_t ps[2] = {0, 0};
          uint32_t pk[32];
#pragma unroll
          for (int e = 0; e < 64; e += 2) {
            const float2 x = unpack_f32x2(
                fma_f32x2(pack_f32x2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), sl22, off2));
            const float p0 = ex2_approx(x.x), p1 = ex2_approx(x.y);
            ps[(e >> 1) & 1] = add_f32x2(ps[(e >> 1) & 1], pack_f32x2(p0, p1));
            pk[e >> 1] = pack_bf16x2(p0, p1);
          }
          // P(t - 2) has been read: its product was issued before S(t), whose commit covers it
          tmem_st32(tP + (t & 1) * 64 + lanes + 32 * hh, pk);
          const float2 pt = unpack_f32x2(add_f32x2(ps[0], ps[1]));
          l = l * corr + (pt.x + pt.y);
          if (tile > it.tile0 && __any_sync(0xffffffffu, corr != 1.f)) {
            wait(&bar_o[(t - 1) & 1], ((t - 1) >> 1) & 1);   // O holds the tiles before this one
#pragma unroll 1
            for (int c0 = hh * (DH / 2); c0 < (hh + 1) * (DH / 2); c0 += 32) {
              uint32_t ov[32];
              tmem_ld32_nowait(tO + lanes + c0, ov);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * corr);
              tmem_st32(tO + lanes + c0, ov);
            }
          }
          ref = nref;
          tmem_wait_st();
        }
        if (boundary) {
          // Values that a row does not see must not reach it through 0 * NaN: drafted rows that are not
          // finite, and the rows past the drafts in the last step of 16 slots that the product takes, are
          // zeroed where they landed.
          const int pv = G::pieces * (2 * t + 2);            // ring position of V(t)
          for (int p = 0; p < G::pieces; ++p) wait(&full[(pv + p) % G::NS], ((pv + p) / G::NS) & 1);
          constexpr int CPR = DH / 8;                        // 16-byte words per row
          auto word = [&](int r, int c) {
            const int vp = r / G::v_keys;
            return reinterpret_cast<uint4*>(ring + ((pv + vp) % G::NS) * G::piece +
                                            (c >> 3) * (G::v_keys * 128) + (r - vp * G::v_keys) * 128 + (c & 7) * 16);
          };
          uint32_t(&bd)[4] = bad[nbound % 3];
          const int r0 = max(0, len - key0), items = (min(TREE_KEYS, (keys - key0 + 15) & ~15) - r0) * CPR;
          if (ok)
#pragma unroll 4
            for (int i = tid; i < items; i += TA_SOFTMAX) {
              const int r = r0 + i / CPR;
              uint4* x = word(r, i % CPR);
              if (key0 + r >= keys) {
                *x = make_uint4(0, 0, 0, 0);
              } else {
                const uint4 y = *x;
                const uint32_t w[4] = {y.x, y.y, y.z, y.w};
                bool odd = false;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  odd |= (w[e] & 0x7f80u) == 0x7f80u || (w[e] & 0x7f800000u) == 0x7f800000u;
                if (odd) atomicOr(&bd[r >> 5], 1u << (r & 31));
              }
            }
          softmax_barrier();
          const uint32_t odd4[4] = {bd[0], bd[1], bd[2], bd[3]};
          if (odd4[0] | odd4[1] | odd4[2] | odd4[3]) {
            if (ok)
              for (int i = tid; i < items; i += TA_SOFTMAX) {
                const int r = r0 + i / CPR;
                if ((odd4[r >> 5] >> (r & 31)) & 1u) *word(r, i % CPR) = make_uint4(0, 0, 0, 0);
              }
            if ((vis[0] & odd4[2 * hh]) | (vis[1] & odd4[2 * hh + 1])) spoilt = true;
          }
          fence_proxy_async_smem();
          if (tid < 4) bad[(nbound + 2) % 3][tid] = 0;
          ++nbound;
        }
        tc_fence_before();
        __syncwarp();
        if ((tid & 31) == 0) mbar_arrive(&bar_p[t & 1]);
      }
      // ---------------- the segment's rows
      wait(&bar_o[(t - 1) & 1], ((t - 1) >> 1) & 1);
      if (work) {
        // the halves' sums; the sign says that a value row was not finite
        float(&sums)[2][128] = mx_sh[t & 1];   // last read before this tile's barrier
        sums[hh][row] = spoilt ? -l : l;
        pair_barrier(pw);
        const float l0 = sums[0][row], l1 = sums[1][row];
        pair_barrier(pw);                      // before the next tile's maxima
        const float lt = fabsf(l0) + fabsf(l1);
        const float bad_v = signbit(l0) || signbit(l1) ? NAN : 0.f;
        const bool whole = it.tile1 - it.tile0 == it.nb;
        const bool mine = row < Rv && ok;
        const float inv = whole ? (lt == 0.f ? 0.f : 1.f / lt) + bad_v : 1.f;
        __nv_bfloat16* orow = a.o + (static_cast<size_t>(it.b) * a.N + tok) * a.Hq * DH + static_cast<size_t>(hq) * DH;
        // a partial segment's rows: [dh / 4][rows][4] floats, then (reference, sum, spoilt) [rows][4], so
        // that a warp's rows leave side by side
        const int RW = min(128, R);
        float* part = a.scratch + static_cast<size_t>(2 * blockIdx.x + (it.tile0 > 0 ? 0 : 1)) * RW * OLD + 4 * row;
#pragma unroll 1
        for (int c0 = hh * (DH / 2); c0 < (hh + 1) * (DH / 2); c0 += 32) {
          uint32_t ov[32];
          tmem_ld32_nowait(tO + lanes + c0, ov);
          tmem_wait_ld();
          if (!mine) continue;
          if (whole) {
#pragma unroll
            for (int e = 0; e < 32; e += 16) {
              uint32_t w[8];
#pragma unroll
              for (int i = 0; i < 8; ++i)
                w[i] = pack_bf16x2(__uint_as_float(ov[e + 2 * i]) * inv, __uint_as_float(ov[e + 2 * i + 1]) * inv);
              st_global_32(orow + c0 + e, w);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<uint4*>(part + static_cast<size_t>((c0 + e) / 4) * RW * 4) =
                  make_uint4(ov[e], ov[e + 1], ov[e + 2], ov[e + 3]);
          }
        }
        if (mine && hh == 0) {
          if (!whole) {
            *reinterpret_cast<float4*>(part + static_cast<size_t>(DH / 4) * RW * 4) = make_float4(ref, lt, bad_v, 0.f);
          } else if (a.lse) {
            a.lse[(static_cast<size_t>(it.b) * a.Hq + hq) * a.N + tok] =
                ref == -INFINITY ? -INFINITY : (ref + log2f(lt)) * 0.6931471805599453f;
          }
        }
        tc_fence_before();
      }
    }
    if (!ok) {
      *abort_v = 1;
      if ((tid & 31) == 0) report_timeout(a.status, 0x713);
    }
  }
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

// ------------------------------------------------------------------ merge
// Joins the segments of units that lie on several CTAs.  A thread has 16 features of a row and every
// `split`-th segment; grid (row groups, row tiles x KV heads, samples).
constexpr int TM_THREADS = 256;

template <int DH>
__global__ void __launch_bounds__(TM_THREADS) k_tree_merge(const __grid_constant__ TreeArgs a, int split) {
  constexpr int OLD = DH + 4, FG = DH / 16;   // feature groups
  __shared__ long long sh_T, sh_cum;
  __shared__ float red[TM_THREADS][17];       // reference, 16 features (one split's threads after the other's)
  __shared__ float red_l[TM_THREADS], red_x[TM_THREADS];
  const int g = a.Hq / a.Hkv, R = g * a.N, RT = (R + 127) >> 7, NB = (RT + a.rtg - 1) / a.rtg;
  const int U = a.Hkv * NB;
  const int b = blockIdx.z, rt = blockIdx.y % RT, hk = blockIdx.y / RT;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rows = TM_THREADS / FG / split;   // rows per CTA, side by side in a warp
  const int Rv = min(128, R - rt * 128), RW = min(128, R);
  const int sub = tid / (rows * FG), fg = tid / rows % FG, row = blockIdx.x * rows + tid % rows;
  if (warp == 0) {
    const long long T = tiles_before(a, U, a.B);
    if (lane == 0) sh_T = T;
  } else if (warp == 1) {
    const long long c = tiles_before(a, U, b);
    if (lane == 0) sh_cum = c;
  }
  const int nb = sample_tiles(a, b);
  __syncthreads();
  grid_dep_wait();
  if (nb == 0 || blockIdx.x * rows >= Rv) return;
  const long long T = sh_T, t0 = sh_cum + static_cast<long long>(hk * NB + rt / a.rtg) * nb;
  // group c < n holds tiles [T c / n, T (c + 1) / n), at least one
  const int n = static_cast<int>(min(T, static_cast<long long>(a.groups)));
  auto holder = [&](long long t) { return static_cast<int>(div_long((t + 1) * n - 1, T)); };
  const int c0 = holder(t0), c1 = holder(t0 + nb - 1);
  if (c0 == c1) return;   // one segment: written by k_tree_attn
  // a CTA's rows that begin a unit are in its second slot, those that go on with one in its first
  auto slot_of = [&](int c) { return 2 * (c * a.rtg + rt % a.rtg) + (c == c0 ? 1 : 0); };
  float m = -INFINITY, l = 0.f, x = 0.f, o[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) o[e] = 0.f;
  auto add = [&](float m2, float l2, float x2, const float* v) {
    const float mn = fmaxf(m, m2);
    if (mn == -INFINITY) return;
    const float w0 = exp2f(m - mn), w1 = exp2f(m2 - mn);
    m = mn;
    l = l * w0 + l2 * w1;
    x += x2;
#pragma unroll
    for (int e = 0; e < 16; ++e) o[e] = o[e] * w0 + v[e] * w1;
  };
  if (row < Rv) {
    constexpr int UN = 2;   // segments in flight
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
        if (cb + i * split <= c1) add(st[i].x, st[i].y, st[i].z, reinterpret_cast<const float*>(v[i]));
    }
  }
  if (split > 1) {
    red[tid][0] = m;
#pragma unroll
    for (int e = 0; e < 16; ++e) red[tid][e + 1] = o[e];
    red_l[tid] = l;
    red_x[tid] = x;
    __syncthreads();
    if (sub == 0)
      for (int w = tid + rows * FG; w < TM_THREADS; w += rows * FG) add(red[w][0], red_l[w], red_x[w], &red[w][1]);
  }
  if (row >= Rv || sub != 0) return;
  const int rr = rt * 128 + row, tok = rr % a.N, hq = hk * g + rr / a.N;
  const float inv = (l == 0.f ? 0.f : 1.f / l) + x;
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = pack_bf16x2(o[2 * i] * inv, o[2 * i + 1] * inv);
  st_global_32(a.o + (static_cast<size_t>(b) * a.N + tok) * a.Hq * DH + static_cast<size_t>(hq) * DH + fg * 16, w);
  if (a.lse && fg == 0)
    a.lse[(static_cast<size_t>(b) * a.Hq + hq) * a.N + tok] =
        m == -INFINITY ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
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
  k_tree_attn<DH><<<a.groups * a.rtg, TA_THREADS, G::smem, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.S_max <= TREE_KEYS) return e;   // a unit of one tile is never split
  // segments per unit if every sample is as long as can be
  const int64_t units = static_cast<int64_t>(planes) * ((RT + a.rtg - 1) / a.rtg);
  const int per = static_cast<int>(a.groups / std::min<int64_t>(units, a.groups)) + 1;
  const int split = per > 32 ? 8 : per > 16 ? 4 : per > 8 ? 2 : 1;
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

template <int DH>
cudaError_t tree_init() {
  return cudaFuncSetAttribute(k_tree_attn<DH>, cudaFuncAttributeMaxDynamicSharedMemorySize, TreeGeom<DH>::smem);
}

}  // namespace

size_t tree_scratch_bytes(int, int Hq, int Hkv, int N, int S_max, int dh) {
  if (S_max <= TREE_KEYS) return 0;
  return static_cast<size_t>(2) * TA_CTAS * std::min(128, Hq / Hkv * N) * (dh + 4) * 4;
}

cudaError_t launch_tree_attention(const TreeArgs& args, cudaStream_t s) {
  TreeArgs a = args;
  int dev = 0, nsm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  tree_groups(std::min(nsm, TA_CTAS), (a.Hq / a.Hkv * a.N + 127) / 128, a.rtg, a.groups);
  return a.dh == 64 ? launch_tree<64>(a, s) : a.dh == 128 ? launch_tree<128>(a, s) : launch_tree<256>(a, s);
}

cudaError_t cache_ops_init() {
  cudaError_t e;
  if ((e = tree_init<64>()) != cudaSuccess || (e = tree_init<128>()) != cudaSuccess ||
      (e = tree_init<256>()) != cudaSuccess)
    return e;
  if ((e = weights_init()) != cudaSuccess) return e;
  return cache_moves_init();
}

}  // namespace tc
}  // namespace fr

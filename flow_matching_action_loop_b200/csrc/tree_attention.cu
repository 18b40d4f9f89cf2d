// Attention of drafted tokens over a static KV cache (fr_attention_tree).
//
// The rows of a unit (sample, KV head, row tile) are up to 128 of the (query head, token) pairs that read
// the KV head, so that its K and V are read once for the whole group; its keys come in tiles of 128 slots.
// All units' tiles form one line that the CTAs (one per SM) cut into equal ranges, whatever the samples'
// lengths: a CTA runs the segments of units that lie in its range one after the other.  A segment that is
// its whole unit writes o and lse; one that is part of a unit writes its rows (O, reference, sum) to the
// scratch, and k_tree_merge, chained behind, joins them.
//
// Inside a CTA, per tile t:
//   copy warp     K(t+1), V(t) by tensor map (128-byte swizzle) into a ring of shared-memory slots
//   MMA warp      S(t+1) = Q K(t+1)^T, then O += P(t) V(t): tcgen05, fp32 in tensor memory; P is the A
//                 operand from tensor memory, in the columns of the scores it came from
//   softmax warps (8) two threads per row, 64 slots each: running maximum and sum in fp32, P = 2^(s - ref)
// so the tensor core works on S(t+1) and P(t-1) V(t-1) while the softmax of tile t runs.  The reference
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

__device__ __forceinline__ void pair_barrier(int w) { asm volatile("bar.sync %0, 64;" ::"r"(1 + w) : "memory"); }
__device__ __forceinline__ void softmax_barrier() { asm volatile("bar.sync 5, 256;" ::: "memory"); }

template <int DH>
__global__ void __launch_bounds__(TA_THREADS, 1) k_tree_attn(const __grid_constant__ TreeArgs a) {
  using G = TreeGeom<DH>;
  extern __shared__ __align__(1024) uint8_t dsm[];
  __shared__ uint64_t full[G::NS], empty[G::NS], q_full[2], q_empty[2], bar_s[2], bar_o[2], bar_p[2], fin_bar;
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  __shared__ TileRange range;
  __shared__ float mx_sh[2][2][128];       // [tile parity][half][row]; a segment's sums at its end
  __shared__ uint32_t bad[3][4];           // drafted value rows of a tile that are not finite
  constexpr uint32_t IDESC_S = idesc_f32acc(FMT_BF16, 128, TREE_KEYS);
  constexpr uint32_t IDESC_O = idesc_f32acc(FMT_BF16, 128, DH) | IDESC_B_MN_MAJOR;
  constexpr int OLD = DH + 4;              // floats per partial row: O, reference, sum, NaN if spoilt
  const int tid = threadIdx.x, warp = tid >> 5;
  const int g = a.Hq / a.Hkv, R = g * a.N, RT = (R + 127) >> 7, U = a.Hkv * RT;

  if (tid == 0) {
    for (int i = 0; i < G::NS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
      mbar_init(&bar_s[i], 1);
      mbar_init(&bar_o[i], 1);
      mbar_init(&bar_p[i], TA_SOFTMAX / 32);
    }
    mbar_init(&fin_bar, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (tid < 12) bad[tid >> 2][tid & 3] = 0;
  if (warp == 0) {
    tmem_alloc(&tmem_base, 512);
    tmem_relinquish();
  }
  if (warp == 1) {
    const TileRange r = tile_range(a, U);
    if ((tid & 31) == 0) range = r;
  }
  grid_dep_launch();   // the merge kernel waits for this whole grid before it reads
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tS = tmem_base, tO = tmem_base + 256;
  volatile int* abort_v = &abort_flag;
  const TileRange rg = range;
  const int nT = static_cast<int>(min(rg.t1 - rg.t0, static_cast<long long>(INT_MAX)));
  TileIter it;
  it.start(a, rg, U);
  bool ok = true;

  if (warp == TA_SOFTMAX / 32) {
    // ---------------- copies: pieces in the order the MMA warp takes them, K(0), then K(t+1), V(t)
    if ((tid & 31) == 0 && nT > 0) {
      int pos = 0, seg = -1, t_end = 0;       // ring position; segment, first tile after it
      long long vt_cum = 0;
      (void)vt_cum;
      auto slot_for = [&](uint8_t*& dst, uint64_t*& bar) {
        const int s = pos % G::NS, use = pos / G::NS;
        if (use > 0 && !mbar_wait(&empty[s], (use - 1) & 1, WAIT_LIMIT_NS)) return false;
        if (*abort_v) return false;
        dst = dsm + G::QB * G::q_bytes + s * G::piece;
        bar = &full[s];
        mbar_arrive_expect_tx(bar, G::piece);
        ++pos;
        return true;
      };
      // the K side runs one tile ahead of the V side: V's plane and first slot of the tile before
      int v_plane = 0, v_key = 0;
      for (int t = 0; ok && t <= nT; ++t) {
        int k_plane = 0, k_key = 0;
        if (t < nT) {
          if (t == t_end) {   // next segment: its query rows
            it.next(a, RT);
            t_end += it.tile1 - it.tile0;
            ++seg;
            const int qb = seg % G::QB, use = seg / G::QB;
            if (use > 0 && !mbar_wait(&q_empty[qb], (use - 1) & 1, WAIT_LIMIT_NS)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(&q_full[qb], G::q_bytes);
            tma_load_4d(dsm + qb * G::q_bytes, &a.tm_q, 0, it.rt * 128, 0, it.b * a.Hkv + it.hk, &q_full[qb]);
          }
          k_plane = it.b * a.Hkv + it.hk;
          k_key = (it.tile1 - (t_end - t)) * TREE_KEYS;
          for (int p = 0; ok && p < G::pieces; ++p) {
            uint8_t* dst;
            uint64_t* bar;
            ok = slot_for(dst, bar);
            if (ok) tma_load_4d(dst, &a.tm_k, 0, k_key, p * G::k_blocks, k_plane, bar);
          }
        }
        if (t > 0)
          for (int p = 0; ok && p < G::pieces; ++p) {
            uint8_t* dst;
            uint64_t* bar;
            ok = slot_for(dst, bar);
            if (ok) tma_load_4d(dst, &a.tm_v, 0, v_key + p * G::v_keys, 0, v_plane, bar);
          }
        v_plane = k_plane;
        v_key = k_key;
      }
      if (!ok) {
        *abort_v = 1;
        report_timeout(a.status, 0x710);
      }
      // no copy is in flight when the CTA leaves
      for (int p = max(0, pos - G::NS); p < pos; ++p) mbar_wait(&full[p % G::NS], (p / G::NS) & 1, WAIT_LIMIT_NS);
      for (int s = max(0, seg - G::QB + 1); s <= seg; ++s)
        mbar_wait(&q_full[s % G::QB], (s / G::QB) & 1, WAIT_LIMIT_NS);
    }
  } else if (warp == TA_SOFTMAX / 32 + 1) {
    // ---------------- MMAs
    if ((tid & 31) == 0 && nT > 0) {
      int pos = 0, seg = -1, t_end = 0;
      auto piece = [&](uint32_t& addr) {   // the next piece, once it has landed
        const int s = pos % G::NS;
        if (!mbar_wait(&full[s], (pos / G::NS) & 1, WAIT_LIMIT_NS) || *abort_v) return false;
        tc_fence_after();
        addr = smem_u32(dsm + G::QB * G::q_bytes + s * G::piece);
        return true;
      };
      auto issue_s = [&](int t) {
        if (t == t_end) {
          it.next(a, RT);
          t_end += it.tile1 - it.tile0;
          ++seg;
          if (!mbar_wait(&q_full[seg % G::QB], (seg / G::QB) & 1, WAIT_LIMIT_NS)) return false;
        }
        // the columns still hold P(t - 2) until O += P(t - 2) V(t - 2) is done
        if (t >= 2 && !mbar_wait(&bar_o[t & 1], ((t - 2) >> 1) & 1, WAIT_LIMIT_NS)) return false;
        const uint32_t qa = smem_u32(dsm + (seg % G::QB) * G::q_bytes);
#pragma unroll
        for (int p = 0; p < G::pieces; ++p) {
          uint32_t ka;
          if (!piece(ka)) return false;
#pragma unroll
          for (int k = 0; k < G::k_blocks * 4; ++k)
            mma_bf16(tS + (t & 1) * TREE_KEYS,
                     smem_desc_sw128(qa + (p * G::k_blocks + (k >> 2)) * (128 * 128) + (k & 3) * 32, 16, 1024),
                     smem_desc_sw128(ka + (k >> 2) * (TREE_KEYS * 128) + (k & 3) * 32, 16, 1024), IDESC_S,
                     p > 0 || k > 0);
          mma_commit(&empty[pos % G::NS]);
          ++pos;
        }
        mma_commit(&bar_s[t & 1]);
        if (t + 1 == t_end) mma_commit(&q_empty[seg % G::QB]);
        return true;
      };
      TileIter vi = it;   // the V side: where segments begin
      int v_end = 0, v_first = 0;
      ok = issue_s(0);
      for (int t = 0; ok && t < nT; ++t) {
        if (t + 1 < nT) ok = issue_s(t + 1);
        if (t == v_end) {
          vi.next(a, RT);
          v_first = t;
          v_end += vi.tile1 - vi.tile0;
        }
        ok = ok && mbar_wait(&bar_p[t & 1], (t >> 1) & 1, WAIT_LIMIT_NS);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int p = 0; p < G::pieces; ++p) {
          uint32_t va;
          ok = piece(va);
          if (!ok) break;
#pragma unroll
          for (int k = 0; k < G::v_keys / 16; ++k)
            mma_bf16_ta(tO, tS + (t & 1) * TREE_KEYS + (p * (G::v_keys / 16) + k) * 8,
                        smem_desc_sw128(va + k * 2048, G::v_keys * 128, 1024), IDESC_O,
                        (t > v_first || p > 0 || k > 0) ? 1u : 0u);
          mma_commit(&empty[pos % G::NS]);
          ++pos;
        }
        mma_commit(&bar_o[t & 1]);
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
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, WAIT_LIMIT_NS) && !*abort_v);
      tc_fence_after();
    };
    int t = 0, nbound = 0;
    while (it.next(a, RT)) {
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
          // Values that a row does not see must not reach it through 0 * NaN: rows past the drafts, and
          // drafted rows that are not finite, are zeroed where they landed.
          const int pv = G::pieces * (min(t + 2, nT) + t);   // ring position of V(t)
          for (int p = 0; p < G::pieces; ++p) wait(&full[(pv + p) % G::NS], ((pv + p) / G::NS) & 1);
          const int key = key0 + row;
          uint32_t(&bd)[4] = bad[nbound % 3];
          if (key >= len && ok) {
            const int vp = row / G::v_keys;
            uint8_t* v0 = dsm + G::QB * G::q_bytes + ((pv + vp) % G::NS) * G::piece + (row - vp * G::v_keys) * 128;
            constexpr int HB = DH == 64 ? 1 : DH / 128;      // feature blocks per thread (a half-row at dh = 64)
            bool clear = key >= keys;
            if (!clear) {
#pragma unroll 1
              for (int i = 0; i < (DH == 64 ? 4 : HB * 8); ++i) {
                const uint4 x = *reinterpret_cast<const uint4*>(
                    v0 + (DH == 64 ? hh * 64 + i * 16 : (hh * HB + (i >> 3)) * (G::v_keys * 128) + (i & 7) * 16));
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  clear |= (w[e] & 0x7f80u) == 0x7f80u || (w[e] & 0x7f800000u) == 0x7f800000u;
              }
              if (clear) atomicOr(&bd[row >> 5], 1u << (row & 31));
            }
          }
          softmax_barrier();
          if (key >= len && ok && (key >= keys || ((bd[row >> 5] >> (row & 31)) & 1u))) {
            const int vp = row / G::v_keys;
            uint8_t* v0 = dsm + G::QB * G::q_bytes + ((pv + vp) % G::NS) * G::piece + (row - vp * G::v_keys) * 128;
            constexpr int HB = DH == 64 ? 1 : DH / 128;
#pragma unroll 1
            for (int i = 0; i < (DH == 64 ? 4 : HB * 8); ++i)
              *reinterpret_cast<uint4*>(v0 + (DH == 64 ? hh * 64 + i * 16
                                                       : (hh * HB + (i >> 3)) * (G::v_keys * 128) + (i & 7) * 16)) =
                  make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
          }
          if (tid < 4) bad[(nbound + 2) % 3][tid] = 0;
          ++nbound;
          const int j0 = key0 + 64 * hh - len;
          vis[0] = seen_slots(words, tok, a.N, j0);
          vis[1] = seen_slots(words, tok, a.N, j0 + 32);
          if ((vis[0] & bd[2 * hh]) | (vis[1] & bd[2 * hh + 1])) spoilt = true;
        }
        wait(&bar_s[t & 1], (t >> 1) & 1);
        const uint32_t tSt = tS + (t & 1) * TREE_KEYS + lanes;
        if (work) {
          uint32_t s[64];
          tmem_ld32_nowait(tSt + 64 * hh, s);
          tmem_ld32_nowait(tSt + 64 * hh + 32, s + 32);
          tmem_wait_ld();
          if (boundary) {
#pragma unroll
            for (int e = 0; e < 64; ++e)
              if (!((vis[e >> 5] >> (e & 31)) & 1u)) s[e] = 0xff800000u;   // -inf
          }
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int e = 0; e < 64; ++e) m4[e & 3] = fmaxf(m4[e & 3], __uint_as_float(s[e]));
          const float mine = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
          mx_sh[t & 1][hh][row] = mine;
          pair_barrier(pw);   // also: both halves of the scores have left their columns
          const float mx = fmaxf(mine, mx_sh[t & 1][hh ^ 1][row]) * sl2;
          const float nref = mx > ref + TA_RESCALE || ref == -INFINITY ? fmaxf(mx, ref) : ref;
          const float corr = nref == -INFINITY ? 1.f : exp2f(ref - nref);   // first visible slot: 0
          const float off = nref == -INFINITY ? 0.f : nref;
          float ps[4] = {0.f, 0.f, 0.f, 0.f};
          uint32_t pk[32];
#pragma unroll
          for (int e = 0; e < 64; e += 2) {
            const float p0 = ex2_approx(fmaf(__uint_as_float(s[e]), sl2, -off));
            const float p1 = ex2_approx(fmaf(__uint_as_float(s[e + 1]), sl2, -off));
            ps[(e >> 1) & 3] += p0 + p1;
            pk[e >> 1] = pack_bf16x2(p0, p1);
          }
          tmem_st32(tSt + 32 * hh, pk);
          l = l * corr + ((ps[0] + ps[1]) + (ps[2] + ps[3]));
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
        const int slot = 2 * blockIdx.x + (it.first ? 0 : 1);
        float* xrow = whole ? nullptr : a.scratch + (static_cast<size_t>(slot) * min(128, R) + row) * OLD;
#pragma unroll 1
        for (int c0 = hh * (DH / 2); c0 < (hh + 1) * (DH / 2); c0 += 32) {
          uint32_t ov[32];
          tmem_ld32_nowait(tO + lanes + c0, ov);
          tmem_wait_ld();
          if (!mine) continue;
          if (whole) {
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              uint32_t w[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                w[i] = pack_bf16x2(__uint_as_float(ov[e + 2 * i]) * inv, __uint_as_float(ov[e + 2 * i + 1]) * inv);
              *reinterpret_cast<uint4*>(orow + c0 + e) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<uint4*>(xrow + c0 + e) = make_uint4(ov[e], ov[e + 1], ov[e + 2], ov[e + 3]);
          }
        }
        if (mine && hh == 0) {
          if (!whole) {
            *reinterpret_cast<float4*>(xrow + DH) = make_float4(ref, lt, bad_v, 0.f);
          } else if (a.lse) {
            a.lse[(static_cast<size_t>(it.b) * a.Hq + hq) * a.N + tok] =
                ref == -INFINITY ? -INFINITY : (ref + log2f(lt)) * 0.6931471805599453f;
          }
        }
        tc_fence_before();
      }
      it.first = 0;
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
// Joins the segments of units that lie on several CTAs.  `wpr` warps share a row (its segments strided
// over them), 8 / wpr rows per CTA; grid (row groups, row tiles x KV heads, samples).
constexpr int TM_WARPS = 8;

template <int DH>
__global__ void __launch_bounds__(TM_WARPS * 32) k_tree_merge(const __grid_constant__ TreeArgs a, int wpr) {
  constexpr int OLD = DH + 4, VL = DH / 32;   // features per lane
  __shared__ long long sh_T, sh_cum;
  __shared__ float red[TM_WARPS][DH + 4];
  const int g = a.Hq / a.Hkv, R = g * a.N, RT = (R + 127) >> 7, U = a.Hkv * RT;
  const int b = blockIdx.z, u = blockIdx.y, rt = u % RT, hk = u / RT;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rpc = TM_WARPS / wpr;             // rows per CTA
  const int Rv = min(128, R - rt * 128);
  const int row = blockIdx.x * rpc + warp / wpr, sub = warp % wpr;
  if (warp == 0) {
    const long long T = tiles_before(a, U, a.B, nullptr);
    if (lane == 0) sh_T = T;
  } else if (warp == 1) {
    const long long c = tiles_before(a, U, b, nullptr);
    if (lane == 0) sh_cum = c;
  }
  const int nb = sample_tiles(a, b);
  __syncthreads();
  grid_dep_wait();
  if (nb == 0 || blockIdx.x * rpc >= Rv) return;
  const long long T = sh_T, t0 = sh_cum + static_cast<long long>(u) * nb, t1 = t0 + nb;
  // CTA c < n holds tiles [T c / n, T (c + 1) / n), at least one
  const int n = static_cast<int>(min(T, static_cast<long long>(a.ctas)));
  auto holder = [&](long long t) { return static_cast<int>(((t + 1) * n - 1) / T); };
  const int c0 = holder(t0), c1 = holder(t1 - 1);
  if (c0 == c1) return;   // one segment: written by k_tree_attn
  // CTA c0's segment of this unit is its first one only if its range begins with it
  auto part = [&](int c) {
    const int s = 2 * c + (c == c0 && T * c / n != t0 ? 1 : 0);
    return a.scratch + (static_cast<size_t>(s) * min(128, R) + row) * OLD;
  };
  float m = -INFINITY, l = 0.f, x = 0.f, o[VL];
#pragma unroll
  for (int e = 0; e < VL; ++e) o[e] = 0.f;
  auto add = [&](float m2, float l2, float x2, const float* v) {
    const float mn = fmaxf(m, m2);
    if (mn == -INFINITY) return;
    const float w0 = exp2f(m - mn), w1 = exp2f(m2 - mn);
    m = mn;
    l = l * w0 + l2 * w1;
    x += x2;
#pragma unroll
    for (int e = 0; e < VL; ++e) o[e] = o[e] * w0 + v[e] * w1;
  };
  if (row < Rv) {
    constexpr int UN = 4;   // segments in flight
    for (int cb = c0 + sub; cb <= c1; cb += UN * wpr) {
      float v[UN][VL];
      float4 st[UN];
#pragma unroll
      for (int i = 0; i < UN; ++i) {
        const int c = cb + i * wpr;
        st[i] = make_float4(-INFINITY, 0.f, 0.f, 0.f);
        if (c <= c1) {
          const float* p = part(c);
          st[i] = *reinterpret_cast<const float4*>(p + DH);
#pragma unroll
          for (int e = 0; e < VL; e += 2)
            *reinterpret_cast<float2*>(&v[i][e]) = *reinterpret_cast<const float2*>(p + (e / 2) * 64 + 2 * lane);
        }
      }
#pragma unroll
      for (int i = 0; i < UN; ++i)
        if (cb + i * wpr <= c1) add(st[i].x, st[i].y, st[i].z, v[i]);
    }
  }
  if (wpr > 1) {
#pragma unroll
    for (int e = 0; e < VL; e += 2) *reinterpret_cast<float2*>(&red[warp][(e / 2) * 64 + 2 * lane]) = make_float2(o[e], o[e + 1]);
    if (lane == 0) {
      red[warp][DH] = m;
      red[warp][DH + 1] = l;
      red[warp][DH + 2] = x;
    }
    __syncthreads();
    if (sub == 0)
      for (int w = warp + 1; w < warp + wpr; ++w) {
        float v[VL];
#pragma unroll
        for (int e = 0; e < VL; e += 2) *reinterpret_cast<float2*>(&v[e]) = *reinterpret_cast<float2*>(&red[w][(e / 2) * 64 + 2 * lane]);
        add(red[w][DH], red[w][DH + 1], red[w][DH + 2], v);
      }
  }
  if (row >= Rv || sub != 0) return;
  const int rr = rt * 128 + row, tok = rr % a.N, hq = hk * g + rr / a.N;
  const float inv = (l == 0.f ? 0.f : 1.f / l) + x;
  __nv_bfloat16* orow = a.o + (static_cast<size_t>(b) * a.N + tok) * a.Hq * DH + static_cast<size_t>(hq) * DH;
#pragma unroll
  for (int e = 0; e < VL; e += 2)
    *reinterpret_cast<uint32_t*>(orow + (e / 2) * 64 + 2 * lane) = pack_bf16x2(o[e] * inv, o[e + 1] * inv);
  if (a.lse && lane == 0)
    a.lse[(static_cast<size_t>(b) * a.Hq + hq) * a.N + tok] =
        m == -INFINITY ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
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
  k_tree_attn<DH><<<a.ctas, TA_THREADS, G::smem, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.S_max <= TREE_KEYS) return e;   // a unit of one tile is never split
  // segments per unit if every sample is as long as can be
  const int64_t units = static_cast<int64_t>(planes) * RT;
  const int per = static_cast<int>(a.ctas / std::min<int64_t>(units, a.ctas)) + 1;
  const int wpr = per > 32 ? 8 : per > 16 ? 4 : per > 8 ? 2 : 1;
  const int rpc = TM_WARPS / wpr;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((std::min(R, 128) + rpc - 1) / rpc, a.Hkv * RT, a.B);
  cfg.blockDim = dim3(TM_WARPS * 32);
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_tree_merge<DH>, a, wpr);
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
  a.ctas = std::min(nsm, TA_CTAS);
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

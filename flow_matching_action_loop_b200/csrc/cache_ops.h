// Ops on one layer's static KV cache [B][Hkv][S_max][dh] with drafted tokens behind the committed
// ones: launch arguments and launchers (tree_attention.cu, cache_moves.cu; entry points cache_ops.cu).
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

namespace fr {

// Device address of the ops' status word on the current device, looked up once per device (ops.cu).
cudaError_t ops_status_word(unsigned** out, int* dev_out);

namespace tc {

// where-codes of the samples that the cache ops refuse (fr_ops_sync_status)
constexpr uint32_t CACHE_BAD_LEN = 0xC001u, CACHE_BAD_PATH = 0xC002u;

// Extents of the buffers that the cache ops store into, in elements of each (rows: 16-byte words of K or of V), and
// the where-codes of their checks.  Checked builds verify every store against them; the product build carries them
// unused.
struct CacheExtents {
  uint64_t o, lse, scratch, acc, pos, src, lens, rows;
};
constexpr uint32_t CHK_TREE_O = 0x9020u, CHK_TREE_LSE = 0x9021u, CHK_TREE_SCRATCH = 0x9022u, CHK_WEIGHTS_ACC = 0x9030u,
                   CHK_COMMIT_ROWS = 0x9040u, CHK_COMMIT_SLOTS = 0x9041u, CHK_COMMIT_LENS = 0x9042u,
                   CHK_EVICT_ROWS = 0x9050u, CHK_EVICT_SLOTS = 0x9051u, CHK_EVICT_SRC = 0x9052u, CHK_EVICT_LENS = 0x9053u;

struct TreeArgs {
  const __nv_bfloat16* q;      // [B][Hq][N][dh]
  const __nv_bfloat16* k;      // [B][Hkv][S_max][dh]
  const __nv_bfloat16* v;
  const int32_t* lens;         // [B] committed tokens, < 0: padded sample
  const uint32_t* mask;        // [B][N][W] words, or nullptr: a sequence
  const uint32_t* use;         // weights: [B][W] words, or nullptr: all tokens count
  __nv_bfloat16* o;            // [B][N][Hq*dh]
  float* lse;                  // [B][Hq][N] (weights: input), or nullptr
  float* acc;                  // weights: [B][Hkv][S_max]
  float* scratch;
  unsigned* status;
  int B, Hq, Hkv, N, W, S_max, dh;
  float scale;                 // 1/sqrt(dh)
  uint64_t wait_ns;            // bound of a wait (fr_ops_set_wait_limit)
  int rtg, groups;             // CTAs per group (row tiles of a unit), groups that share the tiles
  int whole_extra;             // tiles that keeping a unit whole may cost a group
  int cluster;                 // attention: CTAs of a unit's cluster, 1: none
  CacheExtents ext;
  CUtensorMap tm_q, tm_k, tm_v;   // written by the launchers
};

struct MoveArgs {
  uint8_t* k;                  // [B][Hkv][S_max][row_bytes]
  uint8_t* v;
  float* acc;                  // commit: moved in place, or nullptr
  int32_t* pos;
  const float* acc_in;         // evict: [B][Hkv][S_max]
  const int32_t* pos_in;
  float* acc_out;
  int32_t* pos_out;
  const int32_t* lens;
  const int32_t* path;         // commit: [B][N]
  const int32_t* npath;        // commit: [B]
  int32_t* lens_out;
  int32_t* src;                // evict: [B][Hkv][keep]
  unsigned* status;
  int B, Hkv, N, S_max, row_bytes, keep, recent;
  CacheExtents ext;
};

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();   // tc_kernels.cu
// Attributes of the cache ops' kernels on the current device; *regs becomes the attention kernel's registers per
// thread where these are not what its register moves need.
cudaError_t cache_ops_init(int* regs);
size_t tree_scratch_bytes(int B, int Hq, int Hkv, int N, int S_max, int dh);
cudaError_t launch_tree_attention(const TreeArgs& a, cudaStream_t s);
cudaError_t launch_attention_weights(const TreeArgs& a, cudaStream_t s);
cudaError_t launch_cache_commit(const MoveArgs& a, cudaStream_t s);
cudaError_t launch_cache_evict(const MoveArgs& a, cudaStream_t s);
cudaError_t weights_init();
cudaError_t cache_moves_init();

}  // namespace tc
}  // namespace fr

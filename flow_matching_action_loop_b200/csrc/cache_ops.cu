// Entry points of the cache ops: tree attention, accumulated attention weights, commit of accepted
// drafted tokens, eviction.  Argument checks here, kernels in tree_attention.cu and cache_moves.cu.
#include <atomic>
#include <cmath>
#include <cstring>
#include <mutex>

#include <cuda.h>

#include "cache_ops.h"
#include "internal.h"
#include "tc_kernels.h"

namespace fr {
namespace {

// The driver's query, found once through the runtime (no link-time dependency): eight pointers take 0.5 us of a
// call's 4.7, with the runtime's own query 0.75.
using PointerQuery = CUresult(CUDAAPI*)(unsigned, CUpointer_attribute*, void**, CUdeviceptr);
PointerQuery pointer_query() {
  static const PointerQuery fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q{};
    const bool found = cudaGetDriverEntryPoint("cuPointerGetAttributes", &p, cudaEnableDefault, &q) == cudaSuccess &&
                       q == cudaDriverEntryPointSuccess;
    return found ? reinterpret_cast<PointerQuery>(p) : nullptr;
  }();
  return fn;
}

// Memory of the current device (or managed): what the kernels may dereference.  Anything else would
// fault in the kernel, on a GPU that other work shares.
int check_pointers(const char* op, const void* const* ptrs, int n) {
  int dev = 0;
  FR_CUDA(cudaGetDevice(&dev));
  const PointerQuery query = pointer_query();
  if (!query) {
    set_error("%s: the driver has no cuPointerGetAttributes", op);
    return FR_ERR_CUDA;
  }
  for (int i = 0; i < n; ++i) {
    if (!ptrs[i]) continue;
    unsigned type = 0, managed = 0;   // 0 for memory that the driver does not know
    int owner = -1;
    CUpointer_attribute which[3] = {CU_POINTER_ATTRIBUTE_MEMORY_TYPE, CU_POINTER_ATTRIBUTE_IS_MANAGED,
                                    CU_POINTER_ATTRIBUTE_DEVICE_ORDINAL};
    void* out[3] = {&type, &managed, &owner};
    const CUresult r = query(3, which, out, reinterpret_cast<CUdeviceptr>(ptrs[i]));
    if (r == CUDA_SUCCESS && (managed || (type == CU_MEMORYTYPE_DEVICE && owner == dev))) continue;
    set_error("%s: pointer %d is not memory of the current device (cuda:%d)", op, i, dev);
    return FR_ERR_ARG;
  }
  return FR_OK;
}

// Before a launch: the ops' status word, and the attributes of the cache ops' kernels, set by the first cache op on
// each device (no other op needs them, or fails with them).
constexpr int MAX_DEVICES = 64;
std::once_flag g_init_once[MAX_DEVICES];
cudaError_t g_init_err[MAX_DEVICES];
int g_tree_regs[MAX_DEVICES];   // not 0: refused, see cache_ops_init

cudaError_t cache_op_begin(unsigned** status, int* tree_regs = nullptr) {
  int dev = 0;
  const cudaError_t e = ops_status_word(status, &dev);
  if (e != cudaSuccess) return e;
  if (dev >= MAX_DEVICES) return cudaErrorInvalidDevice;
  std::call_once(g_init_once[dev], [dev] { g_init_err[dev] = tc::cache_ops_init(&g_tree_regs[dev]); });
  if (tree_regs) *tree_regs = g_tree_regs[dev];
  return g_init_err[dev];
}

std::atomic<uint64_t> g_wait_ns{tc::WAIT_LIMIT_NS};

// Extents of a call's buffers, or smaller ones declared for a test of the checks (fr_debug_limit_op_extent).
const char* const EXTENT_NAMES[] = {"o", "lse", "scratch", "acc", "pos", "src", "lens", "rows"};
std::atomic<uint64_t> g_extent_limit[8];

tc::CacheExtents extents(uint64_t o, uint64_t lse, uint64_t scratch, uint64_t slots, uint64_t src, uint64_t lens,
                         uint64_t rows) {
  uint64_t e[8] = {o, lse, scratch, slots, slots, src, lens, rows};
  for (int i = 0; i < 8; ++i) {
    const uint64_t limit = g_extent_limit[i].load(std::memory_order_relaxed);
    if (limit && limit < e[i]) e[i] = limit;
  }
  return {e[0], e[1], e[2], e[3], e[4], e[5], e[6], e[7]};
}

bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

int check_tree_sizes(const char* op, int B, int Hq, int Hkv, int N, int S_max, int dh) {
  if (B < 1 || Hq < 1 || Hkv < 1 || N < 1 || S_max < 1 || dh < 1) {
    set_error("%s: sizes must be positive", op);
    return FR_ERR_ARG;
  }
  if ((dh != 64 && dh != 128 && dh != 256) || Hq % Hkv != 0 || N > FR_TREE_MAX_NODES ||
      S_max > FR_CACHE_MAX_SLOTS || B > 4096 || Hq > 1024) {
    set_error("%s: needs dh in {64,128,256}, Hq %% Hkv == 0, N <= %d, S_max <= %d, B <= 4096, Hq <= 1024", op,
              FR_TREE_MAX_NODES, FR_CACHE_MAX_SLOTS);
    return FR_ERR_UNSUPPORTED;
  }
  // key tiles of all samples, KV heads and (at most) row tiles: the kernels count them in an int
  const int64_t line = static_cast<int64_t>(B) * Hkv * ((static_cast<int64_t>(Hq / Hkv) * N + 127) / 128) *
                       ((static_cast<int64_t>(S_max) + 127) / 128);
  if (line > INT32_MAX) {
    set_error("%s: a cache this long is not served at this batch and number of heads", op);
    return FR_ERR_UNSUPPORTED;
  }
  if (N > S_max) {
    set_error("%s: %d drafted tokens do not fit a cache of %d slots", op, N, S_max);
    return FR_ERR_SHAPE;
  }
  return FR_OK;
}

int check_move_sizes(const char* op, int B, int Hkv, int S_max, int dh, int dtype) {
  if (B < 1 || Hkv < 1 || S_max < 1 || dh < 1 || (dtype != FR_DTYPE_BF16 && dtype != FR_DTYPE_F32)) {
    set_error("%s: sizes must be positive, dtype FR_DTYPE_BF16 or FR_DTYPE_F32", op);
    return FR_ERR_ARG;
  }
  if (dh > 512 || dh * (dtype == FR_DTYPE_F32 ? 4 : 2) % 16 != 0 || B > 4096 || Hkv > 1024 ||
      S_max > FR_CACHE_MAX_SLOTS) {
    set_error("%s: needs dh <= 512 with rows of a multiple of 16 bytes, B <= 4096, Hkv <= 1024, S_max <= %d", op,
              FR_CACHE_MAX_SLOTS);
    return FR_ERR_UNSUPPORTED;
  }
  return FR_OK;
}

}  // namespace
}  // namespace fr

using namespace fr;

extern "C" {

int fr_ops_set_wait_limit(uint64_t limit_ns) {
  if (limit_ns > 10000000000ull) {
    set_error("fr_ops_set_wait_limit: limit above 10 s");
    return FR_ERR_ARG;
  }
  g_wait_ns = limit_ns ? limit_ns : tc::WAIT_LIMIT_NS;
  return FR_OK;
}

int fr_debug_limit_op_extent(const char* buffer, uint64_t elems) {
  if (!buffer) {
    set_error("fr_debug_limit_op_extent: NULL argument");
    return FR_ERR_ARG;
  }
  if (!fr_device_checks()) {
    set_error("fr_debug_limit_op_extent: this library was built without device bounds checks");
    return FR_ERR_UNSUPPORTED;
  }
  for (int i = 0; i < 8; ++i)
    if (!std::strcmp(buffer, EXTENT_NAMES[i])) {
      g_extent_limit[i] = elems;
      return FR_OK;
    }
  set_error("fr_debug_limit_op_extent: no buffer \"%s\"", buffer);
  return FR_ERR_ARG;
}

int fr_tree_mask(const int32_t* parents, int n, uint32_t* mask) {
  if (!parents || !mask) {
    set_error("fr_tree_mask: NULL argument");
    return FR_ERR_ARG;
  }
  if (n < 1 || n > FR_TREE_MAX_NODES) {
    set_error("fr_tree_mask: n must be in [1, %d]", FR_TREE_MAX_NODES);
    return FR_ERR_UNSUPPORTED;
  }
  for (int i = 0; i < n; ++i)
    if (parents[i] < -1 || parents[i] >= i) {
      set_error("fr_tree_mask: parent %d of token %d is not in [-1, %d]", parents[i], i, i - 1);
      return FR_ERR_ARG;
    }
  const int W = (n + 31) / 32;
  for (int i = 0; i < n; ++i) {
    for (int w = 0; w < W; ++w) mask[i * W + w] = parents[i] >= 0 ? mask[parents[i] * W + w] : 0u;
    mask[i * W + i / 32] |= 1u << (i % 32);
  }
  return FR_OK;
}

size_t fr_attention_tree_scratch_bytes(int B, int Hq, int Hkv, int N, int S_max, int dh) {
  if (check_tree_sizes("fr_attention_tree_scratch_bytes", B, Hq, Hkv, N, S_max, dh)) return 0;
  return tc::tree_scratch_bytes(B, Hq, Hkv, N, S_max, dh);
}

int fr_attention_tree(const void* q, const void* k, const void* v, const int32_t* lens, const uint32_t* mask, void* o,
                      float* lse, int B, int Hq, int Hkv, int N, int S_max, int dh, void* scratch,
                      size_t scratch_bytes, fr_stream_t stream) {
  const char* op = "fr_attention_tree";
  if (!q || !k || !v || !lens || !o || misaligned(q, 16) || misaligned(k, 16) || misaligned(v, 16) ||
      misaligned(o, 32) || misaligned(scratch, 16) || misaligned(lens, 4) || misaligned(mask, 4) ||
      misaligned(lse, 4)) {
    set_error("%s: NULL or misaligned tensor", op);
    return FR_ERR_ARG;
  }
  int rc = check_tree_sizes(op, B, Hq, Hkv, N, S_max, dh);
  if (rc) return rc;
  const size_t need = tc::tree_scratch_bytes(B, Hq, Hkv, N, S_max, dh);
  if (need > 0 && (!scratch || scratch_bytes < need)) {
    set_error("%s: scratch of %zu bytes needed, %zu given", op, need, scratch ? scratch_bytes : size_t(0));
    return FR_ERR_SHAPE;
  }
  const void* ptrs[] = {q, k, v, lens, mask, o, lse, need > 0 ? scratch : nullptr};
  if ((rc = check_pointers(op, ptrs, 8))) return rc;
  tc::TreeArgs a{};
  int regs = 0;
  FR_CUDA(cache_op_begin(&a.status, &regs));
  if (regs) {
    set_error("%s: this build's kernel has %d registers a thread, which its register moves do not add up to", op, regs);
    return FR_ERR_UNSUPPORTED;
  }
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.lens = lens;
  a.mask = mask;
  a.o = static_cast<__nv_bfloat16*>(o);
  a.lse = lse;
  a.scratch = static_cast<float*>(scratch);
  a.B = B, a.Hq = Hq, a.Hkv = Hkv, a.N = N, a.W = (N + 31) / 32, a.S_max = S_max, a.dh = dh;
  a.scale = 1.0f / std::sqrt(static_cast<float>(dh));
  a.wait_ns = g_wait_ns.load(std::memory_order_relaxed);
  const uint64_t rows = static_cast<uint64_t>(B) * Hq * N;
  a.ext = extents(rows * dh, rows, need / 4, 0, 0, 0, 0);
  FR_CUDA(tc::launch_tree_attention(a, reinterpret_cast<cudaStream_t>(stream)));
  return FR_OK;
}

int fr_attention_weights(const void* q, const void* k, const float* lse, const int32_t* lens, const uint32_t* mask,
                         const uint32_t* use, float* acc, int B, int Hq, int Hkv, int N, int S_max, int dh,
                         fr_stream_t stream) {
  const char* op = "fr_attention_weights";
  if (!q || !k || !lse || !lens || !acc || misaligned(q, 16) || misaligned(k, 16) || misaligned(lse, 4) ||
      misaligned(lens, 4) || misaligned(mask, 4) || misaligned(use, 4) || misaligned(acc, 4)) {
    set_error("%s: NULL or misaligned tensor", op);
    return FR_ERR_ARG;
  }
  int rc = check_tree_sizes(op, B, Hq, Hkv, N, S_max, dh);
  if (rc) return rc;
  const void* ptrs[] = {q, k, lse, lens, mask, use, acc};
  if ((rc = check_pointers(op, ptrs, 7))) return rc;
  tc::TreeArgs a{};
  FR_CUDA(cache_op_begin(&a.status));
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.lens = lens;
  a.mask = mask;
  a.use = use;
  a.lse = const_cast<float*>(lse);
  a.acc = acc;
  a.B = B, a.Hq = Hq, a.Hkv = Hkv, a.N = N, a.W = (N + 31) / 32, a.S_max = S_max, a.dh = dh;
  a.scale = 1.0f / std::sqrt(static_cast<float>(dh));
  a.wait_ns = g_wait_ns.load(std::memory_order_relaxed);
  a.ext = extents(0, 0, 0, static_cast<uint64_t>(B) * Hkv * S_max, 0, 0, 0);
  FR_CUDA(tc::launch_attention_weights(a, reinterpret_cast<cudaStream_t>(stream)));
  return FR_OK;
}

int fr_cache_commit(void* k, void* v, float* acc, int32_t* pos, const int32_t* lens, const int32_t* path,
                    const int32_t* npath, int32_t* lens_out, int B, int Hkv, int N, int S_max, int dh, int dtype,
                    fr_stream_t stream) {
  const char* op = "fr_cache_commit";
  if (!k || !v || !lens || !path || !npath || !lens_out || lens_out == lens || misaligned(k, 16) ||
      misaligned(v, 16) || misaligned(acc, 4) || misaligned(pos, 4) || misaligned(lens, 4) || misaligned(path, 4) ||
      misaligned(npath, 4) || misaligned(lens_out, 4)) {
    set_error("%s: NULL or misaligned tensor, or lens_out is lens", op);
    return FR_ERR_ARG;
  }
  int rc = check_move_sizes(op, B, Hkv, S_max, dh, dtype);
  if (rc) return rc;
  if (N < 1) {
    set_error("%s: sizes must be positive", op);
    return FR_ERR_ARG;
  }
  if (N > FR_TREE_MAX_NODES) {
    set_error("%s: N must be at most %d", op, FR_TREE_MAX_NODES);
    return FR_ERR_UNSUPPORTED;
  }
  if (N > S_max) {
    set_error("%s: %d drafted tokens do not fit a cache of %d slots", op, N, S_max);
    return FR_ERR_SHAPE;
  }
  const void* ptrs[] = {k, v, acc, pos, lens, path, npath, lens_out};
  if ((rc = check_pointers(op, ptrs, 8))) return rc;
  tc::MoveArgs a{};
  FR_CUDA(cache_op_begin(&a.status));
  a.k = static_cast<uint8_t*>(k);
  a.v = static_cast<uint8_t*>(v);
  a.acc = acc;
  a.pos = pos;
  a.lens = lens;
  a.path = path;
  a.npath = npath;
  a.lens_out = lens_out;
  a.B = B, a.Hkv = Hkv, a.N = N, a.S_max = S_max, a.row_bytes = dh * (dtype == FR_DTYPE_F32 ? 4 : 2);
  const uint64_t slots = static_cast<uint64_t>(B) * Hkv * S_max;
  a.ext = extents(0, 0, 0, slots, 0, B, slots * a.row_bytes / 16);
  FR_CUDA(tc::launch_cache_commit(a, reinterpret_cast<cudaStream_t>(stream)));
  return FR_OK;
}

int fr_cache_evict(void* k, void* v, const float* acc, const int32_t* pos, const int32_t* lens, float* acc_out,
                   int32_t* pos_out, int32_t* lens_out, int32_t* src, int B, int Hkv, int S_max, int dh, int dtype,
                   int keep, int recent, fr_stream_t stream) {
  const char* op = "fr_cache_evict";
  if (!k || !v || !acc || !pos || !lens || !acc_out || !pos_out || !lens_out || !src || acc_out == acc ||
      pos_out == pos || lens_out == lens || misaligned(k, 16) || misaligned(v, 16) || misaligned(acc, 4) ||
      misaligned(pos, 4) || misaligned(lens, 4) || misaligned(acc_out, 4) || misaligned(pos_out, 4) ||
      misaligned(lens_out, 4) || misaligned(src, 4)) {
    set_error("%s: NULL or misaligned tensor, or an output is its input", op);
    return FR_ERR_ARG;
  }
  int rc = check_move_sizes(op, B, Hkv, S_max, dh, dtype);
  if (rc) return rc;
  if (keep < 1 || recent < 0) {
    set_error("%s: keep must be positive, recent not negative", op);
    return FR_ERR_ARG;
  }
  if (S_max > FR_EVICT_MAX_SLOTS) {
    set_error("%s: S_max must be at most %d", op, FR_EVICT_MAX_SLOTS);
    return FR_ERR_UNSUPPORTED;
  }
  if (keep > S_max || recent > keep) {
    set_error("%s: needs recent <= keep <= S_max", op);
    return FR_ERR_SHAPE;
  }
  const void* ptrs[] = {k, v, acc, pos, lens, acc_out, pos_out, lens_out, src};
  if ((rc = check_pointers(op, ptrs, 9))) return rc;
  tc::MoveArgs a{};
  FR_CUDA(cache_op_begin(&a.status));
  a.k = static_cast<uint8_t*>(k);
  a.v = static_cast<uint8_t*>(v);
  a.acc_in = acc;
  a.pos_in = pos;
  a.acc_out = acc_out;
  a.pos_out = pos_out;
  a.lens = lens;
  a.lens_out = lens_out;
  a.src = src;
  a.B = B, a.Hkv = Hkv, a.S_max = S_max, a.row_bytes = dh * (dtype == FR_DTYPE_F32 ? 4 : 2);
  a.keep = keep, a.recent = recent;
  const uint64_t slots = static_cast<uint64_t>(B) * Hkv * S_max;
  a.ext = extents(0, 0, 0, slots, static_cast<uint64_t>(B) * Hkv * keep, B, slots * a.row_bytes / 16);
  FR_CUDA(tc::launch_cache_evict(a, reinterpret_cast<cudaStream_t>(stream)));
  return FR_OK;
}

}  // extern "C"

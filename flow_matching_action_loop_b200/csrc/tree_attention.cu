// Attention of drafted tokens over a static KV cache, and the weights its slots received.
#include <algorithm>

#include "cache_ops.h"
#include "fr.h"
#include "tc_device.h"

namespace fr {
namespace tc {
namespace {

__device__ __forceinline__ void report_sample(unsigned* status, uint32_t where, int sample) {
  if (!(atomicOr(status, ST_BOUNDS_BIT) & ST_BOUNDS_BIT)) {   // the first refused sample reports
    atomicExch(status + 1, where);
    atomicExch(status + 2, static_cast<unsigned>(sample));
  }
}

// Whether token n sees slot s of sample b (len committed tokens).
__device__ __forceinline__ bool sees(const TreeArgs& a, int b, int n, int len, int s) {
  if (s < len) return true;
  const int j = s - len;
  if (j >= a.N) return false;
  if (!a.mask) return j <= n;
  return (a.mask[(static_cast<size_t>(b) * a.N + n) * a.W + (j >> 5)] >> (j & 31)) & 1u;
}

__device__ __forceinline__ float dot_row(const float* q, const __nv_bfloat16* k, int dh) {
  float s = 0.f;
  for (int d = 0; d < dh; ++d) s = fmaf(q[d], __bfloat162float(k[d]), s);
  return s;
}

// One CTA per row (token, head, sample), 128 keys at a time.
__global__ void __launch_bounds__(128) k_tree_rows(const __grid_constant__ TreeArgs a) {
  __shared__ float q[256], p[128], red[4];
  __shared__ bool vis[128];
  __shared__ int poison;   // a drafted value row that this token sees is not finite
  const int n = blockIdx.x, hq = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  const int len = a.lens[b];
  if (len < 0 || len > a.S_max - a.N) {
    if (len > 0 && n == 0 && hq == 0 && tid == 0) report_sample(a.status, CACHE_BAD_LEN, b);
    return;
  }
  const size_t row = (static_cast<size_t>(b) * a.Hq + hq) * a.N + n;
  const size_t kv0 = (static_cast<size_t>(b) * a.Hkv + hq / (a.Hq / a.Hkv)) * a.S_max * a.dh;
  for (int d = tid; d < a.dh; d += 128) q[d] = __bfloat162float(a.q[row * a.dh + d]) * a.scale;
  if (tid == 0) poison = 0;
  float m = -INFINITY, l = 0.f, o[2] = {0.f, 0.f};
  const int S = len + a.N;
  for (int s0 = 0; s0 < S; s0 += 128) {
    __syncthreads();
    const bool v = s0 + tid < S && sees(a, b, n, len, s0 + tid);
    const float sc = v ? dot_row(q, a.k + kv0 + static_cast<size_t>(s0 + tid) * a.dh, a.dh) : -INFINITY;
    float mx = sc;
    for (int w = 16; w; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
    if ((tid & 31) == 0) red[tid >> 5] = mx;
    __syncthreads();
    const float mn = fmaxf(fmaxf(m, fmaxf(red[0], red[1])), fmaxf(red[2], red[3]));
    const float ref = mn == -INFINITY ? 0.f : mn;
    vis[tid] = v;
    p[tid] = v ? expf(sc - ref) : 0.f;
    const float corr = expf(m - ref);
    __syncthreads();
    l *= corr;
    o[0] *= corr;
    o[1] *= corr;
    for (int j = 0; j < min(128, S - s0); ++j) {
      if (!vis[j]) continue;
      l += p[j];
      for (int e = 0; e < 2; ++e)
        if (tid + 128 * e < a.dh) {
          const float v = __bfloat162float(a.v[kv0 + static_cast<size_t>(s0 + j) * a.dh + tid + 128 * e]);
          if (s0 + j >= len && !isfinite(v)) poison = 1;
          o[e] = fmaf(p[j], v, o[e]);
        }
    }
    m = mn;
  }
  __syncthreads();
  const float inv = poison ? NAN : l == 0.f ? 0.f : 1.f / l;
  for (int e = 0; e < 2; ++e)
    if (tid + 128 * e < a.dh)
      a.o[(static_cast<size_t>(b) * a.N + n) * a.Hq * a.dh + hq * a.dh + tid + 128 * e] =
          __float2bfloat16_rn(o[e] * inv);
  if (a.lse && tid == 0) a.lse[row] = m == -INFINITY ? m : m + logf(l);
}

// One thread per slot.
__global__ void __launch_bounds__(128) k_weights_rows(const __grid_constant__ TreeArgs a) {
  __shared__ float q[256];
  const int s = blockIdx.x * 128 + threadIdx.x, hk = blockIdx.y, b = blockIdx.z;
  const int len = a.lens[b];
  if (len < 0 || len > a.S_max - a.N) {
    if (len > 0 && s == 0 && hk == 0) report_sample(a.status, CACHE_BAD_LEN, b);
    return;
  }
  const int g = a.Hq / a.Hkv;
  const size_t slot = (static_cast<size_t>(b) * a.Hkv + hk) * a.S_max + s;
  float w = 0.f;
  for (int r = 0; r < g * a.N; ++r) {
    const size_t row = (static_cast<size_t>(b) * a.Hq + hk * g) * a.N + r;
    const int n = r % a.N;
    __syncthreads();
    for (int d = threadIdx.x; d < a.dh; d += 128) q[d] = __bfloat162float(a.q[row * a.dh + d]) * a.scale;
    __syncthreads();
    const float lse = a.lse[row];
    const bool counts = !a.use || ((a.use[static_cast<size_t>(b) * a.W + (n >> 5)] >> (n & 31)) & 1u);
    if (counts && lse != -INFINITY && s < len + a.N && sees(a, b, n, len, s))
      w += expf(dot_row(q, a.k + slot * a.dh, a.dh) - lse);
  }
  if (s < len + a.N) a.acc[slot] = s < len ? a.acc[slot] + w : w;
}

}  // namespace

size_t tree_scratch_bytes(int, int, int, int, int, int) { return 0; }

cudaError_t launch_tree_attention(const TreeArgs& a, cudaStream_t s) {
  k_tree_rows<<<dim3(a.N, a.Hq, a.B), 128, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_attention_weights(const TreeArgs& a, cudaStream_t s) {
  k_weights_rows<<<dim3((a.S_max + 127) / 128, a.Hkv, a.B), 128, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t cache_ops_init() { return cache_moves_init(); }

}  // namespace tc
}  // namespace fr

// The attention weight that each slot of a static KV cache received.
#include "tree_device.h"

namespace fr {
namespace tc {
namespace {

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

cudaError_t launch_attention_weights(const TreeArgs& a, cudaStream_t s) {
  k_weights_rows<<<dim3((a.S_max + 127) / 128, a.Hkv, a.B), 128, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace tc
}  // namespace fr

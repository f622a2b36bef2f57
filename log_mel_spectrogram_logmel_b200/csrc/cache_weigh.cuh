// Token cache: the attention weight that each cached key received.
#pragma once
#include "cache_common.cuh"

namespace logmel {
namespace cache {

struct WeighArgs {
  CacheView c;
  Batch b;
  Rows q;
  const float* lse;    // [rows, n_q]
  float* out;          // laid out as c.mass
  int n_q, n_kv, group;
  int causal, window;
  float scale, decay;
};

// One warp per cached key, in turn over the stream's new rows and the key
// head's query heads; the lanes hold the head's dimensions.
template <typename T, int D>
__global__ void __launch_bounds__(128) weigh_simple_kernel(const __grid_constant__ WeighArgs a) {
  constexpr int P = D / 64;
  const int lane = threadIdx.x & 31, s = blockIdx.z, hk = blockIdx.y;
  const int n = a.b.count(s);
  if (n == 0) return;
  const int len = a.c.length(s, threadIdx.x == 0), size = 1 << a.c.page_shift;
  for (int j = blockIdx.x * 4 + (threadIdx.x >> 5); j < len; j += gridDim.x * 4) {
    const int p = a.c.page(s, j >> a.c.page_shift), x = j & (size - 1);
    if (p < 0) {
      a.c.flag();
      continue;
    }
    float2 k[P];
    const T* kp = (const T*)a.c.k + p * a.c.k_page + hk * a.c.k_head + x * a.c.k_slot;
#pragma unroll
    for (int i = 0; i < P; ++i) k[i] = Half2<T>::to_float(*(const uint32_t*)(kp + 64 * i + 2 * lane));
    float sum = 0.f;
    for (int i = 0; i < n; ++i) {
      const int2 r = seen(len, n, i, a.causal, a.window);
      if (j < r.x || j >= r.y) continue;
      const int64_t t = a.b.begin(s) + i;
      for (int g = 0; g < a.group; ++g) {
        const int h = hk * a.group + g;
        const T* q = (const T*)a.q.data + t * a.q.row + (int64_t)h * a.q.head;
        float dot = 0.f;
#pragma unroll
        for (int e = 0; e < P; ++e) {
          const float2 y = Half2<T>::to_float(*(const uint32_t*)(q + 64 * e + 2 * lane));
          dot += k[e].x * y.x + k[e].y * y.y;
        }
        for (int d = 16; d; d >>= 1) dot += __shfl_xor_sync(~0u, dot, d);
        sum += expf(dot * a.scale - a.lse[t * a.n_q + h]);
      }
    }
    if (lane == 0) {
      const int64_t at = ((int64_t)p * a.n_kv + hk) * size + x;
      a.out[at] = a.decay * a.c.mass[at] + sum;
    }
  }
}

}  // namespace cache
}  // namespace logmel

// Token cache: attention of new rows over the cached slots.
#pragma once
#include "cache_common.cuh"

namespace logmel {
namespace cache {

struct AttendArgs {
  CacheView c;
  Batch b;
  Rows q, out;
  float* lse;          // [rows, n_q] or null
  int n_q, n_kv, group;
  int causal, window;
  float scale;
};

// One warp per new row and query head: the lanes hold the head's dimensions,
// keys are taken one by one with a running maximum and sum.
template <typename T, int D>
__global__ void __launch_bounds__(128) attend_simple_kernel(const __grid_constant__ AttendArgs a) {
  constexpr int P = D / 64;   // 2-element pieces per lane
  const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (w >= (int64_t)a.b.rows * a.n_q) return;
  const int t = (int)(w / a.n_q), h = (int)(w - (int64_t)t * a.n_q), hk = h / a.group;
  const int s = a.b.stream_of(t), n = a.b.count(s);
  const int len = a.c.length(s, lane == 0);
  const int2 r = seen(len, n, t - a.b.begin(s), a.causal, a.window);
  float2 q[P], o[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    q[i] = Half2<T>::to_float(
        *(const uint32_t*)((const T*)a.q.data + (int64_t)t * a.q.row + (int64_t)h * a.q.head + 64 * i + 2 * lane));
    o[i] = make_float2(0.f, 0.f);
  }
  float m = -INFINITY, l = 0.f;
  for (int j = r.x; j < r.y; ++j) {
    const int p = a.c.page(s, j >> a.c.page_shift), x = j & ((1 << a.c.page_shift) - 1);
    if (p < 0) {
      a.c.flag();
      continue;
    }
    const T* k = (const T*)a.c.k + p * a.c.k_page + hk * a.c.k_head + x * a.c.k_slot;
    const T* v = (const T*)a.c.v + p * a.c.v_page + hk * a.c.v_head + x * a.c.v_slot;
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const float2 y = Half2<T>::to_float(*(const uint32_t*)(k + 64 * i + 2 * lane));
      dot += q[i].x * y.x + q[i].y * y.y;
    }
    for (int d = 16; d; d >>= 1) dot += __shfl_xor_sync(~0u, dot, d);
    dot *= a.scale;
    const float top = fmaxf(m, dot);
    const float c = top == -INFINITY ? 1.f : expf(m - top), e = top == -INFINITY ? 0.f : expf(dot - top);
    l = l * c + e;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const float2 y = Half2<T>::to_float(*(const uint32_t*)(v + 64 * i + 2 * lane));
      o[i].x = o[i].x * c + e * y.x;
      o[i].y = o[i].y * c + e * y.y;
    }
    m = top;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int i = 0; i < P; ++i)
    *(uint32_t*)((T*)a.out.data + (int64_t)t * a.out.row + (int64_t)h * a.out.head + 64 * i + 2 * lane) =
        Half2<T>::from_float(o[i].x * inv, o[i].y * inv);
  if (a.lse && lane == 0) a.lse[(int64_t)t * a.n_q + h] = l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace cache
}  // namespace logmel

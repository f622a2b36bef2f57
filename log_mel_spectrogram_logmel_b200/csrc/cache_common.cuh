// Token cache, device side: what its kernels share.
//
// A launch covers a run of streams.  Its new rows are described by a Batch
// (offsets in the launch parameters, or one count for all streams), its
// pages by a CacheView.  Lengths and page ids are device data that the host
// never sees, so every kernel clamps and checks them before it follows them.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "logmel.h"

namespace logmel {
namespace cache {

// Streams of one launch: ragged batches carry their offsets in the launch
// parameters (2 KB of the 4 KB that every driver takes), so that a call needs
// no copy and can be captured.  Larger batches take several launches.
constexpr int MAX_RAGGED = 512;
constexpr int MAX_UNIFORM = 4096;   // every CTA of the split kernels scans the lengths of its launch

struct Batch {
  int streams;
  int rows;                    // new rows of these streams
  int uniform;                 // > 0: every stream has this many; 0: off[]
  int off[MAX_RAGGED + 1];     // first row of each stream, relative to the launch's first row

  __device__ int begin(int s) const { return uniform ? s * uniform : off[s]; }
  __device__ int count(int s) const { return uniform ? uniform : off[s + 1] - off[s]; }
  // the stream that holds row t
  __device__ int stream_of(int t) const {
    if (uniform) return t / uniform;
    int lo = 0, hi = streams - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (off[mid] <= t) lo = mid;
      else hi = mid - 1;
    }
    return lo;
  }
};

struct CacheView {
  char* k;
  char* v;
  const int* table;
  int* lens;
  float* mass;
  int64_t k_page, k_head, k_slot;   // strides in elements
  int64_t v_page, v_head, v_slot;
  int n_pages;
  int width;                        // table entries per stream
  int capacity;                     // slots a table row can name
  int page_shift;
  int* status;

  // the larger code stays: a wait that ran out must not be hidden, the plan's counters depend on it
  __device__ void flag() const { atomicMax(status, LOGMEL_DEVICE_BAD_CACHE); }
  // lens[s], clamped to what the table holds
  __device__ int length(int s, bool report) const {
    const int len = lens[s];
    if (len >= 0 && len <= capacity) return len;
    if (report) flag();
    return len < 0 ? 0 : capacity;
  }
  // page id of a table entry, or -1 when it names no page
  __device__ int page(int s, int entry) const {
    const int p = table[(int64_t)s * width + entry];
    return (unsigned)p < (unsigned)n_pages ? p : -1;
  }
};

struct Rows {
  char* data;
  int64_t row, head;   // strides in elements
};

// Slots [lo, hi) that new token i of n sees.  Clamping at zero keeps tokens
// whose slot would be negative (a length shorter than the push) empty.
__device__ __forceinline__ int2 seen(int len, int n, int i, int causal, int window) {
  const int p = len - n + i;
  int hi = causal ? min(len, p + 1) : len;
  const int lo = window > 0 ? max(0, p - window + 1) : 0;   // p < 2^31 - 1 - window is not needed: p <= len
  hi = max(hi, 0);
  return make_int2(min(lo, hi), hi);
}

template <typename T>
struct Half2;
template <>
struct Half2<__nv_bfloat16> {
  static __device__ __forceinline__ float2 to_float(uint32_t x) {
    return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
  }
  static __device__ __forceinline__ uint32_t from_float(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  static constexpr uint32_t EXPONENT = 0x7f807f80u;   // both halves' exponent bits
  // acc + 0 * x: turns (and stays) NaN where x is not finite
  static __device__ __forceinline__ uint32_t times_zero(uint32_t x, uint32_t acc) {
    asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(x), "r"(0u));
    return acc;
  }
};
template <>
struct Half2<__half> {
  static __device__ __forceinline__ float2 to_float(uint32_t x) {
    return __half22float2(*reinterpret_cast<const __half2*>(&x));
  }
  static __device__ __forceinline__ uint32_t from_float(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  static constexpr uint32_t EXPONENT = 0x7c007c00u;
  static __device__ __forceinline__ uint32_t times_zero(uint32_t x, uint32_t acc) {
    asm("fma.rn.f16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(x), "r"(0u));
    return acc;
  }
};

}  // namespace cache
}  // namespace logmel

// Token cache: the attention weight that each cached key received (tcgen05).
//
// The scores are computed the other way round than in attention: keys are
// the rows of the tensor-core tile and new rows (token x query head of the key
// head) its columns, so that a thread owns a key and adds up its weights in
// registers; nothing is exchanged between threads, and the order is fixed.
// A weight needs no running maximum: exp(x - lse) with the row's known lse.
//
// An item is 256 slots of one (stream, key head), two 128-key tiles.  Its
// query rows come in steps of N columns that both tiles share.  Items are
// dealt to the CTAs in runs of equal numbers of steps.  N = 16 serves pushes of
// few rows, where reading the keys is the bound and the ring holds 6 tiles of
// them; N = 128 the others, bound by the exponentials (one per pair of row
// and key against 2 x head_dim tensor-core operations).
//
// Roles as in the attention kernel: warps 0-3 and 4-7 own one key tile each,
// warp 8 copies, warp 9 issues the MMAs into two score buffers per tile.
#pragma once
#include "cache_chunk.cuh"

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
  CUtensorMap q_map, k_map;
  int tokens;          // tokens of a step: N / group
  int box_keys;        // slots a key copy brings
};

template <int D, int N>
struct WeighShape {
  static constexpr int K_TILE = TILE_KEYS * D * 2, Q_TILE = N * D * 2;
  static constexpr int K_STAGES = N == 128 ? 3 : 6, Q_STAGES = N == 128 ? 3 : 4;
  static constexpr int SMEM = 1024 + K_STAGES * K_TILE + Q_STAGES * Q_TILE;
  static constexpr int COLUMNS = N == 128 ? 512 : 64;   // tensor memory: two score buffers per tile
};

constexpr int WEIGH_KEYS = 2 * TILE_KEYS;

// Which tokens of a push see some of the slots [k0, k1): [begin, end).
__device__ __forceinline__ int2 tokens_that_see(const WeighArgs& a, int n, int len, int k0, int k1) {
  const int p0 = len - n;   // slot of token 0
  const int begin = a.causal ? max(0, k0 - p0) : 0;
  // token i sees no slot at or below p0 + i - window
  const int end = a.window > 0 ? (int)max((int64_t)0, min((int64_t)n, (int64_t)k1 - 1 - p0 + a.window)) : n;
  return make_int2(min(begin, end), end);
}

struct WeighPlace {
  int s, h, item;
  int n, len, items;

  __device__ void load_stream(const WeighArgs& a) {
    n = a.b.count(s);
    len = a.c.length(s, false);
    items = n == 0 ? 0 : (len + WEIGH_KEYS - 1) / WEIGH_KEYS;
  }
  __device__ int steps_each(const WeighArgs& a) const { return max(1, (n + a.tokens - 1) / a.tokens); }
  // to the next item of the line; false at its end
  __device__ bool next(const WeighArgs& a) {
    if (++item < items) return true;
    item = 0;
    if (++h < a.n_kv) return true;
    h = 0;
    do {
      if (++s >= a.b.streams) return false;
      load_stream(a);
    } while (items == 0);
    return true;
  }
};

template <typename F>
__device__ __forceinline__ void for_items(const WeighArgs& a, WeighPlace p, int64_t u, int64_t u1, F&& f) {
  while (u < u1) {
    const int k0 = p.item * WEIGH_KEYS, k1 = min(p.len, k0 + WEIGH_KEYS);
    const int2 tok = tokens_that_see(a, p.n, p.len, k0, k1);
    if (!f(p, k0, k1, tok, (tok.y - tok.x + a.tokens - 1) / a.tokens)) return;
    u += p.steps_each(a);
    if (u < u1 && !p.next(a)) return;
  }
}

template <typename T, int D, int N>
__global__ void __launch_bounds__(CHUNK_THREADS, 1) weigh_kernel(const __grid_constant__ WeighArgs a) {
  using Shape = WeighShape<D, N>;
  constexpr int KS = Shape::K_STAGES, QS = Shape::Q_STAGES, HALVES = D / 64;
  constexpr int K_HALF = Shape::K_TILE / HALVES, Q_HALF = Shape::Q_TILE / HALVES;
  extern __shared__ char smem_raw[];
  __shared__ alignas(8) uint64_t bars[2 * KS + 2 * QS + 8];
  __shared__ uint32_t tmem_base_sh;
  __shared__ int stop_sh;
  __shared__ int64_t warp_total[CHUNK_THREADS / 32];
  __shared__ WeighPlace start_sh;
  __shared__ int64_t start_u_sh;
  __shared__ alignas(16) float minus_lse[8][N];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  volatile int* stop = &stop_sh;
  int* status = a.c.status;
  const uint32_t smem0 = (smem_address(smem_raw) + 1023) & ~1023u;
  const uint32_t k_ring = smem0, q_ring = smem0 + KS * Shape::K_TILE;
  const uint32_t bar0 = smem_address(bars);
  auto k_full = [&](int i) { return bar0 + 8 * i; };
  auto k_free = [&](int i) { return bar0 + 8 * (KS + i); };
  auto q_full = [&](int i) { return bar0 + 8 * (2 * KS + i); };
  auto q_free = [&](int i) { return bar0 + 8 * (2 * KS + QS + i); };
  auto s_full = [&](int tile, int buf) { return bar0 + 8 * (2 * KS + 2 * QS + 2 * tile + buf); };
  auto s_free = [&](int tile, int buf) { return bar0 + 8 * (2 * KS + 2 * QS + 4 + 2 * tile + buf); };

  if (warp == 9) tmem_alloc(smem_address(&tmem_base_sh), Shape::COLUMNS);
  if (tid == 0) {
    for (int i = 0; i < KS; ++i) {
      mbar_init(k_full(i), 1);
      mbar_init(k_free(i), 1);
    }
    for (int i = 0; i < QS; ++i) {
      mbar_init(q_full(i), 1);
      mbar_init(q_free(i), 1);
    }
    for (int t = 0; t < 2; ++t)
      for (int i = 0; i < 2; ++i) {
        mbar_init(s_full(t, i), 1);
        mbar_init(s_free(t, i), 4);
      }
    stop_sh = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }

  // The line: steps of one key head before every stream, in the ring's memory (which holds no tile yet).
  int64_t* before = (int64_t*)(smem_raw + (k_ring - smem_address(smem_raw)));
  const int S = a.b.streams;
  {
    const int per = (S + CHUNK_THREADS - 1) / CHUNK_THREADS;
    auto work = [&](int s, bool report) -> int64_t {
      const int n = a.b.count(s), len = a.c.length(s, report);
      return n == 0 ? 0 : (int64_t)((len + WEIGH_KEYS - 1) / WEIGH_KEYS) * ((n + a.tokens - 1) / a.tokens);
    };
    for (int s = tid; s < S; s += CHUNK_THREADS) before[s] = work(s, blockIdx.x == 0);
    __syncthreads();
    int64_t sum = 0;
    for (int i = 0; i < per; ++i)
      if (tid * per + i < S) sum += before[tid * per + i];
    int64_t run = sum;
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t y = __shfl_up_sync(~0u, run, d);
      if (lane >= d) run += y;
    }
    if (lane == 31) warp_total[warp] = run;
    __syncthreads();
    run -= sum;
    for (int w = 0; w < warp; ++w) run += warp_total[w];
    for (int i = 0; i < per; ++i) {
      const int s = tid * per + i;
      if (s < S) {
        const int64_t own = before[s];
        before[s] = run;
        run += own;
        if (s == S - 1) before[S] = run;
      }
    }
    __syncthreads();
  }
  const int64_t total = before[S] * a.n_kv;
  const int64_t quota = max((int64_t)1, (total + gridDim.x - 1) / gridDim.x);
  const int64_t u1 = min(total, (int64_t)(blockIdx.x + 1) * quota);
  if (tid == 0) {
    // the first item that begins in [blockIdx.x * quota, u1)
    const int64_t want = (int64_t)blockIdx.x * quota;
    int64_t u = u1;
    if (want < u1) {
      int lo = 0, hi = S - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (before[mid] * a.n_kv <= want) lo = mid;
        else hi = mid - 1;
      }
      WeighPlace p;
      p.s = lo;
      p.load_stream(a);
      const int64_t per_head = before[lo + 1] - before[lo], steps = p.steps_each(a);
      int64_t left = want - before[lo] * a.n_kv;
      p.h = (int)(left / per_head);
      left -= p.h * per_head;
      p.item = (int)((left + steps - 1) / steps);
      u = before[lo] * a.n_kv + p.h * per_head + p.item * steps;
      bool there = true;
      if (p.item >= p.items) {
        p.item = p.items - 1;
        there = p.next(a);
      }
      if (!there) u = u1;
      start_sh = p;
    }
    start_u_sh = u;
  }
  // columns that no copy fills must not hold stale values that are not finite
  for (int i = tid; i < QS * Shape::Q_TILE / 16; i += CHUNK_THREADS)
    asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(q_ring + 16 * i), "r"(0) : "memory");
  fence_async_smem();
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = tmem_base_sh;
  const WeighPlace start = start_sh;
  const int64_t u0 = start_u_sh;

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if (warp == 8) {
      // ---- copies ----
      int ks = 0, qs = 0;
      uint32_t k_phase = 0, q_phase = 0;
      const int in_page = (1 << a.c.page_shift) - 1;
      const int boxes = TILE_KEYS / a.box_keys;
      const uint32_t box_bytes = a.box_keys * 128;
      for_items(a, start, u0, u1, [&](const WeighPlace& p, int k0, int k1, int2 tok, int steps) {
        if (steps == 0) return true;
        for (int key0 = k0; key0 < k1; key0 += TILE_KEYS) {
          const int box = lane / HALVES, half = lane % HALVES, key = key0 + box * a.box_keys;
          int page = -1;
          if (box < boxes && key < k1) {
            page = a.c.page(p.s, key >> a.c.page_shift);
            if (page < 0) a.c.flag();
          }
          const uint32_t live = __ballot_sync(~0u, page >= 0);
          if (!mbar_wait(k_free(ks), k_phase ^ 1, stop, status)) return false;
          if (lane == 0) mbar_expect(k_full(ks), __popc(live) * box_bytes);
          __syncwarp();
          if (page >= 0)
            tma_load_4d(k_ring + ks * Shape::K_TILE + half * K_HALF + box * box_bytes, &a.k_map, 64 * half, key & in_page,
                        p.h, page, k_full(ks));
          if (++ks == KS) ks = 0, k_phase ^= 1;
        }
        const int row = a.b.begin(p.s) + tok.x;
        for (int i = 0; i < steps; ++i) {
          if (!mbar_wait(q_free(qs), q_phase ^ 1, stop, status)) return false;
          if (lane == 0) {
            mbar_expect(q_full(qs), HALVES * a.tokens * a.group * 128);
            for (int c = 0; c < HALVES; ++c)
              tma_load_3d(q_ring + qs * Shape::Q_TILE + c * Q_HALF, &a.q_map, 64 * c, p.h * a.group, row + i * a.tokens,
                          q_full(qs));
          }
          __syncwarp();
          if (++qs == QS) qs = 0, q_phase ^= 1;
        }
        return true;
      });
    } else if (warp == 9) {
      // ---- products ----
      int ks = 0, qs = 0;
      uint32_t k_phase = 0, q_phase = 0, uses[2] = {0, 0};
      constexpr uint32_t KIND = mma_kind<T>(TILE_KEYS, N, false);
      for_items(a, start, u0, u1, [&](const WeighPlace& p, int k0, int k1, int2, int steps) {
        if (steps == 0) return true;
        const int tiles = k1 - k0 > TILE_KEYS ? 2 : 1;
        int k_stage[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (t >= tiles) break;
          if (!mbar_wait(k_full(ks), k_phase, stop, status)) return false;
          k_stage[t] = ks;
          if (++ks == KS) ks = 0, k_phase ^= 1;
        }
        for (int i = 0; i < steps; ++i) {
          if (!mbar_wait(q_full(qs), q_phase, stop, status)) return false;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (t >= tiles) break;
            const int buf = uses[t] & 1;
            if (!mbar_wait(s_free(t, buf), ((uses[t] >> 1) & 1) ^ 1, stop, status)) return false;
            ++uses[t];
            tmem_fence_after();
            if (elect_lane()) {
              const uint32_t k = k_ring + k_stage[t] * Shape::K_TILE, q = q_ring + qs * Shape::Q_TILE;
#pragma unroll
              for (int j = 0; j < D / 16; ++j)
                mma_ss(tmem + (2 * t + buf) * N, desc_k_major(k + (j & 3) * 32 + (j >> 2) * K_HALF),
                       desc_k_major(q + (j & 3) * 32 + (j >> 2) * Q_HALF), KIND, j > 0);
              mma_commit(s_full(t, buf));
            }
            __syncwarp();
          }
          if (elect_lane()) mma_commit(q_free(qs));
          if (++qs == QS) qs = 0, q_phase ^= 1;
        }
        if (elect_lane())
          for (int t = 0; t < tiles; ++t) mma_commit(k_free(k_stage[t]));
        __syncwarp();
        return true;
      });
    }
  } else {
    // ---- weights ----
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int tile = warp >> 2;
    const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);
    const float sc = a.scale * LOG2E;
    const uint64_t sc2 = pack2(sc, sc);
    float* ml = minus_lse[warp];
    uint32_t uses = 0;
    for_items(a, start, u0, u1, [&](const WeighPlace& p, int k0, int k1, int2 tok, int steps) {
      const int key0 = k0 + tile * TILE_KEYS, key = key0 + (tid & 127);
      if (key0 >= k1) return true;
      const bool live = key < k1;
      const int page = live ? a.c.page(p.s, key >> a.c.page_shift) : -1;
      if (live && page < 0) a.c.flag();
      const int64_t at = (((int64_t)page * a.n_kv + p.h) << a.c.page_shift) + (key & ((1 << a.c.page_shift) - 1));
      const float old = page >= 0 ? a.c.mass[at] : 0.f;
      const int2 mine = live ? tokens_that_see(a, p.n, p.len, key, key + 1) : make_int2(0, 0);
      const int64_t row0 = a.b.begin(p.s);
      uint64_t sum0 = pack2(0.f, 0.f), sum1 = sum0;
      for (int i = 0; i < steps; ++i) {
        const int t0 = tok.x + i * a.tokens, full = a.tokens * a.group, cols = min(full, (tok.y - t0) * a.group);
        // this warp's copy of -lse (base 2) of the step's rows; its latency hides behind the wait
        float nl[(N + 31) / 32];
        bool odd = false;   // a row whose lse is not finite
#pragma unroll
        for (int e = 0; e < (N + 31) / 32; ++e) {
          const int c = lane + 32 * e, tk = c / a.group;
          nl[e] = c < cols ? -LOG2E * a.lse[(row0 + t0 + tk) * a.n_q + p.h * a.group + c - tk * a.group] : -INFINITY;
          odd |= c < cols && !(fabsf(nl[e]) < INFINITY);
        }
        __syncwarp();
#pragma unroll
        for (int e = 0; e < (N + 31) / 32; ++e)
          if (lane + 32 * e < N) ml[lane + 32 * e] = nl[e];
        __syncwarp();
        const int buf = uses & 1;
        if (!mbar_wait(s_full(tile, buf), (uses >> 1) & 1, stop, status)) return false;
        ++uses;
        tmem_fence_after();
        const uint32_t s_tmem = lanes + (2 * tile + buf) * N;
        uint32_t x[N];
#pragma unroll
        for (int c = 0; c < N; c += 32) {
          if constexpr (N >= 32) tmem_load32(x + c, s_tmem + c);
          else tmem_load16(x, s_tmem);
        }
        tmem_wait_load();
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(s_free(tile, buf));
        // columns of the tokens that see this key
        const int lo = (max(mine.x, t0) - t0) * a.group, hi = min((mine.y - t0) * a.group, cols);
        const bool plain = __all_sync(~0u, lo == 0 && hi >= full && !odd);
        if (plain) {
#pragma unroll
          for (int c = 0; c < N; c += 4) {   // of every 4 exponentials 2 on the FMA pipe
            const float4 z = *(const float4*)(ml + c);
            const float2 y0 = unpack2(fma2(pack2(__uint_as_float(x[c]), __uint_as_float(x[c + 1])), sc2, pack2(z.x, z.y)));
            const uint64_t y1 = fma2(pack2(__uint_as_float(x[c + 2]), __uint_as_float(x[c + 3])), sc2, pack2(z.z, z.w));
            sum0 = add2(sum0, pack2(exp2_approx(y0.x), exp2_approx(y0.y)));
            sum1 = add2(sum1, exp2_fit(y1));
          }
        } else {
#pragma unroll
          for (int c = 0; c < N; c += 2) {
            const float2 z = *(const float2*)(ml + c);
            const float e0 = exp2_approx(fmaf(__uint_as_float(x[c]), sc, z.x));
            const float e1 = exp2_approx(fmaf(__uint_as_float(x[c + 1]), sc, z.y));
            sum0 = add2(sum0, pack2(c >= lo && c < hi ? e0 : 0.f, c + 1 >= lo && c + 1 < hi ? e1 : 0.f));
          }
        }
      }
      const float2 both = unpack2(add2(sum0, sum1));
      if (page >= 0) a.out[at] = a.decay * old + (both.x + both.y);
      return true;
    });
  }
  if (*stop)
    for (int i = 0; i < 1000; ++i) __nanosleep(1000);
  tmem_fence_before();
  __syncthreads();
  if (warp == 9) tmem_free(tmem, Shape::COLUMNS);
}

}  // namespace cache
}  // namespace logmel

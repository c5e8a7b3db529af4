// Routing rows to experts and back: the router's top-k with its gradient, the stable order of the
// assignments by expert, and the row moves (gather to the sorted order, combine with weights, and
// the combine's gradient). An assignment a = t * topk + j is token t's j-th expert.
//
// The row moves are bound by HBM: one warp a token, so that a token's own row crosses once however
// many experts it goes to. The router and the sort are bound by latency.
#include "kernels.h"
#include "rows.cuh"

namespace ss {

// ---- router ---------------------------------------------------------------------------------
// Floats in an order that unsigned integers keep: larger float, larger key. -inf and NaN (a closed
// expert) give key 0, which no other float has.
__device__ __forceinline__ uint32_t rank_key(float v) {
  if (!(v > -INFINITY)) return 0u;
  const uint32_t u = __float_as_uint(v + 0.0f);   // -0.0 ties with +0.0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

// One warp a token, V logits a lane (expert v * 32 + lane). Each of the k rounds takes the largest key
// left (two warp reductions: the key, then the lowest expert that has it).
template <int V>
__global__ void __launch_bounds__(256) k_expert_route(const float* __restrict__ logits,
                                                      int32_t* __restrict__ ids,
                                                      float* __restrict__ weight, int T, int E,
                                                      int topk, int renorm) {
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (t >= T) return;
  uint32_t key[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = v * 32 + lane;
    key[v] = e < E ? rank_key(__ldg(logits + (size_t)t * E + e)) : 0u;
  }
  float top = 0.f, total = 0.f, mine = 0.f;
  int my_id = -1;
  for (int j = 0; j < topk; ++j) {
    uint32_t best = key[0];
#pragma unroll
    for (int v = 1; v < V; ++v) best = best > key[v] ? best : key[v];
    best = __reduce_max_sync(0xffffffffu, best);
    if (best == 0u) break;   // every expert left is closed
    int at = 1 << 30;
#pragma unroll
    for (int v = V - 1; v >= 0; --v)
      if (key[v] == best) at = v * 32 + lane;
    at = __reduce_min_sync(0xffffffffu, at);
    const float value = key_value(best);
    if (j == 0) {
      top = value;
      if (!renorm) {
        float s = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v)
          if (key[v]) s += expf(key_value(key[v]) - top);
        total = warp_sum(s);
      }
    }
    const float ex = expf(value - top);
    if (renorm) total += ex;
    if (lane == j) {
      mine = ex;
      my_id = at;
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (v * 32 + lane == at) key[v] = 0u;
  }
  if (lane < topk) {
    ids[(size_t)t * topk + lane] = my_id;
    weight[(size_t)t * topk + lane] = my_id >= 0 ? mine / total : 0.f;
  }
}

cudaError_t launch_expert_route(const float* logits, int32_t* ids, float* weight, int T, int E,
                                int topk, bool renorm, cudaStream_t st) {
  const dim3 grid((T + 7) / 8), block(256);
  auto go = [&](auto kernel) {
    return launch_pdl(kernel, grid, block, 0, st, logits, ids, weight, T, E, topk,
                      renorm ? 1 : 0);
  };
  if (E <= 32) return go(k_expert_route<1>);
  if (E <= 64) return go(k_expert_route<2>);
  if (E <= 128) return go(k_expert_route<4>);
  if (E <= 256) return go(k_expert_route<8>);
  return go(k_expert_route<16>);
}

// Gradient of the weights for the logits. Renormalised: w is the softmax of the chosen logits, so
// dlogit_j = w_j (dw_j - sum_i dw_i w_i) there and zero elsewhere. Otherwise w_j = p[id_j] of the
// softmax p over all open experts: dlogit_e = p_e (dw_e - sum_i dw_i w_i), dw_e = 0 if not chosen.
template <int V>
__global__ void __launch_bounds__(256)
    k_expert_route_backward(const float* __restrict__ logits, const int32_t* __restrict__ ids,
                            const float* __restrict__ weight, const float* __restrict__ dweight,
                            float* __restrict__ dlogits, int T, int E, int topk, int renorm,
                            int* status) {
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (t >= T) return;
  int id = -1;
  float w = 0.f, dw = 0.f;
  if (lane < topk) {
    id = __ldg(ids + (size_t)t * topk + lane);
    if (id < -1 || id >= E) {
      record_bad_index(status);
      id = -1;
    }
    if (id >= 0) {
      w = __ldg(weight + (size_t)t * topk + lane);
      dw = __ldg(dweight + (size_t)t * topk + lane);
    }
  }
  const float mean = warp_sum(w * dw);
  float d[V];
  if (renorm) {
#pragma unroll
    for (int v = 0; v < V; ++v) d[v] = 0.f;
  } else {
    uint32_t key[V], best = 0u;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = v * 32 + lane;
      key[v] = e < E ? rank_key(__ldg(logits + (size_t)t * E + e)) : 0u;
      best = best > key[v] ? best : key[v];
    }
    best = __reduce_max_sync(0xffffffffu, best);
    const float top = best ? key_value(best) : 0.f;
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      d[v] = key[v] ? expf(key_value(key[v]) - top) : 0.f;
      s += d[v];
    }
    const float total = warp_sum(s);
#pragma unroll
    for (int v = 0; v < V; ++v) d[v] = d[v] > 0.f ? -mean * (d[v] / total) : 0.f;
  }
  for (int j = 0; j < topk; ++j) {
    const int e = __shfl_sync(0xffffffffu, id, j);
    const float add = __shfl_sync(0xffffffffu, renorm ? w * (dw - mean) : w * dw, j);
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (v * 32 + lane == e) d[v] += add;
  }
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (v * 32 + lane < E) dlogits[(size_t)t * E + v * 32 + lane] = d[v];
}

cudaError_t launch_expert_route_backward(const float* logits, const int32_t* ids,
                                         const float* weight, const float* dweight, float* dlogits,
                                         int T, int E, int topk, bool renorm, int* status,
                                         cudaStream_t st) {
  const dim3 grid((T + 7) / 8), block(256);
  auto go = [&](auto kernel) {
    return launch_pdl(kernel, grid, block, 0, st, logits, ids, weight, dweight, dlogits, T, E,
                      topk, renorm ? 1 : 0, status);
  };
  if (E <= 32) return go(k_expert_route_backward<1>);
  if (E <= 64) return go(k_expert_route_backward<2>);
  if (E <= 128) return go(k_expert_route_backward<4>);
  if (E <= 256) return go(k_expert_route_backward<8>);
  return go(k_expert_route_backward<16>);
}

// ---- sort -----------------------------------------------------------------------------------
// A stable counting sort. Each of the CTAs owns a contiguous chunk of the assignments, each of its
// 16 warps a contiguous part of that, walked 32 at a time: __match_any_sync groups the lanes of one
// expert, whose order in the group is their order in the sort. With more than one CTA a first
// launch counts each CTA's experts; the placing launch then adds up the CTAs before its own.
constexpr int kSortWarps = 16;
constexpr int kSortThreads = kSortWarps * 32;

// Expert of assignment a, or -1 (routed nowhere; an id outside [-1, E) is recorded and dropped).
__device__ __forceinline__ int sort_expert(const int32_t* ids, int a, int E, int* status) {
  const int e = __ldg(ids + a);
  if (e < -1 || e >= E) {
    record_bad_index(status);
    return -1;
  }
  return e;
}

// counts[e] += the experts of [a0, a1), by this warp.
__device__ __forceinline__ void sort_count(const int32_t* ids, int a0, int a1, int E, int* counts,
                                           int* status) {
  const int lane = threadIdx.x & 31;
  for (int a = a0; a < a1; a += 32) {
    const int e = a + lane < a1 ? sort_expert(ids, a + lane, E, status) : -1;
    const uint32_t same = __match_any_sync(0xffffffffu, e);
    if (e >= 0 && (same & ((1u << lane) - 1)) == 0) counts[e] += __popc(same);
    __syncwarp();
  }
}

__global__ void __launch_bounds__(kSortThreads) k_expert_count(const int32_t* __restrict__ ids,
                                                               int32_t* __restrict__ hist, int n,
                                                               int chunk, int E, int* status) {
  extern __shared__ int counts[];   // [warps][E]
  griddep_wait();
  griddep_launch();
  const int warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < kSortWarps * E; i += kSortThreads) counts[i] = 0;
  __syncthreads();
  const int c0 = blockIdx.x * chunk, c1 = min(n, c0 + chunk);
  const int part = ((chunk + kSortWarps - 1) / kSortWarps + 31) / 32 * 32;
  sort_count(ids, min(c1, c0 + warp * part), min(c1, c0 + (warp + 1) * part), E, counts + warp * E,
             status);
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kSortThreads) {
    int s = 0;
    for (int w = 0; w < kSortWarps; ++w) s += counts[w * E + e];
    hist[(size_t)blockIdx.x * E + e] = s;
  }
}

__global__ void __launch_bounds__(kSortThreads)
    k_expert_place(const int32_t* __restrict__ ids, const int32_t* __restrict__ hist,
                   int32_t* __restrict__ order, int32_t* __restrict__ slot,
                   int32_t* __restrict__ offsets, int n, int chunk, int E, int* status) {
  extern __shared__ int counts[];   // [warps][E]: counts, then the next place of each expert
  __shared__ int s_sum[kSortWarps];
  __shared__ int s_total;
  griddep_wait();
  griddep_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < kSortWarps * E; i += kSortThreads) counts[i] = 0;
  __syncthreads();
  const int c0 = blockIdx.x * chunk, c1 = min(n, c0 + chunk);
  const int part = ((chunk + kSortWarps - 1) / kSortWarps + 31) / 32 * 32;
  const int a0 = min(c1, c0 + warp * part), a1 = min(c1, c0 + (warp + 1) * part);
  sort_count(ids, a0, a1, E, counts + warp * E, status);
  __syncthreads();
  // Thread e (E <= the CTA's threads): its expert's total over all CTAs and over those before.
  int total = 0, before = 0;
  const int e = threadIdx.x;
  if (e < E) {
    if (gridDim.x == 1) {
      for (int w = 0; w < kSortWarps; ++w) total += counts[w * E + e];
    } else {
#pragma unroll 8
      for (int b = 0; b < gridDim.x; ++b) {
        const int h = __ldg(hist + (size_t)b * E + e);
        total += h;
        before += b < blockIdx.x ? h : 0;
      }
    }
  }
  // Exclusive sum of the totals over the experts.
  int x = total;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s_sum[warp] = x;
  __syncthreads();
  if (threadIdx.x < kSortWarps) {
    int y = s_sum[threadIdx.x];
#pragma unroll
    for (int o = 1; o < kSortWarps; o <<= 1) {
      const int z = __shfl_up_sync((1u << kSortWarps) - 1, y, o);
      if (threadIdx.x >= o) y += z;
    }
    s_sum[threadIdx.x] = y;
  }
  __syncthreads();
  const int first = x - total + (warp ? s_sum[warp - 1] : 0);
  if (e < E) {
    int at = first + before;
    for (int w = 0; w < kSortWarps; ++w) {
      const int c = counts[w * E + e];
      counts[w * E + e] = at;
      at += c;
    }
    if (offsets && blockIdx.x == 0) {
      offsets[e] = first;
      if (e == E - 1) offsets[E] = first + total;
    }
    if (e == E - 1) s_total = first + total;
  }
  __syncthreads();
  int* next = counts + warp * E;
  for (int a = a0; a < a1; a += 32) {
    const bool live = a + lane < a1;
    const int ex = live ? sort_expert(ids, a + lane, E, status) : -1;
    const uint32_t same = __match_any_sync(0xffffffffu, ex);
    const uint32_t lower = same & ((1u << lane) - 1);
    const int at = ex >= 0 ? next[ex] + __popc(lower) : -1;
    __syncwarp();
    if (ex >= 0 && lower == 0) next[ex] += __popc(same);
    __syncwarp();
    if (live) {
      if (slot) slot[a + lane] = at;
      if (order && at >= 0) order[at] = a + lane;
      // places past the routed assignments hold none
      if (order && a + lane >= s_total) order[a + lane] = -1;
    }
  }
}

// CTAs the sort takes: one up to kSortOne assignments, else one per kSortOne / 8 up to kSortMaxCtas.
int sort_ctas(long long n) {
  if (n <= kSortOne) return 1;
  const long long c = (n + kSortOne / 8 - 1) / (kSortOne / 8);
  return (int)(c < kSortMaxCtas ? c : kSortMaxCtas);
}

cudaError_t launch_expert_count(const int32_t* ids, int32_t* hist, int n, int E, int* status,
                                cudaStream_t st) {
  const int ctas = sort_ctas(n), chunk = (n + ctas - 1) / ctas;
  return launch_pdl(k_expert_count, dim3(ctas), dim3(kSortThreads),
                    (size_t)kSortWarps * E * sizeof(int), st, ids, hist, n, chunk, E, status);
}

cudaError_t launch_expert_place(const int32_t* ids, const int32_t* hist, int32_t* order,
                                int32_t* slot, int32_t* offsets, int n, int E, int* status,
                                cudaStream_t st) {
  const int ctas = sort_ctas(n), chunk = n > 0 ? (n + ctas - 1) / ctas : 0;
  return launch_pdl(k_expert_place, dim3(ctas), dim3(kSortThreads),
                    (size_t)kSortWarps * E * sizeof(int), st, ids, hist, order, slot, offsets, n,
                    chunk, E, status);
}

// ---- row moves ------------------------------------------------------------------------------
// The sorted place of assignment a, or -1 (none; one outside [-1, n) is recorded and skipped).
__device__ __forceinline__ int row_slot(const int32_t* slot, long long a, int n, int* status) {
  const int p = __ldg(slot + a);
  if (p < -1 || p >= n) {
    record_bad_index(status);
    return -1;
  }
  return p;
}

// xs[slot[t, j]] = x[t]: the token's row is loaded once, up to eight chunks a lane in flight.
template <class T>
__global__ void __launch_bounds__(256)
    k_expert_gather(const typename T::Store* __restrict__ x, const int32_t* __restrict__ slot,
                    typename T::Store* __restrict__ xs, int tokens, int topk, int C, long long ld,
                    int* status) {
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (t >= tokens) return;
  int my = -1;
  if (lane < topk) my = row_slot(slot, (long long)t * topk + lane, tokens * topk, status);
  const int chunks = C / 8;
  constexpr int kFlight = T::kWords == 4 ? 8 : 4;
  for (int cb = 0; cb < chunks; cb += 32 * kFlight) {
    Chunk<T> buf[kFlight];
#pragma unroll
    for (int i = 0; i < kFlight; ++i) {
      const int c = cb + 32 * i + lane;
      if (c < chunks) chunk_load(buf[i], x + (size_t)t * ld + c * 8);
    }
    for (int j = 0; j < topk; ++j) {
      const int p = __shfl_sync(0xffffffffu, my, j);
      if (p < 0) continue;
#pragma unroll
      for (int i = 0; i < kFlight; ++i) {
        const int c = cb + 32 * i + lane;
        if (c < chunks) chunk_store(xs + (size_t)p * C + c * 8, buf[i]);
      }
    }
  }
}

cudaError_t launch_expert_gather(const void* x, const int32_t* slot, void* xs, int tokens,
                                 int topk, int C, long long ld, int dtype, int* status,
                                 cudaStream_t st) {
  return by_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    using S = typename T::Store;
    return launch_pdl(k_expert_gather<T>, dim3((tokens + 7) / 8), dim3(256), 0, st,
                      static_cast<const S*>(x), slot, static_cast<S*>(xs), tokens, topk, C, ld,
                      status);
  });
}

// out[t] = residual[t] + sum_j weight[t, j] * ys[slot[t, j]], the sum in fp32 in the order of j, then the
// residual. Y: the sorted rows' type (fp32 partials of `splits` k-splits, `split_stride` apart, are
// added first, in split order).
template <class T, class Y>
__global__ void __launch_bounds__(256)
    k_expert_combine(const typename Y::Store* __restrict__ ys, const int32_t* __restrict__ slot,
                     const float* __restrict__ weight, const typename T::Store* residual,
                     typename T::Store* out, int tokens, int topk, int C, long long ld, int splits,
                     long long split_stride, int* status) {
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (t >= tokens) return;
  int my = -1;
  float my_w = 0.f;
  if (lane < topk) {
    my = row_slot(slot, (long long)t * topk + lane, tokens * topk, status);
    my_w = weight ? __ldg(weight + (size_t)t * topk + lane) : 1.f;
  }
  const int chunks = C / 8;
  for (int cb = 0; cb < chunks; cb += 64) {
    float acc[2][8];
    Chunk<T> res[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      chunk_zero(res[i]);
#pragma unroll
      for (int q = 0; q < 8; ++q) acc[i][q] = 0.f;
      const int c = cb + 32 * i + lane;
      if (residual && c < chunks) chunk_load(res[i], residual + (size_t)t * ld + c * 8);
    }
#pragma unroll 4
    for (int j = 0; j < topk; ++j) {
      const int p = __shfl_sync(0xffffffffu, my, j);
      const float w = __shfl_sync(0xffffffffu, my_w, j);
      if (p < 0) continue;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int c = cb + 32 * i + lane;
        if (c >= chunks) continue;
        float f[8];
        Chunk<Y> v;
        chunk_load(v, ys + (size_t)p * C + c * 8);
        chunk_floats(v, f);
        for (int s = 1; s < splits; ++s) {
          float g[8];
          chunk_load(v, ys + s * split_stride + (size_t)p * C + c * 8);
          chunk_floats(v, g);
#pragma unroll
          for (int q = 0; q < 8; ++q) f[q] += g[q];
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) acc[i][q] += w * f[q];
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int c = cb + 32 * i + lane;
      if (c >= chunks) continue;
      float r[8];
      chunk_floats(res[i], r);
#pragma unroll
      for (int q = 0; q < 8; ++q) acc[i][q] += r[q];
      Chunk<T> o;
      chunk_round(o, acc[i]);
      chunk_store(out + (size_t)t * ld + c * 8, o);
    }
  }
}

cudaError_t launch_expert_combine(const void* ys, const int32_t* slot, const float* weight,
                                  const void* residual, void* out, int tokens, int topk, int C,
                                  long long ld, int dtype, int splits, int* status,
                                  cudaStream_t st) {
  return by_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    using S = typename T::Store;
    auto go = [&](auto y) {
      using Y = decltype(y);
      return launch_pdl(k_expert_combine<T, Y>, dim3((tokens + 7) / 8), dim3(256), 0, st,
                        static_cast<const typename Y::Store*>(ys), slot, weight,
                        static_cast<const S*>(residual), static_cast<S*>(out), tokens, topk, C, ld,
                        splits > 1 ? splits : 1, (long long)tokens * topk * C, status);
    };
    return splits > 0 ? go(F32{}) : go(t);
  });
}

// The combine's gradient: dys[slot[t, j]] = weight[t, j] * dout[t] (rounded once) and
// dweight[t, j] = dout[t] . ys[slot[t, j]], in one walk over the token's chunks (K assignments' dot
// products at a time).
template <class T>
__global__ void __launch_bounds__(256)
    k_expert_combine_backward(const typename T::Store* __restrict__ dout,
                              const typename T::Store* ys, const int32_t* __restrict__ slot,
                              const float* __restrict__ weight, typename T::Store* dys,
                              float* __restrict__ dweight, int tokens, int topk, int C,
                              long long ld, int* status) {
  constexpr int K = 4;
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (t >= tokens) return;
  int my = -1;
  float my_w = 0.f;
  if (lane < topk) {
    my = row_slot(slot, (long long)t * topk + lane, tokens * topk, status);
    my_w = __ldg(weight + (size_t)t * topk + lane);
  }
  const int chunks = C / 8;
  float my_dw = 0.f;
  for (int j0 = 0; j0 < topk; j0 += K) {
    int p[K];
    float w[K], dot[K];
#pragma unroll
    for (int q = 0; q < K; ++q) {
      p[q] = __shfl_sync(0xffffffffu, my, (j0 + q) & 31);
      w[q] = __shfl_sync(0xffffffffu, my_w, (j0 + q) & 31);
      if (j0 + q >= topk) p[q] = -1;
      dot[q] = 0.f;
    }
    for (int c = lane; c < chunks; c += 32) {
      Chunk<T> d, y[K];
      chunk_load(d, dout + (size_t)t * ld + c * 8);
#pragma unroll
      for (int q = 0; q < K; ++q)
        if (p[q] >= 0) chunk_load(y[q], ys + (size_t)p[q] * C + c * 8);
      float df[8];
      chunk_floats(d, df);
#pragma unroll
      for (int q = 0; q < K; ++q) {
        if (p[q] < 0) continue;
        float yf[8];
        chunk_floats(y[q], yf);
#pragma unroll
        for (int i = 0; i < 8; ++i) dot[q] += df[i] * yf[i];
#pragma unroll
        for (int i = 0; i < 8; ++i) yf[i] = w[q] * df[i];
        Chunk<T> o;
        chunk_round(o, yf);
        chunk_store(dys + (size_t)p[q] * C + c * 8, o);
      }
    }
#pragma unroll
    for (int q = 0; q < K; ++q) {
      const float s = warp_sum(dot[q]);
      if (lane == j0 + q) my_dw = s;
    }
  }
  if (lane < topk) dweight[(size_t)t * topk + lane] = my_dw;
}

cudaError_t launch_expert_combine_backward(const void* dout, const void* ys, const int32_t* slot,
                                           const float* weight, void* dys, float* dweight,
                                           int tokens, int topk, int C, long long ld, int dtype,
                                           int* status, cudaStream_t st) {
  return by_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    using S = typename T::Store;
    return launch_pdl(k_expert_combine_backward<T>, dim3((tokens + 7) / 8), dim3(256), 0, st,
                      static_cast<const S*>(dout), static_cast<const S*>(ys), slot, weight,
                      static_cast<S*>(dys), dweight, tokens, topk, C, ld, status);
  });
}

}  // namespace ss

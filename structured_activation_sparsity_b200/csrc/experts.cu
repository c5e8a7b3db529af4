// Routing rows to experts and back: the router's top-k with its gradient, the stable order of the
// assignments by expert, and the row moves (gather to the sorted order, combine with weights, and
// the combine's gradient). An assignment a = t * topk + j is token t's j-th expert.
//
// The row moves are bound by HBM: warps work by token, so that a token's own row crosses once however
// many experts it goes to (16384 tokens of 1280 bf16 to two experts each and back: 49.0 us, 0.93 of the
// measured copy rate; the gradients of 32768 tokens of 1024: 82.2 us, 0.97). The router and the sort are
// bound by latency and instructions.
#include <algorithm>
#include <type_traits>

#include "kernels.h"
#include "rows.cuh"

namespace ss {

// ---- router ---------------------------------------------------------------------------------
// A logit as it ranks: NaN closes its expert like -inf. -0.0 compares equal to +0.0, so they tie.
__device__ __forceinline__ float open_logit(float v) { return fmaxf(v, -INFINITY); }
// e^(v - top) for two logits and the largest one, to a few ulp at any distance, subnormal results included:
// 2^(p + q) = 2^p (1 + q ln 2), p the product of the rounded difference d and log2 e, q what p and d lost
// (the difference's part by Knuth's exact sum: left out, it alone would cost |d| 2^-24). Past a distance
// of 200, closed logits among them, it is 0. The pair's arithmetic is packed: on 39200 tokens of 64
// experts the router and its gradient take 1.5 us more than with ex2 of the rounded product, and 3.2 with
// expf and scalar sums.
__device__ __forceinline__ void exp_below2(float v0, float v1, float top, float& e0, float& e1) {
  constexpr float kLog2e = 1.4426950408889634f, kLost = (float)(1.4426950408889634 - (double)kLog2e);
  const uint64_t minus = f2_pack(-1.f, -1.f), t = f2_pack(top, top), v = f2_pack(v0, v1);
  const uint64_t d = f2_fma(t, minus, v), b = f2_fma(v, minus, d);      // d = v - top, b = d - v
  const uint64_t r = f2_fma(f2_add(t, b), minus, f2_fma(f2_fma(b, minus, d), minus, v));
  const uint64_t l = f2_pack(kLog2e, kLog2e), p = f2_mul(d, l);
  uint64_t q = f2_fma(d, l, f2_mul(p, minus));
  q = f2_fma(d, f2_pack(kLost, kLost), f2_fma(r, l, q));
  float p0, p1, d0, d1;
  f2_unpack(p, p0, p1);
  f2_unpack(d, d0, d1);
  const uint64_t e = f2_pack(exp2f(p0), exp2f(p1));
  f2_unpack(f2_fma(e, f2_mul(q, f2_pack(0.69314718f, 0.69314718f)), e), e0, e1);
  if (d0 < -200.f) e0 = 0.f;   // (q may be NaN there)
  if (d1 < -200.f) e1 = 0.f;
}
__device__ __forceinline__ float exp_below(float v, float top) {
  float e, unused;
  exp_below2(v, v, top, e, unused);
  return e;
}
// All of a lane's logits to their exponentials; returns the sum.
template <int V>
__device__ __forceinline__ float exps_below(float (&x)[V], float top, float (&e)[V]) {
  float total = 0.f;
#pragma unroll
  for (int v = 0; v < V; v += 2) {
    if (v + 1 < V) {
      exp_below2(x[v], x[v + 1], top, e[v], e[v + 1]);
      total += e[v] + e[v + 1];
    } else {
      e[v] = exp_below(x[v], top);
      total += e[v];
    }
  }
  return total;
}

// L lanes a token (32 / L tokens a warp), V logits a lane (expert v * L + lane): with eight logits a lane a
// round of the top-k is a few compares and log2 L shuffles for several tokens at once, where a whole
// warp a token spends two warp reductions on each. Each round takes the largest logit left and the lowest
// expert that has it. Bound by instructions: 39200 tokens of 64 experts, four each, take about 7 us (10 MB read);
// with their sort and the gradient 25.8 us.
template <int L>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
template <int L>
__device__ __forceinline__ int group_min(int v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v = min(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <int V>
__device__ __forceinline__ float largest(const float (&x)[V]) {
  float best = x[0];
#pragma unroll
  for (int v = 1; v < V; ++v) best = fmaxf(best, x[v]);
  return best;
}

constexpr int kRouteWarps = 4;

template <int V, int L>
__global__ void __launch_bounds__(kRouteWarps * 32)
    k_expert_route(const float* logits, int32_t* ids, float* weight, int T, int E, int topk,
                   int renorm) {
  griddep_wait();
  griddep_launch();
  const int l = threadIdx.x % L;
  const int t = blockIdx.x * (kRouteWarps * 32 / L) + threadIdx.x / L;
  const bool live = t < T;
  float x[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = v * L + l;
    x[v] = live && e < E ? open_logit(logits[(size_t)t * E + e]) : -INFINITY;
  }
  float best = group_max<L>(largest(x));
  const float top = best > -INFINITY ? best : 0.f;
  float total = 0.f, mine = 0.f;
  int my_id = -1;
  if (!renorm) {
    float e[V];
    total = group_sum<L>(exps_below(x, top, e));
  }
  for (int j = 0; j < topk; ++j) {
    if (j > 0) best = group_max<L>(largest(x));
    const bool open = best > -INFINITY;   // else every expert left is closed
    int at = 1 << 30;
#pragma unroll
    for (int v = V - 1; v >= 0; --v)
      if (x[v] == best) at = v * L + l;
    at = group_min<L>(at);
    const float ex = open ? exp_below(best, top) : 0.f;
    if (renorm) total += ex;
    if (l == j && open) {
      mine = ex;
      my_id = at;
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (v * L + l == at) x[v] = -INFINITY;
  }
  if (live && l < topk) {
    ids[(size_t)t * topk + l] = my_id;
    weight[(size_t)t * topk + l] = my_id >= 0 ? mine / total : 0.f;
  }
}

// Gradient of the weights for the logits. Renormalised: w is the softmax of the chosen logits, so
// dlogit_j = w_j (dw_j - sum_i dw_i w_i) there and zero elsewhere. Otherwise w_j = p[id_j] of the
// softmax p over all open experts: dlogit_e = p_e (dw_e - sum_i dw_i w_i), dw_e = 0 if not chosen.
template <int V, int L>
__global__ void __launch_bounds__(kRouteWarps * 32)
    k_expert_route_backward(const float* logits, const int32_t* ids, const float* weight,
                            const float* dweight, float* dlogits, int T, int E, int topk,
                            int renorm, int* status) {
  griddep_wait();
  griddep_launch();
  const int l = threadIdx.x % L;
  const int t = blockIdx.x * (kRouteWarps * 32 / L) + threadIdx.x / L;
  const bool live = t < T;
  int id = -1;
  float w = 0.f, dw = 0.f;
  if (live && l < topk) {
    id = ids[(size_t)t * topk + l];
    if (id < -1 || id >= E) {
      record_bad_index(status);
      id = -1;
    }
    if (id >= 0) {
      w = weight[(size_t)t * topk + l];
      dw = dweight[(size_t)t * topk + l];
    }
  }
  float d[V];
#pragma unroll
  for (int v = 0; v < V; ++v) d[v] = 0.f;
  const float mean = group_sum<L>(w * dw);
  if (!renorm) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = v * L + l;
      d[v] = live && e < E ? open_logit(logits[(size_t)t * E + e]) : -INFINITY;
    }
    const float best = group_max<L>(largest(d)), top = best > -INFINITY ? best : 0.f;
    const float total = group_sum<L>(exps_below(d, top, d));
    const float k = total == 0.f ? 0.f : -mean / total;   // (0: every expert is closed)
#pragma unroll
    for (int v = 0; v < V; ++v) d[v] *= k;
    if (total != total) {
      // A logit of +inf: the softmax is NaN, and so is every open expert's gradient, a closed one's 0.
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int e = v * L + l;
        d[v] = live && e < E && open_logit(logits[(size_t)t * E + e]) > -INFINITY ? total : 0.f;
      }
    }
  }
  const float add = renorm ? w * (dw - mean) : w * dw;
  for (int j = 0; j < topk; ++j) {
    const int e = __shfl_sync(0xffffffffu, id, j, L);
    const float a = __shfl_sync(0xffffffffu, add, j, L);
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (v * L + l == e) d[v] += a;
  }
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (live && v * L + l < E) dlogits[(size_t)t * E + v * L + l] = d[v];
}

// The lanes a token takes: at least topk (each writes one expert), and no more than eight logits a lane
// until a warp is full.
template <class F>
static cudaError_t by_experts(int E, int topk, F&& go) {
  using std::integral_constant;
  int L = 4;
  while (L < 32 && (L < topk || L * 8 < E)) L *= 2;
  const int v = (E + L - 1) / L;
  auto with = [&](auto l) {
    if (v <= 1) return go(integral_constant<int, 1>{}, l);
    if (v <= 2) return go(integral_constant<int, 2>{}, l);
    if (v <= 4) return go(integral_constant<int, 4>{}, l);
    if (v <= 8) return go(integral_constant<int, 8>{}, l);
    return go(integral_constant<int, 16>{}, integral_constant<int, 32>{});
  };
  if (L == 4) return with(integral_constant<int, 4>{});
  if (L == 8) return with(integral_constant<int, 8>{});
  if (L == 16) return with(integral_constant<int, 16>{});
  return with(integral_constant<int, 32>{});
}
static dim3 route_grid(int T, int L) {
  const int per = kRouteWarps * 32 / L;
  return dim3((T + per - 1) / per);
}

cudaError_t launch_expert_route(const float* logits, int32_t* ids, float* weight, int T, int E,
                                int topk, bool renorm, cudaStream_t st) {
  return by_experts(E, topk, [&](auto v, auto l) {
    return launch_pdl(k_expert_route<decltype(v)::value, decltype(l)::value>,
                      route_grid(T, decltype(l)::value), dim3(kRouteWarps * 32), 0, st, logits, ids,
                      weight, T, E, topk, renorm ? 1 : 0);
  });
}

cudaError_t launch_expert_route_backward(const float* logits, const int32_t* ids,
                                         const float* weight, const float* dweight, float* dlogits,
                                         int T, int E, int topk, bool renorm, int* status,
                                         cudaStream_t st) {
  return by_experts(E, topk, [&](auto v, auto l) {
    return launch_pdl(k_expert_route_backward<decltype(v)::value, decltype(l)::value>,
                      route_grid(T, decltype(l)::value), dim3(kRouteWarps * 32), 0, st, logits, ids,
                      weight, dweight, dlogits, T, E, topk, renorm ? 1 : 0, status);
  });
}

// ---- sort -----------------------------------------------------------------------------------
// A stable counting sort. Each of the CTAs owns a contiguous chunk of the assignments, each of its
// 16 warps a contiguous part of that, walked 32 at a time: __match_any_sync groups the lanes of one
// expert, whose order in the group is their order in the sort. With more than one CTA a first
// launch counts each CTA's experts; the placing launch then adds up the CTAs before its own.
constexpr int kSortWarps = 16;
constexpr int kSortThreads = kSortWarps * 32;

// Calls f(a, expert) for every 32 assignments of [a0, a1) in order, by this warp (lane's assignment a, -1 past
// the end), the ids of four steps loaded together.
template <class F>
__device__ __forceinline__ void sort_walk(const int32_t* ids, int a0, int a1, int E, int* status,
                                          F&& f) {
  const int lane = threadIdx.x & 31;
  for (int a = a0 + lane; a - lane < a1; a += 128) {
    int e[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) e[i] = a + 32 * i < a1 ? ids[a + 32 * i] : -1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (a - lane + 32 * i >= a1) break;
      if (e[i] < -1 || e[i] >= E) {   // routed nowhere, and recorded
        record_bad_index(status);
        e[i] = -1;
      }
      f(a + 32 * i, e[i]);
    }
  }
}

// counts[e] += the experts of [a0, a1), by this warp.
__device__ __forceinline__ void sort_count(const int32_t* ids, int a0, int a1, int E, int* counts,
                                           int* status) {
  const int lane = threadIdx.x & 31;
  sort_walk(ids, a0, a1, E, status, [&](int, int e) {
    const uint32_t same = __match_any_sync(0xffffffffu, e);
    if (e >= 0 && (same & ((1u << lane) - 1)) == 0) counts[e] += __popc(same);
    __syncwarp();
  });
}

__global__ void __launch_bounds__(kSortThreads) k_expert_count(const int32_t* ids, int32_t* hist,
                                                               int n, int chunk, int E,
                                                               int* status) {
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
    k_expert_place(const int32_t* ids, const int32_t* hist, int32_t* order, int32_t* slot,
                   int32_t* offsets, int n, int chunk, int E, int* status) {
  extern __shared__ int counts[];   // [warps][E]: counts, then the next place of each expert
  __shared__ int2 s_part[kSortThreads];
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
  // Thread e (E <= the CTA's threads): its expert's total over all CTAs and over those before. The CTAs'
  // counts are read by all threads, `parts` of them an expert, so that few loads follow one another.
  int total = 0, before = 0;
  const int e = threadIdx.x;
  if (gridDim.x == 1) {
    if (e < E)
      for (int w = 0; w < kSortWarps; ++w) total += counts[w * E + e];
  } else {
    const int parts = kSortThreads / E, part_of = threadIdx.x / E, ex = threadIdx.x % E;
    int sum = 0, sum_before = 0;
    if (part_of < parts) {
#pragma unroll 16
      for (int b = part_of; b < gridDim.x; b += parts) {
        const int h = hist[(size_t)b * E + ex];
        sum += h;
        sum_before += b < blockIdx.x ? h : 0;
      }
    }
    s_part[threadIdx.x] = make_int2(sum, sum_before);
    __syncthreads();
    if (e < E)
      for (int q = 0; q < parts; ++q) {
        const int2 v = s_part[q * E + e];
        total += v.x;
        before += v.y;
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
  sort_walk(ids, a0, a1, E, status, [&](int a, int ex) {
    const uint32_t same = __match_any_sync(0xffffffffu, ex);
    const uint32_t lower = same & ((1u << lane) - 1);
    const int at = ex >= 0 ? next[ex] + __popc(lower) : -1;
    __syncwarp();
    if (ex >= 0 && lower == 0) next[ex] += __popc(same);
    __syncwarp();
    if (a < a1) {
      if (slot) slot[a] = at;
      if (order && at >= 0) order[at] = a;
      // places past the routed assignments hold none
      if (order && a >= s_total) order[a] = -1;
    }
  });
}

// The sort's CTAs and the assignments of each, a whole number of steps of all its warps: one CTA up to
// kSortOne assignments (a second launch costs more than the steps), else as few steps as kSortMaxCtas allow.
static int sort_chunk(long long n) {
  if (n <= kSortOne) return (int)n;
  const long long step = kSortThreads;
  return (int)((n + step * kSortMaxCtas - 1) / (step * kSortMaxCtas) * step);
}
int sort_ctas(long long n) {
  return n <= kSortOne ? 1 : (int)((n + sort_chunk(n) - 1) / sort_chunk(n));
}

cudaError_t launch_expert_count(const int32_t* ids, int32_t* hist, int n, int E, int* status,
                                cudaStream_t st) {
  const int ctas = sort_ctas(n), chunk = sort_chunk(n);
  return launch_pdl(k_expert_count, dim3(ctas), dim3(kSortThreads),
                    (size_t)kSortWarps * E * sizeof(int), st, ids, hist, n, chunk, E, status);
}

cudaError_t launch_expert_place(const int32_t* ids, const int32_t* hist, int32_t* order,
                                int32_t* slot, int32_t* offsets, int n, int E, int* status,
                                cudaStream_t st) {
  const int ctas = sort_ctas(n), chunk = sort_chunk(n);
  return launch_pdl(k_expert_place, dim3(ctas), dim3(kSortThreads),
                    (size_t)kSortWarps * E * sizeof(int), st, ids, hist, order, slot, offsets, n,
                    chunk, E, status);
}

// ---- row moves ------------------------------------------------------------------------------
// The sorted place of assignment a, or -1 (none; one outside [-1, n) is recorded and skipped).
__device__ __forceinline__ int row_slot(const int32_t* slot, long long a, int n, int* status) {
  const int p = slot[a];
  if (p < -1 || p >= n) {
    record_bad_index(status);
    return -1;
  }
  return p;
}

// xs[slot[t, j]] = x[t]: the token's row is loaded once, up to eight chunks a lane in flight.
template <class T>
__global__ void __launch_bounds__(256)
    k_expert_gather(const typename T::Store* x, const int32_t* slot, typename T::Store* xs,
                    int tokens, int topk, int C, long long ld, int* status) {
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
// residual. A warp takes 32 U chunks of a token (`parts` warps a token) with all of its rows' loads in
// flight together, and has the next token's slots and weights on their way meanwhile, so that each
// token waits for memory once. K: topk where it is at most 4 (every row's raw words are held until
// they are added, chunk by chunk), else 0 (four experts at a time into running sums).
// CTAs an SM: 16384 tokens of two 1280 bf16 rows take 30.2, 24.3, 22.3 us with 2, 3, 4; 9000 of two 1024 fp32 rows
// 21.1, 19.3, 23.4, of four 37.3, 33.1, 34.2 (registers).
constexpr int kCombineCtas = 3;

template <class T, int U, int K>
__global__ void __launch_bounds__(256, kCombineCtas)
    k_expert_combine(const typename T::Store* ys, const int32_t* slot, const float* weight,
                     const typename T::Store* residual, typename T::Store* out, int tokens,
                     int topk, int C, long long ld, int parts, int* status) {
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31;
  // Item (token t, part): the warps take every (8 grid)-th, stepped without a division.
  const int warps = gridDim.x * 8, step_t = warps / parts, step_part = warps % parts;
  const int chunks = C / 8;
  if (K > 0) topk = K;
  auto lookup = [&](int t, int& p, float& w) {
    p = -1;
    w = 0.f;
    if (t < tokens && lane < topk) {
      const long long a = (long long)t * topk + lane;
      p = row_slot(slot, a, tokens * topk, status);
      w = weight ? weight[a] : 1.f;
    }
  };
  const int item = blockIdx.x * 8 + (threadIdx.x >> 5);
  int t = item / parts, part = item % parts;
  int my;
  float my_w;
  lookup(t, my, my_w);
  while (t < tokens) {
    const int c0 = part * 32 * U + lane;
    int next_t = t + step_t, next_part = part + step_part;
    if (next_part >= parts) {
      next_part -= parts;
      ++next_t;
    }
    int next;
    float next_w;
    Chunk<T> res[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      chunk_zero(res[i]);
      if (residual && c0 + 32 * i < chunks)
        chunk_load(res[i], residual + (size_t)t * ld + (c0 + 32 * i) * 8);
    }
    constexpr int kJ = K > 0 ? K : 4;   // experts whose rows are in flight together
    Chunk<T> y[kJ][U];
    int p[kJ];
    auto load = [&](int j0) {
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
        p[j] = __shfl_sync(0xffffffffu, my, (j0 + j) & 31);
        if (j0 + j >= topk) p[j] = -1;
        if (p[j] < 0) continue;
#pragma unroll
        for (int i = 0; i < U; ++i)
          if (c0 + 32 * i < chunks) chunk_load(y[j][i], ys + (size_t)p[j] * C + (c0 + 32 * i) * 8);
      }
    };
    auto add = [&](int j0, int i, float (&acc)[8]) {
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
        const float w = __shfl_sync(0xffffffffu, my_w, (j0 + j) & 31);
        if (p[j] < 0) continue;
        float f[8];
        chunk_floats(y[j][i], f);
#pragma unroll
        for (int q = 0; q < 8; ++q) acc[q] += w * f[q];
      }
    };
    auto finish = [&](int i, float (&acc)[8]) {
      if (c0 + 32 * i >= chunks) return;
      float r[8];
      chunk_floats(res[i], r);
#pragma unroll
      for (int q = 0; q < 8; ++q) acc[q] += r[q];
      Chunk<T> o;
      chunk_round(o, acc);
      chunk_store(out + (size_t)t * ld + (c0 + 32 * i) * 8, o);
    };
    if constexpr (K > 0) {
      load(0);
      lookup(next_t, next, next_w);
#pragma unroll
      for (int i = 0; i < U; ++i) {
        float acc[8] = {};
        add(0, i, acc);
        finish(i, acc);
      }
    } else {
      float acc[U][8] = {};
      for (int j0 = 0; j0 < topk; j0 += kJ) {
        load(j0);
        if (j0 == 0) lookup(next_t, next, next_w);
#pragma unroll
        for (int i = 0; i < U; ++i) add(j0, i, acc[i]);
      }
#pragma unroll
      for (int i = 0; i < U; ++i) finish(i, acc[i]);
    }
    t = next_t;
    part = next_part;
    my = next;
    my_w = next_w;
  }
}

// The same over fp32 partials [splits][tokens * topk][C] of fc2's k-splits, added in split order; one chunk a lane.
__global__ void __launch_bounds__(256)
    k_expert_combine_splits(const float* ys, const int32_t* slot, const float* weight,
                            const uint16_t* residual, uint16_t* out, int tokens, int topk, int C,
                            long long ld, int parts, int splits, int* status) {
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31;
  const long long item = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int t = (int)(item / parts), c = ((int)(item % parts) * 32 + lane) * 8;
  if (t >= tokens) return;
  int my = -1;
  float my_w = 0.f;
  if (lane < topk) {
    my = row_slot(slot, (long long)t * topk + lane, tokens * topk, status);
    my_w = weight ? weight[(size_t)t * topk + lane] : 1.f;
  }
  float acc[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) acc[q] = 0.f;
  const long long step = (long long)tokens * topk * C;
  for (int j = 0; j < topk; ++j) {
    const int p = __shfl_sync(0xffffffffu, my, j);
    const float w = __shfl_sync(0xffffffffu, my_w, j);
    if (p < 0 || c >= C) continue;
    float f[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) f[q] = 0.f;
#pragma unroll 4
    for (int s = 0; s < splits; ++s) {
      Chunk<F32> v;
      float g[8];
      chunk_load(v, ys + s * step + (size_t)p * C + c);
      chunk_floats(v, g);
#pragma unroll
      for (int q = 0; q < 8; ++q) f[q] += g[q];
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[q] += w * f[q];
  }
  if (c >= C) return;
  Chunk<Bf16> o;
  if (residual) {
    float r[8];
    chunk_load(o, residual + (size_t)t * ld + c);
    chunk_floats(o, r);
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[q] += r[q];
  }
  chunk_round(o, acc);
  chunk_store(out + (size_t)t * ld + c, o);
}

cudaError_t launch_expert_combine(const void* ys, const int32_t* slot, const float* weight,
                                  const void* residual, void* out, int tokens, int topk, int C,
                                  long long ld, int dtype, int splits, int* status,
                                  cudaStream_t st) {
  const int chunks = C / 8;
  auto grid = [&](int parts) {
    return dim3((unsigned)(((long long)tokens * parts + 7) / 8));
  };
  if (splits > 0) {
    const int parts = (chunks + 31) / 32;
    return launch_pdl(k_expert_combine_splits, grid(parts), dim3(256), 0, st,
                      static_cast<const float*>(ys), slot, weight,
                      static_cast<const uint16_t*>(residual), static_cast<uint16_t*>(out), tokens,
                      topk, C, ld, parts, splits, status);
  }
  return by_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    using S = typename T::Store;
    auto go = [&](auto u, auto k) {
      constexpr int U = decltype(u)::value, K = decltype(k)::value;
      const int parts = (chunks + 32 * U - 1) / (32 * U);
      const int ctas = (int)std::min<long long>(((long long)tokens * parts + 7) / 8,
                                                kCombineCtas * kRowCtas);
      return launch_pdl(k_expert_combine<T, U, K>, dim3(ctas), dim3(256), 0, st,
                        static_cast<const S*>(ys), slot, weight, static_cast<const S*>(residual),
                        static_cast<S*>(out), tokens, topk, C, ld, parts, status);
    };
    using std::integral_constant;
    // As few warps a token as hold its rows' words in registers, its chunks spread evenly; one chunk a
    // lane where there are few tokens.
    auto with = [&](auto k, auto most) {
      constexpr int kMost = decltype(most)::value;
      const int lanes = (chunks + 31) / 32, parts = (lanes + kMost - 1) / kMost;
      const bool few = (long long)tokens * lanes <= 8 * kCombineCtas * kRowCtas;
      const int u = few ? 1 : (lanes + parts - 1) / parts;
      if (u == 1) return go(integral_constant<int, 1>{}, k);
      if (u == 2) return go(integral_constant<int, kMost < 2 ? 1 : 2>{}, k);
      if (u == 3) return go(integral_constant<int, kMost < 3 ? 1 : 3>{}, k);
      if (u == 4) return go(integral_constant<int, kMost < 4 ? 1 : 4>{}, k);
      return go(integral_constant<int, kMost < 5 ? 1 : 5>{}, k);
    };
    constexpr bool kWide = T::kWords == 8;
    switch (topk) {
      case 1: return with(integral_constant<int, 1>{}, integral_constant<int, kWide ? 3 : 5>{});
      case 2: return with(integral_constant<int, 2>{}, integral_constant<int, kWide ? 2 : 4>{});
      case 3: return with(integral_constant<int, 3>{}, integral_constant<int, kWide ? 1 : 3>{});
      case 4: return with(integral_constant<int, 4>{}, integral_constant<int, kWide ? 1 : 2>{});
      default: return with(integral_constant<int, 0>{}, integral_constant<int, 1>{});
    }
  });
}

// The combine's gradient: dys[slot[t, j]] = weight[t, j] * dout[t] (rounded once) and
// dweight[t, j] = dout[t] . ys[slot[t, j]]. One warp a token, which the dot products need; two experts and
// U chunks a lane at a time, all their loads in flight together.
template <class T, int U>
__global__ void __launch_bounds__(256)
    k_expert_combine_backward(const typename T::Store* dout, const typename T::Store* ys,
                              const int32_t* slot, const float* weight, typename T::Store* dys,
                              float* dweight, int tokens, int topk, int C, long long ld,
                              int* status) {
  constexpr int K = 2;
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (t >= tokens) return;
  int my = -1;
  float my_w = 0.f;
  if (lane < topk) {
    my = row_slot(slot, (long long)t * topk + lane, tokens * topk, status);
    my_w = weight[(size_t)t * topk + lane];
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
    for (int c0 = lane; c0 < chunks; c0 += 32 * U) {
      Chunk<T> d[U], y[K][U];
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (c0 + 32 * i < chunks) chunk_load(d[i], dout + (size_t)t * ld + (c0 + 32 * i) * 8);
#pragma unroll
      for (int q = 0; q < K; ++q)
#pragma unroll
        for (int i = 0; i < U; ++i)
          if (p[q] >= 0 && c0 + 32 * i < chunks)
            chunk_load(y[q][i], ys + (size_t)p[q] * C + (c0 + 32 * i) * 8);
#pragma unroll
      for (int i = 0; i < U; ++i) {
        if (c0 + 32 * i >= chunks) continue;
        float df[8];
        chunk_floats(d[i], df);
#pragma unroll
        for (int q = 0; q < K; ++q) {
          if (p[q] < 0) continue;
          float yf[8];
          chunk_floats(y[q][i], yf);
#pragma unroll
          for (int e = 0; e < 8; ++e) dot[q] += df[e] * yf[e];
#pragma unroll
          for (int e = 0; e < 8; ++e) yf[e] = w[q] * df[e];
          Chunk<T> o;
          chunk_round(o, yf);
          chunk_store(dys + (size_t)p[q] * C + (c0 + 32 * i) * 8, o);
        }
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
    constexpr int U = T::kWords == 8 ? 2 : 4;
    return launch_pdl(k_expert_combine_backward<T, U>, dim3((tokens + 7) / 8), dim3(256), 0, st,
                      static_cast<const S*>(dout), static_cast<const S*>(ys), slot, weight,
                      static_cast<S*>(dys), dweight, tokens, topk, C, ld, status);
  });
}

}  // namespace ss

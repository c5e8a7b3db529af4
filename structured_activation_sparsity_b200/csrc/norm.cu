// The norms after one block and before the next, fused with the block's gate, residual scale and
// residual add (sandwich norms, LayerScale and per-image gates of ViT blocks), and their gradients.
//
//   p     = post norm of y                      (or y itself)
//   x_out = x + gate[group] * scale * p         (rounded once to the rows' type)
//   n     = pre norm of x_out as stored         (what the next block reads)
//
// Every row is read and written once, all sums stay in fp32. Measured on B200 (HBM floor at the measured
// copy rate in brackets): forward, 16384 rows of 1280 bf16 with everything on, 30.8 us (26.0); gradients,
// 32768 rows of 1024 bf16, 79 us (62.4), 4039 rows of 1160 fp32, 35 us (17.4). What keeps them from the floor is
// the latency of the rows' sums and shared memory's bandwidth, not HBM.
#include <type_traits>

#include "kernels.h"
#include "rows.cuh"

namespace ss {

// ---- pairs ------------------------------------------------------------------------------------
// Eight fp32 channels as four packed pairs: the arithmetic below runs two channels an instruction.
struct F8 {
  uint64_t p[4];
};
__device__ __forceinline__ uint64_t f2_same(float a) { return f2_pack(a, a); }
__device__ __forceinline__ void f8_fill(F8& f, float a) {
#pragma unroll
  for (int i = 0; i < 4; ++i) f.p[i] = f2_same(a);
}
template <class T>
__device__ __forceinline__ void f8_unpack(const Chunk<T>& c, F8& f) {
  float v[8];
  chunk_floats(c, v);
#pragma unroll
  for (int i = 0; i < 4; ++i) f.p[i] = f2_pack(v[2 * i], v[2 * i + 1]);
}
template <class T>
__device__ __forceinline__ void f8_store(typename T::Store* ptr, const F8& f) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) f2_unpack(f.p[i], v[2 * i], v[2 * i + 1]);
  Chunk<T> c;
  chunk_round(c, v);
  chunk_store(ptr, c);
}
// Rounds f to the element type, stores it and keeps the stored values.
template <class T>
__device__ __forceinline__ void f8_round(F8& f, typename T::Store* ptr) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) f2_unpack(f.p[i], v[2 * i], v[2 * i + 1]);
  Chunk<T> c;
  chunk_round(c, v);
  chunk_store(ptr, c);
  f8_unpack(c, f);
}
// To and from a vector of C fp32 in shared memory, channels c .. c + 7: the chunks' first halves lie side
// by side, then their second halves, so that the lanes of a warp read 16 bytes next to each other
// (eight consecutive floats a lane would meet in the banks: 45.8 instead of 39.5 us for the ViT-H batch).
__device__ __forceinline__ void f8_put(float* to, int C, int c, const F8& f) {
  *reinterpret_cast<ulonglong2*>(to + c / 2) = make_ulonglong2(f.p[0], f.p[1]);
  *reinterpret_cast<ulonglong2*>(to + C / 2 + c / 2) = make_ulonglong2(f.p[2], f.p[3]);
}
__device__ __forceinline__ void f8_get(F8& f, const float* from, int C, int c) {
  const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(from + c / 2);
  const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(from + C / 2 + c / 2);
  f.p[0] = a.x;
  f.p[1] = a.y;
  f.p[2] = b.x;
  f.p[3] = b.y;
}
__device__ __forceinline__ float f2_sum(uint64_t p) {
  float a, b;
  f2_unpack(p, a, b);
  return a + b;
}
// The four pairs' sum.
__device__ __forceinline__ float f8_sum(const F8& f) {
  return f2_sum(f2_add(f2_add(f.p[0], f.p[1]), f2_add(f.p[2], f.p[3])));
}

// ---- forward --------------------------------------------------------------------------------
// A norm's mean and 1/sqrt over a row that `wpr` warps hold, V chunks a lane, n_w channels in warp w.
// (held = n_w of this warp). Each warp takes its sum and its sum of squared deviations
// from its own mean; those are joined by
//   M2 = sum_w M2_w + n_w (mean_w - mean)^2
// (Chan, Golub and LeVeque's update), so no large mean cancels and one meeting of the warps is enough.
// The means are divisions, not products with 1 / n: a constant row whose sum is exact has exactly its
// value as the mean, and no deviations that 1 / sqrt(eps) would make large.
// LPR lanes share a row (fewer than 32: several rows a warp). chunk(e): whether chunk e is in the row (the
// others hold zeros); red: one float2 a warp of the row; meet(): the row's warps wait for one another.
__device__ __forceinline__ float row_held(int C, int w, int V) {   // n_w: a span of V * 256 channels
  const int left = C - w * V * 256;
  return (float)(left > V * 256 ? V * 256 : left > 0 ? left : 0);
}
template <int V, int LPR, class Live, class Meet>
__device__ __forceinline__ void row_moments(const F8 (&v)[V], Live&& chunk, int C, int wpr, int wr,
                                            float held, bool center, float eps, float2* red,
                                            Meet&& meet, float& mean, float& rstd) {
  const float n_c = (float)C, inv_c = 1.0f / n_c;
  float s = 0.f, m2 = 0.f;
  mean = 0.f;
  if (center) {
#pragma unroll
    for (int e = 0; e < V; ++e) s += f8_sum(v[e]);
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (held > 0.f) mean = s / held;
  }
  const uint64_t off = f2_same(-mean);
#pragma unroll
  for (int e = 0; e < V; ++e) {
    F8 d;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      d.p[q] = f2_add(v[e].p[q], off);
      d.p[q] = f2_mul(d.p[q], d.p[q]);
    }
    if (chunk(e)) m2 += f8_sum(d);
  }
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) m2 += __shfl_xor_sync(0xffffffffu, m2, o);
  if (wpr > 1) {
    if ((threadIdx.x & 31) == 0) red[wr] = make_float2(s, m2);
    meet();
    s = m2 = 0.f;
    for (int w = 0; w < wpr; ++w) {
      const float2 r = red[w];
      s += r.x;
      m2 += r.y;
    }
    if (center) {
      mean = s / n_c;
      for (int w = 0; w < wpr; ++w) {
        const float n = row_held(C, w, V);
        const float d = n > 0.f ? red[w].x / n - mean : 0.f;
        m2 += n * d * d;
      }
    }
  }
  rstd = rsqrtf(m2 * inv_c + eps);
}

// The norm of one chunk, (v - mean) rstd w + b, the same in both kernels. (The mean goes first: v rstd - mean
// rstd is one instruction less, but rounds at the size of mean rstd, which a constant row of 1000 and
// an eps of 1e-6 make 1e6.)
__device__ __forceinline__ void apply_norm(F8& v, float mean, float rstd, const F8& w, const F8& b) {
  const uint64_t m = f2_same(-mean), r = f2_same(rstd);
#pragma unroll
  for (int q = 0; q < 4; ++q)
    v.p[q] = f2_fma(f2_mul(f2_add(v.p[q], m), r), w.p[q], b.p[q]);
}
template <class T>
__device__ __forceinline__ void load_f8(F8& f, const void* ptr, long long at, float none) {
  if (!ptr) {
    f8_fill(f, none);
    return;
  }
  Chunk<T> c;
  chunk_load(c, static_cast<const typename T::Store*>(ptr) + at);
  f8_unpack(c, f);
}
// The gate row of a row (both fit 32 bits: a 64-bit division would be a tenth of the row's instructions).
__device__ __forceinline__ long long gate_row(const NormParams& p, long long row) {
  return (uint32_t)row / (uint32_t)p.rows_per_gate;
}
// The post norm's parameters times the residual scale.
template <class T>
__device__ __forceinline__ void load_scaled(F8& w, F8& b, const NormParams& p, int c) {
  F8 k;
  load_f8<T>(k, p.scale, c, 1.f);
  load_f8<T>(w, p.post_w, c, 1.f);
  load_f8<T>(b, p.post_b, c, 0.f);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    w.p[q] = f2_mul(w.p[q], k.p[q]);
    b.p[q] = f2_mul(b.p[q], k.p[q]);
  }
}

// Few rows: `wpr` warps a row, one chunk of eight channels a thread, everything loaded at once. What
// counts is one trip to memory and the two row sums.
template <class T>
__global__ void __launch_bounds__(512) k_norm_residual_direct(const NormParams p, int wpr) {
  __shared__ float2 red[2][16];
  using S = typename T::Store;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wr = warp % wpr;
  const int c = (wr * 32 + lane) * 8;
  const bool col = c < p.C;
  const long long row = blockIdx.x * (long long)(blockDim.x / 32 / wpr) + warp / wpr;
  const bool live = col && row < p.rows;
  griddep_wait();
  griddep_launch();
  F8 v[1], x, gate, post_w, post_b, pre_w, pre_b;
  f8_fill(v[0], 0.f);
  f8_fill(x, 0.f);
  if (live) {
    Chunk<T> yr, xr;   // (plain loads: the outputs may be these rows)
    chunk_load(yr, static_cast<const S*>(p.y) + row * p.ld_y + c);
    chunk_load(xr, static_cast<const S*>(p.x) + row * p.ld_x + c);
    f8_unpack(yr, v[0]);
    f8_unpack(xr, x);
    load_f8<T>(gate, p.gate, p.gate ? gate_row(p, row) * p.C + c : 0, 1.f);
    load_f8<T>(pre_w, p.pre_w, c, 1.f);
    load_f8<T>(pre_b, p.pre_b, c, 0.f);
    load_scaled<T>(post_w, post_b, p, c);   // (last: its products wait for their loads)
  }
  float4 st = make_float4(0.f, 0.f, 0.f, 0.f);
  const float held = row_held(p.C, wr, 1);
  auto in_row = [&](int) { return col; };
  auto meet = [&] { __syncthreads(); };   // the block's rows share its barriers
  if (p.post_w)
    row_moments<1, 32>(v, in_row, p.C, wpr, wr, held, p.center, p.eps, red[0] + warp - wr, meet, st.x,
                       st.y);
  if (live) {
    apply_norm(v[0], st.x, p.post_w ? st.y : 1.f, post_w, post_b);
#pragma unroll
    for (int q = 0; q < 4; ++q) v[0].p[q] = f2_fma(v[0].p[q], gate.p[q], x.p[q]);
    f8_round<T>(v[0], static_cast<S*>(p.x_out) + row * p.ld_x + c);
  }
  if (p.pre_w) {
    if (!live) f8_fill(v[0], 0.f);
    row_moments<1, 32>(v, in_row, p.C, wpr, wr, held, p.center, p.eps, red[1] + warp - wr, meet, st.z,
                       st.w);
    if (live) {
      apply_norm(v[0], st.z, st.w, pre_w, pre_b);
      f8_store<T>(static_cast<S*>(p.n) + row * p.ld_n + c, v[0]);
    }
  }
  if (p.stats && live && c == 0) reinterpret_cast<float4*>(p.stats)[row] = st;
}

// Many rows: a persistent CTA of 16 warps an SM; `wpr` warps hold a row, each a span of it with V chunks
// of eight channels a lane, so that a row's sums cost a few shuffles per V chunks and nothing waits for
// another warp at wpr == 1. Every warp has a slot of shared memory for its y and one for its x, which
// bulk copies fill with the next row's as soon as this one's values are read: the memory stays busy
// without registers for it. The parameters sit in shared memory in fp32 (scale folded into the post
// norm's); the gate, which changes with the row, is read from L1. LPR < 32: narrow rows, 32 / LPR of them
// a warp. kFull: every lane's V chunks are in the row; kFullOne: and the row is one warp's, so that its
// width is known.
// 16384 rows of 1280 bf16: 38.2 us with 24 warps of 80 registers, 36.1 with the width known (which spills
// less), 32.8 with 20 warps, 30.5 with 16 (128 registers), 31.8 with 12; two rows ahead a warp 33.1 (their shared
// memory comes out of the L1 that holds the gate).
constexpr int kFwdWarps = 16, kFwdThreads = 32 * kFwdWarps;
static_assert(kFwdWarps % 4 == 0, "rows of up to four warps");

enum NormSpan { kRagged, kFull, kFullOne };

template <class T, int V, int LPR, NormSpan SPAN>
__global__ void __launch_bounds__(kFwdThreads, 1) k_norm_residual(const NormParams p, int warps,
                                                                  int* status) {
  using S = typename T::Store;
  constexpr bool FULL = SPAN != kRagged;
  const int wpr = SPAN == kFullOne ? 1 : warps, C = SPAN == kFullOne ? V * LPR * 8 : p.C;
  constexpr int kRows = 32 / LPR;                   // rows a warp holds
  constexpr int kSlot = kRows * V * LPR * 8;        // elements of a warp's y or x
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[2][kFwdWarps];
  __shared__ float2 red[2][kFwdWarps];
  __shared__ int abort_flag;
  S* slots = reinterpret_cast<S*>(smem);            // [warps][y, x][kSlot]
  float* prm = reinterpret_cast<float*>(smem + 2 * kFwdWarps * kSlot * sizeof(S));
  // prm [4][C]: scale * post_w, scale * post_b, pre_w, pre_b
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wr = warp % wpr;
  if (threadIdx.x < 2 * kFwdWarps) mbar_init(&full[0][0] + threadIdx.x, 1);
  if (threadIdx.x == 0) abort_flag = 0;
  fence_barrier_init();
  __syncthreads();
  griddep_wait();
  griddep_launch();

  const int per_cta = kFwdWarps / wpr * kRows;
  // (rows and a step past them fit 32 bits)
  const uint32_t rows = (uint32_t)p.rows, stride = gridDim.x * per_cta;
  const uint32_t first = blockIdx.x * per_cta + warp / wpr * kRows;   // of the warp
  const int c0 = wr * V * LPR * 8;                  // first channel of the warp's span
  const int span = FULL || C - c0 > V * LPR * 8 ? V * LPR * 8 : C > c0 ? C - c0 : 0;
  S* slot_y = slots + (size_t)warp * 2 * kSlot;
  S* slot_x = slot_y + kSlot;
  // The warp's span of its rows from `row` on (rows kSlot / kRows apart in the slot).
  auto fetch = [&](S* to, const void* src, long long ld, uint32_t row, uint64_t* bar) {
    const int n = rows - row < kRows ? (int)(rows - row) : kRows;
    mbar_expect_tx(bar, (uint32_t)(n * span * (int)sizeof(S)));
    if (span > 0)
      for (int i = 0; i < n; ++i)
        bulk_load(to + i * (kSlot / kRows), static_cast<const S*>(src) + (row + i) * ld + c0,
                  (uint32_t)(span * (int)sizeof(S)), bar);
  };
  if (lane == 0 && first < rows) {
    fetch(slot_y, p.y, p.ld_y, first, &full[0][warp]);
    fetch(slot_x, p.x, p.ld_x, first, &full[1][warp]);
  }
  for (int c = threadIdx.x * 8; c < C; c += kFwdThreads * 8) {
    F8 a, b;
    load_scaled<T>(a, b, p, c);
    f8_put(prm, C, c, a);
    f8_put(prm + C, C, c, b);
    load_f8<T>(a, p.pre_w, c, 1.f);
    load_f8<T>(b, p.pre_b, c, 0.f);
    f8_put(prm + 2 * C, C, c, a);
    f8_put(prm + 3 * C, C, c, b);
  }
  __syncthreads();
  const int l = lane % LPR, sub = lane / LPR;
  const int mine = sub * (kSlot / kRows) + l * 8;    // in a slot; chunk e is LPR * 8 further on
  const int cl = c0 + l * 8;                        // the lane's first channel
  const float held = (float)span;
  auto in_row = [&](int e) { return FULL || l * 8 + e * LPR * 8 < span; };
  auto meet = [&] { named_barrier(1 + warp / wpr, wpr * 32); };
  // Once a wait gave up (recorded), the lane waits no more and lane 0 asks for no more rows; the walk goes on to
  // its end, so that no barrier is left with missing threads (the addresses do not depend on the data),
  // and lane 0 then waits for the copies still in flight. Bit 0 of state is the row's parity; bit 1 says that a
  // wait gave up, bits 2 and 3 then hold the parities of the slots' last copies.
  int state = 0;
  for (uint32_t at = first; at < rows; at += stride, state ^= 1) {
    const uint32_t row = at + sub;
    const bool live = LPR == 32 || row < rows;
    F8 v[V];
    if (state < 2 && !mbar_wait(&full[0][warp], state, &abort_flag, status))
      state |= 2 | state << 2 | state << 3;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      f8_fill(v[e], 0.f);
      if (live && in_row(e)) {
        Chunk<T> t;
        chunk_load(t, slot_y + mine + e * LPR * 8);
        f8_unpack(t, v[e]);
      }
    }
    // The next row may come into a slot only behind the proxy fence, which orders every lane's reads before
    // the copies. (A warp barrier alone lets the copies win against a queue of reads: rows with channels
    // of the row 592 further on.)
    auto fetch_next = [&](S* to, const void* src, long long ld, uint64_t* bar) {
      if (lane == 0 && state < 2 && at + stride < rows) fetch(to, src, ld, at + stride, bar);
    };
    auto slots_read = [&] {
      fence_proxy_async_smem();
      __syncwarp();
    };
    slots_read();
    fetch_next(slot_y, p.y, p.ld_y, &full[0][warp]);
    float4 st = make_float4(0.f, 0.f, 0.f, 0.f);
    if (p.post_w)
      row_moments<V, LPR>(v, in_row, C, wpr, wr, held, p.center, p.eps, red[0] + warp - wr, meet, st.x,
                          st.y);
    const float rstd = p.post_w ? st.y : 1.f;
    const S* gate = static_cast<const S*>(p.gate);
    if (gate && live) gate += gate_row(p, row) * C;
    S* out = static_cast<S*>(p.x_out) + row * p.ld_x;
    // The gate's chunks come together ahead of the loop's stores, as far as the registers hold them. (One by
    // one between the stores, as plain loads must stay, the ViT-H batch took 37.4 us instead of 31.8, and
    // 2048 channels 54.6 instead of 47.8 in halves. With several warps a row what spills costs more:
    // six chunks a lane 101 us, two at a time 87, 16384 x 4096 bf16 128 two at a time, 119 one by one.)
    constexpr int kAhead = SPAN == kFullOne ? (V > 7 ? V / 2 : V) : V > 6 ? 1 : V > 4 ? 2 : V;
    Chunk<T> gates[kAhead];
    auto load_gates = [&](int e0) {
      if (!gate) return;
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (e0 + i < V && live && in_row(e0 + i)) chunk_load(gates[i], gate + cl + (e0 + i) * LPR * 8);
    };
    load_gates(0);
    if (state < 2 && !mbar_wait(&full[1][warp], state, &abort_flag, status))
      state |= 2 | (at + stride < rows ? state ^ 1 : state) << 2 | state << 3;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      // (one chunk's operands at a time: gathering them ahead would cost the registers)
      asm volatile("" ::: "memory");
      if (e > 0 && e % kAhead == 0) load_gates(e);
      if (!live || !in_row(e)) {
        f8_fill(v[e], 0.f);
        continue;
      }
      const int c = cl + e * LPR * 8;
      F8 w, b, x;
      Chunk<T> t;
      chunk_load(t, slot_x + mine + e * LPR * 8);
      f8_unpack(t, x);
      f8_get(w, prm, C, c);
      f8_get(b, prm + C, C, c);
      apply_norm(v[e], st.x, rstd, w, b);
      if (gate) {
        f8_unpack(gates[e % kAhead], w);
#pragma unroll
        for (int q = 0; q < 4; ++q) v[e].p[q] = f2_fma(v[e].p[q], w.p[q], x.p[q]);
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) v[e].p[q] = f2_add(v[e].p[q], x.p[q]);
      }
      f8_round<T>(v[e], out + c);
    }
    slots_read();
    fetch_next(slot_x, p.x, p.ld_x, &full[1][warp]);
    if (p.pre_w) {
      row_moments<V, LPR>(v, in_row, C, wpr, wr, held, p.center, p.eps, red[1] + warp - wr, meet, st.z,
                          st.w);
      S* nrow = static_cast<S*>(p.n) + row * p.ld_n;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        asm volatile("" ::: "memory");
        if (!live || !in_row(e)) continue;
        const int c = cl + e * LPR * 8;
        F8 w, b;
        f8_get(w, prm + 2 * C, C, c);
        f8_get(b, prm + 3 * C, C, c);
        apply_norm(v[e], st.z, st.w, w, b);
        f8_store<T>(nrow + c, v[e]);
      }
    }
    if (p.stats && live && wr == 0 && l == 0) reinterpret_cast<float4*>(p.stats)[row] = st;
    // One norm only: its next meeting must not overtake a warp that still reads this one's sums.
    if (wpr > 1 && (p.post_w == nullptr) != (p.pre_w == nullptr)) meet();
  }
  if (lane == 0 && state >= 2) {
    mbar_drain(&full[0][warp], state >> 2 & 1);
    mbar_drain(&full[1][warp], state >> 3 & 1);
  }
}

// ---- shared by the persistent backward ------------------------------------------------------
constexpr int kNormThreads = 512;
constexpr int kNormSmem = 225 * 1024;
constexpr int kNormMaxStages = 4;

struct NormShape {
  int workers, wpg, rl;     // workers in all; warps per worker; workers per CTA
  int stages, stage_bytes;  // ring of one worker
};

// Worker w's first row of `rows` shared evenly by `workers`, and the worker of row r.
__host__ __device__ inline long long first_row(long long rows, int workers, int w) {
  return rows * w / workers;
}
__host__ __device__ inline long long worker_of(long long rows, int workers, long long r) {
  return ((r + 1) * workers - 1) / rows;
}

// The workers' geometry for `tensors` rows of C channels and R rows at a time: as many workers a CTA as have
// two stages each.
static NormShape norm_shape(long long rows, int C, int es, int tensors, int R) {
  NormShape g;
  g.wpg = (C / 8 + 31) / 32;
  g.stage_bytes = R * (tensors * C * es + 16);
  const int kept = 4 * C * (int)sizeof(float);   // what a worker keeps besides its ring
  g.rl = kNormThreads / 32 / g.wpg;
  while (g.rl > 1 && g.rl * (2 * g.stage_bytes + kept) > kNormSmem) --g.rl;
  g.stages = (kNormSmem / g.rl - kept) / g.stage_bytes;
  if (g.stages > kNormMaxStages) g.stages = kNormMaxStages;
  const long long most = (long long)kNormMaxCtas * g.rl;
  g.workers = (int)(rows < most ? rows : most);
  return g;
}

template <class T, int V, int LPR>
static cudaError_t launch_fwd(const NormParams& p, int wpr, int* status, cudaStream_t st) {
  // (A row of fewer than 32 lanes has one warp.)
  const auto kernel = p.C != V * LPR * wpr * 8 ? k_norm_residual<T, V, LPR, kRagged>
                      : wpr == 1               ? k_norm_residual<T, V, LPR, kFullOne>
                                 : k_norm_residual<T, V, LPR, LPR == 32 ? kFull : kFullOne>;
  const size_t smem = (size_t)2 * kFwdWarps * V * 32 * 8 * sizeof(typename T::Store) +
                      (size_t)4 * p.C * sizeof(float);
  const cudaError_t e =
      allow_smem(reinterpret_cast<const void*>(kernel), (int)smem);
  if (e != cudaSuccess) return e;
  const int per_cta = kFwdWarps / wpr * (32 / LPR);
  const long long ctas = (p.rows + per_cta - 1) / per_cta;
  return launch_pdl(kernel, dim3((unsigned)(ctas < kNormMaxCtas ? ctas : kNormMaxCtas)),
                    dim3(kFwdThreads), smem, st, p, wpr, status);
}

cudaError_t launch_norm_residual(const NormParams& p, int dtype, int* status, cudaStream_t st) {
  return by_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    const int chunks = p.C / 8;
    int wide = 1;   // warps of a row at one chunk a lane
    while (wide * 32 < chunks) wide *= 2;
    if (p.rows * wide <= norm_direct_warps(T::kWords == 8, wide)) {
      const int wpr = wide;
      const int rpb = wpr < 4 ? 4 / wpr : 1;
      return launch_pdl(k_norm_residual_direct<T>, dim3((unsigned)((p.rows + rpb - 1) / rpb)),
                        dim3(wpr * rpb * 32), 0, st, p, wpr);
    }
    if (chunks <= 8) return launch_fwd<T, 1, 8>(p, 1, status, st);
    if (chunks <= 16) return launch_fwd<T, 1, 16>(p, 1, status, st);
    // The fewest warps a row with at most 64 values a lane (fp32: 40, for the slots' size): 16384 rows of
    // 2048 bf16 take 46.3 us with one warp a row, 59.0 with two; of 4096 fp32 229 with four, 284 with eight.
    constexpr int kMost = T::kWords == 8 ? 5 : 8;
    int wpr = 1;
    while (chunks > 32 * kMost * wpr) wpr *= 2;
    switch ((chunks + 32 * wpr - 1) / (32 * wpr)) {
      case 1: return launch_fwd<T, 1, 32>(p, wpr, status, st);
      case 2: return launch_fwd<T, 2, 32>(p, wpr, status, st);
      case 3: return launch_fwd<T, 3, 32>(p, wpr, status, st);
      case 4: return launch_fwd<T, 4, 32>(p, wpr, status, st);
      case 5: return launch_fwd<T, 5, 32>(p, wpr, status, st);
      case 6: return launch_fwd<T, kMost < 6 ? 5 : 6, 32>(p, wpr, status, st);
      case 7: return launch_fwd<T, kMost < 7 ? 5 : 7, 32>(p, wpr, status, st);
      default: return launch_fwd<T, kMost < 8 ? 5 : 8, 32>(p, wpr, status, st);
    }
  });
}

// ---- backward -------------------------------------------------------------------------------
// With h = (v - mean) * rstd of a norm and g the gradient of h, the norm's input gradient is
//   rstd * (g - mean_c(g) - h * mean_c(g h))          (RMS norm: without the mean_c(g) term),
// so a row needs two sums per norm, taken together. For D = the gradient of x_out (dx_out plus the
// pre norm's part): dx = D, dy = post norm gradient of D * gate * scale. The parameters' gradients
// follow from column sums over rows t of group b:
//   A_b = sum D * h_post,  B_b = sum D      (h_post = y without a post norm)
//   dgate_b = scale * (post_w * A_b + post_b * B_b)
//   P1 = sum_b gate_b * A_b,  P0 = sum_b gate_b * B_b:
//   dscale = post_w * P1 + post_b * P0,  dpost_w = scale * P1,  dpost_b = scale * P0
//   dpre_w = sum dn * h_pre,  dpre_b = sum dn
// so four fp32 accumulators a channel serve all six.
//
// A worker is a group of `wpg` warps (one chunk of eight channels a thread) that walks its own
// contiguous rows, R at a time (two rows share the row sums' meetings): bulk copies bring the rows of
// all inputs, with their statistics, into the worker's ring of shared-memory stages ahead of use.
// Several workers share a CTA (one per SM); at the end their column sums are added in worker order
// and written as one partial per CTA, which k_norm_reduce adds in CTA order: no atomics, the same
// result every run.
template <class T, int R, bool PRE, bool POST, bool FULL>
__global__ void __launch_bounds__(kNormThreads, 1)
    k_norm_residual_backward(const NormBwdParams p, const NormShape g, int* status) {
  using S = typename T::Store;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[16 * kNormMaxStages];
  __shared__ __align__(8) float red[2][16 * 2 * R];   // [buffer][warp][row][sum]
  __shared__ int abort_flag;
  constexpr int kTensors = PRE ? 4 : 2;
  constexpr bool kStats = PRE || POST;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rl = warp / g.wpg, wg = warp % g.wpg;
  const int tw = wg * 32 + lane, c = tw * 8;
  const int worker = blockIdx.x * g.rl + rl;
  const bool col = (FULL || c < p.C) && rl < g.rl;
  if (threadIdx.x == 0) {
    for (int i = 0; i < g.rl * g.stages; ++i) mbar_init(full + i, 1);
    abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  griddep_wait();
  griddep_launch();

  const long long r0 = worker < g.workers ? first_row(p.rows, g.workers, worker) : p.rows;
  const long long r1 = worker < g.workers ? first_row(p.rows, g.workers, worker + 1) : p.rows;
  uint8_t* ring = smem + (size_t)rl * g.stages * g.stage_bytes;
  // Behind the rings, of each worker: pre_w, coef = gate * scale * post_w (as f8_put lays them out: two
  // vectors read once a step cost less than the 16 registers, which spilled), and P1 and P0 of its
  // closed groups (with a gate).
  float* kept = reinterpret_cast<float*>(smem + (size_t)g.rl * g.stages * g.stage_bytes) +
                (size_t)rl * 4 * p.C;
  float* closed = kept + 2 * p.C + c;
  uint64_t* bar = full + rl * g.stages;
  const int row_bytes = p.C * (int)sizeof(S);
  const bool dense = p.ld_x == p.C && p.ld_y == p.C && p.ld_n == p.C;
  // Up to R rows from r into stage st: [R stats][dx_out rows][y][x_out][dn].
  auto fetch = [&](long long r, int st) {
    const int n = (int)(r1 - r < R ? r1 - r : R);
    uint8_t* to = ring + (size_t)st * g.stage_bytes;
    mbar_expect_tx(bar + st, (uint32_t)(n * (kTensors * row_bytes + (kStats ? 16 : 0))));
    if (kStats) bulk_load(to, p.stats + r * 4, (uint32_t)n * 16, bar + st);
    to += R * 16;
    auto rows = [&](const void* src, long long ld) {
      const S* from = static_cast<const S*>(src) + r * ld;
      if (dense) {
        bulk_load(to, from, (uint32_t)(n * row_bytes), bar + st);
      } else {
        for (int i = 0; i < n; ++i)
          bulk_load(to + i * row_bytes, from + i * ld, (uint32_t)row_bytes, bar + st);
      }
      to += R * row_bytes;
    };
    rows(p.dx_out, p.ld_x);
    rows(p.y, p.ld_y);
    if (PRE) {
      rows(p.x, p.ld_x);
      rows(p.dn, p.ld_n);
    }
  };
  long long ahead = r0;
  bool gave_up = false;   // a wait did (recorded): no more waits, no more rows asked for
  if (rl < g.rl && tw == 0)
    for (int s = 0; s < g.stages && ahead < r1; ++s, ahead += R) fetch(ahead, s);

  F8 acc_pw, acc_pb, acc_a, acc_b;
  f8_fill(acc_pw, 0.f);
  f8_fill(acc_pb, 0.f);
  f8_fill(acc_a, 0.f);
  f8_fill(acc_b, 0.f);
  auto load_coef = [&](long long group) {
    F8 coef, f;
    load_f8<T>(coef, p.post_w, c, 1.f);
    load_f8<T>(f, p.scale, c, 1.f);
#pragma unroll
    for (int q = 0; q < 4; ++q) coef.p[q] = f2_mul(coef.p[q], f.p[q]);
    if (p.gate) {
      load_f8<T>(f, p.gate, group * p.C + c, 1.f);
#pragma unroll
      for (int q = 0; q < 4; ++q) coef.p[q] = f2_mul(coef.p[q], f.p[q]);
    }
    f8_put(kept + p.C, p.C, c, coef);
  };
  if (col) {
    if (PRE) {
      F8 w;
      load_f8<T>(w, p.pre_w, c, 1.f);
      f8_put(kept, p.C, c, w);
    }
    if (!p.gate) load_coef(0);
    if (p.gate) {
#pragma unroll
      for (int j = 0; j < 8; ++j) closed[j] = closed[p.C + j] = 0.f;
    }
  }
  auto meet = [&] {
    if (g.wpg > 1) named_barrier(1 + rl, g.wpg * 32);
    else __syncwarp();
  };
  // (a, b) of each of N rows summed over the worker's threads: after the first exchange the two halves of a
  // warp carry one sum each (two rows: after the second, the quarters), so that N rows cost five or six
  // shuffles. The warps' sums meet in shared memory as [warp][row][sum] and are added in warp order.
  int buf = 0;
  auto worker_sums = [&](auto& a, auto& b, auto&& met) {
    constexpr int N = sizeof(a) / sizeof(float);
    const bool hi = lane & 16;
    float v;
    if constexpr (N == 1) {
      v = hi ? b[0] : a[0];
      v += __shfl_xor_sync(0xffffffffu, hi ? a[0] : b[0], 16);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    } else {
      float v0 = hi ? b[0] : a[0], v1 = hi ? b[1] : a[1];
      v0 += __shfl_xor_sync(0xffffffffu, hi ? a[0] : b[0], 16);
      v1 += __shfl_xor_sync(0xffffffffu, hi ? a[1] : b[1], 16);
      const bool second = lane & 8;
      v = second ? v1 : v0;
      v += __shfl_xor_sync(0xffffffffu, second ? v0 : v1, 8);
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    }
    // lane 16 h + 8 i holds row i's sum h
    if (g.wpg > 1) {
      float* all = &red[buf][(warp - wg) * 2 * R];
      if ((lane & (N == 1 ? 15 : 7)) == 0)
        all[wg * 2 * N + (N == 1 ? lane >> 4 : ((lane >> 2) & 2) + (lane >> 4))] = v;
      met();
#pragma unroll
      for (int i = 0; i < N; ++i) a[i] = b[i] = 0.f;
#pragma unroll 4
      for (int w = 0; w < g.wpg; ++w)
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float2 e = reinterpret_cast<const float2*>(all)[w * N + i];
          a[i] += e.x;
          b[i] += e.y;
        }
      buf ^= 1;
    } else {
      met();
#pragma unroll
      for (int i = 0; i < N; ++i) {
        a[i] = __shfl_sync(0xffffffffu, v, 8 * i);
        b[i] = __shfl_sync(0xffffffffu, v, 16 + 8 * i);
      }
    }
  };
  const float inv_c = 1.0f / (float)p.C;
  const float mean_on = p.center ? inv_c : 0.f;
  long long group = -1, group_end = p.gate ? 0 : p.rows;
  // The gate row of the finished group: final if all its rows were this worker's, else a partial in
  // the worker's first slot (its first group) or second.
  auto close_group = [&]() {
    if (group < 0 || !col) return;
    const long long g0 = group * p.rows_per_gate;
    const bool whole = g0 >= r0 && (group_end <= r1 || r1 == p.rows);
    float a[8], b[8], f[8], dg[8];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      f2_unpack(acc_a.p[q], a[2 * q], a[2 * q + 1]);
      f2_unpack(acc_b.p[q], b[2 * q], b[2 * q + 1]);
    }
    auto floats = [&](const void* ptr, long long at, float none) {
      F8 t;
      load_f8<T>(t, ptr, at, none);
#pragma unroll
      for (int q = 0; q < 4; ++q) f2_unpack(t.p[q], f[2 * q], f[2 * q + 1]);
    };
    floats(p.post_w, c, 1.f);
#pragma unroll
    for (int j = 0; j < 8; ++j) dg[j] = f[j] * a[j];
    floats(p.post_b, c, 0.f);
#pragma unroll
    for (int j = 0; j < 8; ++j) dg[j] += f[j] * b[j];
    floats(p.scale, c, 1.f);
#pragma unroll
    for (int j = 0; j < 8; ++j) dg[j] *= f[j];
    if (!whole || p.dgate) {
      float* out = whole ? p.dgate + group * p.C + c
                         : p.gate_partial + ((long long)worker * 2 + (g0 > r0 ? 1 : 0)) * p.C + c;
      reinterpret_cast<float4*>(out)[0] = make_float4(dg[0], dg[1], dg[2], dg[3]);
      reinterpret_cast<float4*>(out)[1] = make_float4(dg[4], dg[5], dg[6], dg[7]);
    }
    floats(p.gate, group * p.C + c, 1.f);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      closed[j] += f[j] * a[j];
      closed[p.C + j] += f[j] * b[j];
    }
    f8_fill(acc_a, 0.f);
    f8_fill(acc_b, 0.f);
  };
  S* dx = static_cast<S*>(p.dx) + r0 * p.ld_x + c;
  S* dy = static_cast<S*>(p.dy) + r0 * p.ld_y + c;
  // One step: N rows (N <= R), rows `at`.. of stage st; `last`: nothing of the stage is needed after it.
  auto step = [&](auto rows_n, int at, int st, bool last) {
    constexpr int N = decltype(rows_n)::value;
    const uint8_t* sp = ring + (size_t)st * g.stage_bytes;
    const float4* stat = reinterpret_cast<const float4*>(sp) + at;
    const S* rows = reinterpret_cast<const S*>(sp + R * 16) + at * p.C + c;
    const int next = R * p.C;   // from one input's rows to the next's
    auto read = [&](F8& f, int which, int i) {
      Chunk<T> t;
      if (FULL || col) chunk_load(t, rows + which * next + i * p.C);
      else chunk_zero(t);
      f8_unpack(t, f);
    };
    // The last meeting of the worker's warps also frees the stage: every thread has its chunks, its reads
    // ordered before the copies that come in their place.
    auto release = [&] {
      fence_proxy_async_smem();
      meet();
      if (last && tw == 0 && !gave_up && ahead < r1) {
        fetch(ahead, st);
        ahead += R;
      }
    };
    F8 D[N], h[N];
    float a[N], b[N], rstd[N];
    if constexpr (PRE) {
      F8 dn[N], w_pre;
      if (FULL || col) f8_get(w_pre, kept, p.C, c);
      else f8_fill(w_pre, 0.f);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        read(h[i], 2, i);
        read(dn[i], 3, i);
        const float2 t = reinterpret_cast<const float2*>(stat + i)[1];
        const uint64_t rs = f2_same(t.y), m = f2_same(-t.x);   // (the mean first: see apply_norm)
        uint64_t s1 = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          h[i].p[q] = f2_mul(f2_add(h[i].p[q], m), rs);
          acc_pw.p[q] = f2_fma(dn[i].p[q], h[i].p[q], acc_pw.p[q]);
          acc_pb.p[q] = f2_add(acc_pb.p[q], dn[i].p[q]);
          dn[i].p[q] = f2_mul(dn[i].p[q], w_pre.p[q]);
          s1 = f2_fma(dn[i].p[q], h[i].p[q], s1);
        }
        a[i] = f8_sum(dn[i]);
        b[i] = f2_sum(s1);
      }
      worker_sums(a, b, meet);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        read(D[i], 0, i);
        const float r = stat[i].w;
        const uint64_t rs = f2_same(r);
        const uint64_t k0 = f2_same(-r * (a[i] * mean_on)), k1 = f2_same(-r * (b[i] * inv_c));
#pragma unroll
        for (int q = 0; q < 4; ++q)
          D[i].p[q] = f2_add(D[i].p[q], f2_fma(dn[i].p[q], rs, f2_fma(h[i].p[q], k1, k0)));
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) read(D[i], 0, i);
    }
    F8 coef;
    if (FULL || col) f8_get(coef, kept + p.C, p.C, c);
    else f8_fill(coef, 0.f);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      // h_post (or y), the column sums and, with a post norm, the row sums.
      read(h[i], 1, i);
      if (FULL || col) f8_store<T>(dx + i * p.ld_x, D[i]);
      if constexpr (POST) {
        const float2 t = *reinterpret_cast<const float2*>(stat + i);
        rstd[i] = t.y;
        const uint64_t rs = f2_same(t.y), m = f2_same(-t.x);
#pragma unroll
        for (int q = 0; q < 4; ++q) h[i].p[q] = f2_mul(f2_add(h[i].p[q], m), rs);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        acc_a.p[q] = f2_fma(D[i].p[q], h[i].p[q], acc_a.p[q]);
        acc_b.p[q] = f2_add(acc_b.p[q], D[i].p[q]);
        D[i].p[q] = f2_mul(D[i].p[q], coef.p[q]);
      }
      if constexpr (POST) {
        uint64_t s1 = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) s1 = f2_fma(D[i].p[q], h[i].p[q], s1);
        a[i] = f8_sum(D[i]);
        b[i] = f2_sum(s1);
      }
    }
    if constexpr (POST) {
      worker_sums(a, b, release);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const uint64_t rs = f2_same(rstd[i]);
        const uint64_t k0 = f2_same(-rstd[i] * (a[i] * mean_on));
        const uint64_t k1 = f2_same(-rstd[i] * (b[i] * inv_c));
#pragma unroll
        for (int q = 0; q < 4; ++q)
          D[i].p[q] = f2_fma(D[i].p[q], rs, f2_fma(h[i].p[q], k1, k0));
      }
    }
    if constexpr (!POST) release();
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (FULL || col) f8_store<T>(dy + i * p.ld_y, D[i]);
    dx += N * p.ld_x;
    dy += N * p.ld_y;
  };
  if (rl < g.rl) {
    int st = 0, phase = 0;
    for (long long r = r0; r < r1; r += R) {
      const int n = (int)(r1 - r < R ? r1 - r : R);
      // After a wait that gives up the walk goes on to its end, so that no barrier is left with missing
      // threads (the addresses do not depend on the data).
      if (!gave_up) gave_up = !mbar_wait(bar + st, phase, &abort_flag, status);
      // Rows of one step share a gate row: a stage with a border between its rows takes a step each.
      int done = 0;
      do {
        const long long at = r + done;
        if (at >= group_end) {
          close_group();
          group = at / p.rows_per_gate;
          group_end = (group + 1) * p.rows_per_gate;
          if (col) load_coef(group);
        }
        if (R == 2 && done == 0 && n == 2 && group_end - at >= 2) {
          step(std::integral_constant<int, R>{}, 0, st, true);
          done = 2;
        } else {
          step(std::integral_constant<int, 1>{}, done, st, done + 1 == n);
          ++done;
        }
      } while (done < n);
      if (++st == g.stages) {
        st = 0;
        phase ^= 1;
      }
    }
    if (p.gate) close_group();
    if (gave_up && tw == 0) {   // the copies still in flight: of the last fetch of each stage
      const int n = (int)((ahead - r0) / R);
      for (int k = n > g.stages ? n - g.stages : 0; k < n; ++k)
        mbar_drain(bar + k % g.stages, k / g.stages & 1);
    }
  }
  // The CTA's column sums, in worker order: [pre_w, pre_b, P1, P0][C], over what the workers kept (the closed
  // groups' sums are read before they are overwritten).
  F8 p1 = acc_a, p0 = acc_b;
  if (p.gate && col) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      p1.p[q] = f2_pack(closed[2 * q], closed[2 * q + 1]);
      p0.p[q] = f2_pack(closed[p.C + 2 * q], closed[p.C + 2 * q + 1]);
    }
  }
  __syncthreads();
  float* sums = kept - (size_t)rl * 4 * p.C;
  if (col) {
    float* mine = sums + (size_t)rl * 4 * p.C + c;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      f2_unpack(acc_pw.p[q], mine[2 * q], mine[2 * q + 1]);
      f2_unpack(acc_pb.p[q], mine[p.C + 2 * q], mine[p.C + 2 * q + 1]);
      f2_unpack(p1.p[q], mine[2 * p.C + 2 * q], mine[2 * p.C + 2 * q + 1]);
      f2_unpack(p0.p[q], mine[3 * p.C + 2 * q], mine[3 * p.C + 2 * q + 1]);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 4 * p.C; i += blockDim.x) {
    float s = 0.f;
    for (int w = 0; w < g.rl; ++w) s += sums[(size_t)w * 4 * p.C + i];
    p.partial[(size_t)blockIdx.x * 4 * p.C + i] = s;
  }
}

// Adds the CTAs' partials in a fixed order and forms the parameters' gradients; a CTA owns 32 channels, its
// 16 warps every 16th partial. CTAs y == 0: the column sums. CTAs y > 0: the gate rows whose group
// several workers shared.
template <class T>
__global__ void __launch_bounds__(512) k_norm_reduce(const NormBwdParams p, const NormShape g,
                                                     int ctas) {
  __shared__ float part[4][16][32];
  griddep_wait();
  griddep_launch();
  using S = typename T::Store;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  if (blockIdx.y == 0) {
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    if (c < p.C)
#pragma unroll 4
      for (int b = warp; b < ctas; b += 16)
#pragma unroll
        for (int q = 0; q < 4; ++q) s[q] += p.partial[((size_t)b * 4 + q) * p.C + c];
#pragma unroll
    for (int q = 0; q < 4; ++q) part[q][warp][lane] = s[q];
    __syncthreads();
    if (warp != 0 || c >= p.C) return;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      s[q] = 0.f;
      for (int w = 0; w < 16; ++w) s[q] += part[q][w][lane];
    }
    auto param = [&](const void* ptr, float none) {
      if (!ptr) return none;
      const S v = static_cast<const S*>(ptr)[c];
      if constexpr (sizeof(S) == 4) {
        return (float)v;
      } else {
        float lo, hi;
        T::unpack(v, lo, hi);
        return lo;
      }
    };
    const float scale = param(p.scale, 1.f);
    if (p.dpre_w) p.dpre_w[c] = s[0];
    if (p.dpre_b) p.dpre_b[c] = s[1];
    if (p.dscale) p.dscale[c] = param(p.post_w, 1.f) * s[2] + param(p.post_b, 0.f) * s[3];
    if (p.dpost_w) p.dpost_w[c] = scale * s[2];
    if (p.dpost_b) p.dpost_b[c] = scale * s[3];
    return;
  }
  const long long groups = (p.rows + p.rows_per_gate - 1) / p.rows_per_gate;
  for (long long gr = blockIdx.y - 1; gr < groups; gr += gridDim.y - 1) {
    const long long g0 = gr * p.rows_per_gate;
    long long g1 = g0 + p.rows_per_gate;
    if (g1 > p.rows) g1 = p.rows;
    const long long w0 = worker_of(p.rows, g.workers, g0);
    const long long w1 = worker_of(p.rows, g.workers, g1 - 1);
    if (w0 == w1) continue;   // one worker's: written by it
    float s = 0.f;
    if (c < p.C)
#pragma unroll 4
      for (long long w = w0 + warp; w <= w1; w += 16)
        s += p.gate_partial[(w * 2 + (g0 > first_row(p.rows, g.workers, (int)w) ? 1 : 0)) * p.C + c];
    part[0][warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < p.C) {
      s = 0.f;
      for (int w = 0; w < 16; ++w) s += part[0][w][lane];
      p.dgate[gr * p.C + c] = s;
    }
    __syncthreads();
  }
}

// Two rows a step, or one where two rows' stages would cost more than a third of the workers.
static NormShape bwd_shape(long long rows, int C, int es, bool pre, int* R) {
  *R = 2;
  NormShape g = norm_shape(rows, C, es, pre ? 4 : 2, 2);
  if (g.stages < 2 || 3 * g.rl < 2 * (kNormThreads / 32 / g.wpg)) {
    *R = 1;
    g = norm_shape(rows, C, es, pre ? 4 : 2, 1);
  }
  return g;
}
static int norm_ctas(const NormShape& g) { return (g.workers + g.rl - 1) / g.rl; }

size_t norm_backward_partial(long long rows, int C, int es, bool pre, bool gate,
                             size_t* gate_offset) {
  int R;
  const NormShape g = bwd_shape(rows, C, es, pre, &R);
  *gate_offset = (size_t)norm_ctas(g) * 4 * C * sizeof(float);
  return *gate_offset + (gate ? (size_t)norm_ctas(g) * g.rl * 2 * C * sizeof(float) : 0);
}

template <class T, int R, bool PRE, bool POST>
static cudaError_t launch_bwd(const NormBwdParams& p, const NormShape& g, int* status,
                              cudaStream_t st) {
  const size_t smem = (size_t)g.rl * g.stages * g.stage_bytes +
                      (size_t)g.rl * 4 * p.C * sizeof(float);
  const auto kernel = p.C % 256 == 0 ? k_norm_residual_backward<T, R, PRE, POST, true>
                                     : k_norm_residual_backward<T, R, PRE, POST, false>;
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel),
                                   kNormSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(norm_ctas(g)), dim3(kNormThreads), smem, st, p, g, status);
}

cudaError_t launch_norm_backward(const NormBwdParams& p, int dtype, int* status, cudaStream_t st) {
  if (p.rows == 0) return cudaSuccess;
  return by_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    int R;
    const NormShape g = bwd_shape(p.rows, p.C, sizeof(typename T::Store), p.pre_w != nullptr, &R);
    auto go = [&](auto r) {
      constexpr int kR = decltype(r)::value;
      if (p.pre_w)
        return p.post_w ? launch_bwd<T, kR, true, true>(p, g, status, st)
                        : launch_bwd<T, kR, true, false>(p, g, status, st);
      return p.post_w ? launch_bwd<T, kR, false, true>(p, g, status, st)
                      : launch_bwd<T, kR, false, false>(p, g, status, st);
    };
    return R == 2 ? go(std::integral_constant<int, 2>{}) : go(std::integral_constant<int, 1>{});
  });
}

cudaError_t launch_norm_reduce(const NormBwdParams& p, int dtype, cudaStream_t st) {
  return by_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    int R;
    const NormShape g = bwd_shape(p.rows, p.C, sizeof(typename T::Store), p.pre_w != nullptr, &R);
    const int ctas = p.rows == 0 ? 0 : norm_ctas(g);   // sums over no rows: zeros
    long long ny = 1;
    if (p.dgate && p.rows > 0) {
      const long long groups = (p.rows + p.rows_per_gate - 1) / p.rows_per_gate;
      ny += groups < 64 ? groups : 64;
    }
    return launch_pdl(k_norm_reduce<T>, dim3((p.C + 31) / 32, (unsigned)ny), dim3(512), 0, st, p, g,
                      ctas);
  });
}

cudaError_t set_wait_limit_norm(uint64_t ns) { return set_wait_limit_here(ns); }

}  // namespace ss

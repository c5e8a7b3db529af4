// The norms after one block and before the next, fused with the block's gate, residual scale and
// residual add (sandwich norms, LayerScale and per-image gates of ViT blocks), and their gradients.
//
//   p     = post norm of y                      (or y itself)
//   x_out = x + gate[group] * scale * p         (rounded once to the rows' type)
//   n     = pre norm of x_out as stored         (what the next block reads)
//
// Both directions are bound by HBM: every row is read and written once, all sums stay in fp32.
#include "kernels.h"
#include "rows.cuh"

namespace ss {

// ---- forward --------------------------------------------------------------------------------
// `wpr` warps hold a row, V chunks of eight channels a lane (chunk (e * wpr + warp) * 32 + lane), so
// the row stays in registers from its load to the second norm. Mean, then the sum of squared
// deviations from it (two passes over registers): no cancellation at a large mean.
template <class T, int V>
__global__ void __launch_bounds__(256) k_norm_residual(const NormParams p, int wpr) {
  __shared__ float red[2][8];
  griddep_wait();
  griddep_launch();
  using S = typename T::Store;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rpb = 8 / wpr, wr = warp % wpr;
  const long long row = (long long)blockIdx.x * rpb + warp / wpr;
  const bool live = row < p.rows;
  const int chunks = p.C / 8;
  int buf = 0;
  // Sum over the row's lanes (wpr > 1: through shared memory, two buffers in turn).
  auto row_sum = [&](float s) {
    s = warp_sum(s);
    if (wpr > 1) {
      if (lane == 0) red[buf][warp] = s;
      __syncthreads();
      s = 0.f;
      for (int i = 0; i < wpr; ++i) s += red[buf][warp - wr + i];
      buf ^= 1;
    }
    return s;
  };
  float v[V][8];
  Chunk<T> xr[V];
  const S* yrow = static_cast<const S*>(p.y) + row * p.ld_y;
  const S* xrow = static_cast<const S*>(p.x) + row * p.ld_x;
  {
    Chunk<T> yr[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const int c = (e * wpr + wr) * 32 + lane;
      chunk_zero(yr[e]);
      chunk_zero(xr[e]);
      if (live && c < chunks) {
        chunk_load(yr[e], yrow + c * 8);
        chunk_load(xr[e], xrow + c * 8);
      }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) chunk_floats(yr[e], v[e]);
  }
  const float inv_c = 1.0f / (float)p.C;
  // v := (v - mean) * rstd (RMS norm: mean 0); channels past the row hold zeros before and after.
  auto normalise = [&](float& mean, float& rstd) {
    mean = 0.f;
    if (p.center) {
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < V; ++e)
#pragma unroll
        for (int j = 0; j < 8; ++j) s += v[e][j];
      mean = row_sum(s) * inv_c;
    }
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < V; ++e)
      if ((e * wpr + wr) * 32 + lane < chunks) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float d = v[e][j] - mean;
          ss += d * d;
        }
      }
    rstd = 1.0f / sqrtf(row_sum(ss) * inv_c + p.eps);
#pragma unroll
    for (int e = 0; e < V; ++e)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[e][j] = (v[e][j] - mean) * rstd;
  };
  auto params = [&](const void* ptr, long long off, int c, float (&f)[8]) {
    Chunk<T> w;
    chunk_load(w, static_cast<const S*>(ptr) + off + c * 8);
    chunk_floats(w, f);
  };
  float st[4] = {0.f, 0.f, 0.f, 0.f};
  if (p.post_w) normalise(st[0], st[1]);
  S* orow = static_cast<S*>(p.x_out) + row * p.ld_x;
  const long long gate_off = p.gate && live ? row / p.rows_per_gate * p.C : 0;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const int c = (e * wpr + wr) * 32 + lane;
    if (!live || c >= chunks) continue;
    float f[8], x[8];
    if (p.post_w) {
      params(p.post_w, 0, c, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[e][j] *= f[j];
      if (p.post_b) {
        params(p.post_b, 0, c, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[e][j] += f[j];
      }
    }
    if (p.gate) {
      params(p.gate, gate_off, c, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[e][j] *= f[j];
    }
    if (p.scale) {
      params(p.scale, 0, c, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[e][j] *= f[j];
    }
    chunk_floats(xr[e], x);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[e][j] += x[j];
    Chunk<T> o;
    chunk_round(o, v[e]);
    chunk_store(orow + c * 8, o);
    chunk_floats(o, v[e]);   // the pre norm is of the stored row
  }
  if (p.pre_w) {
    // Channels past the row must not count: they hold -mean * rstd of the post norm.
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (!live || (e * wpr + wr) * 32 + lane >= chunks) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[e][j] = 0.f;
      }
    normalise(st[2], st[3]);
    S* nrow = static_cast<S*>(p.n) + row * p.ld_n;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const int c = (e * wpr + wr) * 32 + lane;
      if (!live || c >= chunks) continue;
      float f[8];
      params(p.pre_w, 0, c, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[e][j] *= f[j];
      if (p.pre_b) {
        params(p.pre_b, 0, c, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[e][j] += f[j];
      }
      Chunk<T> o;
      chunk_round(o, v[e]);
      chunk_store(nrow + c * 8, o);
    }
  }
  if (p.stats && live && wr == 0 && lane == 0)
    reinterpret_cast<float4*>(p.stats)[row] = make_float4(st[0], st[1], st[2], st[3]);
}

template <class T, int V>
static cudaError_t launch_fwd(const NormParams& p, int wpr, cudaStream_t st) {
  const int rpb = 8 / wpr;
  return launch_pdl(k_norm_residual<T, V>, dim3((unsigned)((p.rows + rpb - 1) / rpb)), dim3(256), 0,
                    st, p, wpr);
}

cudaError_t launch_norm_residual(const NormParams& p, int dtype, cudaStream_t st) {
  // The fewest warps a row with at most five chunks a lane (40 fp32 values, C = 1280 in one warp).
  const int chunks = p.C / 8;
  int wpr = 1;
  while (wpr < 8 && chunks > 32 * 5 * wpr) wpr *= 2;
  const int v = (chunks + 32 * wpr - 1) / (32 * wpr);
  return by_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    switch (v) {
      case 1: return launch_fwd<T, 1>(p, wpr, st);
      case 2: return launch_fwd<T, 2>(p, wpr, st);
      case 3: return launch_fwd<T, 3>(p, wpr, st);
      case 4: return launch_fwd<T, 4>(p, wpr, st);
      default: return launch_fwd<T, 5>(p, wpr, st);
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
// contiguous rows, R at a time: bulk copies bring the rows of all four inputs into the worker's ring
// of shared-memory stages, well ahead of use, so that the row sums' barriers do not idle the memory.
// Several workers share a CTA (one per SM); at the end their column sums are added in worker order
// and written as one partial per CTA, which k_norm_reduce adds in CTA order: no atomics, the same
// result every run.
constexpr int kNormThreads = 512;
constexpr int kNormRingBytes = 192 * 1024;
constexpr int kNormMaxStages = 4;

struct NormBwdShape {
  long long rows_per_worker;
  int workers, wpg, rl;     // workers in all; warps per worker; workers per CTA
  int stages, stage_bytes;  // ring of one worker
  int tensors;              // rows brought per stage: dx_out, y, then x and dn with a pre norm
};

template <class T, int R>
__global__ void __launch_bounds__(kNormThreads, 1)
    k_norm_residual_backward(const NormBwdParams p, const NormBwdShape g, int* status) {
  using S = typename T::Store;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[16 * kNormMaxStages];
  __shared__ float red[2][16][2 * R];   // [buffer][warp][sums]
  __shared__ int abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rl = warp / g.wpg, wg = warp % g.wpg;
  const int tw = wg * 32 + lane;            // thread in the worker
  const int worker = blockIdx.x * g.rl + rl;
  const int chunks = p.C / 8;
  const bool col = tw < chunks && rl < g.rl;
  if (threadIdx.x == 0) {
    for (int i = 0; i < g.rl * g.stages; ++i) mbar_init(full + i, 1);
    abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  griddep_wait();
  griddep_launch();

  const long long r0 = (long long)worker * g.rows_per_worker;
  long long r1 = r0 + g.rows_per_worker;
  if (r1 > p.rows) r1 = p.rows;
  uint8_t* ring = smem + (size_t)rl * g.stages * g.stage_bytes;
  uint64_t* bar = full + rl * g.stages;
  const int row_bytes = p.C * (int)sizeof(S);
  // Batches never cross a group of rows that share a gate row.
  auto batch_rows = [&](long long r) {
    long long e = r1;
    if (p.gate) {
      const long long ge = (r / p.rows_per_gate + 1) * p.rows_per_gate;
      if (ge < e) e = ge;
    }
    return (int)(e - r < R ? e - r : R);
  };
  const void* src[4] = {p.dx_out, p.y, p.x, p.dn};
  const long long ld[4] = {p.ld_x, p.ld_y, p.ld_x, p.ld_n};
  auto fetch = [&](long long r, int st) {
    const int n = batch_rows(r);
    mbar_expect_tx(bar + st, (uint32_t)(g.tensors * n * row_bytes));
    for (int t = 0; t < g.tensors; ++t)
      for (int i = 0; i < n; ++i)
        bulk_load(ring + (size_t)st * g.stage_bytes + (size_t)(t * R + i) * row_bytes,
                  static_cast<const S*>(src[t]) + (r + i) * ld[t], (uint32_t)row_bytes, bar + st);
    return r + n;
  };
  long long ahead = r0;
  if (rl < g.rl && tw == 0)
    for (int s = 0; s < g.stages && ahead < r1; ++s) ahead = fetch(ahead, s);

  auto params = [&](const void* ptr, long long off, float (&f)[8]) {
    Chunk<T> w;
    chunk_load(w, static_cast<const S*>(ptr) + off + tw * 8);
    chunk_floats(w, f);
  };
  const bool pre = p.pre_w != nullptr, post = p.post_w != nullptr;
  float wpre[8], coef[8], base[8];   // base = scale * post_w; coef = gate * base
  float acc_pw[8], acc_pb[8], acc_a[8], acc_b[8], tot_a[8], tot_b[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    wpre[j] = 0.f;
    base[j] = 1.f;
    acc_pw[j] = acc_pb[j] = acc_a[j] = acc_b[j] = tot_a[j] = tot_b[j] = 0.f;
  }
  if (col) {
    float f[8];
    if (pre) params(p.pre_w, 0, wpre);
    if (p.scale) {
      params(p.scale, 0, base);
    }
    if (post) {
      params(p.post_w, 0, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) base[j] *= f[j];
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) coef[j] = base[j];

  // The sums of 2 R values over the worker's threads.
  int buf = 0;
  auto worker_sums = [&](float (&s)[2 * R]) {
#pragma unroll
    for (int i = 0; i < 2 * R; ++i) s[i] = warp_sum(s[i]);
    if (g.wpg > 1) {
      if (lane == 0) {
#pragma unroll
        for (int i = 0; i < 2 * R; ++i) red[buf][warp][i] = s[i];
      }
      named_barrier(1 + rl, g.wpg * 32);
#pragma unroll
      for (int i = 0; i < 2 * R; ++i) s[i] = 0.f;
      for (int w = 0; w < g.wpg; ++w)
#pragma unroll
        for (int i = 0; i < 2 * R; ++i) s[i] += red[buf][warp - wg + w][i];
      buf ^= 1;
    }
  };
  const float inv_c = 1.0f / (float)p.C;
  const float mean_on = p.center ? 1.f : 0.f;
  long long group = -1;
  int it = 0;
  // The gate row of the finished group: final if all its rows were this worker's, else a partial in
  // the worker's first slot (its first group) or second.
  auto close_group = [&]() {
    if (!p.gate || group < 0 || !col) return;
    const long long g0 = group * p.rows_per_gate;
    long long g1 = g0 + p.rows_per_gate;
    if (g1 > p.rows) g1 = p.rows;
    const bool whole = g0 >= r0 && g1 <= r1;
    float gate[8], f[8], dg[8];
    params(p.gate, group * p.C, gate);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = 1.f;
    if (post) params(p.post_w, 0, f);
#pragma unroll
    for (int j = 0; j < 8; ++j) dg[j] = f[j] * acc_a[j];
    if (p.post_b) {
      params(p.post_b, 0, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) dg[j] += f[j] * acc_b[j];
    }
    if (p.scale) {
      params(p.scale, 0, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) dg[j] *= f[j];
    }
    float* out = whole ? p.dgate + group * p.C
                       : p.gate_partial + ((long long)worker * 2 + (g0 > r0 ? 1 : 0)) * p.C;
    if (!whole || p.dgate) {
#pragma unroll
      for (int j = 0; j < 8; j += 4)
        reinterpret_cast<float4*>(out + tw * 8 + j)[0] =
            make_float4(dg[j], dg[j + 1], dg[j + 2], dg[j + 3]);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      tot_a[j] += gate[j] * acc_a[j];
      tot_b[j] += gate[j] * acc_b[j];
      acc_a[j] = acc_b[j] = 0.f;
    }
  };
  if (rl < g.rl) {
    for (long long r = r0; r < r1; ++it) {
      const int n = batch_rows(r);
      const int st = it % g.stages;
      if (p.gate) {
        const long long gr = r / p.rows_per_gate;
        if (gr != group) {
          close_group();
          group = gr;
          if (col) {
            float f[8];
            params(p.gate, group * p.C, f);
#pragma unroll
            for (int j = 0; j < 8; ++j) coef[j] = base[j] * f[j];
          }
        }
      }
      // A wait that gives up is recorded; the walk goes on to its end, so that no barrier is left
      // with missing threads (the addresses do not depend on the data).
      mbar_wait(bar + st, (it / g.stages) & 1, &abort_flag, status);
      Chunk<T> c_d[R], c_y[R], c_x[R], c_n[R];
      float4 stat[R];
      const uint8_t* sp = ring + (size_t)st * g.stage_bytes + (size_t)tw * 8 * sizeof(S);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        chunk_zero(c_d[i]);
        chunk_zero(c_y[i]);
        chunk_zero(c_x[i]);
        chunk_zero(c_n[i]);
        stat[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (col && i < n) {
          const size_t ro = (size_t)i * row_bytes;
          const size_t to = (size_t)R * row_bytes;
          chunk_load(c_d[i], reinterpret_cast<const S*>(sp + ro));
          chunk_load(c_y[i], reinterpret_cast<const S*>(sp + to + ro));
          if (pre) {
            chunk_load(c_x[i], reinterpret_cast<const S*>(sp + 2 * to + ro));
            chunk_load(c_n[i], reinterpret_cast<const S*>(sp + 3 * to + ro));
          }
          stat[i] = __ldg(reinterpret_cast<const float4*>(p.stats) + r + i);
        }
      }
      // Every thread has its chunks: the stage can be filled again.
      if (g.wpg > 1) named_barrier(1 + rl, g.wpg * 32);
      else __syncwarp();
      if (tw == 0 && ahead < r1) ahead = fetch(ahead, st);
      float D[R][8];
#pragma unroll
      for (int i = 0; i < R; ++i) chunk_floats(c_d[i], D[i]);
      if (pre) {
        float s[2 * R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
          float x[8], dn[8];
          chunk_floats(c_x[i], x);
          chunk_floats(c_n[i], dn);
          s[2 * i] = s[2 * i + 1] = 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float h = (x[j] - stat[i].z) * stat[i].w;
            const float gg = dn[j] * wpre[j];
            s[2 * i] += gg;
            s[2 * i + 1] += gg * h;
            acc_pw[j] += dn[j] * h;
            acc_pb[j] += dn[j];
          }
        }
        worker_sums(s);
#pragma unroll
        for (int i = 0; i < R; ++i) {
          float x[8], dn[8];
          chunk_floats(c_x[i], x);
          chunk_floats(c_n[i], dn);
          const float m0 = s[2 * i] * inv_c * mean_on, m1 = s[2 * i + 1] * inv_c;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float h = (x[j] - stat[i].z) * stat[i].w;
            D[i][j] += stat[i].w * (dn[j] * wpre[j] - m0 - h * m1);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (col && i < n) {
          Chunk<T> o;
          chunk_round(o, D[i]);
          chunk_store(static_cast<S*>(p.dx) + (r + i) * p.ld_x + tw * 8, o);
        }
      // h_post (or y), the column sums and, with a post norm, the row sums.
      float s[2 * R];
#pragma unroll
      for (int i = 0; i < R; ++i) {
        float y[8];
        chunk_floats(c_y[i], y);
        s[2 * i] = s[2 * i + 1] = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float h = post ? (y[j] - stat[i].x) * stat[i].y : y[j];
          acc_a[j] += D[i][j] * h;
          acc_b[j] += D[i][j];
          const float q = D[i][j] * coef[j];
          s[2 * i] += q;
          s[2 * i + 1] += q * h;
        }
      }
      if (post) worker_sums(s);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (!col || i >= n) continue;
        float y[8], o8[8];
        chunk_floats(c_y[i], y);
        const float m0 = s[2 * i] * inv_c * mean_on, m1 = s[2 * i + 1] * inv_c;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float q = D[i][j] * coef[j];
          o8[j] = post ? stat[i].y * (q - m0 - (y[j] - stat[i].x) * stat[i].y * m1) : q;
        }
        Chunk<T> o;
        chunk_round(o, o8);
        chunk_store(static_cast<S*>(p.dy) + (r + i) * p.ld_y + tw * 8, o);
      }
      r += n;
    }
    close_group();
  }
  if (!p.gate) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      tot_a[j] = acc_a[j];
      tot_b[j] = acc_b[j];
    }
  }
  // The CTA's column sums, in worker order: [pre_w, pre_b, P1, P0][C]. The ring is free now: every
  // copy into it has been waited for.
  __syncthreads();
  float* sums = reinterpret_cast<float*>(smem);
  if (col) {
    float* mine = sums + (size_t)rl * 4 * p.C + tw * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      mine[j] = acc_pw[j];
      mine[p.C + j] = acc_pb[j];
      mine[2 * p.C + j] = tot_a[j];
      mine[3 * p.C + j] = tot_b[j];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 4 * p.C; i += blockDim.x) {
    float s = 0.f;
    for (int w = 0; w < g.rl; ++w) s += sums[(size_t)w * 4 * p.C + i];
    p.partial[(size_t)blockIdx.x * 4 * p.C + i] = s;
  }
}

// Adds the CTAs' partials in a fixed order and forms the parameters' gradients. Blocks x < ceil(C / 32)
// with y == 0 own 32 channels; the rows y > 0 own the gate rows whose group several workers shared.
template <class T>
__global__ void __launch_bounds__(512) k_norm_reduce(const NormBwdParams p, const NormBwdShape g,
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
  // Gate rows: one warp a group, in turn.
  if (c >= p.C) return;
  const long long groups = (p.rows + p.rows_per_gate - 1) / p.rows_per_gate;
  const long long step = (long long)(gridDim.y - 1) * 16;
  for (long long gr = (long long)(blockIdx.y - 1) * 16 + warp; gr < groups; gr += step) {
    const long long g0 = gr * p.rows_per_gate;
    long long g1 = g0 + p.rows_per_gate;
    if (g1 > p.rows) g1 = p.rows;
    const long long w0 = g0 / g.rows_per_worker, w1 = (g1 - 1) / g.rows_per_worker;
    if (w0 == w1) continue;   // one worker's: written by it
    float s = 0.f;
    for (long long w = w0; w <= w1; ++w)
      s += p.gate_partial[(w * 2 + (g0 > w * g.rows_per_worker ? 1 : 0)) * p.C + c];
    p.dgate[gr * p.C + c] = s;
  }
}

// The workers' geometry; `ctas` CTAs at most are planned for.
static NormBwdShape bwd_shape(long long rows, int C, int es, bool pre, int* R, int* ctas) {
  NormBwdShape g;
  g.wpg = (C / 8 + 31) / 32;
  g.rl = (kNormThreads / 32) / g.wpg;
  g.tensors = pre ? 4 : 2;
  const int row = g.tensors * C * es;
  // Two rows at a time share the row sums' barriers; one where two would leave fewer than three
  // stages.
  *R = kNormRingBytes / (g.rl * 2 * row) >= 3 ? 2 : 1;
  while (g.rl > 1 && kNormRingBytes / (g.rl * *R * row) < 2) --g.rl;
  g.stage_bytes = *R * row;
  g.stages = kNormRingBytes / (g.rl * g.stage_bytes);
  if (g.stages > kNormMaxStages) g.stages = kNormMaxStages;
  const long long most = (long long)kNormMaxCtas * g.rl;
  g.rows_per_worker = (rows + most - 1) / most;
  if (g.rows_per_worker < 1) g.rows_per_worker = 1;
  g.workers = (int)((rows + g.rows_per_worker - 1) / g.rows_per_worker);
  *ctas = (g.workers + g.rl - 1) / g.rl;
  return g;
}

size_t norm_backward_partial(long long rows, int C, int es, bool pre, bool gate,
                             size_t* gate_offset) {
  int R, ctas;
  const NormBwdShape g = bwd_shape(rows, C, es, pre, &R, &ctas);
  *gate_offset = (size_t)ctas * 4 * C * sizeof(float);
  return *gate_offset + (gate ? (size_t)ctas * g.rl * 2 * C * sizeof(float) : 0);
}

template <class T, int R>
static cudaError_t launch_bwd(const NormBwdParams& p, const NormBwdShape& g, int ctas, int* status,
                              cudaStream_t st) {
  size_t smem = (size_t)g.rl * g.stages * g.stage_bytes;
  const size_t sums = (size_t)g.rl * 4 * p.C * sizeof(float);
  if (sums > smem) smem = sums;
  cudaError_t e = cudaFuncSetAttribute(k_norm_residual_backward<T, R>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kNormRingBytes);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_norm_residual_backward<T, R>, dim3(ctas), dim3(kNormThreads), smem, st, p, g,
                    status);
}

cudaError_t launch_norm_backward(const NormBwdParams& p, int dtype, int* status, cudaStream_t st) {
  if (p.rows == 0) return cudaSuccess;
  const int es = dtype == SS_F32 ? 4 : 2;
  int R, ctas;
  const NormBwdShape g = bwd_shape(p.rows, p.C, es, p.pre_w != nullptr, &R, &ctas);
  return by_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    return R == 2 ? launch_bwd<T, 2>(p, g, ctas, status, st)
                  : launch_bwd<T, 1>(p, g, ctas, status, st);
  });
}

cudaError_t launch_norm_reduce(const NormBwdParams& p, int dtype, cudaStream_t st) {
  const int es = dtype == SS_F32 ? 4 : 2;
  int R, ctas;
  const NormBwdShape g = bwd_shape(p.rows, p.C, es, p.pre_w != nullptr, &R, &ctas);
  if (p.rows == 0) ctas = 0;   // sums over no rows: zeros
  int ny = 1;
  if (p.dgate && p.rows > 0) {
    const long long groups = (p.rows + p.rows_per_gate - 1) / p.rows_per_gate;
    ny += (int)((groups + 15) / 16 < 64 ? (groups + 15) / 16 : 64);
  }
  const dim3 grid((p.C + 31) / 32, ny);
  return by_dtype(dtype, [&](auto t) {
    return launch_pdl(k_norm_reduce<decltype(t)>, grid, dim3(512), 0, st, p, g, ctas);
  });
}

cudaError_t set_wait_limit_norm(uint64_t ns) { return set_wait_limit_here(ns); }

}  // namespace ss

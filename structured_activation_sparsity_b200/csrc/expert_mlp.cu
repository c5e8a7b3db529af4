// The experts' products on tcgen05 / TMEM: for rows sorted by expert, H = GELU(X W1_e^T + b1_e) and
// Y = H W2_e^T + b2_e, each expert over its own rows, in one launch per product.
//
// The product is taken transposed, D[features, rows] = W_e[features, Kd] X[rows, Kd]^T: the weights are
// the 128-row operand and the tokens the narrow one. An expert's row count is whatever the router
// gave it; the tensor core's N (a multiple of 16 up to 256) follows it, where an M of 128 tokens
// would be mostly padding at a few rows an expert, and the weights, which bound that case, are always
// read in whole tiles. With many rows a tile is 128 x 256 like the dense GEMM's.
//
// The row counts are on the device only (the sort's offsets): every CTA turns them into the same
// list of tiles, and takes units (tile, feature tile, k-split) c, c + grid, c + 2 grid, ...
#include "kernels.h"
#include "rows.cuh"

namespace ss {

// warp 0 TMA producer, warp 1 TMEM allocation and MMA issue, warps 2-3 idle, warps 4-11 epilogue.
constexpr int kXThreads = 384;
constexpr int kXEpiThreads = 256;
constexpr uint32_t kXRegsProducer = 56, kXRegsEpilogue = 224;
static_assert(128 * kXRegsProducer + 256 * kXRegsEpilogue <= 384 * 168,
              "expert GEMM register split too large");

// Token tile TN: a stage holds one 64-wide k-block of 128 weight rows and TN token rows.
template <int TN>
struct XCfg {
  static constexpr int kABytes = 128 * 128;
  static constexpr int kBBytes = TN * 128;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kStages = (192 * 1024) / kStageBytes < 10 ? (192 * 1024) / kStageBytes : 10;
  static constexpr int kBar = kStages * kStageBytes;
  static constexpr int kTiles = kBar + 256;                       // tile_start[E + 1], offsets[E + 1]
  static constexpr int kAlloc = kTiles + 2 * (kMaxExperts + 1) * 4 + 1024;
  static constexpr int kTmemCols = 2 * TN <= 32 ? 32 : 2 * TN;    // two accumulators
  static_assert((2 * kStages + 5) * 8 <= 256, "barriers");
};

// GELU(z) = z/2 (1 + erf(z / sqrt 2)) by the polynomial of k_gemm's epilogue (Abramowitz & Stegun
// 7.1.26, |error| <= 1.5e-7), on one value.
__device__ __forceinline__ float gelu_erf1(float z) {
  const float x = fabsf(z) * 0.70710678118654752f;
  const float t = rcp_mufu(fmaf(0.3275911f, x, 1.0f));
  float q = fmaf(1.061405429f, t, -1.453152027f);
  q = fmaf(q, t, 1.421413741f);
  q = fmaf(q, t, -0.284496736f);
  q = fmaf(q, t, 0.254829592f);
  const float erfc = t * q * ex2_mufu(-1.4426950408889634f * x * x);
  return 0.5f * z * (z >= 0.f ? 2.0f - erfc : erfc);
}

struct XUnit {
  int e, row0, rows;     // expert, first sorted row, rows of the tile (1..TN)
  int m0, s, kb0, kb1;   // first feature, k-split and its k-blocks
};

template <int TN>
__global__ void __launch_bounds__(kXThreads, 1)
    k_expert_gemm(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
                  const ExpertGemm g, int* status) {
  using G = XCfg<TN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + G::kBar);
  uint64_t* empty = full + G::kStages;
  uint64_t* acc_full = empty + G::kStages;   // [2]
  uint64_t* acc_empty = acc_full + 2;        // [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* tile_start = reinterpret_cast<int*>(smem + G::kTiles);   // [E + 1]
  int* offs = tile_start + kMaxExperts + 1;                     // [E + 1]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < G::kStages; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full + b, 1);
      mbar_init(acc_empty + b, kXEpiThreads);
    }
    *abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc(tmem_slot, G::kTmemCols);
  griddep_wait();
  griddep_launch();
  // The experts' tiles: warp 2 sums ceil(rows / TN) over the experts, 32 at a time.
  if (warp == 2) {
    int base = 0;
    for (int e0 = 0; e0 < g.E; e0 += 32) {
      const int e = e0 + lane;
      const int lo = e < g.E ? __ldg(g.offsets + e) : 0, hi = e < g.E ? __ldg(g.offsets + e + 1) : 0;
      int x = (hi - lo + TN - 1) / TN;
      const int own = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (e < g.E) {
        tile_start[e] = base + x - own;
        offs[e] = lo;
        if (e == g.E - 1) {
          tile_start[g.E] = base + x;
          offs[g.E] = hi;
        }
      }
      base += __shfl_sync(0xffffffffu, x, 31);
    }
  }
  tc_fence_before();
  cta_sync_converged();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int units = tile_start[g.E] * g.m_tiles * g.splits;

  auto decode = [&](int u) {
    XUnit r;
    r.s = u % g.splits;
    const int v = u / g.splits;
    r.m0 = v % g.m_tiles * 128;
    const int t = v / g.m_tiles;
    int lo = 0, hi = g.E;   // tile_start[lo] <= t < tile_start[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (tile_start[mid] <= t) lo = mid;
      else hi = mid;
    }
    r.e = lo;
    r.row0 = offs[lo] + (t - tile_start[lo]) * TN;
    const int left = offs[lo + 1] - r.row0;
    r.rows = left < TN ? left : TN;
    r.kb0 = (int)((long long)r.s * g.kb_total / g.splits);
    r.kb1 = (int)((long long)(r.s + 1) * g.kb_total / g.splits);
    return r;
  };

  if (warp < 4) {
    setmaxnreg_dec<kXRegsProducer>();
    if (warp == 0 && lane == 0) {
      tma_prefetch_desc(&ta);
      tma_prefetch_desc(&tb);
      int it = 0;
      bool ok = true;
      for (int u = blockIdx.x; ok && u < units; u += gridDim.x) {
        const XUnit r = decode(u);
        const int nk = r.kb1 - r.kb0;
        for (int j = 0; j < nk; ++j, ++it) {
          const int st = it % G::kStages;
          if (it >= G::kStages &&
              !(ok = mbar_wait(empty + st, ((it / G::kStages) - 1) & 1, abort, status)))
            break;
          uint8_t* sa = smem + st * G::kStageBytes;
          mbar_expect_tx(full + st, G::kStageBytes);
          tma_load_2d(sa, &ta, full + st, (r.kb0 + j) * 64, r.e * g.features + r.m0);
          tma_load_2d(sa + G::kABytes, &tb, full + st, (r.kb0 + j) * 64, r.row0);
        }
      }
    } else if (warp == 1 && lane == 0) {
      int it = 0, i = 0;
      bool ok = true;
      for (int u = blockIdx.x; ok && u < units; u += gridDim.x, ++i) {
        const XUnit r = decode(u);
        const uint32_t idesc = idesc_bf16_f32(128, (r.rows + 15) & ~15, false, false);
        const int buf = i & 1;
        if (i >= 2 && !(ok = mbar_wait(acc_empty + buf, ((i >> 1) - 1) & 1, abort, status))) break;
        tc_fence_after();
        const uint32_t d = tmem + buf * TN;
        const int nk = r.kb1 - r.kb0;
        bool ready = mbar_test(full + it % G::kStages, (it / G::kStages) & 1);
        for (int j = 0; j < nk; ++j, ++it) {
          const int st = it % G::kStages;
          if (!__builtin_expect(ready, 1) &&
              !(ok = mbar_wait(full + st, (it / G::kStages) & 1, abort, status)))
            break;
          if (j + 1 < nk) ready = mbar_test(full + (it + 1) % G::kStages, ((it + 1) / G::kStages) & 1);
          tc_fence_after();
          const uint32_t a_addr = smem_u32(smem + st * G::kStageBytes);
          const uint32_t b_addr = a_addr + G::kABytes;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_bf16_ss(d, smem_desc(a_addr + kk * 32, 16, 1024, kSwizzle128B),
                         smem_desc(b_addr + kk * 32, 16, 1024, kSwizzle128B), idesc,
                         (j > 0 || kk > 0) ? 1u : 0u);
          umma_commit(empty + st);
        }
        if (ok) umma_commit(acc_full + buf);
      }
    }
  } else {
    setmaxnreg_inc<kXRegsEpilogue>();
    // Warp w reads TMEM lanes 32 (w % 4) ..: a thread holds one feature, and 16 rows at a time (the two
    // warps of a lane quadrant take every other group of 16).
    const int quad = warp & 3, half = (warp - 4) >> 2;
    const uint32_t lane_off = uint32_t(32 * quad) << 16;
    int i = 0;
    for (int u = blockIdx.x; u < units; u += gridDim.x, ++i) {
      const XUnit r = decode(u);
      const int buf = i & 1;
      const int f = r.m0 + 32 * quad + lane;
      const bool live = f < g.features;
      float bias = 0.f;
      if (live && g.bias && r.s == 0)
        bias = __uint_as_float((uint32_t)__ldg(g.bias + (size_t)r.e * g.features + f) << 16);
      const bool ok = __all_sync(0xffffffffu, mbar_wait(acc_full + buf, (i >> 1) & 1, abort, status));
      if (!ok) break;
      tc_fence_after();
      const uint32_t t_acc = tmem + buf * TN + lane_off;
      for (int c = half * 16; c < r.rows; c += 32) {
        uint32_t v[16];
        tmem_ld16(t_acc + c, v);
        const int n = r.rows - c < 16 ? r.rows - c : 16;
        if (g.partial) {
          float* out = g.partial + ((size_t)r.s * g.n + r.row0 + c) * g.features + f;
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (live && e < n) out[(size_t)e * g.features] = __uint_as_float(v[e]) + bias;
        } else {
          uint16_t* out = g.out + (size_t)(r.row0 + c) * g.features + f;
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float z = __uint_as_float(v[e]) + bias;
            if (g.gelu) z = gelu_erf1(z);
            if (live && e < n) {
              const __nv_bfloat16 h = __float2bfloat16_rn(z);
              out[(size_t)e * g.features] = *reinterpret_cast<const uint16_t*>(&h);
            }
          }
        }
      }
      tc_fence_before();
      mbar_arrive(acc_empty + buf);
    }
  }
  tc_fence_before();
  cta_sync_converged();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, G::kTmemCols);
  }
}

ExpertGemmPlan expert_gemm_plan(long long n, int E, int features, int Kd, bool split, int sms) {
  ExpertGemmPlan p;
  p.m_tiles = (features + 127) / 128;
  // The narrowest token tile that holds an average expert's rows.
  const long long avg = (n + E - 1) / E;
  p.tn = avg <= 32 ? 32 : avg <= 64 ? 64 : avg <= 128 ? 128 : 256;
  // Tiles at most: one per expert with rows, and one more per full tile.
  long long tiles = n / p.tn + (n < E ? n : E);
  if (tiles > n) tiles = n;
  p.max_units = tiles * p.m_tiles;
  p.splits = 1;
  const int kb = (Kd + 63) / 64;
  if (split)
    while (p.splits < 8 && p.max_units * (p.splits + 1) <= sms && kb / (p.splits + 1) >= 4)
      ++p.splits;
  p.max_units *= p.splits;
  return p;
}

template <int TN>
static cudaError_t launch_x(const CUtensorMap* ta, const CUtensorMap* tb, const ExpertGemm& g,
                            int grid, int* status, cudaStream_t st) {
  using G = XCfg<TN>;
  cudaError_t e = cudaFuncSetAttribute(k_expert_gemm<TN>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, G::kAlloc);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_expert_gemm<TN>, dim3(grid), dim3(kXThreads), G::kAlloc, st, *ta, *tb, g,
                    status);
}

cudaError_t launch_expert_gemm(const CUtensorMap* ta, const CUtensorMap* tb,
                               const ExpertGemmPlan& p, const ExpertGemm& g, int sms, int* status,
                               cudaStream_t st) {
  const int grid = (int)(p.max_units < sms ? p.max_units : sms);
  switch (p.tn) {
    case 32: return launch_x<32>(ta, tb, g, grid, status, st);
    case 64: return launch_x<64>(ta, tb, g, grid, status, st);
    case 128: return launch_x<128>(ta, tb, g, grid, status, st);
    default: return launch_x<256>(ta, tb, g, grid, status, st);
  }
}

cudaError_t set_wait_limit_expert_mlp(uint64_t ns) { return set_wait_limit_here(ns); }

}  // namespace ss

// The experts' products on tcgen05 / TMEM: for rows sorted by expert, H = GELU(X W1_e^T + b1_e) and
// Y = H W2_e^T + b2_e, each expert over its own rows, in one launch per product.
//
// The product is taken transposed, D[features, rows] = W_e[features, Kd] X[rows, Kd]^T: the weights are
// the 128-row operand and the tokens the narrow one. An expert's row count is whatever the router
// gave it; the tensor core's N (a multiple of 16 up to 256) follows it, where an M of 128 tokens
// would be mostly padding at a few rows an expert, and the weights, which bound that case, are always
// read in whole tiles. With many rows two CTAs take a tile of 256 features x 256 rows together
// (tcgen05 cta_group::2), each bringing its half of both operands.
//
// Measured on B200: 16384 tokens x 2 of 8 experts, C 1280, hidden 5120: fc1 358 us, fc2 304 us (1.20 and 1.41
// PFLOP/s; the measured cuBLAS burst is 1.63, sustained 1.38); the whole call 767 us in a burst, 833 back to
// back under the power cap. 784 tokens x 2 of 16 experts, C 1024, hidden 4096, 98 rows an expert: 38 us a
// product, whose weights take HBM 20.8 us. Loading those weights alone in the same boxes takes 28.8 us shared
// evenly and 32.9 in whole tiles (a plain read 22.6), the token rows 2 more; asking for the weights ahead in
// L2, as tiles or as whole rows, made it slower (89 to 98 us instead of 82 for the call).
//
// The row counts are on the device only (the sort's offsets): every CTA turns them into the same
// list of tiles, and takes units (tile, feature tile, k-split) c, c + grid, c + 2 grid, ...
//
// Part of mlp.cu, whose GELU it uses.
#pragma once

#include "kernels.h"
#include "rows.cuh"

namespace ss {

// warp 0 TMA producer, warp 1 TMEM allocation and MMA issue, warps 2-3 idle, warps 4-11 epilogue.
constexpr int kXThreads = 384;
constexpr int kXEpiThreads = 256;
constexpr uint32_t kXRegsProducer = 56, kXRegsEpilogue = 224;
static_assert(128 * kXRegsProducer + 256 * kXRegsEpilogue <= 384 * 168,
              "expert GEMM register split too large");

// Each epilogue warp turns 32 rows at a time from feature-major (a thread holds one feature) to row-major
// in 2 KB of shared memory: 64 bytes a row, so that it stores 16 bytes a lane, eight rows an instruction.
constexpr int kXTurn = 32 * 64;

// Token tile TN: a stage holds one 64-wide k-block of 128 weight rows and up to TN token rows. These come in
// one box, of all the tile's rows or of half of them if that holds what the tile has: the issue of a load
// costs its thread over a hundred cycles, and with a box per 32 rows the tensor cores waited for that
// half of the time. PAIR: two CTAs work on a tile of 256 weight rows, each with 128 of them and half of
// the token rows.
template <int TN, bool PAIR>
struct XCfg {
  static constexpr int kBox = expert_box(TN, PAIR);   // rows of the larger box
  static constexpr int kABytes = 128 * 128;  static constexpr int kBBytes = kBox * 128;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kStages = (192 * 1024) / kStageBytes < 10 ? (192 * 1024) / kStageBytes : 10;
  static constexpr int kBar = kStages * kStageBytes;
  static constexpr int kTiles = kBar + 256;                       // tile_start[E + 1], offsets[E + 1]
  static constexpr int kTurn = kTiles + (2 * (kMaxExperts + 1) * 4 + 15) / 16 * 16;
  static constexpr int kAlloc = kTurn + 8 * kXTurn + 1024;
  static constexpr int kTmemCols = 2 * TN <= 32 ? 32 : 2 * TN;    // two accumulators
  static_assert((2 * kStages + 5) * 8 <= 256, "barriers");
};

struct XUnit {
  int e, row0, rows;     // expert, first sorted row, rows of the tile (1..TN)
  int m0, s, kb0, kb1;   // first feature, k-split and its k-blocks
};

template <int TN, bool PAIR>
__global__ void __launch_bounds__(kXThreads, 1)
    k_expert_gemm(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
                  const __grid_constant__ CUtensorMap tb_half, const ExpertGemm g, int* status) {
  using G = XCfg<TN, PAIR>;
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
      mbar_init(acc_empty + b, (PAIR ? 2 : 1) * kXEpiThreads / 32);
    }
    *abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    if constexpr (PAIR) tmem_alloc_pair(tmem_slot, G::kTmemCols);
    else tmem_alloc(tmem_slot, G::kTmemCols);
  }
  griddep_wait();
  griddep_launch();
  // The experts' tiles: warp 2 sums ceil(rows / TN) over the experts, 32 at a time.
  if (warp == 2) {
    int base = 0;
    for (int e0 = 0; e0 < g.E; e0 += 32) {
      const int e = e0 + lane;
      const int lo = e < g.E ? g.offsets[e] : 0, hi = e < g.E ? g.offsets[e + 1] : 0;
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
  // The whole cluster (PAIR: the barriers that the other CTA arrives on are set up, too).
  auto meet = [&] {
    if constexpr (PAIR) cluster_sync_converged();
    else cta_sync_converged();
  };
  tc_fence_before();
  meet();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int units = tile_start[g.E] * g.m_tiles * g.splits;
  // The pair takes its units together; its first CTA issues the MMAs.
  const int rank = PAIR ? (int)cluster_rank() : 0;
  const int first = PAIR ? blockIdx.x / 2 : blockIdx.x, step = PAIR ? gridDim.x / 2 : gridDim.x;
  // Columns of the tile's MMA: its rows, rounded up to the instruction's step (PAIR: of each half).
  auto columns = [](int rows) { return PAIR ? (rows + 31) & ~31 : (rows + 15) & ~15; };

  auto decode = [&](int u) {
    XUnit r;
    r.s = u % g.splits;
    const int v = u / g.splits;
    r.m0 = v % g.m_tiles * (PAIR ? 256 : 128) + rank * 128;
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
      tma_prefetch_desc(&tb_half);
      // (One thread's instructions between two loads are time the tensor cores may wait: the loop keeps
      // its stage and phase, and addresses are added up.)
      const uint32_t bar0 = PAIR ? cluster_addr(full, 0) : smem_u32(full);
      int st = 0, phase = 1;   // the first round finds every stage free
      bool ok = true;
      for (int u = first; ok && u < units; u += step) {
        const XUnit r = decode(u);
        // This CTA's token rows (PAIR: its half of the columns).
        const int mine = PAIR ? columns(r.rows) / 2 : r.rows, row0 = r.row0 + rank * mine;
        const bool half = mine <= G::kBox / 2;
        const CUtensorMap* map = half ? &tb_half : &tb;
        const uint32_t bytes = G::kABytes + (half ? G::kBBytes / 2 : G::kBBytes);
        const int f = r.e * g.features + r.m0;
        for (int kc = r.kb0 * 64; kc < r.kb1 * 64; kc += 64) {
          if (!(ok = mbar_wait(empty + st, phase, abort, status))) break;
          uint8_t* sa = smem + st * G::kStageBytes;
          if constexpr (PAIR) {
            // Both CTAs' loads count on the first one's barrier, whose MMAs read both.
            if (rank == 0) mbar_expect_tx(full + st, 2 * bytes);
            tma_load_2d_pair(sa, &ta, bar0 + st * 8, kc, f);
            tma_load_2d_pair(sa + G::kABytes, map, bar0 + st * 8, kc, row0);
          } else {
            mbar_expect_tx(full + st, bytes);
            tma_load_2d(sa, &ta, full + st, kc, f);
            tma_load_2d(sa + G::kABytes, map, full + st, kc, row0);
          }
          if (++st == G::kStages) {
            st = 0;
            phase ^= 1;
          }
        }
      }
    } else if (warp == 1 && lane == 0 && rank == 0) {
      // Descriptors of the first stage; others are added to (addresses count in 16 bytes).
      const uint64_t desc0 = smem_desc(smem_u32(smem), 16, 1024, kSwizzle128B);
      int st = 0, phase = 0, i = 0;
      bool ok = true, ready = mbar_test(full, 0);
      for (int u = first; ok && u < units; u += step, ++i) {
        const XUnit r = decode(u);
        const uint32_t idesc = idesc_bf16_f32(PAIR ? 256 : 128, columns(r.rows), false, false);
        const int buf = i & 1;
        if (i >= 2 &&
            !(ok = PAIR ? mbar_wait_cluster(acc_empty + buf, ((i >> 1) - 1) & 1, abort, status)
                        : mbar_wait(acc_empty + buf, ((i >> 1) - 1) & 1, abort, status)))
          break;
        tc_fence_after();
        const uint32_t d = tmem + buf * TN;
        uint32_t more = 0;   // the unit's first MMA clears the accumulator
        for (int left = r.kb1 - r.kb0; left > 0; --left) {
          if (!__builtin_expect(ready, 1) && !(ok = mbar_wait(full + st, phase, abort, status)))
            break;
          const int cur = st;
          if (++st == G::kStages) {
            st = 0;
            phase ^= 1;
          }
          ready = mbar_test(full + st, phase);   // the next stage's, behind this one's MMAs
          tc_fence_after();
          const uint64_t a = desc0 + (uint64_t)cur * (G::kStageBytes >> 4);
          const uint64_t b = a + (G::kABytes >> 4);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            if constexpr (PAIR) umma_bf16_ss_pair(d, a + 2 * kk, b + 2 * kk, idesc, more);
            else umma_bf16_ss(d, a + 2 * kk, b + 2 * kk, idesc, more);
            more = 1;
          }
          if constexpr (PAIR) umma_commit_pair(empty + cur);
          else umma_commit(empty + cur);
        }
        if (ok) {
          if constexpr (PAIR) umma_commit_pair(acc_full + buf);
          else umma_commit(acc_full + buf);
        }
      }
    }
  } else {
    setmaxnreg_inc<kXRegsEpilogue>();
    // Warp w reads TMEM lanes 32 (w % 4) ..: a thread holds one feature, and 32 rows at a time (the two
    // warps of a lane quadrant take every other group of 32).
    const int quad = warp & 3, half = (warp - 4) >> 2;
    const uint32_t lane_off = uint32_t(32 * quad) << 16;
    uint16_t* turn = reinterpret_cast<uint16_t*>(smem + G::kTurn + (warp - 4) * kXTurn);
    int i = 0;
    for (int u = first; u < units; u += step, ++i) {
      const XUnit r = decode(u);
      const int buf = i & 1;
      const int f0 = r.m0 + 32 * quad, f = f0 + lane;
      const bool live = f < g.features;
      float bias = 0.f;
      if (live && g.bias && r.s == 0)
        bias = __uint_as_float((uint32_t)__ldg(g.bias + (size_t)r.e * g.features + f) << 16);
      const bool ok = __all_sync(0xffffffffu, mbar_wait(acc_full + buf, (i >> 1) & 1, abort, status));
      if (!ok) break;
      tc_fence_after();
      const uint32_t t_acc = tmem + buf * TN + lane_off;
      for (int c = half * 32; c < r.rows; c += 64) {
        uint32_t v[32];
        tmem_ld32(t_acc + c, v);
        const int n = r.rows - c < 32 ? r.rows - c : 32;
        if (g.partial) {
          float* out = g.partial + ((size_t)r.s * g.n + r.row0 + c) * g.features + f;
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (live && e < n) out[(size_t)e * g.features] = __uint_as_float(v[e]) + bias;
          continue;
        }
        __syncwarp();   // the previous group's rows have been read
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float z0, z1;
          f2_unpack(f2_add(f2_pack(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])),
                           f2_pack(bias, bias)), z0, z1);
          if (g.gelu) gelu_erf2(z0, z1);
          const uint32_t h = pack_bf16(z0, z1);
          turn[(2 * e) * 32 + lane] = (uint16_t)h;
          turn[(2 * e + 1) * 32 + lane] = (uint16_t)(h >> 16);
        }
        __syncwarp();
        // Eight rows an instruction, four lanes a row of 64 bytes (features are a multiple of 8).
        const int q = lane & 3;
        uint16_t* out = g.out + (size_t)(r.row0 + c + (lane >> 2)) * g.features + f0 + 8 * q;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint4 w = reinterpret_cast<const uint4*>(turn)[e * 32 + lane];
          if (8 * e + (lane >> 2) < n && f0 + 8 * q < g.features)
            *reinterpret_cast<uint4*>(out + (size_t)(8 * e) * g.features) = w;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (PAIR) mbar_arrive_cluster(cluster_addr(acc_empty + buf, 0));
        else mbar_arrive(acc_empty + buf);
      }
    }
  }
  tc_fence_before();
  abort_drain(abort);
  meet();   // (PAIR: nothing of the other CTA's is in use any more, either)
  if (warp == 1) {
    tc_fence_after();
    if constexpr (PAIR) tmem_dealloc_pair(tmem, G::kTmemCols);
    else tmem_dealloc(tmem, G::kTmemCols);
  }
}

ExpertGemmPlan expert_gemm_plan(long long n, int E, int features, int Kd, bool split, int sms) {
  ExpertGemmPlan p;
  // A token tile of twice an average expert's rows: an expert with one row more than the tile reads its
  // weights again for a second one (784 tokens over 16 experts, 98 rows on average: 98 us with tiles of
  // 128, 87 us with 256), while what a tile does not fill is not loaded. Measured on B200 at 24, 32, 48, 64, 80 and
  // 98 rows an expert, 16 experts of 1024 - 4096: tiles of 64 rows 66, 67, 69, 92, 101, 102 us; of 128 68, 68, 72, 74,
  // 75, 76 (128 rows: 100); pairs of 256 69, 70, 72, 73, 76, 77 (81). 64 experts of 512 - 2048: 72, 74, 80, 100, 116;
  // 72, 74, 75, 78, 80; 74, 77, 82, 87, 92.
  const long long avg = (n + E - 1) / E;
  p.tn = avg <= 32 ? 64 : avg <= 64 ? 128 : 256;
  // Pairs of CTAs where tiles are wide.
  p.pair = p.tn == 256;
  p.box = expert_box(p.tn, p.pair);
  const int workers = p.pair ? sms / 2 : sms;
  p.m_tiles = (features + (p.pair ? 255 : 127)) / (p.pair ? 256 : 128);
  // Tiles at most: one per expert with rows, and one more per full tile.
  long long tiles = n / p.tn + (n < E ? n : E);
  if (tiles > n) tiles = n;
  p.max_units = tiles * p.m_tiles;
  p.splits = 1;
  const int kb = (Kd + 63) / 64;
  if (split)
    while (p.splits < 8 && p.max_units * (p.splits + 1) <= workers && kb / (p.splits + 1) >= 4)
      ++p.splits;
  p.max_units *= p.splits;
  return p;
}

template <int TN, bool PAIR>
static cudaError_t launch_x(const CUtensorMap* ta, const CUtensorMap* tb,
                            const CUtensorMap* tb_half, const ExpertGemmPlan& p,
                            const ExpertGemm& g, int sms, int* status, cudaStream_t st) {
  using G = XCfg<TN, PAIR>;
  const auto kernel = k_expert_gemm<TN, PAIR>;
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), G::kAlloc);
  if (e != cudaSuccess) return e;
  const int workers = PAIR ? sms / 2 : sms;
  const int grid = (int)(p.max_units < workers ? p.max_units : workers) * (PAIR ? 2 : 1);
  return launch_pdl_clusters(kernel, PAIR ? 2 : 1, dim3(grid), dim3(kXThreads), G::kAlloc, st, *ta,
                             *tb, *tb_half, g, status);
}

cudaError_t launch_expert_gemm(const CUtensorMap* ta, const CUtensorMap* tb,
                               const CUtensorMap* tb_half, const ExpertGemmPlan& p,
                               const ExpertGemm& g, int sms, int* status, cudaStream_t st) {
  if (p.tn == 64) return launch_x<64, false>(ta, tb, tb_half, p, g, sms, status, st);
  if (p.tn == 128) return launch_x<128, false>(ta, tb, tb_half, p, g, sms, status, st);
  return launch_x<256, true>(ta, tb, tb_half, p, g, sms, status, st);
}

// ---- few rows -----------------------------------------------------------------------------------
// A handful of assignments read an expert's weights for one row each, and that is all that counts: 2 C
// hidden bf16 an assignment. Two launches without sort or gather: fc1 over (features, assignments), fc2
// over (channels, tokens), which also weights and adds the token's experts and its residual. A warp has
// four weight rows (fc2: two channels of two experts), or its span of them where several warps share
// long rows, in flight at once: up to twenty 16-byte loads a lane and no loop, so that a token of two
// experts at ViT-H widths is on its way from HBM whole, in one wave of blocks, a microsecond after the
// launch. fc2 requests its first weights before it waits for fc1.
constexpr int kVecRows = 4;                    // weight rows of a warp
constexpr int kVecSpan = 5;                    // chunks a lane of each, at most
constexpr int kVecMostK = 8 * 32 * kVecSpan * 8;

// Warps an SM. At five chunks a lane one warp more a scheduler is worth what it spills (C 1280, hidden 5120, one
// token of two experts: 16.6 us, 19.8 with 16 warps: then not all blocks are resident at once); at four it is
// not (9.5 us for four experts of C 768, hidden 2048, 11.3 with 20).
__host__ __device__ constexpr int vec_warps(int V) { return V == kVecSpan ? 20 : 16; }

struct ExpertVec {
  const uint16_t* x;        // fc1: [tokens, ld]; fc2: hidden rows [n, K]
  const int32_t* ids;       // [n]
  const uint16_t *w, *bias; // [E, rows, K], [E, rows]
  uint16_t* out;            // fc1: hidden rows [n, rows]; fc2: [tokens, ld]
  const float* weight;      // fc2: [n] or null
  const uint16_t* residual; // fc2: [tokens, ld] or null
  long long ld;
  int E, topk, rows, K;
  int kw;                   // warps that share a row's K
};

// s[0..3] summed over the warp: lane 8 q (and its seven neighbours) get the sum of s[q].
__device__ __forceinline__ float warp_sum4(const float (&s)[4]) {
  const int lane = threadIdx.x & 31;
  const bool a = lane & 16, b = lane & 8;
  const float x0 = (a ? s[2] : s[0]) + __shfl_xor_sync(0xffffffffu, a ? s[0] : s[2], 16);
  const float x1 = (a ? s[3] : s[1]) + __shfl_xor_sync(0xffffffffu, a ? s[1] : s[3], 16);
  float v = (b ? x1 : x0) + __shfl_xor_sync(0xffffffffu, b ? x0 : x1, 8);
  v += __shfl_xor_sync(0xffffffffu, v, 4);
  v += __shfl_xor_sync(0xffffffffu, v, 2);
  return v + __shfl_xor_sync(0xffffffffu, v, 1);
}

template <int V>
struct VecTile {
  Chunk<Bf16> w[kVecRows][V];
  // The span [first, end) of rows row0 .. row0 + ROWS - 1 of expert e's matrix into w[at ..]; zeros for rows
  // past the last, or without an expert.
  template <int ROWS>
  __device__ __forceinline__ void load(const ExpertVec& g, int e, int row0, int first, int end,
                                       int at) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const uint16_t* from = g.w + ((size_t)e * g.rows + row0 + r) * g.K;
      const bool live = e >= 0 && row0 + r < g.rows;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = first + 32 * v + lane;
        if (live && c < end) chunk_ldg(w[at + r][v], from + c * 8);
        else chunk_zero(w[at + r][v]);
      }
    }
  }
  // The products of w[0], w[1] with x0 and of w[2], w[3] with x1 (their spans), over the warp: the lane's
  // as in warp_sum4.
  template <bool SAME>
  __device__ __forceinline__ float dot(const uint16_t* x0, const uint16_t* x1, int first,
                                       int end) const {
    const int lane = threadIdx.x & 31;
    uint64_t acc[kVecRows] = {};
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = first + 32 * v + lane;
      Chunk<Bf16> xc[2];
      chunk_zero(xc[0]);
      chunk_zero(xc[1]);
      if (c < end) {
        chunk_load(xc[0], x0 + c * 8);
        if (!SAME) chunk_load(xc[1], x1 + c * 8);
      }
      float xf[2][8], wf[8];
      chunk_floats(xc[0], xf[0]);
      if (!SAME) chunk_floats(xc[1], xf[1]);
#pragma unroll
      for (int r = 0; r < kVecRows; ++r) {
        const int h = SAME ? 0 : r / 2;
        chunk_floats(w[r][v], wf);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          acc[r] = f2_fma(f2_pack(wf[2 * q], wf[2 * q + 1]), f2_pack(xf[h][2 * q], xf[h][2 * q + 1]),
                          acc[r]);
      }
    }
    float s[kVecRows];
#pragma unroll
    for (int r = 0; r < kVecRows; ++r) {
      float lo, hi;
      f2_unpack(acc[r], lo, hi);
      s[r] = lo + hi;
    }
    return warp_sum4(s);
  }
};

// The expert of assignment a, or -1 (one out of range is recorded).
__device__ __forceinline__ int vec_expert(const ExpertVec& g, long long a, int* status) {
  const int e = g.ids[a];
  if (e < -1 || e >= g.E) {
    record_bad_index(status);
    return -1;
  }
  return e;
}
__device__ __forceinline__ float vec_bias(const ExpertVec& g, int e, int row) {
  return g.bias ? __uint_as_float((uint32_t)__ldg(g.bias + (size_t)e * g.rows + row) << 16) : 0.f;
}

// hidden[a] = GELU(W1_e x[a / topk] + b1_e), rounded to bf16. WARPS of a block: kw a group of four features.
template <int V, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, vec_warps(V) / WARPS)
    k_expert_vec_fc1(const ExpertVec g, int* status) {
  __shared__ float part[WARPS * kVecRows][WARPS];   // [row][piece]
  griddep_wait();
  griddep_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kw = g.kw, piece = warp % kw, grp = warp / kw;
  const int per_block = WARPS / kw * kVecRows;
  const long long a = blockIdx.y;
  const int e = vec_expert(g, a, status);
  if (e < 0) return;
  const int chunks = g.K / 8, per = (chunks + kw - 1) / kw;
  const int first = piece * per, end = min(chunks, first + per);
  const int row0 = blockIdx.x * per_block + grp * kVecRows;
  VecTile<V> tile;
  tile.template load<kVecRows>(g, e, row0, first, end, 0);
  const int r = threadIdx.x, f = blockIdx.x * per_block + r;
  const bool mine = r < per_block && f < g.rows;
  float z = mine ? vec_bias(g, e, f) : 0.f;
  const uint16_t* x = g.x + a / g.topk * g.ld;
  const float v = tile.template dot<true>(x, x, first, end);
  if ((lane & 7) == 0) part[grp * kVecRows + lane / 8][piece] = v;
  __syncthreads();
  if (!mine) return;
  for (int q = 0; q < kw; ++q) z += part[r][q];
  float unused = 0.f;
  gelu_erf2(z, unused);
  const __nv_bfloat16 h = __float2bfloat16_rn(z);
  g.out[a * g.rows + f] = *reinterpret_cast<const uint16_t*>(&h);
}

// out[t] = residual[t] + sum_j weight[t, j] (W2_e hidden[t, j] + b2_e), the sum in the order of j.
template <int V, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, vec_warps(V) / WARPS)
    k_expert_vec_fc2(const ExpertVec g, int* status) {
  constexpr int kRows = kVecRows / 2;                      // channels of a warp
  __shared__ float part[kMaxTopk][WARPS * kRows][WARPS];   // [expert][row][piece]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kw = g.kw, piece = warp % kw, grp = warp / kw;
  const int per_block = WARPS / kw * kRows;
  const long long t = blockIdx.y;
  const int chunks = g.K / 8, per = (chunks + kw - 1) / kw;
  const int first = piece * per, end = min(chunks, first + per);
  const int row0 = blockIdx.x * per_block + grp * kRows;
  const int r = threadIdx.x, c = blockIdx.x * per_block + r;
  const bool mine = r < per_block && c < g.rows;
  VecTile<V> tile;
  auto load = [&](int j0) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int e = j0 + q < g.topk ? vec_expert(g, t * g.topk + j0 + q, status) : -1;
      tile.template load<kRows>(g, e, row0, first, end, q * kRows);
    }
  };
  // ids and weights were final before fc1 began.
  load(0);
  griddep_wait();
  griddep_launch();
  const float res =
      g.residual && mine ? __uint_as_float((uint32_t)g.residual[t * g.ld + c] << 16) : 0.f;
  for (int j0 = 0; j0 < g.topk; j0 += 2) {
    if (j0 > 0) load(j0);
    const long long a = t * g.topk + j0;
    const float v = tile.template dot<false>(
        g.x + a * g.K, g.x + (j0 + 1 < g.topk ? a + 1 : a) * g.K, first, end);
    const int q = lane >> 4;   // warp_sum4: rows 0, 1 are expert j0's, 2 and 3 the next one's
    if ((lane & 7) == 0 && j0 + q < g.topk)
      part[j0 + q][grp * kRows + ((lane >> 3) & 1)][piece] = v;
  }
  __syncthreads();
  if (!mine) return;
  float acc = 0.f;
  for (int j = 0; j < g.topk; ++j) {
    const long long a = t * g.topk + j;
    const int e = g.ids[a];
    if (e < 0 || e >= g.E) continue;
    float y = 0.f;
    for (int q = 0; q < kw; ++q) y += part[j][r][q];
    acc += (g.weight ? g.weight[a] : 1.f) * (y + vec_bias(g, e, c));
  }
  const __nv_bfloat16 o = __float2bfloat16_rn(acc + res);
  g.out[t * g.ld + c] = *reinterpret_cast<const uint16_t*>(&o);
}

bool expert_vec_fits(long long n, int C, int hidden) {
  return n <= kVecMostAssignments && C <= kVecMostK && hidden <= kVecMostK;
}

cudaError_t launch_expert_vec(bool fc2, const uint16_t* x, long long ld, const int32_t* ids,
                              const float* weight, const uint16_t* residual, const uint16_t* w,
                              const uint16_t* bias, uint16_t* out, int n, int topk, int E, int rows,
                              int K, int* status, cudaStream_t st) {
  ExpertVec g = {};
  g.x = x;
  g.ids = ids;
  g.w = w;
  g.bias = bias;
  g.out = out;
  g.weight = weight;
  g.residual = residual;
  g.ld = ld;
  g.E = E;
  g.topk = topk;
  g.rows = rows;
  g.K = K;
  // The fewest warps a row, which leave the fewest lanes without a chunk.
  const int chunks = K / 8;
  g.kw = 1;
  while (g.kw * 32 * kVecSpan < chunks) g.kw *= 2;
  const int v = ((chunks + g.kw - 1) / g.kw + 31) / 32, warps = g.kw > 4 ? 8 : 4;
  const int per_block = warps / g.kw * (fc2 ? kVecRows / 2 : kVecRows);
  const dim3 grid((rows + per_block - 1) / per_block, fc2 ? n / topk : n);
  auto go = [&](auto k1, auto k2) {
    return launch_pdl(fc2 ? k2 : k1, grid, dim3(warps * 32), 0, st, g, status);
  };
  if (warps == 8) {
    if (v <= 3) return go(k_expert_vec_fc1<3, 8>, k_expert_vec_fc2<3, 8>);
    return go(k_expert_vec_fc1<5, 8>, k_expert_vec_fc2<5, 8>);
  }
  switch (v) {
    case 1: return go(k_expert_vec_fc1<1, 4>, k_expert_vec_fc2<1, 4>);
    case 2: return go(k_expert_vec_fc1<2, 4>, k_expert_vec_fc2<2, 4>);
    case 3: return go(k_expert_vec_fc1<3, 4>, k_expert_vec_fc2<3, 4>);
    case 4: return go(k_expert_vec_fc1<4, 4>, k_expert_vec_fc2<4, 4>);
    default: return go(k_expert_vec_fc1<5, 4>, k_expert_vec_fc2<5, 4>);
  }
}

}  // namespace ss

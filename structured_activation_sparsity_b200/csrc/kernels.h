// Host-side launchers of the library's kernels (internal to the library).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "pattern.h"
#include "sparsesam.h"

namespace ss {

constexpr int kRowCtas = 148;           // CTAs the persistent row kernels are planned for (B200's SMs)
constexpr int kMaxRankTokens = 16384;   // tokens per unit the rank kernel holds in shared memory

// Allows `kernel` `bytes` of dynamic shared memory on the current device (asked of the driver once per
// kernel, device and size).
cudaError_t allow_smem(const void* kernel, int bytes);

// The bounded-wait limit of each source file's kernels (see c_wait_limit_ns), current device.
cudaError_t set_wait_limit_attn(uint64_t ns);
cudaError_t set_wait_limit_mlp(uint64_t ns);
cudaError_t set_wait_limit_norm(uint64_t ns);

// sparsesam_rcmlp's argument checks (same codes, same order) and its workspace bytes in *need.
int rcmlp_validate(const ss_cfg* cfg, const uint16_t* x, int32_t C, int32_t hidden,
                   const uint16_t* w1, const uint16_t* b1, const uint16_t* w2, const uint16_t* b2,
                   const int32_t* keep, int32_t K, size_t* need);

cudaError_t launch_sobel_score(const float* lum, double* score, int B, int H, int W,
                               cudaStream_t st);

// Ranks the unit's tokens by score. With lum non-null the scores are computed from lum (S1 fused
// in) instead of read from `score`, and written to score_out (when non-null).
cudaError_t launch_stripe_rank(const double* score, const float* lum, double* score_out,
                               int window_mode, int B, int Hg, int Wg, int ws, int units, int N,
                               int K, int32_t* perm, int32_t* inv, int32_t* keep,
                               cudaStream_t st);

// score[i] = SplitMix64 output i from `seed`, as a uniform double in [0, 1), i < n.
cudaError_t launch_random_score(double* score, long long n, unsigned long long seed,
                                cudaStream_t st);
// mag[r] = sum over c in order of delta[r, c]^2 in fp64, for rows r < rows of C bf16 (C % 8 == 0).
cudaError_t launch_update_magnitude(const uint16_t* delta, double* mag, long long rows, int C,
                                    cudaStream_t st);

// Gathers q, k, v [U, N, heads, dh] into the block-major permuted layout [U*heads, N, dh].
cudaError_t launch_gather_qkv(const uint16_t* q, const uint16_t* k, const uint16_t* v,
                              const int32_t* perm, uint16_t* qp, uint16_t* kp, uint16_t* vp,
                              int U, int N, int heads, int dh, int b, int* status,
                              cudaStream_t st);

struct AttnParams {
  const int32_t* perm;   // [U, N]
  uint16_t* out;         // [U, N, heads, dh]
  int U, N, heads, L, b, nb, W, g;
  float scale_log2;      // log2(e) / sqrt(dh)
  int sms;               // persistent CTAs to launch (one per SM)
  int whole;             // pair kernel: pairs processed whole (the rest are split)
  int tail_split;        // pair kernel: pieces per split pair
  float* partial;        // per split piece and group, fp32 O [dh][128], m [128], l [128]
  uint16_t* operm;       // pair kernel output: [U*heads, N, dh] in block-major permuted order
  float2* ml;            // null, or [U*heads, N] (block-major): each row's running max m and
                         // sum l of 2^(s*scale_log2 - m) over its kept keys, s = q.k
  // Decomposed relative-position bias (null rel_tab: none; head dim 64). rel_tab [U*heads*N,
  // rel_ld] fp16 in block-major row order: the row's q . Rh[r] * sqrt(dh) at column r <
  // 2*rel_h - 1, then q . Rw[r] * sqrt(dh) from column 2*rel_h - 1 (rel_h x rel_w: the unit
  // grid); the key tiles' one-hot matrices come by the launch's `te` map over [U, npad, 128] fp16;
  // rel_ksteps = the bias MMA's K steps of 16 columns, ceil((rel_h + rel_w) / 16).
  const uint16_t* rel_tab;
  int rel_ld, rel_h, rel_w, rel_ksteps;
};
// Which attention kernel a shape takes, and the scratch beyond the gathered Q, K, V it needs
// (planned for `sms` CTAs).
struct AttnPlan {
  bool pair_kernel;      // the pair kernel (else the short-item kernel)
  int pairs, whole, tail_split;
  size_t partial_bytes;
};
AttnPlan attn_plan(const AttnParams& p, int dh, int sms, bool force_pair = false);
constexpr int kRelPosOneHotCols = 128;   // columns of a one-hot row (Hu + Wu <= 128)
// The relative-position variant's inputs: the tables stacked into rpack [nr, dh] (the bias GEMM's
// B operand) and every key position's one-hot row of E [U, npad, 128] fp16 (1.0 at columns
// Hu-1-kh and Hu+Wu-1-kw; zero rows past N).
cudaError_t launch_relpos_prep(const uint16_t* rel_h, const uint16_t* rel_w, uint16_t* rpack,
                               int dh, int nr, const int32_t* perm, uint16_t* onehot, int U, int N,
                               int npad, int Hu, int Wu, int b, int* status, cudaStream_t st);
// Block-sparse attention over the gathered sequences (tensor maps over [U*heads, N, dh]; the
// tails cover columns 64..79 at head dim 80). The pair kernel writes its output, permuted, through
// `to` / `to_tail` (maps over p.operm laid out like Q), except the rows of split pairs, which
// launch_merge_pieces writes from the pieces' partials; launch_unpermute_out then scatters Op to
// p.out. The short-item kernel writes p.out itself.
cudaError_t launch_attn(const CUtensorMap* tq, const CUtensorMap* tk, const CUtensorMap* tv,
                        const CUtensorMap* tq_tail, const CUtensorMap* tk_tail,
                        const CUtensorMap* to, const CUtensorMap* to_tail, const AttnParams& p,
                        int dh, int* status, cudaStream_t st, const CUtensorMap* te = nullptr);
// Rows of Op for the split pairs: the pieces' (O, m, l) in p.partial combined and normalised
// (nothing when the plan splits no pair).
cudaError_t launch_merge_pieces(const AttnParams& p, int dh, cudaStream_t st);
// out[u, perm[u][p(q)], h, :] = op[u*heads + h, q, :] for every block-major position q.
cudaError_t launch_unpermute_out(const uint16_t* op, const int32_t* perm, uint16_t* out, int U,
                                 int N, int heads, int dh, int b, int* status, cudaStream_t st);

// The partial-token-count variant (prefix tokens before the patch tokens, 2-D RoPE on the patch
// tokens' q and k). q, k, v, out: [U, prefix + N, heads, dh].
constexpr int kMaxPrefix = 4;            // prefix (class) tokens per unit
constexpr int kMaxPrefixHeads = 32;
constexpr size_t kMaxPrefixRowsSmem = 64 * 1024;   // scores of one dense prefix row: prefix + N <= 16384
// Patch tokens (rows prefix + perm[u][p]) into the gathered layout, q and k rotated
// (rope_log2_base = log2 of the RoPE base; 0: none).
cudaError_t launch_gather_rope(const uint16_t* q, const uint16_t* k, const uint16_t* v,
                               const int32_t* perm, uint16_t* qp, uint16_t* kp, uint16_t* vp,
                               int U, int N, int heads, int dh, int b, int prefix, int grid_w,
                               float rope_log2_base, int* status, cudaStream_t st);
// Patch rows: po [U, N, heads, dh] (attention over the kept patch keys, token order) with its
// (m, l) in ml (block-major) merged with the prefix keys, written to out rows prefix + tok.
cudaError_t launch_prefix_merge(const uint16_t* po, const float2* ml, const uint16_t* qp,
                                const uint16_t* k, const uint16_t* v, const int32_t* perm,
                                uint16_t* out, int U, int N, int heads, int dh, int b, int prefix,
                                float scale_log2, int* status, cudaStream_t st);
// Prefix rows: dense attention of each prefix query over all prefix + N keys.
cudaError_t launch_prefix_rows(const uint16_t* q, const uint16_t* k, const uint16_t* v,
                               const uint16_t* kp, const uint16_t* vp, uint16_t* out, int U, int N,
                               int heads, int dh, int prefix, float scale_log2, cudaStream_t st);

// Gathers the kept rows of x [B, T, C] into xk [B*K, C]; zeroes zero[0, nzero). late_wait: keep
// and x are known final at launch (see k_gather_rows), the copy need not wait for the previous
// launch.
cudaError_t launch_gather_rows(const uint16_t* x, const int32_t* keep, uint16_t* xk, int B, int T,
                               int K, int C, int* zero, int nzero, int* status, cudaStream_t st,
                               bool late_wait = false);

// Rows of an encoder block's attention units: row m = u*N + i is token i (enumeration order) of
// unit u. Global blocks: unit u is image u, in raster order. Windowed blocks: the grid is padded
// bottom/right to whole windows of `window` x `window`, unit u = b*windows + w is window w (row-major
// over the padded grid) of image b, its tokens row-major; a token in the padding has no image row.
struct UnitRows {
  int N, T;               // tokens per unit, tokens per image
  int grid_w, grid_h;
  int window;             // 0: global
  int win_per_row, windows;
};
// The image row b*T + t of unit row m, or -1 for a pad token.
__host__ __device__ inline long long unit_row_src(const UnitRows& r, long long m) {
  const long long u = m / r.N;
  const int i = (int)(m - u * r.N);
  if (!r.window) return u * r.T + i;
  const long long b = u / r.windows;
  const int w = (int)(u - b * r.windows);
  const int y = (w / r.win_per_row) * r.window + i / r.window;
  const int x = (w % r.win_per_row) * r.window + i % r.window;
  if (y >= r.grid_h || x >= r.grid_w) return -1;
  return b * r.T + (long long)y * r.grid_w + x;
}

// LayerNorm of rows, bf16 in and out, fp32 statistics: out[m] = (x[src] - mean) / sqrt(var + eps)
// * w + b over the C channels of the source row, or zeros where there is none. keep == null: the
// source of row m < rows is unit_row_src(ur, m) (a block's LN1 over its units, pads zero); else
// it is image m / K's token keep[m] (LN2 over the kept rows; an entry outside the image records
// SS_EINDEX and its row is left unwritten). CTA 0 also zeroes zero[0, nzero).
cudaError_t launch_ln_rows(const uint16_t* x, const uint16_t* w, const uint16_t* b, uint16_t* out,
                           long long rows, int C, const UnitRows& ur, const int32_t* keep, int K,
                           int* zero, int nzero, int* status, cudaStream_t st);

struct GemmEpilogue {
  int kind;                 // 0: out = bf16(GELU(acc + bias)) into out[M, N]
                            // 1: x[b, keep[m], n] = bf16(x + acc + bias)
                            // 2: the q|k|v columns of unit row m into the block-major permuted
                            //    layout: out[which][(u*heads + h)*N + q(inv[m]), d] =
                            //    bf16(acc + bias), q(p) the block-major position of permuted
                            //    position p (pattern block size b, stripe length L)
                            // 3: x[unit_row_src(ur, m), n] = bf16(x + acc + bias), pad rows skipped
                            // 4: out[M, N] = fp16(acc * scale) (the relative-position products)
  const uint16_t* bias;     // [N] or null
  uint16_t* out;            // kind 0; kind 2: gathered Q (K and V follow at which_stride)
  uint16_t* x;              // kind 1: [B, T, N]; kind 3: [B*T, N]
  const int32_t* keep;      // kind 1: [B*K]
  int K_per_image, T;       // kind 1
  const int32_t* inv;       // kind 2: [U*N] permuted position of each unit row
  long long which_stride;   // kind 2: elements from the gathered Q to K (and K to V)
  int heads, dh, C;         // kind 2: C = heads*dh columns per q, k, v
  int b, L;                 // kind 2: the pattern's block size and stripe length
  float scale;              // kind 4
  UnitRows ur;              // kinds 2 (N) and 3
};
// Tile width and k-split of C[M, N] = A[M, Kd] * B[N, Kd]^T for `sms` persistent CTAs.
// tail: without a k-split, the tiles of a last, partial round of units that are each split in two
// along K (two CTAs, finished as a pair), so that round takes half a unit (0: none).
struct GemmPlan {
  int bn, splits, m_tiles, n_tiles, units, tail;
};
GemmPlan gemm_plan(int M, int N, int Kd, int sms);
// Tiles of the tail for `tiles` whole tiles of kb k-blocks over `sms` CTAs (0: no tail).
int gemm_tail(int tiles, int kb, int sms);
// fp32 partial-tile bytes the plan needs (0 without a k-split); plus one int counter per tile.
size_t gemm_partial_bytes(const GemmPlan& p);
// C = A B^T on tcgen05 with the given epilogue. partial / counters: workspace for k-splits
// (counters zero on entry). B must not be written by the launch directly before this one: its
// first tiles are requested before the kernel's dependency wait (weights are the caller's).
cudaError_t launch_gemm(const CUtensorMap* ta, const CUtensorMap* tb, const GemmPlan& p, int M,
                        int N, int Kd, const GemmEpilogue& ep, float* partial, int* counters,
                        int sms, int* status, cudaStream_t st);

// ---- the norms around a block, with its gate, residual scale and residual add ---------------------

constexpr int kMaxNormC = 4096;       // channels of a row: 512 threads of eight hold it
constexpr int kNormMaxCtas = kRowCtas;

struct NormParams {
  const void *y, *x, *gate, *scale, *post_w, *post_b, *pre_w, *pre_b;
  void *x_out, *n;
  float* stats;                        // [rows, 4] or null
  long long rows, rows_per_gate, ld_y, ld_x, ld_n;
  int C, center;                       // center: LayerNorm (else RMS norm)
  float eps;
};
// Up to this many warps of rows the forward takes the direct kernel; a row has `wide` warps (one per 256
// channels, rounded up to a power of two). One wave of it (16 warps an SM), and two for fp32 rows of eight
// warps, whose many-row kernel starts slowest. Measured on B200, direct / many-row, at 2048, 2560 and 4096 warps:
// 16-bit C 64 3.3 / 3.7, 3.2 / 3.7, 4.8 / 3.7 us; C 1280 4.6 / 5.6, 7.4 / 5.6, 8.1 / 5.6; C 4096 6.6 / 10.6,
// 12.2 / 10.6, 12.4 / 10.7; fp32 C 256 3.9 / 3.8, 3.9 / 5.5, 5.9 / 5.7; C 1160 4.9 / 9.7, 8.0 / 9.7, 8.8 / 9.7 (5120:
// 11.9 / 9.7); C 4096 7.6 / 10.5, 14.0 / 10.5, 14.3 / 10.7.
constexpr int kNormDirectWarps = 16 * kRowCtas;
constexpr int norm_direct_warps(bool fp32, int wide) {
  return fp32 && wide == 8 ? 2 * kNormDirectWarps : kNormDirectWarps;
}
cudaError_t launch_norm_residual(const NormParams& p, int dtype, int* status, cudaStream_t st);

struct NormBwdParams {
  const void *y, *x, *gate, *scale, *post_w, *post_b, *pre_w;   // x: the forward's x_out
  const float* stats;
  const void *dx_out, *dn;
  void *dx, *dy;
  float *dgate, *dscale, *dpost_w, *dpost_b, *dpre_w, *dpre_b;  // each may be null
  float* partial;                      // [CTAs][4][C]
  float* gate_partial;                 // [workers][2][C] (with a gate)
  long long rows, rows_per_gate, ld_y, ld_x, ld_n;
  int C, center;
};
// Bytes of the two partials; *gate_offset: where the second begins.
size_t norm_backward_partial(long long rows, int C, int es, bool pre, bool gate,
                             size_t* gate_offset);
// Row gradients and the partial column sums (nothing at rows == 0).
cudaError_t launch_norm_backward(const NormBwdParams& p, int dtype, int* status, cudaStream_t st);
// The parameters' gradients from the partials.
cudaError_t launch_norm_reduce(const NormBwdParams& p, int dtype, cudaStream_t st);

// ---- routed experts --------------------------------------------------------------------------------

constexpr int kMaxExperts = 512;
constexpr int kMaxTopk = 16;
// Assignments one CTA sorts by itself. Measured on B200, one CTA / several: 1024 of 8 experts 3.0 / 4.7 us, 2048
// 3.8 / 4.8, 4096 5.8 / 4.8; of 256 experts 4.5 / 5.7, 6.8 / 6.0, 11.4 / 6.9.
constexpr int kSortOne = 2048;
constexpr int kSortMaxCtas = kRowCtas;

cudaError_t launch_expert_route(const float* logits, int32_t* ids, float* weight, int T, int E,
                                int topk, bool renorm, cudaStream_t st);
cudaError_t launch_expert_route_backward(const float* logits, const int32_t* ids,
                                         const float* weight, const float* dweight, float* dlogits,
                                         int T, int E, int topk, bool renorm, int* status,
                                         cudaStream_t st);
// The sort of n assignments: launch_expert_count (into hist [sort_ctas(n)][E]) when it takes more than one CTA,
// then launch_expert_place.
int sort_ctas(long long n);
cudaError_t launch_expert_count(const int32_t* ids, int32_t* hist, int n, int E, int* status,
                                cudaStream_t st);
cudaError_t launch_expert_place(const int32_t* ids, const int32_t* hist, int32_t* order,
                                int32_t* slot, int32_t* offsets, int n, int E, int* status,
                                cudaStream_t st);
// Rows x, residual, out and dout are ld elements apart; the sorted rows are C apart.
cudaError_t launch_expert_gather(const void* x, const int32_t* slot, void* xs, int tokens,
                                 int topk, int C, long long ld, int dtype, int* status,
                                 cudaStream_t st);
// splits > 0: ys holds that many fp32 partials [tokens * topk, C].
cudaError_t launch_expert_combine(const void* ys, const int32_t* slot, const float* weight,
                                  const void* residual, void* out, int tokens, int topk, int C,
                                  long long ld, int dtype, int splits, int* status,
                                  cudaStream_t st);
cudaError_t launch_expert_combine_backward(const void* dout, const void* ys, const int32_t* slot,
                                           const float* weight, void* dys, float* dweight,
                                           int tokens, int topk, int C, long long ld, int dtype,
                                           int* status, cudaStream_t st);

// One product of all experts: rows [n, Kd] sorted by expert (offsets [E + 1], on the device) times
// W_e [features, Kd]^T. out: bf16 [n, features], with the bias and, if set, the GELU; or partial: fp32
// [splits][n, features], the bias in the first.
struct ExpertGemm {
  const int32_t* offsets;
  const uint16_t* bias;    // [E, features] or null
  uint16_t* out;
  float* partial;
  long long n;
  int E, features, m_tiles, splits, kb_total, gelu;
};
struct ExpertGemmPlan {
  int tn, box;               // rows of a token tile, and of a CTA's box of it
  bool pair;                 // two CTAs a tile of 256 features (else one CTA, 128)
  int m_tiles, splits;       // feature tiles, k-splits
  long long max_units;       // at most
};
ExpertGemmPlan expert_gemm_plan(long long n, int E, int features, int Kd, bool split, int sms);
// Rows of a CTA's token box of a tile of tn rows.
__host__ __device__ constexpr int expert_box(int tn, bool pair) { return pair ? tn / 2 : tn; }
// ta: weights [E * features, Kd], box 128 rows; tb, tb_half: rows [n, Kd], boxes of p.box rows and of half
// as many; all 64 columns.
cudaError_t launch_expert_gemm(const CUtensorMap* ta, const CUtensorMap* tb,
                               const CUtensorMap* tb_half, const ExpertGemmPlan& p,
                               const ExpertGemm& g, int sms, int* status, cudaStream_t st);

// The products of a few assignments, straight from the unsorted tokens (see expert_mlp.cuh): fc1 (x [tokens,
// ld], weights [E, rows, K] -> out: the hidden rows [n, rows]) or fc2 (x: the hidden rows [n, K] -> out
// [tokens, ld], weighted, with the residual).
// Up to this many assignments: their cost grows with each, the products' with each expert that has one.
// Measured on B200, here / sort, gather, products and combine: 8 experts of 1280 - 5120, 2 assignments 16.0 / 29.9
// us, 4 28.8 / 40.4, 8 44.9 / 55.1, 12 63.5 / 55.6, 16 77.5 / 63.2; 64 experts of 768 - 2048, where hardly any share
// an expert, 8 13.5 / 28.8, 12 17.7 / 34.8, 16 26.0 / 36.4, 32 39.4 / 45.1.
constexpr int kVecMostAssignments = 8;
bool expert_vec_fits(long long n, int C, int hidden);
cudaError_t launch_expert_vec(bool fc2, const uint16_t* x, long long ld, const int32_t* ids,
                              const float* weight, const uint16_t* residual, const uint16_t* w,
                              const uint16_t* bias, uint16_t* out, int n, int topk, int E, int rows,
                              int K, int* status, cudaStream_t st);

}  // namespace ss

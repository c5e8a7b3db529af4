// Host side of the C ABI's norm and routed-expert calls (declared in include/sparsesam.h): argument
// validation, workspace carving and the launches.
#include <math.h>

#include "host.h"
#include "kernels.h"

namespace ss {
namespace {

bool dtype_ok(int d) { return d == SS_BF16 || d == SS_F16 || d == SS_F32; }
int dtype_size(int d) { return d == SS_F32 ? 4 : 2; }
// A row stride: 0 stands for the row itself; rows stay 16-byte aligned.
bool stride_ok(int64_t ld, int C) { return ld == 0 || (ld >= C && ld % 8 == 0); }

// ---- norms ------------------------------------------------------------------------------------
int norm_check(const ss_norm_cfg* c) {
  if (!c || c->rows < 0 || c->C < 1) return SS_EINVAL;
  if (!dtype_ok(c->dtype) || (c->norm != SS_LAYERNORM && c->norm != SS_RMSNORM)) return SS_EINVAL;
  if (!(c->eps > 0.f && c->eps < INFINITY) || c->rows_per_gate < 0) return SS_EINVAL;
  if (c->C % 8 != 0 || c->C > kMaxNormC || c->rows >= (int64_t)1 << 31) return SS_EUNSUPPORTED;
  if (!stride_ok(c->ld_y, c->C) || !stride_ok(c->ld_x, c->C) || !stride_ok(c->ld_n, c->C))
    return SS_EINVAL;
  return SS_OK;
}
int64_t or_C(int64_t ld, int C) { return ld ? ld : C; }

// ---- experts ----------------------------------------------------------------------------------
int expert_check(const ss_expert_cfg* c) {
  if (!c || c->tokens < 0 || c->experts < 1 || c->topk < 1 || c->topk > c->experts) return SS_EINVAL;
  if (c->experts > kMaxExperts || c->topk > kMaxTopk) return SS_EUNSUPPORTED;
  if ((int64_t)c->tokens * c->topk >= (int64_t)1 << 30) return SS_EUNSUPPORTED;
  return SS_OK;
}
int expert_rows_check(const ss_expert_cfg* c) {
  int rc = expert_check(c);
  if (rc) return rc;
  if (c->C < 1 || !dtype_ok(c->dtype)) return SS_EINVAL;
  if (c->C % 8 != 0) return SS_EUNSUPPORTED;
  return stride_ok(c->ld, c->C) ? SS_OK : SS_EINVAL;
}

size_t sort_bytes(int64_t n, int E) {
  const int ctas = sort_ctas(n);
  return ctas > 1 ? align256((size_t)ctas * E * sizeof(int32_t)) : 0;
}

int sort_launch(const int32_t* ids, int32_t* order, int32_t* slot, int32_t* offsets, int n, int E,
                void* ws, int* status, cudaStream_t st) {
  int32_t* hist = static_cast<int32_t*>(ws);
  if (sort_ctas(n) > 1) {
    const int rc = cuda_err(traced("expert_count", st, [&] {
      return launch_expert_count(ids, hist, n, E, status, st);
    }));
    if (rc) return rc;
  }
  return cuda_err(traced("expert_place", st, [&] {
    return launch_expert_place(ids, hist, order, slot, offsets, n, E, status, st);
  }));
}

// sparsesam_expert_mlp's workspace: the sort's, the slots and offsets, the sorted rows, the hidden rows,
// and fc2's rows: bf16, or fp32 partials when it is split along K. (Whole rows in fp32 would take the result's
// error from 0.00195 to 0.0018, of which the result's own rounding is 0.00165, and 16384 tokens of two experts
// from 730 to 780 us: twice the bytes to write and to combine.)
struct ExpertMlpLayout {
  ExpertGemmPlan fc1, fc2;
  size_t sort, slot, offsets, xs, h, y, total;
};
void expert_mlp_layout(const ss_expert_cfg* c, ExpertMlpLayout* L) {
  const int64_t n = (int64_t)c->tokens * c->topk;
  L->fc1 = expert_gemm_plan(n, c->experts, c->hidden, c->C, false, kPlanSMs);
  L->fc2 = expert_gemm_plan(n, c->experts, c->C, c->hidden, true, kPlanSMs);
  L->sort = 0;
  L->slot = sort_bytes(n, c->experts);
  L->offsets = L->slot + align256((size_t)n * 4);
  L->xs = L->offsets + align256((size_t)(c->experts + 1) * 4);
  L->h = L->xs + align256((size_t)n * c->C * 2);
  L->y = L->h + align256((size_t)n * c->hidden * 2);
  const size_t y = L->fc2.splits > 1 ? (size_t)L->fc2.splits * n * c->C * 4 : (size_t)n * c->C * 2;
  L->total = L->y + align256(y);
}
int expert_mlp_check(const ss_expert_cfg* c) {
  int rc = expert_rows_check(c);
  if (rc) return rc;
  if (c->hidden < 1) return SS_EINVAL;
  if (c->dtype != SS_BF16 || c->hidden % 8 != 0) return SS_EUNSUPPORTED;
  if ((int64_t)c->experts * c->hidden >= (int64_t)1 << 31 ||
      (int64_t)c->experts * c->C >= (int64_t)1 << 31)
    return SS_EUNSUPPORTED;
  return SS_OK;
}

}  // namespace
}  // namespace ss

using namespace ss;

extern "C" {

int sparsesam_norm_residual(const ss_norm_cfg* cfg, const void* y, const void* x, const void* gate,
                            const void* scale, const void* post_w, const void* post_b,
                            const void* pre_w, const void* pre_b, void* x_out, void* n,
                            float* stats, void* stream) {
  int rc = norm_check(cfg);
  if (rc) return rc;
  if ((pre_w != nullptr) != (n != nullptr) && cfg->rows > 0) return SS_EINVAL;
  if ((post_b && !post_w) || (pre_b && !pre_w) || (gate && cfg->rows_per_gate < 1))
    return SS_EINVAL;
  if (cfg->rows == 0) return SS_OK;
  if (!y || !x || !x_out || n == x_out) return SS_EINVAL;
  // In place over y or x, n's rows have to be theirs: with another stride a row would be written over one
  // that another block has yet to read.
  const int64_t ld_n = or_C(cfg->ld_n, cfg->C);
  if ((n == y && ld_n != or_C(cfg->ld_y, cfg->C)) || (n == x && ld_n != or_C(cfg->ld_x, cfg->C)))
    return SS_EINVAL;
  const void* al[] = {y, x, gate, scale, post_w, post_b, pre_w, pre_b, x_out, n, stats};
  for (const void* a : al)
    if (!aligned(a, 16)) return SS_EINVAL;
  NormParams p = {};
  p.y = y;
  p.x = x;
  p.gate = gate;
  p.scale = scale;
  p.post_w = post_w;
  p.post_b = post_b;
  p.pre_w = pre_w;
  p.pre_b = pre_b;
  p.x_out = x_out;
  p.n = n;
  p.stats = stats;
  p.rows = cfg->rows;
  p.rows_per_gate = gate && cfg->rows_per_gate < cfg->rows ? cfg->rows_per_gate : cfg->rows;
  p.ld_y = or_C(cfg->ld_y, cfg->C);
  p.ld_x = or_C(cfg->ld_x, cfg->C);
  p.ld_n = or_C(cfg->ld_n, cfg->C);
  p.C = cfg->C;
  p.center = cfg->norm == SS_LAYERNORM;
  p.eps = cfg->eps;
  int* status = status_word();
  if (!status) return SS_ECUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return cuda_err(traced("norm_residual", st, [&] {
    return launch_norm_residual(p, cfg->dtype, status, st);
  }));
}

size_t sparsesam_norm_residual_backward_workspace(const ss_norm_cfg* cfg) {
  if (norm_check(cfg) || cfg->rows == 0) return 0;
  // The larger of the layouts with and without a pre norm, with a gate if the rows come in groups.
  size_t most = 0, off;
  for (int pre = 0; pre < 2; ++pre) {
    const size_t b = norm_backward_partial(cfg->rows, cfg->C, dtype_size(cfg->dtype), pre,
                                           cfg->rows_per_gate > 0, &off);
    if (b > most) most = b;
  }
  return most;
}

int sparsesam_norm_residual_backward(const ss_norm_cfg* cfg, const void* y, const void* x_out,
                                     const void* gate, const void* scale, const void* post_w,
                                     const void* post_b, const void* pre_w, const float* stats,
                                     const void* dx_out, const void* dn, void* dx, void* dy,
                                     float* dgate, float* dscale, float* dpost_w, float* dpost_b,
                                     float* dpre_w, float* dpre_b, void* ws, size_t ws_bytes,
                                     void* stream) {
  int rc = norm_check(cfg);
  if (rc) return rc;
  if ((post_b && !post_w) || (gate && cfg->rows_per_gate < 1)) return SS_EINVAL;
  // A gradient is written only of what the call was given.
  if ((dgate && !gate) || (dscale && !scale) || ((dpost_w || dpost_b) && !post_w) ||
      ((dpre_w || dpre_b) && !pre_w))
    return SS_EINVAL;
  if (cfg->rows > 0) {
    if (!y || !dx_out || !dx || !dy || dx == dy || (pre_w != nullptr) != (dn != nullptr) ||
        (pre_w && !x_out) || ((pre_w || post_w) && !stats))
      return SS_EINVAL;
  }
  const void* al[] = {y,  x_out, gate,  scale,  post_w,  post_b,  pre_w,  stats, dx_out, dn,
                      dx, dy,    dgate, dscale, dpost_w, dpost_b, dpre_w, dpre_b};
  for (const void* a : al)
    if (!aligned(a, 16)) return SS_EINVAL;
  size_t gate_off = 0;
  if (cfg->rows > 0) {
    const size_t need = norm_backward_partial(cfg->rows, cfg->C, dtype_size(cfg->dtype),
                                              pre_w != nullptr, gate != nullptr, &gate_off);
    if (!ws || !aligned(ws, 256) || ws_bytes < need) return SS_EWORKSPACE;
  }
  int* status = status_word();
  if (!status) return SS_ECUDA;
  NormBwdParams p = {};
  p.y = y;
  p.x = x_out;
  p.gate = gate;
  p.scale = scale;
  p.post_w = post_w;
  p.post_b = post_b;
  p.pre_w = pre_w;
  p.stats = stats;
  p.dx_out = dx_out;
  p.dn = dn;
  p.dx = dx;
  p.dy = dy;
  p.dgate = dgate;
  p.dscale = dscale;
  p.dpost_w = dpost_w;
  p.dpost_b = dpost_b;
  p.dpre_w = dpre_w;
  p.dpre_b = dpre_b;
  p.partial = static_cast<float*>(ws);
  p.gate_partial =
      gate ? reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + gate_off) : nullptr;
  p.rows = cfg->rows;
  p.rows_per_gate = gate && cfg->rows_per_gate < cfg->rows ? cfg->rows_per_gate : cfg->rows;
  p.ld_y = or_C(cfg->ld_y, cfg->C);
  p.ld_x = or_C(cfg->ld_x, cfg->C);
  p.ld_n = or_C(cfg->ld_n, cfg->C);
  p.C = cfg->C;
  p.center = cfg->norm == SS_LAYERNORM;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cfg->rows > 0) {
    rc = cuda_err(traced("norm_backward", st, [&] {
      return launch_norm_backward(p, cfg->dtype, status, st);
    }));
    if (rc) return rc;
  }
  if (!dgate && !dscale && !dpost_w && !dpost_b && !dpre_w && !dpre_b) return SS_OK;
  return cuda_err(traced("norm_reduce", st, [&] { return launch_norm_reduce(p, cfg->dtype, st); }));
}

int sparsesam_expert_route(const ss_expert_cfg* cfg, const float* logits, int32_t renorm,
                           int32_t* ids, float* weight, void* stream) {
  int rc = expert_check(cfg);
  if (rc) return rc;
  if (cfg->tokens == 0) return SS_OK;
  if (!logits || !ids || !weight) return SS_EINVAL;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return cuda_err(traced("expert_route", st, [&] {
    return launch_expert_route(logits, ids, weight, cfg->tokens, cfg->experts, cfg->topk,
                               renorm != 0, st);
  }));
}

int sparsesam_expert_route_backward(const ss_expert_cfg* cfg, const float* logits, int32_t renorm,
                                    const int32_t* ids, const float* weight, const float* dweight,
                                    float* dlogits, void* stream) {
  int rc = expert_check(cfg);
  if (rc) return rc;
  if (cfg->tokens == 0) return SS_OK;
  if ((!logits && !renorm) || !ids || !weight || !dweight || !dlogits) return SS_EINVAL;
  int* status = status_word();
  if (!status) return SS_ECUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return cuda_err(traced("expert_route_backward", st, [&] {
    return launch_expert_route_backward(logits, ids, weight, dweight, dlogits, cfg->tokens,
                                        cfg->experts, cfg->topk, renorm != 0, status, st);
  }));
}

size_t sparsesam_expert_sort_workspace(const ss_expert_cfg* cfg) {
  if (expert_check(cfg)) return 0;
  return sort_bytes((int64_t)cfg->tokens * cfg->topk, cfg->experts);
}

int sparsesam_expert_sort(const ss_expert_cfg* cfg, const int32_t* ids, int32_t* order,
                          int32_t* slot, int32_t* offsets, void* ws, size_t ws_bytes,
                          void* stream) {
  int rc = expert_check(cfg);
  if (rc) return rc;
  const int n = cfg->tokens * cfg->topk;
  if ((!ids && n > 0) || (!order && !slot && !offsets)) return SS_EINVAL;
  const size_t need = sort_bytes(n, cfg->experts);
  if (need > 0 && (!ws || !aligned(ws, 256) || ws_bytes < need)) return SS_EWORKSPACE;
  int* status = status_word();
  if (!status) return SS_ECUDA;
  return sort_launch(ids, order, slot, offsets, n, cfg->experts, ws, status,
                     static_cast<cudaStream_t>(stream));
}

int sparsesam_expert_gather(const ss_expert_cfg* cfg, const void* x, const int32_t* slot, void* xs,
                            void* stream) {
  int rc = expert_rows_check(cfg);
  if (rc) return rc;
  if (cfg->tokens == 0) return SS_OK;
  if (!x || !slot || !xs || x == xs || !aligned(x, 16) || !aligned(xs, 16)) return SS_EINVAL;
  int* status = status_word();
  if (!status) return SS_ECUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return cuda_err(traced("expert_gather", st, [&] {
    return launch_expert_gather(x, slot, xs, cfg->tokens, cfg->topk, cfg->C,
                                or_C(cfg->ld, cfg->C), cfg->dtype, status, st);
  }));
}

int sparsesam_expert_combine(const ss_expert_cfg* cfg, const void* ys, const int32_t* slot,
                             const float* weight, const void* residual, void* out, void* stream) {
  int rc = expert_rows_check(cfg);
  if (rc) return rc;
  if (cfg->tokens == 0) return SS_OK;
  if (!ys || !slot || !out || ys == out || !aligned(ys, 16) || !aligned(residual, 16) ||
      !aligned(out, 16))
    return SS_EINVAL;
  int* status = status_word();
  if (!status) return SS_ECUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return cuda_err(traced("expert_combine", st, [&] {
    return launch_expert_combine(ys, slot, weight, residual, out, cfg->tokens, cfg->topk, cfg->C,
                                 or_C(cfg->ld, cfg->C), cfg->dtype, 0, status, st);
  }));
}

int sparsesam_expert_combine_backward(const ss_expert_cfg* cfg, const void* dout, const void* ys,
                                      const int32_t* slot, const float* weight, void* dys,
                                      float* dweight, void* stream) {
  int rc = expert_rows_check(cfg);
  if (rc) return rc;
  if (cfg->tokens == 0) return SS_OK;
  if (!dout || !ys || !slot || !weight || !dys || !dweight || dout == dys || !aligned(dout, 16) ||
      !aligned(ys, 16) || !aligned(dys, 16))
    return SS_EINVAL;
  int* status = status_word();
  if (!status) return SS_ECUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return cuda_err(traced("expert_combine_backward", st, [&] {
    return launch_expert_combine_backward(dout, ys, slot, weight, dys, dweight, cfg->tokens,
                                          cfg->topk, cfg->C, or_C(cfg->ld, cfg->C), cfg->dtype,
                                          status, st);
  }));
}

size_t sparsesam_expert_mlp_workspace(const ss_expert_cfg* cfg) {
  if (expert_mlp_check(cfg) || cfg->tokens == 0) return 0;
  ExpertMlpLayout L;
  expert_mlp_layout(cfg, &L);
  return L.total;
}

int sparsesam_expert_mlp(const ss_expert_cfg* cfg, const uint16_t* x, const int32_t* ids,
                         const float* weight, const uint16_t* residual, const uint16_t* w1,
                         const uint16_t* b1, const uint16_t* w2, const uint16_t* b2,
                         uint16_t* out, void* ws, size_t ws_bytes, void* stream) {
  int rc = expert_mlp_check(cfg);
  if (rc) return rc;
  if (cfg->tokens == 0) return SS_OK;
  if (!x || !ids || !w1 || !w2 || !out) return SS_EINVAL;
  const void* al[] = {x, residual, w1, w2, out};
  for (const void* a : al)
    if (!aligned(a, 16)) return SS_EINVAL;
  ExpertMlpLayout L;
  expert_mlp_layout(cfg, &L);
  if (!ws || !aligned(ws, 256) || ws_bytes < L.total) return SS_EWORKSPACE;
  int* status = status_word();
  if (!status) return SS_ECUDA;
  const int E = cfg->experts, C = cfg->C, H = cfg->hidden, n = cfg->tokens * cfg->topk;
  uint8_t* wsb = static_cast<uint8_t*>(ws);
  int32_t* slot = reinterpret_cast<int32_t*>(wsb + L.slot);
  int32_t* offsets = reinterpret_cast<int32_t*>(wsb + L.offsets);
  uint16_t* xs = reinterpret_cast<uint16_t*>(wsb + L.xs);
  uint16_t* h = reinterpret_cast<uint16_t*>(wsb + L.h);
  void* y = wsb + L.y;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (expert_vec_fits(n, C, H)) {
    rc = cuda_err(traced("expert_vec_fc1", st, [&] {
      return launch_expert_vec(false, x, or_C(cfg->ld, C), ids, nullptr, nullptr, w1, b1, h, n,
                               cfg->topk, E, H, C, status, st);
    }));
    if (rc) return rc;
    return cuda_err(traced("expert_vec_fc2", st, [&] {
      return launch_expert_vec(true, h, or_C(cfg->ld, C), ids, weight, residual, w2, b2, out, n,
                               cfg->topk, E, C, H, status, st);
    }));
  }
  CUtensorMap tw1, tx, tx_half, tw2, th, th_half;
  const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
  if (!encode_bf16(&tw1, 2, w1, C, (uint64_t)E * H, 1, (uint64_t)C * 2, 64, 128, sw) ||
      !encode_bf16(&tx, 2, xs, C, n, 1, (uint64_t)C * 2, 64, L.fc1.box, sw) ||
      !encode_bf16(&tx_half, 2, xs, C, n, 1, (uint64_t)C * 2, 64, L.fc1.box / 2, sw) ||
      !encode_bf16(&tw2, 2, w2, H, (uint64_t)E * C, 1, (uint64_t)H * 2, 64, 128, sw) ||
      !encode_bf16(&th, 2, h, H, n, 1, (uint64_t)H * 2, 64, L.fc2.box, sw) ||
      !encode_bf16(&th_half, 2, h, H, n, 1, (uint64_t)H * 2, 64, L.fc2.box / 2, sw))
    return SS_ECUDA;
  if ((rc = sort_launch(ids, nullptr, slot, offsets, n, E, wsb + L.sort, status, st))) return rc;
  rc = cuda_err(traced("expert_gather", st, [&] {
    return launch_expert_gather(x, slot, xs, cfg->tokens, cfg->topk, C, or_C(cfg->ld, C), SS_BF16,
                                status, st);
  }));
  if (rc) return rc;
  ExpertGemm g = {};
  g.offsets = offsets;
  g.n = n;
  g.E = E;
  g.bias = b1;
  g.out = h;
  g.features = H;
  g.m_tiles = L.fc1.m_tiles;
  g.splits = L.fc1.splits;
  g.kb_total = (C + 63) / 64;
  g.gelu = 1;
  rc = cuda_err(traced("expert_fc1", st, [&] {
    return launch_expert_gemm(&tw1, &tx, &tx_half, L.fc1, g, sm_count(), status, st);
  }));
  if (rc) return rc;
  const int splits = L.fc2.splits;
  g.bias = b2;
  g.out = splits > 1 ? nullptr : static_cast<uint16_t*>(y);
  g.partial = splits > 1 ? static_cast<float*>(y) : nullptr;
  g.features = C;
  g.m_tiles = L.fc2.m_tiles;
  g.splits = splits;
  g.kb_total = (H + 63) / 64;
  g.gelu = 0;
  rc = cuda_err(traced("expert_fc2", st, [&] {
    return launch_expert_gemm(&tw2, &th, &th_half, L.fc2, g, sm_count(), status, st);
  }));
  if (rc) return rc;
  return cuda_err(traced("expert_combine", st, [&] {
    return launch_expert_combine(y, slot, weight, residual, out, cfg->tokens, cfg->topk, C,
                                 or_C(cfg->ld, C), SS_BF16, splits > 1 ? splits : 0, status, st);
  }));
}

}  // extern "C"

// forge_layer_host.cpp -- the C ABI declared in include/forge_layer.h: argument checks (before any
// HIP call), the packed table of the step over many tensors, and dispatch.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>
#include <vector>

#include "forge.h"
#include "forge_host_common.h"
#include "forge_layer.h"
#include "forge_layer_internal.h"

using namespace forge::host;

namespace {

// Ranges of one call: written ones overlap nothing, except pairs named as allowed in place.
struct Ranges {
  Range r[16];
  bool written[16];
  int n = 0;
  void add(const void* p, int64_t bytes, const char* name, bool w) {
    r[n] = range_of(p, bytes, name);
    written[n++] = w;
  }
  void add(const forge_tensor* t, const char* name, bool w) { add(t->data, bytes_of(t), name, w); }
  // may: written range i may be exactly range j
  template <class May>
  forge_status check(May&& may) const {
    for (int i = 0; i < n; ++i)
      for (int j = 0; j < n; ++j) {
        if (i == j || !written[i] || (written[j] && j < i)) continue;
        if (!overlap(r[i], r[j])) continue;
        if (r[i].lo == r[j].lo && r[i].hi == r[j].hi && may(r[i].name, r[j].name)) continue;
        return fail(FORGE_ERR_ALIAS, "%s overlaps %s", r[i].name, r[j].name);
      }
    return FORGE_OK;
  }
};
bool never(const char*, const char*) { return false; }

bool is_stream(int32_t dt) { return dt == FORGE_F32 || dt == FORGE_BF16; }

forge_status check_shape(const forge_tensor* t, int64_t rows, int64_t cols, const char* name) {
  if (t->rows != rows || t->cols != cols)
    return fail(FORGE_ERR_SHAPE, "%s is [%lld, %lld], expected [%lld, %lld]", name, (long long)t->rows,
                (long long)t->cols, (long long)rows, (long long)cols);
  return FORGE_OK;
}

forge_status check_gain(const forge_tensor* gain, int64_t D) {
  forge_status st;
  if ((st = check_tensor(gain, "gain")) != FORGE_OK) return st;
  if ((st = check_shape(gain, 1, D, "gain")) != FORGE_OK) return st;
  if (!is_stream(gain->dtype)) return fail(FORGE_ERR_DTYPE, "gain must be F32 or BF16");
  return FORGE_OK;
}

forge_status check_norm_size(int64_t T, int64_t D) {
  if (D < 1 || D >= (int64_t(1) << 31)) return fail(FORGE_ERR_SHAPE, "the width must be 1 .. 2^31 - 1 (got %lld)", (long long)D);
  if (T >= (int64_t(1) << 31)) return fail(FORGE_ERR_SHAPE, "more than 2^31 - 1 rows");
  return FORGE_OK;
}

}  // namespace

extern "C" {

// ------------------------------------------------------------------ RMS norm
forge_status forge_rmsnorm(const forge_tensor* x, const forge_tensor* residual, const forge_tensor* gain, float eps,
                           forge_tensor* h, forge_tensor* y, int32_t scale_mode, float* rstd, float* amax,
                           void* stream) {
  clear_error();
  forge_status st;
  if ((st = check_tensor(x, "x")) != FORGE_OK) return st;
  if (!is_stream(x->dtype)) return fail(FORGE_ERR_DTYPE, "x must be F32 or BF16");
  const int64_t T = x->rows, D = x->cols;
  if ((st = check_norm_size(T, D)) != FORGE_OK) return st;
  if ((st = check_gain(gain, D)) != FORGE_OK) return st;
  if (!(eps >= 0.0f && std::isfinite(eps))) return fail(FORGE_ERR_ARG, "eps must be finite and >= 0");
  if ((residual != nullptr) != (h != nullptr)) return fail(FORGE_ERR_ARG, "residual and h go together: both or neither");
  Ranges rs;
  rs.add(x, "x", false);
  rs.add(gain, "gain", false);
  if (residual) {
    if ((st = check_tensor(residual, "residual")) != FORGE_OK) return st;
    if ((st = check_tensor(h, "h")) != FORGE_OK) return st;
    if ((st = check_shape(residual, T, D, "residual")) != FORGE_OK) return st;
    if ((st = check_shape(h, T, D, "h")) != FORGE_OK) return st;
    if (residual->dtype != x->dtype || h->dtype != x->dtype)
      return fail(FORGE_ERR_DTYPE, "residual and h must have the dtype of x");
    rs.add(residual, "residual", false);
    rs.add(h, "h", true);
  }
  if ((st = check_tensor(y, "y")) != FORGE_OK) return st;
  if ((st = check_shape(y, T, D, "y")) != FORGE_OK) return st;
  rs.add(y, "y", true);
  int y_type;
  if (y->dtype == FORGE_F32) y_type = forge::FORGE_Y_F32;
  else if (y->dtype == FORGE_BF16) y_type = forge::FORGE_Y_BF16;
  else if (y->dtype == FORGE_FP8_E4M3) {
    if (scale_mode != FORGE_SCALE_ROW && scale_mode != FORGE_SCALE_TENSOR)
      return fail(FORGE_ERR_ARG, "unknown scale mode %d", (int)scale_mode);
    if (!y->scale) return fail(FORGE_ERR_ARG, "an fp8 y needs y->scale");
    if (!aligned4(y->scale)) return fail(FORGE_ERR_LAYOUT, "y->scale is not 4-byte aligned");
    const bool row = scale_mode == FORGE_SCALE_ROW;
    y_type = row ? forge::FORGE_Y_FP8_ROW : forge::FORGE_Y_FP8_TENSOR;
    rs.add(y->scale, row ? 4 * T : 4, "y scale", row);
  } else {
    return fail(FORGE_ERR_DTYPE, "y must be F32, BF16 or FP8_E4M3");
  }
  if (rstd) {
    if (!aligned4(rstd)) return fail(FORGE_ERR_LAYOUT, "rstd is not 4-byte aligned");
    rs.add(rstd, 4 * T, "rstd", true);
  }
  if (amax) {
    if (!aligned4(amax)) return fail(FORGE_ERR_LAYOUT, "amax is not 4-byte aligned");
    rs.add(amax, 4, "amax", true);
  }
  st = rs.check([](const char* w, const char* r) {
    return std::strcmp(w, "h") == 0 && (std::strcmp(r, "x") == 0 || std::strcmp(r, "residual") == 0);
  });
  if (st != FORGE_OK) return st;
  if (T == 0) return FORGE_OK;
  if ((st = device_ok()) != FORGE_OK) return st;
  forge::NormArgs a{};
  a.x = x->data;
  a.res = residual ? residual->data : nullptr;
  a.gain = gain->data;
  a.h = h ? h->data : nullptr;
  a.y = y->data;
  a.y_scale = static_cast<float*>(y->scale);
  a.rstd = rstd;
  a.amax = amax;
  a.T = T;
  a.D = (int32_t)D;
  a.eps = eps;
  a.gain_bf16 = gain->dtype == FORGE_BF16;
  return to_status(forge::launch_rmsnorm(x->dtype == FORGE_BF16, y_type, a, stream));
}

int64_t forge_rmsnorm_backward_workspace_bytes(int64_t T, int64_t D) {
  if (T < 0 || D < 0 || T >= (int64_t(1) << 31) || D >= (int64_t(1) << 31)) return -1;
  return forge::norm_bwd_groups(T) * D * 4;
}

forge_status forge_rmsnorm_backward(const forge_tensor* dy, const forge_tensor* dh, const forge_tensor* h,
                                    const forge_tensor* gain, const float* rstd, forge_tensor* dx,
                                    forge_tensor* dgain, void* workspace, int64_t workspace_bytes, void* stream) {
  clear_error();
  forge_status st;
  if ((st = check_tensor(dy, "dy")) != FORGE_OK) return st;
  if (!is_stream(dy->dtype)) return fail(FORGE_ERR_DTYPE, "dy must be F32 or BF16");
  const int64_t T = dy->rows, D = dy->cols;
  if ((st = check_norm_size(T, D)) != FORGE_OK) return st;
  if ((st = check_gain(gain, D)) != FORGE_OK) return st;
  if ((st = check_tensor(h, "h")) != FORGE_OK) return st;
  if ((st = check_tensor(dx, "dx")) != FORGE_OK) return st;
  if (dh && (st = check_tensor(dh, "dh")) != FORGE_OK) return st;
  if ((st = check_shape(h, T, D, "h")) != FORGE_OK) return st;
  if ((st = check_shape(dx, T, D, "dx")) != FORGE_OK) return st;
  if (dh && (st = check_shape(dh, T, D, "dh")) != FORGE_OK) return st;
  if (h->dtype != dy->dtype || dx->dtype != dy->dtype || (dh && dh->dtype != dy->dtype))
    return fail(FORGE_ERR_DTYPE, "dy, dh, h and dx must have the same dtype");
  if (!rstd && T > 0) return fail(FORGE_ERR_ARG, "rstd is NULL");
  if (!aligned4(rstd)) return fail(FORGE_ERR_LAYOUT, "rstd is not 4-byte aligned");
  Ranges rs;
  rs.add(dy, "dy", false);
  if (dh) rs.add(dh, "dh", false);
  rs.add(h, "h", false);
  rs.add(gain, "gain", false);
  rs.add(rstd, 4 * T, "rstd", false);
  rs.add(dx, "dx", true);
  if (dgain) {
    if ((st = check_tensor(dgain, "dgain")) != FORGE_OK) return st;
    if ((st = check_shape(dgain, 1, D, "dgain")) != FORGE_OK) return st;
    if (dgain->dtype != FORGE_F32) return fail(FORGE_ERR_DTYPE, "dgain must be F32");
    rs.add(dgain, "dgain", true);
    const int64_t need = forge_rmsnorm_backward_workspace_bytes(T, D);
    if (!workspace) return fail(FORGE_ERR_ARG, "workspace is NULL");
    if (!aligned16(workspace)) return fail(FORGE_ERR_LAYOUT, "workspace is not 16-byte aligned");
    if (workspace_bytes < need)
      return fail(FORGE_ERR_ARG, "workspace has %lld bytes, the call needs %lld", (long long)workspace_bytes,
                  (long long)need);
    rs.add(workspace, need, "workspace", true);
  }
  st = rs.check([](const char* w, const char* r) {
    return std::strcmp(w, "dx") == 0 && (std::strcmp(r, "dy") == 0 || std::strcmp(r, "dh") == 0);
  });
  if (st != FORGE_OK) return st;
  if (T == 0 && !dgain) return FORGE_OK;
  if ((st = device_ok()) != FORGE_OK) return st;
  forge::NormBwdArgs a{};
  a.dy = dy->data;
  a.dh = dh ? dh->data : nullptr;
  a.h = h->data;
  a.gain = gain->data;
  a.rstd = rstd;
  a.dx = dx->data;
  a.dgain = dgain ? static_cast<float*>(dgain->data) : nullptr;
  a.partial = static_cast<float*>(workspace);
  a.T = T;
  a.D = (int32_t)D;
  a.gain_bf16 = gain->dtype == FORGE_BF16;
  return to_status(forge::launch_rmsnorm_backward(dy->dtype == FORGE_BF16, a, stream));
}

// ------------------------------------------------------------------ products grouped by expert
static forge_status check_groups(const int32_t* ends, int32_t n_groups, int64_t T, int64_t N, int64_t K) {
  if (n_groups < 1 || n_groups > 4096) return fail(FORGE_ERR_ARG, "n_groups must be 1 .. 4096 (got %d)", (int)n_groups);
  if (!ends) return fail(FORGE_ERR_ARG, "ends is NULL");
  if (!aligned4(ends)) return fail(FORGE_ERR_LAYOUT, "ends is not 4-byte aligned");
  if (N < 128 || K < 128 || N % 128 || K % 128)
    return fail(FORGE_ERR_SHAPE, "N = %lld and K = %lld must be positive multiples of 128", (long long)N, (long long)K);
  if (N > (1 << 20) || K > (1 << 20) || N * K >= (int64_t(1) << 31))
    return fail(FORGE_ERR_SHAPE, "N and K must be at most 2^20 and N * K below 2^31");
  if (T >= (int64_t(1) << 31) - 256) return fail(FORGE_ERR_SHAPE, "T must be below 2^31 - 256");
  return FORGE_OK;
}

// Y = A W^T (nn = false: A [T, K], O = N) or A W (nn = true: A [T, N], O = K) by group.
static forge_status grouped_rows(const forge_tensor* A, const forge_tensor* W, const int32_t* ends, int32_t n_groups,
                                 forge_tensor* out, bool nn, void* stream) {
  clear_error();
  const char* an = nn ? "dY" : "X";
  const char* on = nn ? "dX" : "Y";
  forge_status st;
  if ((st = check_tensor(A, an)) != FORGE_OK) return st;
  if ((st = check_tensor(W, "W")) != FORGE_OK) return st;
  if ((st = check_tensor(out, on)) != FORGE_OK) return st;
  const int64_t T = A->rows, N = nn ? A->cols : out->cols, K = nn ? out->cols : A->cols;
  if ((st = check_groups(ends, n_groups, T, N, K)) != FORGE_OK) return st;
  if ((st = check_shape(W, n_groups * N, K, "W")) != FORGE_OK) return st;
  if ((st = check_shape(out, T, nn ? K : N, on)) != FORGE_OK) return st;
  const bool fp8 = !nn && A->dtype == FORGE_FP8_E4M3;
  if (A->dtype != W->dtype || out->dtype != FORGE_BF16 || (A->dtype != FORGE_BF16 && !fp8))
    return fail(FORGE_ERR_DTYPE, nn ? "the grouped dgrad takes BF16 dY and W and writes BF16 dX"
                                    : "the grouped product takes X and W both BF16 or both FP8_E4M3 and writes BF16 Y");
  Ranges rs;
  rs.add(A, an, false);
  rs.add(W, "W", false);
  rs.add(ends, 4 * (int64_t)n_groups, "ends", false);
  rs.add(out, on, true);
  if (fp8) {
    if (!A->scale || !W->scale) return fail(FORGE_ERR_ARG, "fp8 operands need their row scales");
    if (!aligned4(A->scale) || !aligned4(W->scale)) return fail(FORGE_ERR_LAYOUT, "a row scale is not 4-byte aligned");
    rs.add(A->scale, 4 * T, "X scales", false);
    rs.add(W->scale, 4 * n_groups * N, "W scales", false);
  }
  if ((st = rs.check(never)) != FORGE_OK) return st;
  if ((T / 64 + n_groups + 1) * ((out->cols + 255) / 256) >= (int64_t(1) << 31))
    return fail(FORGE_ERR_SHAPE, "too many tiles");
  if (T == 0) return FORGE_OK;
  if ((st = device_ok()) != FORGE_OK) return st;
  forge::GroupedArgs a{};
  a.A = A->data;
  a.W = W->data;
  a.out = out->data;
  a.a_scale = fp8 ? static_cast<const float*>(A->scale) : nullptr;
  a.w_scale = fp8 ? static_cast<const float*>(W->scale) : nullptr;
  a.ends = ends;
  a.E = n_groups;
  a.T = T;
  a.N = N;
  a.K = K;
  const int mode = nn ? forge::FORGE_GROUPED_NN : fp8 ? forge::FORGE_GROUPED_NT8 : forge::FORGE_GROUPED_NT;
  return to_status(forge::launch_grouped_rows(mode, a, stream));
}

forge_status forge_grouped_gemm(const forge_tensor* X, const forge_tensor* W, const int32_t* ends, int32_t n_groups,
                                forge_tensor* Y, void* stream) {
  return grouped_rows(X, W, ends, n_groups, Y, false, stream);
}

forge_status forge_grouped_dgrad(const forge_tensor* dY, const forge_tensor* W, const int32_t* ends, int32_t n_groups,
                                 forge_tensor* dX, void* stream) {
  return grouped_rows(dY, W, ends, n_groups, dX, true, stream);
}

// X, dY and the groups of the weight gradient.
static forge_status check_wgrad(const forge_tensor* X, const forge_tensor* dY, const int32_t* ends, int32_t n_groups,
                                forge::GroupedWgradArgs* a, Ranges* rs) {
  forge_status st;
  if ((st = check_tensor(X, "X")) != FORGE_OK) return st;
  if ((st = check_tensor(dY, "dY")) != FORGE_OK) return st;
  if (X->dtype != FORGE_BF16 || dY->dtype != FORGE_BF16) return fail(FORGE_ERR_DTYPE, "X and dY must be BF16");
  if (X->rows != dY->rows)
    return fail(FORGE_ERR_SHAPE, "X has %lld tokens, dY has %lld", (long long)X->rows, (long long)dY->rows);
  const int64_t T = X->rows, N = dY->cols, K = X->cols;
  if ((st = check_groups(ends, n_groups, T, N, K)) != FORGE_OK) return st;
  // a group's rows are addressed with 32-bit byte offsets (one spare slab of tokens included)
  if ((T + 128) * K * 2 >= (int64_t(1) << 32) || (T + 128) * N * 2 >= (int64_t(1) << 32))
    return fail(FORGE_ERR_SHAPE, "X and dY must each stay below 4 GiB");
  if (n_groups * N >= (int64_t(1) << 31) || n_groups * (N / 128 + 1) * (K / 128) >= (int64_t(1) << 31))
    return fail(FORGE_ERR_SHAPE, "too many tiles");
  rs->add(X, "X", false);
  rs->add(dY, "dY", false);
  rs->add(ends, 4 * (int64_t)n_groups, "ends", false);
  a->X = X->data;
  a->dY = dY->data;
  a->ends = ends;
  a->E = n_groups;
  a->T = T;
  a->N = N;
  a->K = K;
  return FORGE_OK;
}

forge_status forge_grouped_wgrad(const forge_tensor* X, const forge_tensor* dY, const int32_t* ends, int32_t n_groups,
                                 forge_tensor* dW, void* stream) {
  clear_error();
  forge::GroupedWgradArgs a{};
  Ranges rs;
  forge_status st;
  if ((st = check_wgrad(X, dY, ends, n_groups, &a, &rs)) != FORGE_OK) return st;
  if ((st = check_tensor(dW, "dW")) != FORGE_OK) return st;
  if (dW->dtype != FORGE_F32) return fail(FORGE_ERR_DTYPE, "dW must be F32");
  if ((st = check_shape(dW, n_groups * a.N, a.K, "dW")) != FORGE_OK) return st;
  rs.add(dW, "dW", true);
  if ((st = rs.check(never)) != FORGE_OK) return st;
  if ((st = device_ok()) != FORGE_OK) return st;
  return to_status(forge::launch_grouped_wgrad(a, static_cast<float*>(dW->data), stream));
}

forge_status forge_grouped_wgrad_step(const forge_tensor* X, const forge_tensor* dY, const int32_t* ends,
                                      int32_t n_groups, forge_tensor* W, forge_tensor* m, forge_tensor* v,
                                      const forge_hyper* hyper, int32_t opt, int64_t step, uint64_t seed,
                                      const forge_step_opts* opts, void* stream) {
  clear_error();
  forge::GroupedWgradArgs a{};
  Ranges rs;
  forge_status st;
  if ((st = check_wgrad(X, dY, ends, n_groups, &a, &rs)) != FORGE_OK) return st;
  StepPlan plan;
  Range outs[6];
  int n_out = 0;
  if ((st = validate_step_outputs(n_groups * a.N, a.K, W, m, v, hyper, opt, step, seed, opts, &plan, outs, &n_out)) !=
      FORGE_OK)
    return st;
  if (W->dtype != FORGE_BF16) return fail(FORGE_ERR_DTYPE, "W must be BF16");
  for (int i = 0; i < n_out; ++i)
    for (int j = 0; j < rs.n; ++j)
      if (overlap(outs[i], rs.r[j])) return fail(FORGE_ERR_ALIAS, "%s overlaps %s", outs[i].name, rs.r[j].name);
  if ((st = device_ok()) != FORGE_OK) return st;
  return to_status(forge::launch_grouped_step(plan.s_type, opt, a, plan.e, stream));
}

// ------------------------------------------------------------------ the step over many tensors
static int64_t multi_chunks(int64_t n) { return (n + forge::kMultiChunk - 1) / forge::kMultiChunk; }

int64_t forge_multi_table_bytes(const forge_multi_tensor* tensors, int32_t n_tensors) {
  if (n_tensors < 0 || (n_tensors > 0 && !tensors)) return -1;
  int64_t chunks = 0;
  for (int32_t i = 0; i < n_tensors; ++i) {
    if (tensors[i].n < 0 || tensors[i].n > (int64_t(1) << 32) - 8192) return -1;
    chunks += multi_chunks(tensors[i].n);
    if (chunks >= forge::kMultiMaxChunks) return -1;
  }
  return (int64_t)n_tensors * (int64_t)sizeof(forge::MultiEntry) + 4 * chunks;
}

forge_status forge_multi_pack(const forge_multi_tensor* tensors, int32_t n_tensors, int32_t opt, int32_t m_dtype,
                              int32_t v_dtype, void* table, int64_t table_bytes, forge_multi_info* info) {
  clear_error();
  if (!info) return fail(FORGE_ERR_ARG, "info is NULL");
  if (opt < FORGE_ADAMW || opt > FORGE_SGD_MOMENTUM) return fail(FORGE_ERR_ARG, "unknown optimizer %d", (int)opt);
  const bool hm = rule_has_m(opt), hv = rule_has_v(opt);
  if (!hm) m_dtype = -1;
  if (!hv) v_dtype = -1;
  int s_type = -1;
  for (int which = 0; which < 2; ++which) {
    const int32_t dt = which ? v_dtype : m_dtype;
    if (which ? !hv : !hm) continue;
    int ty;
    if (dt == FORGE_F32) ty = forge::FORGE_S_F32;
    else if (dt == (which ? FORGE_U8_B64 : FORGE_I8_B64)) ty = forge::FORGE_S_Q8;
    else if (dt == (which ? FORGE_U8DYN_B64 : FORGE_I8DYN_B64)) ty = forge::FORGE_S_Q8D;
    else return fail(FORGE_ERR_DTYPE, "unsupported dtype %d of %s", (int)dt, which ? "v" : "m");
    if (s_type >= 0 && ty != s_type) return fail(FORGE_ERR_DTYPE, "m and v must both be fp32 or use the same 8-bit map");
    s_type = ty;
  }
  const bool q8 = s_type > forge::FORGE_S_F32;
  const int64_t need = forge_multi_table_bytes(tensors, n_tensors);
  if (need < 0) return fail(FORGE_ERR_SHAPE, "a tensor's n is negative or too large, or there are too many elements");
  if (need > 0 && !table) return fail(FORGE_ERR_ARG, "table is NULL");
  if (table_bytes < need)
    return fail(FORGE_ERR_ARG, "table has %lld bytes, the tensors need %lld", (long long)table_bytes, (long long)need);
  int32_t groups = 0;
  // every range, sorted by address: written ones may overlap nothing
  struct Span {
    Range r;
    bool written;
    int32_t tensor;
  };
  std::vector<Span> spans;
  try {
    spans.reserve((size_t)n_tensors * 6);
    for (int32_t i = 0; i < n_tensors; ++i) {
      const forge_multi_tensor& t = tensors[i];
      if (!is_stream(t.w_dtype) || !is_stream(t.g_dtype))
        return fail(FORGE_ERR_DTYPE, "tensor %d: W and g must be F32 or BF16", (int)i);
      if (t.group < 0 || t.group >= forge::kMultiGroups)
        return fail(FORGE_ERR_ARG, "tensor %d: group must be 0 .. %d", (int)i, forge::kMultiGroups - 1);
      if (t.reserved != 0) return fail(FORGE_ERR_ARG, "tensor %d: reserved must be 0", (int)i);
      groups = std::max(groups, t.group + 1);
      if ((t.m != nullptr || t.m_scale != nullptr) && !hm) return fail(FORGE_ERR_ARG, "tensor %d: this rule keeps no m", (int)i);
      if ((t.v != nullptr || t.v_scale != nullptr) && !hv) return fail(FORGE_ERR_ARG, "tensor %d: this rule keeps no v", (int)i);
      if ((t.m_scale || t.v_scale) && !q8) return fail(FORGE_ERR_ARG, "tensor %d: fp32 moments take no scales", (int)i);
      if (t.n == 0) continue;
      if (!t.W || !t.g || (hm && !t.m) || (hv && !t.v) || (q8 && ((hm && !t.m_scale) || (hv && !t.v_scale))))
        return fail(FORGE_ERR_ARG, "tensor %d: a pointer is NULL", (int)i);
      if (!aligned16(t.W) || !aligned16(t.g) || !aligned16(t.m) || !aligned16(t.v))
        return fail(FORGE_ERR_LAYOUT, "tensor %d: a pointer is not 16-byte aligned", (int)i);
      if (!aligned4(t.m_scale) || !aligned4(t.v_scale))
        return fail(FORGE_ERR_LAYOUT, "tensor %d: a scale is not 4-byte aligned", (int)i);
      const int64_t sb = (t.n + 63) / 64 * 4, ms = q8 ? 1 : 4;
      spans.push_back({range_of(t.W, t.n * dtype_size(t.w_dtype), "W"), true, i});
      spans.push_back({range_of(t.g, t.n * dtype_size(t.g_dtype), "g"), false, i});
      if (hm) spans.push_back({range_of(t.m, t.n * ms, "m"), true, i});
      if (hv) spans.push_back({range_of(t.v, t.n * ms, "v"), true, i});
      if (q8 && hm) spans.push_back({range_of(t.m_scale, sb, "m scales"), true, i});
      if (q8 && hv) spans.push_back({range_of(t.v_scale, sb, "v scales"), true, i});
    }
    std::sort(spans.begin(), spans.end(), [](const Span& a, const Span& b) { return a.r.lo < b.r.lo; });
  } catch (const std::bad_alloc&) {
    return fail(FORGE_ERR_ARG, "out of host memory for %d tensors", (int)n_tensors);
  }
  // a span overlaps an earlier one exactly if it begins before the furthest end so far; of the
  // earlier ones the furthest written and the furthest of any kind are enough
  const Span *any = nullptr, *written = nullptr;
  for (const Span& s : spans) {
    const Span* hit = s.written ? any : written;
    if (hit && s.r.lo < hit->r.hi)
      return fail(FORGE_ERR_ALIAS, "%s of tensor %d overlaps %s of tensor %d", s.r.name, (int)s.tensor, hit->r.name,
                  (int)hit->tensor);
    if (!any || s.r.hi > any->r.hi) any = &s;
    if (s.written && (!written || s.r.hi > written->r.hi)) written = &s;
  }
  unsigned char* entry = static_cast<unsigned char*>(table);
  unsigned char* owner = entry + (size_t)n_tensors * sizeof(forge::MultiEntry);
  int64_t chunk = 0;
  for (int32_t i = 0; i < n_tensors; ++i) {
    const forge_multi_tensor& t = tensors[i];
    forge::MultiEntry e{};
    e.W = t.W;
    e.g = t.g;
    e.m = t.m;
    e.v = t.v;
    e.m_scale = t.m_scale;
    e.v_scale = t.v_scale;
    e.seed = t.seed;
    e.n = (uint32_t)t.n;
    e.chunk0 = (uint32_t)chunk;
    e.group = (uint32_t)t.group;
    e.w_bf16 = t.w_dtype == FORGE_BF16;
    e.g_bf16 = t.g_dtype == FORGE_BF16;
    std::memcpy(entry + (size_t)i * sizeof e, &e, sizeof e);
    const uint32_t who = (uint32_t)i;
    for (int64_t c = multi_chunks(t.n); c > 0; --c, ++chunk) std::memcpy(owner + 4 * chunk, &who, 4);
  }
  info->bytes = need;
  info->chunks = chunk;
  info->tensors = n_tensors;
  info->groups = groups;
  info->opt = opt;
  info->m_dtype = m_dtype;
  info->v_dtype = v_dtype;
  info->reserved = 0;
  return FORGE_OK;
}

forge_status forge_multi_step(const forge_multi_info* info, const void* table, const forge_hyper* hypers,
                              int32_t n_hypers, int64_t step, const float* grad_scale, const forge_step_opts* opts,
                              void* stream) {
  clear_error();
  if (!info) return fail(FORGE_ERR_ARG, "info is NULL");
  if (info->opt < FORGE_ADAMW || info->opt > FORGE_SGD_MOMENTUM)
    return fail(FORGE_ERR_ARG, "unknown optimizer %d", (int)info->opt);
  if (info->tensors < 0 || info->chunks < 0 || info->chunks >= forge::kMultiMaxChunks || info->groups < 0 ||
      info->groups > forge::kMultiGroups ||
      info->bytes != info->tensors * (int64_t)sizeof(forge::MultiEntry) + 4 * info->chunks)
    return fail(FORGE_ERR_ARG, "info is not one that forge_multi_pack wrote");
  if (n_hypers < info->groups || n_hypers > forge::kMultiGroups)
    return fail(FORGE_ERR_ARG, "the tensors use %d hyper-parameter groups, %d were given (at most %d)",
                (int)info->groups, (int)n_hypers, forge::kMultiGroups);
  if (n_hypers > 0 && !hypers) return fail(FORGE_ERR_ARG, "hypers is NULL");
  if (opts && opts->w_preround_out) return fail(FORGE_ERR_ARG, "w_preround_out must be NULL");
  if (!aligned4(grad_scale)) return fail(FORGE_ERR_LAYOUT, "grad_scale is not 4-byte aligned");
  forge::MultiArgs a{};
  forge_status st;
  for (int32_t i = 0; i < n_hypers; ++i)
    if ((st = compute_scalars(info->opt, &hypers[i], step, &a.s[i])) != FORGE_OK) return st;
  if (step < 1) return fail(FORGE_ERR_ARG, "step must be >= 1 (got %lld)", (long long)step);
  const int32_t dt = info->m_dtype >= 0 ? info->m_dtype : info->v_dtype;
  int s_type = forge::FORGE_S_F32;
  if (dt == FORGE_I8_B64 || dt == FORGE_U8_B64) s_type = forge::FORGE_S_Q8;
  else if (dt == FORGE_I8DYN_B64 || dt == FORGE_U8DYN_B64) s_type = forge::FORGE_S_Q8D;
  if (info->chunks == 0) return FORGE_OK;
  if (!table) return fail(FORGE_ERR_ARG, "table is NULL");
  if (!aligned16(table)) return fail(FORGE_ERR_LAYOUT, "table is not 16-byte aligned");
  if ((st = device_ok()) != FORGE_OK) return st;
  a.entries = static_cast<const forge::MultiEntry*>(table);
  a.owner = reinterpret_cast<const uint32_t*>(a.entries + info->tensors);
  a.grad_scale = grad_scale;
  a.step = (uint64_t)step;
  a.sr = opts ? (opts->sr_enable != 0) : 1;
  return to_status(forge::launch_multi_step(s_type, info->opt, a, info->chunks, stream));
}

}  // extern "C"

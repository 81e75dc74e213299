// forge_ffn_host.cpp -- the C ABI declared in include/forge_ffn.h: argument checks (before any HIP
// call) and dispatch.
#include <hip/hip_runtime.h>

#include <cstring>

#include "forge.h"
#include "forge_ffn.h"
#include "forge_ffn_internal.h"
#include "forge_layer_host.h"

using namespace forge::host;

namespace {

bool is_codes(int32_t dt) { return dt == FORGE_FP8_B128 || dt == FORGE_I8_B128; }
int64_t blocks_of(int64_t cols) { return (cols + 127) / 128; }

// Scales of codes: n fp32.
forge_status check_scales(const forge_tensor* t, int64_t n, const char* name, const char* scales, bool written, Ranges* rs) {
  if (!t->scale && n > 0) return fail(FORGE_ERR_ARG, "%s needs %s->scale", name, name);
  if (!aligned4(t->scale)) return fail(FORGE_ERR_LAYOUT, "%s->scale is not 4-byte aligned", name);
  rs->add(t->scale, 4 * n, scales, written);
  return FORGE_OK;
}

forge_status check_act(int32_t act) {
  static_assert(FORGE_ACT_SILU == (int)forge::FORGE_ACT_K_SILU && FORGE_ACT_GELU == (int)forge::FORGE_ACT_K_GELU &&
                    FORGE_ACT_GELU_TANH == (int)forge::FORGE_ACT_K_GELU_TANH && FORGE_ACT_RELU == (int)forge::FORGE_ACT_K_RELU,
                "the kernels' activations");
  if (act < FORGE_ACT_SILU || act > FORGE_ACT_RELU) return fail(FORGE_ERR_ARG, "unknown activation %d", (int)act);
  return FORGE_OK;
}

// Gate and up [T, 2 N] of dtype BF16, `whole` or codes with [T, 2, ceil(N / 128)] scales.
forge_status check_kept(const forge_tensor* t, int64_t T, int64_t N, int32_t whole, bool written, Ranges* rs,
                        forge::KeptArgs* k) {
  forge_status st;
  if ((st = check_tensor(t, "gate_up")) != FORGE_OK) return st;
  if ((st = check_shape(t, T, 2 * N, "gate_up")) != FORGE_OK) return st;
  if (t->dtype != whole && !is_codes(t->dtype))
    return fail(FORGE_ERR_DTYPE, "gate_up must be %s, FP8_B128 or I8_B128", whole == FORGE_F32 ? "F32" : "BF16");
  rs->add(t, "gate_up", written);
  k->data = t->data;
  k->scale = nullptr;
  k->type = t->dtype == FORGE_BF16  ? forge::FORGE_KEEP_BF16
            : t->dtype == FORGE_F32 ? forge::FORGE_KEEP_F32
            : t->dtype == FORGE_FP8_B128 ? forge::FORGE_KEEP_FP8
                                         : forge::FORGE_KEEP_I8;
  if (is_codes(t->dtype)) {
    if ((st = check_scales(t, T * 2 * blocks_of(N), "gate_up", "gate_up scales", written, rs)) != FORGE_OK) return st;
    k->scale = static_cast<float*>(t->scale);
  }
  return FORGE_OK;
}

forge_status check_tiles(int64_t T, int32_t n_groups, int64_t cols) {
  if ((T / 64 + n_groups + 1) * ((cols + 255) / 256) >= (int64_t(1) << 31)) return fail(FORGE_ERR_SHAPE, "too many tiles");
  return FORGE_OK;
}

// x (F32 or BF16) and its codes q.
forge_status check_block(const forge_tensor* x, const char* xn, const forge_tensor* q, bool quantize, forge::BlockArgs* a) {
  clear_error();
  forge_status st;
  if ((st = check_tensor(x, xn)) != FORGE_OK) return st;
  if ((st = check_tensor(q, "q")) != FORGE_OK) return st;
  if (!is_stream(x->dtype)) return fail(FORGE_ERR_DTYPE, "%s must be F32 or BF16", xn);
  if (!is_codes(q->dtype)) return fail(FORGE_ERR_DTYPE, "q must be FP8_B128 or I8_B128");
  const int64_t T = x->rows, D = x->cols;
  if ((st = check_shape(q, T, D, "q")) != FORGE_OK) return st;
  if (D < 1 || D >= (int64_t(1) << 31)) return fail(FORGE_ERR_SHAPE, "D must be 1 .. 2^31 - 1 (got %lld)", (long long)D);
  if (T >= (int64_t(1) << 47) / blocks_of(D)) return fail(FORGE_ERR_SHAPE, "too many blocks");
  Ranges rs;
  rs.add(x, xn, !quantize);
  rs.add(q, "q", quantize);
  if ((st = check_scales(q, T * blocks_of(D), "q", "q scales", quantize, &rs)) != FORGE_OK) return st;
  if ((st = rs.check(never)) != FORGE_OK) return st;
  a->x = quantize ? x->data : q->data;
  a->y = quantize ? q->data : x->data;
  a->scale = static_cast<float*>(q->scale);
  a->T = T;
  a->D = D;
  a->bf16 = x->dtype == FORGE_BF16;
  a->q = q->dtype == FORGE_FP8_B128 ? forge::FORGE_Q_FP8 : forge::FORGE_Q_I8;
  return FORGE_OK;
}

}  // namespace

extern "C" {

forge_status forge_block_quantize(const forge_tensor* x, forge_tensor* q, void* stream) {
  forge::BlockArgs a{};
  forge_status st;
  if ((st = check_block(x, "x", q, true, &a)) != FORGE_OK) return st;
  if (a.T == 0) return FORGE_OK;
  if ((st = device_ok()) != FORGE_OK) return st;
  return to_status(forge::launch_block_quantize(a, stream));
}

forge_status forge_block_dequantize(const forge_tensor* q, forge_tensor* y, void* stream) {
  forge::BlockArgs a{};
  forge_status st;
  if ((st = check_block(y, "y", q, false, &a)) != FORGE_OK) return st;
  if (a.T == 0) return FORGE_OK;
  if ((st = device_ok()) != FORGE_OK) return st;
  return to_status(forge::launch_block_dequantize(a, stream));
}

forge_status forge_block_quantize_weight(const forge_tensor* W, int32_t n_groups, forge_tensor* q, forge_tensor* qt,
                                         void* stream) {
  clear_error();
  forge_status st;
  if ((st = check_tensor(W, "W")) != FORGE_OK) return st;
  if ((st = check_tensor(q, "q")) != FORGE_OK) return st;
  if (!is_stream(W->dtype)) return fail(FORGE_ERR_DTYPE, "W must be F32 or BF16");
  if (q->dtype != FORGE_FP8_B128 || (qt && qt->dtype != FORGE_FP8_B128)) return fail(FORGE_ERR_DTYPE, "q and qt must be FP8_B128");
  if (n_groups < 1) return fail(FORGE_ERR_ARG, "n_groups must be positive (got %d)", (int)n_groups);
  const int64_t E = n_groups, K = W->cols, N = W->rows / E;
  if (N * E != W->rows || N < 128 || K < 128 || N % 128 || K % 128)
    return fail(FORGE_ERR_SHAPE, "W is [%lld, %lld], expected [n_groups * N, K] with multiples of 128", (long long)W->rows,
                (long long)K);
  if (E * (N / 128) * (K / 128) >= (int64_t(1) << 24)) return fail(FORGE_ERR_SHAPE, "W must have fewer than 2^38 elements");
  if ((st = check_shape(q, E * N, K, "q")) != FORGE_OK) return st;
  Ranges rs;
  rs.add(W, "W", false);
  rs.add(q, "q", true);
  const int64_t squares = E * (N / 128) * (K / 128);
  if ((st = check_scales(q, squares, "q", "q scales", true, &rs)) != FORGE_OK) return st;
  if (qt) {
    if ((st = check_tensor(qt, "qt")) != FORGE_OK) return st;
    if ((st = check_shape(qt, E * K, N, "qt")) != FORGE_OK) return st;
    rs.add(qt, "qt", true);
    if ((st = check_scales(qt, squares, "qt", "qt scales", true, &rs)) != FORGE_OK) return st;
  }
  if ((st = rs.check(never)) != FORGE_OK) return st;
  if ((st = device_ok()) != FORGE_OK) return st;
  forge::BlockWeightArgs a{};
  a.W = W->data;
  a.q = static_cast<uint8_t*>(q->data);
  a.scale = static_cast<float*>(q->scale);
  a.qt = qt ? static_cast<uint8_t*>(qt->data) : nullptr;
  a.scale_t = qt ? static_cast<float*>(qt->scale) : nullptr;
  a.E = E;
  a.N = N;
  a.K = K;
  a.bf16 = W->dtype == FORGE_BF16;
  return to_status(forge::launch_block_quantize_weight(a, stream));
}

forge_status forge_grouped_block_gemm(const forge_tensor* X, const forge_tensor* W, const int32_t* ends, int32_t n_groups,
                                      forge_tensor* Y, void* stream) {
  clear_error();
  forge_status st;
  if ((st = check_tensor(X, "X")) != FORGE_OK) return st;
  if ((st = check_tensor(W, "W")) != FORGE_OK) return st;
  if ((st = check_tensor(Y, "Y")) != FORGE_OK) return st;
  const int64_t T = X->rows, N = Y->cols, K = X->cols;
  if ((st = check_groups(ends, n_groups, T, N, K)) != FORGE_OK) return st;
  if ((st = check_shape(W, n_groups * N, K, "W")) != FORGE_OK) return st;
  if ((st = check_shape(Y, T, N, "Y")) != FORGE_OK) return st;
  if (X->dtype != FORGE_FP8_B128 || W->dtype != FORGE_FP8_B128 || Y->dtype != FORGE_BF16)
    return fail(FORGE_ERR_DTYPE, "the block product takes FP8_B128 X and W and writes BF16 Y");
  Ranges rs;
  rs.add(X, "X", false);
  rs.add(W, "W", false);
  rs.add(ends, 4 * (int64_t)n_groups, "ends", false);
  rs.add(Y, "Y", true);
  if ((st = check_scales(X, T * (K / 128), "X", "X scales", false, &rs)) != FORGE_OK) return st;
  if ((st = check_scales(W, n_groups * (N / 128) * (K / 128), "W", "W scales", false, &rs)) != FORGE_OK) return st;
  if ((st = rs.check(never)) != FORGE_OK) return st;
  if ((st = check_tiles(T, n_groups, N)) != FORGE_OK) return st;
  if (T == 0) return FORGE_OK;
  if ((st = device_ok()) != FORGE_OK) return st;
  forge::BlockGemmArgs a{};
  a.X = static_cast<const uint8_t*>(X->data);
  a.W = static_cast<const uint8_t*>(W->data);
  a.x_scale = static_cast<const float*>(X->scale);
  a.w_scale = static_cast<const float*>(W->scale);
  a.ends = ends;
  a.Y = static_cast<uint16_t*>(Y->data);
  a.E = n_groups;
  a.T = T;
  a.N = N;
  a.K = K;
  return to_status(forge::launch_grouped_block_gemm(a, stream));
}

forge_status forge_grouped_gated(const forge_tensor* X, const forge_tensor* W, const int32_t* ends, int32_t n_groups,
                                 int32_t act, forge_tensor* H, forge_tensor* gate_up, void* stream) {
  clear_error();
  forge_status st;
  if ((st = check_tensor(X, "X")) != FORGE_OK) return st;
  if ((st = check_tensor(W, "W")) != FORGE_OK) return st;
  if ((st = check_tensor(H, "H")) != FORGE_OK) return st;
  if ((st = check_act(act)) != FORGE_OK) return st;
  const int64_t T = X->rows, N = H->cols, K = X->cols;
  if (N % 128) return fail(FORGE_ERR_SHAPE, "N = %lld must be a multiple of 128", (long long)N);
  if ((st = check_groups(ends, n_groups, T, 2 * N, K)) != FORGE_OK) return st;  // of the stacked weight
  if ((st = check_shape(W, n_groups * 2 * N, K, "W")) != FORGE_OK) return st;
  if ((st = check_shape(H, T, N, "H")) != FORGE_OK) return st;
  if (X->dtype != FORGE_BF16 || W->dtype != FORGE_BF16 || H->dtype != FORGE_BF16)
    return fail(FORGE_ERR_DTYPE, "X, W and H must be BF16");
  Ranges rs;
  rs.add(X, "X", false);
  rs.add(W, "W", false);
  rs.add(ends, 4 * (int64_t)n_groups, "ends", false);
  rs.add(H, "H", true);
  forge::GatedArgs a{};
  if (gate_up && (st = check_kept(gate_up, T, N, FORGE_BF16, true, &rs, &a.keep)) != FORGE_OK) return st;
  if ((st = rs.check(never)) != FORGE_OK) return st;
  if ((st = check_tiles(T, n_groups, 2 * N)) != FORGE_OK) return st;
  if (T == 0) return FORGE_OK;
  if ((st = device_ok()) != FORGE_OK) return st;
  a.X = X->data;
  a.W = W->data;
  a.ends = ends;
  a.H = static_cast<uint16_t*>(H->data);
  a.E = n_groups;
  a.act = act;
  a.T = T;
  a.N = N;
  a.K = K;
  return to_status(forge::launch_grouped_gated(a, stream));
}

// dgate_up and H of the backward passes, of dtype dt.
static forge_status check_backward_outputs(forge_tensor* dgate_up, forge_tensor* H, int64_t T, int64_t N, int32_t dt,
                                           Ranges* rs) {
  forge_status st;
  if ((st = check_tensor(dgate_up, "dgate_up")) != FORGE_OK) return st;
  if ((st = check_shape(dgate_up, T, 2 * N, "dgate_up")) != FORGE_OK) return st;
  if (dgate_up->dtype != dt) return fail(FORGE_ERR_DTYPE, "dgate_up has the wrong dtype");
  rs->add(dgate_up, "dgate_up", true);
  if (H) {
    if ((st = check_tensor(H, "H")) != FORGE_OK) return st;
    if ((st = check_shape(H, T, N, "H")) != FORGE_OK) return st;
    if (H->dtype != dt) return fail(FORGE_ERR_DTYPE, "H has the wrong dtype");
    rs->add(H, "H", true);
  }
  return FORGE_OK;
}

forge_status forge_gated_backward(const forge_tensor* dH, const forge_tensor* gate_up, int32_t act,
                                  forge_tensor* dgate_up, forge_tensor* H, void* stream) {
  clear_error();
  forge_status st;
  if ((st = check_tensor(dH, "dH")) != FORGE_OK) return st;
  if (!is_stream(dH->dtype)) return fail(FORGE_ERR_DTYPE, "dH must be F32 or BF16");
  if ((st = check_act(act)) != FORGE_OK) return st;
  const int64_t T = dH->rows, N = dH->cols;
  if (N < 1 || N > (int64_t(1) << 30)) return fail(FORGE_ERR_SHAPE, "N must be 1 .. 2^30 (got %lld)", (long long)N);
  Ranges rs;
  rs.add(dH, "dH", false);
  forge::GatedBwdArgs a{};
  if ((st = check_kept(gate_up, T, N, dH->dtype, false, &rs, &a.keep)) != FORGE_OK) return st;
  if ((st = check_backward_outputs(dgate_up, H, T, N, dH->dtype, &rs)) != FORGE_OK) return st;
  st = rs.check([](const char* w, const char* r) {
    return (std::strcmp(w, "H") == 0 && std::strcmp(r, "dH") == 0) ||
           (std::strcmp(w, "dgate_up") == 0 && std::strcmp(r, "gate_up") == 0);
  });
  if (st != FORGE_OK) return st;
  if (T == 0) return FORGE_OK;
  if ((st = device_ok()) != FORGE_OK) return st;
  a.dH = dH->data;
  a.dGU = dgate_up->data;
  a.H = H ? H->data : nullptr;
  a.T = T;
  a.N = N;
  a.act = act;
  a.bf16 = dH->dtype == FORGE_BF16;
  return to_status(forge::launch_gated_backward(a, stream));
}

forge_status forge_grouped_gated_dgrad(const forge_tensor* dY, const forge_tensor* W, const int32_t* ends,
                                       int32_t n_groups, const forge_tensor* gate_up, int32_t act,
                                       forge_tensor* dgate_up, forge_tensor* H, void* stream) {
  clear_error();
  forge_status st;
  if ((st = check_tensor(dY, "dY")) != FORGE_OK) return st;
  if ((st = check_tensor(W, "W")) != FORGE_OK) return st;
  if ((st = check_act(act)) != FORGE_OK) return st;
  const int64_t T = dY->rows, N = W->cols, K = dY->cols;
  if ((st = check_groups(ends, n_groups, T, N, K)) != FORGE_OK) return st;
  if ((st = check_shape(W, n_groups * K, N, "W")) != FORGE_OK) return st;
  if (dY->dtype != FORGE_BF16 || W->dtype != FORGE_BF16) return fail(FORGE_ERR_DTYPE, "dY and W must be BF16");
  Ranges rs;
  rs.add(dY, "dY", false);
  rs.add(W, "W", false);
  rs.add(ends, 4 * (int64_t)n_groups, "ends", false);
  forge::GatedDgradArgs a{};
  if ((st = check_kept(gate_up, T, N, FORGE_BF16, false, &rs, &a.keep)) != FORGE_OK) return st;
  if ((st = check_backward_outputs(dgate_up, H, T, N, FORGE_BF16, &rs)) != FORGE_OK) return st;
  st = rs.check([](const char* w, const char* r) { return std::strcmp(w, "dgate_up") == 0 && std::strcmp(r, "gate_up") == 0; });
  if (st != FORGE_OK) return st;
  if ((st = check_tiles(T, n_groups, N)) != FORGE_OK) return st;
  if (T == 0) return FORGE_OK;
  if ((st = device_ok()) != FORGE_OK) return st;
  a.dY = dY->data;
  a.W = W->data;
  a.ends = ends;
  a.dGU = static_cast<uint16_t*>(dgate_up->data);
  a.H = H ? static_cast<uint16_t*>(H->data) : nullptr;
  a.E = n_groups;
  a.act = act;
  a.T = T;
  a.N = N;
  a.K = K;
  return to_status(forge::launch_grouped_gated_dgrad(a, stream));
}

}  // extern "C"

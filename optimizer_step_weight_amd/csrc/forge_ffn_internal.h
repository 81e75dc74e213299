// forge_ffn_internal.h -- structures shared by the entry points of forge_ffn.h and their kernels.
#pragma once

#include <stdint.h>

#include "forge_layer_internal.h"

namespace forge {

// How an activation tensor is kept (FORGE_Q_FP8, FORGE_Q_I8: forge_layer_internal.h).
enum : int { FORGE_KEEP_NONE = 0, FORGE_KEEP_BF16 = 1, FORGE_KEEP_FP8 = 2, FORGE_KEEP_I8 = 3, FORGE_KEEP_F32 = 4 };
enum : int { FORGE_ACT_K_SILU = 0, FORGE_ACT_K_GELU = 1, FORGE_ACT_K_GELU_TANH = 2, FORGE_ACT_K_RELU = 3 };

// Gate and up [T, 2 N]: blocks of the 8-bit forms begin at column 0 of either half.
struct KeptArgs {
  void* data;
  float* scale;    // 8-bit: [T, 2, ceil(N / 128)]
  int32_t type;    // FORGE_KEEP_*
};

// H = act(X Wg^T) * (X Wu^T), W [E, 2 N, K].
struct GatedArgs {
  const void* X;
  const void* W;
  const int32_t* ends;
  uint16_t* H;     // [T, N] bf16
  KeptArgs keep;   // written
  int32_t E, act;
  int32_t cols;    // least rows of W a tile takes: 256 or 128
  int64_t T, N, K;
};
int launch_grouped_gated(const GatedArgs& a, void* stream);
int launch_gated_few(const GatedArgs& a, void* stream);  // 8-bit gate and up: not there

// dH = dY W, W [E, K, N]; from it and the kept gate and up d(gate, up) and H.
struct GatedDgradArgs {
  const void* dY;
  const void* W;
  const int32_t* ends;
  KeptArgs keep;   // read
  uint16_t* dGU;   // [T, 2 N] bf16
  uint16_t* H;     // or null
  int32_t E, act;
  int32_t cols;
  int64_t T, N, K;
};
int launch_grouped_gated_dgrad(const GatedDgradArgs& a, void* stream);

// The same from dH itself; types F32 or BF16.
struct GatedBwdArgs {
  const void* dH;
  KeptArgs keep;
  void* dGU;
  void* H;         // or null
  int64_t T, N;
  int32_t act, bf16;
};
int launch_gated_backward(const GatedBwdArgs& a, void* stream);

// Codes of blocks of 1 x 128.
struct BlockArgs {
  const void* x;   // F32 or BF16 (quantise), codes (dequantise)
  void* y;
  float* scale;    // [T, ceil(D / 128)]
  int64_t T, D;
  int32_t bf16, q;
};
int launch_block_quantize(const BlockArgs& a, void* stream);
int launch_block_dequantize(const BlockArgs& a, void* stream);

// Codes of blocks of 128 x 128 of E weights [N, K], and their transposed copy.
struct BlockWeightArgs {
  const void* W;
  uint8_t* q;      // [E, N, K]
  float* scale;    // [E, N / 128, K / 128]
  uint8_t* qt;     // [E, K, N] or null
  float* scale_t;
  int64_t E, N, K;
  int32_t bf16;
};
int launch_block_quantize_weight(const BlockWeightArgs& a, void* stream);

// Y_e = X_e W_e^T of codes with block scales.
struct BlockGemmArgs {
  const uint8_t* X;       // [T, K]
  const uint8_t* W;       // [E, N, K]
  const float* x_scale;   // [T, K / 128]
  const float* w_scale;   // [E, N / 128, K / 128]
  const int32_t* ends;
  uint16_t* Y;            // [T, N] bf16
  int32_t E;
  int32_t cols;
  int64_t T, N, K;
};
int launch_grouped_block_gemm(const BlockGemmArgs& a, void* stream);
int launch_block_few(const BlockGemmArgs& a, void* stream);
// Whether the kernels of few rows (forge_few.hip) take a call, by the least tiles of the other kernels that its rows
// and columns make, `cols` columns each: these are slow where they leave CUs without any, those read X again for each
// 16 columns.  In us, few rows against tiles, one weight:
//   gated product  4096 x 4096 (64 tiles): 17 against 41 at 16 rows, 29 against 41 at 64, 54 against 44 at 128;
//                  8192 x 2048 (128): 21 against 25 at 32 rows, 32 against 25 at 64; 1408 x 2048 (22): 10 against 14 at 16
//                  rows, 17 against 14 at 64; 14336 x 4096 (224): 49 against 46 at one row
//   block product  4096 x 14336 (32): 22 against 94 at 16 rows, 49 against 95 at 64, 95 against 105 at 128; 4096 x 4096 (32):
//                  17 against 20 at 64 rows, 32 against 23 at 128; 14336 x 4096 (112): 24 against 31 at 16 rows, 35 against 31
//                  at 32; 2048 x 4096 (16): 17 against 23 at 128 rows, 32 against 29 at 256
inline bool few_rows_call(int64_t T, int32_t E, int64_t N, int64_t cols, int64_t most) {
  const int64_t tiles = (E < T ? E : T) * (N / cols);
  return T <= 256 && tiles <= 128 && T * tiles <= most;
}
constexpr int64_t kFewGated = 4096, kFewBlock = 2048;

}  // namespace forge

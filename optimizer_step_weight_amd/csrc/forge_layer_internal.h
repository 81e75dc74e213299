// forge_layer_internal.h -- structures shared by the entry points of forge_layer.h and their
// kernels.
#pragma once

#include <stdint.h>

#include "forge_internal.h"

namespace forge {

// ------------------------------------------------------------------ RMS norm
enum : int { FORGE_Y_F32 = 0, FORGE_Y_BF16 = 1, FORGE_Y_FP8_ROW = 2, FORGE_Y_FP8_TENSOR = 3 };

struct NormArgs {
  const void* x;
  const void* res;   // or null
  const void* gain;
  void* h;           // null without res
  void* y;
  float* y_scale;    // written per row, or one read for the tensor
  float* rstd;       // or null
  float* amax;       // or null
  int64_t T;
  int32_t D;
  float eps;
  int32_t gain_bf16;
};
int launch_rmsnorm(int x_bf16, int y_type, const NormArgs& a, void* stream);

struct NormBwdArgs {
  const void* dy;
  const void* dh;    // or null
  const void* h;
  const void* gain;
  const float* rstd;
  void* dx;
  float* dgain;      // or null
  float* partial;    // [groups, D]
  int64_t T;
  int32_t D;
  int32_t gain_bf16;
};
// Workgroups of the norm at most: eight of 256 threads on each of 256 CUs.
constexpr int64_t kNormBlocks = 2048;
// Row groups of the gain's gradient: each sums its rows into one row of the workspace.
inline int64_t norm_bwd_groups(int64_t T) { return T < 1024 ? (T < 1 ? 1 : T) : 1024; }
int launch_rmsnorm_backward(int bf16, const NormBwdArgs& a, void* stream);

// ------------------------------------------------------------------ products grouped by expert
struct GroupedArgs {
  const void* A;         // X or dY rows [T, C]
  const void* W;         // [E N, K]
  void* out;             // [T, O] bf16
  const float* a_scale;  // fp8: per row of A, per row of W
  const float* w_scale;
  const int32_t* ends;
  int32_t E;
  int32_t cols;          // least output columns of a tile: 256 or 128
  int64_t T, N, K;
};
enum : int { FORGE_GROUPED_NT = 0, FORGE_GROUPED_NN = 1, FORGE_GROUPED_NT8 = 2 };
int launch_grouped_rows(int mode, const GroupedArgs& a, void* stream);

struct GroupedWgradArgs {
  const void* X;
  const void* dY;
  const int32_t* ends;
  int32_t E;
  int32_t small;         // 128 x 128 tiles throughout
  int64_t T, N, K;
};
int launch_grouped_wgrad(const GroupedWgradArgs& a, float* dW, void* stream);
int launch_grouped_step(int s_type, int opt, const GroupedWgradArgs& a, const EpiArgs& e, void* stream);

// ------------------------------------------------------------------ the step over many tensors
constexpr int kMultiChunk = 4096;   // elements of a workgroup
constexpr int kMultiGroups = 8;
constexpr int64_t kMultiMaxChunks = int64_t(1) << 24;  // of 256 threads: a grid has fewer than 2^32
struct MultiEntry {
  void* W;
  const void* g;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  uint64_t seed;
  uint32_t n;
  uint32_t chunk0;   // first chunk of this tensor
  uint32_t group;
  uint8_t w_bf16, g_bf16, pad[2];
};
static_assert(sizeof(MultiEntry) == 72, "table layout");
// The table: n_tensors entries, then one uint32 per chunk naming its tensor.
struct MultiArgs {
  const MultiEntry* entries;
  const uint32_t* owner;
  const float* grad_scale;
  uint64_t step;
  int32_t sr;
  OptScalars s[kMultiGroups];
};
int launch_multi_step(int s_type, int opt, const MultiArgs& a, int64_t chunks, void* stream);

}  // namespace forge

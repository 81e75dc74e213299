// forge_grouped_wgrad.h -- the optimizer's step of every expert's weight, fused into its gradient
// dW_e = dY_e^T X_e on the LDS-DMA path of forge_mainloop2.h.  (The gradient kept in fp32 takes the
// contraction of forge_grouped.h, whose sums are the same bit for bit.)
//
// One workgroup of 4 waves takes a 256 x 128 tile of an expert's weight (128 x 128 for the last
// rows where N is an odd multiple of 128) and contracts the group's rows alone: the operands'
// buffer ranges begin at the group's first row and end with its last, so a ragged end reads as
// zero and an empty group contracts nothing.  Two workgroups share a CU: a tile is mostly epilogue
// (20 bytes a weight with fp32 moments), and one workgroup's contraction runs beside the other's
// epilogue; a 256 x 256 tile of one workgroup a CU would have nothing beside it.  8 experts of
// 4096 x 4096, 8192 rows, AdamW with fp32 moments: 645-727 us over the cards seen, 3.9-4.4 TB/s of the 2.8 GB that it
// cannot do without (594 us at a copy's 4.75 TB/s) and 380-430 TFLOP/s besides; with 8-bit moments in the linear map 474
// us, in the dynamic map, whose codes take many more operations, 1110 us.  Experts follow each other in the launch, each
// spread over all XCDs, so that a crowded expert does not hold up one XCD.
#pragma once

#include "forge_epilogue.h"
#include "forge_grouped.h"

namespace forge {
namespace grp {

struct WTile {
  GemmArgs g;     // the group's operands
  int n0, k0;     // origin in the expert's weight
  int row0;       // the same row in the stacked weights
  bool half;      // 128 x 128
};

// Tiles of one expert: full ones, then the half ones of the last 128 rows; half ones alone where the
// larger would leave CUs without any (a contraction cannot be split, so the tile is what is halved:
// 5 uneven experts of 512 x 1664, 17679 rows, 130 full tiles: 165 us, 260 half ones: 100 us; the gradient alone
// 147 us in 70 tiles of 256 x 256, 58 us in 260 of 128 x 128; 200 of the former and 800 of the latter
// are equal).
__host__ __device__ inline int wgrad_tiles(int64_t N, int64_t K, bool small) {
  return (int)((small ? N / 128 : N / 256 + (N % 256 ? 1 : 0)) * (K / 128));
}
inline bool wgrad_small(int64_t E, int64_t tiles) { return E * tiles < 256; }

__device__ __forceinline__ void wgrad_tile(const GroupedWgradArgs& a, WTile& t) {
  const int per = wgrad_tiles(a.N, a.K, a.small), e = (int)blockIdx.x / per, b = (int)blockIdx.x - e * per;
  const int nbk = (int)(a.K / 128), full = (int)(a.N / 256) * nbk;
  int start, len, nb, kb;
  group_rows(a.ends, a.E, a.T, e, start, len);
  t.g.X = static_cast<const uint16_t*>(a.X) + (int64_t)start * a.K;
  t.g.dY = static_cast<const uint16_t*>(a.dY) + (int64_t)start * a.N;
  t.g.x_scale = t.g.dy_scale = nullptr;
  t.g.T = len;
  t.g.N = a.N;
  t.g.K = a.K;
  t.half = a.small || b >= full;
  if (a.small) {
    t.n0 = b / nbk * 128;
    t.k0 = b % nbk * 128;
    t.row0 = e * (int)a.N + t.n0;
    return;
  }
  if (t.half) {
    nb = (int)(a.N / 256);
    kb = b - full;
  } else {
    plan::tile_coords_at(b, (int)(a.N / 256), nbk, nb, kb);
  }
  t.n0 = nb * 256;
  t.k0 = kb * 128;
  t.row0 = e * (int)a.N + t.n0;
}

template <int ST, int OPT>
__global__ __launch_bounds__(ml2::THREADS, kOcc2) void grouped_step_kernel(GroupedWgradArgs a, EpiArgs e) {
  __shared__ __attribute__((aligned(1024))) unsigned char smem[kSmem2];
  WTile t;
  wgrad_tile(a, t);
  float* st = reinterpret_cast<float*>(smem);
  if (t.half) {
    floatx4 acc[4][4];
    ml2::contract<Pipe2H>(acc, smem, t.g, t.n0, t.k0);
    tile_epilogue<OPT, FORGE_W_BF16, ST, 1, true>(t.g, e, smem, t.row0, t.k0,
                                                  [&](int) { ml2::stage_acc_all(st, acc, 1.0f); });
  } else {
    floatx4 acc[8][4];
    ml2::contract<Pipe2>(acc, smem, t.g, t.n0, t.k0);
    tile_epilogue<OPT, FORGE_W_BF16, ST, 2, true>(t.g, e, smem, t.row0, t.k0,
                                                  [&](int h) { ml2::stage_acc_half(st, acc, 1.0f, h); });
  }
}

using GroupedStepFn = void (*)(GroupedWgradArgs, EpiArgs);
// Instantiated per moment format in forge_grouped_{f32,q8,q8d}.hip.
template <int ST>
GroupedStepFn select_grouped_step(int opt) {
  switch (opt) {
#define FORGE_CASE(O) \
  case O: return grouped_step_kernel<ST, O>;
    FORGE_FOR_EACH_OPT(FORGE_CASE)
#undef FORGE_CASE
  }
  return nullptr;
}
extern template GroupedStepFn select_grouped_step<FORGE_S_F32>(int);
extern template GroupedStepFn select_grouped_step<FORGE_S_Q8>(int);
extern template GroupedStepFn select_grouped_step<FORGE_S_Q8D>(int);

}  // namespace grp
}  // namespace forge

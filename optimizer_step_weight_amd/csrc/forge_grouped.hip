// forge_grouped.hip -- launchers of the products grouped by expert (forge_grouped.h,
// forge_grouped_wgrad.h), and the weight gradient kept in fp32.
#include <hip/hip_runtime.h>

#include "forge_grouped_wgrad.h"

namespace forge {

int launch_grouped_rows(int mode, const GroupedArgs& given, void* stream) {
  GroupedArgs a = given;
  const int64_t O = mode == FORGE_GROUPED_NN ? a.K : a.N;
  const int64_t row_tiles = a.T / 256 + (a.E < a.T ? a.E : a.T) + 1;
  // the device, which knows the groups, takes the narrow tiles if even the fewest there can be fit
  a.cols = a.T / 256 * ((O + 255) / 256) <= grp::NARROW_TILES ? 128 : 256;
  const int64_t tiles = row_tiles * ((O + a.cols - 1) / a.cols);
  const dim3 grid((unsigned)tiles), block(grp::THREADS);
  hipStream_t st = (hipStream_t)stream;
  switch (mode) {
    case FORGE_GROUPED_NT: hipLaunchKernelGGL(grp::grouped_rows_kernel<FORGE_GROUPED_NT>, grid, block, 0, st, a); break;
    case FORGE_GROUPED_NN: hipLaunchKernelGGL(grp::grouped_rows_kernel<FORGE_GROUPED_NN>, grid, block, 0, st, a); break;
    case FORGE_GROUPED_NT8: hipLaunchKernelGGL(grp::grouped_rows_kernel<FORGE_GROUPED_NT8>, grid, block, 0, st, a); break;
    default: return (int)hipErrorInvalidValue;
  }
  return (int)hipGetLastError();
}

namespace grp {

// dW_e = dY_e^T X_e in fp32, 256 x 256 tiles of the contraction of forge_grouped.h (half as high or
// wide at the end of an odd multiple of 128) over the group's rows alone: the operands' ranges begin
// at the group's first row and end with its last, so a ragged end reads as zero.  32 experts of
// 1408 x 2048, 16384 rows: 143-165 us over the cards seen, 2.9-3.4 TB/s (stores that displace the operands in L2: 158
// us where these took 143); a tile's stores come after its contraction, and nothing else runs on its CU.
template <int HEIGHT, int WIDTH>
__device__ __forceinline__ void wgrad_tile_f32(const GroupedWgradArgs& a, float* dW, int e, int start, int len, int n0,
                                               int k0, unsigned char* smem) {
  using A = Side<2, true, 64 * HEIGHT, true>;
  using B = Side<2, true, 64 * WIDTH, true>;
  using T = Tile<A, B>;
  const int slabs = (len + 63) / 64;
  Feed<A> fa;
  Feed<B> fb;
  fa.open(static_cast<const uint16_t*>(a.dY) + (int64_t)start * a.N + n0, (uint32_t)(len * a.N * 2 - n0 * 2),
          (uint32_t)(a.N * 2), slabs);
  fb.open(static_cast<const uint16_t*>(a.X) + (int64_t)start * a.K + k0, (uint32_t)(len * a.K * 2 - k0 * 2),
          (uint32_t)(a.K * 2), slabs);
  T tile;
  tile.contract(smem, fa, fb, slabs);
  barrier();  // every wave is done with the slabs
  float* out = dW + ((int64_t)e * a.N + n0 + T::row0()) * a.K + k0 + T::col0();
  tile.template store<floatx4>(
      smem + (threadIdx.x >> 6) * WAVE_LDS, [](int, int, floatx4 v) { return v; },
      [&](int row, int col, u32x4 q) { st16_stream(out + (int64_t)row * a.K + col, q); });
}

__global__ __launch_bounds__(THREADS, 1) void grouped_wgrad_kernel(GroupedWgradArgs a, float* dW) {
  __shared__ __attribute__((aligned(1024))) unsigned char smem[5 * 32768];
  const int side = a.small ? 128 : 256;
  const int nbn = (int)((a.N + side - 1) / side), nbk = (int)((a.K + side - 1) / side), per = nbn * nbk;
  const int e = (int)blockIdx.x / per, b = (int)blockIdx.x - e * per;
  int start, len;
  group_rows(a.ends, a.E, a.T, e, start, len);
  const int n0 = side * (b % nbn), k0 = side * (b / nbn);
  const bool low = a.small || a.N - n0 < 256, narrow = a.small || a.K - k0 < 256;
  if (!low && !narrow) wgrad_tile_f32<4, 4>(a, dW, e, start, len, n0, k0, smem);
  else if (!narrow) wgrad_tile_f32<2, 4>(a, dW, e, start, len, n0, k0, smem);
  else if (!low) wgrad_tile_f32<4, 2>(a, dW, e, start, len, n0, k0, smem);
  else wgrad_tile_f32<2, 2>(a, dW, e, start, len, n0, k0, smem);
}

}  // namespace grp

int launch_grouped_wgrad(const GroupedWgradArgs& given, float* dW, void* stream) {
  GroupedWgradArgs a = given;
  int64_t tiles = ((a.N + 255) / 256) * ((a.K + 255) / 256);
  a.small = grp::wgrad_small(a.E, tiles);
  if (a.small) tiles = (a.N / 128) * (a.K / 128);
  const dim3 grid((unsigned)(a.E * tiles));
  hipLaunchKernelGGL(grp::grouped_wgrad_kernel, grid, dim3(grp::THREADS), 0, (hipStream_t)stream, a, dW);
  return (int)hipGetLastError();
}

int launch_grouped_step(int s_type, int opt, const GroupedWgradArgs& given, const EpiArgs& e, void* stream) {
  GroupedWgradArgs a = given;
  a.small = grp::wgrad_small(a.E, grp::wgrad_tiles(a.N, a.K, false));
  grp::GroupedStepFn fn = s_type == FORGE_S_F32  ? grp::select_grouped_step<FORGE_S_F32>(opt)
                          : s_type == FORGE_S_Q8 ? grp::select_grouped_step<FORGE_S_Q8>(opt)
                                                 : grp::select_grouped_step<FORGE_S_Q8D>(opt);
  if (!fn) return (int)hipErrorInvalidValue;
  const dim3 grid((unsigned)(a.E * (int64_t)grp::wgrad_tiles(a.N, a.K, a.small)));
  hipLaunchKernelGGL(fn, grid, dim3(ml2::THREADS), 0, (hipStream_t)stream, a, e);
  return (int)hipGetLastError();
}

}  // namespace forge

// forge_grouped.hip -- launchers of the products grouped by expert (forge_grouped.h,
// forge_grouped_wgrad.h), and the weight gradient kept in fp32.
#include <hip/hip_runtime.h>

#include "forge_grouped_wgrad.h"

namespace forge {

int launch_grouped_rows(int mode, const GroupedArgs& a, void* stream) {
  const int64_t O = mode == FORGE_GROUPED_NN ? a.K : a.N;
  const int64_t tiles = (a.T / 256 + (a.E < a.T ? a.E : a.T) + 1) * ((O + 255) / 256);
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

__global__ __launch_bounds__(ml2::THREADS, kOcc2) void grouped_wgrad_kernel(GroupedWgradArgs a, float* dW) {
  __shared__ __attribute__((aligned(1024))) unsigned char smem[kSmem2];
  grp::WTile t;
  grp::wgrad_tile(a, t);
  float* st = reinterpret_cast<float*>(smem);
  if (t.half) {
    ml2::floatx4 acc[4][4];
    ml2::contract<Pipe2H>(acc, smem, t.g, t.n0, t.k0);
    ml2::stage_acc_all(st, acc, 1.0f);
    __syncthreads();
    store_staged(st, dW, a.K, t.row0, t.k0);
  } else {
    ml2::floatx4 acc[8][4];
    ml2::contract<Pipe2>(acc, smem, t.g, t.n0, t.k0);
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
      ml2::stage_acc_half(st, acc, 1.0f, half);
      __syncthreads();
      store_staged(st, dW, a.K, t.row0 + half * ml2::EPI_ROWS, t.k0);
      __syncthreads();
    }
  }
}

int launch_grouped_wgrad(const GroupedWgradArgs& a, float* dW, void* stream) {
  const dim3 grid((unsigned)(a.E * (int64_t)grp::wgrad_tiles(a.N, a.K)));
  hipLaunchKernelGGL(grouped_wgrad_kernel, grid, dim3(ml2::THREADS), 0, (hipStream_t)stream, a, dW);
  return (int)hipGetLastError();
}

int launch_grouped_step(int s_type, int opt, const GroupedWgradArgs& a, const EpiArgs& e, void* stream) {
  grp::GroupedStepFn fn = s_type == FORGE_S_F32  ? grp::select_grouped_step<FORGE_S_F32>(opt)
                          : s_type == FORGE_S_Q8 ? grp::select_grouped_step<FORGE_S_Q8>(opt)
                                                 : grp::select_grouped_step<FORGE_S_Q8D>(opt);
  if (!fn) return (int)hipErrorInvalidValue;
  const dim3 grid((unsigned)(a.E * (int64_t)grp::wgrad_tiles(a.N, a.K)));
  hipLaunchKernelGGL(fn, grid, dim3(ml2::THREADS), 0, (hipStream_t)stream, a, e);
  return (int)hipGetLastError();
}

}  // namespace forge

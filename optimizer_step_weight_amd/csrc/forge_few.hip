// forge_few.hip -- the gated product and the block product of few rows (a decoded token, or some): a pass over
// the live experts' weights.
//
// A tile of the other kernels (forge_gated.hip, forge_block_gemm.hip) contracts alone, so few columns mean
// few workgroups, each at the latency of its own loads.  Here a workgroup takes 16 columns, and its 8 waves
// share the contraction and join their sums in LDS at the end.  Weights go straight to registers, several
// lines a row in flight: a wave's 16 weight rows are one side of a matrix block, up to 16 rows of X the
// other.  Both sides take the contraction's elements in the same order, which is chosen so that a load
// covers 64 consecutive bytes of each of 16 rows.  Two workgroups fit a CU: with twice the loads ahead of each wave
// one did, and its beginning and end were not covered (block product of 14336 x 4096, one row: 22 us; 19 us now).
//
// One row, gated product: 4096 x 4096 15 us (4.5 TB/s), 1408 x 2048 8.5 us (tiles: 14).  Block product, 4096 x 14336: 15 us
// for one row (3.9 TB/s), 22 us for 16; tiles: 94.  (Lanes without a row could spare their loads of X: no gain.)
#include <hip/hip_runtime.h>

#include "forge_act.h"
#include "forge_ffn_internal.h"
#include "forge_grouped.h"

namespace forge {
namespace grp {

typedef int intx8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int FEW_WAVES = 8, FEW_THREADS = 64 * FEW_WAVES;

// The rows of workgroup row `b`: at most ROWS of one group.
template <int ROWS>
__device__ __forceinline__ bool few_rows(const int32_t* ends, int E, int64_t T, int b, RowTile& t) {
  return find_tile<ROWS>(ends, E, T, 256, 256, b, t);
}

// Adds the waves' sums: wave 0 gets them.  N registers a lane.
template <int N>
__device__ __forceinline__ void join(floatx4 (&v)[N], floatx4* lds) {
  const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
  if (wave > 0)
#pragma unroll
    for (int i = 0; i < N; ++i) lds[((wave - 1) * N + i) * 64 + lane] = v[i];
  __syncthreads();
  if (wave > 0) return;
#pragma unroll
  for (int w = 0; w < FEW_WAVES - 1; ++w)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += lds[(w * N + i) * 64 + lane];
}

// A wave's share of `many` steps: [first, last).
__device__ __forceinline__ void share(int many, int& first, int& last) {
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  first = many * wave / FEW_WAVES;
  last = many * (wave + 1) / FEW_WAVES;
}

// f(M) for batches of at most AHEAD steps (a power of two), the last one no larger than it has to be: M steps are
// loaded together, those from `last` on for nothing.
template <int AHEAD, class F>
__device__ __forceinline__ void in_batches(int& s, int last, F&& f) {
  while (s < last) {
    if (AHEAD >= 8 && last - s > 4) f(std::integral_constant<int, 8>{}), s += 8;
    else if (AHEAD >= 4 && last - s > 2) f(std::integral_constant<int, 4>{}), s += 4;
    else f(std::integral_constant<int, 2>{}), s += 2;
  }
}

// 16 R rows by 16 columns in steps of 64 elements (128 bytes of a row), AHEAD of which are loaded at once.
template <int R, int AHEAD>
__global__ __launch_bounds__(FEW_THREADS) void gated_few_kernel(GatedArgs a) {
  __shared__ floatx4 lds[(FEW_WAVES - 1) * 2 * R * 64];
  RowTile t;
  if (!few_rows<16 * R>(a.ends, a.E, a.T, (int)blockIdx.y, t)) return;
  const int lane = (int)threadIdx.x & 63, row = lane & 15, q = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  floatx4 sum[2 * R];  // gate and up of each 16 rows
#pragma unroll
  for (int i = 0; i < 2 * R; ++i) sum[i] = floatx4{};
  if (t.e < a.E) {
    const uint16_t* x[R];
#pragma unroll
    for (int r = 0; r < R; ++r)
      x[r] = static_cast<const uint16_t*>(a.X) + (int64_t)(t.row0 + (16 * r + row < t.rows ? 16 * r + row : 0)) * a.K + 8 * q;
    const uint16_t* g = static_cast<const uint16_t*>(a.W) + ((int64_t)t.e * 2 * a.N + n0 + row) * a.K + 8 * q;
    const uint16_t* u = g + a.N * a.K;
    int s, last;
    share((int)(a.K / 64), s, last);
    in_batches<AHEAD>(s, last, [&](auto many) {
      constexpr int M = 2 * decltype(many)::value;  // products' 32 elements
      u32x4 wg[M], wu[M], xs[R][M];
#pragma unroll
      for (int i = 0; i < M; ++i) {
        const int at = (s + i / 2 < last ? s + i / 2 : last - 1) * 64 + 32 * (i & 1);
        wg[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(g + at));
        wu[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(u + at));
#pragma unroll
        for (int r = 0; r < R; ++r) xs[r][i] = ld16(x[r] + at);
      }
      __builtin_amdgcn_sched_barrier(0);  // all loads first
#pragma unroll
      for (int i = 0; i < M; ++i) {
        if (s + i / 2 >= last) break;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const bf16x8 xv = __builtin_bit_cast(bf16x8, xs[r][i]);
          sum[2 * r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, wg[i]), xv, sum[2 * r], 0, 0, 0);
          sum[2 * r + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, wu[i]), xv, sum[2 * r + 1], 0, 0, 0);
        }
      }
    });
  }
  join(sum, lds);
  if (threadIdx.x >= 64) return;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (16 * r + row >= t.rows) break;
    // this lane: columns n0 + 4 q .. + 3 of a row
    const int64_t tok = t.row0 + 16 * r + row, n = n0 + 4 * q;
    const floatx4 g = sum[2 * r], u = sum[2 * r + 1];
    floatx4 h;
    by_act(a.act, [&](auto act) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float v, d;
        act_pair<decltype(act)::value>(g[i], v, d);
        h[i] = v * u[i];
      }
    });
    auto put = [](uint16_t* p, const floatx4& v) {
      *reinterpret_cast<u32x2*>(p) = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    };
    put(a.H + tok * a.N + n, h);
    if (a.keep.type == FORGE_KEEP_BF16) {
      uint16_t* p = static_cast<uint16_t*>(a.keep.data) + tok * 2 * a.N + n;
      put(p, g);
      put(p + a.N, u);
    }
  }
}

// The same of codes, in steps of one block of 128.
template <int R, int AHEAD>
__global__ __launch_bounds__(FEW_THREADS) void block_few_kernel(BlockGemmArgs a) {
  __shared__ floatx4 lds[(FEW_WAVES - 1) * R * 64];
  RowTile t;
  if (!few_rows<16 * R>(a.ends, a.E, a.T, (int)blockIdx.y, t)) return;
  const int lane = (int)threadIdx.x & 63, row = lane & 15, q = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  floatx4 sum[R];
#pragma unroll
  for (int r = 0; r < R; ++r) sum[r] = floatx4{};
  if (t.e < a.E) {
    const int KB = (int)(a.K / 128);
    const uint8_t* x[R];
    const float* sx[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t tok = t.row0 + (16 * r + row < t.rows ? 16 * r + row : 0);
      x[r] = a.X + tok * a.K + 16 * q;
      sx[r] = a.x_scale + tok * KB;
    }
    const uint8_t* w = a.W + ((int64_t)t.e * a.N + n0 + row) * a.K + 16 * q;
    const float* sw = a.w_scale + ((int64_t)t.e * (a.N / 128) + n0 / 128) * KB;
    int s, last;
    share(KB, s, last);
    in_batches<AHEAD>(s, last, [&](auto many) {
      constexpr int M = decltype(many)::value;
      u32x4 wv[2 * M], xv[R][2 * M];
      float f[R][M];
#pragma unroll
      for (int i = 0; i < M; ++i) {
        const int b = s + i < last ? s + i : last - 1;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          wv[2 * i + h] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(w + b * 128 + 64 * h));
#pragma unroll
          for (int r = 0; r < R; ++r) xv[r][2 * i + h] = ld16(x[r] + b * 128 + 64 * h);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) f[r][i] = sx[r][b];
      }
      __builtin_amdgcn_sched_barrier(0);  // all loads first
      auto whole = [](u32x4 lo, u32x4 hi) {
        return __builtin_bit_cast(intx8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
      };
#pragma unroll
      for (int i = 0; i < M; ++i) {
        if (s + i >= last) break;
        const float by = sw[s + i];
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const floatx4 part = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              whole(wv[2 * i], wv[2 * i + 1]), whole(xv[r][2 * i], xv[r][2 * i + 1]), floatx4{}, 0, 0, 0, 0, 0, 0);
#pragma unroll
          for (int j = 0; j < 4; ++j) sum[r][j] = __builtin_fmaf(part[j], f[r][i] * by, sum[r][j]);
        }
      }
    });
  }
  join(sum, lds);
  if (threadIdx.x >= 64) return;
#pragma unroll
  for (int r = 0; r < R; ++r)
    if (16 * r + row < t.rows)
      *reinterpret_cast<u32x2*>(a.Y + (int64_t)(t.row0 + 16 * r + row) * a.N + n0 + 4 * q) =
          u32x2{pack_bf16(sum[r][0], sum[r][1]), pack_bf16(sum[r][2], sum[r][3])};
}

}  // namespace grp

// Row tiles of `rows`: every group has at most one more than its rows fill, and so have the rows of no group.
template <class Args, class Kernel>
static int launch_few(Kernel kernel, const Args& a, int rows, void* stream) {
  const dim3 grid((unsigned)(a.N / 16), (unsigned)(a.T / rows + (a.E < a.T ? a.E : a.T) + 1));
  hipLaunchKernelGGL(kernel, grid, dim3(grp::FEW_THREADS), 0, (hipStream_t)stream, a);
  return (int)hipGetLastError();
}

int launch_gated_few(const GatedArgs& a, void* stream) {
  if (a.T <= 16) return launch_few(grp::gated_few_kernel<1, 4>, a, 16, stream);
  if (a.T <= 32) return launch_few(grp::gated_few_kernel<2, 2>, a, 32, stream);
  return launch_few(grp::gated_few_kernel<4, 2>, a, 64, stream);
}
int launch_block_few(const BlockGemmArgs& a, void* stream) {
  if (a.T <= 16) return launch_few(grp::block_few_kernel<1, 4>, a, 16, stream);
  if (a.T <= 32) return launch_few(grp::block_few_kernel<2, 4>, a, 32, stream);
  return launch_few(grp::block_few_kernel<4, 2>, a, 64, stream);
}

}  // namespace forge

// forge_gated.h -- what the products with a gated activation in their epilogue share: a tile's results
// pass through LDS in fp32, and leave by rows.
//
// The activation needs gate and up of one column together and a block's scale needs 128 columns of one
// row, while a wave of the contraction (forge_grouped.h) holds 128 x 128 of the tile.  So all four waves
// put up to 64 rows each into LDS (128 x 256 fp32, 128 KiB of the 160 that the contraction has left), and
// the workgroup takes them from there row after row in a loop of one short body: the activations of a
// tile unrolled over its 256 accumulators would not fit the instruction cache.
#pragma once

#include "forge_act.h"
#include "forge_grouped.h"

namespace forge {
namespace grp {

// The rounds in which a tile of HEIGHT x 64 rows passes: G blocks of 16 rows of each half of the tile.
template <int HEIGHT, int WIDTH>
struct Rounds {
  static constexpr int MB = 2 * HEIGHT, G = MB <= 4 ? MB : MB / 2, N = MB / G;
  static constexpr int ROWS = 32 * G, ROW_BYTES = 256 * WIDTH;  // of a round, of a row of 64 WIDTH floats
  // Row `r` of round `i` in the tile.
  static __device__ __forceinline__ int tile_row(int i, int r) {
    const int half = r / (16 * G);
    return half * 16 * MB + 16 * G * i + (r - half * 16 * G);
  }
  // Chunk c (4 floats) of row r.  16 rows at one chunk fall into 16 places (as they are written), and so do two
  // rows at every other chunk (as 8 threads a row read them).
  static __device__ __forceinline__ unsigned char* at(unsigned char* smem, int r, int c) {
    return smem + r * ROW_BYTES + 16 * (c ^ (r & 15));
  }
  template <int I, class T>
  static __device__ __forceinline__ void put(unsigned char* smem, const T& tile) {
    const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
#pragma unroll
    for (int b = 0; b < G; ++b)
#pragma unroll
      for (int j = 0; j < T::NB; ++j)
        *reinterpret_cast<floatx4*>(at(smem, (wave >> 1) * 16 * G + 16 * b + (lane & 15),
                                       (wave & 1) * 4 * T::NB + 4 * j + (lane >> 4))) = tile.acc[I * G + b][j];
  }
  // Eight columns of row r from chunk c on.
  static __device__ __forceinline__ void get(unsigned char* smem, int r, int c, float* v) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const floatx4 x = *reinterpret_cast<const floatx4*>(at(smem, r, c + j));
#pragma unroll
      for (int i = 0; i < 4; ++i) v[4 * j + i] = x[i];
    }
  }
};

// Calls row_pass(round, first row in LDS) for every round with its rows in LDS.
template <int HEIGHT, int WIDTH, class T, class F>
__device__ __forceinline__ void by_rounds(unsigned char* smem, const T& tile, F&& row_pass) {
  using R = Rounds<HEIGHT, WIDTH>;
  static_for<R::N>([&](auto ic) {
    constexpr int i = decltype(ic)::value;
    __syncthreads();  // the slabs, or the round before, have been read
    R::template put<i>(smem, tile);
    __syncthreads();
    row_pass(i);
  });
}

__device__ __forceinline__ u32x4 to_bf16x8(const float* v) {
  return u32x4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
}

}  // namespace grp
}  // namespace forge

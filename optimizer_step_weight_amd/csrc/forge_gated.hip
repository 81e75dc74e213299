// forge_gated.hip -- H = act(X Wg^T) * (X Wu^T) for the rows of every group, and gate and up as they are
// kept for the backward pass, in one launch.
//
// A tile of forge_grouped.h takes 128 columns of H: its 256 rows of the stacked weight [2 N, K] are the 128
// gate rows of these columns and their 128 up rows, which is all that the products know of the
// activation.  The epilogue is in forge_gated.h.
//
// 8192 rows by 14336 x 4096 with gate and up in e4m3: 1345-1412 us over the cards seen (1.36-1.43 PFLOP/s), 1283 without
// them; the grouped product of the stacked weight alone takes 1272-1281.  The card's power bounds it: matrix cores 71 %
// busy at 1.9 GHz.  16384 rows of 32 uneven experts by 1408 x 2048 with both in bf16: 195-211 us (0.90-0.97 PFLOP/s;
// the grouped product alone 185-188), 43 % busy at 2.2 GHz: 902 tiles on 256 CUs, many of them of few rows.  One row by
// 14336 x 4096: 48-56 us, 4.2-4.9 TB/s of weights.
#include <hip/hip_runtime.h>

#include "forge_gated.h"

namespace forge {
namespace grp {

// The operand of S::WIDTH / 2 rows from `first` on and as many `gap` bytes after them.
template <class S>
__device__ __forceinline__ void open_pair(Feed<S>& f, const void* first, uint32_t gap, uint32_t ld, int slabs) {
  constexpr int HALF = S::WIDTH / 2;
  f.open(first, gap + HALF * ld, ld, slabs);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int j = 0; j < S::DMA; ++j) {
    const int r = S::RPD * (S::DMA * wave + j) + lane / S::CPR;
    if (r >= HALF) f.off[j] += gap - (uint32_t)HALF * ld;
  }
}

// 16 columns of a row of H from gate and up: 8 from column n on, and 8 from n + HALF on.  So a store of 16 bytes a
// thread covers whole lines of a row (16 columns in one piece: gate and up in bf16 205 -> 212 us for 16384 rows of
// 32 experts of 1408 x 2048), and the work on a block's scale is shared by half as many threads as 8 columns would
// have (8192 x 14336 x 4096, codes: 1445 -> 1375 us).
//
// Addresses are the tile's, the same in all lanes, and 32-bit offsets in it (at most 256 rows of 2^20 columns).
struct GatedOut {
  unsigned char *h, *g, *u;   // of the tile's first row and column
  float *gs, *us;             // its scales
  uint32_t ld_h, ld_gu, ld_s; // bytes from row to row
  __device__ __forceinline__ GatedOut(const GatedArgs& a, int64_t row0, int64_t n0) {
    const int esz = a.keep.type == FORGE_KEEP_BF16 ? 2 : 1;
    h = reinterpret_cast<unsigned char*>(a.H + row0 * a.N + n0);
    g = static_cast<unsigned char*>(a.keep.data) + (row0 * 2 * a.N + n0) * esz;
    u = g + a.N * esz;
    gs = a.keep.scale + row0 * (a.N / 64) + n0 / 128;
    us = gs + a.N / 128;
    ld_h = (uint32_t)(2 * a.N);
    ld_gu = (uint32_t)(2 * a.N * esz);
    ld_s = (uint32_t)(a.N / 64);
  }
};

template <int HALF>
__device__ __forceinline__ void gated_row(const GatedArgs& a, const GatedOut& o, int row, int col, bool live,
                                          const float (&g)[16], const float (&u)[16]) {
  float h[16];
  by_act(a.act, [&](auto act) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float v, s;
      act_pair<decltype(act)::value>(g[i], v, s);
      h[i] = v * u[i];
    }
  });
  auto put = [&](unsigned char* base, uint32_t at, const float (&v)[16]) {
    if (!live) return;
    st16_stream(base + at, to_bf16x8(v));
    st16_stream(base + at + 2 * HALF, to_bf16x8(v + 8));
  };
  put(o.h, (uint32_t)row * o.ld_h + 2u * (uint32_t)col, h);
  if (a.keep.type == FORGE_KEEP_BF16) {
    const uint32_t at = (uint32_t)row * o.ld_gu + 2u * (uint32_t)col;
    put(o.g, at, g);
    put(o.u, at, u);
  }
  if constexpr (HALF == 64) {  // 8 lanes have a block's 128 columns
    auto eight = [&](auto qc) {
      constexpr int Q = decltype(qc)::value;
      const uint32_t at = (uint32_t)row * o.ld_gu + (uint32_t)col;
      auto part = [&](const float (&v)[16], unsigned char* base, float* scales) {
        const float scale = block_scale<Q>(max8(amax_bits(v)));
        if (!live) return;
        uint32_t q[4];
        encode<Q>(v, scale, q);
        store_codes<false>(base + at, u32x2{q[0], q[1]}, 8);
        store_codes<false>(base + at + HALF, u32x2{q[2], q[3]}, 8);
        if ((threadIdx.x & 7) == 0) scales[(uint32_t)row * o.ld_s] = scale;
      };
      part(g, o.g, o.gs);
      part(u, o.u, o.us);
    };
    if (a.keep.type == FORGE_KEEP_FP8) eight(std::integral_constant<int, FORGE_Q_FP8>{});
    if (a.keep.type == FORGE_KEEP_I8) eight(std::integral_constant<int, FORGE_Q_I8>{});
  }
}

template <int HEIGHT, int WIDTH>
__device__ __forceinline__ void gated_tile(const GatedArgs& a, const RowTile& t, unsigned char* smem) {
  using A = Side<2, false, 64 * HEIGHT>;
  using B = Side<2, false, 64 * WIDTH>;
  const int64_t n0 = (int64_t)t.n * (32 * WIDTH);  // column of H
  const int slabs = t.e < a.E ? (int)(a.K / 64) : 0;
  const uint32_t ld = (uint32_t)(a.K * 2);
  Feed<A> fa;
  Feed<B> fb;
  fa.open(static_cast<const uint16_t*>(a.X) + (int64_t)t.row0 * a.K, (uint32_t)(t.rows * ld), ld, slabs);
  open_pair(fb, static_cast<const uint16_t*>(a.W) + ((int64_t)t.e * 2 * a.N + n0) * a.K, (uint32_t)(a.N * ld), ld, slabs);
  Tile<A, B> tile;
  tile.contract(smem, fa, fb, slabs);
  using R = Rounds<HEIGHT, WIDTH>;
  constexpr int LANES = 2 * WIDTH;  // of a row
  const GatedOut out(a, t.row0, n0);
  by_rounds<HEIGHT, WIDTH>(smem, tile, [&](int round) {
    const int p = (int)threadIdx.x % LANES;
    for (int r = (int)threadIdx.x / LANES; r < R::ROWS; r += THREADS / LANES) {
      const int row = R::tile_row(round, r);
      float g[16], u[16];
      R::get(smem, r, 2 * p, g);
      R::get(smem, r, 2 * p + 4 * WIDTH, g + 8);
      R::get(smem, r, 2 * p + 8 * WIDTH, u);
      R::get(smem, r, 2 * p + 12 * WIDTH, u + 8);
      gated_row<16 * WIDTH>(a, out, row, 8 * p, row < t.rows, g, u);
    }
  });
}

__global__ __launch_bounds__(THREADS, 1) void gated_kernel(GatedArgs a) {
  __shared__ __attribute__((aligned(1024))) unsigned char smem[5 * 32768];
  RowTile t;
  if (!find_tile<256>(a.ends, a.E, a.T, 2 * a.N, a.cols, (int)blockIdx.x, t)) return;
  switch ((t.rows + 63) / 64 + (t.cols < 256 ? 4 : 0)) {
    case 1: gated_tile<1, 4>(a, t, smem); break;
    case 2: gated_tile<2, 4>(a, t, smem); break;
    case 3: gated_tile<3, 4>(a, t, smem); break;
    case 4: gated_tile<4, 4>(a, t, smem); break;
    case 5: gated_tile<1, 2>(a, t, smem); break;
    case 6: gated_tile<2, 2>(a, t, smem); break;
    case 7: gated_tile<3, 2>(a, t, smem); break;
    case 8: gated_tile<4, 2>(a, t, smem); break;
  }
}

}  // namespace grp

int launch_grouped_gated(const GatedArgs& given, void* stream) {
  if (given.keep.type < FORGE_KEEP_FP8 && few_rows_call(given.T, given.E, given.N, 64, kFewGated)) return launch_gated_few(given, stream);
  GatedArgs a = given;
  const int64_t O = 2 * a.N;
  const int64_t row_tiles = a.T / 256 + (a.E < a.T ? a.E : a.T) + 1;
  // as launch_grouped_rows; a narrow tile has half a block of 8-bit gate and up
  a.cols = a.keep.type < FORGE_KEEP_FP8 && a.T / 256 * ((O + 255) / 256) <= grp::NARROW_TILES ? 128 : 256;
  const int64_t tiles = row_tiles * ((O + a.cols - 1) / a.cols);
  hipLaunchKernelGGL(grp::gated_kernel, dim3((unsigned)tiles), dim3(grp::THREADS), 0, (hipStream_t)stream, a);
  return (int)hipGetLastError();
}

}  // namespace forge

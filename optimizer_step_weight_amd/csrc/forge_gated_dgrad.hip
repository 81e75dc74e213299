// forge_gated_dgrad.hip -- the backward pass of H = act(g) u from the gradient of what the down projection
// makes of H: dH = dY W stays in the tile, whose epilogue reads gate and up and writes
//     dg = dH u act'(g),  du = dH act(g),  H = act(g) u.
// Without it dH would be written and read again, 4 bytes beside the 6 to 10 that an element cannot do without.
#include <hip/hip_runtime.h>

#include "forge_gated.h"

namespace forge {
namespace grp {

// 8 columns of gate or up as loaded, and what they stand for.
struct KeptRaw {
  u32x4 q;
  float scale;
};
__device__ __forceinline__ KeptRaw load_kept(const KeptArgs& k, int64_t row, int64_t N, int64_t col) {
  KeptRaw r{};
  if (k.type == FORGE_KEEP_BF16) {
    r.q = ld16(static_cast<const uint16_t*>(k.data) + row * 2 * N + col);
  } else {
    const u32x2 c = ld8(static_cast<const uint8_t*>(k.data) + row * 2 * N + col);
    r.q[0] = c[0];
    r.q[1] = c[1];
    r.scale = k.scale[row * (N / 64) + (col >> 7)];
  }
  return r;
}
__device__ __forceinline__ void kept_value(int type, const KeptRaw& r, float (&v)[8]) {
  if (type == FORGE_KEEP_BF16) unpack8<true>(Raw8<true>{{r.q}}, v);
  else if (type == FORGE_KEEP_FP8) decode8<FORGE_Q_FP8>(u32x2{r.q[0], r.q[1]}, r.scale, v);
  else decode8<FORGE_Q_I8>(u32x2{r.q[0], r.q[1]}, r.scale, v);
}

template <int HEIGHT, int WIDTH>
__device__ __forceinline__ void gated_dgrad_tile(const GatedDgradArgs& a, const RowTile& t, unsigned char* smem) {
  using A = Side<2, false, 64 * HEIGHT>;
  using B = Side<2, true, 64 * WIDTH>;
  const int64_t n0 = (int64_t)t.n * t.cols;
  const int slabs = t.e < a.E ? (int)(a.K / 64) : 0;
  Feed<A> fa;
  Feed<B> fb;
  fa.open(static_cast<const uint16_t*>(a.dY) + (int64_t)t.row0 * a.K, (uint32_t)(t.rows * a.K * 2), (uint32_t)(a.K * 2),
          slabs);
  fb.open(static_cast<const uint16_t*>(a.W) + (int64_t)t.e * a.N * a.K + n0, (uint32_t)(a.N * a.K * 2 - n0 * 2),
          (uint32_t)(a.N * 2), slabs);
  Tile<A, B> tile;
  tile.contract(smem, fa, fb, slabs);
  using R = Rounds<HEIGHT, WIDTH>;
  constexpr int LANES = 8 * WIDTH, PER = THREADS / LANES;
  by_rounds<HEIGHT, WIDTH>(smem, tile, [&](int round) {
    const int p = (int)threadIdx.x % LANES;
    const int64_t n = n0 + 8 * p;
#pragma unroll 1
    for (int r = (int)threadIdx.x / LANES; r < R::ROWS; r += PER) {
      const int tr = R::tile_row(round, r);
      if (tr >= t.rows) continue;
      const int64_t row = t.row0 + tr;
      float g[8], u[8], d[8], h[8];
      kept_value(a.keep.type, load_kept(a.keep, row, a.N, n), g);
      kept_value(a.keep.type, load_kept(a.keep, row, a.N, a.N + n), u);
      R::get(smem, r, 0, p, d);
      by_act(a.act, [&](auto act) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float v, s;
          act_pair<decltype(act)::value>(g[i], v, s);
          h[i] = v * u[i];
          g[i] = d[i] * u[i] * s;
          u[i] = d[i] * v;
        }
      });
      uint16_t* o = a.dGU + row * 2 * a.N + n;
      if (t.e == a.E) {  // rows of no group
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = u[i] = h[i] = 0.0f;
      }
      st16_stream(o, to_bf16x8(g));
      st16_stream(o + a.N, to_bf16x8(u));
      if (a.H) st16_stream(a.H + row * a.N + n, to_bf16x8(h));
    }
  });
}

__global__ __launch_bounds__(THREADS, 1) void gated_dgrad_kernel(GatedDgradArgs a) {
  __shared__ __attribute__((aligned(1024))) unsigned char smem[5 * 32768];
  RowTile t;
  if (!find_tile<256>(a.ends, a.E, a.T, a.N, a.cols, (int)blockIdx.x, t)) return;
  const bool narrow = t.cols < 256 || a.N - (int64_t)t.n * 256 < 256;
  switch ((t.rows + 63) / 64 + (narrow ? 4 : 0)) {
    case 1: gated_dgrad_tile<1, 4>(a, t, smem); break;
    case 2: gated_dgrad_tile<2, 4>(a, t, smem); break;
    case 3: gated_dgrad_tile<3, 4>(a, t, smem); break;
    case 4: gated_dgrad_tile<4, 4>(a, t, smem); break;
    case 5: gated_dgrad_tile<1, 2>(a, t, smem); break;
    case 6: gated_dgrad_tile<2, 2>(a, t, smem); break;
    case 7: gated_dgrad_tile<3, 2>(a, t, smem); break;
    case 8: gated_dgrad_tile<4, 2>(a, t, smem); break;
  }
}

}  // namespace grp

int launch_grouped_gated_dgrad(const GatedDgradArgs& given, void* stream) {
  GatedDgradArgs a = given;
  const int64_t row_tiles = a.T / 256 + (a.E < a.T ? a.E : a.T) + 1;
  a.cols = a.T / 256 * ((a.N + 255) / 256) <= grp::NARROW_TILES ? 128 : 256;  // as launch_grouped_rows
  const int64_t tiles = row_tiles * ((a.N + a.cols - 1) / a.cols);
  hipLaunchKernelGGL(grp::gated_dgrad_kernel, dim3((unsigned)tiles), dim3(grp::THREADS), 0, (hipStream_t)stream, a);
  return (int)hipGetLastError();
}

}  // namespace forge

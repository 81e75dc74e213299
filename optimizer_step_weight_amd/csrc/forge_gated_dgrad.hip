// forge_gated_dgrad.hip -- the backward pass of H = act(g) u from the gradient of what the down projection
// makes of H: dH = dY W stays in the tile, whose epilogue reads gate and up and writes
//     dg = dH u act'(g),  du = dH act(g),  H = act(g) u.
// Without it dH would be written and read again, 4 bytes beside the 6 to 10 that an element cannot do without.
//
// 8192 rows by 14336 x 4096 from int8: 818-850 us over the cards seen (1.13-1.18 PFLOP/s and 0.95 GB; the grouped input gradient
// and the activation's backward pass one after the other take 667 + 193, and 235 MB for dH).  Without its stores the
// kernel takes 60 us less, without gate and up 65, without the activation 20.  16384 rows of 32 uneven experts by 1408 x
// 2048 from bf16: 135-148 us; apart they take 95 + 41, no longer, but 46 MB for dH.  Tiles whose epilogues come at different times (every other CU, or XCD,
// begins with half a tile) share less in L2: 826 -> 860 and 845 us.  Tiles of few rows or columns are not split further:
// the last 256 tiles of a launch in two halves 145 -> 160 us for the experts.
#include <hip/hip_runtime.h>

#include "forge_gated.h"

namespace forge {
namespace grp {

// The epilogue takes 32 rows of the tile a round, 16 of either half: their dH passes through LDS as in
// forge_gated.h, and so do their gate and up, which are copied there two rounds ahead (64 KiB under way in bf16).
// Loads straight to registers would have to wait there beside accumulators that are not yet out: one pass over
// the threads at a time left 43 us of latency a tile, beside a contraction of 100 us (1018 us for what takes 820 now),
// and several at a time spilled 400 to 1000 registers.
//
// ESZ bytes an element; blocks of 128 columns have their scales where ESZ is 1.
template <int HEIGHT, int WIDTH, int ESZ>
struct KeptRounds {
  static constexpr int N = 2 * HEIGHT, ROWS = 32;
  static constexpr int SEG = 64 * WIDTH * ESZ;                 // bytes of a row's gate, or up
  static constexpr int PART = ROWS * SEG, BYTES = 2 * PART;    // gate, or up, of a round; both
  static constexpr int COPIES = BYTES / 4096;                  // of 1 KiB, of a wave
  static constexpr int STAGE = ROWS * 256 * WIDTH, AHEAD = 3 * BYTES, SCALES = 3 * 1024;
  static constexpr int DMA = COPIES + (ESZ == 1 ? 1 : 0);
  static_assert(STAGE + AHEAD + SCALES <= 5 * 32768 && COPIES >= 1, "LDS");
  u32x4 rsrc, rscale;
  uint32_t off[COPIES], off_scale;   // of this lane's pieces in round 0
  uint32_t step, step_scale, lds;    // 16 rows further

  static __device__ __forceinline__ int tile_row(int round, int r) { return (r >> 4) * 16 * N + 16 * round + (r & 15); }

  __device__ __forceinline__ void open(const KeptArgs& k, const RowTile& t, int64_t N2, int64_t n0, unsigned char* smem) {
    const int lane = (int)threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const uint32_t ld = (uint32_t)(2 * N2 * ESZ);
    lds = lds_address(smem) + STAGE;
    rsrc = make_rsrc(static_cast<const unsigned char*>(k.data) + ((int64_t)t.row0 * 2 * N2 + n0) * ESZ,
                     (uint32_t)t.rows * ld - (uint32_t)(n0 * ESZ));
    step = 16 * ld;
#pragma unroll
    for (int j = 0; j < COPIES; ++j) {
      const int at = (COPIES * wave + j) * 1024 + 16 * lane, part = at / PART, in = at - part * PART, r = in / SEG;
      off[j] = (uint32_t)tile_row(0, r) * ld + (uint32_t)part * (uint32_t)(N2 * ESZ) + (uint32_t)(in - r * SEG);
    }
    if constexpr (ESZ == 1) {  // lane e: row e / 4, gate or up, block of 128
      const int64_t blocks = N2 / 128;
      const int e = 64 * wave + lane, per = 2 * (WIDTH / 2), r = e / per, part = e % per / (WIDTH / 2), b = e % (WIDTH / 2);
      rscale = make_rsrc(k.scale + (int64_t)t.row0 * 2 * blocks, (uint32_t)(t.rows * 2 * blocks * 4));
      off_scale = r < ROWS ? (uint32_t)((tile_row(0, r) * 2 * blocks + part * blocks + n0 / 128 + b) * 4) : 0xFFFFFFF0u;
      step_scale = (uint32_t)(32 * blocks * 4);
      if (r >= ROWS) step_scale = 0;
    }
  }
  // The copies of a round; rows behind the tile's last give zeros.
  __device__ __forceinline__ void copy(int round) {
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const uint32_t to = lds + (uint32_t)(round % 3 * BYTES + wave * COPIES * 1024);
    static_for<COPIES>([&](auto j) { copy_1k<j * 1024>(rsrc, off[j] + (uint32_t)round * step, to); });
    if constexpr (ESZ == 1)
      copy_256(rscale, off_scale + (uint32_t)round * step_scale, lds + (uint32_t)(AHEAD + round % 3 * 1024 + wave * 256));
  }
  // 4 bytes a lane.
  static __device__ __forceinline__ void copy_256(const u32x4& rs, uint32_t o, uint32_t to) {
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(to), "v"(o), "s"(rs) : "memory", "m0");
#pragma clang diagnostic pop
  }
  // Columns 8 p .. of row r of gate (part 0) or up.
  template <int KEEP>
  __device__ __forceinline__ void get(unsigned char* smem, int round, int part, int r, int p, float (&v)[8]) const {
    const unsigned char* at = smem + STAGE + round % 3 * BYTES + part * PART + r * SEG + 8 * ESZ * p;
    if constexpr (ESZ == 2) {
      unpack8<true>(Raw8<true>{{ld16(at)}}, v);
    } else {
      const float* s = reinterpret_cast<const float*>(smem + STAGE + AHEAD + round % 3 * 1024);
      decode8<KEEP == FORGE_KEEP_FP8 ? FORGE_Q_FP8 : FORGE_Q_I8>(ld8(at), s[(r * 2 + part) * (WIDTH / 2) + p / 16], v);
    }
  }
};

template <int HEIGHT, int WIDTH, int KEEP, class T>
__device__ __forceinline__ void gated_dgrad_out(const GatedDgradArgs& a, const RowTile& t, unsigned char* smem, const T& tile,
                                                int64_t n0) {
  using K = KeptRounds<HEIGHT, WIDTH, KEEP == FORGE_KEEP_BF16 ? 2 : 1>;
  constexpr int LANES = 8 * WIDTH, PER = THREADS / LANES;
  static_assert(K::ROWS % (2 * PER) == 0, "whole passes");
  const int p = (int)threadIdx.x % LANES, lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
  // Stores are range-checked: rows behind the tile's last are dropped, but every wave issues the same stores, as the
  // waits below count them (loads and stores of a wave complete in order).
  const uint32_t ld = (uint32_t)(2 * a.N);
  const uint16_t* first = a.dGU + (int64_t)t.row0 * 2 * a.N + n0;
  auto range = [](const uint16_t* p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(p), 0, (int)bytes, 0x00020000);
  };
  const auto rd = range(first, (uint32_t)t.rows * 2 * ld - (uint32_t)(2 * n0));
  const auto rh = range(a.H ? a.H + (int64_t)t.row0 * a.N + n0 : nullptr, a.H ? (uint32_t)t.rows * ld - (uint32_t)(2 * n0) : 0u);
  auto store = [](const u32x4& q, __amdgpu_buffer_rsrc_t rsrc, uint32_t at) {
    __builtin_amdgcn_raw_buffer_store_b128(q, rsrc, at, 0, 2);  // 2: streaming
  };
  const bool none = t.e == a.E;  // rows of no group
  auto chunk = [&](int r, int c) { return reinterpret_cast<floatx4*>(smem + r * 256 * WIDTH + 16 * (c ^ (r & 15))); };
  K kept;
  kept.open(a.keep, t, a.N, n0, smem);
  barrier();  // every wave is done with the slabs
  kept.copy(0);
  if (K::N > 1) kept.copy(1);
#pragma unroll 1
  for (int round = 0; round < K::N; ++round) {
    if (round + 2 < K::N) kept.copy(round + 2);
    static_for<K::N>([&](auto ic) {
      constexpr int i = decltype(ic)::value;
      if (round == i)
#pragma unroll
        for (int j = 0; j < T::NB; ++j)
          *chunk((wave >> 1) * 16 + (lane & 15), (wave & 1) * 4 * T::NB + 4 * j + (lane >> 4)) = tile.acc[i][j];
    });
    // this round's copies have landed; those of the next two rounds may be under way, and the last round's stores
    constexpr int S = 3 * K::ROWS / PER;
    if (round == 0) {
      if (K::N > 2) wait_vm<2 * K::DMA>();
      else wait_vm<K::DMA>();
    } else if (round + 2 < K::N) {
      wait_vm<2 * K::DMA + S>();
    } else if (round + 1 < K::N) {
      wait_vm<K::DMA + S>();
    } else {
      wait_vm<S>();
    }
    __builtin_amdgcn_s_waitcnt(0xF | (0x3 << 14) | (0x7 << 4));  // LDS
    barrier();
    // two passes over the threads at a time, or their waits for LDS and the exponentials would be in the open
    by_act(a.act, [&](auto act) {
#pragma unroll 1
      for (int r = (int)threadIdx.x / LANES; r < K::ROWS; r += 2 * PER) {
        float g[2][8], u[2][8], h[2][8], d[2][8];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int ri = r + PER * i;
          kept.template get<KEEP>(smem, round, 0, ri, p, g[i]);
          kept.template get<KEEP>(smem, round, 1, ri, p, u[i]);
          const floatx4 d0 = *chunk(ri, 2 * p), d1 = *chunk(ri, 2 * p + 1);
#pragma unroll
          for (int j = 0; j < 8; ++j) d[i][j] = j < 4 ? d0[j] : d1[j - 4];
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float v, s;
            act_pair<decltype(act)::value>(g[i][j], v, s);
            h[i][j] = v * u[i][j];
            g[i][j] = d[i][j] * u[i][j] * s;
            u[i][j] = d[i][j] * v;
          }
          const uint32_t at = (uint32_t)K::tile_row(round, r + PER * i) * ld, lane_at = 16u * (uint32_t)p;
          if (none)
#pragma unroll
            for (int j = 0; j < 8; ++j) g[i][j] = u[i][j] = h[i][j] = 0.0f;
          store(to_bf16x8(g[i]), rd, 2 * at + lane_at);
          store(to_bf16x8(u[i]), rd, 2 * at + lane_at + ld);
          store(to_bf16x8(h[i]), rh, at + lane_at);
        }
      }
    });
    barrier();  // the round's rows have been read (their values are in registers, in order)
  }
}

template <int HEIGHT, int WIDTH, int KEEP>
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
  gated_dgrad_out<HEIGHT, WIDTH, KEEP>(a, t, smem, tile, n0);
}

template <int KEEP>
__global__ __launch_bounds__(THREADS, 1) void gated_dgrad_kernel(GatedDgradArgs a) {
  __shared__ __attribute__((aligned(1024))) unsigned char smem[5 * 32768];
  RowTile t;
  if (!find_tile<256>(a.ends, a.E, a.T, a.N, a.cols, (int)blockIdx.x, t)) return;
  const bool narrow = t.cols < 256 || a.N - (int64_t)t.n * 256 < 256;
  switch ((t.rows + 63) / 64 + (narrow ? 4 : 0)) {
    case 1: gated_dgrad_tile<1, 4, KEEP>(a, t, smem); break;
    case 2: gated_dgrad_tile<2, 4, KEEP>(a, t, smem); break;
    case 3: gated_dgrad_tile<3, 4, KEEP>(a, t, smem); break;
    case 4: gated_dgrad_tile<4, 4, KEEP>(a, t, smem); break;
    case 5: gated_dgrad_tile<1, 2, KEEP>(a, t, smem); break;
    case 6: gated_dgrad_tile<2, 2, KEEP>(a, t, smem); break;
    case 7: gated_dgrad_tile<3, 2, KEEP>(a, t, smem); break;
    case 8: gated_dgrad_tile<4, 2, KEEP>(a, t, smem); break;
  }
}

}  // namespace grp

int launch_grouped_gated_dgrad(const GatedDgradArgs& given, void* stream) {
  GatedDgradArgs a = given;
  const int64_t row_tiles = a.T / 256 + (a.E < a.T ? a.E : a.T) + 1;
  a.cols = a.T / 256 * ((a.N + 255) / 256) <= grp::NARROW_TILES ? 128 : 256;  // as launch_grouped_rows
  const int64_t tiles = row_tiles * ((a.N + a.cols - 1) / a.cols);
  auto kernel = a.keep.type == FORGE_KEEP_BF16  ? grp::gated_dgrad_kernel<FORGE_KEEP_BF16>
                : a.keep.type == FORGE_KEEP_FP8 ? grp::gated_dgrad_kernel<FORGE_KEEP_FP8>
                                                : grp::gated_dgrad_kernel<FORGE_KEEP_I8>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)tiles), dim3(grp::THREADS), 0, (hipStream_t)stream, a);
  return (int)hipGetLastError();
}

}  // namespace forge

// forge_block_gemm.hip -- Y_e = X_e W_e^T of e4m3 codes with one fp32 scale for each 1 x 128 of X and each
// 128 x 128 of W:  Y[t, n] = sum over b of sx[t, b] sw[n / 128, b] sum over k in block b of X[t, k] W[n, k].
//
// A block's sum is multiplied by its scales before the next is added, so the matrix cores cannot keep the
// whole contraction in their accumulators: each 16 x 16 block of the output takes one 16 x 16 x 128 product
// from zero (32 cycles) and 4 multiply-adds on the vector unit (16 cycles), which run beside the next
// block's products.  The vector unit cannot read the accumulation registers, so a wave keeps 128 x 64 of
// the output in 128 vector registers, and 8 waves (two a SIMD) a tile of 256 x 256.  (32 x 32 x 64 products,
// two from zero for each block, need 32 registers instead of 16 for results that wait.)
//
// A slab is one block of the contraction, 128 bytes of a row, copied to LDS by DMA in whole lines; LDS holds
// two.  The scales of 8 slabs are loaded 8 slabs ahead and pass through LDS, by slab and row.
//
// 16384 rows of 8 uneven experts by 14336 x 4096: 1038 us, 1.85 PFLOP/s.
#include <hip/hip_runtime.h>

#include "forge_ffn_internal.h"
#include "forge_grouped.h"

namespace forge {
namespace grp {

typedef int intx8 __attribute__((ext_vector_type(8)));

constexpr int BLOCK_THREADS = 512;
constexpr int PANEL_LDS = 32768, STAGE_LDS = 2 * PANEL_LDS;   // of 256 rows of 128 bytes; X and W
constexpr int CHUNK = 8;                                       // slabs whose scales are loaded at once
constexpr int SCALES_AT = 2 * STAGE_LDS, SCALES_LDS = (CHUNK * 256 + 2 * CHUNK) * 4;

__device__ __forceinline__ int block_swz(int row) { return (row >> 1) & 7; }

template <int HEIGHT, int WIDTH>  // of the tile, in 64s
__device__ __forceinline__ void block_tile(const BlockGemmArgs& a, const RowTile& t, unsigned char* smem) {
  constexpr int MB = 2 * HEIGHT, NB = WIDTH;   // blocks of 16 rows and columns of a wave (2 x 4 waves)
  constexpr int DX = HEIGHT, DW = WIDTH;       // copies of 1 KiB of a wave a slab
  const int lane = (int)threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int wr = wave >> 2, wc = wave & 3;
  const int64_t n0 = (int64_t)t.n * t.cols;
  const int KB = (int)(a.K / 128), slabs = t.e < a.E ? KB : 0;
  const uint32_t ld = (uint32_t)a.K;
  const u32x4 rx = make_rsrc(a.X + (int64_t)t.row0 * a.K, (uint32_t)t.rows * ld);
  const u32x4 rw = make_rsrc(a.W + ((int64_t)t.e * a.N + n0) * a.K, (uint32_t)(64 * WIDTH) * ld);
  const uint32_t lds = lds_address(smem);
  uint32_t ox[DX], ow[DW];  // this lane's pieces of the wave's copies
  auto piece_of = [&](int copy) {
    const int r = 8 * copy + (lane >> 3);
    return (uint32_t)r * ld + 16u * (uint32_t)((lane & 7) ^ block_swz(r));
  };
#pragma unroll
  for (int j = 0; j < DX; ++j) ox[j] = piece_of(DX * wave + j);
#pragma unroll
  for (int j = 0; j < DW; ++j) ow[j] = piece_of(DW * wave + j);
  auto copy = [&](int s) {
    const uint32_t at = lds + (uint32_t)((s & 1) * STAGE_LDS), k = (uint32_t)s * 128u;
    static_for<DX>([&](auto j) { copy_1k<j * 1024>(rx, ox[j] + k, at + (uint32_t)(wave * DX * 1024)); });
    static_for<DW>([&](auto j) { copy_1k<PANEL_LDS + j * 1024>(rw, ow[j] + k, at + (uint32_t)(wave * DW * 1024)); });
  };
  // Scales: two threads a row of X, four slabs each; 2 x 8 threads those of W.
  auto scales = [&](int chunk) { return reinterpret_cast<float*>(smem + SCALES_AT + (chunk & 1) * SCALES_LDS); };
  const int sr = (int)threadIdx.x >> 1, sh = ((int)threadIdx.x & 1) * (CHUNK / 2);
  float sx[CHUNK / 2], sw;
  auto fetch_scales = [&](int chunk) {
    const int s0 = chunk * CHUNK;
#pragma unroll
    for (int j = 0; j < CHUNK / 2; ++j) {
      const int s = s0 + sh + j;
      sx[j] = sr < t.rows && s < slabs ? a.x_scale[(int64_t)(t.row0 + sr) * KB + s] : 0.0f;
    }
    const int s = s0 + ((int)threadIdx.x & (CHUNK - 1)), b = WIDTH == 4 ? ((int)threadIdx.x / CHUNK) & 1 : 0;
    sw = s < slabs ? a.w_scale[((int64_t)t.e * (a.N / 128) + n0 / 128 + b) * KB + s] : 0.0f;
  };
  auto put_scales = [&](int chunk) {
    float* p = scales(chunk);
#pragma unroll
    for (int j = 0; j < CHUNK / 2; ++j) p[(sh + j) * 256 + sr] = sx[j];
    if (threadIdx.x < 2 * CHUNK) p[CHUNK * 256 + threadIdx.x] = sw;
  };

  floatx4 acc[MB][NB];
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = floatx4{};
  if (slabs > 0) {
    copy(0);
    fetch_scales(0);
    put_scales(0);
  }
  // addresses of a lane's two pieces: the row's swizzle is the same in every block of 16
  const int row = lane & 15, q = lane >> 4;
  const uint32_t piece0 = (uint32_t)(row * 128 + 16 * ((2 * q) ^ block_swz(row)));
  const uint32_t piece1 = (uint32_t)(row * 128 + 16 * ((2 * q + 1) ^ block_swz(row)));
  using P4 = __attribute__((address_space(3))) const u32x4*;
  auto frag = [&](uint32_t p0, uint32_t p1, int block) {
    const u32x4 lo = *(P4)(p0 + block * 2048), hi = *(P4)(p1 + block * 2048);
    return __builtin_bit_cast(intx8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  for (int s = 0; s < slabs; ++s) {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if (s + 1 < slabs) copy(s + 1);
    const int c = s & (CHUNK - 1);
    if (c == 0) fetch_scales(s / CHUNK + 1);
    const float* sc = scales(s / CHUNK);
    const uint32_t px = lds + (uint32_t)((s & 1) * STAGE_LDS + wr * MB * 2048);
    const uint32_t pw = lds + (uint32_t)((s & 1) * STAGE_LDS + PANEL_LDS + wc * NB * 2048);
    const uint32_t x0 = px + piece0, x1 = px + piece1, w0 = pw + piece0, w1 = pw + piece1;
    intx8 w[NB], x[2];
#pragma unroll
    for (int j = 0; j < NB; ++j) w[j] = frag(w0, w1, j);
    x[0] = frag(x0, x1, 0);
    const float w_scale = sc[CHUNK * 256 + (WIDTH == 4 ? (wc >> 1) * CHUNK : 0) + c];
    float scale[MB];
#pragma unroll
    for (int i = 0; i < MB; ++i) scale[i] = sc[c * 256 + wr * 16 * MB + 16 * i + row];
    __builtin_amdgcn_sched_barrier(0);
    floatx4 part[2][NB];
    auto add = [&](auto ic) {
      constexpr int i = decltype(ic)::value;
      const float f = scale[i] * w_scale;
#pragma unroll
      for (int j = 0; j < NB; ++j) {
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(part[i & 1][j][r], f, acc[i][j][r]);
        asm volatile("" : "+v"(acc[i][j]));  // here, not after all the products: their results would not fit
      }
    };
    static_for<MB>([&](auto ic) {
      constexpr int i = decltype(ic)::value;
      if constexpr (i + 1 < MB) x[(i + 1) & 1] = frag(x0, x1, i + 1);
#pragma unroll
      for (int j = 0; j < NB; ++j)
        part[i & 1][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w[j], x[i & 1], floatx4{}, 0, 0, 0, 0, 0, 0);
      if constexpr (i > 0) add(std::integral_constant<int, i - 1>{});
      __builtin_amdgcn_sched_barrier(0);
    });
    add(std::integral_constant<int, MB - 1>{});
    if (c == CHUNK - 1) put_scales(s / CHUNK + 1);
  }
  __syncthreads();
  // out by rows through LDS in bf16: 16-byte chunks are XOR-swizzled with the row
  constexpr int ROW = 128 * WIDTH, CH = ROW / 16;
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int r = wr * 16 * MB + 16 * i + row, c4 = wc * 4 * NB + 4 * j + q;  // column / 4
      *reinterpret_cast<u32x2*>(smem + r * ROW + 16 * ((c4 >> 1) ^ (r & 15)) + 8 * (c4 & 1)) =
          u32x2{pack_bf16(acc[i][j][0], acc[i][j][1]), pack_bf16(acc[i][j][2], acc[i][j][3])};
    }
  __syncthreads();
  for (int p = (int)threadIdx.x; p < t.rows * CH; p += BLOCK_THREADS) {
    const int r = p / CH, c = p % CH;
    st16_stream(a.Y + (int64_t)(t.row0 + r) * a.N + n0 + 8 * c, *reinterpret_cast<const u32x4*>(smem + r * ROW + 16 * (c ^ (r & 15))));
  }
}

__global__ __launch_bounds__(BLOCK_THREADS, 2) void block_gemm_kernel(BlockGemmArgs a) {
  __shared__ __attribute__((aligned(1024))) unsigned char smem[SCALES_AT + 2 * SCALES_LDS];
  RowTile t;
  if (!find_tile<256>(a.ends, a.E, a.T, a.N, a.cols, (int)blockIdx.x, t)) return;
  const bool narrow = t.cols < 256 || a.N - (int64_t)t.n * 256 < 256;
  switch ((t.rows + 63) / 64 + (narrow ? 4 : 0)) {
    case 1: block_tile<1, 4>(a, t, smem); break;
    case 2: block_tile<2, 4>(a, t, smem); break;
    case 3: block_tile<3, 4>(a, t, smem); break;
    case 4: block_tile<4, 4>(a, t, smem); break;
    case 5: block_tile<1, 2>(a, t, smem); break;
    case 6: block_tile<2, 2>(a, t, smem); break;
    case 7: block_tile<3, 2>(a, t, smem); break;
    case 8: block_tile<4, 2>(a, t, smem); break;
  }
}

}  // namespace grp

int launch_grouped_block_gemm(const BlockGemmArgs& given, void* stream) {
  if (few_rows_call(given.T, given.E, given.N, 128)) return launch_block_few(given, stream);
  BlockGemmArgs a = given;
  const int64_t row_tiles = a.T / 256 + (a.E < a.T ? a.E : a.T) + 1;
  a.cols = a.T / 256 * ((a.N + 255) / 256) <= grp::NARROW_TILES ? 128 : 256;  // as launch_grouped_rows
  const int64_t tiles = row_tiles * ((a.N + a.cols - 1) / a.cols);
  hipLaunchKernelGGL(grp::block_gemm_kernel, dim3((unsigned)tiles), dim3(grp::BLOCK_THREADS), 0, (hipStream_t)stream, a);
  return (int)hipGetLastError();
}

}  // namespace forge

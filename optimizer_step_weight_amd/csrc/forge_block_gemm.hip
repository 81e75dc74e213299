// forge_block_gemm.hip -- Y_e = X_e W_e^T of e4m3 codes with one fp32 scale for each 1 x 128 of X and each
// 128 x 128 of W:  Y[t, n] = sum over b of sx[t, b] sw[n / 128, b] sum over k in block b of X[t, k] W[n, k].
//
// A block's sum is multiplied by its scales before the next is added, so the matrix cores cannot keep the
// whole contraction in their accumulators: each 32 x 32 block of the output takes two 32 x 32 x 64 products
// from zero (128 of the contraction, 128 cycles) and 16 multiply-adds on the vector unit (64 cycles), which
// run beside the next block's products.  The vector unit cannot read the accumulation registers, so a wave
// keeps 128 x 64 of the output in 128 vector registers, and 8 waves (two a SIMD) a tile of 256 x 256.
//
// A slab is one block of the contraction, 128 bytes of a row, copied to LDS by DMA in whole lines; LDS holds
// two.  The scales of 8 slabs are loaded 8 slabs ahead and pass through LDS, by slab and row.
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

template <int MB, int NB>  // blocks of 32 rows and columns of a wave: a tile of 64 MB rows and 128 NB columns
__device__ __forceinline__ void block_tile(const BlockGemmArgs& a, const RowTile& t, unsigned char* smem) {
  const int lane = (int)threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int wr = wave >> 2, wc = wave & 3;
  const int64_t n0 = (int64_t)t.n * t.cols;
  const int KB = (int)(a.K / 128), slabs = t.e < a.E ? KB : 0;
  const uint32_t ld = (uint32_t)a.K;
  const u32x4 rx = make_rsrc(a.X + (int64_t)t.row0 * a.K, (uint32_t)t.rows * ld);
  const u32x4 rw = make_rsrc(a.W + ((int64_t)t.e * a.N + n0) * a.K, (uint32_t)(128 * NB) * ld);
  const uint32_t lds = lds_address(smem);
  uint32_t ox[MB], ow[2 * NB];  // this lane's pieces of the wave's copies
#pragma unroll
  for (int j = 0; j < MB; ++j) {
    const int r = 8 * (MB * wave + j) + (lane >> 3);
    ox[j] = (uint32_t)r * ld + 16u * (uint32_t)((lane & 7) ^ block_swz(r));
  }
#pragma unroll
  for (int j = 0; j < 2 * NB; ++j) {
    const int r = 8 * (2 * NB * wave + j) + (lane >> 3);
    ow[j] = (uint32_t)r * ld + 16u * (uint32_t)((lane & 7) ^ block_swz(r));
  }
  auto copy = [&](int s) {
    const uint32_t at = lds + (uint32_t)((s & 1) * STAGE_LDS), k = (uint32_t)s * 128u;
    static_for<MB>([&](auto j) { copy_1k<j * 1024>(rx, ox[j] + k, at + (uint32_t)(wave * MB * 1024)); });
    static_for<2 * NB>([&](auto j) { copy_1k<PANEL_LDS + j * 1024>(rw, ow[j] + k, at + (uint32_t)(wave * 2 * NB * 1024)); });
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
    const int s = s0 + ((int)threadIdx.x & (CHUNK - 1)), b = ((int)threadIdx.x / CHUNK) & (NB - 1);
    sw = s < slabs ? a.w_scale[((int64_t)t.e * (a.N / 128) + n0 / 128 + b) * KB + s] : 0.0f;
  };
  auto put_scales = [&](int chunk) {
    float* p = scales(chunk);
#pragma unroll
    for (int j = 0; j < CHUNK / 2; ++j) p[(sh + j) * 256 + sr] = sx[j];
    if (threadIdx.x < 2 * CHUNK) p[CHUNK * 256 + threadIdx.x] = sw;
  };

  floatx16 acc[MB][NB];
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = floatx16{};
  if (slabs > 0) {
    copy(0);
    fetch_scales(0);
    put_scales(0);
  }
  // addresses of a row's pieces: the row's swizzle is the same in every block of 32
  const int row = lane & 31, q = 2 * (lane >> 5);
  uint32_t piece[4];
#pragma unroll
  for (int x = 0; x < 4; ++x) piece[x] = (uint32_t)(row * 128 + 16 * ((4 * (x >> 1) + q + (x & 1)) ^ block_swz(row)));
  using P4 = __attribute__((address_space(3))) const u32x4*;
  auto frag = [&](uint32_t panel, int half) {
    const u32x4 lo = *(P4)(panel + piece[2 * half]), hi = *(P4)(panel + piece[2 * half + 1]);
    return __builtin_bit_cast(intx8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  auto product = [&](const intx8& w, const intx8& x, const floatx16& c) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, x, c, 0, 0, 0, 0, 0, 0);
  };
  for (int s = 0; s < slabs; ++s) {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if (s + 1 < slabs) copy(s + 1);
    const int c = s & (CHUNK - 1);
    if (c == 0) fetch_scales(s / CHUNK + 1);
    const float* sc = scales(s / CHUNK);
    const float w_scale = sc[CHUNK * 256 + (NB == 2 ? (wc >> 1) * CHUNK : 0) + c];
    const uint32_t px = lds + (uint32_t)((s & 1) * STAGE_LDS + wr * MB * 4096);
    const uint32_t pw = lds + (uint32_t)((s & 1) * STAGE_LDS + PANEL_LDS + wc * NB * 4096);
    intx8 w[NB][2];
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      w[j][0] = frag(pw + j * 4096, 0);
      w[j][1] = frag(pw + j * 4096, 1);
    }
    floatx16 part[2];
    float scale[MB];
#pragma unroll
    for (int i = 0; i < MB; ++i) scale[i] = sc[c * 256 + wr * 32 * MB + 32 * i + row] * w_scale;
    auto add = [&](auto bc) {
      constexpr int b = decltype(bc)::value, i = b / NB, j = b % NB;
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = __builtin_fmaf(part[b & 1][r], scale[i], acc[i][j][r]);
    };
    static_for<MB>([&](auto ic) {
      constexpr int i = decltype(ic)::value;
      const intx8 x0 = frag(px + i * 4096, 0), x1 = frag(px + i * 4096, 1);
      static_for<NB>([&](auto jc) {
        constexpr int j = decltype(jc)::value, b = i * NB + j;
        part[b & 1] = product(w[j][0], x0, floatx16{});
        part[b & 1] = product(w[j][1], x1, part[b & 1]);
        if constexpr (b > 0) add(std::integral_constant<int, b - 1>{});
        __builtin_amdgcn_sched_barrier(0);
      });
    });
    add(std::integral_constant<int, MB * NB - 1>{});
    if (c == CHUNK - 1) put_scales(s / CHUNK + 1);
  }
  __syncthreads();
  // out by rows through LDS in bf16: 16-byte chunks are XOR-swizzled with the row
  constexpr int ROW = 256 * NB, CH = ROW / 16;
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int r = wr * 32 * MB + 32 * i + row, c4 = wc * 8 * NB + 8 * j + 2 * g + (lane >> 5);  // column / 4
        *reinterpret_cast<u32x2*>(smem + r * ROW + 16 * ((c4 >> 1) ^ (r & 15)) + 8 * (c4 & 1)) =
            u32x2{pack_bf16(acc[i][j][4 * g], acc[i][j][4 * g + 1]), pack_bf16(acc[i][j][4 * g + 2], acc[i][j][4 * g + 3])};
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
    case 1: block_tile<1, 2>(a, t, smem); break;
    case 2: block_tile<2, 2>(a, t, smem); break;
    case 3: block_tile<3, 2>(a, t, smem); break;
    case 4: block_tile<4, 2>(a, t, smem); break;
    case 5: block_tile<1, 1>(a, t, smem); break;
    case 6: block_tile<2, 1>(a, t, smem); break;
    case 7: block_tile<3, 1>(a, t, smem); break;
    case 8: block_tile<4, 1>(a, t, smem); break;
  }
}

}  // namespace grp

int launch_grouped_block_gemm(const BlockGemmArgs& given, void* stream) {
  BlockGemmArgs a = given;
  const int64_t row_tiles = a.T / 256 + (a.E < a.T ? a.E : a.T) + 1;
  a.cols = a.T / 256 * ((a.N + 255) / 256) <= grp::NARROW_TILES ? 128 : 256;  // as launch_grouped_rows
  const int64_t tiles = row_tiles * ((a.N + a.cols - 1) / a.cols);
  hipLaunchKernelGGL(grp::block_gemm_kernel, dim3((unsigned)tiles), dim3(grp::BLOCK_THREADS), 0, (hipStream_t)stream, a);
  return (int)hipGetLastError();
}

}  // namespace forge

// forge_block_gemm.hip -- Y_e = X_e W_e^T of e4m3 codes with one fp32 scale for each 1 x 128 of X and each
// 128 x 128 of W:  Y[t, n] = sum over b of sx[t, b] sw[n / 128, b] sum over k in block b of X[t, k] W[n, k].
//
// A block's sum is multiplied by its scales before the next is added, so the matrix cores cannot keep the
// whole contraction in their accumulators: each 16 x 16 block of the output takes one 16 x 16 x 128 product
// from zero (32 cycles) and 4 multiply-adds on the vector unit (16 cycles), which run beside the next
// block's products.  The vector unit cannot read the accumulation registers, so a wave keeps 112 x 64 of
// the output in 112 vector registers, and 8 waves (two a SIMD) a tile of 224 x 256.  (32 x 32 x 64 products,
// two from zero for each block, need 64 registers instead of 16 for results that wait.)
//
// A slab is one block of the contraction, 128 bytes of a row, copied to LDS by DMA in whole lines.  LDS holds three
// slabs of X and two of W, whose fragments a wave reads half a slab ahead: with one barrier a slab, all of
// a slab's copies have most of a slab's time to land, and they go out at an even pace.  224 rows a tile leave room for
// the scales: those of 4 slabs are copied 4 slabs ahead, by row, where they lie on 16 bytes, else by slab.
//
// 16384 rows of 8 uneven experts by 14336 x 4096: 979-1032 us over the cards seen, 1.86-1.97 PFLOP/s (row scales,
// forge_grouped.h: 845-860); in even groups 832-847 us, 2.25 PFLOP/s.  A longer contraction adds 2.4 PFLOP/s.  What bounds
// it is LDS: fragments and copies together move 240 KiB a slab, 1900 cycles at 128 bytes each beside the
// products' 1792.  Without the copies' data the same loop takes 645 us, without those of X 765, with all of them
// hits in L2 790.  4 waves of 96 x 128 read less from LDS, but a wave alone on its SIMD then issues everything: 872 us.
// Copies in bursts 888 us; one slab of each ahead and W's fragments read when they are used 930.
#include <hip/hip_runtime.h>

#include "forge_ffn_internal.h"
#include "forge_grouped.h"

namespace forge {
namespace grp {

typedef int intx8 __attribute__((ext_vector_type(8)));

constexpr int BLOCK_THREADS = 512, BLOCK_ROWS = 224;           // of a whole tile
// LDS: three slabs of X, two of W, the scales of two chunks of 4 slabs of X and of one of 64 of W, and a place
// for copies of nothing.
constexpr int X_SLAB = BLOCK_ROWS * 128, W_SLAB = 256 * 128;
constexpr int W_AT = 3 * X_SLAB, XS_AT = W_AT + 2 * W_SLAB, XS_CHUNK = 4096, WS_AT = XS_AT + 2 * XS_CHUNK;
constexpr int WS_SLABS = 64, DUMP_AT = WS_AT + 2 * WS_SLABS * 4, BLOCK_LDS = DUMP_AT + 1024;
static_assert(BLOCK_LDS <= 5 * 32768, "LDS");

__device__ __forceinline__ int block_swz(int row) { return (row >> 1) & 7; }

// FOURS: four scales of a row of X lie on 16 bytes, and are copied at once.
template <int HEIGHT, int WIDTH, bool FOURS>  // of the tile, in 64s (4 rows: 224)
__device__ __forceinline__ void block_tile(const BlockGemmArgs& a, const RowTile& t, unsigned char* smem) {
  constexpr int MB = HEIGHT == 4 ? 7 : 2 * HEIGHT, NB = WIDTH;  // blocks of 16 rows and columns of a wave (2 x 4 waves)
  constexpr int DX = HEIGHT, DW = WIDTH;                        // copies of 1 KiB of a wave a slab
  const int lane = (int)threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int wr = wave >> 2, wc = wave & 3;
  const int64_t n0 = (int64_t)t.n * t.cols;
  const int KB = (int)(a.K / 128), slabs = t.e < a.E ? KB : 0;
  const uint32_t ld = (uint32_t)a.K, lds = lds_address(smem);
  const u32x4 rx = make_rsrc(a.X + (int64_t)t.row0 * a.K, (uint32_t)t.rows * ld);
  const u32x4 rw = make_rsrc(a.W + ((int64_t)t.e * a.N + n0) * a.K, (uint32_t)(64 * WIDTH) * ld);
  const u32x4 rs = make_rsrc(a.x_scale + (int64_t)t.row0 * KB, (uint32_t)(t.rows * KB * 4));
  uint32_t ox[DX], ow[DW];  // this lane's pieces of the wave's copies
  auto piece_of = [&](int copy) {
    const int r = 8 * copy + (lane >> 3);
    return (uint32_t)r * ld + 16u * (uint32_t)((lane & 7) ^ block_swz(r));
  };
#pragma unroll
  for (int j = 0; j < DX; ++j) ox[j] = piece_of(DX * wave + j);
#pragma unroll
  for (int j = 0; j < DW; ++j) ow[j] = piece_of(DW * wave + j);
  // wave 7 of a whole tile has no rows of X: its copies are of rows behind the tile's, to a place that nobody reads
  const bool idle = HEIGHT == 4 && wave == 7;
  // Copy j of slab s; of slabs behind the last, nothing (past the operand's end: zeros, which nobody reads).
  auto copy_x = [&](auto j, uint32_t k, uint32_t slot) {
    copy_1k<j * 1024>(rx, ox[j] + k, idle ? lds + DUMP_AT - j * 1024 : lds + slot + (uint32_t)(wave * DX * 1024));
  };
  auto copy_w = [&](auto j, uint32_t k, int s) {
    copy_1k<j * 1024>(rw, ow[j] + k, lds + (uint32_t)(W_AT + (s & 1) * W_SLAB + wave * DW * 1024));
  };
  auto place = [&](int s) { return s < slabs ? (uint32_t)s * 128u : 0x80000000u; };
  const uint32_t skip = idle ? 0x80000000u : 0u;
  // Scales of X of slabs 4 c .. 4 c + 3, to [row][slab] (FOURS) or [slab][row].
  auto copy_scales = [&](int c) {
    const uint32_t at = lds + (uint32_t)(XS_AT + (c & 1) * XS_CHUNK);
    if constexpr (FOURS) {
      const int r = 64 * wave + lane;  // rows from 256 on: behind the tile
      copy_1k<0>(rs, (uint32_t)(r * KB + 4 * c) * 4u, wave < 4 ? at + (uint32_t)(wave * 1024) : lds + DUMP_AT);
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int g = 2 * wave + i, s = 4 * c + (g >> 2), r = 64 * (g & 3) + lane;
        const uint32_t o = s < KB ? (uint32_t)(r * KB + s) * 4u : 0xFFFFFFF0u;
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(at + (uint32_t)(g * 256)), "v"(o), "s"(rs)
                     : "memory", "m0");
      }
    }
  };
  const int row = lane & 15, q = lane >> 4;
  const float* xs = reinterpret_cast<const float*>(smem + XS_AT) + (wr * 16 * MB + row) * (FOURS ? 4 : 1);
  float* ws = reinterpret_cast<float*>(smem + WS_AT);
  // Scales of W of slabs s0 .. s0 + 63.
  auto fetch_w_scales = [&](int s0) {
    const int b = (int)threadIdx.x / WS_SLABS, s = s0 + (int)threadIdx.x % WS_SLABS;
    if (b < WIDTH / 2) ws[threadIdx.x] = s < KB ? a.w_scale[((int64_t)t.e * (a.N / 128) + n0 / 128 + b) * KB + s] : 0.0f;
  };

  floatx4 acc[MB][NB];
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = floatx4{};
  // addresses of a lane's two pieces: the row's swizzle is the same in every block of 16
  const uint32_t piece0 = (uint32_t)(row * 128 + 16 * ((2 * q) ^ block_swz(row)));
  const uint32_t piece1 = (uint32_t)(row * 128 + 16 * ((2 * q + 1) ^ block_swz(row)));
  using P4 = __attribute__((address_space(3))) const u32x4*;
  struct Frag {
    u32x4 lo, hi;
    __device__ __forceinline__ intx8 whole() const { return __builtin_bit_cast(intx8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7)); }
  };
  const uint32_t x_at = lds + (uint32_t)(wr * MB * 2048), w_at = lds + (uint32_t)(W_AT + wc * NB * 2048);
  auto read = [&](Frag& f, uint32_t panel, int block, int half) {
    if (half == 0) f.lo = *(P4)(panel + piece0 + block * 2048);
    else f.hi = *(P4)(panel + piece1 + block * 2048);
  };
  // A product's result is added N_LATE products later, the last ones' in the next slab.
  constexpr int BLOCKS = MB * NB, N_LATE = NB == 4 ? 3 : 1;
  floatx4 part[N_LATE + 1];
#pragma unroll
  for (int i = 0; i <= N_LATE; ++i) part[i] = floatx4{};
  float factor[2] = {0.0f, 0.0f};  // of the present and the last block of rows
  Frag x[2];
  uint32_t slot = 0;  // of slab s in the ring of X
  // Slab s, whose W is in w; then that of slab s + 1 is in next, and its first rows of X are read.
  // MID products in, slab s + 1 has landed for all waves (barrier), none of which needs slab s - 1 or W in LDS any
  // more: slab s + 2 is copied there, and W of slab s + 1 read.
  auto step = [&](auto pc, Frag (&w)[NB], Frag (&next)[NB], int s) {
    constexpr int P = decltype(pc)::value;  // the first rows of X are in x[P]
    constexpr int MID = 2 * NB < BLOCKS - 4 ? 2 * NB : BLOCKS / 2;
    const float w_scale = ws[(WIDTH == 4 ? (wc >> 1) * WS_SLABS : 0) + s % WS_SLABS];
    const float* sc = xs + ((s >> 2) & 1) * (XS_CHUNK / 4) + (s & 3) * (FOURS ? 1 : 256);
    const uint32_t px = x_at + slot, after = slot == 2 * X_SLAB ? 0 : slot + X_SLAB;
    const uint32_t px1 = x_at + after, pw1 = w_at + (uint32_t)(((s + 1) & 1) * W_SLAB);
    const uint32_t k2 = place(s + 2), slot2 = slot == 0 ? 2 * X_SLAB : slot - X_SLAB;
    float scale = sc[0];
    static_for<BLOCKS>([&](auto nc) {
      constexpr int n = decltype(nc)::value, i = n / NB, j = n % NB;
      if constexpr (n == MID) {
        wait_vm<0>();
        barrier();
        if ((s & 3) == 0 && s + 4 < slabs) copy_scales(s / 4 + 1);
        if ((s + 1) % WS_SLABS == 0) {
          fetch_w_scales(s + 1);
          asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        }
      }
      // slab s + 2, at an even pace: in a burst the waves wait for each other to issue their copies
      if constexpr (n >= MID) {
        constexpr int c0 = (DX + DW) * (n - MID) / (BLOCKS - MID), c1 = (DX + DW) * (n + 1 - MID) / (BLOCKS - MID);
        static_for<c1 - c0>([&](auto k) {
          constexpr int c = c0 + decltype(k)::value;
          if constexpr (c < DX) copy_x(std::integral_constant<int, c>{}, k2 | skip, slot2);
          else copy_w(std::integral_constant<int, c - DX>{}, k2, s);
        });
      }
      // the next rows of X, two pieces a block of rows
      if constexpr (j < 2) read(x[(i + 1 + P) & 1], i + 1 < MB ? px : px1, (i + 1) % MB, j);
      // pieces of W of the next slab, evenly over what is left
      constexpr int FROM = MID, LEFT = BLOCKS - FROM;
      constexpr int p0 = n < FROM ? 0 : 2 * NB * (n - FROM) / LEFT, p1 = n < FROM ? 0 : 2 * NB * (n + 1 - FROM) / LEFT;
      static_for<p1 - p0>([&](auto k) { read(next[(p0 + decltype(k)::value) / 2], pw1, (p0 + decltype(k)::value) / 2, (p0 + decltype(k)::value) % 2); });
      if constexpr (j == 0) {
        factor[1] = factor[0];
        factor[0] = scale * w_scale;
        if constexpr (i + 1 < MB) scale = sc[16 * (i + 1) * (FOURS ? 4 : 1)];
      }
      part[n % (N_LATE + 1)] =
          __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w[j].whole(), x[(i + P) & 1].whole(), floatx4{}, 0, 0, 0, 0, 0, 0);
      constexpr int m = (n - N_LATE + BLOCKS) % BLOCKS;  // the block whose result is added
#pragma unroll
      for (int r = 0; r < 4; ++r)
        acc[m / NB][m % NB][r] = __builtin_fmaf(part[(n + 1) % (N_LATE + 1)][r], factor[j < N_LATE ? 1 : 0], acc[m / NB][m % NB][r]);
      asm volatile("" : "+v"(acc[m / NB][m % NB]));  // here, not after all the products
      __builtin_amdgcn_sched_barrier(0);
    });
    slot = after;
  };
  if (slabs > 0) {
    fetch_w_scales(0);
    copy_scales(0);
    static_for<2>([&](auto sc) {
      constexpr int s = decltype(sc)::value;
      static_for<DX>([&](auto j) { copy_x(j, place(s) | skip, s * X_SLAB); });
      static_for<DW>([&](auto j) { copy_w(j, place(s), s); });
    });
    wait_vm<DX + DW>();
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    Frag wa[NB], wb[NB];
#pragma unroll
    for (int j = 0; j < 2 * NB; ++j) read(wa[j / 2], w_at, j / 2, j % 2);
    read(x[0], x_at, 0, 0);
    read(x[0], x_at, 0, 1);
    for (int s = 0; s < slabs; s += 2) {
      step(std::integral_constant<int, 0>{}, wa, wb, s);
      if (s + 1 < slabs) step(std::integral_constant<int, MB & 1>{}, wb, wa, s + 1);
    }
    wait_vm<0>();  // no copy may land in what LDS takes next
    // the last products' results
#pragma unroll
    for (int k = 0; k < N_LATE; ++k) {
      constexpr int at = BLOCKS - N_LATE;
      const int m = at + k;
#pragma unroll
      for (int r = 0; r < 4; ++r)
        acc[m / NB][m % NB][r] = __builtin_fmaf(part[m % (N_LATE + 1)][r], factor[0], acc[m / NB][m % NB][r]);
    }
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

template <bool FOURS>
__global__ __launch_bounds__(BLOCK_THREADS, 2) void block_gemm_kernel(BlockGemmArgs a) {
  __shared__ __attribute__((aligned(1024))) unsigned char smem[BLOCK_LDS];
  RowTile t;
  if (!find_tile<BLOCK_ROWS>(a.ends, a.E, a.T, a.N, a.cols, (int)blockIdx.x, t)) return;
  const bool narrow = t.cols < 256 || a.N - (int64_t)t.n * 256 < 256;
  switch ((t.rows + 63) / 64 + (narrow ? 4 : 0)) {
    case 1: block_tile<1, 4, FOURS>(a, t, smem); break;
    case 2: block_tile<2, 4, FOURS>(a, t, smem); break;
    case 3: block_tile<3, 4, FOURS>(a, t, smem); break;
    case 4: block_tile<4, 4, FOURS>(a, t, smem); break;
    case 5: block_tile<1, 2, FOURS>(a, t, smem); break;
    case 6: block_tile<2, 2, FOURS>(a, t, smem); break;
    case 7: block_tile<3, 2, FOURS>(a, t, smem); break;
    case 8: block_tile<4, 2, FOURS>(a, t, smem); break;
  }
}

}  // namespace grp

int launch_grouped_block_gemm(const BlockGemmArgs& given, void* stream) {
  if (few_rows_call(given.T, given.E, given.N, 128, kFewBlock)) return launch_block_few(given, stream);
  BlockGemmArgs a = given;
  const int64_t row_tiles = a.T / grp::BLOCK_ROWS + (a.E < a.T ? a.E : a.T) + 1;
  a.cols = a.T / grp::BLOCK_ROWS * ((a.N + 255) / 256) <= grp::NARROW_TILES ? 128 : 256;  // as launch_grouped_rows
  const int64_t tiles = row_tiles * ((a.N + a.cols - 1) / a.cols);
  // four scales of X on 16 bytes: a row's begin there too, and so does the tensor
  const bool fours = a.K % 512 == 0 && (reinterpret_cast<uintptr_t>(a.x_scale) & 15) == 0;
  hipLaunchKernelGGL((fours ? grp::block_gemm_kernel<true> : grp::block_gemm_kernel<false>), dim3((unsigned)tiles),
                     dim3(grp::BLOCK_THREADS), 0, (hipStream_t)stream, a);
  return (int)hipGetLastError();
}

}  // namespace forge

// forge_grouped.h -- tiles of the matrix products grouped by expert: the lookup of a workgroup's
// expert and rows in the groups' ends, and the row products Y_e = X_e W_e^T and dX_e = dY_e W_e.
//
// Rows are sorted by expert and the groups' ends live on the device, so the host cannot know how
// many row tiles there are: at most T / BM + E + 1 (each group adds at most one partial tile, and
// so do the rows of no group).  The grid covers that bound; every wave scans the ends and finds
// the tile of its workgroup, and workgroups past the last tile end.  Tiles are ordered by
// expert, within an expert in blocks of 8 row tiles over all column tiles, and given to the 8
// XCDs in contiguous runs: an XCD's resident tiles share their weight and row panels in its L2.
#pragma once

#include "forge_layer_internal.h"
#include "forge_mainloop2.h"

namespace forge {
namespace grp {

using ml2::barrier;
using ml2::dma16;
using ml2::floatx4;
using ml2::make_rsrc;
using ml2::wait_vm;
typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef int intx8 __attribute__((ext_vector_type(8)));

// Position of workgroup b in an order of `total` tiles in which each XCD (b mod 8) has a
// contiguous run.
__device__ __forceinline__ int xcd_run(int b, int total) {
  const int per = total >> 3, rem = total & 7, x = b & 7, loc = b >> 3;
  return (x < rem ? x * (per + 1) : rem * (per + 1) + (x - rem) * per) + loc;
}

// The groups' ends, 64 at a time: lane l of the wave holds group 64 c + l.  Ends are clamped to
// [0, T] and made ascending (a running maximum), so whatever the device holds, the groups cover
// disjoint ranges of rows in bounds.  Group E holds the rows after the last end.
struct Chunk {
  int64_t start, end;  // this lane's group (empty past group E)
};
__device__ __forceinline__ Chunk load_chunk(const int32_t* ends, int E, int64_t T, int c, int64_t carry) {
  const int lane = (int)(threadIdx.x & 63), e = 64 * c + lane;
  int64_t v = e < E ? (int64_t)ends[e] : (e == E ? T : 0);
  v = v < 0 ? 0 : (v > T ? T : v);
  if (lane == 0 && v < carry) v = carry;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int up = __shfl_up((int)v, o);
    if (lane >= o && up > v) v = up;
  }
  const int prev = __shfl_up((int)v, 1);
  Chunk k;
  k.end = v;
  k.start = lane == 0 ? carry : prev;
  return k;
}

// Rows [start, start + len) of group e (e < E), by the same rule.
__device__ __forceinline__ void group_rows(const int32_t* ends, int E, int64_t T, int e, int& start, int& len) {
  int64_t carry = 0;
  Chunk k{};
  for (int c = 0; c <= e / 64; ++c) {
    k = load_chunk(ends, E, T, c, carry);
    carry = __builtin_amdgcn_readlane((int)k.end, 63);
  }
  start = __builtin_amdgcn_readlane((int)k.start, e & 63);
  len = __builtin_amdgcn_readlane((int)k.end, e & 63) - start;
}

struct RowTile {
  int e;          // expert, or E for rows of no group
  int row0;       // first row
  int rows;       // rows of this tile, 1 .. BM
  int n;          // column tile
};

// The tile of workgroup b among the row tiles of BM rows x nbn column tiles; false: none left.
template <int BM>
__device__ __forceinline__ bool find_tile(const int32_t* ends, int E, int64_t T, int nbn, int b, RowTile& out) {
  const int lane = (int)(threadIdx.x & 63), chunks = E / 64 + 1;
  auto tiles_of = [&](const Chunk& k) { return (int)((k.end - k.start + BM - 1) / BM); };
  auto scan = [&](int v) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int up = __shfl_up(v, o);
      if (lane >= o) v += up;
    }
    return v;
  };
  int64_t carry = 0;
  int total = 0;  // the host keeps the grid, and with it every tile number, below 2^31
  Chunk k{};
  int incl = 0;
  for (int c = 0; c < chunks; ++c) {
    k = load_chunk(ends, E, T, c, carry);
    incl = scan(tiles_of(k));
    total += __builtin_amdgcn_readlane(incl, 63);
    carry = __builtin_amdgcn_readlane((int)k.end, 63);
  }
  total *= nbn;
  if (b >= total) return false;
  const int t = xcd_run(b, total);
  int before = 0;  // tiles of earlier chunks
  carry = 0;
  for (int c = 0; c < chunks; ++c) {
    if (chunks > 1) {
      k = load_chunk(ends, E, T, c, carry);
      incl = scan(tiles_of(k));
      carry = __builtin_amdgcn_readlane((int)k.end, 63);
    }
    const uint64_t past = __ballot((before + incl) * nbn > t);
    if (past == 0) {
      before += __builtin_amdgcn_readlane(incl, 63);
      continue;
    }
    const int l = __builtin_ctzll(past);
    const int cnt = __shfl(tiles_of(k), l), last = __shfl(incl, l);
    const int start = __shfl((int)k.start, l), end = __shfl((int)k.end, l);
    const int local = t - (before + last - cnt) * nbn;
    // blocks of G row tiles, row tiles fastest
    constexpr int G = 8;
    const int gid = local / (G * nbn), first = gid * G, gsz = cnt - first < G ? cnt - first : G;
    const int r = local - gid * G * nbn;
    const int row0 = start + (first + r % gsz) * BM;
    // the same in every lane; readfirstlane tells the compiler
    out.n = __builtin_amdgcn_readfirstlane(r / gsz);
    out.e = __builtin_amdgcn_readfirstlane(64 * c + l);
    out.row0 = __builtin_amdgcn_readfirstlane(row0);
    out.rows = __builtin_amdgcn_readfirstlane(end - row0 < BM ? end - row0 : BM);
    return true;
  }
  return false;
}

// ------------------------------------------------------------------ row products
// A BM x 256 tile of the output by one workgroup of 8 waves (2 of rows x 4 of 64 columns), the
// contraction in slabs of 64 bytes (32 bf16 or 64 fp8 elements) held in 4 stages of LDS, three
// in flight by LDS DMA while one is multiplied (the data path of forge_mainloop2.h):
//  * A: BM rows of 64 bytes, read as 16-byte pieces (dY of the dgrad tiles); rows past the
//    tile's last and contractions past the operand read as zero (buffer range check);
//  * NT: W's rows n0 .. n0 + 255 the same way.  With both operands contraction-contiguous a
//    lane's 8 (fp8: 32) contraction elements are consecutive;
//  * NN: 32 rows of W of 512 bytes (256 columns), read by LDS transpose reads.
// 16-byte chunks of the 64-byte rows are XOR-swizzled with (row / 4) mod 4: a group of 16 lanes
// reads 16 rows in 16 distinct bank windows.
template <int BM_, int MODE_>
struct RowsPipe {
  static constexpr int BM = BM_, MODE = MODE_, BN = 256, STAGES = 4, ROW = 64;
  static constexpr int MB = BM / 32;                      // 16-row blocks of a wave
  static constexpr int PANEL_A = BM * ROW, PANEL_B = 16384;
  static constexpr int STAGE = PANEL_A + PANEL_B, SMEM = STAGES * STAGE;
  static constexpr int DMA_A = BM >= 128 ? BM / 128 : 1, DMA = DMA_A + 2;  // 1 KiB copies per wave per slab
  static constexpr int ESZ = MODE == FORGE_GROUPED_NT8 ? 1 : 2;
  static_assert(BM == 64 || BM == 128 || BM == 256, "tile height");
};

struct RowsFeed {
  u32x4 rA, rB;
  uint32_t offA[2], offB[2];
  uint32_t stepB;
};

__device__ __forceinline__ int swz_d(int row) { return (row >> 2) & 3; }

template <class P>
__device__ __forceinline__ void make_feed(RowsFeed& f, const GroupedArgs& a, const RowTile& t) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t C = P::MODE == FORGE_GROUPED_NN ? a.N : a.K;  // contraction length
  const int64_t crow = C * P::ESZ;
  f.rA = make_rsrc(static_cast<const unsigned char*>(a.A) + (int64_t)t.row0 * crow, (uint32_t)(t.rows * crow));
#pragma unroll
  for (int j = 0; j < P::DMA_A; ++j) {
    // BM = 64 has 4 copies for 8 waves: waves 4-7 repeat those of waves 0-3 (the same bytes)
    const int d = P::BM == 64 ? (wave & 3) : P::DMA_A * wave + j;
    const int r = 16 * d + (lane >> 2), p = lane & 3;
    f.offA[j] = (uint32_t)(r * crow + 16 * (p ^ swz_d(r)));
  }
  const unsigned char* W = static_cast<const unsigned char*>(a.W) + (int64_t)t.e * a.N * a.K * P::ESZ;
  if constexpr (P::MODE == FORGE_GROUPED_NN) {
    const int64_t k0 = (int64_t)t.n * P::BN;
    f.rB = make_rsrc(W + k0 * 2, (uint32_t)(a.N * a.K * 2 - k0 * 2));
    f.stepB = (uint32_t)(32 * a.K * 2);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int r = 2 * (2 * wave + j) + (lane >> 5), p = lane & 31;
      f.offB[j] = (uint32_t)(r * a.K * 2 + 16 * (p ^ ml2::swz(r)));
    }
  } else {
    const int64_t n0 = (int64_t)t.n * P::BN, left = a.N - n0;
    f.rB = make_rsrc(W + n0 * crow, (uint32_t)((left < P::BN ? left : P::BN) * crow));
    f.stepB = P::ROW;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int r = 16 * (2 * wave + j) + (lane >> 2), p = lane & 3;
      f.offB[j] = (uint32_t)(r * crow + 16 * (p ^ swz_d(r)));
    }
  }
}

template <class P>
__device__ __forceinline__ void issue(const RowsFeed& f, unsigned char* stage, int slab) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t sa = (uint32_t)slab * P::ROW, sb = (uint32_t)slab * f.stepB;
#pragma unroll
  for (int j = 0; j < P::DMA_A; ++j) {
    const int d = P::BM == 64 ? (wave & 3) : P::DMA_A * wave + j;
    dma16(f.rA, f.offA[j] + sa, stage + d * 1024);
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) dma16(f.rB, f.offB[j] + sb, stage + P::PANEL_A + (2 * wave + j) * 1024);
}

// 16 bytes at chunk c of row r of a 64-byte-row panel.
__device__ __forceinline__ u32x4 piece(const unsigned char* panel, int r, int c) {
  return *reinterpret_cast<const u32x4*>(panel + r * 64 + 16 * (c ^ swz_d(r)));
}

template <class P>
struct Acc {
  floatx4 v[P::MB][4];
};
template <int BM>
struct Acc<RowsPipe<BM, FORGE_GROUPED_NT8>> {
  floatx16 v[BM / 64][2];
};

// One slab: wave (wm, wn) multiplies rows wm BM / 2 .. and columns 64 wn ...
template <class P>
__device__ __forceinline__ void mma(Acc<P>& acc, const unsigned char* stage, int wm, int wn) {
  const int lane = threadIdx.x & 63;
  const unsigned char* pa = stage;
  const unsigned char* pb = stage + P::PANEL_A;
  if constexpr (P::MODE == FORGE_GROUPED_NT8) {
    // 32 x 32 x 64: lane l holds the 32 codes 32 (l / 32) .. of row l mod 32
    const int i = lane & 31, h = 2 * (lane >> 5);
    auto frag8 = [&](const unsigned char* p, int row) {
      const u32x4 lo = piece(p, row, h), hi = piece(p, row, h + 1);
      intx8 x;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[j] = (int)lo[j];
        x[4 + j] = (int)hi[j];
      }
      return x;
    };
    intx8 b[2];
#pragma unroll
    for (int bj = 0; bj < 2; ++bj) b[bj] = frag8(pb, 64 * wn + 32 * bj + i);
#pragma unroll
    for (int bi = 0; bi < P::BM / 64; ++bi) {
      const intx8 a = frag8(pa, wm * (P::BM / 2) + 32 * bi + i);
#pragma unroll
      for (int bj = 0; bj < 2; ++bj)
        acc.v[bi][bj] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b[bj], acc.v[bi][bj], 0, 0, 0, 127, 0, 127);
    }
  } else {
    const int q = lane >> 4, i = lane & 15;
    ml2::bf16x8 b[4];
#pragma unroll
    for (int bj = 0; bj < 4; ++bj) {
      if constexpr (P::MODE == FORGE_GROUPED_NN)
        b[bj] = ml2::frag(pb, 512, 4 * q + (i >> 2), 16 + 4 * q + (i >> 2), 64 * wn + 16 * bj, i);
      else b[bj] = __builtin_bit_cast(ml2::bf16x8, piece(pb, 64 * wn + 16 * bj + i, q));
    }
#pragma unroll
    for (int bi = 0; bi < P::MB; ++bi) {
      const int row = wm * (P::BM / 2) + 16 * bi + i;
      ml2::bf16x8 a;
      if constexpr (P::MODE == FORGE_GROUPED_NN) a = ml2::dy_frag(pa, row, q);
      else a = __builtin_bit_cast(ml2::bf16x8, piece(pa, row, q));
#pragma unroll
      for (int bj = 0; bj < 4; ++bj)
        acc.v[bi][bj] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b[bj], acc.v[bi][bj], 0, 0, 0);
    }
  }
}

// The whole contraction (none for rows of no group).  Ends with a barrier.
template <class P>
__device__ __forceinline__ void contract(Acc<P>& acc, unsigned char* smem, const GroupedArgs& a, const RowTile& t) {
  const int wave = threadIdx.x >> 6, wm = wave >> 2, wn = wave & 3;
  constexpr int NI = P::MODE == FORGE_GROUPED_NT8 ? P::BM / 64 : P::MB, NJ = P::MODE == FORGE_GROUPED_NT8 ? 2 : 4;
  constexpr int NR = P::MODE == FORGE_GROUPED_NT8 ? 16 : 4;
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int r = 0; r < NR; ++r) acc.v[i][j][r] = 0.0f;
  if (t.e >= a.E) return;  // nothing was staged: no barrier is needed
  RowsFeed f;
  make_feed<P>(f, a, t);
  const int nsl = (int)((P::MODE == FORGE_GROUPED_NN ? a.N : a.K) * P::ESZ / P::ROW);
#pragma unroll
  for (int s = 0; s < P::STAGES - 1; ++s)
    if (s < nsl) issue<P>(f, smem + s * P::STAGE, s);
  for (int s = 0; s < nsl; ++s) {
    const int ahead = min(nsl - 1 - s, P::STAGES - 2);
    if (ahead >= 2) wait_vm<2 * P::DMA>();
    else if (ahead == 1) wait_vm<P::DMA>();
    else wait_vm<0>();
    barrier();
    if (s + P::STAGES - 1 < nsl) issue<P>(f, smem + ((s + P::STAGES - 1) % P::STAGES) * P::STAGE, s + P::STAGES - 1);
    mma<P>(acc, smem + (s % P::STAGES) * P::STAGE, wm, wn);
  }
  barrier();
}

// Epilogue: the accumulators pass through LDS in fp32, 64 rows at a time (32 of either wave
// row), and leave as bf16 (nearest even) in 16-byte stores; fp8 sums take their row's and
// column's scales on the way.
constexpr int OUT_LD = 256 + 4;                 // floats per staged row
constexpr int OUT_BYTES = 64 * OUT_LD * 4;

template <class P>
__device__ __forceinline__ void store_tile(const Acc<P>& acc, unsigned char* smem, const GroupedArgs& a,
                                           const RowTile& t) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, wm = wave >> 2, wn = wave & 3;
  float* st = reinterpret_cast<float*>(smem);
  const int64_t O = P::MODE == FORGE_GROUPED_NN ? a.K : a.N, o0 = (int64_t)t.n * P::BN;
  uint16_t* out = static_cast<uint16_t*>(a.out);
#pragma unroll
  for (int part = 0; part < P::BM / 64; ++part) {
    // staged row 32 wm + y is tile row wm BM / 2 + 32 part + y
    if constexpr (P::MODE == FORGE_GROUPED_NT8) {
      // 32 x 32 output: lane l, register r: row 8 (r / 4) + 4 (l / 32) + r mod 4, column l mod 32
#pragma unroll
      for (int bj = 0; bj < 2; ++bj)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          st[(32 * wm + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3)) * OUT_LD + 64 * wn + 32 * bj + (lane & 31)] =
              acc.v[part][bj][r];
    } else {
#pragma unroll
      for (int b2 = 0; b2 < 2; ++b2)
#pragma unroll
        for (int bj = 0; bj < 4; ++bj)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            st[(32 * wm + 16 * b2 + 4 * (lane >> 4) + r) * OUT_LD + 64 * wn + 16 * bj + (lane & 15)] =
                acc.v[2 * part + b2][bj][r];
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < 4; ++s) {  // 64 rows x 32 pieces of 8 columns
      const int id = tid + 512 * s, y = id >> 5, c = 8 * (id & 31);
      const int row = (y >> 5) * (P::BM / 2) + 32 * part + (y & 31);
      if (row >= t.rows || o0 + c >= O) continue;
      const float* p = st + y * OUT_LD + c;
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = p[j];
      if constexpr (P::MODE == FORGE_GROUPED_NT8) {
        if (t.e < a.E) {
          const float sa = a.a_scale[t.row0 + row];
          const float* sw = a.w_scale + (int64_t)t.e * a.N + o0 + c;
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] *= sa * sw[j];
        }
      }
      u32x4 q;
#pragma unroll
      for (int j = 0; j < 4; ++j) q[j] = f32_to_bf16_rne(v[2 * j]) | (f32_to_bf16_rne(v[2 * j + 1]) << 16);
      st16(out + (int64_t)(t.row0 + row) * O + o0 + c, q);
    }
    __syncthreads();
  }
}

template <int BM, int MODE>
__global__ __launch_bounds__(512, BM == 64 ? 4 : 2) void grouped_rows_kernel(GroupedArgs a) {
  using P = RowsPipe<BM, MODE>;
  __shared__ __attribute__((aligned(1024))) unsigned char smem[P::SMEM > OUT_BYTES ? P::SMEM : OUT_BYTES];
  const int64_t O = MODE == FORGE_GROUPED_NN ? a.K : a.N;
  RowTile t;
  if (!find_tile<BM>(a.ends, a.E, a.T, (int)((O + P::BN - 1) / P::BN), (int)blockIdx.x, t)) return;
  Acc<P> acc;
  contract<P>(acc, smem, a, t);
  store_tile<P>(acc, smem, a, t);
}

}  // namespace grp
}  // namespace forge

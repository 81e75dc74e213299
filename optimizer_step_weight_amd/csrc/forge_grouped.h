// forge_grouped.h -- tiles of the matrix products grouped by expert: the lookup of a workgroup's
// expert and rows in the groups' ends, and the row products Y_e = X_e W_e^T and dX_e = dY_e W_e.
//
// Rows are sorted by expert and the groups' ends live on the device, so the host cannot know how
// many row tiles there are: at most T / BM + E + 1 (each group adds at most one partial tile, and
// so do the rows of no group).  The grid covers that bound; every wave scans the ends and finds
// the tile of its workgroup, and workgroups past the last tile end.  Tiles are ordered by
// expert, within an expert in blocks of 8 row tiles over all column tiles, and given to the 8
// XCDs in contiguous runs: an XCD's resident tiles share their weight and row panels in its L2
// (16384 x 14336 x 4096: 79 % of the L2's requests hit).
//
// Measured, over the cards seen: 16384 rows of 8 uneven experts by 14336 x 4096 in bf16 1.41-1.51 ms
// (1.27-1.36 PFLOP/s); in even groups 1.36 ms, where eight calls of the library, one an expert, take 1.42 and
// its product of one weight of that size 1.26.  16384 rows of 32 experts by 4096 x 4096 in fp8
// 0.29-0.33 ms (1.7-1.9 PFLOP/s).  Input gradient of 32768 rows of 64 experts by 1408 x 2048 0.20-0.22 ms.
// The card's power bounds the bf16 product: the clock falls to 1.6-1.7 GHz while the matrix cores are
// 85 % busy within a tile (74 % over the launch).  The others are at 41 % and 42 % and 2 GHz: shorter
// contractions over more, ragged groups.  There it is what a workgroup alone on its CU cannot hide:
// 2.4 thousand cycles to find its tile, 5 until its first slabs have come, 7 to store, beside 2.3 a slab.
#pragma once

#include "forge_layer_internal.h"
#include "forge_mainloop2.h"

namespace forge {
namespace grp {

using ml2::barrier;
using ml2::floatx4;
using ml2::make_rsrc;
using ml2::wait_vm;
typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef float floatx4u __attribute__((ext_vector_type(4), aligned(4)));

// Position of workgroup b in an order of `total` tiles in which each XCD (b mod 8) has a
// contiguous run.
__device__ __forceinline__ int xcd_run(int b, int total) {
  const int per = total >> 3, rem = total & 7, x = b & 7, loc = b >> 3;
  return (x < rem ? x * (per + 1) : rem * (per + 1) + (x - rem) * per) + loc;
}

// Inclusive scans over the wave by data-parallel moves within the vector unit: a workgroup finds its
// tile before it can load anything, and shuffles through LDS took 1.3 of the 3.4 thousand cycles.
template <class F>
__device__ __forceinline__ int wave_scan(int v, F&& join) {
  // lanes without a source take 0, which both joins leave as it is (no value is negative)
  v = join(v, __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false));  // 1, 2, 4, 8 lanes up in a row of 16
  v = join(v, __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false));
  v = join(v, __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false));
  v = join(v, __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false));
  v = join(v, __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false));  // last lane of a row to the next row
  v = join(v, __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false));  // lane 31 to the upper half
  return v;
}
__device__ __forceinline__ int scan_max(int v) {
  return wave_scan(v, [](int a, int b) { return a > b ? a : b; });
}
__device__ __forceinline__ int scan_sum(int v) {
  return wave_scan(v, [](int a, int b) { return a + b; });
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
  v = scan_max((int)v);
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
  int cols;       // columns of a column tile
};

// Up to this many tiles of 256 columns, the tiles take 128, all still on CUs at once: a product of
// few rows is a pass over the live experts' weights, and wants many CUs to read.  Experts of 1024 x
// 2048 in bf16: 30 live ones 29.3 us in 120 wide tiles, 26.0 us in 240 narrow ones (4.8 TB/s); 39 live
// ones 38.5 us in 156 wide tiles, 50.9 us in 312 narrow ones.  Contractions of other lengths were not compared.
constexpr int NARROW_TILES = 128;

// The tile of workgroup b among the row tiles of BM rows x the column tiles of O columns, of 256
// columns or, where there are few tiles and `least` is 128, of 128; false: none left.
template <int BM>
__device__ __forceinline__ bool find_tile(const int32_t* ends, int E, int64_t T, int64_t O, int least, int b, RowTile& out) {
  const int chunks = E / 64 + 1;
  auto tiles_of = [&](const Chunk& k) { return (int)((k.end - k.start + BM - 1) / BM); };
  int64_t carry = 0;
  int total = 0;  // the host keeps the grid, and with it every tile number, below 2^31
  Chunk k{};
  int incl = 0;
  for (int c = 0; c < chunks; ++c) {
    k = load_chunk(ends, E, T, c, carry);
    incl = scan_sum(tiles_of(k));
    total += __builtin_amdgcn_readlane(incl, 63);
    carry = __builtin_amdgcn_readlane((int)k.end, 63);
  }
  const int wide = (int)((O + 255) / 256);
  out.cols = least < 256 && (int64_t)total * wide <= NARROW_TILES ? 128 : 256;
  const int nbn = out.cols < 256 ? (int)((O + 127) / 128) : wide;
  total *= nbn;
  if (b >= total) return false;
  const int t = xcd_run(b, total);
  int before = 0;  // tiles of earlier chunks
  carry = 0;
  for (int c = 0; c < chunks; ++c) {
    if (chunks > 1) {
      k = load_chunk(ends, E, T, c, carry);
      incl = scan_sum(tiles_of(k));
      carry = __builtin_amdgcn_readlane((int)k.end, 63);
    }
    const uint64_t past = __ballot((before + incl) * nbn > t);
    if (past == 0) {
      before += __builtin_amdgcn_readlane(incl, 63);
      continue;
    }
    const int l = __builtin_ctzll(past);
    const int cnt = __builtin_amdgcn_readlane(tiles_of(k), l), last = __builtin_amdgcn_readlane(incl, l);
    const int start = __builtin_amdgcn_readlane((int)k.start, l), end = __builtin_amdgcn_readlane((int)k.end, l);
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

// ------------------------------------------------------------------ the contraction
// D[second, first] = sum over c of second[c] first[c]: a tile of 64 to 256 rows ("second") by 128 or 256
// columns ("first", contiguous in the output) by one workgroup of 4 waves (2 x 2).  256 x 256 tiles
// read the least of L2 and LDS for their products, one wave a SIMD holding 128 x 128 of it: eight
// waves of 128 x 64 read half as much again from LDS, and what they gained in cycles they lost in
// clock (power).  bf16 is multiplied in 16 x 16 x 32 blocks: in 32 x 32 x 16 ones the same loop was 75 %
// busy at 1.69 GHz instead of 69 % at 1.99, and slower (1439 against 1345 us).  fp8 takes
// 32 x 32 x 64 blocks, whose contraction is half a slab.  The accumulators are fp32, but the fp8 matrix
// instructions (16 x 16 x 32 ones alike) cut the products of eight consecutive elements at 2^-13 of the
// largest one's power of two before they add them.  Of 4096-long sums of a norm's rows 1.2 % are rounded to the bf16
// neighbour, at most 2^-19 of the sum of magnitudes off; the library's fp8 product gives the same bits.  Exact products
// would need the bf16 instructions, at half the rate.
//
// The contraction goes in slabs of 128 bytes of a row (64 bf16 or 128 fp8 elements), copied to LDS
// by DMA in whole 128-byte lines: L2 answers a request a line, and with half lines (slabs of 64
// bytes) its request rate, not its bytes, held the matrix cores at 62 % busy.  LDS holds three slabs of the
// second operand and two of the first (160 KiB for 256 x 256).  A wave holds the fragments of two
// half slabs in registers: while it multiplies one it reads the next from LDS.  step() has the
// timetable.
//
// An operand lies in memory either
//  * contraction-contiguous (TR = false: X, dY, W of the forward product): rows of 128 bytes in
//    LDS, a fragment (lane l: row l mod 16, 8 bf16 from 8 (l / 16); row l mod 32, 32 fp8 from
//    32 (l / 32)) read in 16-byte pieces.  The eight 16-byte chunks of a row are XOR-swizzled with
//    (row / 2) mod 8: 16 consecutive rows at one chunk fall in 16 distinct bank windows; or
//  * contraction-strided (TR = true: W of dgrad, X and dY of wgrad): 64 rows of the tile's width,
//    read by LDS transpose reads: lane i of 16 points at row base + i / 4, columns 4 (i mod 4)
//    .. + 3 and receives rows base .. base + 3 of column i.  Chunks are XOR-swizzled with
//    4 (row mod 4) + 2 (q mod 2): the eight half-windows that 32 lanes read are distinct.
// Reads past an operand's last row give zero (buffer range check).
constexpr int THREADS = 256;

// Element bytes, layout, rows (or columns) of the tile.  A lane's 8 contraction elements of a k-step of
// 32 are 8 q .. 8 q + 7 (q = l / 16), or with FOURS 4 q .. + 3 and 16 + 4 q .. + 3: the order of the
// fused step's contraction (forge_mainloop2.h), which gives its sums bit for bit.
template <int E_, bool TR_, int WIDTH_, bool FOURS_ = false>
struct Side {
  static constexpr int ESZ = E_, WIDTH = WIDTH_;
  static constexpr bool TR = TR_, FOURS = FOURS_;
  static constexpr int R_LANE = FOURS ? 4 : 8, R_HIGH = FOURS ? 16 : 4;  // TR: rows from q to q + 1, to the second read
  static constexpr int PANEL = WIDTH * 128;                // bytes a slab
  static constexpr int ROW = TR ? WIDTH * 2 : 128;         // bytes of a row in LDS
  static constexpr int CPR = ROW / 16, RPD = 64 / CPR;     // chunks of a row, rows of a 1 KiB copy
  static constexpr int DMA = PANEL / 4096;                 // copies of a wave a slab
  static constexpr int M = ESZ == 2 ? 16 : 32;             // side of a matrix block
  static constexpr int BLOCKS = WIDTH / 2 / M;             // blocks of a wave
  static_assert(TR || !FOURS, "only transpose reads take the rows in fours");
  static_assert(!TR || (ESZ == 2 && WIDTH >= 128), "transpose reads are of 16-bit elements");
  static __device__ __forceinline__ int swz(int r) { return TR ? 4 * (r & 3) + 2 * ((r / R_LANE) & 1) : (r >> 1) & 7; }
};

// One copy of 1 KiB: 16 bytes a lane from rsrc + off to LDS address `lds` + AT + 16 lane.  Two
// instructions, because a wave issues one in 4 cycles: three fit beside a 16 x 16 x 32 product, and
// more would keep the matrix core waiting.  Completion is awaited with wait_vm.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
template <int AT>
__device__ __forceinline__ void copy_1k(const u32x4& rsrc, uint32_t off, uint32_t lds) {
  asm volatile("s_add_u32 m0, %0, %1\n\tbuffer_load_dwordx4 %2, %3, 0 offen lds" ::"s"(lds), "i"(AT), "v"(off), "s"(rsrc)
               : "memory", "m0", "scc");
}
#pragma clang diagnostic pop
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p);
}

// Copies of an operand, slab after slab.
template <class S>
struct Feed {
  u32x4 rsrc;               // from the next slab to be copied to the operand's end
  uint32_t step;            // bytes from slab to slab
  int slabs;                // left from there
  uint32_t off[S::DMA];     // of this lane's pieces

  // first: the tile's first element; bytes: from there to the operand's end; ld: row length in bytes.
  __device__ __forceinline__ void open(const void* first, uint32_t bytes, uint32_t ld, int slabs_) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    rsrc = make_rsrc(first, bytes);
    step = S::TR ? 64u * ld : 128u;
    slabs = slabs_;
#pragma unroll
    for (int j = 0; j < S::DMA; ++j) {
      const int r = S::RPD * (S::DMA * wave + j) + lane / S::CPR;
      off[j] = (uint32_t)r * ld + 16u * (uint32_t)((lane % S::CPR) ^ S::swz(r));
    }
  }
  // To the next slab, in two parts.  Past the last one the buffer is empty: its copies touch no
  // memory, so that the loop has one body for all slabs.
  __device__ __forceinline__ void next_base() {
    const uint64_t b = ((uint64_t)rsrc.y << 32 | rsrc.x) + step;
    rsrc.x = (uint32_t)b;
    rsrc.y = (uint32_t)(b >> 32);
    asm volatile("" : "+s"(rsrc));
  }
  __device__ __forceinline__ void next_bytes() {
    const uint32_t left = rsrc.z - step;
    --slabs;
    rsrc.z = slabs > 0 ? left : 0u;
    asm volatile("" : "+s"(rsrc));
  }
  __device__ __forceinline__ void next() {
    next_base();
    next_bytes();
  }
};

typedef short v8i16 __attribute__((ext_vector_type(8)));

// A block over half a slab: bf16 16 rows x 32, fp8 32 rows x 64.
template <int ESZ>
struct Frag {
  u32x4 q[ESZ == 2 ? 1 : 2];
};
// A wave's blocks in LDS: the addresses of this lane's pieces in a panel at address 0.  One piece is
// read at v + the panel's place + a constant, so a half slab takes an addition for each v, not for
// each piece.
template <class S>
struct View {
  static constexpr int N = S::TR ? S::BLOCKS : (S::ESZ == 2 ? 2 : 4);
  uint32_t v[N], at[2];
  // first: the wave's first row (TR: column); less: taken off, as the places have it.
  __device__ __forceinline__ void open(int first, int less) {
    const int lane = threadIdx.x & 63;
    if constexpr (S::TR) {
      const int i = lane & 15, r = S::R_LANE * (lane >> 4) + (i >> 2);
#pragma unroll
      for (int b = 0; b < N; ++b)
        v[b] = (uint32_t)(r * S::ROW + 16 * ((first / 8 + 2 * b + ((i & 3) >> 1)) ^ S::swz(r)) + 8 * (i & 1) - less);
    } else {
      const int r = first + (lane & (S::M - 1));  // `first` and M are multiples of 16: one swizzle for all blocks
#pragma unroll
      for (int x = 0; x < N; ++x) {
        const int c = S::ESZ == 2 ? 4 * x + (lane >> 4) : 4 * (x >> 1) + 2 * (lane >> 5) + (x & 1);
        v[x] = (uint32_t)(r * 128 + 16 * (c ^ S::swz(r)) - less);
      }
    }
  }
  // Piece KK of half H of block B.  Block 0 is read first.  (The empty asm keeps the compiler from
  // folding the constants into v and adding the place for every piece.)
  template <int B, int H, int KK>
  __device__ __forceinline__ u32x4 read(uint32_t place) {
    using P4 = __attribute__((address_space(3))) const u32x4*;
    if constexpr (S::TR) {
      using P2 = __attribute__((address_space(3))) ml2::v4i16*;
      // rows r and r + R_HIGH have the same swizzle
      uint32_t at = v[B] + place;
      asm("" : "+v"(at));
      const ml2::v4i16 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P2)(at + 32 * H * S::ROW));
      const ml2::v4i16 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P2)(at + (32 * H + S::R_HIGH) * S::ROW));
      return __builtin_bit_cast(u32x4, (v8i16)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      if constexpr (B == 0) {
        at[KK] = v[S::ESZ == 2 ? H : 2 * H + KK] + place;
        asm("" : "+v"(at[KK]));
      }
      return *(P4)(at[KK] + B * S::M * 128);
    }
  }
};

constexpr int WAVE_LDS = 32768;  // of the tile's 160 KiB, once they are free

template <class A, class B>  // second (rows), first (columns)
struct Tile {
  static constexpr int MB = A::BLOCKS, NB = B::BLOCKS, ESZ = A::ESZ, M = A::M;
  static constexpr int PIECES = ESZ == 2 ? 1 : 2, READS = PIECES * (MB + NB);  // of half a slab
  using Acc = std::conditional_t<ESZ == 2, floatx4, floatx16>;
  static constexpr int STAGES_A = 3, STAGES_B = 2;
  static constexpr int SMEM = STAGES_A * A::PANEL + STAGES_B * B::PANEL;
  Acc acc[MB][NB];

  struct Frags {
    Frag<ESZ> a[MB], b[NB];
  };

  // d += b a.  A tile of 256 x 256 has 256 accumulators a lane, all the AGPRs that there are; the
  // allocator then moves some to and fro within the loop.  The register kind is therefore named here:
  // three quarters of them AGPRs, the rest VGPRs, with room left in both.  The compiler does not see
  // that these are matrix instructions: settle() is due before anything else reads d.
  template <int BLOCK>
  static __device__ __forceinline__ void mma(Acc& d, const Frag<ESZ>& b, const Frag<ESZ>& a) {
    constexpr bool AGPR = BLOCK * (M * M / 64) < 192;
    if constexpr (ESZ == 2) {
      if constexpr (AGPR) asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(d) : "v"(b.q[0]), "v"(a.q[0]));
      else asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+v"(d) : "v"(b.q[0]), "v"(a.q[0]));
    } else {
      auto whole = [](const Frag<1>& f) { return __builtin_shufflevector(f.q[0], f.q[1], 0, 1, 2, 3, 4, 5, 6, 7); };
      if constexpr (AGPR) asm volatile("v_mfma_f32_32x32x64_f8f6f4 %0, %1, %2, %0" : "+a"(d) : "v"(whole(b)), "v"(whole(a)));
      else asm volatile("v_mfma_f32_32x32x64_f8f6f4 %0, %1, %2, %0" : "+v"(d) : "v"(whole(b)), "v"(whole(a)));
    }
  }

  // After the matrix instructions that the compiler does not see: their last results are written
  // (19 wait states at most, after a 32 x 32 x 64 product).
  static __device__ __forceinline__ void settle() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  }

  View<A> va;
  View<B> vb;
  // Read n of the fragments of half h of a slab at (pa, pb).
  template <int H, int n>
  __device__ __forceinline__ void read(Frags& f, uint32_t pa, uint32_t pb) {
    constexpr int kk = n % PIECES, i = n / PIECES;
    if constexpr (i < NB) f.b[i].q[kk] = vb.template read<i, H, kk>(pb);
    else f.a[i - NB].q[kk] = va.template read<i - NB, H, kk>(pa);
  }

  // LDS addresses of the panels of slab s and slab s + 1 in either ring, and of the A panel that is
  // being filled.  They include the wave's
  // first copy, which the views' addresses take off again.
  struct Places {
    uint32_t a, a_next, a_fill, a_first, a_end, b, b_next, b_sum;
    __device__ __forceinline__ void find_next() {
      a_next = a + A::PANEL;
      a_next = a_next == a_end ? a_first : a_next;
      asm volatile("" : "+s"(a_next));
      b_next = b_sum - b;
      asm volatile("" : "+s"(b_next));
    }
  };

  // How many of `many` things, spread evenly over the products [from, to), come before product n.
  static constexpr int due(int many, int from, int to, int n) {
    return n <= from ? 0 : n >= to ? many : (many * (n - from) + (to - from) - 1) / (to - from);
  }

  // Slab s, whose first half is in f, up to the first half of slab s + 1 in f.  In sixteenths of
  // the H products of half a slab:
  //    0 ..  7  the second half is read to g
  //         10  it has been read by all waves (barrier): the place of slab s is free
  //   10 .. 26  B of slab s + 2 is copied there, 26 .. 42 (10 of the next slab) A of slab s + 3
  //         22  slab s + 1 has landed for all waves (barrier)
  //   22 .. 29  its first half is read to f
  // The copies keep one pace throughout, half of what the address unit takes: a faster one makes
  // waves wait to issue them.  A copy has at least 1.75 H products' time to land, a read 3 / 16 H.
  __device__ __forceinline__ void step(Frags& f, Frags& g, Feed<A>& fa, Feed<B>& fb, Places& at) {
    constexpr int H = MB * NB;
    constexpr int FREE = 10 * H / 16, LANDED = 22 * H / 16, G_END = 7 * H / 16, F_END = 29 * H / 16;
    constexpr int A_FROM = 26 * H / 16;
    // two wait states from a vector instruction that writes an accumulator (the zeroes before the first
    // slab) to a matrix instruction that reads it
    asm volatile("s_nop 1" ::: "memory");
    static_for<2 * H>([&](auto nc) {
      constexpr int n = decltype(nc)::value;
      // the scalar work, a few instructions at a time
      if constexpr (n == (G_END < FREE ? G_END : FREE)) fb.next_base();
      if constexpr (n == (G_END + 1 < FREE ? G_END + 1 : FREE)) fb.next_bytes();
      if constexpr (n == (FREE + 2 < A_FROM ? FREE + 2 : A_FROM)) fa.next_base();
      if constexpr (n == (FREE + 3 < A_FROM ? FREE + 3 : A_FROM)) fa.next_bytes();
      if constexpr (n == (FREE + 4 < LANDED ? FREE + 4 : LANDED)) at.find_next();
      if constexpr (n == FREE) {
        __builtin_amdgcn_s_waitcnt(0xF | (0x3 << 14) | (0x7 << 4));
        barrier();
      }
      if constexpr (n == LANDED) {
        // copied later than slab s + 1: A of s + 2 and the first copies of B of s + 2
        wait_vm<A::DMA + due(B::DMA, FREE, A_FROM, n)>();
        barrier();
      }
      if constexpr (n == A_FROM) at.a_fill = at.a;
      constexpr int b0 = due(B::DMA, FREE, A_FROM, n), b1 = due(B::DMA, FREE, A_FROM, n + 1);
      static_for<b1 - b0>([&](auto k) {
        constexpr int j = b0 + decltype(k)::value;
        copy_1k<j * 1024>(fb.rsrc, fb.off[j], at.b);
      });
      constexpr int an = n < FREE ? n + 2 * H : n;
      constexpr int a0 = due(A::DMA, A_FROM, FREE + 2 * H, an), a1 = due(A::DMA, A_FROM, FREE + 2 * H, an + 1);
      static_for<a1 - a0>([&](auto k) {
        constexpr int j = a0 + decltype(k)::value;
        copy_1k<j * 1024>(fa.rsrc, fa.off[j], at.a_fill);
      });
      constexpr int g0 = due(READS, 0, G_END, n), g1 = due(READS, 0, G_END, n + 1);
      static_for<g1 - g0>([&](auto k) { read<1, g0 + decltype(k)::value>(g, at.a, at.b); });
      constexpr int f0 = due(READS, LANDED, F_END, n), f1 = due(READS, LANDED, F_END, n + 1);
      static_for<f1 - f0>([&](auto k) { read<0, f0 + decltype(k)::value>(f, at.a_next, at.b_next); });
      if constexpr (n < H) mma<n>(acc[n / NB][n % NB], f.b[n % NB], f.a[n / NB]);
      else mma<n - H>(acc[n / NB - MB][n % NB], g.b[n % NB], g.a[n / NB - MB]);
      __builtin_amdgcn_sched_barrier(0);
    });
    at.a = at.a_next;
    at.b = at.b_next;
  }
  // Copies of A that a slab's end starts, before the next slab's beginning goes on.
  static constexpr int A_EARLY = due(A::DMA, 26 * (MB * NB) / 16, 10 * (MB * NB) / 16 + 2 * MB * NB, 2 * MB * NB);

  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int r = 0; r < M * M / 64; ++r) acc[i][j][r] = 0.0f;
  }

  // The whole contraction over `slabs` slabs.  All waves call it; LDS must be free when it is
  // called, and is free again after a further barrier.
  __device__ __forceinline__ void contract(unsigned char* smem, Feed<A>& fa, Feed<B>& fb, int slabs) {
    if (slabs == 0) return zero();
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t to_a = lds_address(smem) + (uint32_t)(wave * A::DMA * 1024);
    const uint32_t to_b = lds_address(smem) + STAGES_A * A::PANEL + (uint32_t)(wave * B::DMA * 1024);
    static_for<3>([&](auto sc) {  // two slabs and the first copies of A of the third
      constexpr int s = decltype(sc)::value;
      if constexpr (s > 0) fa.next();
      static_for<(s < 2 ? A::DMA : A_EARLY)>(
          [&](auto j) { copy_1k<s * A::PANEL + j * 1024>(fa.rsrc, fa.off[j], to_a); });
      if constexpr (s == 1) fb.next();
      if constexpr (s < 2)
        static_for<B::DMA>([&](auto j) { copy_1k<s * B::PANEL + j * 1024>(fb.rsrc, fb.off[j], to_b); });
    });
    __builtin_amdgcn_sched_barrier(0);
    zero();  // while the copies fly
    va.open(M * MB * (wave >> 1), wave * A::DMA * 1024);
    vb.open(M * NB * (wave & 1), wave * B::DMA * 1024);
    wait_vm<A::DMA + B::DMA + A_EARLY>();
    barrier();
    Frags f, g;
    static_for<READS>([&](auto n) { read<0, n>(f, to_a, to_b); });
    Places at{to_a, 0, to_a + 2 * A::PANEL, to_a, to_a + STAGES_A * A::PANEL, to_b, 0, 2 * to_b + B::PANEL};
    for (int s = slabs; s > 0; --s) step(f, g, fa, fb, at);
    settle();
    wait_vm<0>();  // no copy may land after the workgroup's end
  }

  // First row and column of this wave in the tile.
  static __device__ __forceinline__ int row0() { return M * MB * (int)(threadIdx.x >> 7); }
  static __device__ __forceinline__ int col0() { return M * NB * (int)((threadIdx.x >> 6) & 1); }

  // The tile to memory by rows.  A lane holds 4 consecutive columns of one of a block's M rows, and a
  // store from there would touch 16 rows at once, 32 or 64 bytes of each.  So rows of blocks pass, some
  // at a time, through 32 KiB of the wave's own in LDS (no barrier: a wave's LDS accesses are in
  // order), and leave as whole rows of the wave's M NB columns, 16 bytes a lane.  Chunks of 16 bytes
  // are XOR-swizzled with the row.  pack(row, column, v): the 4 values of a row of the wave from that
  // column on as they are stored (8 bytes bf16 or 16 fp32); put(row, column, q): stores 16 bytes.
  template <class Unit, class Pack, class Put>
  __device__ __forceinline__ void store(unsigned char* wave_lds, Pack&& pack, Put&& put) const {
    constexpr int SIZE = sizeof(Unit) / 4;              // of an element
    constexpr int ROW = M * NB * SIZE, CH = ROW / 16;   // bytes and chunks of a row
    constexpr int MASK = (CH < 16 ? CH : 16) - 1;
    constexpr int FIT = WAVE_LDS / (M * ROW), G = FIT < MB ? FIT : MB;  // rows of blocks at a time
    const int lane = (int)threadIdx.x & 63, row = lane & (M - 1);
#pragma unroll
    for (int i0 = 0; i0 < MB; i0 += G) {
#pragma unroll
      for (int i = i0; i < (i0 + G < MB ? i0 + G : MB); ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
          for (int g = 0; g < M * M / 256; ++g) {
            const int c4 = M / 4 * j + 64 / M * g + lane / M;  // column / 4
            const Unit u = pack(M * i + row, 4 * c4, floatx4{acc[i][j][4 * g], acc[i][j][4 * g + 1],
                                                             acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]});
            const int byte = c4 * (int)sizeof(Unit);
            *reinterpret_cast<Unit*>(wave_lds + ((i - i0) * M + row) * ROW + 16 * ((byte >> 4) ^ (row & MASK)) +
                                     (byte & 15)) = u;
          }
      __builtin_amdgcn_wave_barrier();
      asm volatile("" ::: "memory");
#pragma unroll
      for (int t = 0; t < (i0 + G < MB ? G : MB - i0) * M * CH / 64; ++t) {
        const int p = lane + 64 * t, r = p / CH, c = p % CH;
        put(M * i0 + r, 16 / SIZE * c, *reinterpret_cast<const u32x4*>(wave_lds + r * ROW + 16 * (c ^ (r & MASK))));
      }
      __builtin_amdgcn_wave_barrier();
      asm volatile("" ::: "memory");
    }
  }
};

// A store that is not kept in L2 in favour of the operands.
__device__ __forceinline__ void st16_stream(void* p, u32x4 q) {
  __builtin_nontemporal_store(q, reinterpret_cast<u32x4*>(p));
}

// Two values to bf16, nearest even, in one instruction.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)lo, (__bf16)hi});
}

// ------------------------------------------------------------------ row products
// Y_e = X_e W_e^T and dX_e = dY_e W_e.  A row tile is 256 rows, or the last rows of a group in the
// least multiple of 64; the last columns of an odd multiple of 128 take a tile half as wide.
template <int MODE, int HEIGHT, int WIDTH>  // of the tile, in 64s
__device__ __forceinline__ void rows_tile(const GroupedArgs& a, const RowTile& t, unsigned char* smem) {
  constexpr bool NN = MODE == FORGE_GROUPED_NN, FP8 = MODE == FORGE_GROUPED_NT8;
  constexpr int ESZ = FP8 ? 1 : 2;
  using A = Side<ESZ, false, 64 * HEIGHT>;
  using B = Side<ESZ, NN, 64 * WIDTH>;
  using T = Tile<A, B>;
  const int64_t C = NN ? a.N : a.K, O = NN ? a.K : a.N, o0 = (int64_t)t.n * t.cols;
  const int slabs = t.e < a.E ? (int)(C * ESZ / 128) : 0;  // rows of no group: zeros
  Feed<A> fa;
  Feed<B> fb;
  fa.open(static_cast<const unsigned char*>(a.A) + (int64_t)t.row0 * C * ESZ, (uint32_t)(t.rows * C * ESZ),
          (uint32_t)(C * ESZ), slabs);
  const unsigned char* W = static_cast<const unsigned char*>(a.W) + (int64_t)t.e * a.N * a.K * ESZ;
  if constexpr (NN) fb.open(W + o0 * 2, (uint32_t)(a.N * a.K * 2 - o0 * 2), (uint32_t)(a.K * 2), slabs);
  else fb.open(W + o0 * C * ESZ, (uint32_t)(64 * WIDTH * C * ESZ), (uint32_t)(C * ESZ), slabs);
  T tile;
  tile.contract(smem, fa, fb, slabs);

  barrier();  // every wave is done with the slabs
  const int row0 = T::row0(), col0 = T::col0();
  uint16_t* out = static_cast<uint16_t*>(a.out) + (int64_t)(t.row0 + row0) * O + o0 + col0;
  const float* ws = FP8 && t.e < a.E ? a.w_scale + (int64_t)t.e * a.N + o0 + col0 : nullptr;
  const float* as = FP8 ? a.a_scale + t.row0 + row0 : nullptr;
  const int rows = t.rows - row0;
  tile.template store<u32x2>(
      smem + (threadIdx.x >> 6) * WAVE_LDS,
      [&](int row, int col, floatx4 v) {
        if constexpr (FP8) {
          if (ws) {
            const float sa = row < rows ? as[row] : 0.0f;
            const floatx4u sw = *reinterpret_cast<const floatx4u*>(ws + col);
#pragma unroll
            for (int x = 0; x < 4; ++x) v[x] = (v[x] * sa) * sw[x];  // the scales' product may leave fp32's range
          }
        }
        return u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
      },
      [&](int row, int col, u32x4 q) {
        if (row < rows) st16_stream(out + (int64_t)row * O + col, q);
      });
}

template <int MODE>
__global__ __launch_bounds__(THREADS, 1) void grouped_rows_kernel(GroupedArgs a) {
  __shared__ __attribute__((aligned(1024))) unsigned char smem[5 * 32768];
  const int64_t O = MODE == FORGE_GROUPED_NN ? a.K : a.N;
  RowTile t;
  if (!find_tile<256>(a.ends, a.E, a.T, O, a.cols, (int)blockIdx.x, t)) return;
  const bool narrow = t.cols < 256 || O - (int64_t)t.n * 256 < 256;
  switch ((t.rows + 63) / 64 + (narrow ? 4 : 0)) {
    case 1: rows_tile<MODE, 1, 4>(a, t, smem); break;
    case 2: rows_tile<MODE, 2, 4>(a, t, smem); break;
    case 3: rows_tile<MODE, 3, 4>(a, t, smem); break;
    case 4: rows_tile<MODE, 4, 4>(a, t, smem); break;
    case 5: rows_tile<MODE, 1, 2>(a, t, smem); break;
    case 6: rows_tile<MODE, 2, 2>(a, t, smem); break;
    case 7: rows_tile<MODE, 3, 2>(a, t, smem); break;
    case 8: rows_tile<MODE, 4, 2>(a, t, smem); break;
  }
}

}  // namespace grp
}  // namespace forge

// forge_block.hip -- 8-bit codes in blocks of 128: activations by rows (1 x 128), weights by squares
// (128 x 128) with a transposed copy, and the activation's backward pass that reads such codes.
//
// All are bound by memory: every element is read and written once.  A thread takes 8 consecutive columns,
// 16 threads a block, whose largest magnitude they find by exchanges within the vector unit.
//
// 16384 x 5120 bf16 to int8 49 us and back 46 (5.3-5.5 TB/s); activation's backward pass of 4099 x 17408 from e4m3 112-116
// us (6.2-6.4 TB/s); weights of 8 x 14336 x 4096 with the transposed copy 403 us (4.7 TB/s, a copy's rate; its bytes
// turn in LDS, which is busy throughout but not what it waits for).
#include <hip/hip_runtime.h>

#include "forge_act.h"

namespace forge {

namespace {

constexpr int kThreads = 256;
constexpr int64_t kMaxBlocks = int64_t(1) << 16;  // workgroups of a launch; each walks on from there

// Group g of 16 threads takes block g of the T x ceil(D / 128) blocks: its row, first column, and this
// thread's columns in it.
struct Place {
  int64_t row, at;  // element index of this thread's first column
  int block, n;     // block of the row, columns of this thread in the row (0 .. 8)
};
__device__ __forceinline__ Place place_of(int64_t g, int64_t D, int blocks) {
  Place p;
  p.row = g / blocks;
  p.block = (int)(g - p.row * blocks);
  const int64_t c = (int64_t)p.block * 128 + 8 * (threadIdx.x & 15);
  p.at = p.row * D + c;
  p.n = D - c < 0 ? 0 : D - c > 8 ? 8 : (int)(D - c);
  return p;
}

template <bool BF, int Q, bool ODD>
__global__ __launch_bounds__(kThreads) void quantize_kernel(BlockArgs a) {
  const int blocks = (int)((a.D + 127) / 128);
  const int64_t total = a.T * blocks, step = (int64_t)gridDim.x * (kThreads / 16);
  for (int64_t g = (int64_t)blockIdx.x * (kThreads / 16) + threadIdx.x / 16; g < total; g += step) {
    const Place p = place_of(g, a.D, blocks);
    float v[8] = {};
    if (p.n) unpack8<BF>(load_cols<BF, ODD>(a.x, p.at, p.n), v);
    const float scale = block_scale<Q>(max16(amax_bits(v)));
    if (p.n) store_codes<ODD>(static_cast<uint8_t*>(a.y) + p.at, encode8<Q>(v, scale), p.n);
    if ((threadIdx.x & 15) == 0) a.scale[g] = scale;
  }
}

template <bool BF, int Q, bool ODD>
__global__ __launch_bounds__(kThreads) void dequantize_kernel(BlockArgs a) {
  const int blocks = (int)((a.D + 127) / 128);
  const int64_t total = a.T * blocks, step = (int64_t)gridDim.x * (kThreads / 16);
  for (int64_t g = (int64_t)blockIdx.x * (kThreads / 16) + threadIdx.x / 16; g < total; g += step) {
    const Place p = place_of(g, a.D, blocks);
    if (!p.n) continue;
    float v[8];
    decode8<Q>(load_codes<ODD>(static_cast<const uint8_t*>(a.x) + p.at, p.n), a.scale[g], v);
    store_cols<BF, ODD>(a.y, p.at, v, p.n);
  }
}

// One workgroup a square: thread (r, c) has rows r, r + 16, .. and columns 8 c .. 8 c + 7.
template <bool BF, bool TURN>
__global__ __launch_bounds__(kThreads) void quantize_weight_kernel(BlockWeightArgs a) {
  __shared__ uint32_t red[4];
  __shared__ __attribute__((aligned(16))) uint8_t turned[128 * 144];
  const int kb = (int)(a.K / 128), nb = (int)(a.N / 128);
  const int64_t sq = blockIdx.x, e = sq / ((int64_t)nb * kb);
  const int in = (int)(sq - e * nb * kb), bn = in / kb, bk = in - bn * kb;
  const int r0 = threadIdx.x >> 4, c = threadIdx.x & 15;
  const int64_t base = (e * a.N + bn * 128) * a.K + bk * 128 + 8 * c;
  Raw8<BF> raw[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) raw[i] = load8<BF>(a.W, base + (int64_t)(r0 + 16 * i) * a.K);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float v[8];
    unpack8<BF>(raw[i], v);
    m = umax(m, amax_bits(v));
  }
  m = max16(m);
  m = umax(m, __shfl_xor(m, 16));
  m = umax(m, __shfl_xor(m, 32));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
  __syncthreads();
  m = umax(umax(red[0], red[1]), umax(red[2], red[3]));
  const float scale = block_scale<FORGE_Q_FP8>(m);
  if (threadIdx.x == 0) {
    a.scale[sq] = scale;
    if constexpr (TURN) a.scale_t[(e * kb + bk) * nb + bn] = scale;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float v[8];
    unpack8<BF>(raw[i], v);
    const u32x2 q = encode8<FORGE_Q_FP8>(v, scale);
    store_codes<false>(a.q + base + (int64_t)(r0 + 16 * i) * a.K, q, 8);
    if constexpr (TURN)
#pragma unroll
      for (int j = 0; j < 8; ++j) turned[(8 * c + j) * 144 + r0 + 16 * i] = (uint8_t)(q[j >> 2] >> (8 * (j & 3)));
  }
  if constexpr (TURN) {
    __syncthreads();
    uint8_t* out = a.qt + (e * a.K + bk * 128) * a.N + bn * 128;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = (threadIdx.x >> 3) + 32 * i, x = 16 * (threadIdx.x & 7);
      __builtin_nontemporal_store(ld16(turned + r * 144 + x), reinterpret_cast<u32x4*>(out + (int64_t)r * a.N + x));
    }
  }
}

// Gate and up of 8 columns of a row: KEEP F32, BF16 or codes.
template <int KEEP, bool ODD>
__device__ __forceinline__ void load_kept8(const KeptArgs& k, int64_t at, int64_t scale_at, int n, float (&v)[8]) {
  if constexpr (KEEP == FORGE_KEEP_F32 || KEEP == FORGE_KEEP_BF16)
    unpack8<KEEP == FORGE_KEEP_BF16>(load_cols<KEEP == FORGE_KEEP_BF16, ODD>(k.data, at, n), v);
  else
    decode8<KEEP == FORGE_KEEP_FP8 ? FORGE_Q_FP8 : FORGE_Q_I8>(load_codes<ODD>(static_cast<const uint8_t*>(k.data) + at, n),
                                                             k.scale[scale_at], v);
}

template <bool BF, int KEEP, bool ODD>
__global__ __launch_bounds__(kThreads) void gated_backward_kernel(GatedBwdArgs a) {
  const int blocks = (int)((a.N + 127) / 128);
  const int64_t total = a.T * blocks, step = (int64_t)gridDim.x * (kThreads / 16);
  for (int64_t i = (int64_t)blockIdx.x * (kThreads / 16) + threadIdx.x / 16; i < total; i += step) {
    const Place p = place_of(i, a.N, blocks);
    if (!p.n) continue;
    const int64_t at = p.at + p.row * a.N, sc = p.row * 2 * blocks + p.block;  // of gate; up is N, `blocks` further
    float d[8], g[8], u[8], h[8];
    unpack8<BF>(load_cols<BF, ODD>(a.dH, p.at, p.n), d);
    load_kept8<KEEP, ODD>(a.keep, at, sc, p.n, g);
    load_kept8<KEEP, ODD>(a.keep, at + a.N, sc + blocks, p.n, u);
    by_act(a.act, [&](auto act) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float v, s;
        act_pair<decltype(act)::value>(g[j], v, s);
        h[j] = v * u[j];
        g[j] = d[j] * u[j] * s;
        u[j] = d[j] * v;
      }
    });
    store_cols<BF, ODD>(a.dGU, at, g, p.n);
    store_cols<BF, ODD>(a.dGU, at + a.N, u, p.n);
    if (a.H) store_cols<BF, ODD>(a.H, p.at, h, p.n);
  }
}

unsigned grid_of(int64_t T, int64_t D) {
  const int64_t g = (T * ((D + 127) / 128) + kThreads / 16 - 1) / (kThreads / 16);
  return (unsigned)(g < kMaxBlocks ? g : kMaxBlocks);
}

template <class F>
void by_flags(bool a, bool b, bool c, F&& f) {
  using std::bool_constant;
  auto third = [&](auto x, auto y) { c ? f(x, y, bool_constant<true>{}) : f(x, y, bool_constant<false>{}); };
  auto second = [&](auto x) { b ? third(x, bool_constant<true>{}) : third(x, bool_constant<false>{}); };
  a ? second(bool_constant<true>{}) : second(bool_constant<false>{});
}

}  // namespace

int launch_block_quantize(const BlockArgs& a, void* stream) {
  by_flags(a.bf16, a.q == FORGE_Q_FP8, a.D % 8 != 0, [&](auto bf, auto fp8, auto odd) {
    hipLaunchKernelGGL((quantize_kernel<bf.value, fp8.value ? FORGE_Q_FP8 : FORGE_Q_I8, odd.value>), dim3(grid_of(a.T, a.D)),
                       dim3(kThreads), 0, (hipStream_t)stream, a);
  });
  return (int)hipGetLastError();
}

int launch_block_dequantize(const BlockArgs& a, void* stream) {
  by_flags(a.bf16, a.q == FORGE_Q_FP8, a.D % 8 != 0, [&](auto bf, auto fp8, auto odd) {
    hipLaunchKernelGGL((dequantize_kernel<bf.value, fp8.value ? FORGE_Q_FP8 : FORGE_Q_I8, odd.value>), dim3(grid_of(a.T, a.D)),
                       dim3(kThreads), 0, (hipStream_t)stream, a);
  });
  return (int)hipGetLastError();
}

int launch_block_quantize_weight(const BlockWeightArgs& a, void* stream) {
  const dim3 grid((unsigned)(a.E * (a.N / 128) * (a.K / 128)));
  by_flags(a.bf16, a.qt != nullptr, false, [&](auto bf, auto turn, auto) {
    hipLaunchKernelGGL((quantize_weight_kernel<bf.value, turn.value>), grid, dim3(kThreads), 0, (hipStream_t)stream, a);
  });
  return (int)hipGetLastError();
}

int launch_gated_backward(const GatedBwdArgs& a, void* stream) {
  by_flags(a.bf16, a.N % 8 != 0, false, [&](auto bf, auto odd, auto) {
    auto go = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3(grid_of(a.T, a.N)), dim3(kThreads), 0, (hipStream_t)stream, a);
    };
    constexpr bool BF = bf.value, ODD = odd.value;
    switch (a.keep.type) {
      case FORGE_KEEP_FP8: go(gated_backward_kernel<BF, FORGE_KEEP_FP8, ODD>); break;
      case FORGE_KEEP_I8: go(gated_backward_kernel<BF, FORGE_KEEP_I8, ODD>); break;
      default: go(gated_backward_kernel<BF, BF ? FORGE_KEEP_BF16 : FORGE_KEEP_F32, ODD>); break;
    }
  });
  return (int)hipGetLastError();
}

}  // namespace forge

// forge_norm_backward.h -- kernels of the RMS norm's backward pass (forge_norm.hip has the formulas), from h
// itself or from its 8-bit codes in blocks of 128 columns, and the reductions that all norm kernels use.
//
// Codes halve or quarter what is read of h; they are decoded as they are used, and the sums are the same.  8192 x
// 4096 in bf16 from int8: 53 us (4.4 TB/s), of which the rows' kernel 40 and the gain's sum 5; 57 from bf16 h.
#pragma once

#include <hip/hip_runtime.h>

#include "forge_rows.h"

namespace forge {

void launch_rmsnorm_backward_q8(int bf16, const NormBwdArgs& a, int64_t groups, void* stream);

namespace {

struct Sum {
  static __device__ __forceinline__ float join(float a, float b) { return a + b; }
};
struct Max {
  static __device__ __forceinline__ float join(float a, float b) { return amax2(a, b); }
};

// Reduction over the TPR threads of a row; red: TPR / 64 floats of this use (TPR > 64).
template <class Op, int TPR>
__device__ __forceinline__ float row_reduce(float v, float* red) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = Op::join(v, __shfl_xor(v, o));
  if constexpr (TPR > 64) {
    constexpr int NW = TPR / 64;
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int w = 1; w < NW; ++w) v = Op::join(v, red[w]);
  }
  return v;
}

// Eight columns of h as loaded.
template <bool BF, int HQ>
struct RawH {
  u32x2 q;
  float scale;
};
template <bool BF>
struct RawH<BF, FORGE_Q_NONE> {
  Raw8<BF> r;
};
template <bool BF, int HQ, bool ODD>
__device__ __forceinline__ RawH<BF, HQ> load_h(const NormBwdArgs& a, int64_t row, int64_t at, int col, int n) {
  if constexpr (HQ == FORGE_Q_NONE) return {load_cols<BF, ODD>(a.h, at, n)};
  else return {load_codes<ODD>(static_cast<const uint8_t*>(a.h) + at, n), a.h_scale[row * ((a.D + 127) / 128) + (col >> 7)]};
}
template <bool BF, int HQ>
__device__ __forceinline__ void unpack_h(const RawH<BF, HQ>& x, float (&v)[8]) {
  if constexpr (HQ == FORGE_Q_NONE) unpack8<BF>(x.r, v);
  else decode8<HQ>(x.q, x.scale, v);
}
// One column of h.
template <bool BF, int HQ>
__device__ __forceinline__ float h1(const NormBwdArgs& a, int64_t row, int64_t c) {
  if constexpr (HQ == FORGE_Q_NONE) {
    return load1<BF>(a.h, row * a.D + c);
  } else {
    float v[8];
    decode8<HQ>(u32x2{static_cast<const uint8_t*>(a.h)[row * a.D + c], 0}, a.h_scale[row * (((int64_t)a.D + 127) / 128) + (c >> 7)], v);
    return v[0];
  }
}

// Row group u (TPR threads) takes rows u T / G .. (u + 1) T / G - 1 and writes their share of
// dgain to row u of the partial sums; dgain_kernel adds the rows in order.
template <bool BF, bool DH, bool DG, bool ODD, int TPR, int NV, int HQ>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void rmsnorm_bwd_kernel(NormBwdArgs a, int64_t groups) {
  constexpr int RPB = TPR >= 256 ? 1 : 256 / TPR;
  __shared__ float red[2][16];
  const int lane = (int)threadIdx.x % TPR, sub = (int)threadIdx.x / TPR;
  const int64_t u = (int64_t)blockIdx.x * RPB + sub;
  if (u >= groups) return;
  int64_t row = u * a.T / groups;
  const int64_t end = (u + 1) * a.T / groups;
  constexpr bool AHEAD = NV == 1;  // next row's loads in flight, gain in registers
  int in[NV];
  float gain[NV][8], acc[DG ? NV : 1][8];
  auto fetch_gain = [&](int i) {
    const int c = (lane + i * TPR) * 8;
    if (a.gain_bf16) unpack8<true>(load_cols<true, ODD>(a.gain, c, in[i]), gain[i]);
    else unpack8<false>(load_cols<false, ODD>(a.gain, c, in[i]), gain[i]);
  };
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    in[i] = cols_in((lane + i * TPR) * 8, a.D);
    if constexpr (DG)
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[i][j] = 0.0f;
    if (AHEAD && in[i]) fetch_gain(i);
  }
  Raw8<BF> rdy[NV], rdh[DH ? NV : 1];
  RawH<BF, HQ> rh[NV];
  float rs = 0.0f;
  auto fetch = [&](int64_t t) {
    rs = a.rstd[t];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!in[i]) continue;
      const int64_t at = t * a.D + (lane + i * TPR) * 8;
      rdy[i] = load_cols<BF, ODD>(a.dy, at, in[i]);
      rh[i] = load_h<BF, HQ, ODD>(a, t, at, (lane + i * TPR) * 8, in[i]);
      if constexpr (DH && AHEAD) rdh[i] = load_cols<BF, ODD>(a.dh, at, in[i]);
    }
  };
  if (AHEAD && row < end) fetch(row);
  const float inv_d = 1.0f / (float)a.D;
  for (int par = 0; row < end; ++row, par ^= 1) {
    if (!AHEAD) fetch(row);
    float dy[NV][8], h[NV][8], dh[DH ? NV : 1][8], c = 0.0f;
    const float s = rs;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!in[i]) continue;
      unpack8<BF>(rdy[i], dy[i]);
      unpack_h<BF, HQ>(rh[i], h[i]);
      if constexpr (DH && AHEAD) unpack8<BF>(rdh[i], dh[i]);
      if (!AHEAD) fetch_gain(i);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        h[i][j] *= s;
        c = __builtin_fmaf(dy[i][j] * gain[i][j], h[i][j], c);
      }
    }
    if (AHEAD && row + 1 < end) fetch(row + 1);
    c = row_reduce<Sum, TPR>(c, red[par]);
    c *= inv_d;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!in[i]) continue;
      if (!AHEAD) {
        fetch_gain(i);
        if constexpr (DH) unpack8<BF>(load_cols<BF, ODD>(a.dh, row * a.D + (lane + i * TPR) * 8, in[i]), dh[i]);
      }
      float dx[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        dx[j] = s * __builtin_fmaf(-h[i][j], c, dy[i][j] * gain[i][j]);
        if constexpr (DH) dx[j] += dh[i][j];
        if constexpr (DG) acc[i][j] = __builtin_fmaf(dy[i][j], h[i][j], acc[i][j]);
      }
      store_cols<BF, ODD>(a.dx, row * a.D + (lane + i * TPR) * 8, dx, in[i]);
    }
  }
  if constexpr (DG)
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (in[i]) store_cols<false, ODD>(a.partial, u * a.D + (lane + i * TPR) * 8, acc[i], in[i]);
}

template <bool BF, int HQ>
__global__ __launch_bounds__(256) void rmsnorm_bwd_loop_kernel(NormBwdArgs a, int64_t groups) {
  __shared__ float red[2][16];
  const int64_t u = blockIdx.x, first = u * a.T / groups, end = (u + 1) * a.T / groups;
  float* part = a.partial + u * a.D;
  if (a.dgain)
    for (int64_t c = threadIdx.x; c < a.D; c += 256) part[c] = 0.0f;
  int par = 0;
  for (int64_t row = first; row < end; ++row, par ^= 1) {
    const int64_t base = row * a.D;
    const float s = a.rstd[row];
    float sum = 0.0f;
    for (int64_t c = threadIdx.x; c < a.D; c += 256)
      sum = __builtin_fmaf(load1<BF>(a.dy, base + c) * gain1(a.gain, a.gain_bf16, c), h1<BF, HQ>(a, row, c) * s, sum);
    const float mean = row_reduce<Sum, 256>(sum, red[par]) * (1.0f / (float)a.D);
    for (int64_t c = threadIdx.x; c < a.D; c += 256) {
      const float dy = load1<BF>(a.dy, base + c), u = h1<BF, HQ>(a, row, c) * s;
      float dx = s * __builtin_fmaf(-u, mean, dy * gain1(a.gain, a.gain_bf16, c));
      if (a.dh) dx += load1<BF>(a.dh, base + c);
      store1<BF>(a.dx, base + c, dx);
      if (a.dgain) part[c] = __builtin_fmaf(dy, u, part[c]);
    }
  }
}

inline bool in_registers(int D) { return D <= 16384; }

// The backward pass holds three rows and the gain's sums besides the gain: one vector a thread
// keeps it at 5 waves a SIMD; two (1024 threads, 128 registers) fit without the next row's
// loads in flight and the gain in registers.
template <class F>
void by_width_backward(int D, F&& f) {
  using std::integral_constant;
  if (D <= 512) f(integral_constant<int, 64>{}, integral_constant<int, 1>{});
  else if (D <= 2048) f(integral_constant<int, 256>{}, integral_constant<int, 1>{});
  else if (D <= 4096) f(integral_constant<int, 512>{}, integral_constant<int, 1>{});
  else if (D <= 8192) f(integral_constant<int, 1024>{}, integral_constant<int, 1>{});
  else f(integral_constant<int, 1024>{}, integral_constant<int, 2>{});
}

template <bool BF, bool DH, bool DG, int HQ>
void backward(const NormBwdArgs& a, int64_t groups, hipStream_t st) {
  by_width_backward(a.D, [&](auto tpr, auto nv) {
    constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value;
    constexpr int RPB = TPR >= 256 ? 1 : 256 / TPR, THREADS = TPR > 256 ? TPR : 256;
    hipLaunchKernelGGL((a.D % 8 ? rmsnorm_bwd_kernel<BF, DH, DG, true, TPR, NV, HQ> : rmsnorm_bwd_kernel<BF, DH, DG, false, TPR, NV, HQ>),
                       dim3((unsigned)((groups + RPB - 1) / RPB)), dim3(THREADS), 0, st, a, groups);
  });
}

template <int HQ>
void backward_by_flags(int bf16, const NormBwdArgs& a, int64_t groups, hipStream_t st) {
  if (!in_registers(a.D)) {
    if (bf16) hipLaunchKernelGGL((rmsnorm_bwd_loop_kernel<true, HQ>), dim3((unsigned)groups), dim3(256), 0, st, a, groups);
    else hipLaunchKernelGGL((rmsnorm_bwd_loop_kernel<false, HQ>), dim3((unsigned)groups), dim3(256), 0, st, a, groups);
    return;
  }
  switch ((bf16 ? 4 : 0) + (a.dh ? 2 : 0) + (a.dgain ? 1 : 0)) {
    case 0: backward<false, false, false, HQ>(a, groups, st); break;
    case 1: backward<false, false, true, HQ>(a, groups, st); break;
    case 2: backward<false, true, false, HQ>(a, groups, st); break;
    case 3: backward<false, true, true, HQ>(a, groups, st); break;
    case 4: backward<true, false, false, HQ>(a, groups, st); break;
    case 5: backward<true, false, true, HQ>(a, groups, st); break;
    case 6: backward<true, true, false, HQ>(a, groups, st); break;
    case 7: backward<true, true, true, HQ>(a, groups, st); break;
  }
}

}  // namespace

}  // namespace forge

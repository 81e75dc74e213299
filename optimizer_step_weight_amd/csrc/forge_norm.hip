// forge_norm.hip -- RMS norm with the residual's addition and an fp8 output, and its backward.
//
// h = x + r (rounded to the stream's dtype), s = 1 / sqrt(mean(h^2) + eps), y = (h s) gain, and
// for fp8 rne(y / scale) with the row's scale amax / 448 or a given one.  Backward, with
// a = dy gain, u = h s and c = mean(a u): dx = s (a - u c) + dh, dgain = sum over rows of dy u.  No power
// of s is formed: its cube leaves fp32 for rows of an rms of 10^13 or 10^-13.
//
// Both are bound by memory: every element is read and written once.  A row is held in the
// registers of one wave (D <= 2048) or of one workgroup of 256 or 512 threads (D <= 16384), 8
// consecutive elements a thread and vector, so its two sums need no second read; a workgroup
// walks over rows with the next row's loads in flight while it works on the present one, and
// keeps its columns' gains (and in the backward pass their gradient's sum) in registers.  Rows whose
// bytes are no multiple of 16 (ODD) are loaded by the same vectors, which then straddle lines, their last
// columns one by one.  Rows that are longer take the loop kernels at the end of each part.
// Sums and statistics are fp32.  Stores are streaming ones, so that they do not displace what is yet
// to be read: 16384 x 5120 with residual to fp8 118 instead of 125 us (116 us now, 5.1 TB/s), backward of 8192 x
// 4096 47 instead of 49 us; streaming loads as well gain 2 % more there and lose 16 % on 8192 x 4096.
#include <hip/hip_runtime.h>

#include "forge_device.h"
#include "forge_layer_internal.h"
#include "forge_norm_backward.h"

namespace forge {

namespace {

// y / scale, rounded once to fp32: the product with the inverse can be a step off and lie on the other
// side of a tie between two codes, so it is corrected by its remainder (with it, the 1.2 thousand million
// quotients of every 24-bit divisor that are next to a tie of e4m3 all equal the division's).  Two
// operations an element; the division's own sequence would take 5 to 14 % of the kernel's time.
// Factors of 2 keep the inverse and the remainder in range.
struct Divisor {
  float m, s, inv, most;
  __device__ __forceinline__ explicit Divisor(float scale) {
    const float mag = fabsf(scale);
    m = mag < 0x1p-70f ? 0x1p80f : mag > 0x1p100f ? 0x1p-64f : 1.0f;
    s = scale * m;
    inv = 1.0f / s;
    most = kFp8Max * fabsf(s);
    if (isinf(s)) s = 0.0f;  // finite ones give zero, infinite ones NaN
  }
};

// The quotient y / (scale m), clamped to the fp8 range; NaN stays.  The clamp comes first, so that what is
// divided is 448 scale at most, and the quotient a step over 448 at most, which the conversion rounds to 448.
// By the row's own scale nothing is larger.
template <bool ROW>
__device__ __forceinline__ float quotient8(float y, const Divisor& d) {
  if constexpr (!ROW) y = __builtin_elementwise_maximum(__builtin_elementwise_minimum(y, d.most), -d.most);
  const float q = y * d.inv, r = __builtin_fmaf(q, d.s, -y);
  return __builtin_fmaf(-r, d.inv, q);
}

// Raises *amax to v (both non-negative or NaN: the bits order as unsigned integers, NaN above
// all).  The plain read spares most calls the atomic; a stale one only costs it.
__device__ __forceinline__ void raise_amax(float* amax, float v) {
  const uint32_t u = __float_as_uint(v) & 0x7FFFFFFFu;
  if (u > *reinterpret_cast<volatile uint32_t*>(amax)) atomicMax(reinterpret_cast<uint32_t*>(amax), u);
}

// ------------------------------------------------------------------ forward
template <bool BF, bool RES, bool ODD, int YT, int TPR, int NV>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void rmsnorm_kernel(NormArgs a) {
  constexpr int RPB = TPR >= 256 ? 1 : 256 / TPR;  // rows at a time
  __shared__ float red[2][2][8];                   // by row parity and use: one barrier a reduction
  const int lane = (int)threadIdx.x % TPR, sub = (int)threadIdx.x / TPR;
  const int64_t step = (int64_t)gridDim.x * RPB;
  int64_t row = (int64_t)blockIdx.x * RPB + sub;
  if (row >= a.T) return;  // a whole row's threads; with TPR > 64 a whole workgroup
  int in[NV];  // columns of the row in this thread's vector: 0 or 8, or the last few (ODD)
  float gain[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (lane + i * TPR) * 8;
    in[i] = cols_in(c, a.D);
    if (!in[i]) continue;
    if (a.gain_bf16) unpack8<true>(load_cols<true, ODD>(a.gain, c, in[i]), gain[i]);
    else unpack8<false>(load_cols<false, ODD>(a.gain, c, in[i]), gain[i]);
  }
  Raw8<BF> x[NV], r[RES ? NV : 1];
  auto fetch = [&](int64_t t) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!in[i]) continue;
      const int64_t at = t * a.D + (lane + i * TPR) * 8;
      x[i] = load_cols<BF, ODD>(a.x, at, in[i]);
      if constexpr (RES) r[i] = load_cols<BF, ODD>(a.res, at, in[i]);
    }
  };
  fetch(row);
  const float inv_d = 1.0f / (float)a.D;
  float top = 0.0f;
  for (int par = 0; row < a.T; row += step, par ^= 1) {
    float v[NV][8], ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!in[i]) continue;
      unpack8<BF>(x[i], v[i]);
      if constexpr (RES) {
        float w[8];
        unpack8<BF>(r[i], w);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = round_to<BF>(v[i][j] + w[j]);
        store_cols<BF, ODD>(a.h, row * a.D + (lane + i * TPR) * 8, v[i], in[i]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = __builtin_fmaf(v[i][j], v[i][j], ss);
    }
    if (row + step < a.T) fetch(row + step);
    ss = row_reduce<Sum, TPR>(ss, red[par][0]);
    const float s = 1.0f / sqrtf(__builtin_fmaf(ss, inv_d, a.eps));
    if (a.rstd && lane == 0) a.rstd[row] = s;
    float mx = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!in[i]) continue;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[i][j] = (v[i][j] * s) * gain[i][j];
        if (!ODD || j < in[i]) mx = amax2(mx, fabsf(v[i][j]));
      }
    }
    float scale = 1.0f;
    if constexpr (YT == FORGE_Y_FP8_ROW) {
      mx = row_reduce<Max, TPR>(mx, red[par][1]);
      scale = mx / kFp8Max;
      scale = scale < kScaleMin ? kScaleMin : scale;
      if (lane == 0) a.y_scale[row] = scale;
    } else if constexpr (YT == FORGE_Y_FP8_TENSOR) {
      scale = a.y_scale[0];
    }
    top = amax2(top, mx);
    const Divisor d(scale);
    // a wave has one row, and a row one scale
    if (YT != FORGE_Y_F32 && YT != FORGE_Y_BF16 && __builtin_amdgcn_readfirstlane(__float_as_int(d.m)) != 0x3F800000)
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] *= d.m;
    auto code = [&](float y) { return quotient8<YT == FORGE_Y_FP8_ROW>(y, d); };
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!in[i]) continue;
      const int64_t at = row * a.D + (lane + i * TPR) * 8;
      if constexpr (YT == FORGE_Y_F32 || YT == FORGE_Y_BF16) {
        store_cols<YT == FORGE_Y_BF16, ODD>(a.y, at, v[i], in[i]);
      } else {
        u32x2 q;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          int w = 0;
          w = __builtin_amdgcn_cvt_pk_fp8_f32(code(v[i][4 * j]), code(v[i][4 * j + 1]), w, false);
          w = __builtin_amdgcn_cvt_pk_fp8_f32(code(v[i][4 * j + 2]), code(v[i][4 * j + 3]), w, true);
          q[j] = (uint32_t)w;
        }
        uint8_t* y = static_cast<uint8_t*>(a.y) + at;
        if constexpr (!ODD) {
          __builtin_nontemporal_store(q, reinterpret_cast<u32x2*>(y));
        } else if (in[i] == 8) {
          *reinterpret_cast<u32x2u*>(y) = q;
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j < in[i]) y[j] = (uint8_t)(q[j >> 2] >> (8 * (j & 3)));
        }
      }
    }
  }
  if (a.amax) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) top = amax2(top, __shfl_xor(top, o));
    if ((threadIdx.x & 63) == 0) raise_amax(a.amax, top);
  }
}

// Rows too long for registers: one workgroup a row, the row read again for each pass (every thread
// its own columns).
template <bool BF, int YT>
__global__ __launch_bounds__(256) void rmsnorm_loop_kernel(NormArgs a) {
  __shared__ float red[2][16];
  const int64_t base = (int64_t)blockIdx.x * a.D;
  const void* hp = a.res ? a.h : a.x;
  float ss = 0.0f;
  for (int64_t c = threadIdx.x; c < a.D; c += 256) {
    float v = load1<BF>(a.x, base + c);
    if (a.res) {
      v = round_to<BF>(v + load1<BF>(a.res, base + c));
      store1<BF>(a.h, base + c, v);
    }
    ss = __builtin_fmaf(v, v, ss);
  }
  ss = row_reduce<Sum, 256>(ss, red[0]);
  const float s = 1.0f / sqrtf(__builtin_fmaf(ss, 1.0f / (float)a.D, a.eps));
  if (a.rstd && threadIdx.x == 0) a.rstd[blockIdx.x] = s;
  auto y_at = [&](int64_t c) { return (load1<BF>(hp, base + c) * s) * gain1(a.gain, a.gain_bf16, c); };
  float mx = 0.0f, scale = 1.0f;
  if (YT == FORGE_Y_FP8_ROW || a.amax) {
    for (int64_t c = threadIdx.x; c < a.D; c += 256) mx = amax2(mx, fabsf(y_at(c)));
    mx = row_reduce<Max, 256>(mx, red[1]);
    if (a.amax && threadIdx.x == 0) raise_amax(a.amax, mx);
  }
  if constexpr (YT == FORGE_Y_FP8_ROW) {
    scale = mx / kFp8Max;
    scale = scale < kScaleMin ? kScaleMin : scale;
    if (threadIdx.x == 0) a.y_scale[blockIdx.x] = scale;
  } else if constexpr (YT == FORGE_Y_FP8_TENSOR) {
    scale = a.y_scale[0];
  }
  const Divisor d(scale);
  for (int64_t c = threadIdx.x; c < a.D; c += 256) {
    const float y = y_at(c);
    if constexpr (YT == FORGE_Y_F32 || YT == FORGE_Y_BF16) {
      store1<YT == FORGE_Y_BF16>(a.y, base + c, y);
    } else {
      const int w = __builtin_amdgcn_cvt_pk_fp8_f32(quotient8<YT == FORGE_Y_FP8_ROW>(y * d.m, d), 0.0f, 0, false);
      static_cast<uint8_t*>(a.y)[base + c] = (uint8_t)(w & 0xFF);
    }
  }
}

// dgain[c] = sum over the groups' partial rows, in a fixed order: thread (x, y) of 32 x 16 adds
// rows y, y + 16, ..., then the 16 sums are added in order.  A workgroup takes 32 columns, and further
// ones where D has more than a grid may (2^32 threads).
constexpr int kGainBlocks = 1 << 16;
__global__ __launch_bounds__(512) void dgain_kernel(const float* partial, float* dgain, int64_t groups, int64_t D) {
  __shared__ float part[16][33];
  const int x = (int)threadIdx.x & 31, y = (int)threadIdx.x >> 5;
  for (int64_t c0 = (int64_t)blockIdx.x * 32; c0 < D; c0 += (int64_t)kGainBlocks * 32) {
    const int64_t c = c0 + x;
    float s = 0.0f;
    if (c < D) {
#pragma unroll 8
      for (int64_t g = y; g < groups; g += 16) s += partial[g * D + c];
    }
    part[y][x] = s;
    __syncthreads();
    if (y == 0 && c < D) {
#pragma unroll
      for (int i = 1; i < 16; ++i) s += part[i][x];
      dgain[c] = s;
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------ dispatch
// f(threads of a row, vectors of a thread): the least that holds D.
template <class F>
void by_width(int D, F&& f) {
  using std::integral_constant;
  if (D <= 512) f(integral_constant<int, 64>{}, integral_constant<int, 1>{});
  else if (D <= 1024) f(integral_constant<int, 64>{}, integral_constant<int, 2>{});
  else if (D <= 2048) f(integral_constant<int, 64>{}, integral_constant<int, 4>{});
  else if (D <= 4096) f(integral_constant<int, 256>{}, integral_constant<int, 2>{});
  else if (D <= 6144) f(integral_constant<int, 256>{}, integral_constant<int, 3>{});
  else if (D <= 8192) f(integral_constant<int, 256>{}, integral_constant<int, 4>{});
  else f(integral_constant<int, 512>{}, integral_constant<int, 4>{});
}

template <bool BF, int YT>
void forward(const NormArgs& a, hipStream_t st) {
  if (!in_registers(a.D)) {
    hipLaunchKernelGGL((rmsnorm_loop_kernel<BF, YT>), dim3((unsigned)a.T), dim3(256), 0, st, a);
    return;
  }
  by_width(a.D, [&](auto tpr, auto nv) {
    constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value;
    constexpr int RPB = TPR >= 256 ? 1 : 256 / TPR, THREADS = TPR > 256 ? TPR : 256;
    const int64_t blocks = (a.T + RPB - 1) / RPB;
    const unsigned grid = (unsigned)(blocks < kNormBlocks ? blocks : kNormBlocks);
    auto launch = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(grid), dim3(THREADS), 0, st, a); };
    if (a.D % 8) launch(a.res ? rmsnorm_kernel<BF, true, true, YT, TPR, NV> : rmsnorm_kernel<BF, false, true, YT, TPR, NV>);
    else launch(a.res ? rmsnorm_kernel<BF, true, false, YT, TPR, NV> : rmsnorm_kernel<BF, false, false, YT, TPR, NV>);
  });
}

}  // namespace

int launch_rmsnorm(int x_bf16, int y_type, const NormArgs& a, void* stream) {
  hipStream_t st = (hipStream_t)stream;
  switch (y_type * 2 + (x_bf16 ? 1 : 0)) {
    case FORGE_Y_F32 * 2: forward<false, FORGE_Y_F32>(a, st); break;
    case FORGE_Y_F32 * 2 + 1: forward<true, FORGE_Y_F32>(a, st); break;
    case FORGE_Y_BF16 * 2: forward<false, FORGE_Y_BF16>(a, st); break;
    case FORGE_Y_BF16 * 2 + 1: forward<true, FORGE_Y_BF16>(a, st); break;
    case FORGE_Y_FP8_ROW * 2: forward<false, FORGE_Y_FP8_ROW>(a, st); break;
    case FORGE_Y_FP8_ROW * 2 + 1: forward<true, FORGE_Y_FP8_ROW>(a, st); break;
    case FORGE_Y_FP8_TENSOR * 2: forward<false, FORGE_Y_FP8_TENSOR>(a, st); break;
    case FORGE_Y_FP8_TENSOR * 2 + 1: forward<true, FORGE_Y_FP8_TENSOR>(a, st); break;
    default: return (int)hipErrorInvalidValue;
  }
  return (int)hipGetLastError();
}

int launch_rmsnorm_backward(int bf16, const NormBwdArgs& a, void* stream) {
  hipStream_t st = (hipStream_t)stream;
  const int64_t groups = norm_bwd_groups(a.T);
  if (a.h_q != FORGE_Q_NONE) launch_rmsnorm_backward_q8(bf16, a, groups, stream);
  else backward_by_flags<FORGE_Q_NONE>(bf16, a, groups, st);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess || !a.dgain) return (int)err;
  const int64_t blocks = ((int64_t)a.D + 31) / 32;
  hipLaunchKernelGGL(dgain_kernel, dim3((unsigned)(blocks < kGainBlocks ? blocks : kGainBlocks)), dim3(512), 0, st, a.partial,
                     a.dgain, groups, (int64_t)a.D);
  return (int)hipGetLastError();
}

}  // namespace forge

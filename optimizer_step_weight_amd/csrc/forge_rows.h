// forge_rows.h -- eight consecutive elements of a row: loads and stores from any alignment, and the
// 8-bit codes of blocks of 128 columns.
#pragma once

#include <hip/hip_runtime.h>

#include "forge_device.h"
#include "forge_layer_internal.h"

namespace forge {

constexpr float kFp8Max = 448.0f;
constexpr float kScaleMin = 1.17549435e-38f;  // 2^-126: keeps 1 / scale finite

// 8 consecutive elements as loaded.
template <bool BF>
struct Raw8 {
  u32x4 q[BF ? 1 : 2];
};
template <bool BF>
__device__ __forceinline__ Raw8<BF> load8(const void* p, int64_t i) {
  Raw8<BF> r;
  if constexpr (BF) {
    r.q[0] = ld16(static_cast<const uint16_t*>(p) + i);
  } else {
    r.q[0] = ld16(static_cast<const float*>(p) + i);
    r.q[1] = ld16(static_cast<const float*>(p) + i + 4);
  }
  return r;
}
template <bool BF>
__device__ __forceinline__ void unpack8(const Raw8<BF>& r, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if constexpr (BF) v[j] = (j & 1) ? __uint_as_float(r.q[0][j >> 1] & 0xFFFF0000u) : __uint_as_float(r.q[0][j >> 1] << 16);
    else v[j] = __uint_as_float(r.q[j >> 2][j & 3]);
  }
}
template <bool BF>
__device__ __forceinline__ void store8(void* p, int64_t i, const float (&v)[8]) {
  if constexpr (BF) {
    u32x4 q;
#pragma unroll
    for (int j = 0; j < 4; ++j) q[j] = f32_to_bf16_rne(v[2 * j]) | (f32_to_bf16_rne(v[2 * j + 1]) << 16);
    __builtin_nontemporal_store(q, reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p) + i));
  } else {
    u32x4 a, b;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      a[j] = __float_as_uint(v[j]);
      b[j] = __float_as_uint(v[4 + j]);
    }
    st16(static_cast<float*>(p) + i, a);
    st16(static_cast<float*>(p) + i + 4, b);
  }
}
// The same from any alignment, and n < 8 elements one by one (the others are 0): rows whose bytes are
// no multiple of 16.
typedef uint32_t u32x4u __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2u __attribute__((ext_vector_type(2), aligned(1)));
template <bool BF>
__device__ __forceinline__ Raw8<BF> load_any(const void* p, int64_t i, int n) {
  Raw8<BF> r;
  const int64_t at = i * (BF ? 2 : 4);
  const char* b = static_cast<const char*>(p) + at;
  if (n == 8) {
    r.q[0] = *reinterpret_cast<const u32x4u*>(b);
    if constexpr (!BF) r.q[1] = *reinterpret_cast<const u32x4u*>(b + 16);
    return r;
  }
  uint32_t v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j)
    v[j] = j >= n ? 0u : BF ? (uint32_t)reinterpret_cast<const uint16_t*>(b)[j] : reinterpret_cast<const uint32_t*>(b)[j];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (BF) r.q[0][j] = v[2 * j] | (v[2 * j + 1] << 16);
    else {
      r.q[0][j] = v[j];
      r.q[1][j] = v[4 + j];
    }
  }
  return r;
}
template <bool BF>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  if constexpr (BF) return bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
  else return static_cast<const float*>(p)[i];
}
template <bool BF>
__device__ __forceinline__ void store1(void* p, int64_t i, float v) {
  if constexpr (BF) static_cast<uint16_t*>(p)[i] = (uint16_t)f32_to_bf16_rne(v);
  else static_cast<float*>(p)[i] = v;
}
__device__ __forceinline__ float gain1(const void* p, int bf, int64_t i) {
  return bf ? load1<true>(p, i) : load1<false>(p, i);
}
template <bool BF>
__device__ __forceinline__ float round_to(float v) {
  if constexpr (BF) return bf16_to_f32(f32_to_bf16_rne(v));
  else return v;
}

template <bool BF>
__device__ __forceinline__ void store_any(void* p, int64_t i, const float (&v)[8], int n) {
  char* b = static_cast<char*>(p) + i * (BF ? 2 : 4);
  if (n == 8) {
    u32x4 q[BF ? 1 : 2];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (BF) q[0][j] = f32_to_bf16_rne(v[2 * j]) | (f32_to_bf16_rne(v[2 * j + 1]) << 16);
      else {
        q[0][j] = __float_as_uint(v[j]);
        q[1][j] = __float_as_uint(v[4 + j]);
      }
    }
    *reinterpret_cast<u32x4u*>(b) = q[0];
    if constexpr (!BF) *reinterpret_cast<u32x4u*>(b + 16) = q[1];
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < n) store1<BF>(b, j, v[j]);
}

// A thread's 8 columns of a row, n of them in the row (ODD: the row's bytes are no multiple of 16).
template <bool BF, bool ODD>
__device__ __forceinline__ Raw8<BF> load_cols(const void* p, int64_t i, int n) {
  if constexpr (ODD) return load_any<BF>(p, i, n);
  else return load8<BF>(p, i);
}
template <bool BF, bool ODD>
__device__ __forceinline__ void store_cols(void* p, int64_t i, const float (&v)[8], int n) {
  if constexpr (ODD) store_any<BF>(p, i, v, n);
  else store8<BF>(p, i, v);
}
__device__ __forceinline__ int cols_in(int c, int D) { return D - c < 0 ? 0 : D - c > 8 ? 8 : D - c; }

// Larger of two magnitudes; NaN wins.
__device__ __forceinline__ float amax2(float a, float b) { return (a > b || a != a) ? a : b; }

// ------------------------------------------------------------------ 8-bit blocks of 128 columns
// value = code * scale with one fp32 scale for each 128 consecutive columns of a row:
//   scale = max(amax / most, 2^-126), code = rne(x * (1 / scale)), both quotients rounded to fp32;
// most is 448 (e4m3) or 127 (int8).  The product is at most 1.5 steps of fp32 above `most`, which
// either rounding takes back to it.  A block that holds NaN or an infinity gets a NaN scale and zero
// codes: all of it reads back as NaN.
//
// Magnitudes are compared as bits, where NaN is above infinity and that above all else.  The quotients are
// the divisions' own, in 3 operations each: a product with the inverse, corrected by its remainder (compared
// with the division for every fp32 amax of either `most`, and every scale up to 2^121).
__device__ __forceinline__ uint32_t mag_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
template <int N>
__device__ __forceinline__ uint32_t amax_bits(const float (&v)[N]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) m = umax(m, mag_bits(v[i]));
  return m;
}
template <int Q>
__device__ __forceinline__ float block_scale(uint32_t amax) {
  if (amax >= 0x7F800000u) return __uint_as_float(0x7FC00000u);
  constexpr float most = Q == FORGE_Q_FP8 ? kFp8Max : 127.0f, inv = 1.0f / most;
  const float x = __uint_as_float(amax), q = x * inv, s = __builtin_fmaf(__builtin_fmaf(-q, most, x), inv, q);
  return s < kScaleMin ? kScaleMin : s;
}
__device__ __forceinline__ float inverse(float scale) {
  const float y = __builtin_amdgcn_rcpf(scale);
  return __builtin_fmaf(__builtin_fmaf(-scale, y, 1.0f), y, y);
}
// Codes of 4 values, by the inverse of their scale.
template <int Q>
__device__ __forceinline__ uint32_t encode4(const float* v, float inv) {
  if constexpr (Q == FORGE_Q_FP8) {
    int w = 0;
    w = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * inv, v[1] * inv, w, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[2] * inv, v[3] * inv, w, true);
  } else {
    // x + 1.5 * 2^23 rounds x to a whole number, whose low byte is the sum's
    uint32_t b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = __float_as_uint(v[i] * inv + 12582912.0f);
    const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0C0C0400u), hi = __builtin_amdgcn_perm(b[3], b[2], 0x04000C0Cu);
    return lo | hi;
  }
}
// Codes of N values by their block's scale.
template <int Q, int N>
__device__ __forceinline__ void encode(const float (&v)[N], float scale, uint32_t (&q)[N / 4]) {
  const float inv = inverse(scale);
  const bool bad = scale != scale;
#pragma unroll
  for (int j = 0; j < N / 4; ++j) q[j] = bad ? 0u : encode4<Q>(v + 4 * j, inv);
}
template <int Q>
__device__ __forceinline__ u32x2 encode8(const float (&v)[8], float scale) {
  uint32_t q[2];
  encode<Q>(v, scale, q);
  return u32x2{q[0], q[1]};
}
template <int Q>
__device__ __forceinline__ void decode8(u32x2 q, float scale, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    if constexpr (Q == FORGE_Q_FP8) {
      const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[j], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[j], true);
      v[4 * j] = lo[0] * scale;
      v[4 * j + 1] = lo[1] * scale;
      v[4 * j + 2] = hi[0] * scale;
      v[4 * j + 3] = hi[1] * scale;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[4 * j + i] = (float)(int8_t)(q[j] >> (8 * i)) * scale;
    }
  }
}
// Eight codes from any address, n < 8 of them one by one (the others are 0), and back.
template <bool ODD>
__device__ __forceinline__ u32x2 load_codes(const uint8_t* p, int n) {
  if constexpr (!ODD) return *reinterpret_cast<const u32x2*>(p);
  if (n == 8) return *reinterpret_cast<const u32x2u*>(p);
  u32x2 q = {0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < n) q[j >> 2] |= (uint32_t)p[j] << (8 * (j & 3));
  return q;
}
template <bool ODD>
__device__ __forceinline__ void store_codes(uint8_t* p, u32x2 q, int n) {
  if constexpr (!ODD) {
    __builtin_nontemporal_store(q, reinterpret_cast<u32x2*>(p));
  } else if (n == 8) {
    *reinterpret_cast<u32x2u*>(p) = q;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) p[j] = (uint8_t)(q[j >> 2] >> (8 * (j & 3)));
  }
}
// The largest over each 8, or 16, consecutive lanes, in all of them.
__device__ __forceinline__ uint32_t max8(uint32_t v) {
  v = umax(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xf, 0xf, false));   // 1 0 3 2 of each four
  v = umax(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xf, 0xf, false));   // 2 3 0 1
  return umax(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xf, 0xf, false));  // 7 .. 0 of each eight
}
__device__ __forceinline__ uint32_t max16(uint32_t v) {
  v = max8(v);
  return umax(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xf, 0xf, false));  // 15 .. 0 of each sixteen
}

}  // namespace forge

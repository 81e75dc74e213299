// forge_multi.hip -- the optimizer's step of many tensors in one launch, from materialised
// gradients: the element-wise rules of the fused step (forge_device.h) for parameters of any
// size.
//
// Bound by memory: every gradient is read once, every weight and moment read and written once
// (26 bytes an element for fp32 weights and moments with bf16 gradients).  A workgroup updates
// one chunk of 4096 consecutive elements of one tensor; the table's owner word names the tensor,
// so that no workgroup searches for it.  Within a chunk the layouts are those of the unfused
// optimizer kernel: fp32 moments in 4-element units with consecutive lanes on consecutive units,
// all of a thread's four units in flight; 8-bit moments in 16-element segments, four lanes to a
// block of 64.  Elements past the last whole unit (n mod 4) or block (n mod 64) are updated by
// one wave, a lane to an element.
//
// Measured, over the cards seen: 120 tensors of 1000 .. 20 M elements in fp32 with bf16 gradients 1.12-1.24 ms
// (5.3-5.8 TB/s; a large copy: 4.75), 40 of 4096 .. 50 M in bf16 with 8-bit moments in the linear map 0.45 ms (5.3), in
// the dynamic map, whose codes take many more operations, 1.0 ms; 65 gains of 256 .. 5120 elements 4.4 us.  Chunks of 4096 elements keep every workgroup's loads in flight at once.
#include <hip/hip_runtime.h>

#include "forge_device.h"
#include "forge_layer_internal.h"
#include "forge_paths.h"

namespace forge {

namespace {

constexpr int kMultiThreads = 256;

// 4 gradients at element i (a multiple of 4), times the gradient scale.
__device__ __forceinline__ void grad4(float (&g)[4], const MultiEntry& t, uint32_t i, float gs) {
  if (t.g_bf16) {
    const u32x2 q = ld8(static_cast<const uint16_t*>(t.g) + i);
    g[0] = __uint_as_float(q.x << 16) * gs;
    g[1] = __uint_as_float(q.x & 0xFFFF0000u) * gs;
    g[2] = __uint_as_float(q.y << 16) * gs;
    g[3] = __uint_as_float(q.y & 0xFFFF0000u) * gs;
  } else {
    const u32x4 q = ld16(static_cast<const float*>(t.g) + i);
#pragma unroll
    for (int c = 0; c < 4; ++c) g[c] = __uint_as_float(q[c]) * gs;
  }
}

// Whole units and blocks of the chunk at `base`.
template <int WT, int ST, int OPT>
__device__ __forceinline__ void chunk_body(const MultiEntry& t, uint32_t base, const EpiArgs& e, float gs) {
  if constexpr (ST == FORGE_S_F32) {
    const int lane = (int)(threadIdx.x & 63);
    const uint32_t first = base + (threadIdx.x >> 6) * 1024u;
    const uint32_t whole = t.n & ~3u;
    uint32_t i[4];
    bool in[4];
    UnitIn x[4];
    float g[4][4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      i[r] = first + 256u * r + 4u * lane;   // n < 2^32 - 4096: no wrap
      in[r] = i[r] < whole;
      if (!in[r]) continue;
      grad4(g[r], t, i[r], gs);
      unit_load<OPT, WT, ST>(x[r], i[r], e);
    }
    uint64_t w[4] = {0ull, 0ull, 0ull, 0ull};
    if (WT == FORGE_W_BF16 && e.sr) sr_words4(i, e, w);  // by whole quads, in range or not
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (in[r]) unit_apply<OPT, WT, ST>(g[r], i[r], x[r], w[r], e);
  } else {
    const uint32_t i0 = base + threadIdx.x * 16u;
    if (i0 < (t.n & ~63u)) {  // the four lanes of a block together
      float g[16];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float h[4];
        grad4(h, t, i0 + 4 * q, gs);
#pragma unroll
        for (int c = 0; c < 4; ++c) g[4 * q + c] = h[c];
      }
      step_segment16<OPT, WT, ST>(g, i0, e);
    }
  }
}

// The elements [first, n), fewer than 64 of them, first a multiple of 4 (fp32 moments) or 64
// (8-bit: they are the tensor's last, short block): one wave, a lane to an element.
template <int WT, int ST, int OPT>
__device__ __forceinline__ void chunk_tail(const MultiEntry& t, uint32_t first, const EpiArgs& e, float gs) {
  constexpr bool HM = RuleStates<OPT>::m, HV = RuleStates<OPT>::v, DYN = ST == FORGE_S_Q8D;
  const uint32_t lane = threadIdx.x & 63u, i = first + lane, blk = first >> 6;
  const bool in = i < t.n;
  float g = 0.0f, w = 0.0f, m = 0.0f, v = 0.0f;
  if (in) {
    g = (t.g_bf16 ? bf16_to_f32(static_cast<const uint16_t*>(t.g)[i]) : static_cast<const float*>(t.g)[i]) * gs;
    w = WT == FORGE_W_BF16 ? bf16_to_f32(static_cast<const uint16_t*>(e.W)[i]) : static_cast<const float*>(e.W)[i];
    if constexpr (ST == FORGE_S_F32) {
      if (HM) m = static_cast<const float*>(e.m)[i];
      if (HV) v = static_cast<const float*>(e.v)[i];
    } else {
      if (HM) m = dequant8<true, DYN>(static_cast<const uint8_t*>(e.m)[i], e.m_scale[blk]);
      if (HV) v = dequant8<false, DYN>(static_cast<const uint8_t*>(e.v)[i], e.v_scale[blk]);
    }
  }
  const float wn = rule<OPT>(g, w, m, v, e.s);
  if (in) {
    if constexpr (WT == FORGE_W_BF16) {
      uint32_t q;
      if (e.sr) {
        const U64x4 o = philox4x64_10((uint64_t)(i >> 4), e.step, 0ull, 0ull, e.seed, 0ull);
        q = f32_to_bf16_sr(wn, (uint32_t)(pick4(o, (int)((i & 15u) >> 2)) >> (16 * (i & 3u))) & 0xFFFFu);
      } else {
        q = f32_to_bf16_rne(wn);
      }
      static_cast<uint16_t*>(e.W)[i] = (uint16_t)q;
    } else {
      static_cast<float*>(e.W)[i] = wn;
    }
  }
  if constexpr (ST == FORGE_S_F32) {
    if (HM && in) static_cast<float*>(e.m)[i] = m;
    if (HV && in) static_cast<float*>(e.v)[i] = v;
  } else {
    if constexpr (HM) {
      const float x[1] = {in ? m : 0.0f};
      uint32_t code[1];
      const float scale = quant_block64<true, DYN, 1, 64>(x, code);
      if (in) static_cast<uint8_t*>(e.m)[i] = (uint8_t)code[0];
      if (lane == 0) e.m_scale[blk] = scale;
    }
    if constexpr (HV) {
      const float x[1] = {in ? v : 0.0f};
      uint32_t code[1];
      const float scale = quant_block64<false, DYN, 1, 64>(x, code);
      if (in) static_cast<uint8_t*>(e.v)[i] = (uint8_t)code[0];
      if (lane == 0) e.v_scale[blk] = scale;
    }
  }
}

template <int ST, int OPT>
__global__ __launch_bounds__(kMultiThreads) void multi_step_kernel(MultiArgs a) {
  const MultiEntry t = a.entries[a.owner[blockIdx.x]];
  const uint32_t base = (blockIdx.x - t.chunk0) * (uint32_t)kMultiChunk;
  EpiArgs e;
  e.W = t.W;
  e.m = t.m;
  e.v = t.v;
  e.m_scale = t.m_scale;
  e.v_scale = t.v_scale;
  e.w_pre = nullptr;
  e.seed = t.seed;
  e.step = a.step;
  e.sr = a.sr;
  e.s = a.s[t.group];
  const float gs = a.grad_scale ? a.grad_scale[0] : 1.0f;
  const uint32_t tail = ST == FORGE_S_F32 ? (t.n & ~3u) : (t.n & ~63u);
  const bool mine = tail < t.n && tail >= base && tail - base < (uint32_t)kMultiChunk && threadIdx.x < 64;
  if (t.w_bf16) {
    chunk_body<FORGE_W_BF16, ST, OPT>(t, base, e, gs);
    if (mine) chunk_tail<FORGE_W_BF16, ST, OPT>(t, tail, e, gs);
  } else {
    chunk_body<FORGE_W_F32, ST, OPT>(t, base, e, gs);
    if (mine) chunk_tail<FORGE_W_F32, ST, OPT>(t, tail, e, gs);
  }
}

using MultiFn = void (*)(MultiArgs);
template <int ST>
MultiFn multi_for(int opt) {
  switch (opt) {
#define FORGE_CASE(O) \
  case O: return multi_step_kernel<ST, O>;
    FORGE_FOR_EACH_OPT(FORGE_CASE)
#undef FORGE_CASE
  }
  return nullptr;
}

}  // namespace

int launch_multi_step(int s_type, int opt, const MultiArgs& a, int64_t chunks, void* stream) {
  MultiFn fn = s_type == FORGE_S_F32  ? multi_for<FORGE_S_F32>(opt)
               : s_type == FORGE_S_Q8 ? multi_for<FORGE_S_Q8>(opt)
                                      : multi_for<FORGE_S_Q8D>(opt);
  if (!fn) return (int)hipErrorInvalidValue;
  hipLaunchKernelGGL(fn, dim3((unsigned)chunks), dim3(kMultiThreads), 0, (hipStream_t)stream, a);
  return (int)hipGetLastError();
}

}  // namespace forge

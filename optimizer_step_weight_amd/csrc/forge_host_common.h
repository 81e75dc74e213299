// forge_host_common.h -- argument checks and per-step scalars shared by the translation units of
// the C ABI (defined in forge_host.cpp).  They run before any HIP call; `fail` keeps the text
// that forge_last_error() returns.
#pragma once

#include <stdint.h>

#include "forge.h"
#include "forge_internal.h"

namespace forge {
namespace host {

void clear_error();
forge_status fail(forge_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));

struct Range {
  uintptr_t lo = 0, hi = 0;  // [lo, hi)
  const char* name = "";
};
Range range_of(const void* p, int64_t bytes, const char* name);
inline bool overlap(const Range& a, const Range& b) {
  return a.lo < b.hi && b.lo < a.hi && a.hi > a.lo && b.hi > b.lo;
}
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

int64_t dtype_size(int32_t dt);  // 0 for an unknown dtype
bool rule_has_m(int32_t opt);
bool rule_has_v(int32_t opt);
forge_status check_tensor(const forge_tensor* t, const char* name);
int64_t bytes_of(const forge_tensor* t);
forge_status device_ok();
forge_status to_status(int herr);

forge_status compute_scalars(int32_t opt, const forge_hyper* h, int64_t step, forge::OptScalars* out);

struct StepPlan {
  int w_type = 0, s_type = 0;
  forge::EpiArgs e{};
};
// Checks W [N, K], its moments, the rule and its scalars; outs receives the written ranges
// (at most 6).
forge_status validate_step_outputs(int64_t N, int64_t K, forge_tensor* W, forge_tensor* m, forge_tensor* v,
                                   const forge_hyper* hyper, int32_t opt, int64_t step, uint64_t seed,
                                   const forge_step_opts* opts, StepPlan* plan, Range* outs, int* n_outs);

}  // namespace host
}  // namespace forge

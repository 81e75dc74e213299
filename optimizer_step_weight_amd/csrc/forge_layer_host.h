// forge_layer_host.h -- argument checks shared by the entry points of forge_layer.h and forge_ffn.h.
#pragma once

#include "forge_host_common.h"

namespace forge {
namespace host {

// Ranges of one call: written ones overlap nothing, except pairs named as allowed in place.
struct Ranges {
  Range r[16];
  bool written[16];
  int n = 0;
  void add(const void* p, int64_t bytes, const char* name, bool w) {
    r[n] = range_of(p, bytes, name);
    written[n++] = w;
  }
  void add(const forge_tensor* t, const char* name, bool w) { add(t->data, bytes_of(t), name, w); }
  // may: written range i may be exactly range j
  template <class May>
  forge_status check(May&& may) const {
    for (int i = 0; i < n; ++i)
      for (int j = 0; j < n; ++j) {
        if (i == j || !written[i] || (written[j] && j < i)) continue;
        if (!overlap(r[i], r[j])) continue;
        if (r[i].lo == r[j].lo && r[i].hi == r[j].hi && may(r[i].name, r[j].name)) continue;
        return fail(FORGE_ERR_ALIAS, "%s overlaps %s", r[i].name, r[j].name);
      }
    return FORGE_OK;
  }
};
inline bool never(const char*, const char*) { return false; }

inline bool is_stream(int32_t dt) { return dt == FORGE_F32 || dt == FORGE_BF16; }

inline forge_status check_shape(const forge_tensor* t, int64_t rows, int64_t cols, const char* name) {
  if (t->rows != rows || t->cols != cols)
    return fail(FORGE_ERR_SHAPE, "%s is [%lld, %lld], expected [%lld, %lld]", name, (long long)t->rows,
                (long long)t->cols, (long long)rows, (long long)cols);
  return FORGE_OK;
}


inline forge_status check_groups(const int32_t* ends, int32_t n_groups, int64_t T, int64_t N, int64_t K) {
  if (n_groups < 1 || n_groups > 4096) return fail(FORGE_ERR_ARG, "n_groups must be 1 .. 4096 (got %d)", (int)n_groups);
  if (!ends) return fail(FORGE_ERR_ARG, "ends is NULL");
  if (!aligned4(ends)) return fail(FORGE_ERR_LAYOUT, "ends is not 4-byte aligned");
  if (N < 128 || K < 128 || N % 128 || K % 128)
    return fail(FORGE_ERR_SHAPE, "N = %lld and K = %lld must be positive multiples of 128", (long long)N, (long long)K);
  if (N > (1 << 20) || K > (1 << 20) || N * K >= (int64_t(1) << 31))
    return fail(FORGE_ERR_SHAPE, "N and K must be at most 2^20 and N * K below 2^31");
  if (T >= (int64_t(1) << 31) - 256) return fail(FORGE_ERR_SHAPE, "T must be below 2^31 - 256");
  return FORGE_OK;
}

}  // namespace host
}  // namespace forge

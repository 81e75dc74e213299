// forge_norm_q8.hip -- the RMS norm's backward pass from 8-bit codes of h.
#include "forge_norm_backward.h"

namespace forge {

void launch_rmsnorm_backward_q8(int bf16, const NormBwdArgs& a, int64_t groups, void* stream) {
  if (a.h_q == FORGE_Q_FP8) backward_by_flags<FORGE_Q_FP8>(bf16, a, groups, (hipStream_t)stream);
  else backward_by_flags<FORGE_Q_I8>(bf16, a, groups, (hipStream_t)stream);
}

}  // namespace forge

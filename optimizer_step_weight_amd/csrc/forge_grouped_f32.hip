// forge_grouped_f32.hip -- the step grouped by expert (forge_grouped_wgrad.h): fp32 moments.
#include "forge_grouped_wgrad.h"

namespace forge {
namespace grp {
template GroupedStepFn select_grouped_step<FORGE_S_F32>(int);
}
}  // namespace forge

// forge_grouped_q8.hip -- the step grouped by expert (forge_grouped_wgrad.h): 8-bit moments, linear map.
#include "forge_grouped_wgrad.h"

namespace forge {
namespace grp {
template GroupedStepFn select_grouped_step<FORGE_S_Q8>(int);
}
}  // namespace forge

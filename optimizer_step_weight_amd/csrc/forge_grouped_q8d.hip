// forge_grouped_q8d.hip -- the step grouped by expert (forge_grouped_wgrad.h): 8-bit moments, dynamic map.
#include "forge_grouped_wgrad.h"

namespace forge {
namespace grp {
template GroupedStepFn select_grouped_step<FORGE_S_Q8D>(int);
}
}  // namespace forge

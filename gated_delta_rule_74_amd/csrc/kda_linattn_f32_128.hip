// kda_linattn_f32_128.hip -- linear attention's sweeps and local passes over
// fp32 data with 128-channel rows on the summed side.
#include "kda_linattn_impl.h"

namespace kda {
KDA_LIN_DEFINE(f32, float, 128)
}  // namespace kda

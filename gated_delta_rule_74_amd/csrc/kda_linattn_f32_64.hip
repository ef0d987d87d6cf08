// kda_linattn_f32_64.hip -- linear attention's sweeps and local passes over
// fp32 data with 64-channel rows on the summed side.
#include "kda_linattn_impl.h"

namespace kda {
KDA_LIN_DEFINE(f32, float, 64)
}  // namespace kda

// kda_linattn_bf16_32.hip -- linear attention's sweeps and local passes over
// bf16 data with 32-channel rows on the summed side.
#include "kda_linattn_impl.h"

namespace kda {
KDA_LIN_DEFINE(bf16, bf16, 32)
}  // namespace kda

// kda_linattn_bf16_128.hip -- linear attention's sweeps and local passes over
// bf16 data with 128-channel rows on the summed side.
#include "kda_linattn_impl.h"

namespace kda {
KDA_LIN_DEFINE(bf16, bf16, 128)
}  // namespace kda

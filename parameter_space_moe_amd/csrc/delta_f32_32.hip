// Delta rule, fp32 inputs, up to 32 keys.
#include "delta.hpp"

namespace swimba {
SWIMBA_DELTA_DEFINE(delta_f32_32, float, 1)
}  // namespace swimba

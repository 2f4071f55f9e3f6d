// Delta rule, fp32 inputs, up to 128 keys.
#include "delta.hpp"

namespace swimba {
SWIMBA_DELTA_DEFINE(delta_f32_128, float, 4)
}  // namespace swimba

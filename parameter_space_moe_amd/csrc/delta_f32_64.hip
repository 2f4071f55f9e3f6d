// Delta rule, fp32 inputs, up to 64 keys.
#include "delta.hpp"

namespace swimba {
SWIMBA_DELTA_DEFINE(delta_f32_64, float, 2)
}  // namespace swimba

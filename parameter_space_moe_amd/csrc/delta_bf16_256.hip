// Delta rule, bf16 inputs, up to 256 keys.
#include "delta.hpp"

namespace swimba {
SWIMBA_DELTA_DEFINE(delta_bf16_256, bf16_t, 8)
}  // namespace swimba

// Delta rule, bf16 inputs, up to 128 keys.
#include "delta.hpp"

namespace swimba {
SWIMBA_DELTA_DEFINE(delta_bf16_128, bf16_t, 4)
}  // namespace swimba

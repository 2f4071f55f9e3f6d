// Delta rule, bf16 inputs, up to 32 keys.
#include "delta.hpp"

namespace swimba {
SWIMBA_DELTA_DEFINE(delta_bf16_32, bf16_t, 1)
}  // namespace swimba

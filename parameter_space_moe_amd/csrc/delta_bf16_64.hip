// Delta rule, bf16 inputs, up to 64 keys.
#include "delta.hpp"

namespace swimba {
SWIMBA_DELTA_DEFINE(delta_bf16_64, bf16_t, 2)
}  // namespace swimba

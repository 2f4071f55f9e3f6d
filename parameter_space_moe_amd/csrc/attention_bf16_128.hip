// Linear attention walks, bf16 operands, rows of up to 128 (attention.hpp).
#include "attention.hpp"

namespace swimba {
int attn_bf16_128(const AttnParams& p, bool state, bool exact, hipStream_t s) {
  return attn_launch_waves<bf16_t, 4>(p, state, exact, s);
}
}  // namespace swimba

// Linear attention walks, f32 operands, rows of up to 64 (attention.hpp).
#include "attention.hpp"

namespace swimba {
int attn_f32_64(const AttnParams& p, bool state, bool exact, hipStream_t s) {
  return attn_launch_waves<float, 2>(p, state, exact, s);
}
}  // namespace swimba

// The 4-bit tile kernel for bf16 activations.
#include "w4_tile_inst.hpp"

namespace gek {
const void* w4_tile_bf16(int cfg, bool gated, int64_t group) { return w4_tile_pick<BF16>(cfg, gated, group); }
}  // namespace gek

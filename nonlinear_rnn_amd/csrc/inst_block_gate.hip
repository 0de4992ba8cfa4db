// Block boundary kernels: bf16 gate and normed stream, float32 stream.
#include "block_launch.hpp"

namespace pararnn {

PARARNN_DEFINE_BLOCK_LAUNCHER(gate, (kNormedBf16 | kGateBf16))

}  // namespace pararnn

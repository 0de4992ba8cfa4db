// Block boundary kernels: float32 gate, bf16 streams.
#include "block_launch.hpp"

namespace pararnn {

PARARNN_DEFINE_BLOCK_LAUNCHER(stream, (kNormedBf16 | kStreamBf16))

}  // namespace pararnn

// Block boundary kernels: float32 gate and stream, bf16 normed stream.
#include "block_launch.hpp"

namespace pararnn {

PARARNN_DEFINE_BLOCK_LAUNCHER(f32, (kNormedBf16))

}  // namespace pararnn

// Block boundary kernels: all of them bf16.
#include "block_launch.hpp"

namespace pararnn {

PARARNN_DEFINE_BLOCK_LAUNCHER(bf16, (kNormedBf16 | kGateBf16 | kStreamBf16))

}  // namespace pararnn

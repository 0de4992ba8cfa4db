// Block boundary kernels: a float32 normed stream, the other types read from the arguments.
#include "block_launch.hpp"

namespace pararnn {

PARARNN_DEFINE_BLOCK_LAUNCHER(args, (kTypesFromArgs))

}  // namespace pararnn

// Block boundary kernels: the norm alone, without states; types from the arguments.
#include "block_launch.hpp"

namespace pararnn {

PARARNN_DEFINE_BLOCK_LAUNCHER(norm, (kTypesFromArgs | kNoStates))

}  // namespace pararnn

// Delta rule: kernels for bfloat16 inputs, keys of up to 64 channels.
#include "delta_inst.hpp"

namespace pararnn {
namespace delta {
template pararnn_status_t run_scan<true, 64>(const Args &, bool, bool, void *);
template pararnn_status_t run_adjoint<true, 64>(const Args &, bool, bool, void *);
}  // namespace delta
}  // namespace pararnn

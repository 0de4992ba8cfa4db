// Launches of the delta rule's chunked kernels, one translation unit for each
// type of the inputs and room for the keys' channels (inst_delta_*.hip).
#pragma once

#include "pararnn.h"

namespace pararnn {
namespace delta {

struct Args;

// Columns of the values a workgroup of the chains takes, 16 a pair of waves.  A
// chain goes along its chunks one after the other, so narrow ones while that
// gives more workgroups than CUs have none of.
constexpr int kNarrow = 32, kWide = 64;

// time_first: the steps of queries and keys lie side by side.
template <bool HALF, int DK>
pararnn_status_t run_scan(const Args &A, bool time_first, bool wide, void *stream);
template <bool HALF, int DK>
pararnn_status_t run_adjoint(const Args &A, bool time_first, bool wide, void *stream);


}  // namespace delta
}  // namespace pararnn

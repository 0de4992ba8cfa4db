// Launches of the delta rule's chunked kernels, one translation unit for each
// type of the inputs and room for the keys' channels (inst_delta_*.hip).
#pragma once

#include "pararnn.h"

namespace pararnn {
namespace delta {

struct Args;

// Columns of the values a workgroup of the chains takes: their state's share
// and the operands made from it fill the LDS at 256 channels.
constexpr int value_block(int room) { return room > 128 ? 16 : 32; }

// time_first: the steps of queries and keys lie side by side.
template <bool HALF, int DK>
pararnn_status_t run_scan(const Args &A, bool time_first, void *stream);
template <bool HALF, int DK>
pararnn_status_t run_adjoint(const Args &A, bool time_first, void *stream);


}  // namespace delta
}  // namespace pararnn

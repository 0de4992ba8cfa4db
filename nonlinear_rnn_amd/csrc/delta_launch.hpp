// Launches of the delta rule's chunked kernels, one translation unit for each
// type of the inputs and room for the keys' channels (inst_delta_*.hip).
#pragma once

#include "pararnn.h"

namespace pararnn {
namespace delta {

struct Args;

// Columns of the values a workgroup of the chains takes, 16 a state's wave.  A
// chain goes along its chunks one after the other, so narrow workgroups, whose
// visits are shorter, until wide ones are as many as the CUs: 8 x 4096 x 8 heads of
// 128 x 128 bfloat16 226 us (wide 315), 4 x 16384 x 32 heads 1114 us (narrow 1409).
constexpr int kNarrow = 32, kWide = 64;

// time_first: the steps of queries and keys lie side by side.
template <bool HALF, int DK>
pararnn_status_t run_scan(const Args &A, bool time_first, bool wide, void *stream);
template <bool HALF, int DK>
pararnn_status_t run_adjoint(const Args &A, bool time_first, bool wide, void *stream);


}  // namespace delta
}  // namespace pararnn

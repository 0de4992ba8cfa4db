// What inst_delta_*.hip instantiate.
#pragma once

#include "delta.hpp"
#include "delta_launch.hpp"

namespace pararnn {
namespace delta {

inline pararnn_status_t launched() { return hipGetLastError() == hipSuccess ? PARARNN_OK : PARARNN_ERR_HIP; }

template <bool HALF, int DK, bool TF, bool OUTPUT>
pararnn_status_t run_chain(const Args &A, bool wide, hipStream_t s)
{
    if (A.chunks > 0) {
        hipLaunchKernelGGL((delta_inverse_kernel<HALF, TF>), dim3((unsigned)(A.B * A.Hv * A.chunks)),
                           dim3(kInverseThreads), 0, s, A);
        const pararnn_status_t st = launched();
        if (st != PARARNN_OK) return st;
    }
    constexpr int W = DK < 256 ? 4 : 2;
    const dim3 grid((unsigned)(A.B * A.Hv * A.blocks));
    if (wide)
        hipLaunchKernelGGL((delta_chain_kernel<HALF, DK, W, TF, OUTPUT>), grid, dim3(Roles<W>::waves(OUTPUT) * kWave), 0, s, A);
    else
        hipLaunchKernelGGL((delta_chain_kernel<HALF, DK, 2, TF, OUTPUT>), grid, dim3(Roles<2>::waves(OUTPUT) * kWave), 0, s, A);
    return launched();
}
template <bool HALF, int DK, bool TF>
pararnn_status_t run_back(const Args &A, bool wide, hipStream_t s)
{
    if (A.chunks > 0) {
        const pararnn_status_t st = run_chain<HALF, DK, TF, false>(A, wide, s);
        if (st != PARARNN_OK) return st;
    }
    const dim3 grid((unsigned)(A.B * A.Hv * A.blocks));
    constexpr int W = DK < 256 ? 4 : 2;
    if (wide)
        hipLaunchKernelGGL((delta_back_kernel<HALF, DK, W, TF>), grid, dim3(2 * W * kWave), 0, s, A);
    else
        hipLaunchKernelGGL((delta_back_kernel<HALF, DK, 2, TF>), grid, dim3(4 * kWave), 0, s, A);
    const pararnn_status_t st = launched();
    if (st != PARARNN_OK || A.chunks == 0) return st;
    hipLaunchKernelGGL((delta_grad_kernel<HALF, DK, TF>), dim3((unsigned)(A.B * A.Hk * A.chunks)), dim3(kThreads), 0,
                       s, A);
    return launched();
}
template <bool HALF, int DK>
pararnn_status_t run_scan(const Args &A, bool time_first, bool wide, void *stream)
{
    hipStream_t s = static_cast<hipStream_t>(stream);
    return time_first ? run_chain<HALF, DK, true, true>(A, wide, s) : run_chain<HALF, DK, false, true>(A, wide, s);
}
template <bool HALF, int DK>
pararnn_status_t run_adjoint(const Args &A, bool time_first, bool wide, void *stream)
{
    hipStream_t s = static_cast<hipStream_t>(stream);
    return time_first ? run_back<HALF, DK, true>(A, wide, s) : run_back<HALF, DK, false>(A, wide, s);
}

}  // namespace delta
}  // namespace pararnn

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
    constexpr int W = DK < 256 ? 4 : 2;
    const dim3 grid((unsigned)(A.B * A.Hv * A.segments * A.blocks));
    if (wide)
        hipLaunchKernelGGL((delta_chain_kernel<HALF, DK, W, TF, OUTPUT>), grid,
                           dim3(Roles<DK, W, OUTPUT>::kWaves * kWave), 0, s, A);
    else
        hipLaunchKernelGGL((delta_chain_kernel<HALF, DK, 2, TF, OUTPUT>), grid,
                           dim3(Roles<DK, 2, OUTPUT>::kWaves * kWave), 0, s, A);
    return launched();
}
template <bool HALF, int DK, bool TF>
pararnn_status_t run_back_chain(const Args &A, bool wide, hipStream_t s)
{
    constexpr int W = DK < 256 ? 4 : 2;
    const dim3 grid((unsigned)(A.B * A.Hv * A.segments * A.blocks));
    if (wide)
        hipLaunchKernelGGL((delta_back_kernel<HALF, DK, W, TF>), grid,
                           dim3(Roles<DK, W, true>::kWaves * kWave), 0, s, A);
    else
        hipLaunchKernelGGL((delta_back_kernel<HALF, DK, 2, TF>), grid,
                           dim3(Roles<DK, 2, true>::kWaves * kWave), 0, s, A);
    return launched();
}
// The inverses, and where the chain goes in segments the state before each.
template <bool HALF, int DK, bool TF>
pararnn_status_t run_before(const Args &A, hipStream_t s)
{
    if (A.chunks == 0) return PARARNN_OK;
    hipLaunchKernelGGL((delta_inverse_kernel<HALF, TF>), dim3((unsigned)(A.B * A.Hv * A.chunks)), dim3(kInverseThreads),
                       0, s, A);
    pararnn_status_t st = launched();
    if (st != PARARNN_OK || A.segments == 1) return st;
    Args ends = A;
    ends.ends = 1;
    ends.blocks = (A.value_pad + A.key_pad + kNarrow - 1) / kNarrow;
    st = run_chain<HALF, DK, TF, false>(ends, false, s);
    if (st != PARARNN_OK) return st;
    hipLaunchKernelGGL((delta_segments_kernel<DK, false>), dim3((unsigned)(A.B * A.Hv * (A.value_pad / 16))),
                       dim3(4 * kWave), 0, s, A);
    return launched();
}
template <bool HALF, int DK, bool TF>
pararnn_status_t run_forward(const Args &A, bool wide, hipStream_t s)
{
    const pararnn_status_t st = run_before<HALF, DK, TF>(A, s);
    return st == PARARNN_OK ? run_chain<HALF, DK, TF, true>(A, wide, s) : st;
}
template <bool HALF, int DK, bool TF>
pararnn_status_t run_back(const Args &A, bool wide, hipStream_t s)
{
    pararnn_status_t st = run_before<HALF, DK, TF>(A, s);
    if (st == PARARNN_OK && A.chunks > 0) st = run_chain<HALF, DK, TF, false>(A, wide, s);
    if (st == PARARNN_OK && A.segments > 1) {
        Args ends = A;
        ends.ends = 1;
        st = run_back_chain<HALF, DK, TF>(ends, wide, s);
        if (st != PARARNN_OK) return st;
        hipLaunchKernelGGL((delta_segments_kernel<DK, true>), dim3((unsigned)(A.B * A.Hv * (A.value_pad / 16))),
                           dim3(4 * kWave), 0, s, A);
        st = launched();
    }
    if (st == PARARNN_OK) st = run_back_chain<HALF, DK, TF>(A, wide, s);
    if (st != PARARNN_OK || A.chunks == 0) return st;
    const dim3 grid((unsigned)(A.B * A.Hk * A.chunks));
    if (A.Hv == A.Hk)
        hipLaunchKernelGGL((delta_grad_kernel<HALF, DK, TF, false>), grid, dim3(kThreads), 0, s, A);
    else
        hipLaunchKernelGGL((delta_grad_kernel<HALF, DK, TF, true>), grid, dim3(kThreads), 0, s, A);
    return launched();
}
template <bool HALF, int DK>
pararnn_status_t run_scan(const Args &A, bool time_first, bool wide, void *stream)
{
    hipStream_t s = static_cast<hipStream_t>(stream);
    return time_first ? run_forward<HALF, DK, true>(A, wide, s) : run_forward<HALF, DK, false>(A, wide, s);
}
template <bool HALF, int DK>
pararnn_status_t run_adjoint(const Args &A, bool time_first, bool wide, void *stream)
{
    hipStream_t s = static_cast<hipStream_t>(stream);
    return time_first ? run_back<HALF, DK, true>(A, wide, s) : run_back<HALF, DK, false>(A, wide, s);
}

}  // namespace delta
}  // namespace pararnn

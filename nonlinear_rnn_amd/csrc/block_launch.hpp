// Launchers of the block boundary's register kernels, one set per combination
// of types, each in its own translation unit (inst_block_*.hip) so that they
// compile in parallel.
#pragma once

#include "block.hpp"

namespace pararnn {

// (waves, groups of 4 steps, channel pairs a lane, steps loaded 4 at a time)
// Widths between the powers of two, for lanes that would idle.  Against the
// powers of two alone: forward B=8 T=4736 D=700 134 -> 117 us, B=2 T=6528
// D=2944 142 -> 123; backward B=53 T=4736 D=142 406 -> 356, B=4 T=4736 D=1500
// 323 -> 297.
#define PARARNN_BLOCK_TILINGS(X)                                                                 \
    X(1, 1, 1, true) X(4, 1, 1, true) X(8, 1, 1, true) X(16, 1, 1, true) X(16, 1, 2, true)       \
    X(2, 2, 1, true) X(8, 2, 1, true) X(16, 2, 1, true) X(16, 2, 2, true) X(16, 2, 4, true)      \
    X(4, 4, 1, true) X(8, 4, 1, true) X(16, 4, 1, true) X(16, 4, 2, true) X(16, 4, 4, true)      \
    X(6, 4, 1, true) X(12, 4, 1, true) X(12, 4, 2, true) X(12, 4, 4, true) X(12, 2, 4, true)     \
    X(16, 1, 4, true) X(16, 1, 4, false)                                                         \
    X(1, 1, 1, false) X(4, 1, 1, false) X(8, 1, 1, false) X(16, 1, 1, false) X(16, 1, 2, false)
#define PARARNN_BLOCK_ADJOINT_TILINGS(X)                                                         \
    X(1, 1, 1, true) X(2, 1, 2, true) X(4, 1, 2, true) X(8, 1, 2, true) X(8, 1, 4, true)         \
    X(2, 2, 2, true) X(4, 2, 2, true) X(4, 2, 4, true) X(8, 2, 4, true) X(8, 2, 8, true)         \
    X(4, 4, 2, true) X(4, 4, 4, true) X(4, 4, 8, true) X(8, 4, 8, true)                          \
    X(3, 4, 2, true) X(3, 4, 4, true) X(3, 4, 8, true) X(6, 4, 8, true) X(6, 2, 8, true)         \
    X(16, 1, 4, true) X(16, 1, 4, false)                                                         \
    X(1, 1, 1, false) X(2, 1, 2, false) X(4, 1, 2, false) X(8, 1, 2, false) X(8, 1, 4, false)
inline int tiling_code(int waves, int groups, int pairs, bool quads)
{
    return waves * 1000 + groups * 100 + pairs * 10 + quads;
}

#define PARARNN_BLOCK_LAUNCHER(NAME)                                                             \
    hipError_t launch_block_##NAME(bool adjoint, int tiling, dim3 grid, dim3 block,              \
                                   hipStream_t st, const BlockArgs &A)
PARARNN_BLOCK_LAUNCHER(f32);
PARARNN_BLOCK_LAUNCHER(gate);
PARARNN_BLOCK_LAUNCHER(stream);
PARARNN_BLOCK_LAUNCHER(bf16);
PARARNN_BLOCK_LAUNCHER(args);
PARARNN_BLOCK_LAUNCHER(norm);

#define PARARNN_TILING_CASE(W, G, P, Q)                                                          \
    case W * 1000 + G * 100 + P * 10 + Q:                                                        \
        hipLaunchKernelGGL((block_tile_kernel<W, G, P, Q, kTypes>), grid, block, 0, st, A);      \
        break;
#define PARARNN_ADJOINT_TILING_CASE(W, G, P, Q)                                                  \
    case W * 1000 + G * 100 + P * 10 + Q:                                                        \
        hipLaunchKernelGGL((block_tile_adjoint_kernel<W, G, P, Q, kTypes>), grid, block, 0, st,  \
                           A);                                                                   \
        break;
#define PARARNN_DEFINE_BLOCK_LAUNCHER(NAME, TYPES)                                               \
    PARARNN_BLOCK_LAUNCHER(NAME)                                                                 \
    {                                                                                            \
        constexpr int kTypes = TYPES;                                                            \
        if (adjoint) {                                                                           \
            switch (tiling) {                                                                    \
                PARARNN_BLOCK_ADJOINT_TILINGS(PARARNN_ADJOINT_TILING_CASE)                       \
            default: return hipErrorInvalidValue;                                                \
            }                                                                                    \
        } else {                                                                                 \
            switch (tiling) {                                                                    \
                PARARNN_BLOCK_TILINGS(PARARNN_TILING_CASE)                                       \
            default: return hipErrorInvalidValue;                                                \
            }                                                                                    \
        }                                                                                        \
        return hipGetLastError();                                                                \
    }

}  // namespace pararnn

// Host-side helpers shared by the entry points: argument checks and
// workspace alignment.
#pragma once

#include <cstddef>
#include <cstdint>
#include <utility>

#include "pararnn.h"

namespace pararnn {

constexpr size_t kAlign = 256;
constexpr int64_t kComputeUnits = 256;  // MI355X

inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Elements (b, d, t) of a plane must not overlap: with the dimensions of
// extent > 1 taken in increasing stride, each stride must exceed the largest
// offset the smaller ones reach.  Covers channel-major [B][D][T], time-major
// [B][T][D] and any padded or permuted variant of them.
inline bool planes_disjoint(int64_t B, int64_t T, int64_t D, int64_t sb, int64_t sd, int64_t st)
{
    if (sb < 0 || sd < 0 || st < 0) return false;
    if (B == 0 || D == 0 || T == 0) return true;  // no elements
    int64_t n[3] = {B, D, T}, str[3] = {sb, sd, st};
    for (int i = 0; i < 3; ++i)  // sort by stride
        for (int j = i + 1; j < 3; ++j)
            if (str[j] < str[i]) {
                std::swap(str[i], str[j]);
                std::swap(n[i], n[j]);
            }
    __int128 reach = 0;  // largest offset of the smaller dimensions
    for (int i = 0; i < 3; ++i) {
        if (n[i] <= 1) continue;
        if ((__int128)str[i] <= reach) return false;
        reach += (__int128)str[i] * (n[i] - 1);
        if (reach > (__int128)INT64_MAX) return false;
    }
    return true;
}

inline pararnn_status_t check_shape(const pararnn_shape_t *sh)
{
    if (!sh) return PARARNN_ERR_INVALID;
    if (sh->B < 0 || sh->T < 0 || sh->D < 0) return PARARNN_ERR_INVALID;
    if (sh->B > (int64_t(1) << 31) || sh->D > (int64_t(1) << 31) || sh->T > (int64_t(1) << 40))
        return PARARNN_ERR_UNSUPPORTED;
    if (!planes_disjoint(sh->B, sh->T, sh->D, sh->u_stride_b, sh->u_stride_d, sh->u_stride_t))
        return PARARNN_ERR_INVALID;
    if (!planes_disjoint(sh->B, sh->T, sh->D, sh->s_stride_b, sh->s_stride_d, sh->s_stride_t))
        return PARARNN_ERR_INVALID;
    return PARARNN_OK;
}

}  // namespace pararnn

// rope.cuh -- what the head kernels with a position rotation share (rope.cu,
// rope_bwd.cu): a token's row of the angle table and the row factor of a head.
#pragma once

#include "rope_args.h"
#include "device_common.cuh"

namespace rmsnorm {

__device__ inline void record_bad_index(int *status)
{
    atomicCAS(status, 0, static_cast<int>(RMSNORM_ERR_BAD_INDEX));
}

// The token's row of the table (null without a rotation); false when its
// position lies outside the table.
__device__ inline bool rope_row(const RopeTable &t, int64_t token, const float *&row)
{
    row = nullptr;
    if (t.rd == 0)
        return true;
    const int64_t p = t.pos[token];
    if (p < 0 || p >= t.max_pos)
        return false;
    row = t.cs + p * t.rd;
    return true;
}

// The factor of a row held as x = (x * pre) * r: pre is 1 but where the range
// guard scales x up by 2^100 (device_common.cuh).  For the bodies that read a
// head or row again from memory; `resum(k)` returns the sum of (k x)^2.
struct RowScale {
    float r, pre;
};
template <int DT, typename Resum>
__device__ inline RowScale row_scale(float S, float n, float eps, Resum resum)
{
    RowScale f = {row_factor(S, n, eps), 1.f};
    if constexpr (kRangeGuard<DT>) {
        if (sum_needs_rescale(S, eps)) {
            const float k = rescale_k(S);
            const Factor g = rescaled_factor(resum(k), k, n, eps);
            f.r = g.r;
            f.pre = g.up ? 0x1p100f : 1.f;
        }
    }
    return f;
}

} // namespace rmsnorm

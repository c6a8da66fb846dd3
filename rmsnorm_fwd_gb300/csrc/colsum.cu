// colsum.cu -- sums of the columns of fp32 partial results, the second step
// of the weights' gradients.
#include <algorithm>

#include "rope_args.h"
#include "device_common.cuh"

namespace rmsnorm {
namespace {

// 32 columns a block, 32 rows at once: the partial rows come from L2, where
// the first step has just left them, so the loads' latency bounds it.  Every
// thread adds its rows in order, then the 32 sums of a column are added in
// order: the same bits each time.
__global__ void __launch_bounds__(1024) colsum_kernel(const ColSum a, const ColSum b, int a_blocks)
{
    __shared__ float sums[32][33];
    pdl_begin();
    const bool second = static_cast<int>(blockIdx.x) >= a_blocks;
    const ColSum &c = second ? b : a;
    const int64_t col0 = static_cast<int64_t>(second ? blockIdx.x - a_blocks : blockIdx.x) * 32;
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    float s = 0.f;
    if (col0 + tx < c.cols)
#pragma unroll 8
        for (int64_t r = ty; r < c.rows; r += 32)
            s += c.part[r * c.ld + col0 + tx];
    sums[ty][tx] = s;
    __syncthreads();
    const float t = group_allreduce<32>(sums[tx][ty]); // warp ty: column col0 + ty
    if (tx == 0 && col0 + ty < c.cols)
        c.out[col0 + ty] = t;
}

} // namespace

cudaError_t launch_colsum(const ColSum &a, const ColSum &b, const LaunchArgs &base)
{
    const int64_t na = (a.cols + 31) / 32, nb = (b.cols + 31) / 32;
    return launch_kernel(colsum_kernel, static_cast<int>(na + nb), 1024, 0, base, a, b,
                         static_cast<int>(na));
}

} // namespace rmsnorm
